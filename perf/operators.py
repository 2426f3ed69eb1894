"""Cases of the operators that verify trees of drafted tokens over a paged KV cache.

Four operators, as one verify step of a hybrid (gated DeltaNet + attention)
stage uses them:

* ``norm_rope``  RMSNorm of every query and key head and the rotation of their
  leading dimensions by position, from the in-projection's rows to the 16-bit
  q, k, v that attention reads;
* ``attention``  attention of the drafted tokens over the sequence's cached rows
  (in pages) and over their own ancestors in the tree of drafts; one token is
  the tree of one node;
* ``deltanet``   the gated DeltaNet state step along a tree of drafts: a node
  starts from its parent's state;
* ``commit``     the accepted path's key and value rows written into the cache's
  pages, all layers in one call;
* ``branch``     the pages themselves: branches of a sequence freed, forked again
  from their root and extended (shared pages are counted, a shared last page is
  copied before it is written).

A tree is ``parent``: for each drafted token the index of its parent within its
sequence's tokens, smaller than its own; -1 continues the cached sequence; -2
marks a padded token, which sees nothing (its output is 0).
"""
import math

import torch

own = False

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = {"f16": F16, "bf16": BF16, "f32": F32}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # plain decoding of one sequence early in a chat
        dict(name="attention_decode_1000", op="attention", batch=1, nodes=1, ctx=1000, heads=24, kv_heads=4, dim=256,
             page=64, dtype="f16", ragged=False),
        # one 16-token draft tree of the 27B hybrid at the benchmark's context
        dict(name="attention_tree16_4096", op="attention", batch=1, nodes=16, ctx=4096, heads=24, kv_heads=4, dim=256,
             page=64, dtype="f16", ragged=False),
        # the same tree at the end of the longest cache a stage accepts
        dict(name="attention_tree16_262001", op="attention", batch=1, nodes=16, ctx=262001, heads=24, kv_heads=4, dim=256,
             page=256, dtype="bf16", ragged=False),
        # a served batch of ragged sequences with small pages
        dict(name="attention_batch24_ragged", op="attention", batch=24, nodes=12, ctx=16384, heads=32, kv_heads=8, dim=128,
             page=16, dtype="bf16", ragged=True),
        # wide trees over long contexts: bound by the products
        dict(name="attention_tree64_65536", op="attention", batch=4, nodes=64, ctx=65536, heads=24, kv_heads=4, dim=256,
             page=128, dtype="f16", ragged=False),
        # one token's heads
        dict(name="norm_rope_1", op="norm_rope", rows=1, heads=24, kv_heads=4, dim=256, rope=64, src="f32", dtype="f16",
             far=262144),
        # the tokens of a large served batch, or of a long prompt
        dict(name="norm_rope_8191", op="norm_rope", rows=8191, heads=24, kv_heads=4, dim=256, rope=64, src="f32", dtype="bf16",
             far=262144),
        # one 16-token draft tree
        dict(name="deltanet_tree16", op="deltanet", batch=1, nodes=16, k_heads=16, v_heads=48, ragged=False),
        # a served batch of ragged trees
        dict(name="deltanet_batch8_ragged", op="deltanet", batch=8, nodes=24, k_heads=16, v_heads=48, ragged=True),
        # accepted drafts of a served batch, the 16 attention layers of the 64-layer model
        dict(name="commit_batch8", op="commit", batch=8, nodes=16, ctx=3001, layers=16, kv_heads=4, dim=256, page=64, dtype="f16"),
        # two alternatives of one sequence
        dict(name="branch_2", op="branch", roots=1, branches=2, ctx=1001, add=16, layers=16, kv_heads=4, dim=256, page=64,
             dtype="f16"),
        # a search over many sequences
        dict(name="branch_96", op="branch", roots=12, branches=8, ctx=2037, add=40, layers=16, kv_heads=4, dim=256, page=64,
             dtype="bf16"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "norm_rope", "deltanet", "commit", "branch"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "attention":
        dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 6, 8])
        batch, nodes = _log(rng, 1, 32), _log(rng, 1, 64)
        # rows of keys x query vectors, and rows of keys, at most the largest listed case's
        most = min(4 * 65536 * 64 * 24 * 256 // (nodes * heads * dim * batch), 262144 * 4 * 256 // (batch * kv_heads * dim))
        return dict(op=op, batch=batch, nodes=nodes, ctx=_log(rng, 1, max(2, min(262001, most))), heads=heads, kv_heads=kv_heads,
                    dim=dim, page=rng.choice([16, 32, 64, 128, 256]), dtype=dtype, ragged=rng.random() < 0.6)
    if op == "norm_rope":
        dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = min(kv_heads * rng.choice([1, 2, 4, 6, 8]), 24 * 256 // dim)
        heads -= heads % kv_heads
        rope = rng.choice([dim, dim // 2, min(64, dim)])
        return dict(op=op, rows=_log(rng, 1, 8191), heads=heads, kv_heads=kv_heads, dim=dim, rope=rope,
                    src=rng.choice(["f32", "f16", "bf16"]), dtype=dtype, far=rng.choice([4096, 262144]))
    if op == "deltanet":
        k_heads = rng.choice([4, 8, 16])
        batch = _log(rng, 1, 8)
        return dict(op=op, batch=batch, nodes=_log(rng, 1, 24), k_heads=k_heads, v_heads=k_heads * rng.choice([1, 2, 3]),
                    ragged=rng.random() < 0.6)
    if op == "commit":
        batch = _log(rng, 1, 24)
        return dict(op=op, batch=batch, nodes=_log(rng, 1, 24), ctx=_log(rng, 1, 4000), layers=rng.choice([1, 4, 16]),
                    kv_heads=rng.choice([1, 4]), dim=rng.choice([64, 128, 256]), page=rng.choice([16, 64, 256]), dtype=dtype)
    page = rng.choice([16, 32, 64])
    # contexts that end inside a page, so that every branch copies one
    ctx = _log(rng, 2, 2000)
    ctx += ctx % page == 0
    return dict(op=op, roots=_log(rng, 1, 12), branches=_log(rng, 1, 8), ctx=ctx, add=_log(rng, 1, 64),
                layers=rng.choice([1, 4, 16]), kv_heads=rng.choice([1, 4]), dim=rng.choice([64, 128, 256]), page=page, dtype=dtype)


# -------------------------------------------------------------------- inputs

def _generator(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _lengths(case):
    """Cached rows and drafted tokens of each sequence, on the host.  They go by the case, so that every seed's outputs have the
    same shapes."""
    g = _generator(case["ctx"] * 64 + case["nodes"], "cpu")
    b = case["batch"]
    ctx, nodes = [case["ctx"]] * b, [case["nodes"]] * b
    if case["ragged"]:
        ctx = [int(x) for x in (torch.rand(b, generator=g) * (case["ctx"] + 1)).long()]
        nodes = [int(x) for x in torch.randint(1, case["nodes"] + 1, (b,), generator=g)]
        ctx[-1], nodes[-1] = case["ctx"], case["nodes"]
    return ctx, nodes


def _roots(case, count):
    """Cached rows of `count` sequences, on the host: the first has the case's, the others between half of it and all."""
    g = _generator(case["ctx"], "cpu")
    return [case["ctx"]] + [int(x) for x in torch.randint(max(1, case["ctx"] // 2), case["ctx"] + 1, (count - 1,), generator=g)]


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _parents(nodes, seed, padded):
    """A random tree for each sequence: mostly chains with side branches; now and then a padded last token."""
    g = _generator(seed + 7, "cpu")
    out = []
    for n in nodes:
        p = []
        for i in range(n):
            r = float(torch.rand((), generator=g))
            p.append(i - 1 if r < 0.6 else int(torch.randint(-1, max(i, 1), (), generator=g)) if i else -1)
        if padded and n > 3:
            p[-1] = -2
        out += p
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _pages_of(counts, n_pages, max_pages, seed):
    """A page table whose sequences hold pages of a pool in no order."""
    g = _generator(seed + 13, "cpu")
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(counts), max_pages), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(counts):
        table[s, :n] = order[at:at + n]
        at += n
    return table.cuda()


def _handle(s):
    """What a serving program makes of its cache once, before any call."""
    if own:
        import quantized_hybrid_layer_b200 as q
        s["kv"] = q.KvPages(s["k"], s["v"], s["table"], s["lens"], s["held"], s["refs"])
    return s


def _prepare_attention(case, seed):
    g = _generator(seed)
    dt = TYPES[case["dtype"]]
    ctx, nodes = _lengths(case)
    P, D, H = case["page"], case["dim"], case["kv_heads"]
    counts = [-(-c // P) for c in ctx]
    max_pages, n_pages = max(1, max(counts)), sum(counts) + 3
    rows = sum(nodes)
    k = torch.randn(1, n_pages, H, P, D, generator=g, device="cuda", dtype=dt)
    v = torch.randn(1, n_pages, H, P, D, generator=g, device="cuda", dtype=dt)
    table = _pages_of(counts, n_pages, max_pages, seed)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    used = table.flatten()
    refs.scatter_add_(0, used.clamp(min=0).long(), (used >= 0).int())
    b = len(ctx)
    # sequences in another order than their rows in the page table
    seqs = torch.randperm(b, generator=_generator(seed + 5, "cpu")).to(torch.int32).cuda()
    lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    by_batch = [nodes[int(i)] for i in seqs.tolist()]
    return _handle(dict(
        op="attention", k=k, v=v, table=table, lens=lens, held=torch.tensor(counts, dtype=torch.int32, device="cuda"), refs=refs,
        seqs=seqs, q_start=torch.tensor(_starts(by_batch), dtype=torch.int32, device="cuda"),
        parent=_parents(by_batch, seed, True), max_nodes=case["nodes"], scale=1.0 / math.sqrt(D),
        q=torch.randn(rows, case["heads"], D, generator=g, device="cuda", dtype=dt),
        k_new=torch.randn(rows, H, D, generator=g, device="cuda", dtype=dt),
        v_new=torch.randn(rows, H, D, generator=g, device="cuda", dtype=dt),
        out=torch.zeros(rows, case["heads"], D, device="cuda", dtype=dt),
        lse=torch.zeros(rows, case["heads"], device="cuda")))


def _prepare_norm_rope(case, seed):
    g = _generator(seed)
    H, K, D, n = case["heads"], case["kv_heads"], case["dim"], case["rows"]
    dt = TYPES[case["dtype"]]
    width = 2 * H * D + 2 * K * D          # q | gate | k | v, as the in-projection leaves them
    return dict(
        op="norm_rope", heads=H, kv_heads=K, dim=D, rope=case["rope"], theta=1.0e7, eps=1.0e-6,
        y=torch.randn(n, width, generator=g, device="cuda").to(TYPES[case["src"]]),
        pos=torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32),
        gamma_q=1 + 0.02 * torch.randn(D, generator=g, device="cuda"), gamma_k=1 + 0.02 * torch.randn(D, generator=g, device="cuda"),
        q=torch.zeros(n, H, D, device="cuda", dtype=dt), k=torch.zeros(n, K, D, device="cuda", dtype=dt),
        v=torch.zeros(n, K, D, device="cuda", dtype=dt))


def _prepare_deltanet(case, seed):
    g = _generator(seed)
    _, nodes = _lengths(dict(case, ctx=1))
    hk, hv, rows, b = case["k_heads"], case["v_heads"], sum(nodes), case["batch"]
    y = torch.randn(rows, 2 * hk * 128 + hv * 128 + 2 * hv, generator=g, device="cuda")
    n_states = b + 2
    return dict(
        op="deltanet", k_heads=hk, v_heads=hv, y=y, max_nodes=case["nodes"],
        q_start=torch.tensor(_starts(nodes), dtype=torch.int32, device="cuda"), parent=_parents(nodes, seed, False),
        states=0.1 * torch.randn(n_states, hv, 128, 128, generator=g, device="cuda"),
        index=torch.randperm(n_states, generator=_generator(seed + 5, "cpu"))[:b].to(torch.int32).cuda(),
        snaps=torch.zeros(rows, hv, 128, 128, device="cuda"), o=torch.zeros(rows, hv * 128, device="cuda"))


def _cache(case, g, counts, n_pages, max_pages, lens, seed):
    shape = (case["layers"], n_pages, case["kv_heads"], case["page"], case["dim"])
    dt = TYPES[case["dtype"]]
    table = _pages_of(counts, n_pages, max_pages, seed)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    used = table.flatten()
    refs.scatter_add_(0, used.clamp(min=0).long(), (used >= 0).int())
    return dict(k=torch.randn(shape, generator=g, device="cuda", dtype=dt), v=torch.randn(shape, generator=g, device="cuda", dtype=dt),
                table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                held=torch.tensor(counts, dtype=torch.int32, device="cuda"), refs=refs)


def _prepare_commit(case, seed):
    g, c = _generator(seed), _generator(seed + 3, "cpu")
    b, n, P = case["batch"], case["nodes"], case["page"]
    ctx = _roots(case, b)
    counts = [-(-(x + n) // P) for x in ctx]
    s = _cache(case, g, counts, sum(counts) + 5, max(counts) + 1, ctx, seed)
    path = torch.full((b, n), -1, dtype=torch.int32)
    accepted = torch.randint(1, n + 1, (b,), generator=c)
    for i in range(b):
        a = int(accepted[i])
        path[i, :a] = torch.randperm(n, generator=c)[:a].sort().values.to(torch.int32)
    new = (case["layers"], b * n, case["kv_heads"], case["dim"])
    s.update(op="commit", seqs=torch.randperm(b, generator=c).to(torch.int32).cuda(),
             q_start=torch.arange(0, b * n + 1, n, dtype=torch.int32, device="cuda"), path=path.cuda(),
             accepted=accepted.to(torch.int32).cuda(),
             k_new=torch.randn(new, generator=g, device="cuda", dtype=s["k"].dtype),
             v_new=torch.randn(new, generator=g, device="cuda", dtype=s["k"].dtype),
             status=torch.zeros(b, dtype=torch.int32, device="cuda"))
    s["pos"] = s["lens"][s["seqs"].long()].clone()
    return _handle(s)


def _prepare_branch(case, seed):
    g, c = _generator(seed), _generator(seed + 3, "cpu")
    r, n, P = case["roots"], case["branches"], case["page"]
    ctx = [x + (x % P == 0) for x in _roots(case, r)]
    counts = [-(-x // P) for x in ctx] + [0] * (r * n)
    new = -(-(case["add"] + P) // P) + 1
    s = _cache(case, g, counts, sum(counts) + r * n * new + 3, max(counts) + new, ctx + [0] * (r * n), seed)
    s.update(op="branch", src=torch.arange(r, dtype=torch.int32).repeat_interleave(n).cuda(),
             dst=torch.arange(r, r + r * n, dtype=torch.int32).cuda(),
             add=torch.randint(1, case["add"] + 1, (r * n,), generator=c).to(torch.int32).cuda(),
             status=torch.zeros(r * n, dtype=torch.int32, device="cuda"))
    return _handle(s)


def prepare(case, seed):
    return {"attention": _prepare_attention, "norm_rope": _prepare_norm_rope, "deltanet": _prepare_deltanet,
            "commit": _prepare_commit, "branch": _prepare_branch}[case["op"]](case, seed)


# --------------------------------------------------------------------- calls

def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


def _own_attention(s):
    import quantized_hybrid_layer_b200 as q
    q.qhl_tree_attention(s["kv"], 0, s["seqs"], s["q_start"], s["parent"], s["max_nodes"], s["q"], s["k_new"], s["v_new"], s["out"],
                         lse=s["lse"], scale=s["scale"])
    return s["out"], s["lse"]


def _own_norm_rope(s):
    import quantized_hybrid_layer_b200 as q
    q.qhl_qk_norm_rope(s["heads"], s["kv_heads"], s["dim"], s["rope"], s["theta"], s["eps"], s["y"], s["pos"], s["gamma_q"],
                       s["gamma_k"], s["q"], s["k"], s["v"])
    return s["q"], s["k"], s["v"]


def _own_deltanet(s):
    import quantized_hybrid_layer_b200 as q
    q.qhl_deltanet_tree(s["k_heads"], s["v_heads"], s["y"], s["q_start"], s["parent"], s["max_nodes"], s["states"], s["index"],
                        s["snaps"], s["o"])
    return s["o"], s["snaps"]


def _own_commit(s):
    import quantized_hybrid_layer_b200 as q
    q.qhl_pages_commit(s["kv"], s["seqs"], s["q_start"], s["path"], s["accepted"], s["pos"], s["k_new"], s["v_new"], s["status"])
    return s["k"], s["v"], s["lens"], s["status"]


def _own_branch(s):
    import quantized_hybrid_layer_b200 as q
    q.qhl_pages_free(s["kv"], s["dst"], s["status"])
    q.qhl_pages_fork(s["kv"], s["src"], s["dst"], s["status"])
    q.qhl_pages_extend(s["kv"], s["dst"], s["add"], s["status"])
    return s["k"], s["v"], s["table"], s["lens"], s["held"], s["refs"], s["status"]


_OWN = {"attention": _own_attention, "norm_rope": _own_norm_rope, "deltanet": _own_deltanet, "commit": _own_commit,
        "branch": _own_branch}


# --------------------------------------------------------------- plain forms

def _ancestors(q_start, parent, max_nodes):
    """[batch, nodes, nodes]: whether node j is node i or one of its ancestors; padded tokens have none."""
    b = q_start.numel() - 1
    first, count = q_start[:-1].long(), (q_start[1:] - q_start[:-1]).long()
    at = torch.arange(max_nodes, device="cuda")
    there = at[None, :] < count[:, None]
    row = (first[:, None] + at[None, :]).clamp(max=parent.numel() - 1)
    p = torch.where(there, parent[row].long(), -2)
    dead = p == -2
    # reach by doubling: after k rounds all ancestors up to 2^k steps away
    reach = torch.eye(max_nodes, device="cuda")[None].expand(b, -1, -1) + ((at[None, None, :] == p[:, :, None]) & (p >= 0)[:, :, None]).float()
    step = 1
    while step < max_nodes:
        reach = (reach @ reach).clamp(max=1)
        step *= 2
    gone = (reach @ dead.float()[:, :, None])[:, :, 0] > 0
    return (reach > 0) & ~gone[:, :, None], row, there, ~gone & there


def _plain_attention(s):
    k, v, P = s["k"][0], s["v"][0], s["k"].shape[3]
    H, D, n = k.shape[1], k.shape[3], s["max_nodes"]
    G = s["q"].shape[1] // H
    seqs = s["seqs"].long()
    b = seqs.numel()
    lens = s["lens"][seqs].long()
    table = s["table"][seqs].long().clamp(min=0)
    width = table.shape[1] * P
    ck = k[table].transpose(2, 3).reshape(b, width, H, D).permute(0, 2, 1, 3)
    cv = v[table].transpose(2, 3).reshape(b, width, H, D).permute(0, 2, 1, 3)
    visible, row, there, alive = _ancestors(s["q_start"], s["parent"], n)
    nk, nv = s["k_new"][row].permute(0, 2, 1, 3), s["v_new"][row].permute(0, 2, 1, 3)
    # masked places may hold anything
    in_ctx = torch.arange(width, device="cuda")[None, :] < lens[:, None]
    keys = torch.cat([ck, nk], 2).float()
    values = torch.where(torch.cat([in_ctx, there], 1)[:, None, :, None], torch.cat([cv, nv], 2).float(), 0.0)
    q = s["q"][row].float().reshape(b, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(b, H, n * G, D)
    scores = (q @ keys.transpose(2, 3)) * s["scale"]
    seen = torch.cat([in_ctx[:, None, :] & alive[:, :, None], visible & there[:, None, :]], 2)
    seen = seen[:, None, :, None, :].expand(b, H, n, G, width + n).reshape(b, H, n * G, width + n)
    scores = torch.where(seen, scores, float("-inf"))
    top = scores.amax(3, keepdim=True)
    p = torch.exp(scores - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(3, keepdim=True)
    out = (p @ values) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + torch.where(top == float("-inf"), 0.0, top))[..., 0]
    out = out.reshape(b, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(b, n, H * G, D)
    lse = lse.reshape(b, H, n, G).permute(0, 2, 1, 3).reshape(b, n, H * G)
    # the rows of all sequences, in order: those that are there
    order = torch.argsort(torch.where(there, row, row.new_tensor(1 << 60)).flatten())[: s["q"].shape[0]]
    return out.reshape(b * n, H * G, D)[order].to(s["q"].dtype), lse.reshape(b * n, H * G)[order]


def _plain_norm_rope(s):
    H, K, D, R = s["heads"], s["kv_heads"], s["dim"], s["rope"]
    y = s["y"].float()
    n = y.shape[0]
    q = y[:, :H * D].reshape(n, H, D)
    k = y[:, 2 * H * D:2 * H * D + K * D].reshape(n, K, D)
    v = y[:, 2 * H * D + K * D:].reshape(n, K, D)
    i = torch.arange(R // 2, device="cuda", dtype=torch.float64)
    angle = s["pos"].double()[:, None] * torch.exp(-2 * i / R * math.log(s["theta"]))[None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    x = torch.cat([q * torch.rsqrt((q * q).mean(2, keepdim=True) + s["eps"]) * s["gamma_q"],
                   k * torch.rsqrt((k * k).mean(2, keepdim=True) + s["eps"]) * s["gamma_k"]], 1)
    a, b = x[..., :R // 2], x[..., R // 2:R]
    x = torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., R:]], 2).to(s["q"].dtype)
    return x[:, :H].contiguous(), x[:, H:].contiguous(), v.to(s["q"].dtype)


def _plain_deltanet(s):
    hk, hv = s["k_heads"], s["v_heads"]
    y, first = s["y"], s["q_start"][:-1].long()
    count = (s["q_start"][1:] - s["q_start"][:-1]).long()
    n, rows = s["max_nodes"], y.shape[0]
    rep = hv // hk
    q = y[:, :hk * 128].reshape(rows, hk, 128)
    k = y[:, hk * 128:2 * hk * 128].reshape(rows, hk, 128)
    v = y[:, 2 * hk * 128:(2 * hk + hv) * 128].reshape(rows, hv, 128)
    beta = torch.sigmoid(y[:, (2 * hk + hv) * 128:(2 * hk + hv) * 128 + hv])
    alpha = torch.sigmoid(-y[:, (2 * hk + hv) * 128 + hv:])
    q = (q * torch.rsqrt((q * q).sum(2, keepdim=True) + 1e-6)).repeat_interleave(rep, 1)
    k = (k * torch.rsqrt((k * k).sum(2, keepdim=True) + 1e-6)).repeat_interleave(rep, 1)
    snaps, o = torch.zeros_like(s["snaps"]), torch.zeros_like(s["o"])
    start = s["states"][s["index"].long()]
    # one step for the i-th node of every sequence; a sequence that has fewer repeats its last
    for i in range(n):
        row = first + torch.clamp(count - 1, max=i)
        p = s["parent"][row].long()
        S = torch.where((p < 0)[:, None, None, None], start, snaps[first + p.clamp(min=0)])
        kk, al = k[row], alpha[row][:, :, None]
        u = beta[row][:, :, None] * (v[row] - al * (S * kk[:, :, None, :]).sum(3))
        S = al[..., None] * S + u[..., None] * kk[:, :, None, :]
        snaps[row] = S
        o[row] = (S * q[row][:, :, None, :]).sum(3).reshape(-1, hv * 128)
    return o, snaps


def _plain_commit(s):
    P, seqs = s["k"].shape[3], s["seqs"].long()
    j = torch.arange(s["path"].shape[1], device="cuda")[None, :]
    there = (j < s["accepted"][:, None]).flatten()
    # what is not accepted repeats the first accepted row: the same values to the same place
    at = torch.where(there, torch.arange(there.numel(), device="cuda"), there.int().argmax())
    row = (s["q_start"][:-1, None] + s["path"].clamp(min=0)).flatten()[at].long()
    to = (s["pos"][:, None] + j).long()
    page = torch.gather(s["table"][seqs].long(), 1, (to // P).clamp(max=s["table"].shape[1] - 1)).flatten()[at]
    r = (to % P).flatten()[at]
    s["k"][:, page, :, r] = s["k_new"][:, row].transpose(0, 1)
    s["v"][:, page, :, r] = s["v_new"][:, row].transpose(0, 1)
    s["lens"][seqs] = s["pos"] + s["accepted"]
    return s["k"], s["v"], s["lens"], s["status"].zero_()


def _plain_branch(s):
    k, v, table, lens, held, refs = s["k"], s["v"], s["table"], s["lens"], s["held"], s["refs"]
    P, src, dst = k.shape[3], s["src"].long(), s["dst"].long()
    at = torch.arange(table.shape[1], device="cuda")[None, :]
    # free
    gone = table[dst]
    refs.scatter_add_(0, gone.clamp(min=0).flatten().long(), -(at < held[dst][:, None]).int().flatten())
    # fork: the pages that hold rows are shared
    n = lens[src]
    n_pages = (n + P - 1) // P
    mine = at < n_pages[:, None]
    row = torch.where(mine, table[src], -1)
    refs.scatter_add_(0, row.clamp(min=0).flatten().long(), mine.int().flatten())
    # extend: a shared last page is copied, new pages follow; free pages in order of their number
    last = torch.gather(row, 1, (n_pages - 1).clamp(min=0).long()[:, None])[:, 0]
    same = (last[:, None] == last[None, :]).int().tril(-1).sum(1)
    copied = ((n % P != 0) & (refs[last.long()] - same > 1)).int()
    fresh = (n + s["add"] + P - 1) // P - n_pages
    need = copied + fresh
    before = torch.cumsum(need, 0) - need
    free = torch.argsort((refs != 0).int(), stable=True).int()
    to = torch.where(copied > 0, free[before.long()], last)
    # the place of each page of a row in the list of free ones
    j = at - n_pages[:, None] + copied[:, None]
    new = (at >= n_pages[:, None] - copied[:, None]) & (j < need[:, None])
    ids = free[(before[:, None] + j).clamp(0, free.numel() - 1).long()]
    refs.scatter_add_(0, last.long(), -copied)
    refs.scatter_add_(0, ids.flatten().long(), new.int().flatten())
    table[dst] = torch.where(new, ids, row)
    lens[dst], held[dst] = n, (n_pages + fresh).to(torch.int32)
    kept = (torch.arange(P, device="cuda")[None, :] < (n % P)[:, None])[None, :, None, :, None]
    k[:, to.long()] = torch.where(kept, k[:, last.long()], k[:, to.long()])
    v[:, to.long()] = torch.where(kept, v[:, last.long()], v[:, to.long()])
    return k, v, table, lens, held, refs, s["status"].zero_()


_PLAIN = {"attention": _plain_attention, "norm_rope": _plain_norm_rope, "deltanet": _plain_deltanet, "commit": _plain_commit,
          "branch": _plain_branch}


# ---------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "attention":
        ctx, nodes = _lengths(case)
        kv = 2 * (sum(ctx) + sum(nodes)) * case["kv_heads"] * case["dim"] * 2
        qo = sum(nodes) * case["heads"] * (2 * case["dim"] * 2 + 4)
        return {"bytes": kv + qo, "flops": 4 * case["heads"] * case["dim"] * sum(n * (c + 1) for c, n in zip(ctx, nodes))}
    if op == "norm_rope":
        vectors = case["rows"] * (case["heads"] + 2 * case["kv_heads"])
        size = 4 if case["src"] == "f32" else 2
        return {"bytes": vectors * case["dim"] * (size + 2) + case["rows"] * 4, "flops": vectors * case["dim"] * 6}
    if op == "deltanet":
        nodes = sum(_lengths(dict(case, ctx=1))[1])
        state = case["v_heads"] * 128 * 128
        row = (2 * case["k_heads"] + 2 * case["v_heads"]) * 128 + 2 * case["v_heads"]
        return {"bytes": (case["batch"] + nodes) * state * 4 + nodes * row * 4, "flops": nodes * state * 7}
    row = case["layers"] * case["kv_heads"] * case["dim"] * 2 * 2
    if op == "commit":
        # about half of the drafts are accepted
        rows = case["batch"] * (case["nodes"] + 1) // 2
        return {"bytes": 2 * rows * row + case["batch"] * (case["nodes"] + 8) * 4, "flops": 0}
    ctx = [x + (x % case["page"] == 0) for x in _roots(case, case["roots"])]
    rows = case["branches"] * sum(x % case["page"] for x in ctx)
    return {"bytes": 2 * rows * row + case["branches"] * sum(x // case["page"] + 8 for x in ctx) * 4, "flops": 0}


# --------------------------------------------------------------------- exact

def _exact_attention(case, seed):
    s = _prepare_attention(case, seed)
    q, D, H = s["q"], case["dim"], case["kv_heads"]
    G, P = case["heads"] // H, case["page"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    start, parent, lens = s["q_start"].tolist(), s["parent"].tolist(), s["lens"].tolist()
    for i, seq in enumerate(s["seqs"].tolist()):
        a, e, c = start[i], start[i + 1], lens[seq]
        pages = s["table"][seq, :-(-c // P)].long()
        mask = torch.zeros(e - a, c + e - a, dtype=torch.bool)
        for x in range(e - a):
            line, at = [], x
            while at >= 0:
                line.append(at)
                at = parent[a + at]
            if at == -1:
                mask[x, :c] = True
                mask[x, [c + z for z in line]] = True
        mask = mask.cuda()
        for h in range(H):
            K = torch.cat([s["k"][0, pages, h].reshape(-1, D)[:c], s["k_new"][a:e, h]]).double()
            V = torch.cat([s["v"][0, pages, h].reshape(-1, D)[:c], s["v_new"][a:e, h]]).double()
            for x in range(h * G, h * G + G):
                z = (q[a:e, x].double() @ K.T) / math.sqrt(D)
                z = z.masked_fill(~mask, float("-inf"))
                lse[a:e, x] = torch.logsumexp(z, 1)
                w = torch.exp(z - lse[a:e, x].nan_to_num(neginf=0.0)[:, None])
                out[a:e, x] = w @ V
    return out, lse


def _exact_norm_rope(case, seed):
    s = _prepare_norm_rope(case, seed)
    y = s["y"].double()
    H, K, D, R = case["heads"], case["kv_heads"], case["dim"], case["rope"]
    n = y.shape[0]

    def turned(x, gamma):
        x = x.reshape(n, -1, D)
        x = x / (x.square().sum(2, keepdim=True) / D + 1.0e-6).sqrt() * gamma.double()
        z = torch.complex(x[..., :R // 2], x[..., R // 2:R])
        turn = s["pos"].double()[:, None] * 1.0e7 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        z = z * torch.polar(torch.ones_like(turn), turn)[:, None, :]
        return torch.cat([z.real, z.imag, x[..., R:]], 2)

    return (turned(y[:, :H * D], s["gamma_q"]), turned(y[:, 2 * H * D:(2 * H + K) * D], s["gamma_k"]),
            y[:, (2 * H + K) * D:].reshape(n, K, D))


def _exact_deltanet(case, seed):
    s = _prepare_deltanet(case, seed)
    hk, hv = case["k_heads"], case["v_heads"]
    y, start, parent = s["y"].double(), s["q_start"].tolist(), s["parent"].tolist()
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    snaps = torch.zeros(s["snaps"].shape, dtype=torch.float64, device="cuda")
    head = torch.arange(hv, device="cuda") // (hv // hk)
    for i, at in enumerate(s["index"].tolist()):
        for x in range(start[i], start[i + 1]):
            S = s["states"][at].double() if parent[x] < 0 else snaps[start[i] + parent[x]]
            parts = torch.split(y[x], [hk * 128, hk * 128, hv * 128, hv, hv])
            q, k, v = parts[0].view(hk, 128)[head], parts[1].view(hk, 128)[head], parts[2].view(hv, 128)
            q = q / (q.square().sum(1, keepdim=True) + 1e-6).sqrt()
            k = k / (k.square().sum(1, keepdim=True) + 1e-6).sqrt()
            beta, alpha = torch.sigmoid(parts[3])[:, None, None], torch.exp(-torch.nn.functional.softplus(parts[4]))[:, None, None]
            kept = S - beta * torch.einsum("hij,hj->hi", S, k)[:, :, None] * k[:, None, :]
            S = alpha * kept + beta * v[:, :, None] * k[:, None, :]
            snaps[x] = S
            o[x] = torch.einsum("hij,hj->hi", S, q).reshape(-1)
    return o, snaps


def exact(case, seed):
    op = case["op"]
    if op == "attention":
        return _exact_attention(case, seed)
    if op == "norm_rope":
        return _exact_norm_rope(case, seed)
    if op == "deltanet":
        return _exact_deltanet(case, seed)
    return None          # rows are moved, not computed
