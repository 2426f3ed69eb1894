"""The tree-verification operators on the GPU: the forms, sizes and calls that only a served batch or a long cache reaches."""
import math

import numpy as np
import pytest
import torch

import verify_helpers as vh
from test_gpu_verify import check_attention, check_norm_rope, dn_inputs, dn_run, q, run_attention  # noqa: F401  (q is a fixture)
from verify_helpers import DTYPES, Trees, gen, half_step, random_tree, tiny_step

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- attention

@pytest.mark.parametrize("dim,page", [(64, 256), (128, 64), (256, 16)])
@pytest.mark.parametrize("more", [1, 64, 130])
def test_attention_many_laps_of_the_ring(q, dim, page, more):
    """Every CTA's run goes around the ring of tiles several times before the tiles that need care."""
    rows = 148 * 20 * (64 if dim == 256 else 128)
    check_attention(q, Trees([rows + more], [[-1, 0, 0]], 2, 1, dim, page, DTYPES["bf16"], seed=more))


@pytest.mark.parametrize("dim,page,dtype", [(256, 16, "f16"), (256, 64, "bf16"), (128, 16, "bf16"), (128, 256, "f16"), (64, 32, "f16"), (64, 128, "bf16")])
@pytest.mark.parametrize("which", ["first", "last", "middle", "several", "all"])
def test_attention_rows_of_a_page_that_does_not_exist_are_absent(q, dim, page, dtype, which):  # noqa: F811
    """A sequence with bad page numbers attends over its other rows; the call reports it."""
    ctx = 3 * page + 450
    t = Trees([ctx, 70], [[-1, 0, 0, -2], [-1]], 4, 2, dim, page, DTYPES[dtype], seed=dim + page)
    s, n = int(t.seqs[0]), -(-ctx // page)
    gone = {"first": [0], "last": [n - 1], "middle": [n // 2], "several": [0, 1, n // 2, n - 2], "all": list(range(n))}[which]
    for i, p in enumerate(gone):
        t.table[s, p] = (-1, int(t.refs.numel()), 2 ** 31 - 1, -2 ** 31)[i % 4]
    keep = torch.tensor([r for r in range(ctx) if r // page not in gone], dtype=torch.long)
    t.K[0], t.V[0] = t.K[0][keep], t.V[0][keep]
    with pytest.raises(q.StageError) as e:
        check_attention(q, t)                            # its last line is the report
    assert e.value.code == -7


def test_attention_pages_that_do_not_exist_in_a_long_run_of_small_ones(q):  # noqa: F811
    """Bad pages here and there among thousands, many to a CTA's run."""
    page, ctx = 16, 148 * 300
    t = Trees([ctx], [random_tree(5, gen(2))], 2, 1, 256, page, torch.float16, seed=12)
    gone = torch.randperm(ctx // page, generator=gen(3))[:400]
    t.table[0, gone] = -1
    keep = ~torch.isin(torch.arange(ctx) // page, gone)
    t.K[0], t.V[0] = t.K[0][keep], t.V[0][keep]
    with pytest.raises(q.StageError) as e:
        check_attention(q, t)
    assert e.value.code == -7


def ragged(n, seed):
    """n trees: empty ones, single tokens, small trees and a few of several M tiles, over caches from none to 3000 rows."""
    g = gen(seed)
    size = torch.tensor([0, 1, 1, 1, 3, 7, 40])[torch.randint(0, 7, (n,), generator=g)].tolist()
    ctx = torch.randint(0, 60, (n,), generator=g).tolist()
    size[n // 3], ctx[n // 3], ctx[n - 1] = 70, 3000, 900
    size[n - 1] = 0                                      # a long cache that nobody asks for
    return Trees(ctx, [random_tree(m, g) for m in size], 4, 1, 64, 32, torch.bfloat16, seed=seed, extra_rows=2)


@pytest.mark.parametrize("n", [32, 33, 100, 255, 256, 257])
def test_attention_batches_that_a_cta_plans_for_itself(q, n):  # noqa: F811
    """Up to 32 trees are planned by a warp, up to 256 by every CTA, more by a kernel of their own."""
    check_attention(q, ragged(n, n))


@pytest.mark.parametrize("n", [40, 200])
def test_attention_large_batches_of_equal_trees_of_several_tiles(q, n):  # noqa: F811
    """Trees of two M tiles each, for which a group of CTAs has one for each."""
    g = gen(n)
    check_attention(q, Trees(torch.randint(0, 150, (n,), generator=g).tolist(), [random_tree(17, g) for _ in range(n)], 8, 1, 64, 16,
                             torch.float16, seed=n))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 256])
def test_attention_a_long_cache_of_values_of_one_sign(q, dtype, dim):  # noqa: F811
    """Values with a mean, so that a part that is lost or counted twice shows; the weights' subnormal numbers count 2^-31."""
    t = Trees([9001], [random_tree(4, gen(1))], 4, 2, dim, 64, DTYPES[dtype], seed=8)
    t.V[0], t.v_new = (1 + 0.2 * t.V[0].float()).to(t.dtype), (1 + 0.2 * t.v_new.float()).to(t.dtype)
    s = int(t.seqs[0])
    for j in range(-(-9001 // 64)):
        m = min(64, 9001 - 64 * j)
        t.v[0, int(t.table[s, j]), :, :m] = t.V[0][64 * j:64 * j + m].transpose(0, 1)
    out, _ = run_attention(q, t)
    ref, _, tol, _ = t.reference(subnormal=2.0 ** -31)
    assert bool(((out.double() - ref).abs() <= tol).all())
    q.qhl_sync()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_f16_weights_of_a_long_tail_are_kept(q, dim):  # noqa: F811
    """One key in 64 has nearly all the weight and values of 0, the others less than 2^-25 of it each and values of 1024: alone,
    such a weight rounds to 0 in f16."""
    n, P = 9000, 64
    t = Trees([n], [[-1]], 1, 1, dim, P, torch.float16, seed=5)
    g = gen(31)
    score = -25.5 * math.log(2) + 0.4 * (torch.rand(n, generator=g) - 0.5)
    score[::64] = 0
    t.q.zero_(), t.k_new.zero_(), t.v_new.zero_()
    t.q[:, :, 0] = math.sqrt(dim)                        # the scale undoes it: a key's first element is its score
    t.K[0] = torch.zeros(n, 1, dim, dtype=torch.float16)
    t.K[0][:, 0, 0] = score.half()
    t.V[0] = torch.where(score == 0, 0.0, 1024.0)[:, None, None].expand(n, 1, dim).half()
    s = int(t.seqs[0])
    for j in range(-(-n // P)):
        m = min(P, n - P * j)
        t.k[0, int(t.table[s, j]), :, :m] = t.K[0][P * j:P * j + m].transpose(0, 1)
        t.v[0, int(t.table[s, j]), :, :m] = t.V[0][P * j:P * j + m].transpose(0, 1)
    out, _ = run_attention(q, t)
    w = torch.softmax(torch.cat([t.K[0][:, 0, 0].double(), torch.zeros(1, dtype=torch.float64)]), 0)
    ref = float((w[:n] * t.V[0][:, 0, 0].double()).sum())
    # every part of the sum has its own largest key, so a weight's half step is 2^-31 of a sum of at least n / 64 (+ 1 drafted):
    # n 2^-31 1024 / (n / 64); the scores are exact products, 2^-22 of 18 for the exponent; u for normal weights and the result
    u = half_step(torch.float16)
    tol = 64 * 2.0 ** -31 * 1024 + ref * (2.02 * u + 2 * 18 * 2.0 ** -22 + (n + 16) * 2.0 ** -23) + tiny_step(torch.float16)
    assert tol < 0.05 * ref
    assert bool(((out.double() - ref).abs() <= tol).all())
    q.qhl_sync()


@pytest.mark.parametrize("kv_heads,group,nodes,ctx", [
    (149, 1, [2], [130]),                                # more heads than CTAs, and a prime number of them
    (256, 1, [1, 3], [70, 0]),
    (1, 128, [128], [40]),                               # 128 M tiles
    (1, 128, [128, 1, 2], [40, 700, 9]),
    (2, 100, [77], [200]),                               # a group that is no divisor of a tile's rows
])
def test_attention_the_most_heads_and_tiles(q, kv_heads, group, nodes, ctx):  # noqa: F811
    g = gen(sum(nodes))
    check_attention(q, Trees(ctx, [random_tree(n, g) for n in nodes], kv_heads * group, kv_heads, 64, 16, torch.float16, seed=kv_heads))


def test_attention_the_most_trees(q):  # noqa: F811
    g = gen(1)
    size = torch.randint(0, 3, (2048,), generator=g).tolist()
    check_attention(q, Trees(torch.randint(0, 40, (2048,), generator=g).tolist(), [random_tree(m, g) for m in size], 2, 1, 64, 16, torch.bfloat16, seed=6))


def test_attention_calls_on_two_streams_at_once(q):  # noqa: F811
    """Calls that overlap have scratch of their own, also where the caller gives none."""
    t = [Trees([c, 60], [random_tree(9, gen(c)), [-1]], 6, 2, 256, 64, torch.float16, seed=c) for c in (5000, 3001)]
    want = [run_attention(q, x) for x in t]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = []
    for x in t:
        kv = q.KvPages(x.k.cuda(), x.v.cuda(), x.table.cuda(), x.lens.cuda(), x.held.cuda(), x.refs.cuda())
        ins = [y.cuda() for y in (x.seqs, x.q_start, x.parent, x.q, x.k_new, x.v_new)]
        calls.append((kv, ins, [torch.zeros(x.rows, 6, 256, dtype=x.dtype, device="cuda") for _ in range(20)], x))
    torch.cuda.synchronize()
    for r in range(20):
        for (kv, ins, out, x), s in zip(calls, streams):
            with torch.cuda.stream(s):
                q.qhl_tree_attention(kv, 0, *ins[:3], x.max_nodes, *ins[3:], out[r], scale=x.scale)
    torch.cuda.synchronize()
    for (_, _, out, _), w in zip(calls, want):
        assert all(torch.equal(o.cpu(), w[0]) for o in out)
    q.qhl_sync()


# ------------------------------------------------------------- norm and rope

@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 2])
def test_norm_rope_of_a_view_whose_width_is_not_a_multiple_of_16_bytes(q, src, n):  # noqa: F811
    """One row of padded rows is as good as two: the width of a view is no stride."""
    st = {"f32": torch.float32, **DTYPES}[src]
    full = torch.randn(n, 1024, generator=gen(n)).to(st).cuda()
    pos, one = torch.arange(n, dtype=torch.int32, device="cuda"), torch.ones(64, device="cuda")

    def run(y):
        out = [torch.zeros(n, h, 64, dtype=torch.float16, device="cuda") for h in (4, 2, 2)]
        return q.qhl_qk_norm_rope(4, 2, 64, 64, 1e4, 1e-6, y, pos, one, one, *out, offsets=(0, 512, 768))

    want = run(full)
    for width in (897, 898, 1023):                       # the last head ends at 896
        assert all(torch.equal(a, b) for a, b in zip(run(full[:, :width]), want))


@pytest.mark.parametrize("src,dst", [("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("f16", "bf16"), ("bf16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("dim,rope", [(256, 64), (256, 256), (128, 128), (128, 48), (64, 64), (64, 32), (64, 0), (128, 0), (256, 200)])
def test_norm_rope_of_many_rows(q, src, dst, dim, rope):  # noqa: F811
    """Four passes per warp: 2501 rows of 9 vectors, the last pass and the last CTA partly filled."""
    check_norm_rope(q, 2501, 7, 1, dim, rope, src, dst, seed=dim + rope)


def test_norm_rope_of_many_strided_rows(q):  # noqa: F811
    check_norm_rope(q, 2501, 6, 2, 128, 64, "bf16", "bf16", pad=24, offsets=(512, 0, 256))


@pytest.mark.parametrize("src,dim,rope", [("f32", 256, 64), ("bf16", 128, 128), ("f16", 64, 32)])
def test_norm_rope_gives_a_row_the_same_bits_alone_and_among_many(q, src, dim, rope):  # noqa: F811
    st, n = {"f32": torch.float32, **DTYPES}[src], 2501
    y = torch.randn(n, 16 * dim, generator=gen(dim)).to(st).cuda()
    pos = torch.randint(0, 262144, (n,), generator=gen(2), dtype=torch.int32).cuda()
    gamma = torch.randn(2, dim, generator=gen(3)).cuda()

    def run(rows):
        out = [torch.zeros(rows.stop - rows.start, h, dim, dtype=torch.bfloat16, device="cuda") for h in (7, 1, 1)]
        return q.qhl_qk_norm_rope(7, 1, dim, rope, 1e7, 1e-6, y[rows], pos[rows], gamma[0], gamma[1], *out)

    many = run(slice(0, n))
    for r in (0, 1, 1250, n - 1):
        assert all(torch.equal(a[0], b[r]) for a, b in zip(run(slice(r, r + 1)), many))


# ------------------------------------------------------------------ DeltaNet

def served(n, seed, most=40):
    """n trees of 0 to `most` tokens, some with padded ones, the largest not first."""
    g = gen(seed)
    size = torch.randint(0, 4, (n,), generator=g).tolist()
    size[n - 2], size[1] = most, 17
    trees = [random_tree(m, g) for m in size]
    trees[1][5], trees[1][9] = -2, -2
    assert max(len(vh.lineage(t, i) or []) for t in trees for i in range(len(t))) <= 13
    return trees


# 13 trees of 6 heads, or 2 of 48, are as many CTAs as take 32 rows each; beyond 32 trees they are not ordered by size
@pytest.mark.parametrize("n,Hk,Hv", [(13, 2, 6), (32, 2, 4), (33, 1, 4), (40, 2, 2), (2, 16, 48), (3, 16, 48)])
def test_deltanet_tree_batches_match_the_64_bit_form(q, n, Hk, Hv):  # noqa: F811
    assert Hv * 4 * n > 2 * 148
    parents = served(n, n) if n > 3 else [random_tree(18, gen(2)), [-1, -2, 0], [-1, 0, 0]][:n]
    y, states, starts, parent = dn_inputs(parents, Hk, Hv, 5, n, extra=2)
    index = [(3 * b) % 6 - 1 for b in range(n)]
    o, snaps = dn_run(q, y, states, starts, parent, index, Hk, Hv)
    ro, rs = vh.deltanet_tree(y, starts, parent.tolist(), states, index, Hk, Hv)
    end = starts[-1]
    dead = np.isnan(rs[:end]).any((1, 2, 3))
    assert dead.any()
    for r in range(end):                                 # the tolerance of test_deltanet_tree_matches_the_64_bit_form
        if dead[r]:
            assert bool((o[r] == 0).all()) and bool((snaps[r] == 9).all())
        else:
            assert np.abs(snaps[r].numpy() - rs[r]).max() <= 2.0 ** -16 * max(1, np.abs(rs[r]).max())
            assert np.abs(o[r].numpy() - ro[r]).max() <= 2.0 ** -16 * max(1, np.abs(ro[r]).max())
    assert bool((o[end:] == 9).all()) and bool((snaps[end:] == 9).all())
    q.qhl_sync()


@pytest.mark.parametrize("n,Hk,Hv,most", [(13, 2, 6, 40), (40, 2, 2, 128), (2, 16, 48, 35)])
def test_deltanet_tree_paths_in_a_batch_have_the_bits_of_the_chained_step(q, n, Hk, Hv, most):  # noqa: F811
    g = gen(most)
    parents = [random_tree(int(m), g) for m in torch.randint(1, 4, (n,), generator=g)]
    parents[n - 1] = random_tree(most, g)
    y, states, starts, parent = dn_inputs(parents, Hk, Hv, 2, n)
    o, snaps = dn_run(q, y, states, starts, parent, [b % 2 for b in range(n)], Hk, Hv)
    for b in (0, n - 1):
        tree = parents[b]
        deepest = max(range(len(tree)), key=lambda i: len(vh.lineage(tree, i)))
        for leaf in {len(tree) - 1, deepest}:
            S = states[b % 2:b % 2 + 1].cuda().contiguous()
            for i in vh.lineage(tree, leaf)[::-1]:
                r = starts[b] + i
                s1, o1 = torch.empty(1, Hv, 128, 128, device="cuda"), torch.empty(1, Hv * 128, device="cuda")
                q.qhl_deltanet_step(Hk, Hv, y[r:r + 1].cuda(), S, s1, o1)
                assert torch.equal(o1[0].cpu(), o[r]) and torch.equal(s1[0].cpu(), snaps[r])
                S = s1
    q.qhl_sync()


# --------------------------------------------------------------------- pages

def test_strides_along_an_axis_of_one_element_do_not_count(q):  # noqa: F811
    """A cache of one layer cut out of a larger one, and one drafted row of every layer: k and v may come from tensors of
    other sizes as long as the strides that are used agree."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
    half = lambda *s: torch.randn(s, generator=gen(1)).half().cuda()   # noqa: E731
    k, v = half(3, 4, 2, 16, 64)[1:2], half(1, 4, 2, 16, 64)
    assert k.stride(1) == v.stride(1)
    v3 = torch.as_strided(v, v.shape, (8, *v.stride()[1:]))
    kv = q.KvPages(k, v3, i32(1, 2), i32(1) + 4, i32(1) + 1, i32(4) + 1)
    new_k, new_v = half(1, 1, 2, 64), half(2, 3, 2, 64)[:1, 1:2]
    assert new_k.stride() != new_v.stride()
    status = i32(1) + 9
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    q.qhl_pages_commit(kv, i32(1), starts, i32(1, 1), i32(1) + 1, i32(1) + 4, new_k, new_v, status)
    assert status.tolist() == [0] and kv.lens.tolist() == [5]
    assert torch.equal(k[0, 0, :, 4], new_k[0, 0]) and torch.equal(v[0, 0, :, 4], new_v[0, 0])
    q.qhl_sync()


def test_pages_needs_beyond_32_bits_are_refused(q):  # noqa: F811
    """34 requests of 2^27 pages each: their sum passes 2^31 and 2^32, the pool has eight."""
    S, most = 34, 1 << 27
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
    pool = torch.zeros(1, 8, 1, 16, 64, dtype=torch.float16, device="cuda")
    table = torch.empty(S, most, dtype=torch.int32, device="cuda")       # 17 GB, of which nothing is read
    kv = q.KvPages(pool, pool.clone(), table, i32(S), i32(S), i32(8))
    seqs, status = torch.arange(S, dtype=torch.int32, device="cuda"), i32(S) + 9
    add = torch.full((S,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    q.qhl_pages_extend(kv, seqs, add, status)
    assert status.tolist() == [-3] * S
    assert kv.held.tolist() == [0] * S and kv.refs.tolist() == [0] * 8
    add[0] = 100                                         # what the pool has goes to the requests before the one that fails
    q.qhl_pages_extend(kv, seqs, add, status)
    assert status.tolist() == [0] + [-3] * (S - 1)
    assert kv.held.tolist() == [7] + [0] * (S - 1) and kv.refs.tolist() == [1] * 7 + [0] and table[0, :7].tolist() == list(range(7))
    q.qhl_sync()


def test_pages_beyond_2_31_elements_are_copied_and_written(q):  # noqa: F811
    """A pool of more than 2^31 elements whose last pages are used: a shared page is copied among them, a path committed."""
    n_pages, H, P, D = 33000, 4, 64, 256
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    k = torch.empty(1, n_pages, H, P, D, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    assert k[0, n_pages - 4].data_ptr() - k.data_ptr() > 2 * 2 ** 31
    old, new, after = n_pages - 2, n_pages - 4, n_pages - 3
    refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
    refs[old], refs[new], refs[after] = 2, 0, 0
    for c, base in ((k, 1), (v, 2)):
        c[0, old:old + 1] = torch.randn(1, H, P, D, generator=gen(base)).half().cuda()
        c[0, new], c[0, after] = 7, 7
    kv = q.KvPages(k, v, i32([[old, -1], [old, -1]]), i32([40, 40]), i32([1, 1]), refs)
    status = i32([9])
    q.qhl_pages_extend(kv, i32([1]), i32([30]), status)
    assert status.tolist() == [0] and kv.table.tolist() == [[old, -1], [new, after]] and refs[old:].tolist() == [1, 1]
    for c in (k, v):
        assert torch.equal(c[0, new, :, :40], c[0, old, :, :40]) and bool((c[0, new, :, 40:] == 7).all()) and bool((c[0, after] == 7).all())
    kn, vn = (torch.randn(1, 30, H, D, generator=gen(s)).half().cuda() for s in (3, 4))
    path = torch.randperm(30, generator=gen(5)).tolist()
    q.qhl_pages_commit(kv, i32([1]), i32([0, 30]), i32([path]), i32([30]), i32([40]), kn, vn, status)
    assert status.tolist() == [0] and kv.lens.tolist() == [40, 70]
    for c, x in ((k, kn), (v, vn)):
        rows = torch.cat([c[0, new, :, 40:], c[0, after, :, :6]], 1)
        assert torch.equal(rows, x[0, path].transpose(0, 1)) and bool((c[0, after, :, 6:] == 7).all())
    q.qhl_sync()


# ------------------------------------------- a step of a layer, and its oracle

def test_a_layer_of_the_stage_as_a_tree_over_pages(q):  # noqa: F811
    """The in-projections of the 27B-class shapes (quantised GEMV), then the tree operators, against the oracle's mixers run
    along every path: an attention layer over 100 cached rows in pages, and a DeltaNet layer."""
    import oracle
    import synth
    from synth import FULL, Q4_0
    Hq, H, D, ctx, P, seed = FULL.att_q_heads, FULL.att_kv_heads, FULL.att_dim, 100, 64, 7
    tree = [-1, 0, 0, 2, 1, -1]
    n = len(tree)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    x = oracle.rmsnorm(synth.hidden(FULL, seed, 0, n), np.ones(FULL.hidden), FULL.eps).astype(np.float32)
    t = {**synth.layer_tensors(FULL, Q4_0, seed, 2), **synth.layer_tensors(FULL, Q4_0, seed, 3)}

    def project(name, rows):
        W = t[name]
        packed = torch.empty(q.qhl_packed_bytes(Q4_0, rows, FULL.hidden), dtype=torch.uint8, device="cuda")
        q.qhl_repack(Q4_0, rows, FULL.hidden, torch.from_numpy(np.ascontiguousarray(W).reshape(-1)).cuda(), packed)
        y = torch.empty(n, rows, device="cuda")
        q.qhl_qgemv(Q4_0, rows, FULL.hidden, packed, torch.from_numpy(x).cuda(), y)
        return y, oracle.qgemv(Q4_0, W, x)

    # attention: y is q | gate | k | v
    y, ry = project("blk.3.attn_in", FULL.attn_in_rows)
    gq, gk = t["blk.3.attn_q_norm"], t["blk.3.attn_k_norm"]
    K, V = synth.kv_prefill(FULL, seed, 3, ctx, ctx + n)
    k, v = (torch.from_numpy(np.pad(c[:, :ctx], ((0, 0), (0, 2 * P - ctx), (0, 0)), constant_values=np.nan).reshape(H, 2, P, D)).permute(1, 0, 2, 3)[None]
            .contiguous().cuda() for c in (K, V))
    kv = q.KvPages(k, v, i32([[0, 1]]), i32([ctx]), i32([2]), i32([1, 1]))
    pos = [ctx + len(vh.lineage(tree, i)) - 1 for i in range(n)]
    qq, out = (torch.empty(n, Hq, D, dtype=torch.float16, device="cuda") for _ in range(2))
    kn, vn = (torch.empty(n, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    q.qhl_qk_norm_rope(Hq, H, D, FULL.rope_dims, FULL.rope_theta, FULL.eps, y, i32(pos), torch.from_numpy(gq).cuda(), torch.from_numpy(gk).cuda(), qq, kn, vn)
    q.qhl_tree_attention(kv, 0, i32([0]), i32([0, n]), i32(tree), n, qq, kn, vn, out)
    gate = torch.sigmoid(y[:, Hq * D:2 * Hq * D].double()).cpu().numpy()
    got = out.double().cpu().numpy().reshape(n, -1) * gate
    u = half_step(torch.float16)
    for i in range(n):
        line = vh.lineage(tree, i)[::-1]
        Kp, Vp = K.copy(), V.copy()
        for j, node in enumerate(line):                  # the oracle keeps one chain: its path
            ref = oracle.attention_token(ry[node], ctx + j, Kp, Vp, gq, gk, FULL)
        end = ctx + len(line)
        qi = oracle.rope(oracle.rmsnorm(ry[i][:Hq * D].reshape(Hq, D), gq, FULL.eps), pos[i], FULL.rope_dims, FULL.rope_theta)
        for h in range(Hq):
            Kh, Vh = Kp[h // (Hq // H), :end].astype(np.float64), Vp[h // (Hq // H), :end].astype(np.float64)
            s = Kh @ qi[h] / 16
            w = np.exp(s - s.max())
            w /= w.sum()
            # q is rounded to f16 (u), a drafted k and v may be one rounding apart from the oracle's (2 u each), the projections
            # and the f32 sums are good to 2^-14 of their magnitudes; the errors of different elements of q and k are
            # independent, but the bound adds them up
            ds = (3 * u + 2.0 ** -14) * (np.abs(Kh) @ np.abs(qi[h])).max() / 16
            A = w @ np.abs(Vh)
            tol = (A * (2 * ds + 3.01 * u + 2.0 ** -14) + u * np.abs(w @ Vh)) * gate[i, h * D:(h + 1) * D] + 2.0 ** -14 * A
            assert (np.abs(got[i, h * D:(h + 1) * D] - ref[h * D:(h + 1) * D]) <= tol).all()
            # and on the whole: independent errors of 256 elements of q and k leave a few half steps of the output's size
            assert oracle.max_rel_err(got[i, h * D:(h + 1) * D], ref[h * D:(h + 1) * D]) <= 8 * u

    # DeltaNet: y is q | k | v | b | a
    y, ry = project("blk.2.dn_in", FULL.dn_in_rows)
    S0 = synth.dn_state(FULL, seed, 2)
    snaps, o = torch.empty(n, FULL.dn_v_heads, 128, 128, device="cuda"), torch.empty(n, FULL.dn_o, device="cuda")
    q.qhl_deltanet_tree(FULL.dn_k_heads, FULL.dn_v_heads, y, i32([0, n]), i32(tree), n, torch.from_numpy(S0)[None].cuda(), i32([0]), snaps, o)
    for i in range(n):
        S = S0.astype(np.float64)
        for node in vh.lineage(tree, i)[::-1]:
            S, ro = oracle.deltanet_token(S, *oracle.split_dn_in(ry[node], FULL), FULL)
        assert oracle.max_rel_err(o[i].cpu().numpy(), ro.reshape(-1)) <= 2e-3          # the stage's own bounds
        for h in range(FULL.dn_v_heads):
            assert oracle.max_rel_err(snaps[i, h].cpu().numpy(), S[h]) <= 2e-3
    q.qhl_sync()
