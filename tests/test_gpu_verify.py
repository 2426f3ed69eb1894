"""The tree-verification operators on the GPU against plain 64-bit forms.

QK-norm with rotation, the gated DeltaNet step along trees, the page operations,
tree attention over a paged cache, and a whole verify step that uses them
together (with the quantised GEMV before them)."""
import numpy as np
import pytest
import torch

import verify_helpers as vh
from verify_helpers import DTYPES, Trees, gen, half_step, random_tree, tiny_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU test needs CUDA"
    import quantized_hybrid_layer_b200 as q
    q.qhl_sync()
    return q


def test_the_binding_refuses_wrong_tensors_on_the_gpu(q):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
    k = torch.zeros(2, 4, 2, 16, 64, dtype=torch.float16, device="cuda")
    kv = q.KvPages(k, k.clone(), i32(3, 2), i32(3), i32(3), i32(4))
    x, n = torch.zeros(2, 4, 64, dtype=torch.float16, device="cuda"), torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")

    def refused(f, good, bad):
        f(**good)
        for o in bad:
            with pytest.raises((ValueError, q.StageError)):
                f(**{**good, **o})

    refused(q.qhl_tree_attention, dict(kv=kv, layer=0, seqs=i32(1), q_start=i32(2), parent=i32(2) - 1, max_nodes=2, q=x, k_new=n, v_new=n, out=x.clone()),
            [dict(q=x.bfloat16()), dict(q=x.transpose(0, 1)), dict(q=x.cpu()), dict(k_new=x), dict(v_new=torch.cat([n, n], 1)[:, :2]), dict(out=x[:1]),
             dict(lse=torch.zeros(2, 2, device="cuda")), dict(lse=torch.zeros(2, 4)), dict(parent=i32(3)), dict(parent=i32(2).long()), dict(q_start=i32(1)),
             dict(seqs=i32(1).cpu()), dict(seqs=i32(1, 1)), dict(layer=2), dict(max_nodes=0), dict(max_nodes=129), dict(scale=-1.0), dict(scale="x"),
             dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")), dict(workspace=torch.zeros(1 << 24, dtype=torch.uint8)), dict(stream="x")])
    y, p = torch.zeros(2, 768, device="cuda"), i32(2)
    one = torch.ones(64, device="cuda")
    refused(lambda **a: q.qhl_qk_norm_rope(4, 2, 64, a.get("rope", 64), 1e4, 1e-6, *(a[c] for c in ("y", "p", "gq", "gk", "q", "k", "v")), **a["kw"]),
            dict(y=y, p=p, gq=one, gk=one, q=x, k=n, v=n.clone(), kw={}),
            [dict(y=y[:, :760]), dict(y=y.double()), dict(y=y.cpu()), dict(y=y.t()), dict(p=p[:1]), dict(p=p.long()), dict(gq=one[:32]), dict(gk=one.half()),
             dict(q=x.float()), dict(k=n.bfloat16()), dict(v=n[:1]), dict(rope=60), dict(kw=dict(offsets=(0, 640, 700))), dict(kw=dict(offsets=(0, -8, 640)))])
    st, sn = torch.zeros(1, 4, 128, 128, device="cuda"), torch.zeros(2, 4, 128, 128, device="cuda")
    refused(lambda **a: q.qhl_deltanet_tree(4, 4, a["y"], a["s"], a["p"], 2, a["st"], a["ix"], a["sn"], a["o"]),
            dict(y=torch.zeros(2, 1544, device="cuda"), s=i32(2), p=i32(2) - 1, st=st, ix=i32(1), sn=sn, o=torch.zeros(2, 512, device="cuda")),
            [dict(y=torch.zeros(2, 1540, device="cuda")), dict(s=i32(1)), dict(p=i32(3)), dict(st=st[:, :2]), dict(st=st.half()), dict(sn=sn[:1]),
             dict(st=sn), dict(o=torch.zeros(2, 512)), dict(ix=i32(1).long())])
    for f, good in ((q.qhl_pages_free, (i32(1), i32(1))), (q.qhl_pages_fork, (i32(1), i32(1) + 1, i32(1))), (q.qhl_pages_extend, (i32(1), i32(1), i32(1)))):
        f(kv, *good)
        for at in range(len(good)):
            for bad in (good[at].long(), i32(2), good[at].cpu()):
                with pytest.raises(ValueError):
                    f(kv, *good[:at], bad, *good[at + 1:])
        with pytest.raises(q.StageError):
            f(kv, *(g[:0] for g in good))                # no requests
    new = torch.zeros(2, 2, 2, 64, dtype=torch.float16, device="cuda")
    refused(lambda **a: q.qhl_pages_commit(kv, a["s"], a["q"], a["p"], a["n"], a["at"], a["k"], a["v"], a["st"]),
            dict(s=i32(1), q=i32(2), p=i32(1, 2), n=i32(1), at=i32(1), k=new, v=new, st=i32(1)),
            [dict(s=i32(2)), dict(q=i32(1)), dict(p=i32(2)), dict(p=i32(2, 2)), dict(n=i32(2)), dict(at=i32(1).cpu()), dict(k=new[:1]), dict(v=new.float()),
             dict(k=new.transpose(1, 2)), dict(st=i32(0))])
    q.qhl_sync()


# ------------------------------------------------------------- norm and rope

def check_norm_rope(q, n, hq, hkv, dim, rope, src, dst, theta=1e7, far=262144, seed=0, pad=0, offsets=None):
    g = gen(seed)
    st, dt = {"f32": torch.float32, **DTYPES}[src], DTYPES[dst]
    width = 2 * hq * dim + 2 * hkv * dim
    off = offsets or (0, 2 * hq * dim, 2 * hq * dim + hkv * dim)
    full = (torch.randn(n, width + pad, generator=g) * 3).to(st)
    if n > 2:
        full[1] = 0                                     # a row of zeros: the norm's eps alone
        full[2] *= 1e-4
    y = full[:, :width]
    pos = torch.randint(0, far, (n,), generator=g, dtype=torch.int32)
    gq, gk = 1 + 0.1 * torch.randn(dim, generator=g), 1 + 0.1 * torch.randn(dim, generator=g)
    out = [torch.full((n, h + 1, dim), 7.0, dtype=dt, device="cuda")[:, :h] for h in (hq, hkv, hkv)]   # rows with room behind them
    q.qhl_qk_norm_rope(hq, hkv, dim, rope, theta, 1e-6, full.cuda()[:, :width], pos.cuda(), gq.cuda(), gk.cuda(), *out, offsets=off)
    torch.cuda.synchronize()
    for t, h, o, gamma in ((out[0], hq, off[0], gq), (out[1], hkv, off[1], gk)):
        ref, mag = vh.norm_rope(y[:, o:o + h * dim].reshape(n, h, dim), gamma, pos, rope, theta, 1e-6)
        # rounded once; before that about a dozen f32 roundings of the parts and an angle good to 2^-21
        tol = half_step(dt) * ref.abs() + 2.0 ** -19 * mag + tiny_step(dt)
        assert bool(((t.cpu().double() - ref).abs() <= tol).all())
    v = y[:, off[2]:off[2] + hkv * dim].reshape(n, hkv, dim).float().to(dt)
    assert torch.equal(out[2].cpu(), v)
    for t, h in zip(out, (hq, hkv, hkv)):               # what lies between the rows is left as it was
        assert bool((t._base[:, h] == 7).all())


@pytest.mark.parametrize("src,dst", [("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("dim,rope", [(256, 64), (256, 256), (128, 128), (128, 48), (64, 64), (64, 32), (256, 0), (256, 8), (256, 200)])
def test_norm_rope_types_and_sizes(q, src, dst, dim, rope):
    check_norm_rope(q, 5, 6, 2, dim, rope, src, dst, seed=dim + rope)


@pytest.mark.parametrize("n,hq,hkv", [(1, 24, 4), (1, 1, 1), (3, 7, 7), (37, 5, 1), (2000, 24, 4)])
def test_norm_rope_rows_and_heads(q, n, hq, hkv):
    check_norm_rope(q, n, hq, hkv, 256, 64, "f32", "bf16", seed=n)


def test_norm_rope_strided_rows_and_other_offsets(q):
    check_norm_rope(q, 9, 4, 2, 128, 64, "f32", "f16", pad=64)
    check_norm_rope(q, 9, 4, 2, 128, 64, "bf16", "bf16", pad=8, offsets=(512, 0, 256))


def test_norm_rope_negative_and_extreme_positions(q):
    dt, dim = torch.float16, 64
    x = torch.randn(4, 4 * dim, generator=gen(3))
    pos = torch.tensor([-5, 0, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    out = [torch.empty(4, 1, dim, dtype=dt, device="cuda") for _ in range(3)]
    one = torch.ones(dim, device="cuda")
    q.qhl_qk_norm_rope(1, 1, dim, dim, 1e4, 1e-6, x.cuda(), pos.cuda(), one, one, *out)
    ref, mag = vh.norm_rope(x[:, :dim].reshape(4, 1, dim), one.cpu(), pos, dim, 1e4, 1e-6)
    # the angle's own 64-bit roundings: 2^31 rad off by 2^-21 (ten roundings of 2^-53 relative)
    assert bool(((out[0].cpu().double() - ref).abs() <= half_step(dt) * ref.abs() + 2.0 ** -17 * mag + tiny_step(dt)).all())


# ------------------------------------------------------------------ DeltaNet

def dn_inputs(parents, Hk, Hv, n_states, seed, extra=0):
    g = gen(seed)
    n = sum(map(len, parents)) + extra
    y = torch.randn(n, 2 * Hk * 128 + Hv * 128 + 2 * Hv, generator=g)
    states = 0.1 * torch.randn(n_states, Hv, 128, 128, generator=g)
    starts = np.cumsum([0] + [len(p) for p in parents])
    parent = torch.tensor(sum(parents, []) + [-1] * extra, dtype=torch.int32)
    return y, states, [int(x) for x in starts], parent


def dn_run(q, y, states, starts, parent, index, Hk, Hv, fill=9.0):
    n = y.shape[0]
    snaps = torch.full((n, Hv, 128, 128), fill, device="cuda")
    o = torch.full((n, Hv * 128), fill, device="cuda")
    q.qhl_deltanet_tree(Hk, Hv, y.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), parent.cuda(),
                        max(1, max(b - a for a, b in zip(starts, starts[1:]))), states.cuda(), torch.tensor(index, dtype=torch.int32).cuda(), snaps, o)
    torch.cuda.synchronize()
    return o.cpu(), snaps.cpu()


TREES = {
    "one": [[-1]],
    "chain": [[-1, 0, 1, 2, 3]],
    "star": [[-1, 0, 0, 0, -1, -1]],
    "far_parents": [[-1, 0, 1, 2, 0, 4, 1, 6, 3, 8, -1, 10, 5]],
    "padded": [[-1, 0, -2, 2, 1, -2]],
    "first_padded": [[-2, -1, 0, 1]],
    "all_padded": [[-2, -2]],
    "ragged": [[-1, 0, 0], [], [-1], [-1, -1, 1, 1, 0]],
}


@pytest.mark.parametrize("name", TREES)
@pytest.mark.parametrize("Hk,Hv", [(2, 6), (4, 4)])
def test_deltanet_tree_matches_the_64_bit_form(q, name, Hk, Hv):
    parents = TREES[name]
    y, states, starts, parent = dn_inputs(parents, Hk, Hv, 5, 11, extra=2)
    index = [3, -1, 0, 4][:len(parents)]
    o, snaps = dn_run(q, y, states, starts, parent, index, Hk, Hv)
    ro, rs = vh.deltanet_tree(y, starts, parent.tolist(), states, index, Hk, Hv)
    end = starts[-1]
    # per step about a hundred f32 roundings of terms no larger than the state's largest: 2^-16 of it after 13 steps
    dead = np.isnan(rs[:end]).any((1, 2, 3))
    for r in range(end):
        if dead[r]:
            assert bool((o[r] == 0).all()) and bool((snaps[r] == 9).all())   # padded: output 0, no snapshot
        else:
            assert np.abs(snaps[r].numpy() - rs[r]).max() <= 2.0 ** -16 * max(1, np.abs(rs[r]).max())
            assert np.abs(o[r].numpy() - ro[r]).max() <= 2.0 ** -16 * max(1, np.abs(ro[r]).max())
    assert bool((o[end:] == 9).all()) and bool((snaps[end:] == 9).all())       # rows behind the last tree


@pytest.mark.parametrize("n", [1, 16, 17, 40, 128])
def test_deltanet_tree_paths_have_the_bits_of_the_chained_step(q, n):
    Hk, Hv = 2, 4
    tree = random_tree(n, gen(n))
    y, states, starts, parent = dn_inputs([tree], Hk, Hv, 1, n)
    o, snaps = dn_run(q, y, states, starts, parent, [0], Hk, Hv)
    deepest = max(range(n), key=lambda i: len(vh.lineage(tree, i)))
    for leaf in {n - 1, deepest}:
        line = vh.lineage(tree, leaf)[::-1]
        S = states[:1].cuda().contiguous()
        for i in line:
            s1, o1 = torch.empty(1, Hv, 128, 128, device="cuda"), torch.empty(1, Hv * 128, device="cuda")
            q.qhl_deltanet_step(Hk, Hv, y[i:i + 1].cuda(), S, s1, o1)
            assert torch.equal(o1[0].cpu(), o[i]) and torch.equal(s1[0].cpu(), snaps[i])
            S = s1


def test_deltanet_tree_reports_bad_indices_and_does_not_follow_them(q):
    Hk, Hv = 1, 2
    y, states, starts, parent = dn_inputs([[-1, 0], [-1, 0]], Hk, Hv, 2, 5)
    ref = dn_run(q, y, states, starts, parent, [0, 1], Hk, Hv)
    q.qhl_sync()
    bad = parent.clone()
    bad[1], bad[3] = 1, 7                                # its own index; beyond its tree
    o, snaps = dn_run(q, y, states, starts, bad, [0, 1], Hk, Hv)
    assert torch.equal(o[0], ref[0][0]) and torch.equal(o[2], ref[0][2]) and bool((o[[1, 3]] == 0).all())
    with pytest.raises(q.StageError) as e:
        q.qhl_sync()
    assert e.value.code == -7 and "index" in str(e.value)
    o, _ = dn_run(q, y, states, starts, parent, [0, 2], Hk, Hv)      # state 2 of 2: the zero state
    assert torch.equal(o[:2], ref[0][:2])
    zero = dn_run(q, y, states, starts, parent, [0, -1], Hk, Hv)
    assert torch.equal(o, zero[0])
    with pytest.raises(q.StageError):
        q.qhl_sync()
    o, _ = dn_run(q, y, states, [0, 2, 9], parent, [0, 1], Hk, Hv)   # a tree beyond the rows is left out
    assert torch.equal(o[:2], ref[0][:2]) and bool((o[2:] == 9).all())
    with pytest.raises(q.StageError):
        q.qhl_sync()
    q.qhl_sync()


# --------------------------------------------------------------------- pages

class Both:
    """A cache on the GPU beside its plain form."""

    def __init__(self, q, n_pages=24, page=16, seqs=10, max_pages=8, layers=3, heads=2, dim=64, dtype=torch.float16, seed=0, permute=False):
        self.q, self.plain = q, vh.Pages(n_pages, page, seqs, max_pages)
        g = gen(seed)
        self.ref_k = torch.randn(layers, n_pages, heads, page, dim, generator=g).to(dtype)
        self.ref_v = torch.randn(layers, n_pages, heads, page, dim, generator=g).to(dtype)
        put = (lambda x: x.cuda().permute(1, 3, 0, 2, 4).contiguous().permute(2, 0, 3, 1, 4)) if permute else (lambda x: x.cuda())
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
        self.kv = q.KvPages(put(self.ref_k), put(self.ref_v), i32(seqs, max_pages) - 1, i32(seqs), i32(seqs), i32(n_pages))

    def call(self, name, *args):
        t = [torch.tensor(a, dtype=torch.int32, device="cuda") for a in args]
        status = torch.full((len(args[0]),), 5, dtype=torch.int32, device="cuda")
        getattr(self.q, "qhl_pages_" + name)(self.kv, *t, status)
        got, want = status.tolist(), getattr(self.plain, name)(*args)
        if name == "extend":
            for a, b, rows in self.plain.copies:
                self.ref_k[:, b, :, :rows] = self.ref_k[:, a, :, :rows]
                self.ref_v[:, b, :, :rows] = self.ref_v[:, a, :, :rows]
        assert got == want, name
        self.check()
        return want

    def grow(self, seq, rows):
        """Committed rows for a sequence that has room for them."""
        self.plain.lens[seq] = rows
        self.kv.lens[seq] = rows

    def check(self):
        p = self.plain
        assert self.kv.refs.tolist() == p.refs
        assert self.kv.lens.tolist() == p.lens
        assert self.kv.held.tolist() == [len(r) for r in p.rows]
        for s, r in enumerate(p.rows):
            assert self.kv.table[s, :len(r)].tolist() == r
        assert torch.equal(self.kv.k.cpu(), self.ref_k) and torch.equal(self.kv.v.cpu(), self.ref_v)


@pytest.mark.parametrize("permute", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_pages_fork_extend_free(q, permute, dtype):
    c = Both(q, permute=permute, dtype=dtype)
    c.call("extend", [0, 4], [37, 16])
    c.grow(0, 37)
    c.grow(4, 16)                                        # ends with its page
    c.call("fork", [0, 0, 4, 0], [1, 2, 5, 3])
    c.call("extend", [1, 5, 2], [3, 1, 20])              # a shared page that is copied, one that is full
    c.call("extend", [0, 3], [1, 1])                     # two holders are left: the first copies, the second keeps
    c.call("free", [2, 0])
    c.call("extend", [6], [40])
    c.call("free", [1, 3, 4, 5, 6, 9])
    assert c.plain.refs == [0] * 24
    q.qhl_sync()


def test_pages_requests_that_fail_change_nothing(q):
    c = Both(q, n_pages=6)
    c.call("extend", [0, 0, -1, 10, 1, 2], [20, 1, 1, 1, -4, 16 * 8 + 1])
    c.grow(0, 20)
    c.call("fork", [0, 1, 0, 0, 3, -1, 0], [1, 2, 1, 0, 3, 4, 10])
    c.call("fork", [0, 4], [1, 6])                       # 1 holds pages
    c.call("extend", [3, 4, 5, 6], [40, 40, 1, 0])       # four pages are free: 3, then none, then none, then nothing asked
    c.call("free", [3, 3, -5, 99, 8])
    c.call("extend", [1, 0], [1, 1])
    q.qhl_sync()


def test_pages_that_run_out_while_the_last_page_is_shared(q):
    c = Both(q, n_pages=3)
    c.call("extend", [0], [20])
    c.grow(0, 20)
    c.call("fork", [0, 0], [1, 2])
    c.call("extend", [0, 1, 2], [1, 1, 1])               # one page is free: 0 copies, 1 fails, 2 shares and fails with it
    c.call("extend", [1], [1])
    q.qhl_sync()


def test_pages_shared_beyond_the_next_row_are_refused(q):
    c = Both(q)
    c.call("extend", [0], [60])
    c.grow(0, 60)
    c.call("fork", [0], [1])
    c.grow(1, 20)                                        # taken back: pages 2 and 3 stay shared
    c.call("extend", [1], [30])
    c.call("extend", [1], [5])
    q.qhl_sync()


def test_pages_random_operations(q):
    g = gen(77)
    c = Both(q, n_pages=40, seqs=14, max_pages=6, layers=1, heads=1)
    pick = lambda n, hi, lo=0: torch.randint(lo, hi, (n,), generator=g).tolist()   # noqa: E731
    for step in range(40):
        n = int(torch.randint(1, 8, (), generator=g))
        op = ("extend", "fork", "free", "extend")[step % 4]
        a = pick(n, 15, -1)
        if op == "extend":
            add = pick(n, 30)
            for s, m, rc in zip(a, add, c.call("extend", a, add)):
                if rc == 0 and 0 <= s < 14:
                    c.grow(s, c.plain.lens[s] + m)
        elif op == "fork":
            c.call("fork", a, pick(n, 15, -1))
        else:
            c.call("free", a)
    q.qhl_sync()


def test_pages_many_requests_and_pages(q):
    c = Both(q, n_pages=20000, seqs=1024, max_pages=16, layers=1, heads=1)
    order = torch.randperm(1024, generator=gen(4)).tolist()
    add = torch.randint(0, 250, (1024,), generator=gen(5)).tolist()
    c.call("extend", order, add)
    c.call("free", order[::3])
    c.call("extend", order[::-1], add)
    q.qhl_sync()


@pytest.mark.parametrize("dim,heads,page,permute", [(256, 4, 64, False), (64, 1, 16, True), (128, 3, 256, True)])
def test_pages_commit(q, dim, heads, page, permute):
    c = Both(q, n_pages=12, page=page, seqs=5, max_pages=3, layers=2, heads=heads, dim=dim, dtype=torch.bfloat16, permute=permute)
    c.call("extend", [0, 1, 2, 3], [2 * page, page, page + 9, 2 * page])
    lens = [page - 1, 3, page, 5]
    for s, n in enumerate(lens):
        c.grow(s, n)
    g = gen(9)
    starts = [0, 6, 7, 7, 15]
    rows = 17
    # rows of a larger tensor
    k_new = torch.randn(2, rows, heads + 1, dim, generator=g).bfloat16()
    v_new = torch.randn(2, rows, heads + 1, dim, generator=g).bfloat16()
    seqs, path = [1, 0, 2, 3], [[5, 0, 0, 3], [0, -1, -1, -1], [-1] * 4, [0, 1, 6, 7]]
    acc, pos = [4, 1, 0, 4], [3, page - 1, page - 2, 0]
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    status = t([9] * 4)
    q.qhl_pages_commit(c.kv, t(seqs), t(starts), t(path), t(acc), t(pos), k_new.cuda()[:, :, :heads], v_new.cuda()[:, :, :heads], status)
    assert status.tolist() == [0, 0, 0, 0]
    for b, s in enumerate(seqs):
        for j in range(acc[b]):
            r = pos[b] + j
            p = c.plain.rows[s][r // page]
            c.ref_k[:, p, :, r % page] = k_new[:, starts[b] + path[b][j], :heads]
            c.ref_v[:, p, :, r % page] = v_new[:, starts[b] + path[b][j], :heads]
        c.plain.lens[s] = pos[b] + acc[b]
    c.check()
    # refused one by one: nothing changes (the first change takes sequence 0 back to 7 rows and
    # the second sequence 3 to none, so their positions are too far where they come again)
    c.call("fork", [1], [4])
    bad = [(dict(seqs=[0, 0, 5, -1]), [0, -1, -1, -1]), (dict(acc=[5, -1, 0, 0]), [-1, -1, 0, 0]), (dict(pos=[8, -1, page - 2, 4]), [-1, -1, 0, -1]),
           (dict(path=[[6, 0, 0, 0], [1, 0, 0, 0], [0] * 4, [-1] * 4]), [-1, -1, 0, -1]), (dict(seqs=[4, 0, 2, 3]), [-2, -1, 0, 0])]
    for change, want in bad:
        a = dict(seqs=seqs, path=path, acc=acc, pos=[3, page - 1, page - 2, 0])
        a.update(change)
        before = c.kv.lens.tolist()
        q.qhl_pages_commit(c.kv, t(a["seqs"]), t(starts), t(a["path"]), t(a["acc"]), t(a["pos"]), k_new.cuda()[:, :, :heads],
                           v_new.cuda()[:, :, :heads], status)
        # 1 and 4 share their page now, so tree 0 fails with E_STATE where nothing else is wrong
        want = [(-2 if b == 0 and w == 0 and a["seqs"][0] == 1 else w) for b, w in enumerate(want)]
        assert status.tolist() == want, change
        after = c.kv.lens.tolist()
        for b, s in enumerate(a["seqs"]):
            if want[b] and 0 <= s < 5 and s not in [x for x, w in zip(a["seqs"], want) if w == 0]:
                assert after[s] == before[s]
        assert torch.equal(c.kv.k.cpu()[:, c.plain.rows[1][0]], c.ref_k[:, c.plain.rows[1][0]])
    q.qhl_sync()


# ----------------------------------------------------------------- attention

def run_attention(q, t: Trees, kv=None, workspace=None, lse=True, stream=None, fill=9.0):
    kv = kv or q.KvPages(t.k.cuda(), t.v.cuda(), t.table.cuda(), t.lens.cuda(), t.held.cuda(), t.refs.cuda())
    out = torch.full((t.rows, t.heads, t.dim), fill, dtype=t.dtype, device="cuda")
    ls = torch.full((t.rows, t.heads), fill, device="cuda") if lse else None
    q.qhl_tree_attention(kv, 0, t.seqs.cuda(), t.q_start.cuda(), t.parent.cuda(), t.max_nodes, t.q.cuda(), t.k_new.cuda(), t.v_new.cuda(), out,
                         lse=ls, scale=t.scale, workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), None if ls is None else ls.cpu()


def check_attention(q, t: Trees, **kw):
    out, lse = run_attention(q, t, **kw)
    ref, rl, tol, ltol = t.reference()
    end = int(t.q_start[-1])
    d = (out[:end].double() - ref[:end]).abs()
    assert bool((d <= tol[:end]).all()), f"out off by {float((d / tol[:end].clamp(min=1e-30)).max()):.3g} of what is allowed"
    seen = rl[:end] > -float("inf")
    assert torch.equal(lse[:end] == -float("inf"), ~seen)
    dl = (lse[:end].double() - rl[:end]).abs()[seen]
    assert bool((dl <= ltol[:end][seen]).all()), f"lse off by {float(dl.max()):.3g}"
    assert bool((out[end:] == 9).all()) and bool((lse[end:] == 9).all())
    q.qhl_sync()
    return out, lse


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,page", [(256, 64), (256, 16), (128, 128), (64, 32), (256, 256), (128, 16), (64, 256)])
@pytest.mark.parametrize("ctx", [0, 1, 63, 64, 65, 129, 700])
def test_attention_one_token(q, dtype, dim, page, ctx):
    check_attention(q, Trees([ctx], [[-1]], 6, 2, dim, page, DTYPES[dtype], seed=ctx + dim))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("nodes,heads,kv_heads", [(2, 4, 4), (16, 6, 1), (21, 6, 1), (22, 6, 1), (33, 8, 2), (64, 6, 1), (65, 2, 2), (128, 1, 1),
                                                  (3, 128, 1), (43, 6, 1)])
def test_attention_trees(q, dim, nodes, heads, kv_heads):
    t = Trees([150], [random_tree(nodes, gen(nodes))], heads, kv_heads, dim, 32, torch.bfloat16, seed=nodes)
    check_attention(q, t)


@pytest.mark.parametrize("dim,page,dtype", [(256, 64, "f16"), (128, 16, "bf16"), (64, 128, "f16")])
def test_attention_ragged_batch(q, dim, page, dtype):
    g = gen(5)
    ctx = [0, 300, 17, 1, 511, 128, 0, 64]
    parents = [random_tree(n, g) for n in (1, 5, 0, 30, 7, 1, 12, 70)]
    parents[4][3] = -2                                   # padded tokens, with what descends from them
    parents[6] = [-2] * 12                               # a tree of nothing
    check_attention(q, Trees(ctx, parents, 8, 2, dim, page, DTYPES[dtype], seed=1, extra_rows=3))


@pytest.mark.parametrize("kv_heads,group,nodes,ctx", [
    (3, 2, [4, 4], [1200, 700]),                         # heads that share a run
    (7, 1, [3], [2000]),
    (16, 3, [2, 5], [900, 30]),                          # more heads than a group takes
    (2, 8, [40, 37, 40], [500, 900, 0]),                 # trees of three M tiles: a CTA for each
    (2, 8, [64] + [1] * 30, [300] + [400] * 30),         # sizes too different for that: M tiles by themselves
    (1, 128, [5, 3], [1500, 100]),
    (1, 4, [128, 128], [3000, 5]),
])
@pytest.mark.parametrize("dim", [64, 256])
def test_attention_groups_of_heads_and_tiles(q, kv_heads, group, nodes, ctx, dim):
    g = gen(sum(nodes))
    check_attention(q, Trees(ctx, [random_tree(n, g) for n in nodes], kv_heads * group, kv_heads, dim, 16, torch.float16, seed=len(nodes)))


def test_attention_infinities_in_a_tree_of_several_tiles_and_parts(q):
    """The same as above for a tree whose rows and keys are spread over many CTAs."""
    n, D = 100, 256
    tree = [i - 2 if i > 1 else -1 for i in range(n)]    # two chains: odd tokens do not see even ones
    t = Trees([1500], [tree], 4, 2, D, 64, torch.bfloat16, seed=4)
    clean, clean_lse = run_attention(q, t)
    t.v_new[10, 0, 7], t.v_new[70, 1, 200] = float("inf"), float("nan")
    out, lse = run_attention(q, t)
    assert torch.equal(out[1::2], clean[1::2]) and torch.equal(lse, clean_lse)
    assert torch.equal(out[:10], clean[:10])
    assert bool((out[10::2, :2, 7] == float("inf")).all()) and bool(out[70::2, 2:, 200].isnan().all())
    same = torch.ones(n, 4, D, dtype=torch.bool)
    same[10::2, :2, 7], same[70::2, 2:, 200] = False, False
    assert torch.equal(out[same], clean[same])
    q.qhl_sync()


def test_attention_more_trees_than_a_cta_plans_for_itself(q):
    g = gen(9)
    ctx = [2500] + torch.randint(0, 40, (270,), generator=g).tolist() + [1100, 0]
    trees = [random_tree(6, g)] + [[-1]] * 270 + [random_tree(30, g), []]
    check_attention(q, Trees(ctx, trees, 8, 1, 64, 32, torch.bfloat16, seed=3))


def test_attention_many_sequences(q):
    g = gen(6)
    ctx = torch.randint(0, 90, (300,), generator=g).tolist()
    check_attention(q, Trees(ctx, [random_tree(1 + i % 3, g) for i in range(300)], 4, 2, 64, 16, torch.float16, seed=2))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_long_context_split_over_the_sms(q, dtype):
    check_attention(q, Trees([9001, 20], [random_tree(9, gen(1)), [-1]], 4, 2, 256, 64, DTYPES[dtype], seed=8))


@pytest.mark.parametrize("dim", [64, 256])
def test_attention_maxima_that_rise_from_tile_to_tile(q, dim):
    """Scores whose maximum grows by more than the rescaling threshold many times, down to weights that vanish."""
    t = Trees([1000], [[-1, 0, 0]], 2, 1, dim, 64, torch.float16, seed=3)
    t.q[:] = t.q.sign()
    ramp = torch.linspace(-30, 60, 1000)[:, None, None] / dim ** 0.5
    t.K[0] = (t.q[0, 0].sign().float() * ramp * torch.ones(1000, 1, dim)).half()
    s = int(t.seqs[0])
    for j in range(-(-1000 // 64)):
        m = min(64, 1000 - 64 * j)
        t.k[0, int(t.table[s, j]), :, :m] = t.K[0][64 * j:64 * j + m].transpose(0, 1)
    check_attention(q, t)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 256])
def test_attention_hidden_infinities_stay_hidden(q, dtype, dim):
    """A drafted token with infinities and NaN in k and v changes the tokens that see it, and no others."""
    tree = [-1, 0, 0, 1, 2, -1]                          # tokens 1 and 3 descend through 1; 2, 4, 5 do not see 1
    t = Trees([70], [tree], 4, 2, dim, 64, DTYPES[dtype], seed=4)
    clean, clean_lse = run_attention(q, t)
    t.v_new[1, 0, 3], t.v_new[1, 1, dim - 1], t.v_new[1, 0, 5] = float("inf"), float("nan"), -float("inf")
    out, lse = run_attention(q, t)
    hidden = [0, 2, 4, 5]
    assert torch.equal(out[hidden], clean[hidden]) and torch.equal(lse, clean_lse)
    for i in (1, 3):
        assert bool((out[i, :2, 3] == float("inf")).all()) and bool((out[i, :2, 5] == -float("inf")).all())
        assert bool(out[i, 2:, dim - 1].isnan().all())
        same = torch.ones(4, dim, dtype=torch.bool)
        same[:2, [3, 5]], same[2:, dim - 1] = False, False
        assert torch.equal(out[i][same], clean[i][same])
    t.k_new[1, 0, 2] = float("nan")
    out, lse = run_attention(q, t)
    assert torch.equal(out[hidden], clean[hidden]) and torch.equal(lse[hidden], clean_lse[hidden])
    assert bool(out[[1, 3], :2].isnan().all()) and bool(lse[[1, 3], :2].isnan().all())
    q.qhl_sync()


@pytest.mark.parametrize("ctx", [0, 40, 3000])
def test_attention_a_token_whose_own_key_is_nan(q, ctx):
    """NaN stays NaN where the parts of a token are joined, also from a part whose scores are all NaN."""
    t = Trees([ctx], [[-1, -1]], 2, 1, 256, 64, torch.float16, seed=4)
    clean, clean_lse = run_attention(q, t)
    t.k_new[1, 0, 9] = float("nan")
    out, lse = run_attention(q, t)
    assert torch.equal(out[0], clean[0]) and torch.equal(lse[0], clean_lse[0])
    assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
    q.qhl_sync()


def test_attention_padded_tokens_over_a_cache_with_infinities(q):
    t = Trees([100], [[-1, -2]], 2, 1, 256, 64, torch.bfloat16, seed=4)
    t.v[0, int(t.table[0, 0]), 0, 5, 7] = float("inf")
    out, lse = run_attention(q, t)
    assert bool((out[1] == 0).all()) and bool((lse[1] == -float("inf")).all())
    assert bool((out[0, :, 7] == float("inf")).all())


@pytest.mark.parametrize("layout", ["rows_heads", "contiguous_cache", "heads_outermost"])
def test_attention_cache_layouts(q, layout):
    t = Trees([333], [random_tree(4, gen(2))], 6, 2, 256, 32, torch.float16, seed=6, poison=0.0)
    ref = run_attention(q, t)
    order = {"rows_heads": (0, 1, 3, 2, 4), "contiguous_cache": (0, 2, 1, 3, 4), "heads_outermost": (2, 0, 3, 1, 4)}[layout]
    back = [order.index(i) for i in range(5)]
    put = lambda x: x.cuda().permute(*order).contiguous().permute(*back)   # noqa: E731
    kv = q.KvPages(put(t.k), put(t.v), t.table.cuda(), t.lens.cuda(), t.held.cuda(), t.refs.cuda())
    out = run_attention(q, t, kv=kv)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


def test_attention_layers_strided_rows_and_repeated_sequences(q):
    t = Trees([80, 80], [[-1, 0], [-1, 0]], 4, 2, 128, 16, torch.bfloat16, seed=6)
    ref, _ = run_attention(q, t)
    k = torch.stack([torch.full_like(t.k[0], float("nan")), t.k[0]]).cuda()
    v = torch.stack([torch.full_like(t.v[0], float("nan")), t.v[0]]).cuda()
    kv = q.KvPages(k, v, t.table.cuda(), t.lens.cuda(), t.held.cuda(), t.refs.cuda())
    wide = lambda x: torch.cat([x, torch.full_like(x[:, :1], float("nan"))], 1).cuda()[:, :x.shape[1]]   # noqa: E731
    out = torch.full((t.rows, 5, 128), 9.0, dtype=t.dtype, device="cuda")
    q.qhl_tree_attention(kv, 1, t.seqs.cuda(), t.q_start.cuda(), t.parent.cuda(), 2, wide(t.q), wide(t.k_new), wide(t.v_new), out[:, :4], scale=t.scale)
    assert torch.equal(out[:, :4].cpu(), ref) and bool((out[:, 4] == 9).all())
    # both trees over the same sequence
    seqs = t.seqs.clone()
    seqs[1] = seqs[0]
    a = run_attention(q, t)[0]
    t.seqs = seqs
    b = run_attention(q, t)[0]
    assert torch.equal(a[:2], b[:2])
    t.K[1], t.V[1] = t.K[0], t.V[0]
    check_attention(q, t)


def test_attention_is_the_same_alone_and_in_a_batch_of_the_same_split(q):
    """Two calls give the same bits: no result depends on the order in which CTAs end."""
    t = Trees([2500, 900], [random_tree(12, gen(1)), random_tree(5, gen(2))], 6, 2, 256, 64, torch.bfloat16, seed=9)
    a = run_attention(q, t)
    for _ in range(5):
        b = run_attention(q, t)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_bad_indices_are_reported_and_not_followed(q):
    t = Trees([200, 40], [[-1, 0], [-1]], 2, 1, 256, 64, torch.float16, seed=3)
    ref = run_attention(q, t)[0]
    q.qhl_sync()
    good = t.table.clone()
    s = int(t.seqs[0])
    for bad in (-1, int(t.refs.numel()), 2 ** 31 - 1):
        t.table[s, 1] = bad
        out = run_attention(q, t)[0]
        assert torch.equal(out[2], ref[2])               # the other sequence
        with pytest.raises(q.StageError) as e:
            q.qhl_sync()
        assert e.value.code == -7
    t.table = good
    for name, at, bad in (("seqs", 0, 2), ("seqs", 0, -1), ("parent", 1, 1), ("parent", 1, -3), ("lens", s, -1), ("lens", s, 10 ** 6), ("q_start", 1, 5)):
        kept = getattr(t, name).clone()
        getattr(t, name)[at] = bad
        out = run_attention(q, t)[0]
        if name != "q_start":
            assert torch.equal(out[2], ref[2])
        with pytest.raises(q.StageError):
            q.qhl_sync()
        setattr(t, name, kept)
    assert torch.equal(run_attention(q, t)[0], ref)
    q.qhl_sync()


def test_attention_on_another_stream_and_from_a_graph(q):
    """One captured graph serves lengths, trees and pages that change between replays; two graphs with a workspace
    each may run at once."""
    first = Trees([700, 90], [random_tree(7, gen(1)), random_tree(3, gen(2))], 6, 2, 256, 64, torch.float16, seed=1)
    other = Trees([120, 650], [random_tree(4, gen(3)), random_tree(6, gen(4))], 6, 2, 256, 64, torch.float16, seed=2)
    s = torch.cuda.Stream()
    want = [run_attention(q, t, stream=s) for t in (first, other)]
    pad = lambda x, n: torch.cat([x, torch.zeros((n - x.shape[0],) + x.shape[1:], dtype=x.dtype)])   # noqa: E731
    pages, width = max(first.refs.numel(), other.refs.numel()), max(first.table.shape[1], other.table.shape[1])

    def held(t):
        tab = torch.full((2, width), -1, dtype=torch.int32)
        tab[:, :t.table.shape[1]] = t.table
        return [pad(t.k[0], pages)[None], pad(t.v[0], pages)[None], tab, t.lens, t.held, pad(t.refs, pages), t.seqs, t.q_start, t.parent, t.q,
                t.k_new, t.v_new]

    graphs = []
    for _ in range(2):
        d = [x.cuda() for x in held(first)]
        kv = q.KvPages(*d[:6])
        out, lse = torch.zeros(10, 6, 256, dtype=torch.float16, device="cuda"), torch.zeros(10, 6, device="cuda")
        ws = torch.empty(q.qhl_tree_attention_workspace(kv, 6, 10, 2, 7), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.qhl_tree_attention(kv, 0, *d[6:9], 7, *d[9:12], out, lse=lse, scale=first.scale, workspace=ws)
        graphs.append((g, d, out, lse, ws))              # the graph's workspace lives as long as the graph
    g, d, out, lse, _ = graphs[0]
    for t, w in ((first, want[0]), (other, want[1]), (first, want[0])):
        for x, y in zip(d, held(t)):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), w[0]) and torch.equal(lse.cpu(), w[1])
    for x, y in zip(graphs[1][1], held(other)):
        x.copy_(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (g, *_), st in zip(graphs, streams):
        with torch.cuda.stream(st):
            for _ in range(20):
                g.replay()
    torch.cuda.synchronize()
    for (g, d, out, lse, _), w in zip(graphs, want):
        assert torch.equal(out.cpu(), w[0]) and torch.equal(lse.cpu(), w[1])
    q.qhl_sync()


def test_attention_pages_beyond_32_bits(q):
    """A pool of more than 2^31 elements, its last pages used."""
    n_pages, H, P, D = 33000, 4, 64, 256
    t = Trees([150], [[-1, 0]], 8, 4, D, P, torch.float16, seed=5, poison=0.0)
    k = torch.empty(1, n_pages, H, P, D, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 31
    table = t.table.clone()
    m = t.refs.numel()
    for p in range(m):
        k[0, n_pages - 1 - p], v[0, n_pages - 1 - p] = t.k[0, p].cuda(), t.v[0, p].cuda()
    table[table >= 0] = n_pages - 1 - table[table >= 0]
    kv = q.KvPages(k, v, table.cuda(), t.lens.cuda(), t.held.cuda(), torch.zeros(n_pages, dtype=torch.int32, device="cuda"))
    check_attention(q, t, kv=kv)


# -------------------------------------------------------------- a verify step

def test_a_verify_step_with_all_operators(q):
    """Two decoding steps of a batch, each: in-projection rows -> norm and rotation -> attention over a draft tree -> the
    accepted path committed; the second step over pages that a fork shares.  Held against one long attention over all
    accepted rows, and a branch against its own history."""
    Hq, H, D, P, L = 6, 2, 64, 16, 2
    dt, theta = torch.bfloat16, 1e4
    g = gen(12)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    n_pages = 16
    kv = q.KvPages(torch.full((L, n_pages, H, P, D), float("nan"), dtype=dt, device="cuda"),
                   torch.full((L, n_pages, H, P, D), float("nan"), dtype=dt, device="cuda"), i32([[-1] * 6] * 4), i32([0] * 4), i32([0] * 4),
                   i32([0] * n_pages))
    gq, gk = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
    width = 2 * Hq * D + 2 * H * D
    history = {0: [], 1: [], 2: []}                      # accepted (k, v) rows of each sequence, per layer

    def step(seqs, trees, paths):
        starts = np.cumsum([0] + [len(t) for t in trees]).tolist()
        n = starts[-1]
        lens = [len(history[s]) for s in seqs]
        status = i32([0] * len(seqs))
        q.qhl_pages_extend(kv, i32(seqs), i32([len(t) for t in trees]), status)
        assert status.tolist() == [0] * len(seqs)
        pos = [lens[b] + len(vh.lineage(t, i)) - 1 for b, t in enumerate(trees) for i in range(len(t))]
        k_new, v_new = (torch.zeros(L, n, H, D, dtype=dt, device="cuda") for _ in range(2))
        for layer in range(L):
            y = torch.randn(n, width, generator=g).cuda()
            qq, out = torch.zeros(n, Hq, D, dtype=dt, device="cuda"), torch.zeros(n, Hq, D, dtype=dt, device="cuda")
            q.qhl_qk_norm_rope(Hq, H, D, D, theta, 1e-6, y, i32(pos), gq, gk, qq, k_new[layer], v_new[layer])
            q.qhl_tree_attention(kv, layer, i32(seqs), i32(starts), i32(sum(trees, [])), max(map(len, trees)), qq, k_new[layer], v_new[layer], out)
            for b, t in enumerate(trees):
                for i in range(len(t)):
                    rows = [starts[b] + x for x in vh.lineage(t, i)[::-1]]
                    K = torch.stack([r[layer][0] for r in history[seqs[b]]] + [k_new[layer, r] for r in rows]).cpu().double()
                    V = torch.stack([r[layer][1] for r in history[seqs[b]]] + [v_new[layer, r] for r in rows]).cpu().double()
                    for j in range(Hq):
                        w = torch.softmax(K[:, j // 3] @ qq[starts[b] + i, j].cpu().double() / D ** 0.5, 0)
                        ref, A = w @ V[:, j // 3], w @ V[:, j // 3].abs()
                        # u for the result, u for each weight, and the f32 parts (see Trees.reference)
                        assert bool(((out[starts[b] + i, j].cpu().double() - ref).abs() <= half_step(dt) * ref.abs() + A * (1.01 * half_step(dt) + 2.0 ** -10)).all())
        most = max(map(len, paths))
        q.qhl_pages_commit(kv, i32(seqs), i32(starts), i32([p + [-1] * (most - len(p)) for p in paths]), i32([len(p) for p in paths]), i32(lens), k_new,
                           v_new, status)
        assert status.tolist() == [0] * len(seqs)
        for b, s in enumerate(seqs):
            history[s] = history[s] + [[(k_new[x, starts[b] + i], v_new[x, starts[b] + i]) for x in range(L)] for i in paths[b]]

    step([0, 1], [[-1, 0, 0, 2, 3], list(range(-1, 20))], [[0, 2, 3], list(range(19))])
    step([1, 0], [[-1], [-1, 0, 1]], [[0], [0, 1]])
    status = i32([9])
    q.qhl_pages_fork(kv, i32([1]), i32([2]), status)
    assert status.tolist() == [0]
    history[2] = list(history[1])
    step([2, 1], [[-1, -1, 1], [-1, 0]], [[1, 2], [0]])
    step([0, 2, 1], [[-1], [-1], [-1, 0, 0]], [[0], [], [0, 2]])
    assert kv.lens.tolist()[:3] == [len(history[s]) for s in range(3)]
    q.qhl_pages_free(kv, i32([0, 1, 2]), i32([0, 0, 0]))
    assert kv.refs.tolist() == [0] * n_pages
    q.qhl_sync()


def test_a_verify_step_captured_in_a_graph(q):
    """Every operator of a step in one graph, with scratch from the allocator, replayed with other inputs; and on a
    stream of its own."""
    Hq, H, D, P, L, n = 4, 2, 64, 16, 2, 5
    dt = torch.float16
    g = gen(21)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    width = 2 * Hq * D + 2 * H * D
    Hk, Hv = 2, 2

    def fresh(seed):
        g = gen(seed)
        r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
        table = torch.full((3, 5), -1, dtype=torch.int32)
        table[0, :3], table[1, :2] = torch.tensor([4, 1, 7]), torch.tensor([0, 6])
        refs = torch.zeros(14, dtype=torch.int32)
        refs[[4, 1, 7, 0, 6]] = 1
        k = torch.full((L, 14, H, P, D), float("nan")).to(dt)
        v = k.clone()
        for p in (4, 1, 7, 0, 6):
            k[:, p], v[:, p] = r(L, H, P, D).to(dt), r(L, H, P, D).to(dt)
        dn = r(n, 2 * Hk * 128 + Hv * 128 + 2 * Hv)
        return dict(k=k, v=v, table=table, lens=torch.tensor([35 + seed % 5, 30, 0], dtype=torch.int32), held=torch.tensor([3, 2, 0], dtype=torch.int32),
                    refs=refs, at=torch.tensor([35 + seed % 5, 30], dtype=torch.int32), y=r(L, n, width), dn=dn, states=0.1 * r(2, Hv, 128, 128))

    seqs, starts, parent = i32([2, 1]), i32([0, 3, 5]), i32([-1, 0, 0, -1, 0])
    path, acc = i32([[0, 2], [0, 1]]), i32([2, 2])

    def make(d):
        kv = q.KvPages(d["k"], d["v"], d["table"], d["lens"], d["held"], d["refs"])
        o = dict(status=i32([9, 9]), st=i32([9]), qq=torch.zeros(L, n, Hq, D, dtype=dt, device="cuda"), kn=torch.zeros(L, n, H, D, dtype=dt, device="cuda"),
                 vn=torch.zeros(L, n, H, D, dtype=dt, device="cuda"), out=torch.zeros(L, n, Hq, D, dtype=dt, device="cuda"),
                 lse=torch.zeros(L, n, Hq, device="cuda"), snaps=torch.zeros(n, Hv, 128, 128, device="cuda"), o=torch.zeros(n, Hv * 128, device="cuda"),
                 pos=i32([0] * n), one=torch.ones(D, device="cuda"), zero=i32([0, 1]), src=i32([0]), dst=i32([2]), add=i32([3, 2]), kv=kv)
        return o

    def step(d, o, stream=None):
        q.qhl_pages_free(o["kv"], o["dst"], o["st"], stream=stream)
        q.qhl_pages_fork(o["kv"], o["src"], o["dst"], o["st"], stream=stream)
        q.qhl_pages_extend(o["kv"], seqs, o["add"], o["status"], stream=stream)
        for layer in range(L):
            q.qhl_qk_norm_rope(Hq, H, D, D, 1e4, 1e-6, d["y"][layer], o["pos"], o["one"], o["one"], o["qq"][layer], o["kn"][layer], o["vn"][layer], stream=stream)
            q.qhl_tree_attention(o["kv"], layer, seqs, starts, parent, 3, o["qq"][layer], o["kn"][layer], o["vn"][layer], o["out"][layer],
                                 lse=o["lse"][layer], stream=stream)
        q.qhl_deltanet_tree(Hk, Hv, d["dn"], starts, parent, 3, d["states"], o["zero"], o["snaps"], o["o"], stream=stream)
        q.qhl_pages_commit(o["kv"], seqs, starts, path, acc, d["at"], o["kn"], o["vn"], o["status"], stream=stream)

    def results(d, o):
        torch.cuda.synchronize()
        return [x.clone() for x in (d["table"], d["lens"], d["held"], d["refs"], o["status"], o["out"], o["lse"], o["snaps"], o["o"])] + [
            d["k"].nan_to_num(7.0), d["v"].nan_to_num(7.0)]

    def eager(seed, stream=None):
        d = {k: x.cuda() for k, x in fresh(seed).items()}
        o = make(d)
        torch.cuda.synchronize()
        step(d, o, stream=stream)
        return results(d, o)

    want = [eager(s) for s in (1, 2)]
    for s, w in zip((1, 2), want):
        assert w[4].tolist() == [0, 0]
        side = torch.cuda.Stream()
        for stream in (side, side.cuda_stream):
            assert all(torch.equal(a, b) for a, b in zip(eager(s, stream), w))
    d = {k: x.cuda() for k, x in fresh(1).items()}
    o = make(d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(d, o)
    for s, w in ((1, want[0]), (2, want[1]), (1, want[0])):
        for k, x in fresh(s).items():
            d[k].copy_(x)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(d, o), w))
    q.qhl_sync()
