"""Refusals of the tree-verification operators, before any device work: the C
calls' argument checks, the binding's, and the plain page operations that the
GPU tests compare with."""
import ctypes
import os
import re

import pytest
import torch

from verify_helpers import E_ARG, E_OOM, E_STATE, OK, Pages


@pytest.fixture(scope="module")
def q():
    from quantized_hybrid_layer_b200 import build as b
    b.build()
    import quantized_hybrid_layer_b200 as q
    return q


def cache(q, **over):
    f = dict(k_dev=1 << 20, v_dev=1 << 21, dtype=q.QHL_F16, n_layers=2, n_pages=8, kv_heads=4, page_rows=64, dim=256,
             stride_layer=8 * 4 * 64 * 256, stride_page=4 * 64 * 256, stride_head=64 * 256, stride_row=256, n_seqs=4, max_pages=8,
             table_dev=1 << 12, len_dev=1 << 12, held_dev=1 << 12, refs_dev=1 << 12)
    f.update(over)
    return q.KvPagesStruct(**f)


BAD_CACHES = [dict(k_dev=0), dict(v_dev=None), dict(refs_dev=0), dict(dtype=0), dict(dtype=3), dict(dim=96), dict(page_rows=24),
              dict(page_rows=512), dict(n_layers=0), dict(n_pages=0), dict(kv_heads=0), dict(kv_heads=257), dict(n_seqs=0),
              dict(max_pages=0), dict(k_dev=(1 << 20) + 8), dict(stride_row=252), dict(stride_row=128), dict(stride_head=0),
              dict(stride_page=4), dict(stride_layer=4), dict(stride_layer=0), dict(stride_page=1 << 50)]


def tree_call(q, kv, layer=0, hq=24, rows=4, batch=1, nodes=4, qp=16, stride=24 * 256, new=4 * 256, scale=0.1, ws=16, nbytes=1 << 40):
    return q.lib().qhl_tree_attention(ctypes.byref(kv) if kv is not None else None, layer, hq, rows, batch, nodes, 16, 16, 16, qp, stride,
                                      16, 16, new, 16, stride, None, scale, ws, nbytes, None)


@pytest.mark.parametrize("over", BAD_CACHES)
def test_caches_that_the_kernels_cannot_use_are_refused(q, over):
    kv, lib = cache(q, **over), q.lib()
    want = -6 if set(over) <= {"dtype", "dim", "page_rows"} else -1
    p = ctypes.byref(kv)
    assert tree_call(q, kv) == want
    assert lib.qhl_pages_free(p, 1, 16, 16, None) == want
    assert lib.qhl_pages_fork(p, 1, 16, 16, 16, None) == want
    assert lib.qhl_pages_extend(p, 1, 16, 16, 16, 16, 16, None) == want
    assert lib.qhl_pages_commit(p, 1, 4, 16, 16, 16, 4, 16, 16, 16, 16, 4096, 1024, 16, None) == want
    assert lib.qhl_tree_attention_workspace(p, 24, 4, 1, 4) == 0
    assert lib.qhl_last_error()


@pytest.mark.parametrize("over", [dict(layer=-1), dict(layer=2), dict(hq=0), dict(hq=23), dict(hq=4 * 129), dict(rows=-1), dict(batch=0),
                                  dict(batch=2049), dict(nodes=0), dict(nodes=129), dict(qp=0), dict(qp=24), dict(stride=24 * 256 - 8),
                                  dict(stride=24 * 256 + 4), dict(new=1016), dict(new=1028), dict(scale=0.0), dict(scale=-1.0),
                                  dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=0), dict(ws=24)])
def test_tree_attention_refuses_bad_arguments(q, over):
    assert tree_call(q, cache(q), **over) == -1
    assert b"qhl_tree_attention" in q.lib().qhl_last_error()


def test_null_caches_are_refused(q):
    lib = q.lib()
    assert tree_call(q, None) == -1
    assert lib.qhl_pages_free(None, 1, 16, 16, None) == -1
    assert lib.qhl_tree_attention_workspace(None, 24, 4, 1, 4) == 0


def test_page_calls_refuse_bad_arguments(q):
    kv, lib = cache(q), q.lib()
    p = ctypes.byref(kv)
    for n in (0, -1, 1025):
        assert lib.qhl_pages_free(p, n, 16, 16, None) == -1
        assert lib.qhl_pages_fork(p, n, 16, 16, 16, None) == -1
        assert lib.qhl_pages_extend(p, n, 16, 16, 16, 16, 1 << 20, None) == -1
        assert lib.qhl_pages_commit(p, n, 4, 16, 16, 16, 4, 16, 16, 16, 16, 4096, 1024, 16, None) == -1
    assert lib.qhl_pages_free(p, 1, None, 16, None) == -1
    assert lib.qhl_pages_fork(p, 1, 16, None, 16, None) == -1
    assert lib.qhl_pages_commit(p, 1, 4, 16, 16, None, 4, 16, 16, 16, 16, 4096, 1024, 16, None) == -1
    assert lib.qhl_pages_commit(p, 1, 4, 16, 16, 16, 0, 16, 16, 16, 16, 4096, 1024, 16, None) == -1      # path_stride
    assert lib.qhl_pages_commit(p, 1, 4, 16, 16, 16, 4, 16, 16, 24, 16, 4096, 1024, 16, None) == -1      # k_new misaligned
    assert lib.qhl_pages_commit(p, 1, 4, 16, 16, 16, 4, 16, 16, 16, 16, 4096, 1016, 16, None) == -1      # rows too short
    assert lib.qhl_pages_commit(p, 1, 4, 16, 16, 16, 4, 16, 16, 16, 16, 512, 1024, 16, None) == -1       # layers overlap


def norm_call(q, hq=24, hkv=4, dim=256, rope=64, theta=1e7, eps=1e-6, y=16, yt=0, ys=14336, off=(0, 12288, 13312), n=1, dt=1, out=16, qs=6144):
    return q.lib().qhl_qk_norm_rope(hq, hkv, dim, rope, theta, eps, y, yt, ys, *off, n, 16, 16, 16, dt, out, qs, 16, 1024, 16, 1024, None)


@pytest.mark.parametrize("over,want", [(dict(hq=0), -1), (dict(hkv=0), -1), (dict(dim=96), -6), (dict(rope=60), -1), (dict(rope=264), -1),
                                       (dict(rope=-8), -1), (dict(theta=0.0), -1), (dict(theta=float("nan")), -1), (dict(eps=-1.0), -1),
                                       (dict(eps=float("nan")), -1), (dict(y=0), -1), (dict(y=20), -1), (dict(yt=3), -6), (dict(dt=0), -6),
                                       (dict(ys=14338), -1), (dict(off=(0, 12290, 13312)), -1), (dict(off=(0, 12288, 13316)), -1),
                                       (dict(off=(-8, 12288, 13312)), -1), (dict(n=-1), -1), (dict(out=8), -1), (dict(qs=6136), -1),
                                       (dict(qs=6148), -1)])
def test_norm_rope_refuses_bad_arguments(q, over, want):
    assert norm_call(q, **over) == want
    assert b"qhl_qk_norm_rope" in q.lib().qhl_last_error()


def test_norm_rope_of_no_rows_does_nothing(q):
    assert norm_call(q, n=0) == 0


def dn_call(q, hk=16, hv=48, y=16, n=4, batch=1, nodes=4, st=1 << 40, ns=2, sn=1 << 30, o=16):
    return q.lib().qhl_deltanet_tree(hk, hv, y, n, batch, nodes, 16, 16, st, ns, 16, sn, o, None)


@pytest.mark.parametrize("over,want", [(dict(hk=0), -1), (dict(hv=47), -1), (dict(y=0), -1), (dict(y=20), -1), (dict(st=0), -1),
                                       (dict(o=8), -1), (dict(n=-1), -1), (dict(batch=0), -1), (dict(batch=2049), -1), (dict(nodes=0), -1),
                                       (dict(nodes=129), -1), (dict(ns=0), -1), (dict(hk=1, hv=1), -6), (dict(sn=1 << 40), -1),
                                       (dict(sn=(1 << 40) - 48 * 65536), -1)])
def test_deltanet_tree_refuses_bad_arguments(q, over, want):
    assert dn_call(q, **over) == want
    assert b"qhl_deltanet_tree" in q.lib().qhl_last_error()


def test_the_binding_refuses_wrong_tensors(q):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)   # noqa: E731
    k = torch.zeros(1, 4, 2, 16, 64, dtype=torch.float16)
    good = (k, k.clone(), i32(3, 2), i32(3), i32(3), i32(4))
    kv = q.KvPages(*good)
    for at, t in ((1, k.float()), (1, k[:, :2]), (0, k.transpose(3, 4)), (2, i32(3)), (2, i32(3, 2).long()), (3, i32(2)), (4, i32(4)),
                  (5, i32(3)), (2, i32(3, 4)[:, ::2])):
        with pytest.raises(ValueError):
            q.KvPages(*(good[:at] + (t,) + good[at + 1:]))
    x, n = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, 2, 64, dtype=torch.float16)
    call = lambda **o: q.qhl_tree_attention(**{**dict(kv=kv, layer=0, seqs=i32(1), q_start=i32(2), parent=i32(2), max_nodes=2, q=x,   # noqa: E731
                                                      k_new=n, v_new=n, out=x.clone()), **o})
    for o in (dict(q=x.bfloat16()), dict(q=x.transpose(0, 1)), dict(k_new=x), dict(out=x[:1]), dict(lse=torch.zeros(2, 2)), dict(parent=i32(3)),
              dict(q_start=i32(1)), dict(seqs=torch.zeros(1)), dict()):       # the last: everything right, but on the CPU
        with pytest.raises(ValueError):
            call(**o)
    with pytest.raises(ValueError):
        q.qhl_pages_free(kv, i32(1), i32(2))
    with pytest.raises(ValueError):
        q.qhl_qk_norm_rope(4, 2, 64, 64, 1e4, 1e-6, torch.zeros(2, 100), i32(2), torch.ones(64), torch.ones(64), x, n, n.clone())
    with pytest.raises(ValueError):
        q.qhl_deltanet_tree(4, 4, torch.zeros(2, 10), i32(2), i32(2), 2, torch.zeros(1, 4, 128, 128), i32(1), torch.zeros(2, 4, 128, 128),
                            torch.zeros(2, 512))


def test_plain_page_operations():
    p = Pages(6, 4, 4, 4)
    assert p.extend([0], [6]) == [OK] and p.rows[0] == [0, 1]
    p.lens[0] = 6
    # a src that is a dst of the call, a dst named again, a number out of range
    assert p.fork([0, 1, 0, 9], [1, 2, 1, 3]) == [OK, E_ARG, E_ARG, E_ARG]
    assert p.fork([0, 0], [2, 1]) == [OK, E_STATE]
    assert p.refs == [3, 3, 0, 0, 0, 0]
    # two of the three holders of page 1 ask: both copy; then the last keeps it
    assert p.extend([1, 2], [1, 3]) == [OK, OK]
    assert p.copies == [(1, 2, 2), (1, 3, 2)] and p.rows[1] == [0, 2] and p.rows[2] == [0, 3, 4]
    assert p.refs == [3, 1, 1, 1, 1, 0]
    assert p.extend([0, 1, 2], [7, 3, 0]) == [E_OOM, E_OOM, OK]
    assert p.extend([0, 0, 3, 3], [99, 1, -1, 0]) == [E_ARG, E_ARG, E_ARG, E_ARG]
    assert p.free([2, 2, 7]) == [OK, E_ARG, E_ARG]
    assert p.refs == [2, 1, 1, 0, 0, 0]


def test_kernels_that_start_before_their_predecessor_ends_use_coherent_loads():
    """A non-coherent load (__ldg, ld.global.nc) promises that its data does not change while the kernel runs; these kernels
    run beside the one that writes their inputs until they have waited for it."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_hybrid_layer_b200", "csrc")
    for name in ("norm_rope.cu", "tree_attention.cu", "deltanet_tree.cu", "pages.cu", "verify.cuh"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        assert not re.search(r"__ldg\b|\.nc\b|__restrict__", text), name
