"""The packed-row and page calls check their arguments on the host, before any
launch (no GPU is touched; the pointers are never dereferenced)."""
import ctypes
import os

import pytest
import torch

from sparse_decode_attention_head_gb300 import build_lib, sa

A, M = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4)
FAR = [ctypes.c_void_p((i + 2) << 32) for i in range(8)]      # addresses far from one another
BAD, UNSUP = sa.SA_ERR_INVALID_ARG, sa.SA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sa.LIB_PATH):
        build_lib.build()
    return sa.lib()


def _prob(**kw):
    base = dict(B=2, Hq=8, Hk=2, max_pages_per_seq=64, num_pages=128, sink=4, window=64,
                block_sizes=[16, 16], k_per_head=[3] * 8, kcap=8)
    base.update(kw)
    return sa.Problem(**base)


def _rope(pairs=(64,), layout=0, axes=None):
    c = sa._Rope(layout, len(pairs) if axes is None else axes, (ctypes.c_int32 * 4)(*pairs))
    return c


def _rotate(lib, p, n=4, q=FAR[0], qs=1024, k=FAR[1], ks=256, v=FAR[2], vs=256, qw=None, kw=None, eps=1e-6, rope=None,
            freq=A, pos=None, off=A, lens=A, table=A, q_out=FAR[3], kp=FAR[4], vp=FAR[5], ws=A):
    return lib.sa_qk_norm_rope(p.ref, n, q, qs, k, ks, v, vs, qw, kw, eps, None if rope is None else ctypes.byref(rope),
                               freq, pos, off, lens, table, q_out, kp, vp, ws, None)


def test_workspace_size(lib):
    assert lib.sa_rows_workspace_size(_prob().ref) > 0
    assert lib.sa_rows_workspace_size(_prob(num_pages=1 << 22).ref) >= 16 << 22     # four counts a page
    assert lib.sa_rows_workspace_size(_prob(D=64).ref) == 0
    assert lib.sa_rows_workspace_size(None) == 0


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(q=None), dict(k=None), dict(v=None), dict(off=None), dict(lens=None), dict(table=None),
    dict(q_out=None), dict(kp=None), dict(vp=None), dict(ws=None), dict(q=M), dict(k=M), dict(v=M), dict(q_out=M),
    dict(kp=M), dict(vp=M), dict(ws=M), dict(qw=M), dict(kw=M), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(qs=1020), dict(qs=1016), dict(ks=248), dict(vs=0),
    dict(q=FAR[3], qs=2048),                                  # q_out over a strided q
    dict(k=FAR[3]),                                           # q_out over k
    dict(rope=_rope((64,)), freq=None), dict(rope=_rope((64,), layout=2)), dict(rope=_rope((64, 8))),
    dict(rope=_rope((-8, 16))), dict(rope=_rope((0,))), dict(rope=_rope((64,), axes=0)), dict(rope=_rope((64,), axes=5)),
])
def test_rotation_refusals(lib, kw):
    assert _rotate(lib, _prob(), **kw) == BAD


def test_rotation_limits(lib):
    p = _prob()
    assert _rotate(lib, p, rope=_rope((20,))) == UNSUP             # pairs not a multiple of 8
    assert _rotate(lib, _prob(D=64)) == BAD
    assert _rotate(lib, p, n=0, q=None, k=None, v=None, q_out=None) == sa.SA_OK
    assert _rotate(lib, p, n=0, rope=_rope((20,))) == UNSUP        # settings are checked without rows too


def _attend(lib, p, tree=None, n=4, q=FAR[0], kp=A, vp=A, table=A, lens=A, off=A, out=FAR[1], ws=A, words=A):
    if tree:
        return lib.sa_tree_attention(p.ref, n, q, kp, vp, table, lens, off, words, out, None, ws, None)
    return lib.sa_prompt_attention(p.ref, n, q, kp, vp, table, lens, off, out, None, ws, None)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(q=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None), dict(off=None),
    dict(out=None), dict(ws=None), dict(q=M), dict(kp=M), dict(vp=M), dict(out=M), dict(ws=M), dict(out=FAR[0]),
    dict(out=ctypes.c_void_p(FAR[0].value + 4096))])
def test_attention_refusals(lib, kw, tree):
    assert _attend(lib, _prob(), tree, **kw) == BAD


def test_attention_limits(lib):
    assert _attend(lib, _prob(), True, words=None) == BAD
    assert _attend(lib, _prob(D=64)) == BAD
    assert _attend(lib, _prob(page_size=32)) == UNSUP
    assert _attend(lib, _prob(Hq=32, k_per_head=[1] * 32)) == UNSUP         # 16 query heads a KV head
    for tree in (False, True):
        assert _attend(lib, _prob(), tree, n=0, q=None, out=None, words=None) == sa.SA_OK


def test_page_call_refusals(lib):
    p = _prob()
    far, n = FAR[6], None
    plan, pack, copy, acc = lib.sa_plan_pages, lib.sa_compact_pages, lib.sa_copy_pages, lib.sa_accept_rows
    full = [A, A, A, A, far, A, A, A, A]
    for i in range(9):
        args = list(full)
        args[i] = n
        assert plan(p.ref, *args, None) == BAD, i
    assert plan(p.ref, A, A, A, A, A, A, A, A, A, None) == BAD                # table_out is table_in
    assert plan(p.ref, A, A, A, A, ctypes.c_void_p(A.value + 256), A, A, A, A, None) == BAD   # they overlap
    assert plan(p.ref, *full[:8], M, None) == BAD
    big = _prob(B=1025)
    assert plan(big.ref, *full, None) == UNSUP
    full = [A, A, far, A, A, A, A]
    for i in range(7):
        args = list(full)
        args[i] = n
        assert pack(p.ref, *args, None) == BAD, i
    assert pack(p.ref, A, A, A, A, A, A, A, None) == BAD
    for i in (0, 1, 2, 3, 4, 6):
        args = [A, A, A, A, A, 4, A]
        args[i] = n
        assert copy(p.ref, *args, None) == BAD, i
    assert copy(p.ref, M, A, A, A, A, 4, A, None) == BAD
    assert copy(p.ref, A, A, A, A, A, -1, A, None) == BAD
    assert copy(p.ref, A, A, A, A, A, 0, A, None) == sa.SA_OK
    for i in (0, 1, 2, 3, 4, 6, 7):
        args = [A, A, A, A, A, 4, A, A]
        args[i] = n
        assert acc(p.ref, *args, None) == BAD, i
    assert acc(p.ref, A, A, A, A, A, 0, A, A, None) == BAD
    assert acc(p.ref, A, A, A, A, A, 65, A, A, None) == UNSUP
    assert acc(p.ref, A, M, A, A, A, 4, A, A, None) == BAD


def test_binding_refuses_host_tensors_and_a_small_workspace():
    p = _prob()
    t = torch.zeros(4)
    ws = object()
    for c in (lambda: sa.qk_norm_rope(p, t, t, t, t, t, t, t, t, t, ws),
              lambda: sa.prompt_attention(p, t, t, t, t, t, t, t, ws),
              lambda: sa.tree_attention(p, t, t, t, t, t, t, t, t, ws),
              lambda: sa.accept_rows(p, t, t, t, t, t, t, ws),
              lambda: sa.plan_pages(p, t, t, t, t, t, t, t, t, ws),
              lambda: sa.compact_pages(p, t, t, t, t, t, t, ws),
              lambda: sa.copy_pages(p, t, t, t, t, t, ws)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            c()
    with pytest.raises(ValueError):
        sa.Rope([])
    with pytest.raises(ValueError):
        sa.Rope([8] * 5)
    assert sa.Rope([16, 24, 24]).pairs == 64
