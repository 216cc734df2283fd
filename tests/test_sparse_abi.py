"""sa_select_rows and sa_sparse_row_attention check their arguments on the host,
before any launch (no GPU is touched; the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests.test_rows_abi import A, BAD, FAR, M, UNSUP, _prob, lib  # noqa: F401


def test_workspace_size(lib):  # noqa: F811
    p = _prob()
    assert lib.sa_sparse_workspace_size(p.ref, 0) >= lib.sa_rows_workspace_size(p.ref)
    assert lib.sa_sparse_workspace_size(p.ref, 100000) > 0
    assert lib.sa_sparse_workspace_size(p.ref, -1) == 0
    assert lib.sa_sparse_workspace_size(_prob(D=64).ref, 1) == 0
    assert lib.sa_sparse_workspace_size(None, 1) == 0
    big = _prob(Hq=512 // 2, Hk=64, block_sizes=[16] * 64, k_per_head=[1] * 256)
    assert lib.sa_sparse_workspace_size(big.ref, 2 ** 31 - 1) == 0       # more than 2^30 items


def _attend(lib, p, n=4, q=FAR[0], kp=A, vp=A, table=A, lens=A, off=A, idx=A, cnt=A, out=FAR[1], ws=A):  # noqa: F811
    return lib.sa_sparse_row_attention(p.ref, n, q, kp, vp, table, lens, off, idx, cnt, out, None, ws, None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(q=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None), dict(off=None),
    dict(idx=None), dict(cnt=None), dict(out=None), dict(ws=None), dict(q=M), dict(kp=M), dict(vp=M), dict(out=M),
    dict(ws=M), dict(out=FAR[0]), dict(out=ctypes.c_void_p(FAR[0].value + 4096))])
def test_attention_refusals(lib, kw):  # noqa: F811
    assert _attend(lib, _prob(), **kw) == BAD


def test_attention_limits(lib):  # noqa: F811
    assert _attend(lib, _prob(D=64)) == BAD
    assert _attend(lib, _prob(page_size=32)) == UNSUP
    assert _attend(lib, _prob(B=1, max_pages_per_seq=819201), n=0) == UNSUP
    assert _attend(lib, _prob(B=1, max_pages_per_seq=819200), n=0) == sa.SA_OK
    assert _attend(lib, _prob(B=1 << 20, max_pages_per_seq=1 << 10)) == UNSUP
    assert _attend(lib, _prob(), n=0, q=None, out=None) == sa.SA_OK


def _select(lib, p, n=4, q=A, summ=A, lens=A, off=A, idx=A, cnt=A, ws=A):  # noqa: F811
    return lib.sa_select_rows(p.ref, n, q, summ, lens, off, idx, cnt, ws, None)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(q=None), dict(summ=None), dict(lens=None), dict(off=None), dict(idx=None),
                                dict(cnt=None), dict(ws=None), dict(q=M), dict(summ=M), dict(ws=M)])
def test_selection_refusals(lib, kw):  # noqa: F811
    assert _select(lib, _prob(), **kw) == BAD


def test_selection_limits(lib):  # noqa: F811
    assert _select(lib, _prob(D=64)) == BAD
    assert _select(lib, _prob(k_per_head=[9] + [3] * 7)) == sa.SA_ERR_CAPACITY
    assert _select(lib, _prob(selection=sa.SELECT_GROUP, k_per_head=[1, 2, 1, 1, 1, 1, 1, 1])) == BAD
    assert _select(lib, _prob(), n=0, q=None, idx=None, cnt=None) == sa.SA_OK
    assert _select(lib, _prob(B=1, max_pages_per_seq=65536, block_sizes=[16, 64]), n=0) == sa.SA_OK
    assert _select(lib, _prob(B=1, max_pages_per_seq=65537, block_sizes=[16, 64]), n=0) == UNSUP      # 65537 block slots


def test_binding_refuses_host_tensors():
    p, t, ws = _prob(), torch.zeros(4), object()
    for c in (lambda: sa.select_rows(p, t, t, t, t, t, t, ws),
              lambda: sa.sparse_row_attention(p, t, t, t, t, t, t, t, t, t, ws)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            c()
