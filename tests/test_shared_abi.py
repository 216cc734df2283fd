"""sa_shared_prefixes and sa_shared_attention check their arguments on the host,
before any launch (no GPU is touched; the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests.test_rows_abi import A, BAD, FAR, M, UNSUP, _prob, lib  # noqa: F401


def test_workspace_size(lib):  # noqa: F811
    p = _prob()
    rows = lib.sa_rows_workspace_size(p.ref)
    assert lib.sa_shared_workspace_size(p.ref, 0) >= rows
    assert lib.sa_shared_workspace_size(p.ref, 1000) >= 51 << 20
    assert lib.sa_shared_workspace_size(p.ref, 100000) - lib.sa_shared_workspace_size(p.ref, 0) >= 2 * 100000 * 8 * 130 * 4
    assert lib.sa_shared_workspace_size(p.ref, 2 ** 31 - 1) > 2 ** 31 * 8 * 130 * 4      # in 64 bits
    assert lib.sa_shared_workspace_size(p.ref, -1) == 0
    assert lib.sa_shared_workspace_size(_prob(D=64).ref, 1) == 0
    assert lib.sa_shared_workspace_size(None, 1) == 0


def _attend(lib, p, n=4, q=FAR[0], kp=A, vp=A, table=A, lens=A, off=A, words=None, members=A, prefix=A, out=FAR[1], ws=A):  # noqa: F811
    return lib.sa_shared_attention(p.ref, n, q, kp, vp, table, lens, off, words, members, prefix, out, None, ws, None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(q=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None), dict(off=None),
    dict(members=None), dict(prefix=None), dict(out=None), dict(ws=None), dict(q=M), dict(kp=M), dict(vp=M), dict(out=M),
    dict(ws=M), dict(out=FAR[0]), dict(out=ctypes.c_void_p(FAR[0].value + 4096))])
def test_attention_refusals(lib, kw):  # noqa: F811
    assert _attend(lib, _prob(), **kw) == BAD


def test_attention_limits(lib):  # noqa: F811
    assert _attend(lib, _prob(D=64)) == BAD
    assert _attend(lib, _prob(page_size=32)) == UNSUP
    assert _attend(lib, _prob(Hq=32, k_per_head=[1] * 32)) == UNSUP
    assert _attend(lib, _prob(B=1 << 20, max_pages_per_seq=1 << 10)) == UNSUP      # a table of 2^30 entries
    assert _attend(lib, _prob(), n=0, q=None, out=None) == sa.SA_OK
    assert _attend(lib, _prob(), n=0, q=None, out=None, prefix=None) == BAD


def test_prefix_refusals(lib):  # noqa: F811
    f, p = lib.sa_shared_prefixes, _prob()
    full = [A, A, A, A, 1, 0, A, A, A]
    for i in (0, 1, 2, 3, 6, 7, 8):
        args = list(full)
        args[i] = None
        assert f(p.ref, *args, None) == BAD, i
    assert f(p.ref, A, A, A, A, -1, 0, A, A, A, None) == BAD
    assert f(p.ref, A, A, A, A, 3, 0, A, A, A, None) == BAD          # more groups than sequences
    assert f(p.ref, A, A, A, A, 1, 0, A, A, M, None) == BAD
    assert f(_prob(page_size=32).ref, *full, None) == UNSUP
    assert f(_prob(B=1 << 20, max_pages_per_seq=1 << 10).ref, *full, None) == UNSUP


def test_binding_refuses_host_tensors():
    p, t, ws = _prob(), torch.zeros(4), object()
    for c in (lambda: sa.shared_prefixes(p, t, t, t, t, t, t, ws),
              lambda: sa.shared_attention(p, t, t, t, t, t, t, t, t, t, ws)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            c()
