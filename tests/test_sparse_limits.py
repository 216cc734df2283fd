"""Workspaces of the calls with selected blocks, and the limits that the header
states (no GPU is touched; the pointers are never dereferenced)."""
import pytest

from sparse_decode_attention_head_gb300 import sa
from tests.test_rows_abi import UNSUP, _prob, lib  # noqa: F401
from tests.test_sparse_abi import _attend, _select


def test_no_size_for_a_table_that_both_calls_refuse(lib):  # noqa: F811
    size = lib.sa_sparse_workspace_size
    wide, most = (_prob(B=1, max_pages_per_seq=n, block_sizes=[64, 64]) for n in (819201, 819200))
    assert size(wide.ref, 4) == 0 and size(wide.ref, 0) == 0
    assert _attend(lib, wide, n=0) == UNSUP and _select(lib, wide, n=0) == UNSUP
    # the attention takes this one, with lists of the caller's
    assert size(most.ref, 4) >= lib.sa_rows_workspace_size(most.ref) > 0
    assert _attend(lib, most, n=0) == sa.SA_OK and _select(lib, most, n=0) == UNSUP


def test_the_workspace_of_more_than_65536_slots_serves_the_attention(lib):  # noqa: F811
    # no scratch of the selection in it: a page more does not ask for less
    a, b = (lib.sa_sparse_workspace_size(_prob(B=1, max_pages_per_seq=n, block_sizes=[16, 16]).ref, 1000) for n in (65537, 100000))
    assert 0 < a <= b


@pytest.mark.parametrize("Hq,Hk", [(256, 64), (64, 64), (128, 64), (8, 2)])
def test_number_of_rows(lib, Hq, Hk):  # noqa: F811
    # 2^30 items of 32 / G rows under a KV head, each sequence's last one a part of that
    p = _prob(B=2, Hq=Hq, Hk=Hk, block_sizes=[16] * Hk, k_per_head=[1] * Hq)
    each = 32 // (Hq // Hk)
    most = min(2 ** 31 - 1, ((1 << 30) // Hk - 2) * each + each - 1)
    assert lib.sa_sparse_workspace_size(p.ref, most) > 0
    if most < 2 ** 31 - 1:
        assert lib.sa_sparse_workspace_size(p.ref, most + 1) == 0
        assert _select(lib, p, n=most + 1) == UNSUP
    assert (most < 2 ** 31 - 1) == (Hk == 64)
