"""A page table whose entries, summed over the rows, pass what the calls count
in 32 bits is refused on the host: a plan for 1024 rows of 2^21 pages and more
would take its free pages from behind a sum that has wrapped around (no GPU is
touched; the pointers are never dereferenced)."""
import ctypes
import os

import pytest

from sparse_decode_attention_head_gb300 import build_lib, sa

A = ctypes.c_void_p(1 << 20)
FAR = [ctypes.c_void_p((i + 2) << 40) for i in range(8)]      # further apart than any table


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sa.LIB_PATH):
        build_lib.build()
    return sa.lib()


def _prob(B, mpp):
    return sa.Problem(B=B, Hq=8, Hk=2, max_pages_per_seq=mpp, num_pages=128, sink=4, window=64, block_sizes=[16, 16],
                      k_per_head=[3] * 8, kcap=8)


@pytest.mark.parametrize("B,mpp", [(1024, 1 << 21), (1024, 1 << 20), (64, (1 << 26) - 1), (1 << 30, 1), (2 ** 31 - 1, 1), (65535, 1 << 15)])
def test_a_table_of_too_many_entries(lib, B, mpp):
    p, U = _prob(B, mpp), sa.SA_ERR_UNSUPPORTED
    assert lib.sa_rows_workspace_size(p.ref) == 0
    assert lib.sa_plan_pages(p.ref, FAR[0], A, A, A, FAR[1], A, A, A, A, None) == U
    assert lib.sa_compact_pages(p.ref, FAR[0], A, FAR[1], A, A, A, A, None) == U
    assert lib.sa_copy_pages(p.ref, A, A, A, A, A, 4, A, None) == U
    assert lib.sa_accept_rows(p.ref, A, A, A, A, A, 4, A, A, None) == U
    assert lib.sa_prompt_attention(p.ref, 4, FAR[0], A, A, A, A, A, FAR[1], None, A, None) == U
    assert lib.sa_tree_attention(p.ref, 4, FAR[0], A, A, A, A, A, A, FAR[1], None, A, None) == U
    assert lib.sa_qk_norm_rope(p.ref, 4, FAR[0], 1024, FAR[1], 256, FAR[2], 256, None, None, 0.0, None, None, None, A, A, A,
                               FAR[3], FAR[4], FAR[5], A, None) == U


def test_a_large_table_is_taken(lib):
    for B, mpp in ((1024, (1 << 20) - 1), (15, (1 << 26) - 1), ((1 << 30) - 1, 1)):
        p = _prob(B, mpp)
        assert lib.sa_rows_workspace_size(p.ref) > 0
        assert lib.sa_copy_pages(p.ref, A, A, A, A, A, 0, A, None) == sa.SA_OK
        assert lib.sa_prompt_attention(p.ref, 0, None, A, A, A, A, A, None, None, A, None) == sa.SA_OK
