"""Rows without candidates by their position (sa_select_rows): ahead of the
cache under the widest window, and behind sinks that reach over the table's end."""
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import sparse_ref as Z
from tests.test_gpu_select_rows import _check, _rows, _summaries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
@pytest.mark.parametrize("rows", [60, 1600])      # the form for few rows, and the one for many
@pytest.mark.parametrize("S", [0, 4, 2 ** 31 - 1])
def test_rows_without_a_position_under_the_widest_window(S, rows, mode):
    # the first 40 rows lie ahead of the cache: L - W of such a row is below the least int32
    r = _rows([rows, 3], [0, 900], 8, 2, seed=rows)
    r.lens[0] = rows - 40
    prob = Z.problem(r, 16, 6, S, 2 ** 31 - 1, mode=mode)
    idx, cnt = _check(r, prob, _summaries(prob, 1))
    assert bool((cnt == 0).all())


@pytest.mark.parametrize("rows", [60, 1600])
def test_sinks_behind_the_table(rows):
    # candidates begin behind the sinks, where the table has no blocks
    r = _rows([rows], [5000], 8, 2, seed=rows, mpp=64)
    prob = Z.problem(r, 16, 6, 4096, 64)
    idx, cnt = _check(r, prob, _summaries(prob, 2), status=sa.SA_ERR_CAPACITY)
    assert bool((cnt == 0).all())
    assert cnt.dtype == torch.int32
