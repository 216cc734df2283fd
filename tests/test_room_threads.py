"""Two threads that share a Problem and call with different numbers of rows: each
is checked against the room that its own rows need."""
import os

import pytest
import torch

from sparse_decode_attention_head_gb300 import build_lib, sa
from tests.test_rows_abi import _prob


class _Other(dict):
    """A Problem's notes, into which another thread writes right behind every write of this one."""

    def __init__(self, theirs):
        super().__init__()
        self.theirs = theirs

    def __setitem__(self, key, value):
        super().__setitem__(key, value)
        super().__setitem__(key, self.theirs)


class _Room:
    def __init__(self, n, max_rows):
        self.buf, self.max_rows = torch.empty(n, dtype=torch.uint8), max_rows


@pytest.fixture(autouse=True)
def built():
    if not os.path.exists(sa.LIB_PATH):
        build_lib.build()


@pytest.mark.parametrize("size", ["sa_shared_workspace_size", "sa_sparse_workspace_size"])
def test_the_other_threads_rows_do_not_count(size):
    prob = _prob()
    need = int(getattr(sa.lib(), size)(prob.ref, 100))
    # the other thread asks for more: this one has room
    prob._room = _Other((5000, 1 << 40))
    sa._check_room(prob, _Room(need, 100), size, 100)
    # it asks for less: this one has none
    prob._room = _Other((1, 0))
    with pytest.raises(ValueError, match="max_rows"):
        sa._check_room(prob, _Room(need - 1, 100), size, 100)
    with pytest.raises(ValueError, match="max_rows"):
        sa._check_room(prob, _Room(need, 99), size, 100)


def test_asked_again_when_the_number_changes():
    prob = _prob()
    size = "sa_shared_workspace_size"
    for n in (100, 7, 100, 2000):
        need = int(sa.lib().sa_shared_workspace_size(prob.ref, n))
        for _ in range(2):
            sa._check_room(prob, _Room(need, n), size, n)
            with pytest.raises(ValueError, match="max_rows"):
                sa._check_room(prob, _Room(need - 1, n), size, n)
