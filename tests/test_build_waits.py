"""A kernel that waits for a copy has to look at whether it came: the build
refuses one that drops the answer of a bounded wait and goes on with the data."""
import os
import subprocess

import pytest

from sparse_decode_attention_head_gb300 import build_lib

SOURCE = """#include "sa_common.cuh"
__global__ void k(uint64_t* out, int* status) {
  __shared__ uint64_t bar;
  %s
  out[0] = bar;
}
"""


@pytest.mark.parametrize("wait,builds", [
    ("sa::mbar_wait_bounded(&bar, 0, status);", False),
    ("if (!sa::mbar_wait_bounded(&bar, 0, status)) return;", True),
    ("(void)sa::mbar_wait_bounded(&bar, 0, status);", True),      # at the end of a kernel, nothing is read behind it
])
def test_the_answer_of_a_wait_is_used(tmp_path, wait, builds):
    src = tmp_path / "wait.cu"
    src.write_text(SOURCE % wait)
    cmd = [build_lib.nvcc(), *build_lib._flags(), "-I", build_lib.CSRC, "-c", str(src), "-o", os.devnull]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert (r.returncode == 0) == builds, r.stderr
