"""The 8-bit attention's unit spans on the host: tests/q8_spans_check.cu runs the
kernel's own walk for every CTA of many schedules and compares the spans it records,
which no wait precedes, with brute force; a merge refuses any other span."""
import os
import shutil
import subprocess

import pytest

from block_wise_diffusion_b200 import build

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "q8_spans_check.cu")


def test_spans_come_from_the_walk_alone(tmp_path):
    if shutil.which(build.NVCC) is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "q8_spans_check")
    subprocess.run([build.NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O1",
                    "-I", build.CSRC, SRC, "-o", exe], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "q8_spans: ok" in r.stdout, r.stdout + r.stderr


def test_spans_are_recorded_before_any_wait():
    """In the kernel with waits, by a lane that waits for nothing; the merge asks the
    rule before it uses a span."""
    text = open(os.path.join(build.CSRC, "tt_attn_q8.cu")).read()
    role = text[text.index("-- codes to shared memory"):]
    assert "if (lane == 1) put_spans(" in role[:role.index("mbar_wait")]
    merge = text[text.index("attn_q8_merge_kernel(const"):]
    assert merge.index("span_in_range(") < merge.index("uc.y - uc.x")
