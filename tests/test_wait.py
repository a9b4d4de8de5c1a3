"""The chunk kernel's bounded wait: limited by the GPU's clock, not by a number of tries."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "paged_kv_cache_273_gb300")


def _build(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "wait_check")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(PKG, "csrc"), os.path.join(ROOT, "tests", "native", "wait_check.cu"), "-o", exe], check=True)
    return exe


def test_every_wait_of_the_chunk_kernel_is_limited_by_the_clock():
    with open(os.path.join(PKG, "csrc", "chunk.cu")) as f:
        src = f.read()
    # a try of its own is only the last one, of the MMAs under way, which looks at the clock too
    assert src.count("mbar_try_wait(") == src.count("while (!mbar_try_wait(drain, 0u) && globaltimer_ns()") == 1
    assert src.count("mbar_wait_or_abort(") == src.count("mbar_wait_bounded(") == 1


@pytest.mark.gpu
def test_gpu_wait_runs_out_and_returns(tmp_path):
    r = subprocess.run([_build(tmp_path)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout
