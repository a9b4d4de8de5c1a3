"""The block-list decode kernel's shared-memory carve-up and index helpers,
checked on the host (see tests/native/blocks_layout_check.cu)."""
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_layout_fits_every_batch(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "blocks_layout_check")
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "paged_kv_cache_273_gb300", "csrc"),
                    "-o", exe, os.path.join(HERE, "native", "blocks_layout_check.cu")],
                   check=True, capture_output=True, timeout=600)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "blocks layout check: 0 bad" in r.stdout


def test_quotient_by_fp32_is_exact_below_its_limit():
    # the kernel's x / d for x < 2^20: fp32 (x + 1/2) / d with a quotient off by up to 2 steps
    g = np.random.default_rng(0)
    for d in list(range(1, 400)) + [511, 512, 513, 4095, 4096, 65535, 99991, 2 ** 20]:
        k = np.arange(0, 2 ** 20 // d + 1, max(1, 2 ** 20 // d // 500), dtype=np.int64) * d
        x = np.unique(np.concatenate([k, k - 1, k + 1, g.integers(0, 2 ** 20, 300),
                                      [0, 2 ** 20 - 1]]))
        x = x[(x >= 0) & (x < 2 ** 20)]
        q = (x.astype(np.float32) + np.float32(0.5)) / np.float32(d)
        for step in (-2, -1, 0, 1, 2):
            got = (q * (1 + np.float32(step) * np.float32(2.0 ** -23))).astype(np.int64)
            assert np.array_equal(got, x // d), d


def test_uneven_split_boundaries():
    # cut(c) = c (T / P) + c (T mod P) / P is floor(c T / P), and the CTA of a tile is found from
    # x / (T / P) downwards in few steps
    g = np.random.default_rng(1)
    for _ in range(300):
        P = int(g.integers(1, 153))
        T = int(g.integers(16 * P, 16 * P + int(10 ** g.uniform(1, 8.9))))
        TP, TR = T // P, T % P
        cut = [c * TP + c * TR // P for c in range(P + 1)]
        assert cut == [c * T // P for c in range(P + 1)]
        for x in [0, T - 1] + g.integers(0, T, 20).tolist() + [c for c in cut if c < T]:
            c, steps = min(P - 1, x // TP), 0
            while cut[c] > x:
                c, steps = c - 1, steps + 1
            assert cut[c] <= x < cut[c + 1] and steps <= P // 16 + 1
