"""The attention workspace's size, on the host: enough for every plan of the
sizes it was asked for and of smaller ones, with any window, and never less
for larger sizes."""
import ctypes
import os
import subprocess

import pytest

import nvfp4_quantized_dense_amd as nv

HERE = os.path.dirname(os.path.abspath(__file__))
LENS = [1, 500, 513, 2000, 8156, 8193, 30000, 131072, 648616]


def size(B, q, length, hq=40, h=8, d=128):
    return nv.nvfp4_kv_attention_workspace_bytes(B * q, B, hq, h, d, q, length)


@pytest.mark.parametrize("hq,h,d", [(64, 8, 128), (40, 8, 128), (171, 9, 128), (16, 4, 256), (32, 4, 64), (1, 1, 64)])
def test_size_grows(hq, h, d):
    for q in (1, 2, 5, 16, 64, 300, 1024):
        for length in LENS:
            row = [size(B, q, length, hq, h, d) for B in range(1, 300)]
            assert row == sorted(row), (q, length)
    for B in (1, 4, 65):
        for length in LENS:
            row = [size(B, q, length, hq, h, d) for q in range(1, 300)]
            assert row == sorted(row), (B, length)
        for q in (1, 5, 64, 1024):
            row = [size(B, q, length, hq, h, d) for length in range(1, 70000, 97)]
            assert row == sorted(row), (B, q)


def test_a_buffer_for_the_largest_serves_the_smaller():
    """Sizes between which the split count falls."""
    assert size(127, 1, 8192, 64) <= size(128, 1, 8192, 64) and size(1, 64, 8192, 64) <= size(1, 1024, 8192, 64)
    assert size(1, 16, 8156) <= size(1, 16, 8193)
    assert size(65, 1, 648616, 171, 9) <= size(65, 2, 648616, 171, 9)


@pytest.fixture(scope="module")
def scan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "attention_plan_scan.cpp")], check=True)
    return ctypes.CDLL(so).scan


@pytest.mark.parametrize("seed", range(4))
def test_plans_fit(scan, seed):
    at, tight = (ctypes.c_int64 * 7)(), ctypes.c_double()
    bad = scan(seed, 300000, at, ctypes.byref(tight))
    assert bad == 0, (bad, list(at))
    assert tight.value > 0.5  # the bound is not idle
