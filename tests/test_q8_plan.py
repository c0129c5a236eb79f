"""The plan of the 8-bit products, built for the host and checked over a grid of
shapes: variants that exist, partial sums inside the workspace, launch limits."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def faults():
    out = os.path.join(ROOT, "tests", "_build")
    os.makedirs(out, exist_ok=True)
    so = os.path.join(out, "libq8_plan_check.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                           "-I/opt/rocm/include", "-I",
                           os.path.join(ROOT, "quantization_error_compensation_amd", "csrc"),
                           os.path.join(ROOT, "tests", "q8_plan_check.cpp"), "-o", so])
    return ctypes.CDLL(so).q8_plan_faults


WIDTHS = (16, 48, 128, 144, 1024, 4096, 4112, 8192, 11008, 28672, 65536)
OUTS = (16, 32, 48, 256, 1024, 1040, 4096, 6144, 6160, 8192, 10240, 28672, 100000, 262144)
TOKENS = (1, 2, 8, 9, 16, 17, 32, 33, 48, 49, 64, 65, 100, 128, 129, 200, 257, 500, 777, 1024, 3000, 4096, 20000,
          1 << 17, 1 << 20)


@pytest.mark.parametrize("gated", [0, 1])
def test_every_plan_fits(faults, gated):
    for K in WIDTHS:
        for N in OUTS:
            for i, T in enumerate(TOKENS):
                if T * N > 1 << 37:  # refused
                    continue
                for largest in (T, TOKENS[min(i + 1, len(TOKENS) - 1)], 1 << 20):
                    assert faults(K, N, gated, T, largest) == 0, (K, N, gated, T, largest)


def test_drawn_plans_fit(faults):
    r = random.Random(5)
    for _ in range(20000):
        K, N = (16 * r.randint(1, int(4096 * 16 ** r.random() / 16)) for _ in range(2))
        T = int(2 ** (20 * r.random()))
        assert faults(K, N, r.randint(0, 1), T, min(1 << 20, T + r.randint(0, 300))) == 0, (K, N, T)


def test_products_past_the_launch_limits_are_refused():
    import quantization_error_compensation_amd as q
    from quantization_error_compensation_amd import q8
    d = q.make_q8_desc(16, 262144)
    args = [0x10000 * (i + 1) for i in range(6)]
    call = q8._lib().spear_ec_q8_linear
    assert call(ctypes.byref(d), (1 << 19) + 1, *args, 1 << 40, None) == 2
