"""The 8-bit path's C ABI without a GPU: declared, exported and bound names, the
refusals of every entry point (none of which reaches a HIP call), those of the
binding, and the reference that the GPU tests use."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import q8_reference as ref
import quantization_error_compensation_amd as q
from quantization_error_compensation_amd import binding, q8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from quantization_error_compensation_amd import build
        build.build()
    return q8._lib()


def test_header_binding_and_library_name_the_same_functions(lib):
    text = open(os.path.join(ROOT, "include", "spear_ec_q8.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(spear_ec_\w+)\s*\(", text)))
    assert names == sorted(q.Q8_EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(names) <= set(re.findall(r"\sT\s(spear_ec_\w+)", out))


def ptr(i):
    return 0x10000 * (i + 1)


def quantize(lib, rows=2, width=64, x=ptr(0), f32=0, stride=64, codes=ptr(1), scales=ptr(2)):
    return lib.spear_ec_q8_quantize(rows, width, x, f32, stride, codes, scales, None)


def dequant(lib, rows=2, width=64, codes=ptr(1), scales=ptr(2), out=ptr(3)):
    return lib.spear_ec_q8_dequant_f32(rows, width, codes, scales, out, None)


def norm(lib, rows=2, width=64, x=ptr(0), stride=64, residual=None, sum=None, weight=ptr(4), eps=1e-5, y=None,
         codes=ptr(1), scales=ptr(2)):
    return lib.spear_ec_q8_rmsnorm(rows, width, x, stride, residual, sum, weight, eps, y, codes, scales, None)


def linear(lib, desc, tokens=2, xq=ptr(0), xs=ptr(1), wq=ptr(2), ws=ptr(3), y=ptr(4), work=ptr(5), size=1 << 40):
    return lib.spear_ec_q8_linear(ctypes.byref(desc) if desc else None, tokens, xq, xs, wq, ws, y, work, size, None)


@pytest.mark.parametrize("call", [quantize, dequant, norm])
def test_rows_and_widths_are_checked(lib, call):
    for change, code in ((dict(rows=-1), INVALID), (dict(width=0), INVALID), (dict(width=-16), INVALID),
                         (dict(width=24), UNSUPPORTED), (dict(width=65552), UNSUPPORTED),
                         (dict(codes=ptr(1) + 8), MISALIGNED), (dict(scales=ptr(2) + 2), MISALIGNED),
                         (dict(scales=None), INVALID)):
        assert call(lib, **change) == code, change
        assert q.spear_ec_last_error()
    assert call(lib, rows=0, codes=None, scales=None) == OK   # nothing to do


def test_quantize_and_dequant_refusals(lib):
    for change, code in ((dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(stride=63), INVALID),
                         (dict(stride=-64), INVALID), (dict(stride=1 << 33), INVALID), (dict(stride=68), MISALIGNED),
                         (dict(x=ptr(0) + 4), MISALIGNED), (dict(f32=1, x=ptr(0) + 8), MISALIGNED)):
        assert quantize(lib, **change) == code, change
    assert dequant(lib, out=None) == INVALID
    assert dequant(lib, codes=None) == INVALID
    assert dequant(lib, out=ptr(3) + 4) == MISALIGNED


def test_norm_refusals(lib):
    r, s, y = ptr(6), ptr(7), ptr(8)
    for change, code in ((dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(residual=r), INVALID),
                         (dict(sum=s), INVALID), (dict(codes=None, scales=None), INVALID), (dict(codes=None), INVALID),
                         (dict(eps=0.0), INVALID), (dict(eps=-1e-5), INVALID), (dict(eps=math.nan), INVALID),
                         (dict(eps=math.inf), INVALID), (dict(stride=56), INVALID), (dict(stride=100), MISALIGNED),
                         (dict(weight=ptr(4) + 2), MISALIGNED), (dict(residual=r + 8, sum=s), MISALIGNED),
                         (dict(residual=r, sum=s + 2), MISALIGNED), (dict(y=y + 2), MISALIGNED),
                         (dict(residual=r, sum=ptr(0), stride=72), INVALID), (dict(y=ptr(0)), INVALID),
                         (dict(residual=r, sum=s, y=r), INVALID), (dict(residual=r, sum=s, y=s), INVALID)):
        assert norm(lib, **change) == code, change
        assert q.spear_ec_last_error()


BAD_DESCS = [((0, 64, 0), INVALID), ((64, 0, 0), INVALID), ((-16, 64, 0), INVALID), ((64, 64, 1), INVALID),
             ((64, 64, 32), INVALID), ((64, 64, 16), INVALID), ((24, 64, 0), UNSUPPORTED), ((64, 24, 0), UNSUPPORTED),
             ((65552, 64, 0), UNSUPPORTED), ((64, 262160, 0), UNSUPPORTED)]


def test_linear_refusals(lib):
    assert linear(lib, None) == INVALID
    for fields, code in BAD_DESCS:
        assert linear(lib, q.spear_ec_q8_desc(*fields)) == code, fields
        assert q.spear_ec_q8_workspace_bytes(q.spear_ec_q8_desc(*fields), 1) == 0
    for act in ("none", "silu", "gelu"):
        d = q.make_q8_desc(64, 48, act)
        for change, code in ((dict(tokens=-1), INVALID), (dict(tokens=(1 << 20) + 1), UNSUPPORTED),
                             (dict(xq=None), INVALID), (dict(xs=None), INVALID), (dict(wq=None), INVALID),
                             (dict(ws=None), INVALID), (dict(y=None), INVALID), (dict(work=None), WORKSPACE),
                             (dict(size=64), WORKSPACE), (dict(xq=ptr(0) + 4), MISALIGNED),
                             (dict(xs=ptr(1) + 1), MISALIGNED), (dict(wq=ptr(2) + 8), MISALIGNED),
                             (dict(ws=ptr(3) + 2), MISALIGNED), (dict(y=ptr(4) + 8), MISALIGNED),
                             (dict(work=ptr(5) + 8), MISALIGNED)):
            assert linear(lib, d, **change) == code, change
            assert q.spear_ec_last_error()
        assert linear(lib, d, tokens=0, xq=None, xs=None, wq=None, ws=None, y=None, work=None, size=0) == OK


def test_workspaces_cover_smaller_calls(lib):
    assert q.spear_ec_q8_workspace_bytes(q.make_q8_desc(64, 48), -1) == 0
    assert q.spear_ec_q8_workspace_bytes(q.make_q8_desc(64, 48), (1 << 20) + 1) == 0
    for K, N, act in ((64, 48, "none"), (4096, 4096, "none"), (28672, 8192, "none"), (8192, 28672, "silu"),
                      (65536, 16, "none"), (16, 262144, "gelu"), (8192, 1024, "none")):
        d = q.make_q8_desc(K, N, act)
        sizes = [q.spear_ec_q8_workspace_bytes(d, t) for t in (0, 1, 2, 16, 17, 32, 33, 64, 65, 100, 128, 129, 200, 256,
                                                              257, 300, 384, 512, 513, 700, 1024, 2000, 4096, 9000,
                                                              1 << 17, 1 << 20)]
        assert sizes[0] >= 16 and sizes == sorted(sizes), (K, N, act, sizes)
        assert sizes[-1] <= 256 << 20


def test_the_binding_refuses_what_the_library_cannot_see(lib):
    """Types, shapes and layouts (CPU tensors: each is refused before a call)."""
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    codes, scales = q.alloc_q8(2, 64, "cpu")
    w = torch.zeros(64, dtype=torch.bfloat16)
    d = q.make_q8_desc(64, 48)
    wq, ws = q.alloc_q8(48, 64, "cpu")
    y = torch.zeros((2, 48), dtype=torch.bfloat16)
    work = torch.zeros(1 << 20, dtype=torch.uint8)
    bad = [
        lambda: q.spear_ec_q8_quantize(x.half(), codes, scales),
        lambda: q.spear_ec_q8_quantize(x[0], codes, scales),
        lambda: q.spear_ec_q8_quantize(x.t().contiguous().t(), codes, scales),
        lambda: q.spear_ec_q8_quantize(x, codes[:1], scales),
        lambda: q.spear_ec_q8_quantize(x, codes.view(torch.uint8), scales),
        lambda: q.spear_ec_q8_quantize(x, codes, scales.double()),
        lambda: q.spear_ec_q8_quantize(x, codes, scales[:1]),
        lambda: q.spear_ec_q8_quantize(x, codes, scales),          # not on a GPU
        lambda: q.spear_ec_q8_dequant_f32(codes, scales, y),
        lambda: q.spear_ec_q8_dequant_f32(codes[0], scales, y),
        lambda: q.spear_ec_q8_rmsnorm(x.float(), None, None, w, 1e-5, codes=codes, scales=scales),
        lambda: q.spear_ec_q8_rmsnorm(x, None, None, w[:32], 1e-5, codes=codes, scales=scales),
        lambda: q.spear_ec_q8_rmsnorm(x, x[:1], x, w, 1e-5, codes=codes, scales=scales),
        lambda: q.spear_ec_q8_rmsnorm(x, x, x.float(), w, 1e-5, codes=codes, scales=scales),
        lambda: q.spear_ec_q8_rmsnorm(x, None, None, w, 1e-5, codes=codes),
        lambda: q.spear_ec_q8_rmsnorm(x, None, None, w, 1e-5, y=y),
        lambda: q.spear_ec_q8_linear(d, codes[:, :32], scales, wq, ws, y, work),
        lambda: q.spear_ec_q8_linear(d, codes, scales[:1], wq, ws, y, work),
        lambda: q.spear_ec_q8_linear(d, codes, scales, wq[:47], ws, y, work),
        lambda: q.spear_ec_q8_linear(d, codes, scales, wq, ws[:47], y, work),
        lambda: q.spear_ec_q8_linear(d, codes, scales, wq, ws, y.float(), work),
        lambda: q.spear_ec_q8_linear(d, codes, scales, wq, ws, y[:1], work),
        lambda: q.spear_ec_q8_linear(d, codes, scales, wq, ws, y, None),
        lambda: q.spear_ec_q8_linear(d, codes, scales, wq, ws, y, work),   # not on a GPU
        lambda: q.make_q8_desc(64, 48, "relu"),
        lambda: q.alloc_q8_workspace(q.make_q8_desc(24, 48), 1, "cpu"),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_reference_quantize_by_hand():
    v = torch.tensor([[127.0, 2.5, 3.5, -127.0], [0, 0, 0, 0], [-254.0, 1.0, 3.0, 0.5], [1.0, math.inf, 0, 0]],
                     dtype=torch.float64)
    c, s = ref.quantize(v)
    assert c.tolist() == [[127, 2, 4, -127], [0, 0, 0, 0], [-127, 0, 2, 0], [0, 0, 0, 0]]
    assert s[:3].tolist() == [1.0, 1.0, 2.0] and math.isnan(s[3])


def test_reference_norm_and_product_by_hand():
    x = torch.tensor([[3.0, 4.0]]).bfloat16()
    h, u = ref.norm(x, x, torch.tensor([1.0, 2.0]).bfloat16(), 0.5)
    assert h.tolist() == [[6.0, 8.0]]
    r = 1 / math.sqrt(50.5)
    assert torch.allclose(u, torch.tensor([[6 * r, 16 * r]], dtype=torch.float64), rtol=1e-15)
    xq, wq = torch.tensor([[1, 2]], dtype=torch.int8), torch.tensor([[3, -1], [0, 5]], dtype=torch.int8)
    y, _ = ref.product(xq, torch.tensor([0.5]), wq, torch.tensor([2.0, 1.0]))
    assert y.tolist() == [[1.0, 5.0]]
    for act, f in (("silu", lambda a: a / (1 + math.exp(-a))),
                   ("gelu", lambda a: 0.5 * a * (1 + math.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))))):
        y, tol = ref.product(xq, torch.tensor([0.5]), wq, torch.tensor([2.0, 1.0]), act)
        assert abs(float(y) - f(1.0) * 5.0) < 1e-14 and 0 < float(tol) < 1e-4
