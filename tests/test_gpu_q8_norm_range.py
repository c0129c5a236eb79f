"""The 8-bit path's norm at the ends of what it accepts (needs an MI355X)."""
from __future__ import annotations

import math

import pytest

import quantization_error_compensation_amd as q
from test_gpu_q8 import guarded, note, ref, rng, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def defined(torch, x, residual, weight, eps):  # noqa: F811
    """(h as bf16, u in float64) from the definition; a row is NaN if h or weight
    is not finite there."""
    h = x if residual is None else (x.double() + residual.double()).bfloat16()
    d, w = h.double(), weight.double()
    u = d * w / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    good = torch.isfinite(d).all(1) & bool(torch.isfinite(w).all())
    return h, torch.where(good[:, None], u, torch.full_like(u, math.nan))


def run(torch, x, residual, weight, eps):  # noqa: F811
    """(sum, y, codes, scales), once together and with y and the codes alone: the same."""
    total = None if residual is None else torch.empty_like(x)
    y, y_ok = guarded(torch, x.shape, torch.bfloat16)
    codes, codes_ok = guarded(torch, x.shape, torch.int8)
    scales, scales_ok = guarded(torch, x.shape[:1], torch.float32)
    q.spear_ec_q8_rmsnorm(x, residual, total, weight, eps, y, codes, scales)
    y2, codes2, scales2 = torch.empty_like(y), torch.empty_like(codes), torch.empty_like(scales)
    q.spear_ec_q8_rmsnorm(x, residual, total, weight, eps, y=y2)
    q.spear_ec_q8_rmsnorm(x, residual, total, weight, eps, codes=codes2, scales=scales2)
    torch.cuda.synchronize()
    for ok in (y_ok, codes_ok, scales_ok):
        ok()
    for a, b in ((y, y2), (codes.float(), codes2.float()), (scales, scales2)):
        assert torch.equal(a.nan_to_num(7e7), b.nan_to_num(7e7))
    return total, y, codes, scales


def check(torch, ref, got, h, u, low=0.0):  # noqa: F811
    """y: half a step of bf16 (2^-8 of the value, 2^-134 below its normal range) and
    2^-12 of that for the steps before; low: what the header allows besides for rows
    with products below fp32's normal range.  Codes and scales: the definition's,
    but where a few steps of fp64 (the order of the sum) put a scale on the other
    side of a border of fp32, 2^-23 of it, or a code of a border, 127 * 2^-23 away."""
    total, y, codes, scales = got
    if total is not None:
        assert torch.equal(total, h)
    want, s = ref.quantize(u)
    bad = s.isnan()
    assert torch.equal(y.isnan().all(1), bad) and torch.equal(y.isnan().any(1), bad)
    assert torch.equal(scales.isnan(), bad)
    assert bool((codes[bad] == 0).all())
    past = u.float().bfloat16().isinf()   # past bf16
    bound = (u.abs() * 2.0 ** -8 * (1 + 2.0 ** -12)).clamp(min=low) + 2.0 ** -134
    good = (y.double() - u).abs() <= bound
    assert bool((good | (past & y.isinf() & ((y > 0) == (u > 0))) | bad[:, None]).all())
    assert torch.allclose(scales[~bad], s[~bad], rtol=2.0 ** -23, atol=0)
    near = (u / s.double()[:, None]).abs().frac().sub(0.5).abs() < 127 * 2.0 ** -23
    assert bool(((codes == want) | (near & ((codes.int() - want.int()).abs() <= 1)))[~bad].all())


EPS = (5e-324, 1e-300, 1e-100, 1e-80, 1e-77, 1e-76, 1e-30, 1.0, 1e30, 1e75, 1e76, 1e77, 1e88, 1e90, 1e100, 1e300)


@pytest.mark.parametrize("width", [48, 1040, 4096])
@pytest.mark.parametrize("eps", EPS)
def test_results_for_every_eps(torch, ref, width, eps):  # noqa: F811
    """1 / sqrt(mean(h^2) + eps) from 4.5e161 to 1e-150: past either end of fp32 and
    in its subnormal range."""
    note(f"eps {eps} x {width}")
    g = rng(torch, width)
    for hs, ws in ((0.0, 1.0), (1.0, 1.0), (2.0 ** -130, 2.0 ** 100), (1e18, 1e18), (1.0, 1e30), (1e37, 1.0),
                   (2.0 ** -120, 1.0)):
        x = (torch.randn((9, width), generator=g, device="cuda") * hs).bfloat16()
        x[4] = 0
        w = (torch.randn(width, generator=g, device="cuda") * ws).bfloat16()
        h, u = defined(torch, x, None, w, eps)
        check(torch, ref, run(torch, x, None, w, eps), h, u)
        zero = (h == 0).all(1)
        total, y, codes, scales = run(torch, x, x.flip(0).contiguous(), w, eps)
        h, u = defined(torch, x, x.flip(0), w, eps)
        check(torch, ref, (total, y, codes, scales), h, u)
        assert bool((y[zero & zero.flip(0)] == 0).all())


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,width", [(5, 48), (6, 400), (7, 1936), (12, 4112), (3, 65536)])
def test_products_past_fp32(torch, ref, rows, width, residual):  # noqa: F811
    """Rows of finite h whose products with finite weights leave fp32, among
    ordinary rows, rows of zeros, rows that are not finite, in place too."""
    note(f"products past fp32 {rows} x {width} residual={residual}")
    g = rng(torch, rows + width)
    for hs, ws, eps in ((1e25, 1e20, 1e-5), (1e37, 1e37, 1e-5), (1e20, 1e30, 1e30), (1e38, 1e3, 1e80)):
        x = (torch.randn((rows, width), generator=g, device="cuda").clamp(-3, 3) * hs).bfloat16()
        x[1] = torch.randn(width, generator=g, device="cuda").bfloat16()
        if rows > 3:
            x[2] = 0
            x[3, width // 2] = math.inf
        w = (torch.randn(width, generator=g, device="cuda").clamp(-3, 3) * ws).bfloat16()
        r = (torch.randn((rows, width), generator=g, device="cuda") * 1e-3 * hs).bfloat16() if residual else None
        if residual:
            r[1:3] = 0
        h, u = defined(torch, x, r, w, eps)
        assert bool((h.float() * w.float()).isinf().any()) and bool(u[0].isfinite().all())
        check(torch, ref, run(torch, x, r, w, eps), h, u)
        if residual:
            codes, scales = q.alloc_q8(rows, width)
            q.spear_ec_q8_rmsnorm(x, r, r, w, eps, y := torch.empty_like(x), codes, scales)
            check(torch, ref, (r, y, codes, scales), h, u)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_weights_that_are_not_finite(torch, ref, bad):  # noqa: F811
    g = rng(torch, 3)
    for width in (16, 272, 1040, 8208):
        x = torch.randn((5, width), generator=g, device="cuda").bfloat16()
        x[1] = 0
        x[2] *= 2.0 ** -120
        x[3] *= 1e38
        w = torch.randn(width, generator=g, device="cuda").bfloat16()
        w[width // 2] = bad
        h, u = defined(torch, x, None, w, 1e-5)
        got = run(torch, x, None, w, 1e-5)
        check(torch, ref, got, h, u)
        assert bool(got[1].isnan().all()) and bool(got[3].isnan().all())
