"""Row operators of the 8-bit path (needs an MI355X) for every count of elements that
a lane or thread holds, against the definition in 64 bits."""
from __future__ import annotations

import pytest

import quantization_error_compensation_amd as q
from test_gpu_q8 import guarded, note, ref, rng, special_rows, torch  # noqa: F401
from test_gpu_q8_norm_range import check, defined, run

pytestmark = pytest.mark.gpu

# Rows of at most 256 pieces of 8 elements: 1 a lane of 16, 32, 64 lanes, then 2, 3, 4
# of 64; wider ones 2 to 8 a thread of a workgroup.  In calls of 2048 rows or more
# fewer threads hold 3 or 4 each (bf16).
WIDTHS = [112, 128, 240, 496, 1008, 1520, 1936, 2048, 2064, 4112, 20496, 28688, 36880, 45072, 53264, 61456]
MANY = [2064, 3088, 5136, 7184, 11280, 15376, 20496]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,width", [(9, w) for w in WIDTHS] + [(2049, w) for w in MANY])
def test_quantize_of_every_width(torch, ref, rows, width, kind):  # noqa: F811
    note(f"quantize {rows} x {width} {kind}")
    x = torch.randn((rows, width), generator=rng(torch, rows + width), device="cuda")
    x = special_rows(torch, x.bfloat16() if kind == "bf16" else x, width)
    want, scale = ref.quantize(x.double())
    codes, codes_ok = guarded(torch, (rows, width), torch.int8)
    scales, scales_ok = guarded(torch, (rows,), torch.float32)
    out, out_ok = guarded(torch, (rows, width), torch.float32)
    q.spear_ec_q8_quantize(x, codes, scales)
    q.spear_ec_q8_dequant_f32(codes, scales, out)
    torch.cuda.synchronize()
    assert torch.equal(scales, scale) and torch.equal(codes, want)
    assert torch.equal(out, want.float() * scale[:, None])
    for ok in (codes_ok, scales_ok, out_ok):
        ok()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,width", [(9, w) for w in WIDTHS] + [((6 << 20) // w + 9, w) for w in WIDTHS] +
                         [(2049, w) for w in MANY] + [(2049, 16), (400001, 16)])
def test_norm_of_every_width(torch, ref, rows, width, residual):  # noqa: F811
    """Calls on either side of 6 M elements, from which on results stay in the caches."""
    note(f"norm {rows} x {width} residual={residual}")
    g = rng(torch, 13 * rows + width)
    x = special_rows(torch, torch.randn((rows, width), generator=g, device="cuda").bfloat16(), width)
    r = None
    if residual:
        r = torch.randn((rows, width), generator=g, device="cuda").bfloat16()
        r[1] = 0
        r[3] = -x[3]
    w = (1 + 0.2 * torch.randn(width, generator=g, device="cuda")).bfloat16()
    h, u = defined(torch, x, r, w, 1e-5)
    # products below fp32's normal range, as the header has it
    low = 2.0 ** -149 / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + 1e-5)
    check(torch, ref, run(torch, x, r, w, 1e-5), h, u, low)
