"""The 8-bit path called over and over (needs an MI355X): products whose K is
split meet in memory, in an order that differs from call to call, and must give
the same bits each time on one workspace that no call leaves dirty; row
operators in place; calls on other streams than the current one."""
from __future__ import annotations

import math
import random

import pytest

import quantization_error_compensation_amd as q
from test_gpu_q8 import bits_equal, note, operands, ref, rng, torch  # noqa: F401

pytestmark = pytest.mark.gpu

# tokens, d_in, d_out, act: 2 to 4 splits of four tile shapes, whole tiles and ragged ones, and the streams
SHAPES = [(512, 28672, 2048, "none"), (256, 8192, 8192, "none"), (300, 28672, 1040, "silu"), (1000, 11008, 2064, "none"),
          (72, 4112, 4096, "gelu"), (100, 8192, 1024, "none"), (48, 8192, 10240, "none"), (40, 11008, 4096, "none"),
          (200, 16400, 1040, "silu"), (20, 4096, 4096, "none"), (1, 8192, 1024, "none"), (513, 4112, 528, "none")]


def test_products_repeat_bit_for_bit(torch, ref):  # noqa: F811
    r = random.Random(11)
    cases, size = [], 0
    for i, (T, K, N, act) in enumerate(SHAPES):
        d = q.make_q8_desc(K, N, act)
        x = operands(torch, T, K, q.q8_weight_shape(d)[0], 900 + i)
        size = max(size, q.spear_ec_q8_workspace_bytes(d, T))
        cases.append((d, x, torch.empty((T, N), dtype=torch.bfloat16, device="cuda"), act))
    work = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first = []
    for i, (d, x, y, act) in enumerate(cases):
        note(f"first call {SHAPES[i]}")
        y.fill_(math.nan)
        q.spear_ec_q8_linear(d, *x, y, work)
        want, tol = ref.product(*x, act)
        ref.check(y, want, tol, SHAPES[i])
        first.append(y.clone())
    same = torch.ones(len(cases), dtype=torch.bool, device="cuda")
    for n in range(600):
        i = r.randrange(len(cases))
        d, x, y, _ = cases[i]
        y.fill_(math.nan)
        q.spear_ec_q8_linear(d, *x, y, work)
        same[i] &= (y == first[i]).all()
        if n % 100 == 99:
            torch.cuda.synchronize()
            note(f"  {n + 1} calls")
    assert bool(same.all()), [SHAPES[i] for i in (~same).nonzero().flatten().tolist()]
    assert int(work[:65536].count_nonzero()) == 0


@pytest.mark.parametrize("rows,width", [(5, 48), (9, 1008), (3, 4096), (40, 8208)])
@pytest.mark.parametrize("over", ["x", "residual"])
def test_norm_in_place_of_small_and_usual_rows(torch, ref, rows, width, over):  # noqa: F811
    """Rows near fp32's small end read their sum again after it is written."""
    g = rng(torch, rows * width)
    x = torch.randn((rows, width), generator=g, device="cuda")
    r = torch.randn((rows, width), generator=g, device="cuda")
    scale = torch.tensor([2.0 ** -128, 1.0, 2.0 ** -105, 2.0 ** -133], device="cuda")[torch.arange(rows, device="cuda") % 4]
    x, r = (x * scale[:, None]).bfloat16(), (r * scale[:, None]).bfloat16()
    w = (1 + 0.2 * torch.randn(width, generator=g, device="cuda")).bfloat16()
    h, u = ref.norm(x, r, w, 1e-6)
    want, s = ref.quantize(u)
    codes, scales = q.alloc_q8(rows, width)
    total = x if over == "x" else r
    q.spear_ec_q8_rmsnorm(x, r, total, w, 1e-6, codes=codes, scales=scales)
    assert torch.equal(total, h) and torch.equal(scales, s) and torch.equal(codes, want)


def test_calls_follow_the_current_stream(torch, ref):  # noqa: F811
    d = q.make_q8_desc(4096, 2064)
    x = operands(torch, 200, 4096, 2064, 5)
    want, tol = ref.product(*x)
    work = q.alloc_q8_workspace(d, 200)
    for given in (None, "object", "handle"):
        side = torch.cuda.Stream()
        y = torch.full((200, 2064), math.nan, dtype=torch.bfloat16, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        if given is None:
            with torch.cuda.stream(side):
                q.spear_ec_q8_linear(d, *x, y, work)
        else:
            q.spear_ec_q8_linear(d, *x, y, work, stream=side if given == "object" else side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
        ref.check(y, want, tol, given)


def test_views_of_larger_buffers(torch, ref):  # noqa: F811
    """Operands and results in the middle of larger buffers, 16 bytes apart from aligned ones."""
    K, N, T = 1040, 272, 77
    for act in ("none", "silu"):
        d = q.make_q8_desc(K, N, act)
        rows = q.q8_weight_shape(d)[0]
        xq, xs, wq, ws = operands(torch, T, K, rows, 6)
        bx = torch.zeros(T * K + 48, dtype=torch.int8, device="cuda")
        bw = torch.zeros(rows * K + 48, dtype=torch.int8, device="cuda")
        bs = torch.zeros(T + rows + 8, device="cuda")
        bx[16:16 + T * K] = xq.flatten()
        bw[32:32 + rows * K] = wq.flatten()
        bs[1:1 + T], bs[T + 2:T + 2 + rows] = xs, ws
        by = torch.full((T * N + 24,), 7.0, dtype=torch.bfloat16, device="cuda")
        y = by[8:8 + T * N].view(T, N)
        q.spear_ec_q8_linear(d, bx[16:16 + T * K].view(T, K), bs[1:1 + T], bw[32:32 + rows * K].view(rows, K),
                             bs[T + 2:T + 2 + rows], y, q.alloc_q8_workspace(d, T))
        want, tol = ref.product(xq, xs, wq, ws, act)
        ref.check(y, want, tol, act)
        assert bool((by[:8] == 7).all()) and bool((by[8 + T * N:] == 7).all())
        plain = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        q.spear_ec_q8_linear(d, xq, xs, wq, ws, plain, q.alloc_q8_workspace(d, T))
        assert bits_equal(torch, plain, y)
