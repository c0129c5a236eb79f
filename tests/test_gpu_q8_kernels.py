"""Every compiled kernel of the 8-bit products (needs an MI355X), at the sizes of
q8_shapes.py, against the definition in 64 bits."""
from __future__ import annotations

import math
import random

import pytest

import quantization_error_compensation_amd as q
from q8_shapes import PRODUCTS
from test_gpu_q8 import bits_equal, guarded, note, operands, ref, torch  # noqa: F401

pytestmark = pytest.mark.gpu

GROUPS = sorted({(k // 1000 if k < 10000 else k // 100, g) for k, g, *_ in PRODUCTS})


@pytest.mark.parametrize("group,gated", GROUPS)
def test_products_of_every_kernel(torch, ref, group, gated):  # noqa: F811
    """Both types of y on one workspace, whose counters every call leaves at zero."""
    for i, (k, g, T, K, N) in enumerate(PRODUCTS):
        if (k // 1000 if k < 10000 else k // 100, g) != (group, gated):
            continue
        act = "none" if not g else "silu" if i % 4 < 2 else "gelu"
        note(f"kernel {k} T={T} K={K} N={N} {act}")
        d = q.make_q8_desc(K, N, act)
        x = operands(torch, T, K, q.q8_weight_shape(d)[0], 7000 + i)
        work = q.alloc_q8_workspace(d, T)
        want, tol = ref.product(*x, act)
        for f32 in (False, True):
            d = q.make_q8_desc(K, N, act, out_f32=f32)
            y, ok = guarded(torch, (T, N), torch.float32 if f32 else torch.bfloat16)
            y.fill_(math.nan)
            q.spear_ec_q8_linear(d, *x, y, work)
            torch.cuda.synchronize()
            ref.check(y, want, tol, (k, T, K, N, act, f32))
            ok()
            assert int(work[:65536].count_nonzero()) == 0
        again = torch.empty_like(y)
        q.spear_ec_q8_linear(d, *x, again, work)
        assert bits_equal(torch, again, y)


def test_splits_of_every_tile_repeat_bit_for_bit(torch, ref):  # noqa: F811
    """Products whose K is split meet in memory in an order that differs from call to
    call: every tile shape with every number of splits, in random order on one
    workspace, gives the first call's bits."""
    cases, size = [], 0
    for i, (k, g, T, K, N) in enumerate(PRODUCTS):
        if k < 10000 or k % 100 == 1:
            continue
        d = q.make_q8_desc(K, N, "silu" if g else "none")
        x = operands(torch, T, K, q.q8_weight_shape(d)[0], 8000 + i)
        size = max(size, q.spear_ec_q8_workspace_bytes(d, T))
        cases.append((k, d, x, torch.empty((T, N), dtype=torch.bfloat16, device="cuda")))
    work = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first = []
    for k, d, x, y in cases:
        y.fill_(math.nan)
        q.spear_ec_q8_linear(d, *x, y, work)
        want, tol = ref.product(*x, "silu" if d.flags else "none")
        ref.check(y, want, tol, k)
        first.append(y.clone())
    same = torch.ones(len(cases), dtype=torch.bool, device="cuda")
    r = random.Random(12)
    for n in range(10 * len(cases)):
        i = r.randrange(len(cases))
        k, d, x, y = cases[i]
        y.fill_(math.nan)
        q.spear_ec_q8_linear(d, *x, y, work)
        same[i] &= (y == first[i]).all()
        if n % 200 == 199:
            torch.cuda.synchronize()
            note(f"  {n + 1} calls")
    assert bool(same.all()), [cases[i][0] for i in (~same).nonzero().flatten().tolist()]
    assert int(work[:65536].count_nonzero()) == 0
