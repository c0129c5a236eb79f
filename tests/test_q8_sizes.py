"""Sizes that do not fit the C ABI's 32-bit counts: the 8-bit path's binding
refuses them (tensors without memory; no call is made)."""
import pytest
import torch

import quantization_error_compensation_amd as q
from quantization_error_compensation_amd import q8

MANY = 2 ** 32 + 16   # 16, as 32 bits hold it


@pytest.fixture
def no_call(monkeypatch):
    monkeypatch.setattr(q8, "_run", lambda fn, dev, stream, *args: pytest.fail(f"called with {args}"))


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("rows,width", [(MANY, 16), (2 ** 31, 16), (1, MANY), (1, 2 ** 31)])
def test_rows_and_widths(no_call, rows, width):
    x, codes, scales = empty(rows, width), empty(rows, width, dtype=torch.int8), empty(rows, dtype=torch.float32)
    weight = empty(width)
    for call in (lambda: q.spear_ec_q8_quantize(x, codes, scales),
                 lambda: q.spear_ec_q8_quantize(x.float(), codes, scales),
                 lambda: q.spear_ec_q8_dequant_f32(codes, scales, empty(rows, width, dtype=torch.float32)),
                 lambda: q.spear_ec_q8_rmsnorm(x, None, None, weight, 1e-5, y=empty(rows, width)),
                 lambda: q.spear_ec_q8_rmsnorm(x, None, None, weight, 1e-5, codes=codes, scales=scales)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


@pytest.mark.parametrize("tokens", [MANY, 2 ** 31])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_tokens(no_call, tokens, act):
    d = q.make_q8_desc(16, 32, act)
    rows = q.q8_weight_shape(d)[0]
    with pytest.raises(ValueError, match="2\\^31"):
        q.spear_ec_q8_linear(d, empty(tokens, 16, dtype=torch.int8), empty(tokens, dtype=torch.float32),
                             empty(rows, 16, dtype=torch.int8), empty(rows, dtype=torch.float32),
                             empty(tokens, 32), empty(1 << 20, dtype=torch.uint8))


def test_workspaces():
    d = q.make_q8_desc(16, 32)
    assert q.spear_ec_q8_workspace_bytes(d, 16) > 0
    for tokens in (MANY, -MANY, 2 ** 31, 2 ** 64 + 16):
        assert q.spear_ec_q8_workspace_bytes(d, tokens) == 0
        with pytest.raises(ValueError):
            q.alloc_q8_workspace(d, tokens, "cpu")
