"""The key/value cache's C ABI without a GPU: declared, exported and bound
names, the refusals of every entry point (none of which reaches a HIP call),
and the reference the GPU tests use."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import quantization_error_compensation_amd as q
from quantization_error_compensation_amd import binding, kv
import kv_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from quantization_error_compensation_amd import build
        build.build()
    return kv._lib()


def test_header_binding_and_library_name_the_same_functions(lib):
    text = open(os.path.join(ROOT, "include", "spear_ec_kv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(spear_ec_\w+)\s*\(", text)))
    assert names == sorted(q.KV_EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = set(re.findall(r"\sT\s(spear_ec_\w+)", out))
    assert set(names) <= exported


GOOD = dict(q_heads=8, kv_heads=2, head_dim=128, page_tokens=16, pages=4, max_pages=2, zeros=False)
BAD_DESCS = [
    (dict(q_heads=0), INVALID), (dict(kv_heads=-1), INVALID), (dict(head_dim=0), INVALID),
    (dict(pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(page_tokens=0), INVALID),
    (dict(q_heads=7), UNSUPPORTED), (dict(q_heads=258), UNSUPPORTED),
    (dict(q_heads=257, kv_heads=257), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=256), UNSUPPORTED), (dict(page_tokens=8), UNSUPPORTED),
    (dict(page_tokens=48), UNSUPPORTED), (dict(page_tokens=8192), UNSUPPORTED),
    (dict(page_tokens=4096, max_pages=1 << 19), UNSUPPORTED),
    (dict(pages=1 << 30), UNSUPPORTED),
]


def ptr(i):
    return 0x10000 * (i + 1)


def batch(n=2, tokens=2, off=None, lens=ptr(20), table=ptr(21)):
    return q.spear_ec_kv_batch(n, tokens, off, lens, table)


def call(lib, name, desc, b, **kw):
    d = ctypes.byref(desc) if desc is not None else None
    bb = ctypes.byref(b) if b is not None else None
    g = lambda k, v: kw.get(k, v)  # noqa: E731
    cache = (g("codes", ptr(3)), g("scales", ptr(4)), g("zeros", None))
    if name == "append":
        rope = g("rope", None)
        return lib.spear_ec_kv_append(
            d, bb, g("q", ptr(0)), g("qs", 1024), g("k", ptr(1)), g("ks", 256), g("v", ptr(2)),
            g("vs", 256), ctypes.byref(rope) if rope is not None else None, *cache,
            g("q_out", ptr(5)), g("os", 1024), None)
    if name == "attention":
        return lib.spear_ec_kv_attention(
            d, bb, g("q", ptr(0)), g("qs", 1024), *cache, g("scale", 0.1), g("window", 0),
            g("out", ptr(6)), g("lse", None), g("ws", ptr(7)), g("ws_bytes", 1), None)
    return lib.spear_ec_kv_dequant_f32(d, bb, *cache, g("k_out", ptr(8)), g("v_out", ptr(9)), None)


NAMES = ("append", "attention", "dequant")


@pytest.mark.parametrize("name", NAMES)
def test_descs_and_batches_are_checked(lib, name):
    good = q.make_kv_desc(**GOOD)
    assert call(lib, name, None, batch()) == INVALID
    assert call(lib, name, good, None) == INVALID
    for change, code in BAD_DESCS:
        assert call(lib, name, q.make_kv_desc(**{**GOOD, **change}), batch()) == code, change
        assert q.spear_ec_kv_workspace_bytes(q.make_kv_desc(**{**GOOD, **change}), 1, 1) == 0
    flags = q.make_kv_desc(**GOOD)
    flags.flags = 4
    assert call(lib, name, flags, batch()) == INVALID
    assert call(lib, name, good, batch(n=-1)) == INVALID
    assert call(lib, name, good, batch(tokens=-1)) == INVALID
    assert call(lib, name, good, batch(n=65537, tokens=65537)) == UNSUPPORTED
    assert call(lib, name, good, batch(tokens=(1 << 20) + 1, off=ptr(22))) == UNSUPPORTED
    many = q.make_kv_desc(**{**GOOD, "q_heads": 256})
    assert call(lib, name, many, batch(tokens=(1 << 19) + 1, off=ptr(22))) == UNSUPPORTED
    assert call(lib, name, good, batch(lens=None)) == INVALID
    assert call(lib, name, good, batch(table=None)) == INVALID
    assert call(lib, name, good, batch(tokens=3)) == INVALID          # needs q_offsets
    assert call(lib, name, good, batch(lens=ptr(20) + 2)) == MISALIGNED
    assert call(lib, name, good, batch(off=ptr(22) + 1)) == MISALIGNED
    # nothing to do: no pointer is looked at
    assert call(lib, name, good, batch(n=0, tokens=0, lens=None, table=None), codes=None) == OK
    assert call(lib, name, good, batch(n=2, tokens=0, lens=None, table=None), codes=None) == OK
    for change, code in ((dict(codes=None), INVALID), (dict(scales=None), INVALID),
                         (dict(codes=ptr(3) + 8), MISALIGNED), (dict(scales=ptr(4) + 2), MISALIGNED)):
        assert call(lib, name, good, batch(), **change) == code, change
    asym = q.make_kv_desc(**{**GOOD, "zeros": True})
    assert call(lib, name, asym, batch()) == INVALID
    assert call(lib, name, asym, batch(), zeros=ptr(10) + 4) == MISALIGNED


def test_append_refusals(lib):
    d = q.make_kv_desc(**GOOD)
    rope = lambda *a: q.spear_ec_kv_rope(*a)  # noqa: E731
    for change, code in (
            (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=None), INVALID),
            (dict(q_out=None), INVALID), (dict(k=ptr(1) + 2), MISALIGNED),
            (dict(q_out=ptr(5) + 8), MISALIGNED), (dict(ks=255), INVALID), (dict(qs=1000), INVALID),
            (dict(vs=-256), INVALID), (dict(ks=260), MISALIGNED), (dict(os=1028), MISALIGNED),
            (dict(q_out=ptr(0), os=2048), INVALID),
            (dict(rope=rope(None, 8, 128, 0)), INVALID), (dict(rope=rope(ptr(11), 0, 128, 0)), INVALID),
            (dict(rope=rope(ptr(11), 8, 0, 0)), INVALID),
            (dict(rope=rope(ptr(11), 8, 24, 0)), UNSUPPORTED),
            (dict(rope=rope(ptr(11), 8, 144, 0)), UNSUPPORTED),
            (dict(rope=rope(ptr(11) + 4, 8, 128, 0)), MISALIGNED)):
        assert call(lib, "append", d, batch(), **change) == code, change
        assert q.spear_ec_last_error()


def test_attention_and_dequant_refusals(lib):
    d = q.make_kv_desc(**GOOD)
    for change, code in (
            (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(out=ptr(0)), INVALID),
            (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
            (dict(scale=float("inf")), INVALID), (dict(scale=2.0 ** 65), INVALID), (dict(window=-1), INVALID),
            (dict(qs=1023), INVALID), (dict(qs=1028), MISALIGNED), (dict(q=ptr(0) + 4), MISALIGNED),
            (dict(out=ptr(6) + 2), MISALIGNED), (dict(lse=ptr(12) + 2), MISALIGNED),
            (dict(ws=None), WORKSPACE), (dict(ws=ptr(7) + 8), MISALIGNED), (dict(ws_bytes=64), WORKSPACE)):
        assert call(lib, "attention", d, batch(), **change) == code, change
    assert call(lib, "dequant", d, batch(), k_out=None) == INVALID
    assert call(lib, "dequant", d, batch(), v_out=None) == INVALID
    assert call(lib, "dequant", d, batch(), k_out=ptr(8) + 4) == MISALIGNED


def test_workspace_grows_with_the_call(lib):
    d = q.make_kv_desc(**GOOD)
    assert q.spear_ec_kv_workspace_bytes(d, -1, 1) == 0
    assert q.spear_ec_kv_workspace_bytes(d, 65537, 1) == 0
    assert q.spear_ec_kv_workspace_bytes(d, 1, (1 << 20) + 1) == 0
    sizes = [[q.spear_ec_kv_workspace_bytes(d, n, t) for t in (0, 1, 7, 64, 1000, 1 << 20)]
             for n in (0, 1, 5, 300, 65536)]
    a = np.array(sizes)
    assert (a > 0).all() and (np.diff(a, axis=0) >= 0).all() and (np.diff(a, axis=1) >= 0).all()


def test_binding_refuses_tensors_the_call_would_misread(lib):
    import torch
    d = q.make_kv_desc(**GOOD)
    codes, scales, zeros = q.alloc_kv_cache(d, "cpu")
    lens = torch.ones(2, dtype=torch.int32)
    table = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        q.make_kv_batch(None, lens.long(), table, 2)
    with pytest.raises(ValueError):
        q.make_kv_batch(torch.zeros(2, dtype=torch.int32), lens, table, 2)
    with pytest.raises(ValueError):
        q.make_kv_batch(None, lens, torch.zeros((2, 4), dtype=torch.int32)[:, ::2], 2)
    b = q.make_kv_batch(None, lens, table, 2)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    good = dict(q=bf(2, 8, 128), k=bf(2, 2, 128), v=bf(2, 2, 128), o=bf(2, 8, 128))
    for change in (dict(k=bf(1, 2, 128)), dict(k=bf(2, 2, 64)), dict(v=bf(2, 2, 128).float()),
                   dict(q=bf(2, 128, 8).transpose(1, 2)), dict(o=bf(2, 4, 128))):
        a = {**good, **change}
        with pytest.raises(ValueError):
            q.spear_ec_kv_append(d, b, a["q"], a["k"], a["v"], None, codes, scales, zeros, a["o"])
    with pytest.raises(ValueError):
        q.spear_ec_kv_append(d, b, good["q"], good["k"], good["v"], None, codes[:2], scales, zeros,
                             good["o"])
    with pytest.raises(ValueError):
        q.spear_ec_kv_attention(d, b, good["q"], codes, scales, zeros, 0.1, bf(2, 16, 128)[:, ::2],
                                None)
    wide = q.make_kv_batch(None, lens, torch.zeros((2, 3), dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        q.spear_ec_kv_attention(d, wide, good["q"], codes, scales, zeros, 0.1, good["o"], None)


    with pytest.raises(ValueError, match="on the GPU"):
        q.spear_ec_kv_attention(d, b, good["q"], codes, scales, zeros, 0.1, good["o"], None)


def test_binding_runs_on_the_cache_s_device(monkeypatch):
    """A call for tensors of another device than the current one runs with theirs current, on
    its stream."""
    import contextlib
    import torch
    seen = []

    @contextlib.contextmanager
    def device(i):
        seen.append(("enter", i))
        yield
        seen.append(("leave", i))

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    fn = lambda *a: seen.append(a) or 0  # noqa: E731
    kv._call(fn, 1, None, "x")
    kv._call(fn, 0, None, "y")
    kv._call(fn, 1, 7, "z")
    assert seen == [("enter", 1), ("x", 101), ("leave", 1), ("y", 100), ("enter", 1), ("z", 7),
                    ("leave", 1)]


# ------------------------------------------------------------- the reference
def test_reference_quantizer_by_hand():
    c, s, z = ref.quantize(np.array([7.0, -7.0, 3.5, 0.0]), False)
    assert list(c) == [15, 1, 12, 8] and s == np.float16(1).view(np.uint16) and z == 8   # 3.5 -> 4
    c, s, z = ref.quantize(np.array([-1.0, 14.0, 0.5, 2.5]), True)
    assert list(c) == [0, 15, 1, 3] and s == np.float16(1).view(np.uint16) and z == 1
    c, s, z = ref.quantize(np.zeros(4), False)
    assert list(c) == [8] * 4 and s == np.float16(1).view(np.uint16)
    assert ref.quantize(np.array([1e9, 0.0]), False)[1] == np.float16(65504).view(np.uint16)


def test_reference_layout_and_attention_by_hand():
    cache = ref.Cache(1, 64, 16, 2, True)
    table = np.array([1, 0])
    codes = np.arange(64, dtype=np.uint8) % 16
    cache.put(table, 17, 0, 0, codes, np.float16(0.5).view(np.uint16), 3)
    cache.put(table, 17, 0, 1, codes[::-1].copy(), np.float16(2).view(np.uint16), 9)
    assert cache.codes[0, 0, 0, 32] == 0x10 and cache.codes[0, 0, 0, 33] == 0x32
    assert cache.codes[0, 0, 0, 512 + 1] == 0xEF and cache.codes[0, 0, 0, 512 + 17] == 0xCD
    assert cache.zeros[0, 0, 0, 1] == 0x93
    kc, ks = cache.parts(table, 18, 0, 0, 17)
    vc, vs = cache.parts(table, 18, 0, 1, 17)
    assert np.array_equal(kc[0], codes.astype(float) - 3) and ks[0] == 0.5
    assert np.array_equal(vc[0], codes[::-1].astype(float) - 9) and vs[0] == 2
    # one attended token: its value, lse its score
    q1 = ref.f64_to_bf16(np.ones((1, 1, 64)))
    out, lse, _, _ = ref.attention(cache, q1, [0, 1], [18], [table], 0.25, window=1)
    assert np.allclose(out[0, 0], vc[0] * 2) and np.isclose(lse[0, 0], 0.25 * 0.5 * kc[0].sum())


def test_reference_rotation_keeps_length_and_position_differences():
    rng = np.random.default_rng(3)
    ang = np.outer(np.arange(40), 100.0 ** (-np.arange(16) / 16))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    a, b = rng.standard_normal((2, 64))
    for inter in (False, True):
        ra = [ref.rotate(a, p, cs, 32, inter) for p in (5, 25)]
        rb = [ref.rotate(b, p, cs, 32, inter) for p in (2, 22)]
        assert np.isclose(np.linalg.norm(ra[0]), np.linalg.norm(a))
        assert np.isclose(ra[0] @ rb[0], ra[1] @ rb[1])
        assert np.array_equal(ra[0][32:], a[32:])
