"""The 4-bit paged key/value cache on the GPU against tests/kv_reference.py
(needs an MI355X).

Stored bytes, scales, zero-points and values read back are compared bit for
bit, attention within the tolerances that kv_reference derives.  Every case
prints its sizes before it touches the GPU.  Slots that no token was stored to
hold 0xFF codes and zero-points and NaN scales, and page-table entries past a
sequence's length hold -1, so a read of either shows.
"""
from __future__ import annotations

import numpy as np
import pytest

import kv_reference as ref
import quantization_error_compensation_amd as q

pytestmark = pytest.mark.gpu


# A rotated query is evaluated in fp32 with one product's error added back (two
# roundings, at most 2 * 2^-24 of the value) and then rounded to bf16, half a step
# of which is at least 2^-9 of the value: together at most (1 + 2^-23 / 2^-9) half steps.
Q_ROUNDING = 1 + 2.0 ** -14


def note(msg):
    print(f"[case] {msg}", flush=True)


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    assert _t.cuda.is_available(), "GPU tests need a GPU"
    q.load_library()
    return _t


class Case:
    """A cache, its sequences and the same things on the device."""

    def __init__(self, torch, H, G, D, page, asym, lens, new=None, seed=0, offsets=True, extra=0,
                 q_std=1.0, pos_table=None):
        self.torch, self.H, self.G, self.D, self.page, self.asym = torch, H, G, D, page, asym
        rng = self.rng = np.random.default_rng(seed)
        self.lens = list(lens)
        self.new = list(new) if new is not None else [1] * len(lens)
        self.offsets = np.concatenate([[0], np.cumsum(self.new)]).astype(int)
        self.rows = int(self.offsets[-1]) + extra
        need = [-(-max(n, 0) // page) for n in self.lens]
        self.max_pages = max(max(need), 1) + 1
        self.pages = sum(need) + 2
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), self.max_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = ref.Cache(G, D, page, self.pages, asym, fill=0xFF)
        self.desc = q.make_kv_desc(H, G, D, page, self.pages, self.max_pages, asym)
        self.q = ref.f64_to_bf16(rng.standard_normal((self.rows, H, D)) * q_std)
        self.d_lens, self.d_table = self.dev(np.array(self.lens, np.int32)), self.dev(self.table)
        self.d_offsets = self.dev(self.offsets.astype(np.int32)) if offsets else None
        self.batch = q.make_kv_batch(self.d_offsets, self.d_lens, self.d_table, self.rows)

    def dev(self, a):
        return self.torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def bf16(self, bits):
        return self.dev(np.ascontiguousarray(bits, np.uint16).view(np.int16)).view(self.torch.bfloat16)

    def fill(self, scale_spread=0.3, value_scales=None):
        """Every token of every sequence, straight into the cache."""
        rng, c = self.rng, self.cache
        for b, n in enumerate(self.lens):
            for g in range(self.G):
                for w in (0, 1):
                    codes = np.clip(np.rint(rng.standard_normal((max(n, 0), self.D)) * 2.6 + 8), 0, 15)
                    sc = 0.38 * np.exp(scale_spread * rng.standard_normal(max(n, 0)))
                    if w == 1 and value_scales is not None:
                        sc = value_scales(n)
                    sc = sc.astype(np.float16).view(np.uint16)
                    z = rng.integers(0, 16, max(n, 0)) if self.asym else np.full(max(n, 0), 8)
                    for t in range(max(n, 0)):
                        c.put(self.table[b], t, g, w, codes[t].astype(np.uint8), sc[t], int(z[t]))
        self.upload()
        return self

    def upload(self):
        c, t = self.cache, self.torch
        self.codes = self.dev(c.codes)
        self.scales = self.dev(c.scales.view(np.int16)).view(t.float16)
        self.zeros = self.dev(c.zeros) if self.asym else None
        return self

    def attend(self, scale=None, window=0, ws=None, stream=None, d_q=None, lse=True):
        t = self.torch
        out = t.full((self.rows, self.H, self.D), 7.0, dtype=t.bfloat16, device="cuda")
        l = t.full((self.rows, self.H), 7.0, dtype=t.float32, device="cuda") if lse else None
        ws = ws if ws is not None else q.alloc_kv_workspace(self.desc, len(self.lens), self.rows)
        if stream is not None:
            stream.wait_stream(t.cuda.current_stream())
        q.spear_ec_kv_attention(self.desc, self.batch, self.bf16(self.q) if d_q is None else d_q,
                                self.codes, self.scales, self.zeros,
                                self.D ** -0.5 if scale is None else scale, out, ws, lse=l,
                                window=window, stream=stream)
        t.cuda.synchronize()
        return out, l, ws

    def check(self, out, lse, scale=None, window=0, skip=()):
        ro, rl, tol, ltol = ref.attention(self.cache, self.q, self.offsets, self.lens, self.table,
                                          self.D ** -0.5 if scale is None else scale, window)
        o = ref.bf16_to_f64(out.view(self.torch.int16).cpu().numpy().view(np.uint16))
        n = int(self.offsets[-1])
        keep = [t for t in range(n) if t not in skip]
        err = np.abs(o - ro)[keep] - tol[keep]
        assert np.isfinite(o[keep]).all(), "output not finite"
        assert err.size == 0 or err.max() <= 0, f"off by {err.max():.3g} more than allowed"
        assert (o[n:] == 7.0).all(), "rows behind the last sequence were written"
        if lse is not None:
            v = lse.cpu().numpy().astype(np.float64)
            fin = np.isfinite(rl[keep])
            assert np.array_equal(np.isneginf(v[keep]), ~fin)
            e = np.abs(v[keep] - np.where(fin, rl[keep], 0))[fin] - ltol[keep][fin]
            assert e.size == 0 or e.max() <= 0, f"lse off by {e.max():.3g} more than allowed"
            assert (v[n:] == 7.0).all()


# ------------------------------------------------------------------ append
APPENDS = [  # H, G, D, page, asym, lens, new, rope dim, interleaved
    (4, 4, 64, 16, False, [1], [1], 64, False),
    (8, 2, 128, 16, True, [17, 16, 100], [1, 1, 1], 128, False),
    (32, 8, 128, 64, False, [40, 70], [40, 7], 128, True),
    (12, 2, 64, 32, True, [33, 5, 64, 90], [33, 5, 48, 19], 32, False),
    (6, 3, 128, 16, False, [200], [131], 48, True),
    (16, 1, 128, 256, True, [300, 17], [299, 2], 0, False),
    (40, 20, 64, 16, True, [50] * 70, [1 + i % 5 for i in range(70)], 64, False),
    (8, 2, 64, 16, False, [20 + i for i in range(70)], [9 + i % 12 for i in range(70)], 32, True),
    (4, 2, 128, 32, True, [80 + i % 40 for i in range(66)], [30] * 66, 128, False),
]


@pytest.mark.parametrize("H,G,D,page,asym,lens,new,dim,inter", APPENDS)
def test_append_stores_the_reference_bytes(torch, H, G, D, page, asym, lens, new, dim, inter):
    note(f"append H={H} G={G} D={D} page={page} asym={asym} lens={lens[:4]} new={new[:4]} rope={dim} {inter}")
    c = Case(torch, H, G, D, page, asym, lens, new, seed=H + D + len(lens), extra=2)
    c.upload()
    rng = c.rng
    qkv = ref.f64_to_bf16(rng.standard_normal((c.rows, H + 2 * G, D)) * np.exp(rng.standard_normal((c.rows, 1, 1))))
    qkv[0, H, :] = 0                      # a key of zeros: scale 1
    qkv[0, H + G, 1:] = 0                 # a value with one element
    cs = None
    if dim:
        ang = np.outer(np.arange(max(lens)), 1000.0 ** (-np.arange(dim // 2) / (dim // 2)))
        cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    d = c.bf16(qkv)
    q_out = torch.full((c.rows, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    q.spear_ec_kv_append(c.desc, c.batch, d[:, :H], d[:, H:H + G], d[:, H + G:],
                         c.dev(cs) if dim else None, c.codes, c.scales, c.zeros, q_out,
                         interleaved=inter)
    torch.cuda.synchronize()
    rq = ref.append(c.cache, qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:], c.offsets, lens, c.table,
                    cs, dim, inter)
    assert np.array_equal(c.codes.cpu().numpy(), c.cache.codes)
    assert np.array_equal(c.scales.view(torch.int16).cpu().numpy().view(np.uint16), c.cache.scales)
    if asym:
        assert np.array_equal(c.zeros.cpu().numpy(), c.cache.zeros)
    n = int(c.offsets[-1])
    got = ref.bf16_to_f64(q_out.view(torch.int16).cpu().numpy().view(np.uint16))
    assert (np.abs(got - rq)[:n] <= ref.half_step_bf16(rq)[:n] * Q_ROUNDING).all()
    assert (got[n:] == 7.0).all()

    # the same rows read back: the exact values
    k = torch.full((c.rows, G, D), 7.0, dtype=torch.float32, device="cuda")
    v = torch.full_like(k, 7.0)
    q.spear_ec_kv_dequant_f32(c.desc, c.batch, c.codes, c.scales, c.zeros, k, v)
    torch.cuda.synchronize()
    for which, x in ((0, k.cpu().numpy()), (1, v.cpu().numpy())):
        for b, m in enumerate(lens):
            for g in range(G):
                codes, s = c.cache.parts(c.table[b], m, g, which, m - new[b])
                assert np.array_equal(x[c.offsets[b]:c.offsets[b + 1], g], codes * s[:, None])
        assert (x[n:] == 7.0).all()


def test_append_values_near_borders(torch):
    """Values on and next to the borders between two codes, and extremes: scales that overflow,
    underflow to 0, and are fp16 subnormals."""
    note("append borders")
    G, D = 2, 64
    for asym in (False, True):
        c = Case(torch, G, G, D, 16, asym, [48], [48], seed=5)
        c.upload()
        rng = c.rng
        x = np.zeros((48, G, D))
        for t in range(48):
            m = 2.0 ** (t % 12 - 6)
            x[t] = m * (np.arange(D) % 15 - 7 + 0.5 * (t % 3)) / 7
        x[40], x[41], x[42] = 1e38, 1e-9, rng.standard_normal((G, D)) * 1e-6
        x[43, :, 0], x[44, :, 3] = 65504 * 7.5, -2.0 ** -22
        bits = ref.f64_to_bf16(x)
        bits[45, 0, 5] = 0x7FC0                                  # NaN: code 0, no part of the maximum
        bits[46, 1, 7], bits[46, 1, 8] = 0x7F80, 0xFF80          # infinities
        d = c.bf16(bits)
        q.spear_ec_kv_append(c.desc, c.batch, None, d, d, None, c.codes, c.scales, c.zeros, None)
        torch.cuda.synchronize()
        plain = [t for t in range(48) if t not in (45, 46)]
        sub = ref.Cache(G, D, 16, c.pages, asym, fill=0xFF)
        vals = ref.bf16_to_f64(bits)
        for t in plain:
            for g in range(G):
                for w in (0, 1):
                    sub.put(c.table[0], t, g, w, *ref.quantize(vals[t, g], asym))
        codes = c.codes.cpu().numpy()
        got = ref.Cache(G, D, 16, c.pages, asym)
        got.codes, got.scales = codes, c.scales.view(torch.int16).cpu().numpy().view(np.uint16)
        if asym:
            got.zeros = c.zeros.cpu().numpy()
        for g in range(G):
            for w in (0, 1):
                a, sa = got.parts(c.table[0], 48, g, w)
                b, sb = sub.parts(c.table[0], 48, g, w)
                assert np.array_equal(a[plain], b[plain]) and np.array_equal(sa[plain], sb[plain])
                assert np.isfinite(a).all() and np.isfinite(sa).all()
                raw = a + (8 if not asym else 0)
                if not asym and g == 0:
                    assert raw[45, 5] == 0
                if g == 1:
                    assert sa[46] == 65504


def test_append_in_place_and_keys_only(torch):
    note("append in place")
    H, G, D = 4, 2, 128
    c = Case(torch, H, G, D, 16, False, [9, 30], [3, 4], seed=2)
    c.upload()
    qkv = ref.f64_to_bf16(c.rng.standard_normal((c.rows, H + 2 * G, D)))
    cs = np.concatenate([np.cos(np.outer(np.arange(30), np.arange(1, 65) / 64)),
                         np.sin(np.outer(np.arange(30), np.arange(1, 65) / 64))], 1).astype(np.float32)
    d, tab = c.bf16(qkv), c.dev(cs)
    out = torch.empty((c.rows, H, D), dtype=torch.bfloat16, device="cuda")
    q.spear_ec_kv_append(c.desc, c.batch, d[:, :H], d[:, H:H + G], d[:, H + G:], tab, c.codes, c.scales,
                         c.zeros, out)
    torch.cuda.synchronize()
    codes = c.codes.clone()
    c.upload()
    q.spear_ec_kv_append(c.desc, c.batch, d[:, :H], d[:, H:H + G], d[:, H + G:], tab, c.codes, c.scales,
                         c.zeros, d[:, :H])
    torch.cuda.synchronize()
    assert torch.equal(d[:, :H], out) and torch.equal(c.codes, codes)
    assert np.array_equal(d[:, H:].contiguous().view(torch.int16).cpu().numpy().view(np.uint16), qkv[:, H:])
    c.upload()
    q.spear_ec_kv_append(c.desc, c.batch, None, d[:, H:H + G], d[:, H + G:], tab, c.codes, c.scales,
                         c.zeros, None)
    torch.cuda.synchronize()
    assert torch.equal(c.codes, codes)


def test_append_padding_bad_pages_and_short_tables(torch):
    """Padding rows give zeros, rows without a slot NaN, and nothing else in the cache changes."""
    note("append padding and bad pages")
    H, G, D = 4, 2, 64
    c = Case(torch, H, G, D, 16, True, [2, 20, 40, 60], [5, 4, 4, 4], seed=4)
    c.upload()
    table = c.table.copy()
    table[1, 1] = c.pages                 # positions 16 .. 19 of sequence 1
    table[2, 2] = -5                      # positions 36 .. 39 of sequence 2
    c.d_table.copy_(c.dev(table))
    lens = [2, 20, 40, c.max_pages * 16 + 2]  # sequence 3: two rows past its table row
    c.d_lens.copy_(c.dev(np.array(lens, np.int32)))
    cs = np.ones((c.max_pages * 16 + 8, D), np.float32)
    bits = ref.f64_to_bf16(c.rng.standard_normal((c.rows, H, D)))
    d = c.bf16(bits)
    out = torch.full((c.rows, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    before = c.codes.clone()
    table[3, c.max_pages - 1] = c.table[3, 0]  # a page that exists for the last row of the table
    c.d_table.copy_(c.dev(table))
    q.spear_ec_kv_append(c.desc, c.batch, d, d[:, :G].contiguous(), d[:, G:2 * G].contiguous(), c.dev(cs),
                         c.codes, c.scales, c.zeros, out)
    torch.cuda.synchronize()
    o = out.float().cpu().numpy()
    assert (o[:3] == 0).all() and np.isfinite(o[3:5]).all() and (np.abs(o[3:5]).max(-1) > 0).all()
    assert np.isnan(o[5:9]).all() and np.isnan(o[9:13]).all()
    assert np.isfinite(o[13:15]).all() and np.isnan(o[15:17]).all()
    changed = (c.codes != before).any(-1).any(-1).any(-1).nonzero().flatten().tolist()
    assert set(changed) == {int(table[0, 0]), int(table[3, c.max_pages - 1])}
    # positions past the rotation's table are refused alike
    c.upload()
    c.d_table.copy_(c.dev(c.table))
    c.d_lens.copy_(c.dev(np.array([2, 20, 40, 60], np.int32)))
    q.spear_ec_kv_append(c.desc, c.batch, d, d[:, :G].contiguous(), d[:, G:2 * G].contiguous(),
                         c.dev(cs[:38]), c.codes, c.scales, c.zeros, out)
    torch.cuda.synchronize()
    o = out.float().cpu().numpy()
    assert np.isfinite(o[3:11]).all() and np.isnan(o[11:17]).all()


# --------------------------------------------------------------- attention
ATTEND = [  # H, G, D, page, asym, lens, new, window
    (1, 1, 64, 16, False, [1], [1], 0),
    (8, 1, 128, 16, True, [1, 2, 15, 16, 17], None, 0),
    (4, 4, 128, 16, False, [127, 128, 129, 333], None, 0),
    (32, 4, 64, 64, True, [511, 40, 1000], None, 0),
    (6, 2, 128, 32, True, [255, 1], None, 100),
    (16, 1, 128, 16, False, [700], [1], 1),
    (40, 2, 64, 256, False, [300, 77], None, 0),
    (128, 1, 128, 16, True, [140], [1], 0),
    (8, 2, 128, 64, False, [90, 200, 9], [9, 9, 9], 0),
    (5, 1, 64, 16, True, [64, 65, 33], [3, 1, 33], 0),
    (8, 2, 128, 16, True, [150, 70], [70, 70], 0),
    (4, 1, 128, 64, False, [200], [200], 33),
    (12, 2, 64, 32, True, [129, 300, 1], [129, 17, 1], 64),
    (2, 2, 64, 16, False, [130], [130], 0),
    (8, 8, 128, 16, False, [2000], [1], 0),
    (16, 2, 128, 128, True, [1500, 3], [5, 2], 700),
]


@pytest.mark.parametrize("H,G,D,page,asym,lens,new,window", ATTEND)
def test_attention_matches_the_definition(torch, H, G, D, page, asym, lens, new, window):
    note(f"attention H={H} G={G} D={D} page={page} asym={asym} lens={lens} new={new} window={window}")
    c = Case(torch, H, G, D, page, asym, lens, new, seed=H * 7 + D + lens[0], offsets=new is not None,
             extra=3 if new is not None else 0).fill()
    out, lse, ws = c.attend(window=window)
    c.check(out, lse, window=window)
    assert q.spear_ec_workspace_status(ws) == 0
    again, lse2, _ = c.attend(window=window, ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2), "the same call differs"


SPLITS = [  # the ways a call is cut: H, G, D, page, asym, lens, new, window
    # pieces of one size for uneven lengths
    (8, 8, 64, 16, False, [30] * 9 + [4100] + [25] * 15, None, 0),
    (8, 8, 128, 64, True, [3000, 900, 100, 1500, 2100, 1, 640, 1300, 2900, 40, 1900, 2500], None, 0),
    # more items than workgroups: runs that cross items
    (8, 8, 64, 16, False, [30 + 53 * i % 700 for i in range(40)], None, 0),
    (8, 8, 128, 16, True, [1 + 97 * i % 900 for i in range(34)], [1 + i % 2 for i in range(34)], 500),
    # more than 64 sequences: one token, a few, many rows of 128 and of 256 an item
    (8, 4, 64, 16, True, [1 + 37 * i % 300 for i in range(70)], None, 0),
    (4, 2, 128, 16, False, [40 + 11 * i % 200 for i in range(66)], [1 + i % 3 for i in range(66)], 50),
    (16, 1, 64, 16, False, [20 + 7 * i % 100 for i in range(72)], [6] * 72, 0),
    (16, 1, 64, 32, True, [9 + 5 * i % 90 for i in range(70)], [9] * 70, 0),
    # 256 rows an item: whole items, and items cut into runs, one of them short
    (128, 16, 64, 16, False, [33, 70, 49], [33, 33, 40], 0),
    (32, 32, 128, 64, True, [700, 150], [130, 130], 0),
    (32, 32, 64, 64, False, [1100, 131], [131, 131], 600),
    # 128 rows an item, many runs
    (8, 1, 128, 16, False, [1500], [17], 0),
    (8, 1, 64, 64, True, [2500, 4], [40, 4], 1300),
    # a group of 128 query heads
    (128, 1, 64, 16, False, [77, 30], [2, 3], 0),
]


@pytest.mark.parametrize("H,G,D,page,asym,lens,new,window", SPLITS)
def test_attention_however_it_is_cut(torch, H, G, D, page, asym, lens, new, window):
    note(f"attention cut H={H} G={G} D={D} page={page} asym={asym} {len(lens)} sequences {lens[:3]} "
         f"new={new and new[:3]} window={window}")
    c = Case(torch, H, G, D, page, asym, lens, new, seed=H + D + len(lens), offsets=new is not None,
             extra=2 if new is not None else 0).fill()
    out, lse, ws = c.attend(window=window)
    c.check(out, lse, window=window)
    assert q.spear_ec_workspace_status(ws) == 0
    again, lse2, _ = c.attend(window=window, ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2), "the same call differs"


@pytest.mark.parametrize("G,new", [(2, 300), (2, 2)])
def test_attention_widest_window_with_padding(torch, G, new):
    """The largest window there is takes in everything, also for rows at negative positions."""
    note(f"attention widest window new={new}")
    c = Case(torch, 4, G, 64, 16, True, [200, 150, 1], [new] * 3, seed=12).fill()
    plain = c.attend()
    wide = c.attend(window=2 ** 31 - 1)
    c.check(wide[0], wide[1])
    assert torch.equal(plain[0], wide[0]) and torch.equal(plain[1], wide[1])


@pytest.mark.parametrize("new", [1, 3, 60])
def test_cache_past_four_gigabytes(torch, new):
    """Pages whose codes lie 4 GiB and more into the array, written, attended to and read back."""
    note(f"cache past 4 GiB new={new}")
    H, G, D, page = 4, 1, 128, 256
    c = Case(torch, H, G, D, page, False, [300, 70], [new, new], seed=6).fill()
    pages = (2 ** 32 // (page * D)) + c.pages + 1       # a page's codes: page * D bytes
    up = pages - c.pages
    codes = torch.zeros((pages, *c.codes.shape[1:]), dtype=torch.uint8, device="cuda")
    scales = torch.full((pages, *c.scales.shape[1:]), float("nan"), dtype=torch.float16, device="cuda")
    assert up * page * D > 2 ** 32
    codes[up:], scales[up:] = c.codes, c.scales
    low = c.attend()
    c.desc = q.make_kv_desc(H, G, D, page, pages, c.max_pages, False)
    c.d_table.copy_(c.dev(np.where(c.table < 0, c.table, c.table + up)))
    c.codes, c.scales = codes, scales
    high = c.attend()
    c.check(high[0], high[1])
    assert torch.equal(low[0], high[0]) and torch.equal(low[1], high[1])
    kv = ref.f64_to_bf16(c.rng.standard_normal((c.rows, G, D)))
    d = c.bf16(kv)
    q.spear_ec_kv_append(c.desc, c.batch, None, d, d, None, codes, scales, None, None)
    ref.append(c.cache, np.zeros((c.rows, H, D), np.uint16), kv, kv, c.offsets, c.lens, c.table)
    k = torch.full((c.rows, G, D), 7.0, device="cuda")
    v = torch.full_like(k, 7.0)
    q.spear_ec_kv_dequant_f32(c.desc, c.batch, codes, scales, None, k, v)
    torch.cuda.synchronize()
    assert np.array_equal(codes[up:].cpu().numpy(), c.cache.codes) and not codes[:up].any()
    for b, m in enumerate(c.lens):
        for which, x in ((0, k), (1, v)):
            w, s = c.cache.parts(c.table[b], m, 0, which, m - new)
            assert np.array_equal(x[c.offsets[b]:c.offsets[b + 1], 0].cpu().numpy(), w * s[:, None])


def test_two_captured_calls_share_a_workspace(torch):
    """A call of few rows and one of many, captured with one workspace and replayed in turn,
    with eager calls on it in between."""
    note("captured calls on one workspace")
    a = Case(torch, 8, 2, 128, 16, True, [2300, 40], [1, 1], seed=21).fill()
    b = Case(torch, 8, 1, 128, 16, False, [1400], [40], seed=22).fill()
    both = [(c, c.bf16(c.q)) for c in (a, b)]
    ra, rb = a.attend(), b.attend()
    a.check(*ra[:2])
    b.check(*rb[:2])
    n = max(q.alloc_kv_workspace(c.desc, len(c.lens), c.rows).numel() for c in (a, b))
    ws = torch.zeros(n, dtype=ra[2].dtype, device="cuda")
    outs = [torch.empty_like(r[0]) for r in (ra, rb)]
    lses = [torch.empty_like(r[1]) for r in (ra, rb)]
    graphs, st = [], torch.cuda.Stream()
    torch.cuda.synchronize()
    for i, (c, x) in enumerate(both):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            q.spear_ec_kv_attention(c.desc, c.batch, x, c.codes, c.scales, c.zeros, 128 ** -0.5, outs[i],
                                    ws, lse=lses[i], stream=st)
        graphs.append(g)
    torch.cuda.synchronize()
    for turn in range(4):
        for i, r in ((0, ra), (1, rb), (0, ra)):
            outs[i].fill_(float("nan"))
            lses[i].fill_(float("nan"))
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], r[0]) and torch.equal(lses[i], r[1]), (turn, i)
            c = both[1 - i][0]
            eager = c.attend(ws=ws)
            assert torch.equal(eager[0], (ra, rb)[1 - i][0])
    assert q.spear_ec_workspace_status(ws) == 0


@pytest.mark.parametrize("new", [2, 70])
def test_offsets_that_do_not_ascend_stay_in_bounds(torch, new):
    """Such calls may leave rows out; nothing outside the outputs is touched, and the workspace
    serves the next call."""
    note(f"offsets out of order new={new}")
    c = Case(torch, 8, 2, 64, 16, True, [90, 200, 120], [new] * 3, seed=15, extra=4).fill()
    good, lse, ws = c.attend()
    rows = c.bf16(ref.f64_to_bf16(c.rng.standard_normal((c.rows, 2, 64))))
    for off in ([0, 2 * new, new, 3 * new], [3 * new, 0, 3 * new, 0], [-5, 10 ** 9, -(10 ** 9), 2 ** 31 - 1],
                [0, 3 * new, 3 * new, 3 * new]):
        note(f"  {off}")
        c.d_offsets.copy_(c.dev(np.array(off, np.int32)))
        c.attend(ws=ws)
        back = torch.zeros((c.rows, 2, 64), device="cuda")
        q.spear_ec_kv_dequant_f32(c.desc, c.batch, c.codes, c.scales, c.zeros, back, back.clone())
        q.spear_ec_kv_append(c.desc, c.batch, None, rows, rows, None, c.codes.clone(), c.scales.clone(),
                             c.zeros.clone(), None)
        torch.cuda.synchronize()
        q.spear_ec_workspace_status(ws)
        c.d_offsets.copy_(c.dev(c.offsets.astype(np.int32)))
        again, lse2, _ = c.attend(ws=ws)
        assert torch.equal(good, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new,H,G", [(1, 8, 2), (6, 8, 2), (40, 8, 2), (40, 256, 32)])
def test_attention_empty_and_padded_rows(torch, new, H, G):
    """Sequences of length 0, padding rows, no rows, and rows behind the last sequence."""
    note(f"attention empty rows new={new} H={H} G={G}")
    c = Case(torch, H, G, 64, 16, True, [0, 3, 60, 0, 20], [new, new, new, 0, 1], seed=new, extra=5).fill()
    out, lse, ws = c.attend()
    c.check(out, lse)
    o = out.float()
    assert (o[:new] == 0).all() and torch.isneginf(lse[:new]).all()
    assert q.spear_ec_workspace_status(ws) == 0


@pytest.mark.parametrize("H,G,D,new", [(8, 2, 128, 1), (4, 1, 64, 20), (16, 2, 128, 9), (64, 16, 64, 50)])
def test_attention_peaks_and_value_scales(torch, H, G, D, new):
    """Scores from flat to a single peak, a first token with tiny values that takes most of the
    weight, scales over many powers of two, and softmax scales far from 1 / sqrt(D)."""
    note(f"attention peaks H={H} G={G} D={D} new={new}")
    spread = lambda n: np.exp(6 * np.random.default_rng(n).standard_normal(n)).clip(1e-4, 2e4)  # noqa: E731

    def sink(n):
        s = np.full(n, 0.5)
        s[0] = 1e-3
        return s

    for seed, (vs, std, scale) in enumerate(((None, 0.0, None), (None, 6.0, None), (sink, 3.0, None),
                                             (spread, 1.0, None), (spread, 1.0, 1e-3),
                                             (None, 1.0, 2.0))):
        note(f"  spread {seed}")
        c = Case(torch, H, G, D, 16, seed % 2 == 1, [400, 129], [new, new], seed=40 + seed, q_std=std)
        c.fill(value_scales=vs)
        out, lse, _ = c.attend(scale=scale)
        c.check(out, lse, scale=scale)


def test_attention_query_extremes_stay_in_their_row(torch):
    note("attention query extremes")
    c = Case(torch, 4, 2, 128, 16, False, [70, 70, 300], [1, 3, 20], seed=9)
    c.q[0, 1, 5] = 0x7F80                 # infinity
    c.q[2, 0, 0] = 0x7FC0                 # NaN
    c.q[10, 3, 9] = 0xFF80
    c.q[3] = 0                            # zeros: the mean of the values
    c.q[5] = ref.f64_to_bf16(np.full((4, 128), 2.0 ** -120))
    c.q[6] = ref.f64_to_bf16(c.rng.standard_normal((4, 128)) * 2.0 ** np.arange(128) * 2.0 ** -120)
    c.fill()
    out, lse, _ = c.attend()
    o = out.float().cpu().numpy()
    for t, h in ((0, 1), (2, 0), (10, 3)):
        assert np.isnan(o[t, h]).all()
        c.q[t, h] = 0
    mask = np.ones(o.shape[:2], bool)
    for t, h in ((0, 1), (2, 0), (10, 3)):
        mask[t, h] = False
    ro, _, tol, _ = ref.attention(c.cache, c.q, c.offsets, c.lens, c.table, 128 ** -0.5)
    assert (np.abs(o - ro) <= tol)[mask].all()


@pytest.mark.parametrize("new,H,G", [(1, 8, 2), (9, 8, 2), (50, 8, 2), (50, 64, 16)])
def test_attention_bad_pages_give_nan_and_the_error_bit(torch, new, H, G):
    """Page numbers outside the cache and sequences longer than their page-table row: NaN in the
    rows that attend to them, the workspace's error bit, and nothing else touched."""
    note(f"attention bad pages new={new} H={H} G={G}")
    c = Case(torch, H, G, 128, 16, True, [200, 90, 100, 70], [new] * 4, seed=new).fill()
    good = c.table.copy()
    bad = good.copy()
    bad[0, 3] = c.pages
    bad[2, 1] = -7
    c.d_table.copy_(c.dev(bad))
    out, lse, ws = c.attend()
    assert q.spear_ec_workspace_status(ws) == q.SPEAR_EC_WS_BAD_PAGE
    assert q.spear_ec_workspace_status(ws) == 0
    o = out.float()
    assert torch.isnan(o[:new]).all() and torch.isnan(o[2 * new:3 * new]).all()
    skip = set(range(new)) | set(range(2 * new, 3 * new))
    c.check(out, lse, skip=skip)
    # a window that leaves the bad pages out (positions 48 .. 63 and 16 .. 31; with 50 rows
    # sequence 2's first is at position 50): the rows are whole again
    c.check(*c.attend(window=18, ws=ws)[:2], window=18)
    assert q.spear_ec_workspace_status(ws) == 0
    # a sequence longer than its row of the table
    c.d_table.copy_(c.dev(good))
    c.d_lens[1] = c.max_pages * 16 + new
    out, lse, _ = c.attend(ws=ws)
    assert torch.isnan(out[new:2 * new].float()).all()
    c.check(out, lse, skip=set(range(new, 2 * new)))
    assert q.spear_ec_workspace_status(ws) == q.SPEAR_EC_WS_BAD_PAGE


def test_attention_strided_queries_and_no_lse(torch):
    note("attention strided queries")
    H, G, D = 8, 2, 64
    c = Case(torch, H, G, D, 32, True, [100, 45], [4, 30], seed=3).fill()
    wide = torch.zeros((c.rows, H + 2 * G, D), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = c.bf16(c.q)
    out, _, _ = c.attend(d_q=wide[:, :H], lse=False)
    c.check(out, None)


def test_tensors_of_the_host_are_refused(torch):
    note("tensors of the host")
    c = Case(torch, 4, 2, 64, 16, True, [20, 7], [1, 1], seed=1).fill()
    x, out = c.bf16(c.q), torch.empty((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    kv = x[:, :2].contiguous()
    ws = q.alloc_kv_workspace(c.desc, 2, 2)
    cs = torch.zeros((30, 64), device="cuda")
    cache = (c.codes, c.scales, c.zeros)

    def attend(x=x, cache=cache, out=out, ws=ws, lse=None):
        q.spear_ec_kv_attention(c.desc, c.batch, x, *cache, 0.1, out, ws, lse=lse)

    def append(x=x, k=kv, cs=cs, out=out):
        q.spear_ec_kv_append(c.desc, c.batch, x, k, kv, cs, *cache, out)

    attend()
    append()
    for f, kw in ((attend, dict(x=x.cpu())), (attend, dict(out=out.cpu())), (attend, dict(ws=ws.cpu())),
                  (attend, dict(lse=torch.zeros(2, 4))), (attend, dict(cache=(c.codes, c.scales.cpu(), c.zeros))),
                  (attend, dict(cache=tuple(t.cpu() for t in cache))), (append, dict(x=x.cpu())),
                  (append, dict(k=kv.cpu())), (append, dict(cs=cs.cpu())), (append, dict(out=out.cpu()))):
        with pytest.raises(ValueError):
            f(**kw)
    with pytest.raises(ValueError):
        q.spear_ec_kv_dequant_f32(c.desc, c.batch, *cache, kv.float(), kv.float().cpu())
    with pytest.raises(ValueError):
        q.make_kv_batch(c.d_offsets, c.d_lens.cpu(), c.d_table, 2)
    torch.cuda.synchronize()


def test_attention_on_two_streams_at_once(torch):
    note("attention on two streams")
    a = Case(torch, 8, 2, 128, 16, True, [900, 333], [1, 1], seed=1).fill()
    b = Case(torch, 8, 2, 128, 16, False, [150], [100], seed=2).fill()
    ra, rb = a.attend()[:2], b.attend()[:2]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wb = (q.alloc_kv_workspace(c.desc, len(c.lens), c.rows) for c in (a, b))
    qa, qb = a.bf16(a.q), b.bf16(b.q)
    oa, ob = torch.empty_like(ra[0]), torch.empty_like(rb[0])
    torch.cuda.synchronize()
    for _ in range(5):
        q.spear_ec_kv_attention(a.desc, a.batch, qa, a.codes, a.scales, a.zeros, 128 ** -0.5, oa, wa, stream=s1)
        q.spear_ec_kv_attention(b.desc, b.batch, qb, b.codes, b.scales, b.zeros, 128 ** -0.5, ob, wb, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(oa, ra[0]) and torch.equal(ob, rb[0])


def test_captured_decode_step_follows_its_batch(torch):
    """Append and attention captured once, replayed for several steps while the lengths, the
    page table and the token rows change, with eager calls on the same workspace in between."""
    note("captured decode step")
    H, G, D, page = 8, 2, 128, 16
    start = [5, 130, 31, 0]
    steps = 4
    c = Case(torch, H, G, D, page, True, [n + steps + 1 for n in start], seed=8, offsets=False)
    c.lens = list(start)
    c.fill()
    ang = np.outer(np.arange(200), 10000.0 ** (-np.arange(64) / 64))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    tab = c.dev(cs)
    rows = [ref.f64_to_bf16(c.rng.standard_normal((4, H + 2 * G, D))) for _ in range(steps + 1)]
    x = c.bf16(rows[0])
    q_rot = torch.empty((4, H, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q_rot)
    lse = torch.empty((4, H), dtype=torch.float32, device="cuda")
    ws = q.alloc_kv_workspace(c.desc, 4, 4)

    def step(st):
        q.spear_ec_kv_append(c.desc, c.batch, x[:, :H], x[:, H:H + G], x[:, H + G:], tab, c.codes,
                             c.scales, c.zeros, q_rot, stream=st)
        q.spear_ec_kv_attention(c.desc, c.batch, q_rot, c.codes, c.scales, c.zeros, D ** -0.5, out, ws,
                                lse=lse, stream=st)

    def verify(i):
        r = rows[i]
        qr = ref.append(c.cache, r[:, :H], r[:, H:H + G], r[:, H + G:], range(5), c.lens, c.table, cs,
                        D, False)
        assert np.array_equal(c.codes.cpu().numpy(), c.cache.codes), f"stored codes, step {i}"
        got = q_rot.view(torch.int16).cpu().numpy().view(np.uint16)
        assert (np.abs(ref.bf16_to_f64(got) - qr) <= ref.half_step_bf16(qr) * Q_ROUNDING).all()
        c.q = got
        c.check(out, lse)

    c.lens = [n + 1 for n in start]
    c.d_lens.copy_(c.dev(np.array(c.lens, np.int32)))
    step(None)
    torch.cuda.synchronize()
    verify(0)
    cap, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cap):
        step(cap)
    torch.cuda.synchronize()
    other = Case(torch, H, G, D, page, True, [400, 20, 3, 77], seed=19, offsets=False).fill()
    for i in range(1, steps + 1):
        note(f"  replay {i}")
        c.lens = [n + 1 for n in c.lens]
        c.d_lens.copy_(c.dev(np.array(c.lens, np.int32)))
        x.copy_(c.bf16(rows[i]))
        o2, l2, _ = other.attend(ws=ws)     # eager, on the captured call's workspace
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        verify(i)
        other.check(o2, l2)


def test_decode_layer_from_projection_to_projection(torch):
    """The operators as a serving step uses them: the 4-bit layer's qkv projection, append,
    attention and the output projection, prompts first, then tokens one at a time."""
    import oracle
    import synth
    from helpers import check_bf16_output, from_dev_u16, to_dev_bf16, to_dev_f32
    note("decode layer")
    H, G, D, page = 4, 2, 64, 16
    hid = 256
    s_in = synth.small_spec(hid, (H + 2 * G) * D, 16, 128, True, seed_base=61000)
    s_out = synth.small_spec(H * D, hid, 16, 128, True, seed_base=62000)
    layers = []
    for s in (s_in, s_out):
        W = synth.weights(s) * 4
        A, B, g, b = synth.compensator(s)
        d = q.make_desc(s.d_in, s.d_out, 16, 128, True)
        wq, sc, zs = q.alloc_packed(d)
        q.spear_ec_quantize_rtn(d, to_dev_f32(W), wq, sc, zs)
        layers.append((d, (wq, sc, zs, to_dev_bf16(A), to_dev_bf16(B), to_dev_f32(g), to_dev_f32(b)),
                       oracle.quantize_rtn(W, 128, True), (A, B, g, b)))
    ang = np.outer(np.arange(80), 10000.0 ** (-np.arange(D // 2) / (D // 2)))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    tab = torch.from_numpy(cs).cuda()
    final = [44, 26]
    c = Case(torch, H, G, D, page, True, final, [1, 1], seed=77)
    c.upload()
    rng = c.rng

    def linear(i, x, T):
        d, w, _, _ = layers[i]
        y = torch.empty((T, d.d_out), dtype=torch.bfloat16, device="cuda")
        q.spear_ec_linear(d, x, *w, 1.0, y, q.alloc_workspace(d, T))
        return y

    for new, lens in (([40, 22], [40, 22]), ([1, 1], [41, 23]), ([2, 2], [43, 25]), ([1, 1], final)):
        T = sum(new)
        off = np.concatenate([[0], np.cumsum(new)])
        x = ref.f64_to_bf16(rng.standard_normal((T, hid)))
        qkv = linear(0, c.bf16(x), T).view(T, H + 2 * G, D)
        batch = q.make_kv_batch(c.dev(off.astype(np.int32)), c.dev(np.array(lens, np.int32)), c.d_table, T)
        q_rot = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
        att = torch.empty_like(q_rot)
        q.spear_ec_kv_append(c.desc, batch, qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:], tab, c.codes,
                             c.scales, c.zeros, q_rot)
        q.spear_ec_kv_attention(c.desc, batch, q_rot, c.codes, c.scales, c.zeros, D ** -0.5, att,
                                q.alloc_kv_workspace(c.desc, 2, T))
        y = linear(1, att.view(T, H * D), T)
        torch.cuda.synchronize()
        bits = qkv.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
        yref = oracle.forward(x, *layers[0][2], *layers[0][3], 1.0, 128)
        ok, st = check_bf16_output(bits.reshape(T, -1), yref)
        assert ok, st
        ref.append(c.cache, bits[:, :H], bits[:, H:H + G], bits[:, H + G:], off, lens, c.table, cs, D, False)
        assert np.array_equal(c.codes.cpu().numpy(), c.cache.codes)
        qb = q_rot.view(torch.int16).cpu().numpy().view(np.uint16)
        ro, _, tol, _ = ref.attention(c.cache, qb, off, lens, c.table, D ** -0.5)
        ab = att.view(torch.int16).cpu().numpy().view(np.uint16)
        assert (np.abs(ref.bf16_to_f64(ab) - ro) <= tol).all()
        yref = oracle.forward(ab.reshape(T, -1), *layers[1][2], *layers[1][3], 1.0, 128)
        ok, st = check_bf16_output(from_dev_u16(y), yref)
        assert ok, st
