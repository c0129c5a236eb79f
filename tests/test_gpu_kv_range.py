"""The key/value cache over the whole range of what it may hold: value scales
far apart within a block of 16 tokens, queries far apart within a call,
scores past fp32's integers, padding rows of any content, and infinities that
meet a rotation (needs an MI355X).

Attention is held to what include/spear_ec_kv.h states, with u = 2^-24,
p_j = exp(S_j - m) / l, s_j the value's scale and v_j its codes less z:
  * a score is a sum of D products of q with codes up to 15, less z times the
    sum of q, in fp32, and a few products: |dS| <= (D + 16) u scale s 30 sum|q|;
    p_j is off by twice the largest dS and by exp's and its argument's rounding,
    under 2^-18;
  * a probability and a value are rounded to fp16, 2^-11 of themselves each:
    2^-10 + 2^-22 together;
  * O's sum, in fp32, runs over products with codes and zero-points up to 15
    apart: (n / 16 + 64) u 30 sum p_j s_j;
  * in calls of many rows a p_j s_j is no finer than u times the row's largest:
    weights start at 2^7 and lose at most half of fp16's smallest step, 2^-25,
    for values of up to 2^8 times their token's scale: 2^-25 2^8 / 2^7;
  * in calls of few rows a p_j s_j is no finer than 2^-38 of the row's largest
    p_j times its largest s_j;
  * the output is rounded once to bf16.
"""
from __future__ import annotations

import numpy as np
import pytest

import kv_reference as ref
import quantization_error_compensation_amd as q
from test_gpu_kv import Case, note, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def expected(c, few, scale=None, window=0):
    """(out, lse, tolerance of out, of lse) of a case, by the definition."""
    scale = c.D ** -0.5 if scale is None else scale
    x = ref.bf16_to_f64(c.q)
    T, H, D = x.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    tol, ltol = np.zeros((T, H, D)), np.zeros((T, H))
    R = H // c.G
    for b, length in enumerate(c.lens):
        n = int(c.offsets[b + 1] - c.offsets[b])
        real = np.arange(max(0, n - length), n)          # rows that are no padding
        pos = length - n + real[:, None]
        j = np.arange(length)
        seen = (j <= pos) & (j > pos - window if window else True)
        seen = np.repeat(seen, R, 0)
        for g in range(c.G if len(real) else 0):
            kc, ks = c.cache.parts(c.table[b], length, g, 0)
            vc, vs = c.cache.parts(c.table[b], length, g, 1)
            rows = np.ix_(c.offsets[b] + real, np.arange(g * R, (g + 1) * R))
            xr = x[rows].reshape(-1, D)
            with np.errstate(invalid="ignore", over="ignore"):
                S = np.where(seen, (xr @ kc.T) * ks * scale, -np.inf)
                top = S.max(1)
                e = np.exp(S - top[:, None])
            l = e.sum(1)
            p = e / l[:, None]
            pv = p * vs
            o = pv @ vc
            ls = top + np.log(l)
            dS = scale * np.where(seen, ks, 0).max(1) * (D + 16) * ref.U * 30 * np.abs(xr).sum(1)
            second = np.partition(S, -2, 1)[:, -2] if length > 1 else np.full(len(S), -np.inf)
            # one token has all the weight whatever the scores' errors: p is 1 and 0
            dp = np.where(top - second - 2 * dS > 100, 0.0, 2 * dS)[:, None]
            t = ((dp + 2.0 ** -10 + 2.0 ** -22 + 2.0 ** -18) * (pv @ np.abs(vc))
                 + ((seen.sum(1) / 16 + 64) * ref.U * 30 * pv.sum(1))[:, None])
            floor = 2.0 ** -38 * p.max(1) * np.where(seen, vs, 0).max(1) if few else ref.U * pv.max(1)
            t += floor[:, None] * (seen.astype(float) @ np.abs(vc))
            t += ref.half_step_bf16(np.abs(o) + t)
            shape = (len(real), R)
            out[rows], tol[rows] = o.reshape(*shape, D), t.reshape(*shape, D)
            lse[rows], ltol[rows] = ls.reshape(shape), (dS + 2.0 ** -20 * (1 + np.abs(ls))).reshape(shape)
    return out, lse, tol, ltol


def check(c, out, lse, few, skip=(), scale=None, window=0):
    ro, rl, tol, ltol = expected(c, few, scale, window)
    o = ref.bf16_to_f64(out.view(c.torch.int16).cpu().numpy().view(np.uint16))
    v = lse.cpu().numpy().astype(np.float64)
    keep = [t for t in range(int(c.offsets[-1])) if t not in skip]
    assert np.isfinite(o[keep]).all(), "output not finite"
    err = np.abs(o - ro)[keep]
    worst = (err - tol[keep]).max()
    assert worst <= 0, f"off by {worst:.3g} more than allowed"
    none = np.isneginf(rl[keep])
    assert np.array_equal(np.isneginf(v[keep]), none)
    e = np.abs(v[keep] - np.where(none, 0, rl[keep]))[~none] - ltol[keep][~none]
    assert e.size == 0 or e.max() <= 0, f"lse off by {e.max():.3g} more than allowed"


# ------------------------------------------------------------ value scales
CALLS = [  # H, G, D, page, asym, lens, new, window, few rows' kernel
    (8, 2, 64, 16, True, [90, 33], [3, 2], 0, True),
    (4, 1, 128, 16, False, [70, 20], [6, 20], 0, True),
    (8, 1, 128, 16, False, [40, 90], [40, 40], 0, False),     # 128 rows an item
    (8, 1, 64, 32, True, [130], [70], 50, False),
    (16, 1, 128, 16, True, [1100], [17], 0, False),           # cut into runs
    (32, 32, 64, 16, False, [130, 131], [130, 131], 0, False),  # 256 rows an item
    (32, 32, 128, 64, True, [140, 130], [130, 130], 70, False),
]


def scales(kind):
    def later(n):               # a larger one that the block's first rows do not see
        s = np.full(n, 2.0 ** -14)
        s[5::16] = 2.0 ** 12
        return s

    def ratios(n):              # two scales a block, 1 to 26 powers of two apart
        s = np.full(n, 2.0 ** -12)
        at = np.arange(n)
        s[at % 16 == 11] *= 2.0 ** (1 + at[at % 16 == 11] // 16 % 26)
        return s

    def wild(n):                # every fp16 exponent, subnormal scales among them
        return np.exp2(np.random.default_rng(n).uniform(-24, 15.9, n))

    def blocks(n):              # alike in a block, far apart from block to block
        r = np.random.default_rng(n)
        return np.exp2(r.uniform(-14, 12, n // 16 + 1))[np.arange(n) // 16] * r.uniform(0.3, 1, n)
    return {"later": later, "ratios": ratios, "wild": wild, "blocks": blocks}[kind]


@pytest.mark.parametrize("kind", ["later", "ratios", "wild", "blocks"])
@pytest.mark.parametrize("H,G,D,page,asym,lens,new,window,few", CALLS)
def test_value_scales_far_apart(torch, H, G, D, page, asym, lens, new, window, few, kind):  # noqa: F811
    note(f"scales {kind} H={H} G={G} D={D} asym={asym} lens={lens} new={new} window={window}")
    c = Case(torch, H, G, D, page, asym, lens, new, seed=D + H).fill(value_scales=scales(kind))
    out, lse, ws = c.attend(window=window)
    check(c, out, lse, few, window=window)
    again, lse2, _ = c.attend(window=window, ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2), "the same call differs"


@pytest.mark.parametrize("bits", [13, 20, 26])
@pytest.mark.parametrize("H,G,D,page,asym,lens,new,window,few", CALLS)
def test_value_scales_that_no_weight_meets(torch, H, G, D, page, asym, lens, new, window, few, bits):  # noqa: F811
    """Every fifth token has scales 2^bits times the others' and scores so low that its weight is
    nothing (2^-40 and less): the row is its neighbours' alone."""
    note(f"scales without weight 2^{bits} H={H} G={G} D={D} asym={asym} lens={lens} new={new}")

    def vs(n):
        s = np.full(n, 2.0 ** -14)
        s[2::5] *= 2.0 ** bits
        return s

    c = Case(torch, H, G, D, page, asym, lens, new, seed=D + bits)
    c.q = ref.f64_to_bf16(1 + 0.3 * c.rng.standard_normal((c.rows, H, D)))
    c.fill(value_scales=vs)
    for b, n in enumerate(lens):
        for g in range(G):
            codes, s = c.cache.parts(c.table[b], n, g, 0)
            for t in range(2, n, 5):
                c.cache.put(c.table[b], t, g, 0, np.zeros(D, np.uint8), np.float16(1.0).view(np.uint16),
                            15 if asym else 8)
    c.upload()
    out, lse, _ = c.attend(window=window)
    check(c, out, lse, few, window=window)


@pytest.mark.parametrize("H,G,D,page,asym,lens,new,window,few", CALLS)
def test_vectors_of_zeros_beside_small_values(torch, H, G, D, page, asym, lens, new, window, few):  # noqa: F811
    """As the append stores them: a vector of zeros has scale 1, whatever stands next to it."""
    note(f"zeros beside small values H={H} G={G} D={D} asym={asym} lens={lens} new={new}")
    c = Case(torch, H, G, D, page, asym, lens, lens, seed=D)
    c.upload()
    kv = c.rng.standard_normal((c.rows, 2 * G, D))
    kv[:, G:] *= 1e-3
    kv[3::7, G:] = 0
    bits = ref.f64_to_bf16(kv)
    d = c.bf16(bits)
    q.spear_ec_kv_append(c.desc, c.batch, None, d[:, :G], d[:, G:], None, c.codes, c.scales, c.zeros, None)
    ref.append(c.cache, np.zeros((c.rows, H, D), np.uint16), bits[:, :G], bits[:, G:], c.offsets, lens, c.table)
    torch.cuda.synchronize()
    assert np.array_equal(c.codes.cpu().numpy(), c.cache.codes)
    c.new = list(new)
    c.offsets = np.concatenate([[0], np.cumsum(new)]).astype(int)
    c.rows = int(c.offsets[-1])
    c.q = c.q[:c.rows]
    c.d_offsets = c.dev(c.offsets.astype(np.int32))
    c.batch = q.make_kv_batch(c.d_offsets, c.d_lens, c.d_table, c.rows)
    out, lse, _ = c.attend(window=window)
    check(c, out, lse, few, window=window)


# ------------------------------------------------------------ query rows
@pytest.mark.parametrize("big", [2.0 ** 20, 2.0 ** 34, 2.0 ** 40, 1e30, 3e38])
@pytest.mark.parametrize("H,G,D,page,asym,lens,new,window,few", CALLS)
def test_a_large_query_row_stays_alone(torch, H, G, D, page, asym, lens, new, window, few, big):  # noqa: F811
    """One (token, head) of each sequence is `big` times the others, one token 2^-40 of them: the
    others' results are theirs alone."""
    note(f"query row of {big:g} H={H} G={G} D={D} lens={lens} new={new}")
    c = Case(torch, H, G, D, page, asym, lens, new, seed=D + 3).fill()
    x = ref.bf16_to_f64(c.q)
    rows = [int(o) + n // 2 for o, n in zip(c.offsets, new)]
    x[[int(o) + n - 1 for o, n in zip(c.offsets, new)]] *= 2.0 ** -40
    for t in rows:
        x[t, H - 1] = np.clip(x[t, H - 1] * big, -3.3e38, 3.3e38)
    c.q = ref.f64_to_bf16(x)
    out, lse, _ = c.attend(window=window)
    ro, rl, tol, ltol = expected(c, few, window=window)
    o = ref.bf16_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16))
    v = lse.cpu().numpy().astype(np.float64)
    keep = np.ones(o.shape[:2], bool)
    keep[rows, H - 1] = False
    assert np.isfinite(o[keep]).all() and np.isfinite(v[keep]).all()
    assert (np.abs(o - ro) - tol)[keep].max() <= 0
    assert (np.abs(v - rl) - ltol)[keep].max() <= 0


@pytest.mark.parametrize("what", [1e30, 3e38, float("inf"), float("nan")])
@pytest.mark.parametrize("H,G,D,new,few", [(8, 2, 64, 6, True), (8, 1, 128, 40, False),
                                           (32, 32, 64, 140, False), (32, 32, 128, 140, False)])
def test_padding_rows_hold_anything(torch, H, G, D, new, few, what):  # noqa: F811
    """Rows at negative positions: zeros and -inf, and nothing of them in the rows beside them."""
    note(f"padding of {what} H={H} G={G} D={D} new={new}")
    c = Case(torch, H, G, D, 16, False, [3, new - 1, new + 9], [new] * 3, seed=D).fill()
    pad = [t for b, n in enumerate(c.lens) for t in range(c.offsets[b], c.offsets[b] + max(0, new - n))]
    x = torch.full((c.rows, H, D), what, device="cuda", dtype=torch.bfloat16)
    keep = [t for t in range(c.rows) if t not in pad]
    x[keep] = c.bf16(c.q)[keep]
    c.q[pad] = 0
    out, lse, ws = c.attend(d_q=x)
    check(c, out, lse, few)
    assert (out[pad] == 0).all() and torch.isneginf(lse[pad]).all()
    assert q.spear_ec_workspace_status(ws) == 0


@pytest.mark.parametrize("bits", [20, 24, 30, 40, 90])
@pytest.mark.parametrize("H,G,D,page,asym,lens,new,window,few", CALLS)
def test_scores_too_large_for_digits_below_one(torch, H, G, D, page, asym, lens, new, window, few, bits):  # noqa: F811
    """Rows of 2^bits beside ordinary ones, value scales alike and far apart: where two tokens'
    scores differ by more than their errors, the larger has all the weight."""
    note(f"scores of 2^{bits} H={H} G={G} D={D} lens={lens} new={new}")
    for kind in (None, "wild"):
        c = Case(torch, H, G, D, page, asym, lens, new, seed=D + bits)
        c.fill(value_scales=kind and scales(kind))
        x = ref.bf16_to_f64(c.q)
        x[::3, ::2] *= 2.0 ** bits
        x[1::3] -= 2.0 ** (bits - 6)       # of every score far below zero, or far above
        c.q = ref.f64_to_bf16(x)
        out, lse, ws = c.attend(window=window)
        check(c, out, lse, few, window=window)
        again, lse2, _ = c.attend(window=window, ws=ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2), "the same call differs"


# ------------------------------------------------------- rotated infinities
def quantize(x, asym):
    """ref.quantize for vectors with infinities and NaN: a NaN is no part of the
    maxima and becomes code 0."""
    f = np.where(np.isnan(x), 0.0, x)
    lo, hi = min(0.0, f.min()), max(0.0, f.max())
    with np.errstate(over="ignore", invalid="ignore"):
        s = min(np.float16((hi - lo) / 15.0 if asym else max(hi, -lo) / 7.0), np.float16(65504.0))
        s = s if s != 0 else np.float16(1.0)
        z = float(np.clip(np.rint(-lo / float(s)), 0, 15)) if asym else 8.0
        codes = np.clip(np.rint(x / float(s)) + z, 0, 15)
    return np.where(np.isnan(x), 0, codes).astype(np.uint8), s.view(np.uint16), int(z)


@pytest.mark.parametrize("n", [5, 40])          # by rows, and by blocks of positions
@pytest.mark.parametrize("D,dim", [(64, 64), (128, 128), (128, 48)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("asym", [False, True])
def test_infinities_that_meet_a_rotation(torch, n, D, dim, inter, asym):  # noqa: F811
    """Keys and queries with an infinity in either half of a pair, in both, with a NaN, and with
    values whose products leave fp32 by the table's factors: what 64-bit arithmetic gives."""
    note(f"rotated infinities n={n} D={D} dim={dim} interleaved={inter} asym={asym}")
    H, G = 4, 2
    c = Case(torch, H, G, D, 16, asym, [n + 3], [n], seed=n + D)
    c.upload()
    ang = np.outer(np.arange(n + 3), 100.0 ** (-np.arange(dim // 2) / (dim // 2))) + 0.1
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    cs[n // 2 + 3:] *= 1.5                       # tables may carry a factor
    x = c.rng.standard_normal((n, H + 2 * G, D))
    a, b = (0, 1) if inter else (0, dim // 2)    # a pair
    bits = ref.f64_to_bf16(x)
    inf, ninf, nan, most = 0x7F80, 0xFF80, 0x7FC0, 0x7F7F
    step = 2 if inter else 1
    plan = [[(a, inf)], [(b, ninf)], [(a, inf), (b, inf)], [(a, ninf), (b + 2 * step, nan)],
            [(a + step, most), (b + step, most)]]
    for t in range(n):
        for h in range(0, H + G):
            if (t + h) % 3 == 0:
                for d, w in plan[(t + h) // 3 % len(plan)]:
                    bits[t, h, d] = w
    bits[n - 1, :H + G, a], bits[n - 1, :H + G, b] = most, most     # 3.4e38 times 1.5
    bits[n - 2, :H + G, a], bits[n - 2, :H + G, b] = most | 0x8000, most
    d = c.bf16(bits)
    out = torch.full((n, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    q.spear_ec_kv_append(c.desc, c.batch, d[:, :H], d[:, H:H + G], d[:, H + G:], c.dev(cs), c.codes, c.scales,
                         c.zeros, out, interleaved=inter)
    torch.cuda.synchronize()
    v = ref.bf16_to_f64(bits)
    got = ref.bf16_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16))
    for i in range(n):
        with np.errstate(invalid="ignore"):
            want = ref.rotate(v[i, :H], 3 + i, cs, dim, inter)
            kr = ref.rotate(v[i, H:H + G], 3 + i, cs, dim, inter)
        big = np.abs(want) > 3.3961775e38        # past the largest bf16 and half a step
        fin = np.isfinite(want) & ~big
        assert np.array_equal(np.isnan(got[i]), np.isnan(want)), i
        assert np.array_equal(got[i][np.isinf(want)], want[np.isinf(want)]), i
        assert (np.isinf(got[i][big]) & (np.sign(got[i][big]) == np.sign(want[big]))).all(), i
        assert (np.abs(got[i][fin] - want[fin]) <= ref.half_step_bf16(want[fin]) * (1 + 2.0 ** -14)).all(), i
        for g in range(G):
            c.cache.put(c.table[0], 3 + i, g, 0, *quantize(kr[g], asym))
            c.cache.put(c.table[0], 3 + i, g, 1, *quantize(v[i, H + G + g], asym))
    assert np.array_equal(c.scales.view(torch.int16).cpu().numpy().view(np.uint16), c.cache.scales)
    assert np.array_equal(c.codes.cpu().numpy(), c.cache.codes)
    if asym:
        assert np.array_equal(c.zeros.cpu().numpy(), c.cache.zeros)


@pytest.mark.parametrize("kind", ["later", "wild"])
@pytest.mark.parametrize("H,G,D,asym,new,few", [(4, 2, 64, True, 3, True), (8, 2, 128, False, 2, True),
                                                (8, 1, 64, False, 9, False), (16, 1, 128, True, 10, False),
                                                (64, 4, 64, True, 17, False), (64, 4, 128, False, 17, False)])
def test_more_than_64_sequences(torch, H, G, D, asym, new, few, kind):  # noqa: F811
    """Scales far apart, a large row and garbage in padding, in calls whose lengths do not fit a wave."""
    note(f"70 sequences {kind} H={H} G={G} D={D} new={new}")
    lens = [new - 1 if i % 9 == 4 else new + 7 * i % 60 for i in range(70)]
    c = Case(torch, H, G, D, 16, asym, lens, [new] * 70, seed=D + new).fill(value_scales=scales(kind))
    pad = [int(c.offsets[b]) for b, n in enumerate(lens) if n < new]
    x = ref.bf16_to_f64(c.q)
    x[2 * new - 1::new * 5, 0] *= 2.0 ** 40
    c.q = ref.f64_to_bf16(x)
    d_q = c.bf16(c.q)
    d_q[pad] = 3e38
    c.q[pad] = 0
    out, lse, ws = c.attend(d_q=d_q)
    check(c, out, lse, few)
    again, lse2, _ = c.attend(d_q=d_q, ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2), "the same call differs"
    assert q.spear_ec_workspace_status(ws) == 0
