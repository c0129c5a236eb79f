"""The 8-bit path on the GPU (needs an MI355X): quantization of rows, norm and
products against their definition in 64 bits, over sizes, layouts and values
where they can go wrong, and a run of them together with the cache and the
4-bit layer as a model's block uses them."""
from __future__ import annotations

import math

import pytest

import quantization_error_compensation_amd as q

pytestmark = pytest.mark.gpu


def note(msg):
    print(f"[case] {msg}", flush=True)


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    assert _t.cuda.is_available(), "GPU tests need a GPU"
    q.load_library()
    return _t


@pytest.fixture(scope="module")
def ref(torch):
    import q8_reference
    return q8_reference


def rng(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def guarded(torch, shape, dtype, fill=77):
    """A tensor in the middle of a larger one, and a check that the rest is untouched."""
    n = math.prod(shape)
    pad = 64
    big = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")

    def untouched():
        assert bool((big[:pad] == fill).all()) and bool((big[n + pad:] == fill).all())
    return big[pad:pad + n].view(shape), untouched


def bits_equal(torch, a, b):
    as_int = {1: torch.int8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(as_int), b.contiguous().view(as_int))


# ---------------------------------------------------------------- row operators
ROWS = [(1, 16), (3, 48), (257, 256), (5, 1008), (2, 4096), (64, 8208), (3, 28672), (2, 65536), (70000, 16)]


def special_rows(torch, x, seed):
    """Rows that go wrong easily: zeros, ties, tiny, huge, one large element."""
    n, d = x.shape
    g = rng(torch, seed)
    rows = [torch.zeros(d, device="cuda"),
            torch.randint(-254, 255, (d,), generator=g, device="cuda") / 2,   # ties of s = 1
            torch.randn(d, generator=g, device="cuda") * 2.0 ** -130,         # subnormal
            torch.randn(d, generator=g, device="cuda") * 1e37,
            torch.randn(d, generator=g, device="cuda") * 2.0 ** -110]
    rows[1][0] = 127
    rows[4][d // 2] = 3e30
    for i, r in enumerate(rows):
        x[(i * 7 + 1) % n] = r.to(x.dtype)
    return x


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,width", ROWS)
def test_quantize_and_read_back(torch, ref, rows, width, kind):
    note(f"quantize {rows} x {width} {kind}")
    dtype = torch.bfloat16 if kind == "bf16" else torch.float32
    x = torch.randn((rows, width), generator=rng(torch, rows + width), device="cuda").to(dtype)
    if rows > 1:
        x = special_rows(torch, x, width)
    wide = torch.full((rows, width + 24), 9e9, dtype=dtype, device="cuda")
    wide[:, 8:8 + width] = x
    want, scale = ref.quantize(x.double())
    out, out_ok = guarded(torch, (rows, width), torch.float32)
    for source in (x, wide[:, 8:8 + width]):
        codes, codes_ok = guarded(torch, (rows, width), torch.int8)
        scales, scales_ok = guarded(torch, (rows,), torch.float32)
        q.spear_ec_q8_quantize(source, codes, scales)
        q.spear_ec_q8_dequant_f32(codes, scales, out)
        torch.cuda.synchronize()
        assert torch.equal(scales, scale)
        assert torch.equal(codes, want)
        assert torch.equal(out, want.float() * scale[:, None])
        for ok in (codes_ok, scales_ok, out_ok):
            ok()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_ties_and_borders_of_codes(torch, ref, kind):
    """Values on and next to the borders between codes, for scales of few and many digits."""
    dtype = torch.bfloat16 if kind == "bf16" else torch.float32
    rows = []
    for top in (127.0, 254.0, 381.0, 1.0, 3.1, 127 * 5.0, 2.0 ** -90, 1e30):
        t = torch.tensor(top).to(dtype).float()
        s = (t.double() / 127).float()
        k = torch.arange(-126, 127)
        half = ((k.double() + 0.5) * s.double()).to(dtype).float()
        steps = torch.cat([half, torch.nextafter(half, torch.tensor(math.inf)),
                           torch.nextafter(half, torch.tensor(-math.inf))])
        row = torch.zeros(784)
        row[:steps.numel()] = steps.clamp(-float(t), float(t))
        row[-1] = t
        rows.append(row)
    x = torch.stack(rows).to(dtype).cuda()
    want, scale = ref.quantize(x.double())
    codes, scales = q.alloc_q8(*x.shape)
    q.spear_ec_q8_quantize(x, codes, scales)
    assert torch.equal(scales, scale) and torch.equal(codes, want)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,width", ROWS)
def test_norm(torch, ref, rows, width, residual):
    note(f"norm {rows} x {width} residual={residual}")
    g = rng(torch, 11 * rows + width)
    x = torch.randn((rows, width), generator=g, device="cuda").bfloat16()
    r = (3 * torch.randn((rows, width), generator=g, device="cuda")).bfloat16() if residual else None
    if rows > 1:
        x = special_rows(torch, x, width)
        if residual:
            r[1] = 0
            r[3 % rows] = -x[3 % rows]                       # sums to zero
    w = (1 + 0.2 * torch.randn(width, generator=g, device="cuda")).bfloat16()
    w[width // 3] = 0
    eps = 1e-5
    h, u = ref.norm(x, r, w, eps)
    want, scale = ref.quantize(u)
    # |h w| below fp32's normal range is off by 2^-150, times 1 / sqrt(mean + eps)
    low = 2.0 ** -149 / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + eps)
    bound = torch.maximum(u.abs() * ref.HALF[torch.bfloat16] * (1 + 2.0 ** -13), low + 2.0 ** -134)
    total = torch.empty_like(x) if residual else None
    y, y_ok = guarded(torch, (rows, width), torch.bfloat16)
    codes, codes_ok = guarded(torch, (rows, width), torch.int8)
    scales, scales_ok = guarded(torch, (rows,), torch.float32)
    for give_y, give_codes in ((True, True), (True, False), (False, True)):
        y.fill_(5)
        codes.fill_(5)
        q.spear_ec_q8_rmsnorm(x, r, total, w, eps, y=y if give_y else None,
                              codes=codes if give_codes else None,
                              scales=scales if give_codes else None)
        torch.cuda.synchronize()
        if residual:
            assert torch.equal(total, h)
        if give_y:
            assert bool(((y.double() - u).abs() <= bound).all())
        if give_codes:
            assert torch.equal(scales, scale)
            assert torch.equal(codes, want)
        for ok in (y_ok, codes_ok, scales_ok):
            ok()


@pytest.mark.parametrize("rows,width", [(1529, 4112), (1531, 4112), (3000, 8208), (140000, 16400)])
def test_norm_of_large_calls(torch, ref, rows, width):
    """Either side of the size up to which results leave the caches early, rows of
    several pieces a thread, and matrices of 4.6 GB: sampled rows."""
    note(f"large norm {rows} x {width}")
    g = rng(torch, rows)
    x = torch.randn((rows, width), generator=g, device="cuda", dtype=torch.bfloat16)
    r = torch.randn((rows, width), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(width, generator=g, device="cuda").bfloat16()
    s, y = torch.empty_like(x), torch.empty_like(x)
    codes, scales = q.alloc_q8(rows, width)
    q.spear_ec_q8_rmsnorm(x, r, s, w, 1e-5, y, codes, scales)
    for at in (slice(0, 3), slice(rows // 2, rows // 2 + 3), slice(65534, 65539), slice(130944, 130947),
               slice(rows - 3, rows)):
        h, u = ref.norm(x[at], r[at], w, 1e-5)
        assert torch.equal(s[at], h), at
        # y: (1 + 2^-12) half steps; bf16's own rounding is check's
        ref.check(y[at], u, u.abs() * 2.0 ** -8 * 2.0 ** -12, at)
        want_c, want_s = ref.quantize(u)
        near = (u / want_s.double()[:, None]).abs().frac().sub(0.5).abs() < 2.0 ** -22
        assert torch.allclose(scales[at], want_s, rtol=2.0 ** -23, atol=0), at
        assert bool(((codes[at] == want_c) | (near & ((codes[at].int() - want_c.int()).abs() <= 1))).all()), at


def test_norm_strides_and_in_place(torch, ref):
    g = rng(torch, 5)
    wide = torch.randn((37, 3 * 512), generator=g, device="cuda").bfloat16()
    x = wide[:, 512:1024]
    r = torch.randn((37, 512), generator=g, device="cuda").bfloat16()
    w = torch.ones(512, device="cuda").bfloat16()
    h, u = ref.norm(x, r, w, 1e-6)
    want, scale = ref.quantize(u)
    codes, scales = q.alloc_q8(37, 512)
    before = wide.clone()
    q.spear_ec_q8_rmsnorm(x, r, r, w, 1e-6, codes=codes, scales=scales)    # sum over residual
    assert torch.equal(r, h) and torch.equal(codes, want) and torch.equal(scales, scale)
    assert torch.equal(wide, before)
    x2, r2 = before[:, 512:1024].contiguous(), torch.zeros_like(r)
    h2, u2 = ref.norm(x2, r2, w, 1e-6)
    want2, scale2 = ref.quantize(u2)
    q.spear_ec_q8_rmsnorm(x2, r2, x2, w, 1e-6, codes=codes, scales=scales)  # sum over x
    assert torch.equal(x2, h2) and torch.equal(codes, want2) and torch.equal(scales, scale2)


def test_rows_that_are_not_finite(torch, ref):
    x = torch.randn((12, 4112), generator=rng(torch, 6), device="cuda").bfloat16()
    x[1, 7], x[4, 4111], x[9, 2000] = math.nan, math.inf, -math.inf
    bad = torch.tensor([i in (1, 4, 9) for i in range(12)], device="cuda")
    w = torch.ones(4112, device="cuda").bfloat16()
    w[7] = 0.0
    codes, scales = q.alloc_q8(12, 4112)
    y = torch.empty_like(x)
    for v in (x, x.float()):
        want, scale = ref.quantize(v.double())
        q.spear_ec_q8_quantize(v, codes, scales)
        assert torch.equal(codes, want) and torch.equal(scales.isnan(), bad)
        assert torch.equal(scales[~bad], scale[~bad])
    q.spear_ec_q8_rmsnorm(x, None, None, w, 1e-5, y=y, codes=codes, scales=scales)
    h, u = ref.norm(x, None, w, 1e-5)
    want, scale = ref.quantize(u)
    assert torch.equal(codes, want) and torch.equal(scales.isnan(), bad)
    assert torch.equal(y.isnan().all(1), bad) and torch.equal(y.isnan().any(1), bad)
    # and a product with them: NaN in those rows alone
    d = q.make_q8_desc(4112, 64)
    wq = torch.randint(-127, 128, (64, 4112), generator=rng(torch, 7), device="cuda").to(torch.int8)
    ws = torch.rand(64, generator=rng(torch, 8), device="cuda")
    out = torch.empty((12, 64), dtype=torch.bfloat16, device="cuda")
    q.spear_ec_q8_linear(d, codes, scales, wq, ws, out, q.alloc_q8_workspace(d, 12))
    assert torch.equal(out.isnan().all(1), bad) and torch.equal(out.isnan().any(1), bad)


@pytest.mark.parametrize("width", [128, 1040, 8208])
def test_norm_of_rows_of_zeros(torch, ref, width):
    """Padding: rows of zeros (of either sign, or cancelled by the residual)
    between others of every size give zeros and the scale 1, but NaN with a
    weight that is not finite."""
    note(f"zeros {width}")
    g = rng(torch, width)
    rows = 65
    x = torch.randn(rows, width, generator=g, device="cuda").bfloat16()
    r = torch.randn(rows, width, generator=g, device="cuda").bfloat16()
    x[5::10] *= 2.0 ** -70
    r[5::10] *= 2.0 ** -70
    x[::3] = 0
    r[::3] = torch.where(torch.rand(rows, width, generator=g, device="cuda") < 0.5, 0.0, -0.0).bfloat16()[::3]
    r[1::6] = -x[1::6]
    w = torch.randn(width, generator=g, device="cuda").bfloat16()
    for last in (1.0, 0.0, math.inf, math.nan):
        w[-1] = last
        s, y = torch.empty_like(x), torch.empty_like(x)
        codes, scales = q.alloc_q8(rows, width)
        q.spear_ec_q8_rmsnorm(x, r, s, w, 1e-6, y, codes, scales)
        h, u = ref.norm(x, r, w, 1e-6)
        assert torch.equal(s, h)
        zero = (h == 0).all(1)
        assert zero.sum() >= 22
        assert bool((codes[zero] == 0).all())
        if math.isfinite(last):
            assert bool((scales[zero] == 1).all()) and bool((y[zero] == 0).all())
        else:
            assert bool(scales[zero].isnan().all()) and bool(y[zero].isnan().all())
        want_c, want_s = ref.quantize(u)
        near = (u / want_s.double()[:, None]).abs().frac().sub(0.5).abs() < 2.0 ** -22
        assert torch.allclose(scales, want_s, rtol=2.0 ** -23, atol=0, equal_nan=True)
        assert bool(((codes == want_c) | (near & ((codes.int() - want_c.int()).abs() <= 1))).all())


def test_norm_weights_and_eps_at_the_ends(torch, ref):
    """Weights and values whose products leave fp32's normal range, and large eps."""
    g = rng(torch, 9)
    for xs, ws, eps in ((1e-25, 1e-25, 1e-30), (1e-38, 1.0, 1e-12), (1e18, 1e-30, 1e-5), (1.0, 1e-36, 1e-5),
                        (1e-3, 1e3, 1e30), (1e15, 1e15, 1e-5)):
        x = (torch.randn((4, 272), generator=g, device="cuda") * xs).bfloat16()
        w = (torch.randn(272, generator=g, device="cuda") * ws).bfloat16()
        h, u = ref.norm(x, None, w, eps)
        want, scale = ref.quantize(u)
        codes, scales = q.alloc_q8(4, 272)
        q.spear_ec_q8_rmsnorm(x, None, None, w, eps, codes=codes, scales=scales)
        assert torch.equal(scales, scale) and torch.equal(codes, want), (xs, ws, eps)


# --------------------------------------------------------------------- products
def operands(torch, T, K, rows, seed):
    g = rng(torch, seed)
    xq = torch.randint(-127, 128, (T, K), generator=g, device="cuda").to(torch.int8)
    wq = torch.randint(-128, 128, (rows, K), generator=g, device="cuda").to(torch.int8)
    xs = torch.rand(T, generator=g, device="cuda") * 0.02 + 0.001
    ws = (torch.rand(rows, generator=g, device="cuda") + 0.1) * (2e-3 / math.sqrt(K))
    return xq, xs, wq, ws


TOKENS = [1, 2, 7, 15, 16, 17, 31, 33, 48, 49, 64, 65, 72, 96, 97, 127, 128, 129, 200, 255, 256, 257, 300, 511, 513, 1000]
WIDTHS = [16, 48, 64, 112, 128, 144, 192, 1040, 2064, 4096]
OUTS = [16, 32, 48, 80, 112, 128, 144, 256, 272, 528, 1040]


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("i", range(len(TOKENS)))
def test_products(torch, ref, i, act):
    """Every token count with widths and outputs that go round, both types of y."""
    T = TOKENS[i]
    for j in range(4):
        K, N = WIDTHS[(i + 3 * j) % len(WIDTHS)], OUTS[(2 * i + 5 * j + len(act)) % len(OUTS)]
        f32 = (i + j) % 2 == 0
        note(f"product T={T} K={K} N={N} {act} f32={f32}")
        d = q.make_q8_desc(K, N, act, out_f32=f32)
        assert q.q8_weight_shape(d) == (N * (1 if act == "none" else 2), K)
        x = operands(torch, T, K, q.q8_weight_shape(d)[0], 100 * i + j)
        y, ok = guarded(torch, (T, N), torch.float32 if f32 else torch.bfloat16)
        y.fill_(math.nan)
        ws = q.alloc_q8_workspace(d, T)
        q.spear_ec_q8_linear(d, *x, y, ws)
        torch.cuda.synchronize()
        want, tol = ref.product(*x, act)
        ref.check(y, want, tol, (T, K, N, act))
        ok()
        assert int(ws[:16384].count_nonzero()) == 0


LARGE = [(1, 28672, 8192, "none"), (3, 11008, 4096, "none"), (1, 4096, 11008, "silu"), (20, 8192, 4112, "gelu"),
         (40, 65536, 1024, "none"), (64, 4096, 4096, "none"), (72, 8192, 7168, "silu"), (130, 28672, 1040, "none"),
         (320, 4096, 4096, "none"), (512, 28672, 2048, "none"), (777, 4112, 5536, "silu"), (2048, 4096, 4096, "none"),
         (2500, 1024, 8192, "gelu"), (4099, 2064, 2064, "none"), (9000, 512, 512, "none"),
         (475, 20224, 3584, "none"), (1252, 9728, 1408, "silu"), (700, 20000, 528, "gelu")]


@pytest.mark.parametrize("T,K,N,act", LARGE)
def test_products_of_usual_sizes(torch, ref, T, K, N, act):
    note(f"large product T={T} K={K} N={N} {act}")
    d = q.make_q8_desc(K, N, act)
    x = operands(torch, T, K, q.q8_weight_shape(d)[0], T + K + N)
    y = torch.full((T, N), math.nan, dtype=torch.bfloat16, device="cuda")
    ws = q.alloc_q8_workspace(d, T)
    for _ in range(2):  # on the workspace as the first call left it
        q.spear_ec_q8_linear(d, *x, y, ws)
    torch.cuda.synchronize()
    want, tol = ref.product(*x, act)
    ref.check(y, want, tol, (T, K, N, act))


@pytest.mark.parametrize("T", [1, 20, 100, 700])
def test_largest_sums_are_exact(torch, T):
    """Every code -128 over the widest rows: sums of 2^30, exact in 32 bits."""
    K, N = 65536, 48
    d = q.make_q8_desc(K, N, out_f32=True)
    xq = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    wq[5], wq[7, 1] = 127, -127
    one = torch.ones(max(T, N), device="cuda")
    y = torch.empty((T, N), device="cuda")
    q.spear_ec_q8_linear(d, xq, one[:T], wq, one[:N], y, q.alloc_q8_workspace(d, T))
    want = torch.full((T, N), 2.0 ** 30, device="cuda", dtype=torch.float64)
    want[:, 5] = -127 * 128 * 65536
    want[:, 7] = 2.0 ** 30 - 128
    assert torch.equal(y, want.float())


@pytest.mark.parametrize("act", ["none", "silu"])
def test_a_row_does_not_depend_on_its_batch(torch, act):
    """The same tokens in calls of every size and way of splitting: the same bits."""
    K, N, T = 4112, 2064, 1100
    d = q.make_q8_desc(K, N, act)
    xq, xs, wq, ws = operands(torch, T, K, q.q8_weight_shape(d)[0], 3)
    work = q.alloc_q8_workspace(d, T)
    whole = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    q.spear_ec_q8_linear(d, xq, xs, wq, ws, whole, work)
    for n in (1, 2, 16, 17, 40, 64, 65, 100, 128, 129, 256, 300, 600):
        part = torch.empty((n, N), dtype=torch.bfloat16, device="cuda")
        q.spear_ec_q8_linear(d, xq[13:13 + n].clone(), xs[13:13 + n].clone(), wq, ws, part, work)
        assert bits_equal(torch, part, whole[13:13 + n]), n


def test_gates_at_the_ends(torch, ref):
    """Pre-activations from far below to far above zero, zeros and infinities."""
    K, N = 16, 272
    xq = torch.zeros((3, K), dtype=torch.int8, device="cuda")
    xq[:, 0] = 1
    wq = torch.zeros((2 * N, K), dtype=torch.int8, device="cuda")
    wq[:N, 0] = 1
    wq[N:, 0] = 64
    xs = torch.ones(3, device="cuda")
    values = torch.cat([torch.linspace(-95, 95, 190), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 300, -300, 1e19, -1e19]),
                        torch.linspace(-9, 9, N - 198)]).cuda()
    ws = torch.cat([values, torch.full((N,), 1 / 64, device="cuda")])
    for act in ("silu", "gelu"):
        d = q.make_q8_desc(K, N, act, out_f32=True)
        y = torch.empty((3, N), device="cuda")
        q.spear_ec_q8_linear(d, xq, xs, wq, ws, y, q.alloc_q8_workspace(d, 3))
        want, tol = ref.product(xq, xs, wq, ws, act)
        ref.check(y, want, tol, act)
    ws[3], ws[N + 5], ws[200] = math.inf, math.inf, math.nan
    q.spear_ec_q8_linear(d, xq, xs, wq, ws, y, q.alloc_q8_workspace(d, 3))
    other = torch.ones(N, dtype=torch.bool, device="cuda")
    other[3] = other[5] = other[200] = False
    ref.check(y[:, other], want[:, other], tol[:, other], "beside infinities")
    assert bool((y[:, 3] == math.inf).all()) and bool(y[:, 200].isnan().all())


def test_offsets_past_32_bits(torch, ref):
    """Weights of 4.3 GB, outputs of 8.6 GB, read-back of 4.6 GB: sampled rows."""
    note("weights past 2^32 bytes")
    g = rng(torch, 1)
    N, K = 262144, 16400
    wq = torch.empty((N, K), dtype=torch.int8, device="cuda")
    for i in range(0, N, 16384):
        wq[i:i + 16384] = torch.randint(-127, 128, (16384, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=g, device="cuda") * 1e-5
    pick = torch.randint(0, N, (500,), generator=g, device="cuda")
    pick[:3] = torch.tensor([0, N - 1, N - 17])
    for T in (1, 40, 300):
        d = q.make_q8_desc(K, N)
        xq = torch.randint(-127, 128, (T, K), generator=g, device="cuda").to(torch.int8)
        xs = torch.rand(T, generator=g, device="cuda")
        y = torch.full((T, N), math.nan, dtype=torch.bfloat16, device="cuda")
        q.spear_ec_q8_linear(d, xq, xs, wq, ws, y, q.alloc_q8_workspace(d, T))
        want, tol = ref.product(xq, xs, wq[pick], ws[pick])
        ref.check(y[:, pick], want, tol, T)
        assert not bool(y.isnan().any())
    del wq
    note("outputs past 2^32 bytes")
    K, T = 16, 16400
    x = operands(torch, T, K, N, 2)
    d = q.make_q8_desc(K, N)
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    y[-1] = math.nan
    q.spear_ec_q8_linear(d, *x, y, q.alloc_q8_workspace(d, T))
    for rows in (slice(0, 3), slice(9000, 9003), slice(T - 3, T)):
        want, tol = ref.product(x[0][rows], x[1][rows], x[2], x[3])
        ref.check(y[rows], want, tol, rows)
    del y
    note("rows past 2^32 bytes")
    rows, width = 70000, 16400
    v = torch.randn((rows, width), generator=g, device="cuda").bfloat16()
    codes, scales = q.alloc_q8(rows, width)
    out = torch.empty((rows, width), device="cuda")
    q.spear_ec_q8_quantize(v, codes, scales)
    q.spear_ec_q8_dequant_f32(codes, scales, out)
    for at in (slice(0, 2), slice(65535, 65538), slice(rows - 2, rows)):
        want, scale = ref.quantize(v[at].double())
        assert torch.equal(codes[at], want) and torch.equal(scales[at], scale)
        assert torch.equal(out[at], want.float() * scale[:, None])


# ------------------------------------------------------------- streams, graphs
def test_no_rows_and_no_tokens(torch):
    codes, scales = q.alloc_q8(0, 64)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    q.spear_ec_q8_quantize(x, codes, scales)
    q.spear_ec_q8_dequant_f32(codes, scales, torch.empty((0, 64), device="cuda"))
    q.spear_ec_q8_rmsnorm(x, None, None, torch.ones(64, device="cuda").bfloat16(), 1e-5, codes=codes,
                          scales=scales)
    d = q.make_q8_desc(64, 32)
    wq, ws = q.alloc_q8(32, 64)
    q.spear_ec_q8_linear(d, codes, scales, wq, ws, torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"),
                         q.alloc_q8_workspace(d, 0))


class Block:
    """A block's feed-forward half at 8 bits and the workspaces it keeps."""

    def __init__(self, torch, T, d, f, seed):
        g = rng(torch, seed)
        self.w = torch.ones(d, device="cuda").bfloat16()
        self.up, self.down = q.make_q8_desc(d, f, "silu"), q.make_q8_desc(f, d)
        self.wu = operands(torch, 1, d, 2 * f, seed + 1)[2:]
        self.wd = operands(torch, 1, f, d, seed + 2)[2:]
        self.x = torch.randn((T, d), generator=g, device="cuda").bfloat16()
        self.r = torch.randn((T, d), generator=g, device="cuda").bfloat16()
        self.sum = torch.empty_like(self.x)
        self.cx, self.cf = q.alloc_q8(T, d), q.alloc_q8(T, f)
        self.f = torch.empty((T, f), dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
        self.ws = [q.alloc_q8_workspace(self.up, T), q.alloc_q8_workspace(self.down, T)]

    def __call__(self, stream=None):
        q.spear_ec_q8_rmsnorm(self.x, self.r, self.sum, self.w, 1e-5, codes=self.cx[0], scales=self.cx[1],
                              stream=stream)
        q.spear_ec_q8_linear(self.up, *self.cx, *self.wu, self.f, self.ws[0], stream=stream)
        q.spear_ec_q8_quantize(self.f, *self.cf, stream=stream)
        q.spear_ec_q8_linear(self.down, *self.cf, *self.wd, self.y, self.ws[1], stream=stream)


@pytest.mark.parametrize("T", [1, 40, 130, 600])
def test_captured_calls_replay(torch, T):
    note(f"graph T={T}")
    b = Block(torch, T, 1040, 2064, T)
    b()
    torch.cuda.synchronize()
    want = [t.clone() for t in (b.sum, b.f, b.y)]
    cap, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cap):
        b(cap)
    first = b.x.clone()
    for rep in range(3):
        b.x.copy_(first.flip(0))
        b()                                      # eager work on the same workspaces
        torch.cuda.synchronize()
        b.x.copy_(first)
        for t in (b.sum, b.f, b.y):
            t.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip((b.sum, b.f, b.y), want):
            assert torch.equal(t, w), rep


def test_two_streams_at_once(torch):
    """Calls on two streams with workspaces of their own do not meet."""
    blocks = [Block(torch, T, 2064, 4112, 50 + T) for T in (20, 200)]
    want = []
    for b in blocks:
        b()
        torch.cuda.synchronize()
        want.append(b.y.clone())
        b.y.fill_(math.nan)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for b, s in zip(blocks, streams):
            b(s)
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        assert torch.equal(b.y, w)


# ------------------------------------------------------------ a block together
def test_a_models_block(torch, ref):
    """Norm, 8-bit projections, the 4-bit cache and its attention, the gated
    feed-forward half: a prompt and then a single token of three chats, each
    call against the definition on the inputs that it was given."""
    H, G, D, d, f, page = 8, 2, 64, 512, 1040, 16
    lens = [5, 40, 17]
    g = rng(torch, 21)
    kv = q.make_kv_desc(H, G, D, page, 16, 4, False)
    cache = q.alloc_kv_cache(kv)
    table = torch.randperm(16, generator=g, device="cuda").to(torch.int32)[:12].view(3, 4).contiguous()
    wn = (1 + 0.1 * torch.randn((2, d), generator=g, device="cuda")).bfloat16()
    weights = {}
    for name, k, n, act in (("qkv", d, (H + 2 * G) * D, "none"), ("out", H * D, d, "none"),
                            ("up", d, f, "silu"), ("down", f, d, "none")):
        desc = q.make_q8_desc(k, n, act)
        rows = q.q8_weight_shape(desc)[0]
        w = torch.randn((rows, k), generator=g, device="cuda") / math.sqrt(k)
        codes, scales = q.alloc_q8(rows, k)
        q.spear_ec_q8_quantize(w, codes, scales)
        want, scale = ref.quantize(w.double())
        assert torch.equal(codes, want) and torch.equal(scales, scale)
        weights[name] = (desc, codes, scales, act)

    def linear(name, xq, xs):
        desc, codes, scales, act = weights[name]
        y = torch.empty((xq.shape[0], desc.d_out), dtype=torch.bfloat16, device="cuda")
        q.spear_ec_q8_linear(desc, xq, xs, codes, scales, y, q.alloc_q8_workspace(desc, xq.shape[0]))
        want, tol = ref.product(xq, xs, codes, scales, act)
        ref.check(y, want, tol, name)
        return y

    def norm(x, r, i):
        codes, scales = q.alloc_q8(*x.shape)
        total = torch.empty_like(x) if r is not None else None
        q.spear_ec_q8_rmsnorm(x, r, total, wn[i], 1e-5, codes=codes, scales=scales)
        h, u = ref.norm(x, r, wn[i], 1e-5)
        want, scale = ref.quantize(u)
        assert torch.equal(codes, want) and torch.equal(scales, scale)
        assert r is None or torch.equal(total, h)
        return codes, scales, x if r is None else total

    for step in (0, 1):
        new = lens if step == 0 else [1, 1, 1]
        total_lens = lens if step == 0 else [n + 1 for n in lens]
        T = sum(new)
        note(f"block, {T} tokens")
        off = torch.tensor([0] + [sum(new[:i + 1]) for i in range(3)], dtype=torch.int32, device="cuda")
        batch = q.make_kv_batch(off, torch.tensor(total_lens, dtype=torch.int32, device="cuda"), table, T)
        x = torch.randn((T, d), generator=g, device="cuda").bfloat16()
        c, s, stream = norm(x, None, 0)
        qkv = linear("qkv", c, s).view(T, H + 2 * G, D)
        q.spear_ec_kv_append(kv, batch, None, qkv[:, H:H + G], qkv[:, H + G:], None, *cache, None)
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
        q.spear_ec_kv_attention(kv, batch, qkv[:, :H], *cache, D ** -0.5, out,
                                q.alloc_kv_workspace(kv, 3, T))
        assert bool(out.isfinite().all())
        c, s = q.alloc_q8(T, H * D)
        q.spear_ec_q8_quantize(out.view(T, H * D), c, s)
        y = linear("out", c, s)
        c, s, stream = norm(y, stream, 1)
        a = linear("up", c, s)
        c, s = q.alloc_q8(T, f)
        q.spear_ec_q8_quantize(a, c, s)
        want, scale = ref.quantize(a.double())
        assert torch.equal(c, want) and torch.equal(s, scale)
        y = linear("down", c, s)
        # and a 4-bit layer on the norm of the block's result
        last = torch.empty_like(y)
        q.spear_ec_q8_rmsnorm(y, stream, stream, wn[0], 1e-5, y=last)
        desc = q.make_desc(d, 256, 0, d, False)
        w4 = torch.randn((256, d), generator=rng(torch, 30), device="cuda")
        packed = q.alloc_packed(desc)
        q.spear_ec_quantize_rtn(desc, w4, *packed)
        values = torch.empty((256, d), device="cuda")
        q.spear_ec_dequant_f32(desc, *packed, values)
        logits = torch.empty((T, 256), dtype=torch.bfloat16, device="cuda")
        q.spear_ec_linear(desc, last, *packed, None, None, None, None, 1.0, logits, q.alloc_workspace(desc, T))
        exact = last.double() @ values.double().t()
        # fp32 sums of 512 products (2^-24 of their magnitudes' sum a step), and bf16's half step
        tol = (last.double().abs() @ values.double().abs().t()) * 512 * 2.0 ** -24
        ref.check(logits, exact, tol, "4-bit layer")
