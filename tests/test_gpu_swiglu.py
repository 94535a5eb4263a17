"""The experts' activation with its FP8 cast, and its gradient, on the GPU
against the 64-bit formulas, row by row of the segments."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import moe_inputs as mi
from gpu_path import dev, to_dev

pytestmark = pytest.mark.gpu

ROUND, WORDS = 1, 2


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_moe_layout_03_amd import capi as c

    return c


def inputs(seed, counts, width, mode="rows", per=0, spread=1.0):
    start, rows = ref.lay_rows(counts, mode, per, 4, 3)
    live = ref.live_rows(start, counts)
    rng = np.random.default_rng(seed)
    x = np.full((rows, width), 0x7FC0, np.uint16)  # NaN where nothing may be read
    x[live] = mi.to_bf16_bits((rng.standard_normal((len(live), width)) * spread).astype(np.float32))
    return start, rows, live, x


def fp8(capi, counts, start, rows, x, I, flags, status=None):
    q = torch.full((rows, I), 0xA5, dtype=torch.uint8, device=dev())
    words = bool(flags & WORDS)
    sc = torch.full((rows, I // 512 if words else I // 128), -5,
                    dtype=torch.int32 if words else torch.float32, device=dev())
    capi.moe_swiglu_fp8(len(counts), I, rows, to_dev(x), to_dev(start),
                        to_dev(np.array(counts, np.int32)), q, sc, flags, status)
    torch.cuda.synchronize()
    return q.cpu().numpy(), sc.cpu().numpy()


def check_fp8(live, x, q, sc, I, flags):
    rows = q.shape[0]
    dead = np.setdiff1d(np.arange(rows), live)
    assert np.all(q[dead] == 0xA5) and np.all(sc[dead] == -5)
    if not len(live):
        return
    *_, h = ref.silu_mul(mi.bf16_bits_to_f32(x[live]))
    # exp (2 steps), sum, quotient, product: 8 half steps of h with a margin of 2;
    # the scale adds its quotient
    n = 10 * ref.EPS24
    hg = h.reshape(len(live), -1, 128)
    want = np.maximum(np.abs(hg).max(-1), np.float32(1e-4)) / 448.0
    if flags & WORDS:
        b = np.stack([(sc[live].astype(np.int64) >> k) & 255 for k in (0, 8, 16, 24)], -1)
        s = np.exp2(b.reshape(len(live), -1) - 127.0)
    else:
        s = sc[live].astype(np.float64)
    if flags & ROUND:
        assert np.array_equal(s, np.exp2(np.round(np.log2(s))))
        assert np.all(s >= want * (1 - n)) and np.all(s / 2 < want * (1 + n))
    else:
        assert np.all(np.abs(s - want) <= n * want)
    v = ref.e4m3_values(q[live]).reshape(hg.shape) * s[..., None]
    # a code is off by at most half an E4M3 step: 2^-4 of the value, 2^-10 below
    # the smallest normal 2^-6; the scaled value by n, or n of the largest where
    # it saturates
    tol = (2.0 ** -4 * np.abs(hg) * (1 + n) + 2.0 ** -10 * s[..., None] + n * np.abs(hg)
           + n * 448 * s[..., None] * (np.abs(hg) >= 440 * s[..., None]))
    assert np.all(np.abs(v - hg) <= tol)
    # signs survive, also those of values that round to zero
    assert np.array_equal((q[live] >> 7).reshape(hg.shape)[hg != 0], np.signbit(hg)[hg != 0])


COUNTS = [[1], [0], [0, 3, 0, 1, 0], [5, 0, 17, 1, 64], [1] * 40, [200, 1, 0, 77]]


@pytest.mark.parametrize("flags", [0, ROUND, ROUND | WORDS])
@pytest.mark.parametrize("I", [128, 512, 640, 2048])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_swiglu_fp8(capi, counts, I, flags):
    if flags & WORDS and I % 512:
        I = 1024
    start, rows, live, x = inputs(sum(counts) + I, counts, 2 * I, spread=2.0)
    q, sc = fp8(capi, counts, start, rows, x, I, flags)
    check_fp8(live, x, q, sc, I, flags)


def test_padded_layout_many_experts(capi):
    rng = np.random.default_rng(4)
    counts = rng.integers(0, 4, size=1024).tolist()
    start, rows, live, x = inputs(6, counts, 512, "padded", 6)
    q, sc = fp8(capi, counts, start, rows, x, 256, 0)
    check_fp8(live, x, q, sc, 256, 0)


def test_extreme_values(capi):
    """Zero groups, subnormals, far negative gates (silu = -0), products past the
    float range (kept at the largest float)."""
    I = 256
    g = np.zeros((6, I), np.float32)
    u = np.ones((6, I), np.float32)
    g[1], u[1] = -3.3e38, 3.3e38
    g[2], u[2] = 1e-39, 1e-3
    g[3, ::2], u[3] = 3e38, 3e38
    g[4], u[4] = np.linspace(-90, 90, I), -2.0
    g[5], u[5] = 1.0, np.linspace(-3e38, 3e38, I)
    x = mi.to_bf16_bits(np.concatenate([g, u], 1))
    start = np.array([0], np.int32)
    q, sc = fp8(capi, [6], start, 6, x, I, 0)
    assert np.isfinite(sc).all() and np.all((q & 0x7F) != 0x7F)
    assert np.all((q[:3] & 0x7F) == 0)
    assert np.all(sc[0] == np.float32(1e-4) / np.float32(448))
    assert np.all(q[3, ::2] == 0x7E) and np.all((q[3, 1::2] & 0x7F) == 0)
    check_fp8(np.array([4, 5]), x, *[np.where(np.isin(np.arange(6), [4, 5])[:, None], a, b)
                                    for a, b in ((q, 0xA5), (sc, -5))], I, 0)


def grad_tol(g, u, s, d, want):
    """A rounding to bf16, and 16 half float steps of each factor: 1 + g (1 - s)
    cancels near g = -1.28, so its rounding counts against 1 + |g|."""
    big = np.concatenate([np.abs(d * u * s) * (1 + np.abs(g)), np.abs(d * g * s)], 1)
    return ref.HALF_BF16 * np.abs(want) + 16 * ref.EPS24 * big + 1e-40


@pytest.mark.parametrize("I", [8, 24, 512, 1416, 2048])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_swiglu_grad(capi, counts, I):
    start, rows, live, x = inputs(sum(counts) * 3 + I, counts, 2 * I, spread=3.0)
    rng = np.random.default_rng(I)
    dh = np.full((rows, I), 0x7FC0, np.uint16)
    dh[live] = mi.to_bf16_bits(rng.standard_normal((len(live), I)).astype(np.float32))
    dx = torch.full((rows, 2 * I), 0x1234, dtype=torch.int16, device=dev())
    cnt = to_dev(np.array(counts, np.int32))
    capi.moe_swiglu_grad(len(counts), I, rows, to_dev(x), to_dev(dh), to_dev(start), cnt, dx)
    torch.cuda.synchronize()
    got = dx.cpu().numpy().view(np.uint16)
    assert np.all(got[np.setdiff1d(np.arange(rows), live)] == 0x1234)
    g, u, s, _ = ref.silu_mul(mi.bf16_bits_to_f32(x[live]))
    d = mi.bf16_bits_to_f32(dh[live]).astype(np.float64)
    want = np.concatenate([d * u * s * (1 + g * (1 - s)), d * g * s], 1)
    have = mi.bf16_bits_to_f32(got[live]).astype(np.float64)
    assert np.all(np.abs(have - want) <= grad_tol(g, u, s, d, want))
    # the derivative by central differences: off by h^2 / 6 of a third
    # derivative, below 1 in size for silu, and by the rounding of h
    if len(live):
        h = 1e-4
        silu = lambda z: z / (1 + np.exp(-z))  # noqa: E731
        num = np.concatenate([d * u * (silu(g + h) - silu(g - h)) / (2 * h),
                              d * silu(g)], 1)
        ext = np.concatenate([np.abs(d * u), np.abs(d * u)], 1) * (h * h + 1e-11 / h)
        assert np.all(np.abs(have - num) <= grad_tol(g, u, s, d, want) + ext)
    # in place: the gradient over x itself
    xin = to_dev(x)
    capi.moe_swiglu_grad(len(counts), I, rows, xin, to_dev(dh), to_dev(start), cnt, xin)
    torch.cuda.synchronize()
    assert np.array_equal(xin.cpu().numpy().view(np.uint16)[live], got[live])


def test_gradient_of_large_factors(capi):
    """d_h * u past the float range where the sigmoid brings the product back, or
    to zero: the gradient is the formula's, not an infinity or NaN."""
    I = 64
    g = np.zeros((4, I), np.float32)
    g[0], g[1], g[2] = -1e30, np.linspace(-80, -30, I), -3.3e38
    g[3] = np.linspace(-85, 85, I)
    u = np.full((4, I), 3e38, np.float32)
    d = np.full((4, I), -10.0, np.float32)
    d[3] = 1e-3
    x, dh = mi.to_bf16_bits(np.concatenate([g, u], 1)), mi.to_bf16_bits(d)
    dx = torch.zeros(4, 2 * I, dtype=torch.int16, device=dev())
    capi.moe_swiglu_grad(1, I, 4, to_dev(x), to_dev(dh), to_dev(np.array([0], np.int32)),
                         to_dev(np.array([4], np.int32)), dx)
    torch.cuda.synchronize()
    have = mi.bf16_bits_to_f32(dx.cpu().numpy().view(np.uint16)).astype(np.float64)
    gg, uu, s, _ = ref.silu_mul(mi.bf16_bits_to_f32(x))
    dd = mi.bf16_bits_to_f32(dh).astype(np.float64)
    want = np.concatenate([dd * uu * s * (1 + gg * (1 - s)), dd * gg * s], 1)
    assert np.isfinite(want).all() and np.isfinite(have).all()
    assert np.all(np.abs(have - want) <= grad_tol(gg, uu, s, dd, want))


def test_bad_segments(capi):
    """Segments outside the buffer are skipped and reported, the others done."""
    I, rows = 128, 32
    rng = np.random.default_rng(0)
    x = mi.to_bf16_bits(rng.standard_normal((rows, 2 * I)).astype(np.float32))
    start = np.array([-1, 30, 4, 2 ** 31 - 1, 8, 12], np.int32)
    counts = [2, 3, 3, 5, -4, 2 ** 31 - 1]
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    q, sc = fp8(capi, counts, start, rows, x, I, 0, st)
    assert int(st.item()) == capi.MOE_STATUS_BAD_SLOT
    check_fp8(np.arange(4, 7), x, q, sc, I, 0)
    st.zero_()
    q, sc = fp8(capi, [0, -3, 2], np.array([-9, 99, 1], np.int32), rows, x, I, 0, st)
    assert int(st.item()) == 0  # empty segments may point anywhere
    check_fp8(np.arange(1, 3), x, q, sc, I, 0)


def test_offsets_past_32_bits(capi):
    """A buffer of more than 2^32 elements, segments at both ends: the same rows
    as in a small buffer, bit for bit."""
    I, rows, counts = 2048, (1 << 20) + 40, [3, 37]
    start = np.array([1, rows - 38], np.int32)
    small = np.array([0, 3], np.int32)
    rng = np.random.default_rng(8)
    part = to_dev(mi.to_bf16_bits(rng.standard_normal((40, 2 * I)).astype(np.float32)))
    dpart = to_dev(mi.to_bf16_bits(rng.standard_normal((40, I)).astype(np.float32)))
    far = torch.cat([torch.arange(1, 4), torch.arange(rows - 38, rows - 1)]).to(dev())
    cnt = to_dev(np.array(counts, np.int32))
    got = []
    for n, st, at in ((40, small, torch.arange(40, device=dev())), (rows, start, far)):
        x = torch.zeros(n, 2 * I, dtype=torch.int16, device=dev())
        dh = torch.zeros(n, I, dtype=torch.int16, device=dev())
        x[at], dh[at] = part.view(torch.int16), dpart.view(torch.int16)
        q = torch.zeros(n, I, dtype=torch.uint8, device=dev())
        sc = torch.zeros(n, I // 128, device=dev())
        dx = torch.zeros(n, 2 * I, dtype=torch.int16, device=dev())
        capi.moe_swiglu_fp8(2, I, n, x, to_dev(st), cnt, q, sc)
        capi.moe_swiglu_grad(2, I, n, x, dh, to_dev(st), cnt, dx)
        torch.cuda.synchronize()
        got.append((q[at].clone(), sc[at].clone(), dx[at].clone()))
        if n == rows:  # nothing else was written
            for t in (q, sc, dx):
                t[at] = 0
                assert all(not bool(c.any()) for c in t.split(1 << 18))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_gradient_of_a_steep_gate(capi):
    """The gate's slope s (1 + g (1 - s)) passes 1 between g = 0 and its tail: a
    factor near the largest bf16 times it leaves the float range where the other
    factor, being small, brings the product back."""
    I = 64
    slopes = np.linspace(0.01, 12.0, I)
    g = np.tile(slopes, (4, 1)).astype(np.float32)
    u, d = np.empty((4, I), np.float32), np.empty((4, I), np.float32)
    u[0], d[0] = 1e-10, 3.38e38
    u[1], d[1] = 3.38e38, -1e-10
    u[2], d[2] = -0.75, 3.38e38   # the product itself in the top binade
    u[3], d[3] = 1e-30, 1e-8      # and far below
    x, dh = mi.to_bf16_bits(np.concatenate([g, u], 1)), mi.to_bf16_bits(d)
    dx = torch.zeros(4, 2 * I, dtype=torch.int16, device=dev())
    capi.moe_swiglu_grad(1, I, 4, to_dev(x), to_dev(dh), to_dev(np.array([0], np.int32)),
                         to_dev(np.array([4], np.int32)), dx)
    torch.cuda.synchronize()
    have = mi.bf16_bits_to_f32(dx.cpu().numpy().view(np.uint16)).astype(np.float64)
    gg, uu, s, _ = ref.silu_mul(mi.bf16_bits_to_f32(x))
    dd = mi.bf16_bits_to_f32(dh).astype(np.float64)
    want = np.concatenate([dd * uu * s * (1 + gg * (1 - s)), dd * gg * s], 1)
    # the largest bf16 is (2 - 2^-7) 2^127; from half a step above, a value rounds
    # to infinity
    top, edge = (2 - 2.0 ** -7) * 2.0 ** 127, (2 - 2.0 ** -8) * 2.0 ** 127
    tol = grad_tol(gg, uu, s, dd, want)
    fits = np.abs(want) + tol < top
    assert fits[:, :I].all() and fits[1].all() and fits[3].all()
    assert np.all(np.abs(have - want)[fits] <= tol[fits])
    past = np.abs(want) - tol > edge
    assert np.all(have[past] == np.copysign(np.inf, want[past]))


@pytest.mark.parametrize("flags", [0, ROUND, ROUND | WORDS])
def test_values_that_are_not_finite_stay_visible(capi, flags):
    """A NaN or infinite gate or up gives its group of 128 channels the scale NaN
    (UE8M0: the byte 255) and NaN codes; every other group is as without it."""
    I, n = 1024, 9
    rng = np.random.default_rng(31)
    clean = mi.to_bf16_bits(rng.standard_normal((n, 2 * I)).astype(np.float32))
    x = clean.copy()
    nan, neg_nan, inf, neg_inf = 0x7FC0, 0xFFFF, 0x7F80, 0xFF80
    bad = {1: (300, nan), 2: (I + 5, inf), 3: (700, neg_inf), 4: (I + 1023, neg_nan),
           5: (128, inf), 6: (I + 130, neg_inf), 7: (127, 0x7F81)}
    for r, (c, v) in bad.items():
        x[r, c] = v
    x[5, I + 128] = 0            # an infinite gate on an up of zero
    x[6, 130] = 0                # and the other way round
    x[8, 0], x[8, I] = 0x7F7F, 0x7F7F  # the product of two finite values is kept finite
    start = np.array([0], np.int32)
    q, sc = fp8(capi, [n], start, n, x, I, flags)
    x[8, 0], x[8, I] = clean[8, 0], clean[8, I]
    q0, sc0 = fp8(capi, [n], start, n, clean, I, flags)

    def groups(s):
        if not flags & WORDS:
            return s
        return np.stack([(s.astype(np.int64) >> k) & 255 for k in (0, 8, 16, 24)],
                        -1).reshape(n, -1)

    s, s0 = groups(sc), groups(sc0)
    q, q0 = q.reshape(n, I // 128, 128), q0.reshape(n, I // 128, 128)
    hit = np.zeros((n, I // 128), bool)
    for r, (c, _) in bad.items():
        hit[r, c % I // 128] = True
    over = np.zeros_like(hit)
    over[8, 0] = True
    assert np.all((q[hit] & 0x7F) == 0x7F)
    assert np.all(s[hit] == 255) if flags & WORDS else np.isnan(s[hit]).all()
    assert np.array_equal(q[~hit & ~over], q0[~hit & ~over])
    assert np.array_equal(s[~hit & ~over], s0[~hit & ~over])
    assert np.all((q[8, 0] & 0x7F) < 0x7F) and (flags or q[8, 0, 0] == 0x7E)
    assert s[8, 0] < 255 if flags & WORDS else np.isfinite(s[8, 0])


def test_gradient_of_values_that_are_not_finite(capi):
    """NaN where the formulas give NaN, an infinity where they give one, and the
    other channels as without them."""
    I = 64
    rng = np.random.default_rng(37)
    g, u, d = (rng.standard_normal((7, I)).astype(np.float32) for _ in range(3))
    clean = [mi.to_bf16_bits(v) for v in (g, u, d)]
    at = np.arange(0, I, 3)
    g, u, d = g.copy(), u.copy(), d.copy()
    g[0, at], u[1, at], d[2, at] = np.nan, np.nan, np.nan
    g[3, at], u[4, at], d[5, at] = np.inf, -np.inf, np.inf
    g[6, at] = -np.inf
    bits = [mi.to_bf16_bits(v) for v in (g, u, d)]
    start, cnt = to_dev(np.array([0], np.int32)), to_dev(np.array([7], np.int32))
    got = []
    for b in (bits, clean):
        dx = torch.zeros(7, 2 * I, dtype=torch.int16, device=dev())
        capi.moe_swiglu_grad(1, I, 7, to_dev(np.concatenate(b[:2], 1)), to_dev(b[2]), start, cnt,
                             dx)
        torch.cuda.synchronize()
        got.append(dx.cpu().numpy().view(np.uint16))
    have = mi.bf16_bits_to_f32(got[0])
    g, u, d = (mi.bf16_bits_to_f32(b).astype(np.float64) for b in bits)
    with np.errstate(all="ignore"):
        s = 1 / (1 + np.exp(-g))
        want = np.concatenate([d * u * s * (1 + g * (1 - s)), d * g * s], 1)
    assert np.array_equal(np.isnan(have), np.isnan(want))
    assert np.array_equal(have[np.isinf(want)], want[np.isinf(want)])
    assert not np.isfinite(want[:, at]).all() and np.isinf(want).any()
    rest = np.setdiff1d(np.arange(2 * I), np.concatenate([at, at + I]))
    assert np.array_equal(got[0][:, rest], got[1][:, rest])


def test_gates_whose_sigmoid_is_subnormal(capi):
    """From -87.5 to -88.5 exp(-g) is finite, but its reciprocal is below the
    smallest normal float; times a large up, value and gradient are not."""
    I = 384
    g = np.repeat(np.array([-87.0, -87.5, -88.0, -88.5, -86.5], np.float32), 3)
    g = np.tile(g, I // 15 + 1)[:I][None].repeat(4, 0)
    u = np.empty((4, I), np.float32)
    u[0], u[1] = 3.3e38, -1e38
    u[2] = np.linspace(1e36, 3e38, I)
    u[3] = -np.geomspace(1e34, 1e38, I)
    x = mi.to_bf16_bits(np.concatenate([g, u], 1))
    start = np.array([0], np.int32)
    q, sc = fp8(capi, [4], start, 4, x, I, 0)
    check_fp8(np.arange(4), x, q, sc, I, 0)
    d = np.where(np.arange(I) % 2, 3e38, -7.0).astype(np.float32)[None].repeat(4, 0)
    d[0], d[1] = 10.0, -1e-3
    dh = mi.to_bf16_bits(d)
    dx = torch.zeros(4, 2 * I, dtype=torch.int16, device=dev())
    capi.moe_swiglu_grad(1, I, 4, to_dev(x), to_dev(dh), to_dev(start),
                         to_dev(np.array([4], np.int32)), dx)
    torch.cuda.synchronize()
    have = mi.bf16_bits_to_f32(dx.cpu().numpy().view(np.uint16)).astype(np.float64)
    gg, uu, s, _ = ref.silu_mul(mi.bf16_bits_to_f32(x))
    dd = mi.bf16_bits_to_f32(dh).astype(np.float64)
    want = np.concatenate([dd * uu * s * (1 + gg * (1 - s)), dd * gg * s], 1)
    # results past the largest bf16 are infinite
    over = np.abs(want) > 3.38e38
    assert not over[:2].any() and not over[:, I:].any()
    tol = grad_tol(gg, uu, s, dd, want)
    assert np.all(np.abs(have - want)[~over] <= tol[~over])


@pytest.mark.parametrize("flags", [0, ROUND, ROUND | WORDS])
def test_codes_are_those_of_the_cast_of_rows(capi, flags):
    """With gates of 128 the sigmoid is 1 and h = 128 u a bf16 value, so the cast
    has to give what moe_quantize_fp8 gives for the same rows, bit for bit: every
    significand of a group's largest value against every one below it, over the
    E4M3 range. Among them are 76 quotients that fall on the middle of two codes,
    which a product with the scale's reciprocal misses."""
    sig = np.arange(128, 256, dtype=np.float32) / 128
    I = 128 * 128                   # a group per significand of its largest value
    binades = 2.0 ** -np.arange(0, 18, dtype=np.float32)
    rows = len(binades) * 2         # 64 of the significands below it in each row's group
    h = np.empty((rows, 128, 128), np.float32)
    for b, two in enumerate(binades):
        for half in range(2):
            v = sig[64 * half:64 * half + 64] * two
            h[2 * b + half, :, :64] = v
            h[2 * b + half, :, 64:] = -v[::-1]
    h = np.minimum(h, sig[None, :, None])
    h = np.maximum(h, -sig[None, :, None])
    h[:, :, 0] = sig
    h = h.reshape(rows, I)
    u = mi.to_bf16_bits(h)
    assert np.array_equal(mi.bf16_bits_to_f32(u), h)
    g = np.full((rows, I), 0x4300, np.uint16)
    start = np.array([0], np.int32)
    q, sc = fp8(capi, [rows], start, rows, np.concatenate([g, u], 1), I, flags)
    want = torch.zeros(rows, I, dtype=torch.uint8, device=dev())
    ws = torch.zeros(sc.shape, device=dev(),
                     dtype=torch.int32 if flags & WORDS else torch.float32)
    capi.moe_quantize_fp8(rows, I, to_dev(mi.to_bf16_bits(128 * h)), want, ws, flags)
    torch.cuda.synchronize()
    assert np.array_equal(sc, ws.cpu().numpy())
    assert np.array_equal(q, want.cpu().numpy()), np.count_nonzero(q != want.cpu().numpy())


def test_rows_that_pass_32_bits_together(capi):
    """Overlapping segments of a buffer near 2^31 rows, whose rows together do not
    fit 31 bits: against the rules, reported, and nothing is read or written.
    (Their sum in units of 1024 rows still fits the buffer.)"""
    I, rows = 8, (1 << 31) - 1
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 96 GiB for the buffers")
    extra = 1000
    counts = np.ones(1 + extra, np.int32)
    counts[0] = rows
    start = np.zeros(1 + extra, np.int32)
    start[1:] = np.arange(extra)
    x = torch.empty(rows * 2 * I, dtype=torch.int16, device=dev())
    dh = torch.empty(rows * I, dtype=torch.int16, device=dev())
    ends = (x[:1 << 20], x[-(1 << 20):], x[rows * I:rows * I + (1 << 20)])
    for t in ends:
        t.fill_(0x1234)
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    capi.moe_swiglu_grad(1 + extra, I, rows, x, dh, to_dev(start), to_dev(counts), x, st)
    torch.cuda.synchronize()
    assert int(st.item()) == capi.MOE_STATUS_BAD_SLOT
    assert all(bool((t == 0x1234).all()) for t in ends)
    del x, dh, ends, t
    torch.cuda.empty_cache()
