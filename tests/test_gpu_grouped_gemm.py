"""The experts' FP8 products on the GPU against 64-bit sums of the codes'
values: every scale layout, segments of every size class, ragged widths."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import moe_inputs as mi
from gpu_path import dev, to_dev

pytestmark = pytest.mark.gpu

ROUND, WORDS, ROWS = 1, 2, 4
SENTINEL = 0x1234


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_moe_layout_03_amd import capi as c

    return c


class Case:
    """Codes and scales of the segments' rows; NaN codes and scales elsewhere."""

    def __init__(self, seed, counts, N, C, flags, per=0, gap=0, max_count=0):
        rng = np.random.default_rng(seed)
        self.counts, self.N, self.C, self.flags = counts, N, C, flags
        E, G = len(counts), C // 128
        self.E, self.max_count = E, max_count
        if flags & ROWS and not per:
            self.start, self.rows = ref.lay_rows(counts, "rows", 0, 1, gap)
        else:
            self.start, self.rows = ref.lay_rows(counts, "padded", per)
        self.live = ref.live_rows(self.start, counts)
        n = len(self.live)
        self.a = np.full((self.rows, C), 0x7F, np.uint8)
        self.a[self.live] = ref.random_codes(rng, (n, C))
        if flags & ROUND:
            e = rng.integers(110, 130, size=(n, G))
            s = np.exp2(e - 127.0)
        else:
            s = np.exp(rng.standard_normal((n, G))) * 0.01
            s = s.astype(np.float32).astype(np.float64)
        self.s = s
        if flags & WORDS:
            e = e.reshape(n, -1, 4)
            word = (e[..., 0] | e[..., 1] << 8 | e[..., 2] << 16 | e[..., 3] << 24)
            full = np.full((self.rows, G // 4), -1, np.int32)
            full[self.live] = word.astype(np.uint32).view(np.int32)
        else:
            full = np.full((self.rows, G), np.nan, np.float32)
            full[self.live] = s
        if not flags & ROWS:
            full = np.ascontiguousarray(
                full.reshape(E, self.rows // E, -1).transpose(0, 2, 1))
        self.scale = full
        self.w = ref.random_codes(rng, (E, N, C))
        self.ws = (np.exp(rng.standard_normal((E, (N + 127) // 128, G)) * 0.5)
                   * 0.01).astype(np.float32)

    def run(self, capi, status=None, stream=None, out=None):
        if out is None:
            out = torch.full((self.rows, self.N), SENTINEL, dtype=torch.int16, device=dev())
        capi.moe_grouped_gemm_fp8(
            self.E, self.N, self.C, to_dev(self.a), to_dev(self.scale), self.rows,
            to_dev(self.start), to_dev(np.array(self.counts, np.int32)), to_dev(self.w),
            to_dev(self.ws), out, self.flags, self.max_count, status, stream)
        torch.cuda.synchronize()
        return out.cpu().numpy().view(np.uint16)

    def check(self, got, experts=None):
        """Each result within half a bf16 step and the matrix unit's bound."""
        G = self.C // 128
        done = np.zeros(self.rows, bool)
        at = 0
        for e, c in enumerate(self.counts):
            c = max(c, 0)
            r = slice(self.start[e], self.start[e] + c)
            src = slice(at, at + c)
            at += c
            if c == 0 or (experts is not None and e not in experts):
                continue
            done[r] = True
            a = ref.e4m3_values(self.a[r]).reshape(c, G, 128) * self.s[src][..., None]
            b = ref.e4m3_values(self.w[e]).reshape(self.N, G, 128)
            b = b * np.repeat(self.ws[e].astype(np.float64), 128, 0)[:self.N, :, None]
            a, b = a.reshape(c, -1), b.reshape(self.N, -1)
            want = a @ b.T
            have = mi.bf16_bits_to_f32(got[r]).astype(np.float64)
            tol = ref.HALF_BF16 * np.abs(want) + ref.product_bound(a, b, G)
            assert np.all(np.abs(have - want) <= tol), (e, np.max(np.abs(have - want) / tol))
        assert np.all(got[~done] == SENTINEL)


COUNTS = [[1], [0, 2, 0], [16, 1, 0, 17, 33], [64, 65, 5], [130, 0, 15, 31, 300]]


@pytest.mark.parametrize("flags", [ROWS, ROWS | ROUND, ROWS | ROUND | WORDS])
@pytest.mark.parametrize("N,C", [(8, 128), (136, 640), (256, 512), (72, 1152)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_row_scales(capi, counts, N, C, flags):
    if flags & WORDS:
        C = (C + 511) // 512 * 512
    c = Case(sum(counts) + N + C, counts, N, C, flags, gap=3)
    c.check(c.run(capi))


@pytest.mark.parametrize("flags", [0, ROUND, ROUND | WORDS])
@pytest.mark.parametrize("N,C", [(8, 128), (200, 896), (256, 2048)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_column_scales(capi, counts, N, C, flags):
    if flags & WORDS:
        C = (C + 511) // 512 * 512
    c = Case(sum(counts) + N + C, counts, N, C, flags, per=max(counts) + 9)
    c.check(c.run(capi))


@pytest.mark.parametrize("flags", [ROWS, ROWS | ROUND | WORDS])
def test_scales_at_any_word(capi, flags):
    """Row-major scales that start on a word, not on 16 bytes, and 16-byte
    aligned operands that start inside their allocation."""
    c = Case(71, [9, 40, 0, 130], 200, 1024, flags)
    want = c.run(capi)
    c.check(want)

    def moved(x, n):  # the same values n elements into a larger buffer
        t = to_dev(x).reshape(-1)
        buf = torch.zeros(t.numel() + n, dtype=t.dtype, device=dev())
        buf[n:] = t
        return buf[n:]

    out = torch.full((c.rows, c.N), SENTINEL, dtype=torch.int16, device=dev())
    capi.moe_grouped_gemm_fp8(
        c.E, c.N, c.C, moved(c.a, 16), moved(c.scale, 1), c.rows, moved(c.start, 1),
        moved(np.array(c.counts, np.int32), 3), moved(c.w, 48), moved(c.ws, 1), out, c.flags)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy().view(np.uint16), want)


@pytest.mark.parametrize("c", [1, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 79, 80, 96, 97,
                               112, 113, 127, 128, 129, 143, 144, 159, 160, 161, 255, 256, 257,
                               511, 513])
def test_every_tile_edge(capi, c):
    """One segment of every size next to a tile's edge, beside a small one."""
    k = Case(c, [c, 2], 264, 384, ROWS)
    k.check(k.run(capi))


@pytest.mark.parametrize("C", [128, 256, 384, 512, 1024, 1408, 7168, 16384])
def test_channel_counts(capi, C):
    for counts in ([3, 1], [150, 20]):
        k = Case(C, counts, 80, C, ROWS)
        k.check(k.run(capi))


def test_wide_and_many_experts(capi):
    k = Case(1, [2, 0, 140], 2824, 256, ROWS)
    k.check(k.run(capi))
    rng = np.random.default_rng(2)
    k = Case(2, rng.integers(0, 5, size=1024).tolist(), 16, 128, 0, per=6)
    k.check(k.run(capi))
    k = Case(3, rng.integers(60, 70, size=40).tolist(), 40, 256, ROWS)
    k.check(k.run(capi))


def test_max_count_bound(capi):
    """A bound on the segments changes nothing for those within it; a larger
    segment is skipped and reported."""
    for bound in (3, 16, 64, 65, 100, 1000):
        counts = [bound, 1, 0, min(bound, 20)]
        k = Case(bound, counts, 64, 256, ROWS, max_count=bound)
        st = torch.zeros(1, dtype=torch.int32, device=dev())
        k.check(k.run(capi, st))
        assert int(st.item()) == 0
        k.counts = [bound + 1, 1, 0, min(bound, 20)]
        k2 = Case(bound + 5, k.counts, 64, 256, ROWS, max_count=bound)
        got = k2.run(capi, st)
        assert int(st.item()) == capi.MOE_STATUS_BAD_SLOT
        k2.check(got, experts=(1, 2, 3))


def test_bad_segments(capi):
    k = Case(7, [4, 4, 4, 4], 24, 128, ROWS)
    for e, (s, n) in enumerate([(-1, 4), (13, 4), (2 ** 31 - 1, 4), (0, 2 ** 31 - 1)]):
        start, counts = k.start.copy(), list(k.counts)
        k.start[e], k.counts[e] = s, n
        st = torch.zeros(1, dtype=torch.int32, device=dev())
        got = k.run(capi, st)
        assert int(st.item()) == capi.MOE_STATUS_BAD_SLOT
        k.start, k.counts = start, counts
        k.check(got, experts=[i for i in range(4) if i != e])
    # column-major scales: a segment may not leave its expert's rows
    k = Case(8, [3, 3], 24, 128, 0, per=8)
    start = k.start.copy()
    k.start[1] = 6
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    got = k.run(capi, st)
    assert int(st.item()) == capi.MOE_STATUS_BAD_SLOT
    k.start = start
    k.check(got, experts=[0])


def test_overlapping_counts_do_not_overflow(capi):
    """1024 segments that each claim a whole large buffer against the rules: the
    call reports them and writes nothing."""
    E, N, C, rows = 1024, 8, 128, 1 << 22
    a = torch.zeros(rows, C, dtype=torch.uint8, device=dev())
    sc = torch.ones(rows, 1, device=dev())
    w = torch.zeros(E, N, C, dtype=torch.uint8, device=dev())
    ws = torch.ones(E, 1, 1, device=dev())
    out = torch.full((rows, N), SENTINEL, dtype=torch.int16, device=dev())
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    capi.moe_grouped_gemm_fp8(E, N, C, a, sc, rows,
                              torch.zeros(E, dtype=torch.int32, device=dev()),
                              torch.full((E,), rows, dtype=torch.int32, device=dev()), w, ws, out,
                              ROWS, 0, st)
    torch.cuda.synchronize()
    assert int(st.item()) == capi.MOE_STATUS_BAD_SLOT
    assert bool((out == SENTINEL).all())


def test_offsets_past_32_bits(capi):
    """A buffer whose codes and results pass 2^31 bytes, segments at both ends."""
    E, N, C, rows = 2, 4096, 7168, 600_000
    rng = np.random.default_rng(12)
    n = (5, 70)
    start = np.array([3, rows - 71], np.int32)
    a = torch.zeros(rows, C, dtype=torch.uint8, device=dev())
    sc = torch.zeros(rows, C // 128, device=dev())
    out = torch.zeros(rows, N, dtype=torch.int16, device=dev())
    w, ws = ref.random_codes(rng, (E, N, C)), np.full((E, N // 128, C // 128), 0.01, np.float32)
    dw = to_dev(w)
    for e in range(E):
        r = slice(int(start[e]), int(start[e]) + n[e])
        a[r] = to_dev(ref.random_codes(rng, (n[e], C)))
        sc[r] = 0.02
    capi.moe_grouped_gemm_fp8(E, N, C, a, sc, rows, to_dev(start),
                              to_dev(np.array(n, np.int32)), dw, to_dev(ws), out, ROWS)
    torch.cuda.synchronize()
    s = float(np.float32(0.02)) * float(np.float32(0.01))
    for e in range(E):
        r = slice(int(start[e]), int(start[e]) + n[e])
        x = ref.e4m3_values(a[r].cpu().numpy())
        b = ref.e4m3_values(w[e])
        want = x @ b.T * s
        have = mi.bf16_bits_to_f32(out[r].cpu().numpy().view(np.uint16)).astype(np.float64)
        assert np.all(np.abs(have - want) <= ref.HALF_BF16 * np.abs(want)
                      + ref.product_bound(x, b * s, C // 128))
    used = [slice(3, 8), slice(rows - 71, rows - 1)]
    for r in used:
        out[r] = 0
    assert not bool(out.any())


def test_transposed_weights_give_the_row_gradient(capi):
    """The gradient with respect to the rows is the call on transposed weights:
    against the product of the cast gradients with the weights as stored."""
    N, C, counts = 256, 384, [20, 70]
    fwd = Case(31, counts, N, C, ROWS)
    bwd = Case(32, counts, C, N, ROWS)  # rows of width N: the cast gradient
    bwd.w = np.ascontiguousarray(fwd.w.transpose(0, 2, 1))
    bwd.ws = np.ascontiguousarray(fwd.ws.transpose(0, 2, 1))
    got = bwd.run(capi)
    bwd.check(got)
    at = 0
    for e, c in enumerate(counts):
        r = slice(bwd.start[e], bwd.start[e] + c)
        g = (ref.e4m3_values(bwd.a[r]).reshape(c, -1, 128)
             * bwd.s[at:at + c][..., None]).reshape(c, N)
        at += c
        w = ref.e4m3_values(fwd.w[e]) * np.repeat(np.repeat(fwd.ws[e], 128, 0), 128, 1)
        want = g @ w
        have = mi.bf16_bits_to_f32(got[r]).astype(np.float64)
        assert np.all(np.abs(have - want) <= ref.HALF_BF16 * np.abs(want)
                      + ref.product_bound(g, w.T, N // 128))


def test_large_beside_small_products(capi):
    """Codes of every size in one group: products 2^26 apart, where the matrix
    unit's alignment shows most. The bound holds, and across blocks of eight
    channels nothing of a small product is lost but the float's own rounding."""
    k = Case(51, [70, 3], 48, 256, ROWS)
    rng = np.random.default_rng(52)
    for arr in (k.a, k.w):
        big = rng.random(arr.shape) < 0.1
        arr[big & (arr != 0x7F)] = 0x7E
        small = rng.random(arr.shape) < 0.5
        arr[small & (arr != 0x7F) & ~big] = 0x01
    k.check(k.run(capi))
    k = Case(53, [5], 16, 128, ROWS)
    k.a[k.live], k.w[:], k.s[:], k.ws[:] = 0, 0, 1.0, 1.0
    k.scale[k.live] = 1.0
    k.a[k.live, 0], k.w[:, :, 0] = 0x78, 0x78      # 256 * 256
    k.a[k.live, 8::8], k.w[:, :, 8::8] = 0x39, 0x39  # 15 products of 1.265625
    got = k.run(capi)
    want = mi.to_bf16_bits(np.array([65536 + 15 * 1.265625], np.float32))[0]
    assert np.all(got[k.live] == want)


@pytest.mark.parametrize("counts", [[3, 2], [70, 20]], ids=["streamed", "tiled"])
def test_nan_stays_in_its_row_and_column(capi, counts):
    """A NaN code or scale of a row spoils that row, one of a weight row its
    column, for that expert alone."""
    k = Case(61, counts, 200, 512, ROWS)
    k.a[k.start[0] + 1, 300] = 0x7F
    k.scale[k.start[1], 2] = np.nan
    k.w[1, 77, 5] = 0xFF
    got = mi.bf16_bits_to_f32(k.run(capi)).astype(np.float64)
    nan = np.zeros(got.shape, bool)
    nan[k.start[0] + 1] = True
    nan[k.start[1]] = True
    nan[k.start[1]:k.start[1] + counts[1], 77] = True
    assert np.array_equal(np.isnan(got), nan & (np.isin(np.arange(k.rows), k.live)[:, None]))
    # a zero scale gives +-0 or nothing, an infinite one NaN or infinities, in its row alone
    k = Case(62, counts, 40, 256, ROWS)
    k.scale[k.start[0]] = 0.0
    k.scale[k.start[1]] = np.inf
    got = mi.bf16_bits_to_f32(k.run(capi)).astype(np.float64)
    assert np.all(got[k.start[0]] == 0) and not np.isfinite(got[k.start[1]]).any()
    rest = np.setdiff1d(k.live, [k.start[0], k.start[1]])
    assert np.isfinite(got[rest]).all()


def test_byte_scales_of_every_exponent(capi):
    """UE8M0 bytes 0 ... 254 as the powers of two they stand for."""
    for counts in ([16], [64]):
        k = Case(63, counts, 8, 512, ROWS | ROUND | WORDS)
        n = counts[0]
        k.a[k.live], k.w[:], k.ws[:] = 0x38, 0x38, 1.0  # ones
        byte = (np.arange(n) * 4 % 255).astype(np.int64)
        k.scale[k.live, 0] = byte.astype(np.int32)  # the first group's; the others' 2^-127
        got = mi.bf16_bits_to_f32(k.run(capi)).astype(np.float64)[k.live]
        want = 128 * (np.exp2(byte - 127.0) + 3 * np.exp2(-127.0))
        fin = want < 3.3e38
        assert np.all(np.abs(got - want[:, None])[fin] <= ref.HALF_BF16 * want[fin, None])
        assert np.all(np.isinf(got[~fin]))


def test_graph_of_both_kernels(capi):
    """A captured product whose segments are streamed and tiled, replayed on new
    rows and counts with eager calls between: every replay equals the eager one."""
    k = Case(71, [40, 3, 0, 100], 264, 512, ROWS)
    d = [to_dev(v) for v in (k.a, k.scale, k.start, np.array(k.counts, np.int32), k.w, k.ws)]
    out = torch.zeros(k.rows, k.N, dtype=torch.int16, device=dev())
    other = torch.zeros_like(out)
    cnt = [[40, 3, 0, 100], [0, 3, 0, 17], [1, 0, 0, 0], [40, 1, 0, 99]]

    def step(o, s):
        capi.moe_grouped_gemm_fp8(k.E, k.N, k.C, d[0], d[1], k.rows, d[2], d[3], d[4], d[5], o,
                                  k.flags, 0, None, s)

    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(out, stream)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step(out, stream)
    for c in cnt:
        d[3].copy_(torch.tensor(c, dtype=torch.int32))
        out.fill_(5)
        other.fill_(5)
        step(other, None)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, other)


def test_streams_and_repeat(capi):
    """Two calls at once on two streams, then again: the same bits."""
    ks = [Case(41, [90, 3, 0, 40], 264, 512, ROWS), Case(42, [1, 2, 3, 200], 128, 1024, ROWS)]
    alone = [k.run(capi) for k in ks]
    streams = [torch.cuda.Stream() for _ in ks]
    d = []
    for k in ks:
        d.append([to_dev(v) for v in (k.a, k.scale, k.start, np.array(k.counts, np.int32), k.w,
                                      k.ws)]
                 + [torch.full((k.rows, k.N), SENTINEL, dtype=torch.int16, device=dev())])
    torch.cuda.synchronize()
    for _ in range(3):
        for k, (a, s, st, c, w, ws, out), stream in zip(ks, d, streams):
            capi.moe_grouped_gemm_fp8(k.E, k.N, k.C, a, s, k.rows, st, c, w, ws, out, k.flags, 0,
                                      None, stream)
    torch.cuda.synchronize()
    for k, t, want in zip(ks, d, alone):
        assert np.array_equal(t[-1].cpu().numpy().view(np.uint16), want)
