"""Gradient of the weighted combine on the GPU: rows bit for bit (one float
product rounded to bf16), weights against the 64-bit sums."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import moe_inputs as mi
from gpu_path import dev, to_dev

pytestmark = pytest.mark.gpu

SENTINEL = 0x7E57


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_moe_layout_03_amd import capi as c

    return c


def bf16(bits):
    return mi.bf16_bits_to_f32(bits)


def case(orc, seed, T, H, E, R, K, A=1, neg=0.1, dup=0.1):
    w = mi.random_case(seed, T, H, E, R, K, A, neg_frac=neg, dup_frac=dup)
    lay = orc.layout(w.topk_idx, E, R, A)
    rng = np.random.default_rng(seed + 1)
    rows = max(lay["rows"], 1)
    y = mi.to_bf16_bits(rng.standard_normal((rows, H)).astype(np.float32))
    do = mi.to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    return w, lay["slot"].astype(np.int32), rows, y, do


def run(capi, w, slot, rows, y, do, weights=True, dweights=True, mask=None, pad=5):
    shape = capi.make_shape(w.T, w.H, w.E, w.R, w.K, w.A)
    dy = torch.full((rows + pad, w.H), SENTINEL, dtype=torch.int16, device=dev())
    dw = torch.full((w.T, w.K), float("nan"), device=dev()) if dweights else None
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    capi.moe_combine_grad(
        shape, to_dev(do), to_dev(y) if dweights else None, rows, to_dev(slot),
        to_dev(w.topk_weights) if weights else None, dy, dw,
        to_dev(w.topk_idx) if mask is not None else None,
        to_dev(mask) if mask is not None else None, st)
    torch.cuda.synchronize()
    return (dy.cpu().numpy().view(np.uint16), None if dw is None else dw.cpu().numpy(),
            int(st.item()))


def check(w, slot, rows, y, do, got_dy, got_dw, weights=True, mask=None):
    want = np.full(got_dy.shape, SENTINEL, np.uint16)
    d32, d64, y64 = bf16(do), bf16(do).astype(np.float64), bf16(y).astype(np.float64)
    L = w.E // w.R
    for t in range(w.T):
        for k in range(w.K):
            s = slot[t, k]
            if not 0 <= s < rows:
                if got_dw is not None:
                    assert got_dw[t, k] == 0
                continue
            e = w.topk_idx[t, k]
            if mask is not None and 0 <= e < w.E and mask[e // L]:
                want[s] = 0
                if got_dw is not None:
                    assert got_dw[t, k] == 0
                continue
            a = w.topk_weights[t, k] if weights else np.float32(1)
            want[s] = mi.to_bf16_bits(a * d32[t])
            if got_dw is not None:
                terms = d64[t] * y64[s]
                # a lane adds up to 8 ceil(H / 2048) products, then 11 more sums
                n = 8 * -(-w.H // 2048) + 12
                assert abs(got_dw[t, k] - terms.sum()) <= n * ref.EPS24 * np.abs(terms).sum()
    assert np.array_equal(got_dy, want)


SHAPES = [(1, 8, 4, 2, 1, 1), (5, 24, 8, 4, 3, 1), (64, 256, 16, 4, 2, 1), (17, 2056, 64, 8, 8, 16),
          (9, 7168, 256, 8, 8, 1), (40, 136, 32, 8, 6, 4), (3, 16392, 8, 8, 4, 1),
          (2, 64, 64, 64, 64, 1)]


@pytest.mark.parametrize("shp", SHAPES)
def test_combine_grad(capi, orc, shp):
    T, H, E, R, K, A = shp
    w, slot, rows, y, do = case(orc, T + H, T, H, E, R, K, A)
    dy, dw, st = run(capi, w, slot, rows, y, do)
    assert st == 0
    check(w, slot, rows, y, do, dy, dw)
    dy, dw, _ = run(capi, w, slot, rows, y, do, weights=False)  # the plain sum's gradient
    check(w, slot, rows, y, do, dy, dw, weights=False)
    dy, dw, _ = run(capi, w, slot, rows, y, do, dweights=False)  # rows alone, y not read
    check(w, slot, rows, y, do, dy, None)


@pytest.mark.parametrize("shp", SHAPES[2:6])
def test_masked_ranks(capi, orc, shp):
    T, H, E, R, K, A = shp
    w, slot, rows, y, do = case(orc, 3 * T + H, T, H, E, R, K, A)
    for on in ([], [1], list(range(R))):
        mask = np.zeros(R, np.int32)
        mask[on] = 3
        # infinities and NaN of a masked rank's rows are never read
        L = E // R
        bad = y.copy()
        for t in range(T):
            for k in range(K):
                e = w.topk_idx[t, k]
                if slot[t, k] >= 0 and 0 <= e < E and mask[e // L]:
                    bad[slot[t, k]] = 0x7FC0
        dy, dw, st = run(capi, w, slot, rows, bad, do, mask=mask)
        assert st == 0
        check(w, slot, rows, bad, do, dy, dw, mask=mask)


def test_special_values_and_bad_slots(capi, orc):
    """Any bf16 pattern in d_out: the product's rounding and NaN code; slots out
    of range are skipped and reported."""
    T, H, E, R, K = 6, 64, 8, 2, 2
    w, slot, rows, y, do = case(orc, 77, T, H, E, R, K, neg=0, dup=0)
    rng = np.random.default_rng(3)
    do = rng.integers(0, 1 << 16, size=do.shape, dtype=np.uint16)
    do[0, :6] = [0x7F80, 0xFF80, 0x8000, 0x0001, 0x7FC0, 0x7F7F]
    w.topk_weights[:] = rng.standard_normal((T, K)).astype(np.float32) * 10
    w.topk_weights[1] = [0.0, np.inf]
    dy, dw, st = run(capi, w, slot, rows, y, do)
    assert st == 0
    with np.errstate(all="ignore"):
        for t in range(T):
            for k in range(K):
                p = w.topk_weights[t, k] * bf16(do)[t]
                want = mi.to_bf16_bits(p)
                got = dy[slot[t, k]]
                nan = np.isnan(p)
                assert np.array_equal(got[~nan], want[~nan])
                assert np.all(got[nan] == 0x7FC0)
    s2 = slot.copy()
    s2[2, 1], s2[4, 0] = rows, -2
    do = mi.to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    w.topk_weights[:] = 0.5
    dy, dw, st = run(capi, w, s2, rows, y, do)
    assert st == capi.MOE_STATUS_BAD_SLOT
    check(w, s2, rows, y, do, dy, dw)


def test_adjoint_of_the_combine(capi, orc):
    """<d_out, combine(y)> = <d_y, y> for unrounded sums, and moving a weight
    moves it by its gradient: the combine is linear in both, so the difference
    of two combines over the step is the derivative but for rounding."""
    w, slot, rows, y, do = case(orc, 5, 12, 512, 16, 4, 3)
    shape = capi.make_shape(w.T, w.H, w.E, w.R, w.K, w.A)
    _, dw, _ = run(capi, w, slot, rows, y, do)

    def value(wt):
        out = torch.empty(w.T, w.H, dtype=torch.int16, device=dev())
        o32 = torch.empty(w.T, w.H, device=dev())
        capi.moe_combine(shape, to_dev(y), rows, to_dev(slot), to_dev(wt), out, o32)
        return (o32.double().cpu().numpy() * bf16(do).astype(np.float64)).sum(1)

    mag = (np.abs(bf16(y)).max() * np.abs(bf16(do)).astype(np.float64).sum(1))
    for k in range(w.K):
        a, b = w.topk_weights.copy(), w.topk_weights.copy()
        a[:, k] += np.float32(0.5)
        b[:, k] -= np.float32(0.5)
        num = (value(a) - value(b)) / (a[:, k].astype(np.float64) - b[:, k])
        # each output of the two combines is off by K + 2 half steps of its terms
        assert np.all(np.abs(num - dw[:, k]) <= 2 * (w.K + 2 + 24) * w.K * ref.EPS24 * 1.5 * mag)


def test_on_another_stream_and_repeat(capi, orc):
    w, slot, rows, y, do = case(orc, 9, 128, 7168, 256, 8, 8, neg=0, dup=0)
    shape = capi.make_shape(w.T, w.H, w.E, w.R, w.K, w.A)
    d, yy, s, wt = to_dev(do), to_dev(y), to_dev(slot), to_dev(w.topk_weights)
    torch.cuda.synchronize()
    got = []
    for _ in range(2):
        st = torch.cuda.Stream()
        dy = torch.zeros(rows, w.H, dtype=torch.int16, device=dev())
        dw = torch.zeros(w.T, w.K, device=dev())
        torch.cuda.synchronize()
        capi.moe_combine_grad(shape, d, yy, rows, s, wt, dy, dw, stream=st)
        st.synchronize()
        got.append((dy, dw))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_offsets_past_32_bits(capi):
    """Expert rows of more than 2^32 elements, slots at both ends and between."""
    T, H, E, R, K, rows = 3, 8192, 8, 2, 2, (1 << 19) + 5
    shape = capi.make_shape(T, H, E, R, K, 1)
    slot = torch.tensor([0, rows - 1, (1 << 18) + 1, rows - 3, -1, 7], dtype=torch.int32,
                        device=dev())
    g = torch.Generator(device="cuda").manual_seed(3)
    y = torch.zeros(rows, H, dtype=torch.bfloat16, device=dev())
    live = slot[slot >= 0].long()
    y[live] = torch.randn(5, H, generator=g, device=dev()).to(torch.bfloat16)
    d_out = torch.randn(T, H, generator=g, device=dev()).to(torch.bfloat16)
    w = torch.rand(T, K, generator=g, device=dev())
    d_y = torch.zeros(rows, H, dtype=torch.bfloat16, device=dev())
    d_w = torch.zeros(T, K, device=dev())
    capi.moe_combine_grad(shape, d_out, y, rows, slot, w, d_y, d_w)
    torch.cuda.synchronize()
    for p in range(T * K):
        t, k, s = p // K, p % K, int(slot[p])
        if s < 0:
            assert float(d_w[t, k]) == 0
            continue
        assert torch.equal(d_y[s], (w[t, k] * d_out[t].float()).to(torch.bfloat16))
        prod = d_out[t].double() * y[s].double()
        # H products added in float: half a step of the running sum each
        tol = H * 2.0 ** -24 * float(prod.abs().sum())
        assert abs(float(d_w[t, k]) - float(prod.sum())) <= tol
    d_y[live] = 0
    assert all(not bool(c.any()) for c in d_y.split(1 << 16))
