"""Router with a balance bias and groups on the GPU against the 64-bit reference:
ids equal, weights within the rounding of the float arithmetic."""
import numpy as np
import pytest
import torch

import dense_ref as ref
from gpu_path import dev

pytestmark = pytest.mark.gpu

BF16, SIG, REN, SUM2 = 1, 2, 4, 8


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_moe_layout_03_amd import capi as c

    return c


def run(capi, x, bias, K, G, KG, flags, scale):
    T, E = x.shape
    idx = torch.full((T + 1, K), -77, dtype=torch.int64, device=dev())
    w = torch.full((T + 1, K), float("nan"), device=dev())
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    b = None if bias is None else torch.from_numpy(bias).to(dev())
    capi.moe_gate_grouped(T, E, K, G, KG, x.to(dev()), b, idx, w, flags, scale, st)
    torch.cuda.synchronize()
    assert bool((idx[T] == -77).all()) and bool(torch.isnan(w[T]).all())
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy().astype(np.float64), int(st.item())


def check(capi, x, bias, K, G, KG, flags, scale=1.0, status=0):
    ids, w, st = run(capi, x, bias, K, G, KG, flags, scale)
    v = x.float().numpy().astype(np.float64)
    sg, rn = bool(flags & SIG), bool(flags & REN)
    want, s = ref.grouped_select(v, bias, K, G, KG, sg, bool(flags & SUM2))
    assert np.array_equal(ids, want)
    ww = ref.grouped_weights(v, want, s, sg, rn, scale)
    # an exponential of a difference D is off by D and four half steps, a
    # log-sigmoid by as much again; the sum over E adds E / 64 + 9, quotients 4
    f = v[np.isfinite(v) & (np.abs(v) < 1e4)]
    n = 2 * (4 * float(np.abs(f).max(initial=0)) + 8) + x.shape[1] / 64 + 16
    assert np.all(np.abs(w - ww) <= n * ref.EPS24 * np.abs(ww) + 1e-37)
    assert st == status
    return ids


def logits(T, E, seed, bf16=False, sd=1.5):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((T, E)) * sd).astype(np.float32))
    return x.to(torch.bfloat16) if bf16 else x


def biases(E, seed, sd=0.1):
    return (np.random.default_rng(seed).standard_normal(E) * sd).astype(np.float32)


@pytest.mark.parametrize("E,G,KG,K", [
    (1, 1, 1, 1), (8, 2, 1, 4), (8, 8, 3, 2), (60, 4, 2, 6), (60, 1, 1, 8), (64, 64, 5, 5),
    (64, 8, 4, 6), (96, 3, 2, 8), (128, 8, 8, 8), (160, 8, 3, 6), (256, 8, 4, 8), (256, 1, 1, 8),
    (256, 64, 9, 16), (320, 5, 2, 8), (512, 8, 4, 12), (1000, 10, 3, 8), (1024, 64, 2, 64),
    (1024, 4, 1, 64)])
@pytest.mark.parametrize("flags", [SIG | REN | SUM2, SIG, REN, SUM2])
def test_shapes(capi, E, G, KG, K, flags):
    for T, bf16 in ((1, True), (37, False)):
        check(capi, logits(T, E, E + G + T, bf16), biases(E, E), K, G, KG, flags, 2.5)
    check(capi, logits(9, E, E + 5, True), None, K, G, KG, flags)


@pytest.mark.parametrize("flags", [SIG | REN | SUM2, SUM2, SIG | REN])
def test_many_tokens(capi, flags):
    """Enough tokens that some choices fall closer together than floats tell apart."""
    x = logits(3000, 256, 11)
    check(capi, x, biases(256, 12), 8, 8, 4, flags, 2.5)
    check(capi, x.to(torch.bfloat16), np.zeros(256, np.float32), 8, 8, 4, flags)


@pytest.mark.parametrize("flags", [SIG, SIG | SUM2, 0, SUM2])
def test_choices_a_float_merges(capi, flags):
    """Logits one float step apart, and biases that make up for all but the last bits."""
    rng = np.random.default_rng(3)
    T, E = 64, 256
    base = np.float32(1.25)
    x = np.full((T, E), base, np.float32)
    for t in range(T):
        for e in rng.permutation(E):
            x[t, e] = np.nextafter(base, np.float32(9), dtype=np.float32) if rng.random() < 0.4 else base
    check(capi, torch.from_numpy(x), None, 8, 8, 4, flags)
    y = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    s = 1 / (1 + np.exp(-y[0].astype(np.float64)))
    bias = (0.75 - s).astype(np.float32)  # row 0: all choices within a float step of 0.75
    y[1:32] = y[0]
    check(capi, torch.from_numpy(y), bias, 8, 8, 4, flags | SIG)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("flags", [SIG | REN | SUM2, SIG, SUM2, REN])
def test_ties_go_to_the_lower_id(capi, bf16, flags):
    x = torch.zeros(5, 256)
    x[1, ::2] = 1.0
    x[2, 200:] = 3.0
    x[3] = torch.arange(256).float() % 3
    x[4] = torch.finfo(torch.float32).min if not bf16 else -1e30
    x = x.to(torch.bfloat16) if bf16 else x
    check(capi, x, None, 8, 8, 4, flags)
    check(capi, x, np.zeros(256, np.float32), 8, 8, 4, flags)
    check(capi, x, np.where(np.arange(256) % 5 == 0, 0.5, -0.5).astype(np.float32), 8, 8, 4, flags)


@pytest.mark.parametrize("flags", [SIG | REN | SUM2, SIG | REN, SUM2, REN, SIG, 0])
def test_masks(capi, flags):
    """Masked experts by logit and by bias, groups without an expert, with one, tokens
    without any."""
    x = logits(8, 64, 21)
    x[0] = -np.inf
    x[1, :56] = -np.inf           # one group is left
    x[2, 1:] = -np.inf            # one expert
    x[3, 8:16] = -np.inf          # a group gone
    x[4, 9:16] = -np.inf          # a group of one
    x[5, ::2] = -np.inf
    ids = check(capi, x, biases(64, 4), 6, 8, 3, flags)
    assert (ids[0] == -1).all() and ids[2, 0] == 0 and (ids[2, 1:] == -1).all()
    b = biases(64, 5)
    b[:32] = -np.inf
    ids = check(capi, x, b, 6, 8, 3, flags)
    assert not np.any((ids >= 0) & (ids < 32))
    b[:] = -np.inf
    assert (check(capi, x, b, 6, 8, 3, flags) == -1).all()


@pytest.mark.parametrize("flags", [SIG | REN | SUM2, SUM2, REN])
def test_bad_values_are_masked_and_reported(capi, flags):
    x = logits(4, 64, 31)
    x[1, 5], x[2, 7], x[3, 9] = float("nan"), float("inf"), -float("nan")
    check(capi, x, None, 8, 8, 4, flags, status=16)
    b = biases(64, 6)
    b[3], b[60] = np.nan, np.inf
    check(capi, logits(4, 64, 32), b, 8, 8, 4, flags, status=16)


def test_extreme_logits(capi):
    big = float(np.finfo(np.float32).max)
    x = logits(4, 64, 41)
    x[0, :4] = torch.tensor([big, -big, 88.0, -104.0])
    x[1] *= 20
    x[2] = torch.linspace(-30, 30, 64)
    for flags in (SIG | REN | SUM2, SIG, REN, 0):
        check(capi, x, biases(64, 7), 8, 8, 4, flags)
    b = biases(64, 8)
    b[::7] *= 1e4  # biases far larger than the scores
    check(capi, x, b, 8, 8, 4, SIG | SUM2)


def test_one_group_is_the_plain_router(capi):
    """Without bias and groups the ids and weights are moe_gate's."""
    for bf16 in (False, True):
        x = logits(100, 256, 51, bf16).to(dev())
        for flags in (0, SIG, REN, SIG | REN):
            a, b = (torch.empty(100, 8, dtype=torch.int64, device=dev()) for _ in range(2))
            u, v = (torch.empty(100, 8, device=dev()) for _ in range(2))
            capi.moe_gate(100, 256, 8, x, a, u, flags, 2.0)
            capi.moe_gate_grouped(100, 256, 8, 1, 1, x, None, b, v, flags, 2.0)
            assert torch.equal(a, b)
            assert bool(((u - v).abs() <= 8 * ref.EPS24 * u).all())


def test_empty(capi):
    e = torch.empty(0, 64, device=dev())
    i, w = torch.empty(0, 4, dtype=torch.int64, device=dev()), torch.empty(0, 4, device=dev())
    capi.moe_gate_grouped(0, 64, 4, 8, 2, e, None, i, w)


@pytest.mark.parametrize("E,G,KG", [(256, 8, 4), (160, 8, 3), (64, 8, 4)])
@pytest.mark.parametrize("bf16", [False, True])
def test_rows_that_start_anywhere(capi, E, G, KG, bf16):
    """Logits and bias aligned to their own type only: the same ids and weights."""
    T, K = 21, 6
    x = logits(T, E, 61, bf16).to(dev())
    b = torch.from_numpy(biases(E, 62)).to(dev())
    want = None
    for off in (0, 1, 2, 3, 5):
        xs = torch.zeros(T * E + 8, dtype=x.dtype, device=dev())[off:off + T * E].view(T, E)
        bs = torch.zeros(E + 8, device=dev())[off:off + E]
        xs.copy_(x)
        bs.copy_(b)
        idx = torch.empty(T, K, dtype=torch.int64, device=dev())
        w = torch.empty(T, K, device=dev())
        capi.moe_gate_grouped(T, E, K, G, KG, xs, bs, idx, w, SIG | SUM2, 1.0)
        if want is None:
            want = idx.clone(), w.clone()
            assert np.array_equal(idx.cpu().numpy(), ref.grouped_select(
                x.float().cpu().numpy().astype(np.float64), b.cpu().numpy(), K, G, KG, True, True)[0])
        assert torch.equal(idx, want[0]) and bool(((w - want[1]).abs() <= 8 * ref.EPS24 * w).all())


@pytest.mark.parametrize("K", [8, 9, 15, 16])
def test_many_places_in_one_lane(capi, K):
    """The best experts all neighbours, so that one lane's list runs out; and near ties
    among them."""
    T, E = 8, 256
    x = logits(T, E, 71) * 0.1
    for t in range(T):
        s = 16 * (t % 15)
        x[t, s:s + 16] += 3.0
        if t % 2:
            x[t, s:s + 16] = 3.0 + torch.arange(16).flip(0) * 2.0 ** -22
        if t % 3 == 2:
            x[t, s + 16:s + 20] = x[t, s + 9]
    for flags in (SIG, SIG | REN | SUM2, 0):
        check(capi, x, np.full(256, 0.25, np.float32), K, 8, 3, flags)
        check(capi, x, None, K, 8, 3, flags)
        check(capi, x.to(torch.bfloat16), None, K, 1, 1, flags)


@pytest.mark.parametrize("flags", [SIG | SUM2, SUM2, SIG])
def test_groups_too_near_to_tell(capi, flags):
    """Groups whose sums differ by less than their floats' errors, or not at all."""
    rng = np.random.default_rng(81)
    T, E = 32, 256
    x = (rng.standard_normal((T, E)) * 0.5 - 3).astype(np.float32)
    for t in range(T):
        for g in range(8):
            x[t, g * 32 + 5] = np.float32(1.0) + np.float32(rng.integers(0, 3)) * 2.0 ** -23
            x[t, g * 32 + 9 + g] = np.float32(0.5) + np.float32(rng.integers(0, 3)) * 2.0 ** -24
    check(capi, torch.from_numpy(x), None, 6, 8, 4, flags)
    check(capi, torch.from_numpy(x), np.full(256, 0.125, np.float32), 6, 8, 4, flags)
    check(capi, torch.from_numpy(x).to(torch.bfloat16), None, 6, 8, 4, flags)


@pytest.mark.parametrize("flags", [0, SUM2, REN])
@pytest.mark.parametrize("E,G,KG", [(256, 8, 4), (64, 1, 1), (96, 3, 2)])
def test_softmax_choices_a_float_merges(capi, flags, E, G, KG):
    """Biases that make up for all but the last bits of a softmax."""
    rng = np.random.default_rng(91)
    y = (rng.standard_normal((16, E)) * 1.5).astype(np.float32)
    y[1:8] = y[0]
    e = np.exp(y[0].astype(np.float64) - y[0].max())
    bias = (0.5 - e / e.sum()).astype(np.float32)
    check(capi, torch.from_numpy(y), bias, 6, G, KG, flags)
    check(capi, torch.from_numpy(y).to(torch.bfloat16), bias, 6, G, KG, flags)
