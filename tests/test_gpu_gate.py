"""Router and its gradient on the GPU against the 64-bit reference: ids equal,
weights and gradients within the rounding of the float arithmetic."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from gpu_path import dev

pytestmark = pytest.mark.gpu

SIG, REN = 2, 4
LOWEST = float(np.finfo(np.float32).min)


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_moe_layout_03_amd import capi as c

    return c


def run(capi, x, K, flags, scale, dw=None, ids=None):
    """x: a CPU tensor, float32 or bfloat16. -> ids, weights, d_logits, status."""
    T, E = x.shape
    d = x.to(dev())
    idx = torch.full((T, K), -77, dtype=torch.int64, device=dev())
    w = torch.full((T, K), float("nan"), device=dev())
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    capi.moe_gate(T, E, K, d, idx, w, flags, scale, st)
    dx = None
    if dw is not None:
        dx = torch.full_like(d, float("nan"))
        use = idx if ids is None else torch.from_numpy(ids).to(dev())
        capi.moe_gate_grad(T, E, K, d, use, torch.from_numpy(dw).to(dev()), dx, flags, scale, st)
    torch.cuda.synchronize()
    return (idx.cpu().numpy(), w.cpu().numpy().astype(np.float64),
            None if dx is None else dx.float().cpu().numpy().astype(np.float64), int(st.item()))


def steps(x, E):
    """Bound on the relative error of a weight, in half float steps. An
    exponential of a difference of up to D is off by D (the difference's own
    rounding), another D for log-sigmoids, and 4 (two steps of the exponential);
    the sum over E adds E / 64 + 9 additions; the quotient and the scale 2."""
    f = x[np.isfinite(x)]
    D = float(np.abs(f[np.abs(f) < 1e4]).max(initial=0)) * 2
    return 2 * (2 * D + 8) + E / 64 + 16


def check(x, ids, w, K, flags, scale, dw=None, dx=None, use=None, bf16=False):
    want_ids = ref.gate_select(x, K)
    assert np.array_equal(ids, want_ids)
    sg, rn = bool(flags & SIG), bool(flags & REN)
    n = steps(x, x.shape[1]) * ref.EPS24
    want = ref.gate_weights(x, want_ids, sg, rn, scale)
    assert np.all(np.abs(w - want) <= n * np.abs(want) + 1e-37)
    assert np.all(w[want_ids < 0] == 0)
    if dw is None:
        return
    use = want_ids if use is None else use
    g = ref.gate_grad(x, use, dw, sg, rn, scale)
    # every term of an entry is off by n relative to itself; their sum cancels,
    # so the bound takes the terms' magnitudes
    p = ref.gate_weights(x, use, sg, rn, 1.0)
    size = np.zeros_like(g)
    a = np.abs(dw.astype(np.float64) * scale)
    total = (a * p).sum(1, keepdims=True)
    for k in range(use.shape[1]):
        t = np.nonzero(use[:, k] >= 0)[0]
        np.add.at(size, (t, use[t, k]), (p * (a + total))[t, k])
    if not sg and not rn:
        with np.errstate(all="ignore"):
            xf = np.where(np.isfinite(x), x, -np.inf).astype(np.float64)
            m = xf.max(1, keepdims=True)
            e = np.exp(xf - np.where(np.isfinite(m), m, 0))
            s = e.sum(1, keepdims=True)
            size += e / np.where(s > 0, s, 1) * total
    tol = 3 * n * size + 1e-37 + (ref.HALF_BF16 * np.abs(g) if bf16 else 0)
    assert np.all(np.abs(dx - g) <= tol), np.max(np.abs(dx - g) - tol)


SHAPES = [(1, 1, 1), (3, 5, 5), (1, 64, 6), (7, 60, 4), (16, 256, 8), (33, 65, 8), (5, 128, 64),
          (130, 160, 6), (2, 1024, 64), (9, 1000, 1), (6, 300, 7), (1025, 64, 2)]


@pytest.mark.parametrize("flags", [0, SIG, REN, SIG | REN])
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_gate_and_gradient(capi, T, E, K, flags):
    rng = np.random.default_rng(T * 7 + E + K + flags)
    for bf16 in (False, True):
        x = torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32))
        if bf16:
            x = x.to(torch.bfloat16)  # many equal logits: ties go to the lower id
        dw = rng.standard_normal((T, K)).astype(np.float32)
        ids, w, dx, st = run(capi, x, K, flags, 2.5, dw)
        check(x.float().numpy(), ids, w, K, flags, 2.5, dw, dx, bf16=bf16)
        assert st == 0


@pytest.mark.parametrize("flags", [0, SIG, REN, SIG | REN])
def test_masks_ties_and_extremes(capi, flags):
    E, K = 70, 4
    inf = np.inf
    rows = {
        "all masked": np.full(E, -inf),
        "three left": np.where(np.isin(np.arange(E), [3, 66, 69]), 0.5, -inf),
        "one left, lowest": np.where(np.arange(E) == 68, LOWEST, -inf),
        "all lowest": np.full(E, LOWEST),
        "lowest but two": np.where(np.arange(E) >= 68, 1.0, LOWEST),
        "all equal": np.zeros(E),
        "zeros of both signs": np.where(np.arange(E) % 2, 0.0, -0.0),
        "far apart": np.where(np.arange(E) == 40, 80.0, -90.0),
        "large": np.arange(E) * 1.0 + 2500.0,
        "very negative": np.arange(E) * 0.5 - 2000.0,
        "largest": np.where(np.arange(E) == 1, -LOWEST, np.arange(E) * 0.01),
        "subnormal": np.arange(E) * 1e-45,
    }
    x = np.stack(list(rows.values())).astype(np.float32)
    rng = np.random.default_rng(5)
    dw = rng.standard_normal((len(rows), K)).astype(np.float32)
    ids, w, dx, st = run(capi, torch.from_numpy(x), K, flags, 1.0, dw)
    assert st == 0
    for i, name in enumerate(rows):
        one = slice(i, i + 1)
        try:
            # rounding a difference of thousands costs that many half steps
            # more: the bound of `steps` holds it
            check(x[one], ids[one], w[one], K, flags, 1.0, dw[one], dx[one])
        except AssertionError as e:
            raise AssertionError(name) from e
    assert np.isfinite(w).all() and np.isfinite(dx).all()


def test_nan_and_infinity_are_masked_and_reported(capi):
    rng = np.random.default_rng(8)
    x = rng.standard_normal((6, 33)).astype(np.float32)
    x[1, 4], x[2, 32], x[3, :] = np.nan, np.inf, np.nan
    x[4, 5] = -np.nan
    dw = rng.standard_normal((6, 3)).astype(np.float32)
    for flags in (0, SIG, REN, SIG | REN):
        ids, w, dx, st = run(capi, torch.from_numpy(x), 3, flags, 1.0, dw)
        assert st == capi.MOE_STATUS_BAD_LOGIT
        check(x, ids, w, 3, flags, 1.0, dw, dx)
        assert (ids[3] == -1).all() and (w[3] == 0).all() and (dx[3] == 0).all()


def test_gradient_of_given_ids(capi):
    """Ids of another selection, the same id twice, -1, masked and bad ids."""
    rng = np.random.default_rng(11)
    T, E, K = 8, 40, 4
    x = rng.standard_normal((T, E)).astype(np.float32)
    x[:, 7] = -np.inf
    ids = np.array([[1, 2, 3, 4], [5, 5, 5, 5], [-1, -1, -1, -1], [7, 0, -1, 39], [9, 9, -1, 2],
                    [7, 7, 7, 7], [39, 0, 38, 1], [3, 3, 12, 12]], dtype=np.int64)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    for flags in (0, SIG, REN, SIG | REN):
        i0, w, dx, st = run(capi, torch.from_numpy(x), K, flags, 1.5, dw, ids)
        assert st == 0
        check(x, i0, w, K, flags, 1.5, dw, dx, use=ids)
        bad = ids.copy()
        bad[0, 0], bad[6, 3], bad[2, 1] = E, -2, 1 << 40
        _, _, dx, st = run(capi, torch.from_numpy(x), K, flags, 1.5, dw, bad)
        assert st == capi.MOE_STATUS_BAD_EXPERT
        good = np.where((bad < 0) | (bad >= E), -1, bad)
        check(x, i0, w, K, flags, 1.5, dw, dx, use=good)


@pytest.mark.parametrize("flags", [0, SIG, REN, SIG | REN])
def test_gradient_against_differences(capi, flags):
    """Central differences of the 64-bit weights. With step h the difference is
    off by h^2 / 6 times a third derivative, which for these functions of the
    logits is at most 6 sum |dw| scale; the GPU's gradient by its rounding."""
    rng = np.random.default_rng(21 + flags)
    T, E, K, h = 3, 12, 4, 1e-4
    x = rng.standard_normal((T, E)).astype(np.float32)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    ids, _, dx, _ = run(capi, torch.from_numpy(x), K, flags, 1.25, dw)
    sg, rn = bool(flags & SIG), bool(flags & REN)
    size = np.abs(dw).sum(1).max() * 1.25
    for e in range(E):
        up, lo = x.astype(np.float64), x.astype(np.float64)
        up, lo = up.copy(), lo.copy()
        up[:, e] += h
        lo[:, e] -= h
        num = ((ref.gate_weights(up, ids, sg, rn, 1.25)
                - ref.gate_weights(lo, ids, sg, rn, 1.25)) * dw).sum(1) / (2 * h)
        assert np.all(np.abs(num - dx[:, e]) <= h * h * size + 1e-11 / h
                      + 3 * steps(x, E) * ref.EPS24 * size)


def test_empty_batch_and_repeat(capi):
    e = torch.empty(0, 16, device=dev())
    capi.moe_gate(0, 16, 2, e, torch.empty(0, 2, dtype=torch.int64, device=dev()),
                  torch.empty(0, 2, device=dev()))
    x = torch.randn(513, 256, device=dev())
    got = []
    for _ in range(2):
        idx = torch.empty(513, 8, dtype=torch.int64, device=dev())
        w = torch.empty(513, 8, device=dev())
        d = torch.empty_like(x)
        capi.moe_gate(513, 256, 8, x, idx, w)
        capi.moe_gate_grad(513, 256, 8, x, idx, w, d)
        got.append((idx.clone(), w.clone(), d.clone()))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_gradient_of_unselected_experts(capi):
    """An unselected expert's own gradient is -p_e times a number: its p_e has to
    be good by itself, also where it is a small part of the sum. The differences
    to the largest logit are whole numbers, so nothing is lost in them. In half
    float steps: the exponential 2, the sum over E = 64 terms 2 + 9 + 1, which
    counts for the selected p and for the quotient (24), two quotients and three
    products 5: 31. (The smallest of them is still a normal float.)"""
    E = 64
    x = np.full((24, E), -90.0, np.float32)
    x[:, 5] = 0.0
    x[:, 20:47] = -np.arange(60, 87)  # 27 distances
    x[12:] += 64.0
    ids = np.full((24, 1), 5, np.int64)
    dw = (np.linspace(1, 3, 24) * np.tile([1, -1], 12)).astype(np.float32)[:, None]
    _, _, dx, st = run(capi, torch.from_numpy(x), 1, 0, 1.0, dw, ids)
    want = ref.gate_grad(x, ids, dw, False, False, 1.0)
    assert st == 0
    off = np.abs(dx - want)[:, 20:47] / np.abs(want)[:, 20:47]
    assert off.max() <= 31 * ref.EPS24, off.max() / ref.EPS24


@pytest.mark.parametrize("E", [40, 200, 700])
@pytest.mark.parametrize("flags", [0, SIG, REN, SIG | REN])
def test_masked_logits_get_zero_from_any_weight_gradient(capi, flags, E):
    """NaN and infinities among d_weights reach unmasked logits only, of their
    own token."""
    K = 4
    rng = np.random.default_rng(E)
    x = rng.standard_normal((6, E)).astype(np.float32)
    x[:, ::3] = -np.inf
    x[5, 1] = np.nan
    dw = rng.standard_normal((6, K)).astype(np.float32)
    clean = dw.copy()
    dw[0, 1], dw[1, 0], dw[2, 3], dw[3, 2], dw[5, 0] = (np.nan, np.inf, -np.inf, 3.4e38, np.nan)
    d = torch.from_numpy(x)
    _, _, dx, _ = run(capi, d, K, flags, 2.0, dw)
    _, _, want, _ = run(capi, d, K, flags, 2.0, clean)
    assert np.all(dx[~np.isfinite(x)] == 0)
    assert np.array_equal(dx[4], want[4])
    assert np.isnan(dx[0]).any() and np.isnan(dx[5]).any()
