"""Groups' scores of the router in the float's far corners, on the GPU against 64 bits:
biases that take a group's sum past the float range, or leave little of it."""
import numpy as np
import pytest
import torch

from gpu_path import dev
from test_gpu_gate_grouped import REN, SIG, SUM2, capi, check, logits  # noqa: F401

pytestmark = pytest.mark.gpu

FLT_MAX = np.finfo(np.float32).max


@pytest.mark.parametrize("E", [64, 128, 256, 96, 112])  # four tokens a wave; one (112)
@pytest.mark.parametrize("flags", [SIG | SUM2, SUM2, SIG | REN | SUM2])
def test_masked_group_beside_lowest_biases(capi, E, flags):
    """Every bias the lowest float: the sum of two passes the range, and still beats a
    group whose experts are all masked."""
    x = logits(5, E, E)
    n = E // 8
    x[:, :n] = -np.inf
    ids = check(capi, x, np.full(E, -FLT_MAX, np.float32), 4, 8, 1, flags)
    assert (ids == n + np.arange(4)).all()


@pytest.mark.parametrize("E", [64, 160, 256, 96, 112])
@pytest.mark.parametrize("flags", [SIG | SUM2, SUM2, SIG, 0])
def test_group_sums_past_the_float_range(capi, E, flags):
    """Sums of either sign past the range differ in 64 bits, and from ordinary ones."""
    rng = np.random.default_rng(E + flags)
    n = E // 8
    for turn in range(12):
        b = (rng.uniform(1.8e38, FLT_MAX, E) * rng.choice([-1, 1], E)).astype(np.float32)
        if turn % 3 == 1:
            b[:3 * n] = rng.standard_normal(3 * n)
        if turn % 3 == 2:  # all alike but for the last bits
            b = np.full(E, rng.choice([-1, 1]) * 3e38, np.float32)
            b = np.where(rng.random(E) < 0.5, b, np.nextafter(b, np.float32(0)))
        x = logits(4, E, turn)
        x[1, n:2 * n] = -np.inf
        check(capi, x, b, 6, 8, 3, flags)


@pytest.mark.parametrize("E,G", [(64, 16), (64, 8), (160, 8), (256, 8), (96, 8), (112, 8)])
@pytest.mark.parametrize("size", [100.0, 1000.0, 10000.0])
@pytest.mark.parametrize("flags", [SIG | SUM2, SUM2, SIG | REN | SUM2])
def test_group_sums_that_cancel(capi, E, G, size, flags):
    """A group's best two of opposite sign, each rounded at its own size: what is left
    is off by many steps of its own, and the groups differ by less."""
    rng = np.random.default_rng(E + G)
    T, n = 48, E // G
    b = np.full(E, -size, np.float32)
    b[::n] = size
    step = size * 2.0 ** -23 * (1 if flags & SIG else G)  # of a choice's float, in these units
    first = rng.uniform(0.2, 0.8, (T, G))
    s = np.full((T, G, n), 1e-3)
    s[..., 0] = first
    s[..., 1] = 1 - first + rng.uniform(0, 2, (T, G)) * step
    x = np.log(s) - (np.log1p(-s) if flags & SIG else 0)
    check(capi, torch.from_numpy(x.reshape(T, E).astype(np.float32)), b, 6, G, 4, flags)


def sigmoid(x):
    return 1 / (1 + np.exp(-x.astype(np.float64)))


def first_above(s):
    """The least float whose sigmoid, in 64 bits, is above s."""
    x = (np.log(s) - np.log1p(-s)).astype(np.float32)
    while np.any(sigmoid(x) > s):
        x = np.where(sigmoid(x) > s, np.nextafter(x, np.float32(-99), dtype=np.float32), x)
    while np.any(sigmoid(x) <= s):
        x = np.where(sigmoid(x) <= s, np.nextafter(x, np.float32(99), dtype=np.float32), x)
    return x


@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("E", [64, 256, 96, 112])
def test_second_best_far_larger_than_the_best(capi, E, first):
    """Second best choices near -1000, whose floats are 2^-14 apart, beside best ones near
    1. Two experts of a group lie just above a border between two such floats, the larger
    one with the score that has fewer bits left, so that its float may fall below; the
    other group's second best lies between the two."""
    m = (np.arange(1 << 14) + 0.5) * 2.0 ** -14
    m = m[(m > 0.86) & (m < 0.94)]
    low = first_above(m - 0.75 + 1e-8)
    mid = np.nextafter(low, np.float32(99), dtype=np.float32)
    high = first_above(sigmoid(mid) + 0.75 + 1e-9)
    T, n = len(m), E // 2
    x = np.full((T, 2, n), -40.0, np.float32)
    b = np.full((2, n), -1000.0, np.float32)
    x[:, :, 0], b[:, 0] = 2.0, 0.0
    x[:, first, 1], b[first, 1] = high, -1000.75
    x[:, first, 2] = low
    x[:, 1 - first, 1] = mid
    x = torch.from_numpy(x.reshape(T, E)).to(dev())
    idx = torch.empty(T, 1, dtype=torch.int64, device=dev())
    w = torch.empty(T, 1, device=dev())
    capi.moe_gate_grouped(T, E, 1, 2, 1, x, torch.from_numpy(b.reshape(-1)).to(dev()), idx, w,
                          SIG | SUM2)
    wrong = int((idx != n * first).sum())
    assert wrong == 0, (wrong, T)
