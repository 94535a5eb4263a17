"""Groups' scores of the router in the float's far corners, on the GPU against 64 bits:
biases that take a group's sum past the float range, or leave little of it."""
import numpy as np
import pytest
import torch

from gpu_path import dev
from test_gpu_gate_grouped import REN, SIG, SUM2, capi, check, logits  # noqa: F401

pytestmark = pytest.mark.gpu

FLT_MAX = np.finfo(np.float32).max


@pytest.mark.parametrize("E", [64, 128, 256, 96])  # four tokens a wave; one (96)
@pytest.mark.parametrize("flags", [SIG | SUM2, SUM2, SIG | REN | SUM2])
def test_masked_group_beside_lowest_biases(capi, E, flags):
    """Every bias the lowest float: the sum of two passes the range, and still beats a
    group whose experts are all masked."""
    x = logits(5, E, E)
    n = E // 8
    x[:, :n] = -np.inf
    ids = check(capi, x, np.full(E, -FLT_MAX, np.float32), 4, 8, 1, flags)
    assert (ids == n + np.arange(4)).all()


@pytest.mark.parametrize("E", [64, 160, 256, 96])
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
