"""The grouped router at every number of experts a lane holds, on the GPU against 64
bits: equal and nearly equal choices at the ends of lanes, lists and groups."""
import numpy as np
import pytest
import torch

from test_gpu_gate_grouped import REN, SIG, SUM2, biases, capi, check, logits  # noqa: F401

pytestmark = pytest.mark.gpu

WIDTHS = [2, 4, 6, 8, 10, 12, 14, 16]


@pytest.mark.parametrize("v", WIDTHS)
@pytest.mark.parametrize("lanes", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("flags", [SIG | REN | SUM2, SIG, SUM2, REN])
def test_groups(capi, v, lanes, flags):
    E, G = 16 * v, 16 // lanes
    KG = max(1, G // 3)
    for T, bf16, K in ((1, True, 1), (37, False, 8), (9, True, 15)):
        x = logits(T, E, E + lanes + T, bf16)
        check(capi, x, biases(E, E), K, G, KG, flags, 2.5)
        check(capi, x, None, K, G, KG, flags)
        if T > 1:
            x[0] = -np.inf
            x[1, ::2] = -np.inf
            x[2, lanes * v:] = -np.inf
            check(capi, x, biases(E, E + 1), K, G, KG, flags)


@pytest.mark.parametrize("v", WIDTHS)
@pytest.mark.parametrize("K", [8, 9, 15])
def test_lists_that_run_out(capi, v, K):
    """The best experts all in one lane, equal or a few float steps apart, and as near
    ones in the next."""
    T, E = 16, 16 * v
    x = logits(T, E, v) * 0.1
    for t in range(T):
        s = v * (t % 15)
        x[t, s:s + v] += 3.0
        if t % 2:
            x[t, s:s + v] = 3.0 + torch.arange(v).flip(0) * 2.0 ** -22
        if t % 3 == 2:
            x[t, s + v:s + v + min(v, 4)] = x[t, s + v // 2]
    for flags in (SIG, SIG | REN | SUM2, 0):
        check(capi, x, np.full(E, 0.25, np.float32), K, 8, 3, flags)
        check(capi, x, None, K, 8, 3, flags)
        check(capi, x.to(torch.bfloat16), None, K, 1, 1, flags)


@pytest.mark.parametrize("v", WIDTHS)
@pytest.mark.parametrize("flags", [SIG | SUM2, SUM2, SIG, 0])
def test_choices_a_float_merges(capi, v, flags):
    """Equal logits but for the last bit, and biases that make up for all but the last bits."""
    rng = np.random.default_rng(v)
    T, E = 16, 16 * v
    base = np.float32(1.25)
    x = np.where(rng.random((T, E)) < 0.4, np.nextafter(base, np.float32(9)), base)
    check(capi, torch.from_numpy(x.astype(np.float32)), None, 6, 8, 4, flags)
    y = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    y[1:] = y[0]
    z = y[0].astype(np.float64)
    s = 1 / (1 + np.exp(-z)) if flags & SIG else np.exp(z - z.max()) / np.exp(z - z.max()).sum()
    check(capi, torch.from_numpy(y), (0.75 - s).astype(np.float32), 6, 8, 4, flags)
