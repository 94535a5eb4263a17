"""Gradient of the weights of a grouped, biased selection on the GPU against 64 bits:
moe_gate_grad with the ids that moe_gate_grouped gave."""
import numpy as np
import pytest
import torch

import dense_ref
import experts_ref as ref
from gpu_path import dev
from test_gpu_gate import steps
from test_gpu_gate_grouped import REN, SIG, SUM2, biases, capi, logits, run  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("E,G,KG,K", [(64, 8, 3, 6), (96, 3, 2, 8), (160, 8, 3, 6), (256, 8, 4, 8),
                                      (1000, 10, 3, 8)])
@pytest.mark.parametrize("flags", [0, SIG, REN, SIG | REN])
@pytest.mark.parametrize("bf16", [False, True])
def test_gradient(capi, E, G, KG, K, flags, bf16):
    T, scale = 33, 2.5
    rng = np.random.default_rng(E + flags)
    x, b = logits(T, E, E + 1, bf16), biases(E, E + 2)
    x[3] = -np.inf             # no expert at all
    x[4, 2:] = -np.inf         # fewer than K
    x[5, ::3] = -np.inf
    ids, _, _ = run(capi, x, b, K, G, KG, flags | SUM2, scale)
    v = x.float().numpy()
    want, _ = dense_ref.grouped_select(v, b, K, G, KG, bool(flags & SIG), True)
    assert np.array_equal(ids, want)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    dx = torch.full((T + 1, E), float("nan"), dtype=x.dtype, device=dev())
    capi.moe_gate_grad(T, E, K, x.to(dev()), torch.from_numpy(ids).to(dev()),
                       torch.from_numpy(dw).to(dev()), dx, flags, scale)
    assert bool(torch.isnan(dx[T].float()).all())
    got = dx[:T].float().cpu().numpy().astype(np.float64)
    sg, rn = bool(flags & SIG), bool(flags & REN)
    g = ref.gate_grad(v, ids, dw, sg, rn, scale)
    # every term of an entry is off by n relative to itself: the bound takes their sizes
    n = steps(v, E) * ref.EPS24
    p = ref.gate_weights(v, ids, sg, rn, 1.0)
    a = np.abs(dw.astype(np.float64) * scale)
    total = (a * p).sum(1, keepdims=True)
    size = np.zeros_like(g)
    t, k = np.nonzero(ids >= 0)
    np.add.at(size, (t, ids[t, k]), (p * (a + total))[t, k])
    if not flags:
        f = np.where(np.isfinite(v), v, -np.inf).astype(np.float64)
        top = f.max(1, keepdims=True)
        e = np.exp(f - np.where(np.isfinite(top), top, 0))
        size += e / np.maximum(e.sum(1, keepdims=True), 1e-300) * total
    tol = 3 * n * size + 1e-37 + (ref.HALF_BF16 * np.abs(g) if bf16 else 0)
    assert np.all(np.abs(got - g) <= tol), np.max(np.abs(got - g) - tol)
