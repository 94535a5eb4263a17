"""The norm's gradient of rows that pass the registers of a workgroup, on the GPU
against 64 bits: several rows to a workgroup, rows that end inside a thread's
vectors, results in place."""
import pytest
import torch

import test_gpu_norm as norm
from dense_ref import HALF_BF16
from gpu_path import dev
from test_gpu_norm import DEPTH, EPS, capi, grads64, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(1, 16384), (1, 16392), (5, 18432), (300, 24584), (600, 18432),
                                 (257, 32768), (261, 65528), (300, 65536)])
@pytest.mark.parametrize("more", [False, True])
def test_gradient(capi, T, H, more):
    norm.test_grad(capi, T, H, more)


@pytest.mark.parametrize("T,H", [(7, 16392), (300, 40008)])
def test_in_place_of_what_reaches_the_sum(capi, T, H):
    x, _, w = inputs(T, H, T)
    g = torch.Generator(device=dev()).manual_seed(2)
    dy, ds = ((torch.randn(T, H, generator=g, device=dev()) * 0.02).to(torch.bfloat16)
              for _ in range(2))
    d, mag, _, _ = grads64(x, w, dy, ds)
    e = ds.clone()
    capi.moe_rms_norm_grad(T, H, x, w, EPS, dy, e, e)
    assert bool(((e.double() - d).abs() <= HALF_BF16 * d.abs() + 4 * DEPTH * mag + 1e-38).all())
    out = torch.empty_like(ds)
    capi.moe_rms_norm_grad(T, H, x, w, EPS, dy, ds, out)
    assert torch.equal(out, e)
