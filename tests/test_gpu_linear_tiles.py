"""Every kernel of the dense product and of its gradients, at ragged sizes, on the GPU
against 64 bits."""
import pytest

from linear_sizes import FORWARD, GRADIENTS, STREAMED
import test_gpu_linear as linear
from test_gpu_linear import capi  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,C,act", FORWARD + STREAMED)
def test_forward(capi, T, N, C, act):
    linear.check(capi, T, N, C, act, True, True, False, act != "none")


@pytest.mark.parametrize("T,N,C,act", [s for s in FORWARD if s[0] > 5000][::2])
def test_forward_float(capi, T, N, C, act):
    linear.check(capi, T, N, C, act, False, False, True, False)


@pytest.mark.parametrize("T,N,C", GRADIENTS)
def test_gradients(capi, T, N, C):
    linear.test_grad(capi, T, N, C)
