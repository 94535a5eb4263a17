"""Which kernels of the dense product the GPU tests' sizes select, by the library's own
rules compiled for the CPU: every variant has to be among them."""
import ctypes as C
import itertools
import os
import subprocess

import pytest

from linear_sizes import FORWARD, GRADIENTS, STREAMED

ACTS = ("none", "silu", "gelu", "swiglu")
WORKSPACE = 64 << 20

SHIM = r"""
#include "linear_plan.hpp"
extern "C" void plan_of(int64_t rows, int64_t cols, int64_t k, int pairs, int64_t ws, int *out) {
  const moe::Plan p = moe::plan(rows, cols, k, pairs, ws);
  out[0] = p.high, out[1] = p.wide, out[2] = p.splits, out[3] = p.steps;
}
extern "C" int stream_of(int64_t rows, int64_t N, int64_t k, int pairs) {
  return moe::streamed(rows, N, k, pairs) ? moe::stream_weight_rows(rows, N, pairs) : 0;
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    from combine_moe_layout_03_amd import build

    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(build.CSRC, "experts"), "-o", str(d / "plan.so"),
                    str(d / "plan.cpp")], check=True)
    lib = C.CDLL(str(d / "plan.so"))
    i64 = C.c_int64
    lib.plan_of.argtypes = [i64, i64, i64, C.c_int, i64, C.POINTER(C.c_int)]
    lib.plan_of.restype = None
    lib.stream_of.argtypes = [i64, i64, i64, C.c_int]
    return lib


def plan_of(rules, rows, cols, k, pairs=False):
    out = (C.c_int * 4)()
    rules.plan_of(rows, cols, k, pairs, WORKSPACE, out)
    return tuple(out)


def forward(rules, T, N, Cc, act):
    """("stream", weight rows) or ("tiles", high, wide, whether parts are joined)"""
    pairs = act == "swiglu"
    w = rules.stream_of(T, N, Cc, pairs)
    if w:
        return "stream", w
    high, wide, splits, _ = plan_of(rules, T, N * (2 if pairs else 1), Cc, pairs)
    return "tiles", high, wide, splits > 1


def gradients(rules, T, N, Cc):
    """(high, wide, joined) of the rows' and of the weights' gradient"""
    x, w = plan_of(rules, T, Cc, N), plan_of(rules, N, Cc, T)
    return (*x[:2], x[2] > 1), (*w[:2], w[2] > 1)


TILES = [(4, 4), (8, 6), (8, 7), (8, 8)]


def test_every_forward_kernel_is_run(rules):
    got = {(act, forward(rules, T, N, Cc, act)) for T, N, Cc, act in FORWARD + STREAMED}
    for act in ACTS:
        for high, wide in TILES:
            if (act, wide) != ("swiglu", 7):  # (pairs of 16 columns: even widths)
                assert (act, ("tiles", high, wide, False)) in got, (act, high, wide)
        assert (act, ("tiles", 4, 4, True)) in got, act
        for w in (8, 16):
            assert (act, ("stream", w)) in got, (act, w)


def test_every_gradient_kernel_is_run(rules):
    got = [gradients(rules, *s) for s in GRADIENTS]
    for side, (high, wide) in itertools.product((0, 1), TILES):
        assert (high, wide, False) in {g[side] for g in got}, (side, high, wide)
    for side in (0, 1):
        assert (4, 4, True) in {g[side] for g in got}, side


def test_large_tiles_have_ragged_edges_and_a_steady_state(rules):
    """Rows, columns and channels that end inside a tile or stage, and enough stages that
    both of a tile's buffers are filled again and again."""
    for T, N, Cc, act in FORWARD:
        kind = forward(rules, T, N, Cc, act)
        if kind[:2] == ("tiles", 8):
            cols = N * (2 if act == "swiglu" else 1)
            assert T % 256 and cols % (32 * kind[2]) and Cc % 64 and Cc >= 8 * 64
    for T, N, Cc in GRADIENTS:
        x, w = gradients(rules, T, N, Cc)
        if x[0] == 8:
            assert T % 256 and Cc % (32 * x[1]) and N % 64 and N >= 8 * 64
        if w[0] == 8:
            assert N % 256 and Cc % (32 * w[1]) and T % 64 and T >= 8 * 64
