"""The operators around the experts on the CPU: the library exports what
moe_experts.h declares, and its host checks and the binding's refuse bad
arguments before a device is touched."""
import ctypes as C
import os
import re
import warnings

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_experts.h")


@pytest.fixture(scope="module")
def lib():
    from combine_moe_layout_03_amd import capi

    return capi


D = C.c_void_p(256)
ODD = C.c_void_p(257)
HALF = C.c_void_p(258)
FOUR = C.c_void_p(260)
NULL, SHAPE, CAPACITY, ALIGN, FLAGS = -1, -2, -3, -5, -10


def test_exports_every_declared_symbol(lib):
    txt = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", txt)))
    assert declared == sorted(lib.EXPORTED_EXPERTS)
    raw = C.CDLL(lib.LIB_PATH)
    for name in declared:
        assert getattr(raw, name) is not None
    values = dict(re.findall(r"#define (MOE_\w+) (\d+)", txt))
    for name, v in values.items():
        assert getattr(lib, name) == int(v)


@pytest.mark.parametrize("T,E,K,flags,scale,code", [
    (-1, 8, 2, 0, 1.0, SHAPE), (4, 0, 1, 0, 1.0, SHAPE), (4, 1025, 1, 0, 1.0, SHAPE),
    (4, 8, 0, 0, 1.0, SHAPE), (4, 8, 9, 0, 1.0, SHAPE), (4, 128, 65, 0, 1.0, SHAPE),
    ((1 << 26) - 63, 8, 2, 0, 1.0, SHAPE), (4, 8, 2, 8, 1.0, FLAGS), (4, 8, 2, -1, 1.0, FLAGS),
    (4, 8, 2, 0, float("nan"), SHAPE), (4, 8, 2, 0, float("inf"), SHAPE)])
def test_gate_shapes(lib, T, E, K, flags, scale, code):
    raw = lib.lib()
    assert raw.moe_gate(T, E, K, D, D, D, flags, scale, None, None) == code
    assert raw.moe_gate_grad(T, E, K, D, D, D, D, flags, scale, None, None) == code


def test_gate_pointers(lib):
    raw = lib.lib()
    assert raw.moe_gate(0, 8, 2, None, None, None, 0, 1.0, None, None) == 0  # empty batch
    assert raw.moe_gate_grad(0, 8, 2, None, None, None, None, 0, 1.0, None, None) == 0
    for bad in range(3):
        args = [D, D, D]
        args[bad] = None
        assert raw.moe_gate(4, 8, 2, *args, 0, 1.0, None, None) == NULL
    for args, flags in (((HALF, D, D), 0), ((ODD, D, D), 1), ((D, FOUR, D), 0),
                        ((D, D, HALF), 0)):
        assert raw.moe_gate(4, 8, 2, *args, flags, 1.0, None, None) == ALIGN
    for bad in range(4):
        args = [D, D, D, D]
        args[bad] = None
        assert raw.moe_gate_grad(4, 8, 2, *args, 0, 1.0, None, None) == NULL
        args[bad] = ODD
        assert raw.moe_gate_grad(4, 8, 2, *args, 0, 1.0, None, None) == ALIGN


def test_combine_grad_checks(lib):
    raw = lib.lib()

    def call(s, do=D, y=D, rows=8, slot=D, w=D, dy=D, dw=D, idx=None, mask=None):
        return raw.moe_combine_grad(C.byref(s) if s else None, do, y, rows, slot, w, dy, dw, idx,
                                    mask, None, None)

    ok = lib.make_shape(4, 16, 16, 4, 2)
    assert call(None) == NULL
    for bad in ((-1, 16, 16, 4, 2), (4, 12, 16, 4, 2), (4, 0, 16, 4, 2), (4, 16, 16, 3, 2),
                (4, 16, 1025, 1, 2), (4, 16, 16, 4, 0), (4, 16, 16, 4, 65), (1 << 23, 16, 16, 4, 2)):
        assert call(lib.make_shape(*bad)) == SHAPE
    assert call(ok, rows=-1) == CAPACITY
    for kw in (dict(do=None), dict(slot=None), dict(dy=None), dict(y=None), dict(idx=D),
               dict(mask=D)):
        assert call(ok, **kw) == NULL
    for kw in (dict(do=FOUR), dict(y=FOUR), dict(dy=FOUR), dict(slot=HALF), dict(w=HALF),
               dict(dw=HALF), dict(idx=FOUR, mask=D)):
        assert call(ok, **kw) == ALIGN
    assert call(lib.make_shape(0, 16, 16, 4, 2), do=None, y=None, slot=None, dy=None) == 0


def test_grouped_gemm_checks(lib):
    raw = lib.lib()

    def call(E=4, N=64, Cc=256, a=D, s=D, rows=8, start=D, count=D, w=D, ws=D, out=D, flags=4,
             most=0):
        return raw.moe_grouped_gemm_fp8(E, N, Cc, a, s, rows, start, count, w, ws, out, flags,
                                        most, None, None)

    for kw in (dict(E=0), dict(E=1025), dict(N=0), dict(N=12), dict(N=(1 << 20) + 8), dict(Cc=0),
               dict(Cc=64), dict(Cc=200), dict(Cc=(1 << 20) + 128), dict(rows=-1),
               dict(rows=1 << 31), dict(most=-1), dict(flags=7, Cc=256),
               dict(flags=0, rows=10)):  # column-major scales: rows % E
        assert call(**kw) == SHAPE, kw
    for f in (2, 6, 8, -1, 16):
        assert call(flags=f, Cc=512) == FLAGS
    for kw in ("a", "s", "start", "count", "w", "ws", "out"):
        assert call(**{kw: None}) == NULL
    for kw in ("a", "w", "out"):
        assert call(**{kw: FOUR}) == ALIGN
    for kw in ("s", "ws", "start", "count"):
        assert call(**{kw: HALF}) == ALIGN
    assert call(rows=0, a=None, s=None, w=None, ws=None, out=None) == 0


def test_swiglu_checks(lib):
    raw = lib.lib()

    def fp8(E=4, I=256, rows=8, x=D, start=D, count=D, q=D, s=D, flags=0):
        return raw.moe_swiglu_fp8(E, I, rows, x, start, count, q, s, flags, None, None)

    def grad(E=4, I=256, rows=8, x=D, dh=D, start=D, count=D, dx=D):
        return raw.moe_swiglu_grad(E, I, rows, x, dh, start, count, dx, None, None)

    for kw in (dict(E=0), dict(E=1025), dict(I=0), dict(I=8), dict(I=192), dict(I=1 << 21),
               dict(rows=-1), dict(rows=1 << 31), dict(flags=3, I=256)):
        assert fp8(**kw) == SHAPE, kw
    for f in (2, 8, -1):
        assert fp8(I=512, flags=f) == FLAGS
    for kw in ("x", "start", "count", "q", "s"):
        assert fp8(**{kw: None}) == NULL
    for kw in ("x", "q"):
        assert fp8(**{kw: FOUR}) == ALIGN
    for kw in ("start", "count", "s"):
        assert fp8(**{kw: HALF}) == ALIGN
    for kw in (dict(E=0), dict(I=4), dict(I=12), dict(I=1 << 21), dict(rows=-1)):
        assert grad(**kw) == SHAPE
    for kw in ("x", "dh", "start", "count", "dx"):
        assert grad(**{kw: None}) == NULL
    for kw in ("x", "dh", "dx"):
        assert grad(**{kw: FOUR}) == ALIGN
    assert fp8(rows=0, x=None, q=None, s=None) == 0
    assert grad(rows=0, x=None, dh=None, dx=None) == 0


def test_binding_refusals(lib):
    """CPU tensors, wrong types and sizes raise before the library is called."""
    x = torch.zeros(4, 8)
    idx, w = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        lib.moe_gate(4, 8, 2, x, idx, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        lib.moe_swiglu_fp8(1, 128, 1, torch.zeros(1, 256, dtype=torch.bfloat16),
                           torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                           torch.zeros(1, 128, dtype=torch.uint8), torch.zeros(1, 1))
    with pytest.raises(ValueError, match="is required"):
        lib.moe_gate(4, 8, 2, None, idx, w)
    with pytest.raises(TypeError, match="MOE_GATE_BF16"):
        lib._logits(x, lib.MOE_GATE_BF16)
    from combine_moe_layout_03_amd import ep

    with pytest.raises(ValueError, match="score"):
        ep.gate(x, 2, score="tanh")


def test_wrapper_refusals(lib):
    """Shapes that do not belong together, which the element counts alone would
    let through: fewer experts, narrower rows, fewer tokens, transposed scales."""
    from combine_moe_layout_03_amd import ep

    shape = lib.make_shape(6, 256, 8, 2, 2, 1)
    h = ep.Handle(shape, lib.LayoutBuffers.empty(shape, "cpu"), 12)
    q, sc = torch.zeros(12, 256, dtype=torch.float8_e4m3fn), torch.ones(12, 2)

    def gemm(E=8, C=256, blocks=(3, 2)):
        return ep.expert_gemm((q, sc), (torch.zeros(E, 384, C, dtype=torch.float8_e4m3fn),
                                        torch.ones(E, *blocks)), h)

    with pytest.raises(ValueError, match="GPU tensor"):  # as it should be, but for the device
        gemm()
    with pytest.raises(ValueError, match="for 8 experts"):
        gemm(E=4)
    with pytest.raises(ValueError, match="rows of 256"):
        gemm(C=128, blocks=(3, 1))
    with pytest.raises(ValueError, match="scales"):
        gemm(blocks=(2, 3))
    x = torch.zeros(12, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not gates and ups"):
        ep.swiglu_fp8(x[:, :255], h)
    with pytest.raises(ValueError, match="rows of 64"):
        ep.swiglu_grad(x, x[:, :64], h)
    with pytest.raises(ValueError, match="for 6 tokens"):
        ep.combine_grad(x[:4], x, h)
    with pytest.raises(ValueError, match="expert rows of 128"):
        ep.combine_grad(x[:6], x[:, :128], h)
    with pytest.raises(ValueError, match="for 6 tokens"):
        ep.gate_grad(torch.zeros(6, 8), torch.zeros(6, 2, dtype=torch.int64), torch.zeros(6, 3))


def test_scales_have_to_match_the_rows(lib):
    """Row scales of another width or layout than the codes', which hold enough
    elements: refused, not read as something else."""
    from combine_moe_layout_03_amd import ep

    shape = lib.make_shape(6, 256, 4, 2, 2, 1)
    lay = lib.LayoutBuffers.empty(shape, "cpu")
    h = ep.Handle(shape, lay, 4 * 8, ll_M=4)  # stripes of 8 rows for each of 4 experts
    q = torch.zeros(32, 256, dtype=torch.float8_e4m3fn)
    w = (torch.zeros(4, 128, 256, dtype=torch.float8_e4m3fn), torch.ones(4, 1, 2))

    def gemm(sc):
        return ep.expert_gemm((q, sc), w, h)

    columns = torch.ones(4, 2, 8)  # as the dispatch stores them
    for good in (torch.ones(32, 2), torch.ones(2, 2, 8, 2), columns.transpose(1, 2),
                 columns.view(2, 2, 2, 8).transpose(2, 3)):
        with pytest.raises(ValueError, match="GPU tensor"):
            gemm(good)
    for bad in (torch.ones(32, 4),                          # of rows twice as wide
                columns,                                    # column-major, but not the view
                torch.ones(32, 1),
                torch.ones(4, 2, 16).transpose(1, 2)):      # stripes of another length
        with pytest.raises(ValueError, match="scales"):
            gemm(bad)


def test_weights_that_would_be_copied_are_reported(lib):
    """Weights that are not contiguous still run, but the copy of all of them
    that each call makes is not silent; nor is a transposed product whose width
    is no whole number of groups of 128 accepted."""
    from combine_moe_layout_03_amd import ep

    shape = lib.make_shape(6, 256, 4, 2, 2, 1)
    h = ep.Handle(shape, lib.LayoutBuffers.empty(shape, "cpu"), 12)
    q, sc = torch.zeros(12, 256, dtype=torch.float8_e4m3fn), torch.ones(12, 2)
    w = torch.zeros(4, 256, 128, dtype=torch.float8_e4m3fn)
    with pytest.warns(UserWarning, match="contiguous"):
        with pytest.raises(ValueError, match="GPU tensor"):
            ep.expert_gemm((q, sc), (w.transpose(1, 2), torch.ones(4, 1, 2)), h)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="GPU tensor"):
            ep.expert_gemm((q, sc), (w.transpose(1, 2).contiguous(), torch.ones(4, 1, 2)), h)
    raw = lib.lib()  # N = 200 forwards, so C = 200 back
    assert raw.moe_grouped_gemm_fp8(4, 200, 256, D, D, 0, D, D, D, D, D, 4, 0, None, None) == 0
    assert raw.moe_grouped_gemm_fp8(4, 256, 200, D, D, 0, D, D, D, D, D, 4, 0, None, None) == SHAPE
