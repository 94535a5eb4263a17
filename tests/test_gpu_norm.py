"""Residual addition and root-mean-square norm, its FP8 codes and its gradient on
the GPU against 64 bits."""
import numpy as np
import pytest
import torch

from dense_ref import EPS24, HALF_BF16, guard_ok, guarded
from gpu_path import dev

pytestmark = pytest.mark.gpu

EPS = 1e-6
ROUND, WORDS = 1, 2
# The mean of squares: positive terms, at most 8 + 8 vectors + 6 lanes + 16 waves
# additions deep for H up to 65536 (fewer than 64), so relative 64 half steps, of
# which the root halves all but its own; products and root add 6.
DEPTH = 40 * EPS24


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_moe_layout_03_amd import capi as c

    return c


def inputs(T, H, seed, scale=1.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = (torch.randn(T, H, generator=g, device=dev())
         * torch.exp(torch.randn(T, 1, generator=g, device=dev())) * scale).to(torch.bfloat16)
    r = (torch.randn(T, H, generator=g, device=dev()) * scale).to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(H, generator=g, device=dev())).to(torch.bfloat16)
    return x, r, w


def y64(s, w, eps=EPS):
    v = s.double()
    rstd = 1.0 / torch.sqrt(v.square().mean(dim=1, keepdim=True) + eps)
    return v * rstd, v * rstd * w.double(), rstd


SIZES = [(1, 8), (3, 72), (5, 512), (700, 512), (600, 1032), (515, 2048), (2, 2048), (129, 4096),
         (16, 7168), (513, 7168), (3, 16392), (2, 65536)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("res", [False, True])
def test_norm(capi, T, H, res):
    x, r, w = inputs(T, H, T * 31 + H)
    yb, y = guarded(T * H, torch.bfloat16, dev())
    sb, s = guarded(T * H, torch.bfloat16, dev())
    capi.moe_rms_norm(T, H, x, r if res else None, w, EPS, s if res else None, y)
    want = (x.float() + r.float()).to(torch.bfloat16) if res else x
    if res:
        assert torch.equal(s.view(T, H), want)
    _, v, _ = y64(want, w)
    assert bool(((y.view(T, H).double() - v).abs() <= (HALF_BF16 + DEPTH) * v.abs() + 1e-38).all())
    assert guard_ok(yb, T * H) and guard_ok(sb, T * H)


def test_sum_in_place_and_alone(capi):
    x, r, w = inputs(7, 4096, 1)
    want = (x.float() + r.float()).to(torch.bfloat16)
    y = torch.empty_like(x)
    for buf in (0, 1):
        a, b = x.clone(), r.clone()
        capi.moe_rms_norm(7, 4096, a, b, w, EPS, (a, b)[buf], y)
        assert torch.equal((a, b)[buf], want)
        first = y.clone()
    capi.moe_rms_norm(7, 4096, x, r, w, EPS, None, y)  # the sum is not written
    assert torch.equal(y, first)


def codes64(capi, q, sc, flags, T, H):
    v = q.float().double()
    if flags & WORDS:
        b = sc.view(torch.uint8).view(T, H // 128).double()
        return v, torch.exp2(b - 127)
    return v, sc.double()


@pytest.mark.parametrize("T,H", [(1, 512), (3, 1536), (520, 512), (600, 1024), (515, 2048),
                                 (16, 7168), (3, 16384), (1, 65536)])
@pytest.mark.parametrize("flags", [0, ROUND, ROUND | WORDS])
def test_codes(capi, T, H, flags):
    x, r, w = inputs(T, H, T + H + flags)
    x[0, :128] = 0
    r[0, :128] = 0  # a group of zeros: the smallest scale
    q = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=dev())
    cols = capi.fp8_scale_cols(H, flags)
    sb = torch.full((T * cols + 64,), -7, device=dev(),
                    dtype=torch.int32 if flags & WORDS else torch.float32)
    sc = sb[:T * cols].view(T, cols)
    capi.moe_rms_norm(T, H, x, r, w, EPS, None, None, q, sc, flags)
    assert bool((sb[T * cols:] == -7).all())
    _, v, _ = y64((x.float() + r.float()).to(torch.bfloat16), w)
    got, s = codes64(capi, q, sc, flags, T, H)
    g = v.view(T, H // 128, 128)
    want = g.abs().amax(-1).clamp_min(1e-4) / 448
    if flags:
        # the smallest power of two not below it, or the next where rounding carries over one
        up, lo = torch.exp2(torch.ceil(torch.log2(want * (1 + 2 * DEPTH)))), torch.exp2(
            torch.ceil(torch.log2(want * (1 - 2 * DEPTH))))
        assert bool(((s == up) | (s == lo)).all())
    else:
        assert bool(((s - want).abs() <= (DEPTH + 2 * EPS24) * want).all())
    # half a code step of y / s (relative 2^-4; below 2^-6 the step is 2^-9), both off by DEPTH
    t = g / s[..., None]
    off = (got.view_as(g) - t).abs()
    assert bool((off <= 2.0 ** -4 * t.abs().clamp_min(2.0 ** -6) + 4 * DEPTH * t.abs()).all())


def test_both_outputs_agree(capi):
    x, r, w = inputs(130, 2048, 9)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    q, q2 = (torch.empty(130, 2048, dtype=torch.float8_e4m3fn, device=dev()) for _ in range(2))
    s, s2 = (torch.empty(130, 16, device=dev()) for _ in range(2))
    capi.moe_rms_norm(130, 2048, x, r, w, EPS, None, y, q, s)
    capi.moe_rms_norm(130, 2048, x, r, w, EPS, None, y2)
    capi.moe_rms_norm(130, 2048, x, r, w, EPS, None, None, q2, s2)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8))


def test_zero_rows_and_eps(capi):
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device=dev())
    x[1, 3] = 2.0
    w = torch.ones(256, dtype=torch.bfloat16, device=dev())
    y = torch.empty_like(x)
    capi.moe_rms_norm(2, 256, x, None, w, EPS, None, y)
    assert bool((y[0] == 0).all()) and float(y[1, 3]) == 16.0  # 2 / sqrt(4 / 256)
    capi.moe_rms_norm(2, 256, x, None, w, 0.0, None, y)  # 0 * infinity
    assert bool(torch.isnan(y[0]).all()) and float(y[1, 3]) == 16.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite_rows_stay_alone(capi, bad):
    x, _, w = inputs(6, 1024, 3)
    x[2, 700] = bad
    y = torch.empty_like(x)
    q = torch.empty(6, 1024, dtype=torch.float8_e4m3fn, device=dev())
    s = torch.empty(6, 8, device=dev())
    capi.moe_rms_norm(6, 1024, x, None, w, EPS, None, y, q, s)
    keep = torch.tensor([0, 1, 3, 4, 5], device=dev())
    _, v, _ = y64(x[keep], w)
    assert bool(((y[keep].double() - v).abs() <= (HALF_BF16 + DEPTH) * v.abs()).all())
    assert bool(torch.isnan(y[2, 700])) and bool(torch.isnan(s[2, 5]))
    assert bool(torch.isnan(q[2, 640:768].float()).all())
    assert bool(torch.isfinite(s[keep]).all())
    if not np.isnan(bad):  # 1 / sqrt(infinity) = 0: the row's other values are zeros
        assert bool((y[2, :700] == 0).all()) and bool(torch.isfinite(s[2, :5]).all())


def grads64(s, w, dy, ds):
    n, _, rstd = y64(s, w)
    g = dy.double() * w.double()
    d = rstd * (g - n * (g * n).mean(dim=1, keepdim=True))
    mag = rstd * (g.abs() + n.abs() * (g * n).abs().mean(dim=1, keepdim=True))
    if ds is not None:
        d = d + ds.double()
        mag = mag + ds.double().abs()
    return d, mag, (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0)


@pytest.mark.parametrize("T,H", SIZES + [(2100, 512), (1030, 4096)])
@pytest.mark.parametrize("more", [False, True])
def test_grad(capi, T, H, more):
    x, r, w = inputs(T, H, T * 7 + H)
    g = torch.Generator(device=dev()).manual_seed(5)
    dy = (torch.randn(T, H, generator=g, device=dev()) * 0.02).to(torch.bfloat16)
    ds = (torch.randn(T, H, generator=g, device=dev()) * 0.02).to(torch.bfloat16) if more else None
    xb, dx = guarded(T * H, torch.bfloat16, dev())
    wb, dw = guarded(H, torch.float32, dev())
    need = capi.moe_rms_norm_grad_workspace_bytes(T, H)
    assert 0 < need <= capi.MOE_WORKSPACE_MAX_BYTES
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=dev())
    capi.moe_rms_norm_grad(T, H, x, w, EPS, dy, ds, dx, dw, ws[:need])
    d, mag, want, total = grads64(x, w, dy, ds)
    tol = HALF_BF16 * d.abs() + 4 * DEPTH * mag + 1e-38
    assert bool(((dx.view(T, H).double() - d).abs() <= tol).all())
    # rows one after the other, then the workgroups': fewer than T + 64 additions
    tol = (min(T, 600) + 64) * EPS24 * total + DEPTH * total + 1e-38
    assert bool(((dw.double() - want).abs() <= tol).all())
    assert guard_ok(xb, T * H) and guard_ok(wb, H) and bool((ws[need:] == 255).all())
    # without the weight's gradient no workspace; in place of d_y; again the same bits
    e = dy.clone()
    capi.moe_rms_norm_grad(T, H, x, w, EPS, e, ds, e)
    assert torch.equal(e.view(-1), dx)
    dw2 = torch.empty_like(dw)
    capi.moe_rms_norm_grad(T, H, x, w, EPS, dy, ds, dx, dw2, ws)
    assert torch.equal(dw, dw2)


def test_grad_against_differences(capi):
    """The gradient of sum(c * y) against central differences of the formula."""
    T, H = 3, 264
    x, _, w = inputs(T, H, 77)
    g = torch.Generator(device=dev()).manual_seed(6)
    c = torch.randn(T, H, generator=g, device=dev()).to(torch.bfloat16)
    dx, dw = torch.empty_like(x), torch.empty(H, device=dev())
    ws = torch.empty(capi.moe_rms_norm_grad_workspace_bytes(T, H), dtype=torch.uint8, device=dev())
    capi.moe_rms_norm_grad(T, H, x, w, EPS, c, None, dx, dw, ws)

    def f(v, u):
        return (v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * u * c.double()).sum()

    step = 1e-5
    for t, h in ((0, 0), (1, 100), (2, 263)):
        e = torch.zeros(T, H, dtype=torch.float64, device=dev())
        e[t, h] = step * float(x[t].double().norm() / H ** 0.5)
        a = float((f(x.double() + e, w.double()) - f(x.double() - e, w.double())) / (2 * e[t, h]))
        assert abs(float(dx[t, h]) - a) <= HALF_BF16 * abs(a) + 1e-5 * (abs(a) + 1)
        e = torch.zeros(H, dtype=torch.float64, device=dev())
        e[h] = step
        a = float((f(x.double(), w.double() + e) - f(x.double(), w.double() - e)) / (2 * step))
        assert abs(float(dw[h]) - a) <= 1e-5 * (abs(a) + 1)


def test_empty(capi):
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=dev())
    w = torch.ones(256, dtype=torch.bfloat16, device=dev())
    capi.moe_rms_norm(0, 256, e, None, w, EPS, None, e)
    dw = torch.full((256,), 3.0, device=dev())
    capi.moe_rms_norm_grad(0, 256, e, w, EPS, e, None, e, dw)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("T,H", [(1, 4096), (3, 4096), (4, 7168), (5, 7168), (9, 512), (17, 512),
                                 (2, 20480)])
@pytest.mark.parametrize("off", [0, 1])
def test_grad_of_few_rows(capi, T, H, off):
    """One workgroup's sums are the result; also where the result starts at any float."""
    x, _, w = inputs(T, H, T)
    g = torch.Generator(device=dev()).manual_seed(8)
    dy = (torch.randn(T, H, generator=g, device=dev()) * 0.02).to(torch.bfloat16)
    b = torch.full((H + 8,), float("nan"), device=dev())
    dw, dx = b[off:off + H], torch.empty_like(x)
    ws = torch.empty(capi.moe_rms_norm_grad_workspace_bytes(T, H), dtype=torch.uint8, device=dev())
    capi.moe_rms_norm_grad(T, H, x, w, EPS, dy, None, dx, dw, ws)
    _, _, want, total = grads64(x, w, dy, None)
    assert bool(((dw.double() - want).abs() <= (T + 64) * EPS24 * total + DEPTH * total).all())
    assert bool(torch.isnan(b[off + H:]).all()) and bool(torch.isnan(b[:off]).all())


def test_past_32_bits(capi):
    """Rows of more than 4 GiB, with codes and their gradient."""
    T, H = 300001, 8192
    g = torch.Generator(device=dev()).manual_seed(3)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=dev())
    for at in torch.arange(T, device=dev()).split(32768):
        x[at] = torch.randn(len(at), H, generator=g, device=dev()).to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(H, generator=g, device=dev())).to(torch.bfloat16)
    y = torch.full_like(x, float("nan"))
    q = torch.zeros(T, H, dtype=torch.float8_e4m3fn, device=dev())
    s = torch.empty(T, H // 128, device=dev())
    capi.moe_rms_norm(T, H, x, None, w, EPS, None, y, q, s)
    dx, dw = torch.empty_like(x), torch.empty(H, device=dev())
    ws = torch.empty(capi.moe_rms_norm_grad_workspace_bytes(T, H), dtype=torch.uint8, device=dev())
    capi.moe_rms_norm_grad(T, H, x, w, EPS, y, None, dx, dw, ws)
    want, total = 0, 0
    for at in torch.arange(T, device=dev()).split(16384):
        _, v, _ = y64(x[at], w)
        assert bool(((y[at].double() - v).abs() <= (HALF_BF16 + DEPTH) * v.abs()).all())
        t = v.view(len(at), -1, 128) / s[at].double()[..., None]
        off = (q[at].float().double().view_as(t) - t).abs()
        assert bool((off <= 2.0 ** -4 * t.abs().clamp_min(2.0 ** -6) + 4 * DEPTH * t.abs()).all())
        d, mag, a, b = grads64(x[at], w, y[at], None)
        assert bool(((dx[at].double() - d).abs() <= HALF_BF16 * d.abs() + 4 * DEPTH * mag).all())
        want, total = want + a, total + b
    assert bool(((dw.double() - want).abs() <= (600 + 64) * EPS24 * total + DEPTH * total).all())
