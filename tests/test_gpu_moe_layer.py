"""Router, FP8 dispatch, the experts' products and activation, combine, and the
gradients, run together through the allocating calls as a layer uses them; and
captured into HIP graphs. Each step is held to the 64-bit reference on what the
step before it handed on."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import moe_inputs as mi
from gpu_path import dev, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_moe_layout_03_amd import ep as e

    return e


def weights(rng, E, N, C):
    w = to_dev(ref.random_codes(rng, (E, N, C))).view(torch.float8_e4m3fn)
    s = (np.exp(rng.standard_normal((E, (N + 127) // 128, C // 128)) * 0.3)
         * 4 / 448 / np.sqrt(C)).astype(np.float32)
    return w, to_dev(s)


def host(t):
    return t.detach().cpu()


def scales64(sc):
    s = host(sc).numpy()
    if s.dtype == np.int32:
        b = np.stack([(s.astype(np.int64) >> k) & 255 for k in (0, 8, 16, 24)], -1)
        return np.exp2(b.reshape(s.shape[:-1] + (-1,)) - 127.0)
    return s.astype(np.float64)


def check_product(x, w, rows_of, got):
    q = host(x[0].reshape(-1, x[0].shape[-1]).view(torch.uint8)).numpy()
    s = scales64(x[1]).reshape(q.shape[0], -1)
    wq, ws = host(w[0].view(torch.uint8)).numpy(), host(w[1]).numpy().astype(np.float64)
    N, C = wq.shape[1:]
    g = host(got.float()).numpy().astype(np.float64)
    for e, r in rows_of.items():
        a = ref.e4m3_values(q[r]) * np.repeat(s[r], 128, 1)
        b = ref.e4m3_values(wq[e]) * np.repeat(np.repeat(ws[e], 128, 0)[:N], 128, 1)
        tol = ref.HALF_BF16 * np.abs(a @ b.T) + ref.product_bound(a, b, C // 128)
        off = np.abs(g[r] - a @ b.T) / tol
        assert off.max() <= 1, (e, off.max(), np.unravel_index(off.argmax(), off.shape))


def check_activation(x, h, rows):
    gu = host(x.float()).numpy()[rows]
    _, _, _, want = ref.silu_mul(gu)
    q = host(h[0].view(torch.uint8)).numpy()[rows]
    s = scales64(h[1])[rows]
    v = ref.e4m3_values(q).reshape(len(rows), -1, 128) * s[..., None]
    want = want.reshape(v.shape)
    assert np.all(np.abs(v - want) <= (2.0 ** -4 + 20 * ref.EPS24) * np.abs(want)
                  + (2.0 ** -10 + 450 * 20 * ref.EPS24) * s[..., None])


@pytest.mark.parametrize("mode", ["ll", "ll_words", "ll_rows", "contiguous"])
def test_forward(ep, orc, mode):
    T, H, E, R, K, I, M = 40, 1024, 32, 4, 4, 512, 64
    rng = np.random.default_rng(17)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(dev())
    logits[:, 8:16] = -float("inf")  # rank 1 is out
    x = to_dev(mi.to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))).view(torch.bfloat16)
    w1, w2 = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
    idx, wt = ep.gate(logits, K, score="sigmoid", renormalize=True, scale=2.5)
    assert np.array_equal(host(idx).numpy(), ref.gate_select(host(logits).numpy(), K))
    words = mode == "ll_words"
    if mode == "contiguous":
        _, _, _, _, handle = ep.get_dispatch_layout(idx, E, R, 16, H)
        qz = orc.quantize_fp8(host(x.view(torch.int16)).numpy().view(np.uint16), 0)
        xq = torch.from_numpy(qz["q"]).to(dev()).view(torch.float8_e4m3fn)
        recv = ep.dispatch((xq, to_dev(qz["scale"])), handle)
    else:
        recv, _, handle = ep.low_latency_dispatch(x, idx, M, E, R, 2, use_fp8=True,
                                                  use_ue8m0=words, scale_rows=mode == "ll_rows")
    start, count = host(handle.layout.offset).numpy(), host(handle.layout.count).numpy()
    assert count.sum() == T * K and np.all(count[8:16] == 0)
    rows_of = {e: np.arange(start[e], start[e] + count[e]) for e in range(E) if count[e]}
    live = np.concatenate(list(rows_of.values()))
    y1 = ep.expert_gemm(recv, w1, handle)
    check_product(recv, w1, rows_of, y1)
    h = ep.swiglu_fp8(y1, handle, use_ue8m0=words)
    check_activation(y1, h, live)
    y2 = ep.expert_gemm(h, w2, handle)
    check_product(h, w2, rows_of, y2)
    out = ep.combine(y2, handle, wt)
    slot = host(handle.layout.slot).numpy().reshape(T, K)
    y64 = host(y2.float()).numpy().astype(np.float64)
    terms = host(wt).numpy().astype(np.float64)[..., None] * y64[slot]
    got = host(out.float()).numpy().astype(np.float64)
    assert np.all(np.abs(got - terms.sum(1)) <= ref.HALF_BF16 * np.abs(terms.sum(1))
                  + 2 * K * ref.EPS24 * np.abs(terms).sum(1))
    assert int(handle.layout.status.item()) == 0


def test_backward(ep, orc):
    """Gradients through combine, activation, dispatch and router."""
    T, H, E, R, K, I = 33, 256, 16, 4, 4, 128
    rng = np.random.default_rng(23)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(dev())
    idx, wt = ep.gate(logits, K)
    x = to_dev(mi.to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))).view(torch.bfloat16)
    recv, handle = ep.dispatch_with_layout(x, idx, E, R, 8)
    rows = handle.recv_rows
    y = to_dev(mi.to_bf16_bits(rng.standard_normal((rows, H)).astype(np.float32))).view(
        torch.bfloat16)
    d_out = to_dev(mi.to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))).view(
        torch.bfloat16)
    d_y, d_w = ep.combine_grad(d_out, y, handle, wt)
    slot = host(handle.layout.slot).numpy().reshape(T, K)
    do, yy = host(d_out.float()).numpy(), host(y.float()).numpy()
    w32 = host(wt).numpy()
    want = mi.bf16_bits_to_f32(mi.to_bf16_bits((w32[..., None] * do[:, None, :]).reshape(-1, H)))
    assert np.array_equal(host(d_y.float()).numpy()[slot.reshape(-1)], want)
    t64 = do.astype(np.float64)[:, None, :] * yy.astype(np.float64)[slot]
    assert np.all(np.abs(host(d_w).numpy() - t64.sum(-1)) <= 20 * ref.EPS24 * np.abs(t64).sum(-1))
    gu = to_dev(mi.to_bf16_bits(rng.standard_normal((rows, 2 * I)).astype(np.float32))).view(
        torch.bfloat16)
    d_h = d_y[:, :I].contiguous()
    d_gu = ep.swiglu_grad(gu, d_h, handle)
    r = slot.reshape(-1)
    g, u, s, _ = ref.silu_mul(host(gu.float()).numpy()[r])
    d = host(d_h.float()).numpy()[r].astype(np.float64)
    want = np.concatenate([d * u * s * (1 + g * (1 - s)), d * g * s], 1)
    big = np.concatenate([np.abs(d * u * s) * (1 + np.abs(g)), np.abs(d * g * s)], 1)
    assert np.all(np.abs(host(d_gu.float()).numpy()[r] - want)
                  <= ref.HALF_BF16 * np.abs(want) + 16 * ref.EPS24 * big + 1e-40)
    # the gradient of the dispatch: the plain sum of a token's rows
    d_x = ep.dispatch_grad(d_gu, handle)
    rows64 = host(d_gu.float()).numpy().astype(np.float64)[slot]
    tot = rows64.sum(1)
    assert np.all(np.abs(host(d_x.float()).numpy() - tot) <= ref.HALF_BF16 * np.abs(tot)
                  + K * ref.EPS24 * np.abs(rows64).sum(1))
    d_logits = host(ep.gate_grad(logits, idx, d_w)).numpy()
    xl, ids, dw = host(logits).numpy(), host(idx).numpy(), host(d_w).numpy()
    want = ref.gate_grad(xl, ids, dw, False, False, 1.0)
    size = (np.abs(dw) * ref.gate_weights(xl, ids, False, False, 1.0)).sum(1, keepdims=True)
    assert np.all(np.abs(d_logits - want) <= 200 * ref.EPS24 * (np.abs(want) + size))
    # a masked rank, as the low-latency combine leaves it out
    recv, _, h2 = ep.low_latency_dispatch(x, idx, 64, E, R, 1)
    y2 = recv.reshape(-1, H)
    mask = torch.tensor([0, 1, 0, 0], dtype=torch.int32, device=dev())
    d_y, d_w = ep.combine_grad(d_out, y2, h2, wt, mask)
    dead = (ids // (E // R)) == 1
    sl = host(h2.layout.slot).numpy().reshape(T, K)
    assert np.all(host(d_w).numpy()[dead] == 0) and np.all(host(d_w).numpy()[~dead] != 0)
    assert np.all(host(d_y.float()).numpy()[sl[dead]] == 0)
    with pytest.raises(ValueError, match="topk_idx"):
        ep.combine_grad(d_out, y, handle, wt, mask)


def test_scale_views_are_told_apart(ep):
    rng = np.random.default_rng(2)
    T, H, E, R, K, M = 9, 256, 8, 2, 2, 16
    x = torch.randn(T, H, device=dev()).to(torch.bfloat16)
    idx = torch.from_numpy(mi._uniform_subsets(rng, T, E, K)).to(dev())
    w = weights(rng, E, 64, H)
    got = []
    for rows in (False, True):
        recv, _, h = ep.low_latency_dispatch(x, idx, M, E, R, 0, use_fp8=True, scale_rows=rows)
        assert recv[1].is_contiguous() == rows
        out = ep.expert_gemm(recv, w, h)
        got.append(out[h.layout.slot.long()])
    assert torch.equal(*got)
    _, _, _, _, hc = ep.get_dispatch_layout(idx, E, R, 1, H)
    with pytest.raises(ValueError, match="row-major"):
        q = torch.zeros(T * K, H, dtype=torch.float8_e4m3fn, device=dev())
        ep.expert_gemm((q, torch.ones(H // 128, T * K, device=dev()).t()), w, hc)


def test_empty_batch(ep):
    w = weights(np.random.default_rng(0), 8, 64, 128)
    logits = torch.empty(0, 8, device=dev())
    idx, wt = ep.gate(logits, 2)
    assert idx.shape == (0, 2) and wt.shape == (0, 2)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device=dev())
    recv, _, h = ep.low_latency_dispatch(x, idx, 4, 8, 2, 0, use_fp8=True)
    out = torch.full((h.recv_rows, 64), 3.0, dtype=torch.bfloat16, device=dev())
    ep.expert_gemm(recv, w, h, out)
    assert bool((out == 3).all())
    assert ep.gate_grad(logits, idx, wt).shape == (0, 8)


def test_layer_in_a_graph(ep):
    """Forward and backward captured once and replayed on new inputs, with eager
    work of the same shapes between the replays: every replay equals the eager
    run on those inputs, bit for bit."""
    T, H, E, R, K, I, M = 48, 512, 16, 4, 4, 256, 48
    rng = np.random.default_rng(29)
    w1, w2 = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
    logits = torch.zeros(T, E, device=dev())
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=dev())
    d_out = torch.zeros(T, H, dtype=torch.bfloat16, device=dev())

    def layer():
        idx, wt = ep.gate(logits, K, renormalize=True)
        recv, _, h = ep.low_latency_dispatch(x, idx, M, E, R, 1, use_fp8=True)
        y1 = ep.expert_gemm(recv, w1, h)
        y2 = ep.expert_gemm(ep.swiglu_fp8(y1, h), w2, h)
        out = ep.combine(y2, h, wt)
        d_y, d_w = ep.combine_grad(d_out, y2, h, wt)
        d_gu = ep.swiglu_grad(y1, d_y[:, :I].contiguous(), h)
        # rows as the tokens see them: the rest of the buffers is not written
        s = h.layout.slot.long()
        return idx, wt, y1[s], y2[s], out, d_y[s], d_w, d_gu[s], ep.gate_grad(
            logits, idx, d_w, renormalize=True)

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        logits.copy_(torch.randn(T, E, generator=g, device=dev()))
        x.copy_(torch.randn(T, H, generator=g, device=dev()))
        d_out.copy_(torch.randn(T, H, generator=g, device=dev()))

    stream = torch.cuda.Stream()
    fill(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        held = layer()
    for seed in (1, 2, 3, 1):
        fill(seed)
        want = [t.clone() for t in layer()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(held, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (seed, i)


@pytest.mark.parametrize("words", [False, True])
@pytest.mark.parametrize("T", [6, 90])
def test_a_diverged_row_stays_visible(ep, T, words):
    """One NaN and one infinity behind the first product: the rows they are in
    come out of the second as NaN throughout, all others as without them."""
    H, E, R, K, I, M = 256, 4, 2, 2, 512, 96
    rng = np.random.default_rng(T)
    w2 = weights(rng, E, H, I)
    idx = torch.from_numpy(mi._uniform_subsets(rng, T, E, K)).to(dev())
    x = torch.randn(T, H, device=dev()).to(torch.bfloat16)
    recv, _, h = ep.low_latency_dispatch(x, idx, M, E, R, 1)
    y1 = torch.randn(h.recv_rows, 2 * I, device=dev()).to(torch.bfloat16)
    slot = h.layout.slot.long()
    bad = slot[torch.tensor([3, len(slot) - 2], device=dev())]
    spoilt = y1.clone()
    spoilt[bad[0], 77], spoilt[bad[1], I + 500] = float("nan"), float("inf")
    out = [ep.expert_gemm(ep.swiglu_fp8(v, h, use_ue8m0=words), w2, h) for v in (y1, spoilt)]
    assert bool(out[1][bad].isnan().all())
    rest = slot[~torch.isin(slot, bad)]
    assert torch.equal(out[0][rest], out[1][rest]) and bool(out[0][slot].isfinite().all())


def test_dispatch_gradient_of_another_width(ep):
    """dispatch_grad sums rows of the width it is given, whatever the width the
    handle was made for."""
    T, E, R, K = 19, 8, 2, 3
    rng = np.random.default_rng(3)
    idx = torch.from_numpy(mi._uniform_subsets(rng, T, E, K)).to(dev())
    for made, H in ((8, 256), (64, 128), (512, 64)):
        _, _, _, _, h = ep.get_dispatch_layout(idx, E, R, 4, made)
        rows = to_dev(mi.to_bf16_bits(rng.standard_normal((h.recv_rows, H)).astype(
            np.float32))).view(torch.bfloat16)
        d_x = ep.dispatch_grad(rows, h)
        assert h.shape.H == made  # the handle is as it was
        t = host(rows.float()).numpy().astype(np.float64)[
            host(h.layout.slot).numpy().reshape(T, K)]
        assert np.all(np.abs(host(d_x.float()).numpy() - t.sum(1))
                      <= ref.HALF_BF16 * np.abs(t.sum(1)) + K * ref.EPS24 * np.abs(t).sum(1))


def transposed(w):
    """Weights stored for the product's gradient: rows and columns changed over,
    the scales' blocks with them (N has to be a multiple of 128)."""
    codes, scale = w
    return (codes.view(torch.uint8).transpose(1, 2).contiguous().view(torch.float8_e4m3fn),
            scale.transpose(1, 2).contiguous())


def cast_rows(x, flags=0):
    from combine_moe_layout_03_amd import capi

    rows, width = x.shape
    q = torch.empty(rows, width, dtype=torch.float8_e4m3fn, device=x.device)
    sc = torch.empty(rows, capi.fp8_scale_cols(width, flags), device=x.device,
                     dtype=torch.int32 if flags & capi.MOE_FP8_UE8M0 else torch.float32)
    capi.moe_quantize_fp8(rows, width, x, q, sc, flags)
    return q, sc


def check_cast(x, h, rows):
    """Codes and scales of the live rows against their definition."""
    v = host(x.float()).numpy()[rows].astype(np.float64).reshape(len(rows), -1, 128)
    s = scales64(h[1])[rows]
    got = ref.e4m3_values(host(h[0].view(torch.uint8)).numpy()[rows]).reshape(v.shape)
    assert np.all(np.abs(got * s[..., None] - v) <= 2.0 ** -4 * np.abs(v) * (1 + 2.0 ** -20)
                  + 2.0 ** -10 * s[..., None])


@pytest.mark.parametrize("mode", ["contiguous", "ll", "ll_words"])
def test_backward_of_the_experts(ep, orc, mode):
    """The whole way back, each step on what the one before it hands on: combine's
    gradient, cast, product with the transposed weights, activation's gradient,
    cast, the other transposed product, sum of a token's rows. Held to 64 bits
    step by step, rows of no segment being whatever the buffers held."""
    T, H, E, R, K, I, M = 37, 512, 16, 4, 4, 256, 64
    rng = np.random.default_rng(41)
    flags = 3 if mode == "ll_words" else 0
    if flags:
        I = 512
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(dev())
    x = to_dev(mi.to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))).view(torch.bfloat16)
    d_out = to_dev(mi.to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))).view(
        torch.bfloat16)
    w1, w2 = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
    w1t, w2t = transposed(w1), transposed(w2)
    idx, wt = ep.gate(logits, K, renormalize=True)
    if mode == "contiguous":
        _, _, _, _, handle = ep.get_dispatch_layout(idx, E, R, 16, H)
        recv = ep.dispatch(cast_rows(x), handle)
    else:
        recv, _, handle = ep.low_latency_dispatch(x, idx, M, E, R, 1, use_fp8=True,
                                                  use_ue8m0=bool(flags))
    start, count = host(handle.layout.offset).numpy(), host(handle.layout.count).numpy()
    rows_of = {e: np.arange(start[e], start[e] + count[e]) for e in range(E) if count[e]}
    live = np.concatenate(list(rows_of.values()))
    y1 = ep.expert_gemm(recv, w1, handle)
    y2 = ep.expert_gemm(ep.swiglu_fp8(y1, handle, use_ue8m0=bool(flags)), w2, handle)

    d_y2, d_w = ep.combine_grad(d_out, y2, handle, wt)
    slot = host(handle.layout.slot).numpy().reshape(T, K)
    do, y64 = (host(t.float()).numpy().astype(np.float64) for t in (d_out, y2))
    w64 = host(wt).numpy().astype(np.float64)[..., None]
    got = host(d_y2.float()).numpy().astype(np.float64)[slot]
    want = w64 * do[:, None]
    assert np.all(np.abs(got - want) <= (ref.HALF_BF16 + 2 * ref.EPS24) * np.abs(want))
    prod = do[:, None] * y64[slot]
    assert np.all(np.abs(host(d_w).numpy() - prod.sum(-1))
                  <= (H / 256 + 16) * ref.EPS24 * np.abs(prod).sum(-1))

    q2 = cast_rows(d_y2, flags)
    check_cast(d_y2, q2, live)
    d_h = ep.expert_gemm(q2, w2t, handle)
    check_product(q2, w2t, rows_of, d_h)
    # the same from the weights as they are stored: out = W^T d per expert
    a = ref.e4m3_values(host(q2[0].view(torch.uint8)).numpy()) * np.repeat(
        scales64(q2[1]), 128, 1)
    wq = ref.e4m3_values(host(w2[0].view(torch.uint8)).numpy())
    full = wq * np.repeat(np.repeat(host(w2[1]).numpy().astype(np.float64), 128, 1), 128, 2)
    g = host(d_h.float()).numpy().astype(np.float64)
    for e, r in rows_of.items():
        b = np.ascontiguousarray(full[e].T)
        tol = ref.HALF_BF16 * np.abs(a[r] @ full[e]) + ref.product_bound(a[r], b, H // 128)
        assert np.all(np.abs(g[r] - a[r] @ full[e]) <= tol)

    d_y1 = ep.swiglu_grad(y1, d_h, handle)
    gg, uu, s, _ = ref.silu_mul(host(y1.float()).numpy()[live])
    d = g[live]
    want = np.concatenate([d * uu * s * (1 + gg * (1 - s)), d * gg * s], 1)
    big = np.concatenate([np.abs(d * uu * s) * (1 + np.abs(gg)), np.abs(d * gg * s)], 1)
    assert np.all(np.abs(host(d_y1.float()).numpy()[live] - want)
                  <= ref.HALF_BF16 * np.abs(want) + 16 * ref.EPS24 * big + 1e-40)

    q1 = cast_rows(d_y1, flags)
    check_cast(d_y1, q1, live)
    d_recv = ep.expert_gemm(q1, w1t, handle)
    check_product(q1, w1t, rows_of, d_recv)
    d_x = ep.dispatch_grad(d_recv, handle)
    rows64 = host(d_recv.float()).numpy().astype(np.float64)[slot]
    tot = rows64.sum(1)
    assert np.all(np.abs(host(d_x.float()).numpy() - tot) <= ref.HALF_BF16 * np.abs(tot)
                  + K * ref.EPS24 * np.abs(rows64).sum(1))
    d_logits = host(ep.gate_grad(logits, idx, d_w, renormalize=True)).numpy()
    xl, ids, dw = host(logits).numpy(), host(idx).numpy(), host(d_w).numpy()
    want = ref.gate_grad(xl, ids, dw, False, True, 1.0)
    size = (np.abs(dw) * ref.gate_weights(xl, ids, False, True, 1.0)).sum(1, keepdims=True)
    assert np.all(np.abs(d_logits - want) <= 200 * ref.EPS24 * (np.abs(want) + size))
    assert int(handle.layout.status.item()) == 0


def test_backward_of_the_experts_in_a_graph(ep):
    """Forward and the whole backward captured once: every replay on new inputs,
    with eager runs between, equals the eager run bit for bit."""
    T, H, E, R, K, I, M = 24, 256, 8, 2, 2, 128, 32
    rng = np.random.default_rng(43)
    w1, w2 = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
    w1t, w2t = transposed(w1), transposed(w2)
    logits = torch.zeros(T, E, device=dev())
    x, d_out = (torch.zeros(T, H, dtype=torch.bfloat16, device=dev()) for _ in range(2))

    def step():
        idx, wt = ep.gate(logits, K)
        recv, _, h = ep.low_latency_dispatch(x, idx, M, E, R, 0, use_fp8=True)
        y1 = ep.expert_gemm(recv, w1, h)
        y2 = ep.expert_gemm(ep.swiglu_fp8(y1, h), w2, h)
        d_y2, d_w = ep.combine_grad(d_out, y2, h, wt)
        d_h = ep.expert_gemm(cast_rows(d_y2), w2t, h)
        d_y1 = ep.swiglu_grad(y1, d_h, h)
        d_recv = ep.expert_gemm(cast_rows(d_y1), w1t, h)
        return (ep.combine(y2, h, wt), ep.dispatch_grad(d_recv, h), ep.gate_grad(logits, idx, d_w),
                d_w)

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (logits, x, d_out):
            t.copy_(torch.randn(t.shape, generator=g, device=dev()))

    stream = torch.cuda.Stream()
    fill(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        held = step()
    for seed in (1, 2, 1):
        fill(seed)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(held, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (seed, i)


@pytest.mark.parametrize("T", [5, 70])
def test_row_gradient_of_a_ragged_product(ep, T):
    """A product of 200 columns has no transposed form (200 is no whole number of
    groups); with rows and weights stored 256 wide, zeros behind, it has one."""
    E, R, K, C, N, P = 4, 2, 2, 256, 200, 256
    rng = np.random.default_rng(T)
    w = weights(rng, E, N, C)
    wide = torch.zeros(E, P, C, dtype=torch.uint8, device=dev())
    wide[:, :N] = w[0].view(torch.uint8)
    wt = transposed((wide.view(torch.float8_e4m3fn), w[1]))
    idx = torch.from_numpy(mi._uniform_subsets(rng, T, E, K)).to(dev())
    _, _, _, _, h = ep.get_dispatch_layout(idx, E, R, 1)
    d_out = torch.zeros(h.recv_rows, P, dtype=torch.bfloat16, device=dev())
    d_out[:, :N] = torch.randn(h.recv_rows, N, device=dev())
    q = cast_rows(d_out)
    d_in = ep.expert_gemm(q, wt, h)
    start, count = host(h.layout.offset).numpy(), host(h.layout.count).numpy()
    check_product(q, wt, {e: np.arange(start[e], start[e] + count[e]) for e in range(E)
                          if count[e]}, d_in)
    a = ref.e4m3_values(host(q[0].view(torch.uint8)).numpy()) * np.repeat(scales64(q[1]), 128, 1)
    wq = ref.e4m3_values(host(w[0].view(torch.uint8)).numpy())
    s = np.repeat(np.repeat(host(w[1]).numpy().astype(np.float64), 128, 1)[:, :N], 128, 2)
    got = host(d_in.float()).numpy().astype(np.float64)
    for e in range(E):
        r = slice(start[e], start[e] + count[e])
        if count[e]:
            b = np.ascontiguousarray((wq[e] * s[e]).T)
            want = a[r, :N] @ (wq[e] * s[e])
            pad = np.pad(b, ((0, 0), (0, P - N)))
            assert np.all(np.abs(got[r] - want) <= ref.HALF_BF16 * np.abs(want)
                          + ref.product_bound(a[r], pad, P // 128))
