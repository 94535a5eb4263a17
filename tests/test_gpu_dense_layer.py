"""Norm, router product, grouped router, FP8 dispatch, experts, combine and shared
expert run together through the allocating calls, forward and back; captured into
HIP graphs, on other streams, and beside each other. Each step is held to 64 bits
on what the step before it handed on."""
import numpy as np
import pytest
import torch

import dense_ref as ref
import experts_ref
from dense_ref import EPS24, HALF_BF16
from gpu_path import dev, to_dev
from test_gpu_moe_layer import check_product, host, weights

pytestmark = pytest.mark.gpu

EPS = 1e-6
T, H, E, R, K, G, KG, I, S = 40, 1024, 32, 4, 4, 8, 3, 512, 264


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_moe_layout_03_amd import ep as e

    return e


def normal(g, *shape, sd=1.0):
    return (torch.randn(*shape, generator=g, device=dev()) * sd).to(torch.bfloat16)


def layer_weights(seed=5):
    g = torch.Generator(device=dev()).manual_seed(seed)
    rng = np.random.default_rng(seed)
    return dict(norm=(1 + 0.2 * torch.randn(H, generator=g, device=dev())).to(torch.bfloat16),
                router=normal(g, E, H, sd=H ** -0.5),
                balance=torch.randn(E, generator=g, device=dev()) * 0.1,
                w1=weights(rng, E, 2 * I, H), w2=weights(rng, E, H, I),
                up=normal(g, 2 * S, H, sd=H ** -0.5), down=normal(g, H, S, sd=S ** -0.5))


def forward(ep, w, x, r):
    """(what the layer adds to, all that was computed on the way)"""
    v = {}
    v["y"], v["sum"], v["fp8"] = ep.rms_norm(x, w["norm"], EPS, r, use_fp8=True)
    v["logits"] = ep.linear(v["y"], w["router"], out_dtype=torch.float32)
    v["idx"], v["wt"] = ep.gate(v["logits"], K, "sigmoid", True, 2.5, bias=w["balance"],
                                num_groups=G, topk_groups=KG, group_score="sum2")
    _, _, _, _, v["handle"] = ep.get_dispatch_layout(v["idx"], E, R, 16, H)
    v["recv"] = ep.dispatch(v["fp8"], v["handle"])
    v["y1"] = ep.expert_gemm(v["recv"], w["w1"], v["handle"])
    v["h"] = ep.swiglu_fp8(v["y1"], v["handle"])
    v["y2"] = ep.expert_gemm(v["h"], w["w2"], v["handle"])
    v["routed"] = ep.combine(v["y2"], v["handle"], v["wt"])
    v["shared"], v["pre"] = ep.linear(v["y"], w["up"], activation="swiglu", save_pre=True)
    v["out"] = ep.linear(v["shared"], w["down"], residual=v["routed"])
    return v


def backward(ep, w, v, d_out):
    """Through shared expert, combine's weights, router and norm (the experts' own way
    back has its tests); d_out also reaches the sum past the layer."""
    d = {}
    d["h"], d["down"], _ = ep.linear_grad(d_out, v["shared"], w["down"])
    d["y_shared"], d["up"], d["up_bias"] = ep.linear_grad(d["h"], v["y"], w["up"], v["pre"],
                                                          "swiglu", with_bias=True)
    _, d["wt"] = ep.combine_grad(d_out, v["y2"], v["handle"], v["wt"])
    d["logits"] = ep.gate_grad(v["logits"], v["idx"], d["wt"], "sigmoid", True, 2.5)
    d["y_router"], d["router"], _ = ep.linear_grad(d["logits"], v["y"], w["router"])
    d["y"] = (d["y_shared"].float() + d["y_router"].float()).to(torch.bfloat16)
    d["x"], d["norm"] = ep.rms_norm_grad(v["sum"], w["norm"], d["y"], EPS, d_out)
    return d


def inputs(seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return normal(g, T, H), normal(g, T, H, sd=2.0), normal(g, T, H, sd=0.02)


def close(got, want, err):
    return bool(((got.double() - want).abs() <= HALF_BF16 * want.abs() + err + 1e-38).all())


def test_forward(ep):
    w = layer_weights()
    x, r, _ = inputs(1)
    v = forward(ep, w, x, r)
    assert torch.equal(v["sum"], (x.float() + r.float()).to(torch.bfloat16))
    s = v["sum"].double()
    y = s / torch.sqrt(s.square().mean(1, keepdim=True) + EPS) * w["norm"].double()
    assert close(v["y"], y, 40 * EPS24 * y.abs())
    z, err = ref.dot_bound(v["y"], w["router"])
    assert bool(((v["logits"].double() - z).abs() <= err).all())
    ids, sc = ref.grouped_select(host(v["logits"]).numpy().astype(np.float64),
                                 host(w["balance"]).numpy(), K, G, KG, True, True)
    assert np.array_equal(host(v["idx"]).numpy(), ids)
    lay = v["handle"].layout
    start, count = host(lay.offset).numpy(), host(lay.count).numpy()
    assert count.sum() == T * K and int(lay.status.item()) == 0
    slot = host(lay.slot).numpy().reshape(T, K)
    for t in range(T):  # the rows that were dispatched are the norm's codes
        assert torch.equal(v["recv"][0].view(torch.uint8)[slot[t, 0]],
                           v["fp8"][0].view(torch.uint8)[t])
    rows_of = {e: np.arange(start[e], start[e] + count[e]) for e in range(E) if count[e]}
    check_product(v["recv"], w["w1"], rows_of, v["y1"])
    check_product(v["h"], w["w2"], rows_of, v["y2"])
    z, err = ref.dot_bound(v["y"], w["up"])
    h, s1, s2 = ref.act64(z, "swiglu", S)
    assert close(v["shared"], h, 2 * s1 * err[:, :S] + 2 * s2 * err[:, S:] + 16 * EPS24 * h.abs()
                 + err.amax() ** 2)
    assert close(v["pre"], z, 1.01 * err)
    z, err = ref.dot_bound(v["shared"], w["down"])
    z = z + v["routed"].double()
    assert close(v["out"], z, 1.01 * err + 2 * EPS24 * z.abs())


def test_backward(ep):
    w = layer_weights()
    x, r, d_out = inputs(2)
    v = forward(ep, w, x, r)
    d = backward(ep, w, v, d_out)
    z, err = ref.dot_bound(d_out, w["down"].t())
    assert close(d["h"], z, 1.01 * err)
    z, err = ref.dot_bound(d_out.t(), v["shared"].t())
    assert bool(((d["down"].double() - z).abs() <= err + 1e-38).all())
    # d_z is rounded to bf16 between: half a step of each term
    dz = ref.act_grad64(v["pre"].double(), d["h"].double(), "swiglu", S)
    mag = dz.abs() * (1 + 2 * v["pre"].double().abs().amax())
    z = dz @ w["up"].double()
    err = 1.2 * HALF_BF16 * (mag @ w["up"].double().abs())
    assert close(d["y_shared"], z, err)
    z, err = dz.t() @ v["y"].double(), 1.2 * HALF_BF16 * (mag.t() @ v["y"].double().abs())
    assert bool(((d["up"].double() - z).abs() <= err + 1e-38).all())
    assert bool(((d["up_bias"].double() - dz.sum(0)).abs() <= 200 * EPS24 * mag.sum(0) + 1e-38).all())
    dl = d["logits"].to(torch.bfloat16)
    z, err = ref.dot_bound(dl, w["router"].t())
    assert close(d["y_router"], z, 1.01 * err)
    z, err = ref.dot_bound(dl.t(), v["y"].t())
    assert bool(((d["router"].double() - z).abs() <= err + 1e-38).all())
    s, g = v["sum"].double(), d["y"].double() * w["norm"].double()
    rstd = 1 / torch.sqrt(s.square().mean(1, keepdim=True) + EPS)
    n = s * rstd
    z = rstd * (g - n * (g * n).mean(1, keepdim=True)) + d_out.double()
    mag = rstd * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True)) + d_out.double().abs()
    assert close(d["x"], z, 160 * EPS24 * mag)
    z, mag = (d["y"].double() * n).sum(0), (d["y"].double() * n).abs().sum(0)
    assert bool(((d["norm"].double() - z).abs() <= 200 * EPS24 * mag + 1e-38).all())


def test_shared_expert_in_fp8(ep):
    """The norm's codes through a product of one expert."""
    w = layer_weights()
    x, r, _ = inputs(3)
    _, _, one = ep.rms_norm(x, w["norm"], EPS, r, use_fp8=True, use_ue8m0=True)
    _, _, _, _, handle = ep.get_dispatch_layout(torch.zeros(T, 1, dtype=torch.int64, device=dev()),
                                                1, 1, 1, H)
    w1 = tuple(t[:1].contiguous() for t in w["w1"])
    y = ep.expert_gemm(one, w1, handle)
    check_product(one, w1, {0: np.arange(T)}, y)


KEEP = ("y", "sum", "logits", "idx", "wt", "routed", "shared", "pre", "out")


def step(ep, w, x, r, d_out):
    v = forward(ep, w, x, r)
    d = backward(ep, w, v, d_out)
    return [v[k] for k in KEEP] + [v["fp8"][0].view(torch.uint8), v["fp8"][1]] + [
        d[k] for k in ("h", "down", "y_shared", "up", "up_bias", "logits", "y_router", "router",
                       "x", "norm")]


def test_in_a_graph(ep):
    """One graph of forward and backward, replayed on new inputs between eager runs."""
    w = layer_weights()
    fixed = [t.clone() for t in inputs(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ep, w, *fixed)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(ep, w, *fixed)
    for seed in (6, 7, 6, 8):
        new = inputs(seed)
        want = [t.clone() for t in step(ep, w, *new)]
        for a, b in zip(fixed, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_graphs_share_nothing(ep):
    """Two captured layers, their replays in turn and beside eager work."""
    w = layer_weights()
    sets = [[t.clone() for t in inputs(s)] for s in (9, 10)]
    want = [[t.clone() for t in step(ep, w, *s)] for s in sets]
    graphs, got = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(step(ep, w, *s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
        eager = step(ep, w, *sets[0])
        torch.cuda.synchronize()
        for a, b in zip(eager, want[0]):
            assert torch.equal(a, b)
        for outs, ref_outs in zip(got, want):
            for a, b in zip(outs, ref_outs):
                assert torch.equal(a, b)


def test_other_streams(ep):
    """Calls go to the current stream, and two of them at once do not disturb each other."""
    w = layer_weights()
    sets = [inputs(s) for s in (11, 12)]
    want = [step(ep, w, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(2):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = step(ep, w, *sets[i])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for p, q in zip(a, b):
                assert torch.equal(p, q)


def test_router_pads_and_rows_are_views(ep):
    """Inputs that are slices of larger tensors, copied where they are not contiguous."""
    w = layer_weights()
    x, r, _ = inputs(13)
    wide = torch.zeros(T, 2 * H, dtype=torch.bfloat16, device=dev())
    wide[:, ::2] = x
    y0 = ep.rms_norm(x, w["norm"], EPS, r)
    y1 = ep.rms_norm(wide[:, ::2], w["norm"], EPS, r)
    assert torch.equal(y0[0], y1[0]) and torch.equal(y0[1], y1[1])
    a = ep.linear(x, w["router"], out_dtype=torch.float32)
    b = ep.linear(wide[:, ::2], w["router"].t().contiguous().t(), out_dtype=torch.float32)
    assert torch.equal(a, b)
