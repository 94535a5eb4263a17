"""The operators before and beside the experts of a mixture-of-experts layer, as cases to measure.

Each is reached through the library's C-ABI binding (``own``) or computed by
elementary torch operations in 32 bits (the plain form):

* ``norm``      residual addition and root-mean-square norm, bf16 rows and FP8 codes with a
                scale per 128 channels, and the gradient with respect to rows and weight;
* ``gate``      router with a balance bias and groups: the best groups, the K best experts
                in them by score + bias, weights from the scores alone;
* ``linear``    x w^T + bias through an activation, plus a residual: router logits in float,
                shared expert;
* ``act_grad``  gradient of that epilogue: d_z and the bias's gradient;
* ``lin_grad``  the product's gradients with respect to rows and weights.
"""
from __future__ import annotations

import math

import torch

own = False

FP8_MAX = 448.0
EPS = 1e-6
GATE_SIGMOID, GATE_RENORM, GATE_GROUP_SUM2 = 2, 4, 8      # router flags of the library
ACTS = ("none", "silu", "gelu", "swiglu")                 # the library's activations 0 ... 3
LINEAR_F32 = 4
WORKSPACE = 64 << 20                                      # no call here needs more
MAX_FLOPS = 9.7e11                                        # the largest listed products
MAX_BYTES = 9.0e8


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step of a small batch: residual, norm, rows for the router and codes to dispatch
        dict(name="norm_16x7168_fp8", op="norm", T=16, H=7168, res=True, fp8=True, grad=False),
        # the skewed batch, forward and backward, with the codes
        dict(name="norm_4096x4096_fp8_train", op="norm", T=4096, H=4096, res=True, fp8=True,
             grad=True),
        # a training batch, forward and backward
        dict(name="norm_8192x7168_train", op="norm", T=8192, H=7168, res=True, fp8=False,
             grad=True),
        # a decoding step: sigmoid scores, a bias, 4 of 8 groups by the sum of their best two
        dict(name="gate_16x256_groups", op="gate", T=16, E=256, K=8, G=8, KG=4, dtype="bf16",
             sigmoid=True, renorm=True, sum2=True, bias=True, scale=2.5),
        # a training batch's router
        dict(name="gate_8192x256_groups", op="gate", T=8192, E=256, K=8, G=8, KG=4, dtype="f32",
             sigmoid=True, renorm=True, sum2=True, bias=True, scale=2.5),
        # router logits of the standard batch, in float
        dict(name="linear_router_128x256", op="linear", T=128, N=256, C=7168, act="none",
             bias=False, res=False, f32=True, pre=False),
        # the shared expert's gates and ups of a decoding step: the weights' bytes
        dict(name="linear_16x2048_swiglu", op="linear", T=16, N=2048, C=7168, act="swiglu",
             bias=False, res=False, f32=False, pre=False),
        # the shared expert's way down of a training batch, added to the combined rows
        dict(name="linear_8192x7168_res", op="linear", T=8192, N=7168, C=2048, act="none",
             bias=True, res=True, f32=False, pre=False),
        # gradient of an epilogue, odd batch and ragged width
        dict(name="act_grad_1001x2824_gelu", op="act_grad", T=1001, N=2824, act="gelu"),
        # gradient of the shared expert's activation, a training batch
        dict(name="act_grad_8192x2048_swiglu", op="act_grad", T=8192, N=2048, act="swiglu"),
        # both gradients of a product, odd batch and ragged width
        dict(name="lin_grad_1001x2824x4096", op="lin_grad", T=1001, N=2824, C=4096),
        # both gradients of the shared expert's first product, a training batch
        dict(name="lin_grad_8192x4096x7168", op="lin_grad", T=8192, N=4096, C=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gate", "linear", "linear", "act_grad", "lin_grad"])
    while True:
        c = dict(op=op, T=_log(rng, 1, 8192))
        if op == "norm":
            c["fp8"] = rng.random() < 0.5
            c["H"] = 128 * _log(rng, 2, 56) if c["fp8"] else 8 * _log(rng, 32, 896)
            c["res"] = rng.random() < 0.7
            c["grad"] = rng.random() < 0.5
        elif op == "gate":
            c["E"], c["G"] = rng.choice([(64, 1), (64, 8), (128, 8), (160, 8), (256, 1), (256, 8),
                                         (256, 16)])
            c["KG"] = 1 if c["G"] == 1 else rng.choice([2, 3, 4])
            c["K"] = rng.choice([1, 2, 4, 6, 8])
            c["dtype"] = rng.choice(["f32", "bf16"])
            c["sigmoid"], c["renorm"] = rng.random() < 0.6, rng.random() < 0.5
            c["sum2"], c["bias"] = rng.random() < 0.5, rng.random() < 0.7
            c["scale"] = rng.choice([1.0, 2.5])
        elif op == "linear":
            c["N"], c["C"] = 8 * _log(rng, 8, 896), 8 * _log(rng, 32, 896)
            c["act"] = rng.choice(ACTS)
            c["bias"], c["res"] = rng.random() < 0.5, rng.random() < 0.3
            c["f32"] = rng.random() < 0.2
            c["pre"] = c["act"] != "none" and rng.random() < 0.5
        else:
            c["N"] = 8 * _log(rng, 8, 896)
            if op == "act_grad":
                c["act"] = rng.choice(ACTS[1:])
            else:
                c["C"] = 8 * _log(rng, 32, 896)
        w = work(c)
        if w["flops"] <= MAX_FLOPS and w["bytes"] <= MAX_BYTES:
            return c


def work(case):
    c, T = case, case["T"]
    if c["op"] == "norm":
        H = c["H"]
        b = T * H * 2 * (4 if c["res"] else 2) + 2 * H + (T * H + T * H // 32 if c["fp8"] else 0)
        f = 6 * T * H
        if c["grad"]:
            b += T * H * 2 * 4 + 4 * H
            f += 10 * T * H
        return {"bytes": b, "flops": f}
    if c["op"] == "gate":
        E = c["E"]
        b = T * E * (4 if c["dtype"] == "f32" else 2) + T * c["K"] * 12 + (4 * E if c["bias"] else 0)
        return {"bytes": b, "flops": 6 * T * E}
    N = c["N"] * (2 if c.get("act") == "swiglu" else 1)
    if c["op"] == "act_grad":
        return {"bytes": 2 * T * (c["N"] + 2 * N) + 4 * N, "flops": 10 * T * N}
    C = c["C"]
    if c["op"] == "linear":
        b = 2 * T * C + 2 * N * C + T * c["N"] * ((4 if c["f32"] else 2) + (2 if c["res"] else 0))
        b += 4 * N * c["bias"] + 2 * T * N * c["pre"]
        return {"bytes": b, "flops": 2 * T * N * C}
    return {"bytes": 2 * (2 * T * C + T * N + N * C) + 4 * N * C, "flops": 4 * T * N * C}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    c, T = case, case["T"]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = dict(c=c)
    if c["op"] == "gate":
        x = normal(T, c["E"]) * 1.5
        s["x"] = x if c["dtype"] == "f32" else x.to(torch.bfloat16)
        s["bias"] = normal(c["E"]) * 0.1 if c["bias"] else None
        s["idx"], s["w"] = empty(T, c["K"], dtype=torch.int64), empty(T, c["K"], dtype=torch.float32)
        return s
    s["ws"] = empty(WORKSPACE, dtype=torch.uint8)
    if c["op"] == "norm":
        H = c["H"]
        # rows of a residual stream: some are much larger than others
        x = normal(T, H) * torch.exp(normal(T, 1))
        s["x"] = x.to(torch.bfloat16)
        s["res"] = (normal(T, H) * 2).to(torch.bfloat16) if c["res"] else None
        s["weight"] = (1 + 0.3 * normal(H)).to(torch.bfloat16)
        s["sum"], s["y"] = empty(T, H) if c["res"] else None, empty(T, H)
        if c["fp8"]:
            s["q"] = empty(T, H, dtype=torch.float8_e4m3fn)
            s["qs"] = empty(T, H // 128, dtype=torch.float32)
        if c["grad"]:
            s["dy"] = (normal(T, H) * 0.02).to(torch.bfloat16)
            s["dsum"] = (normal(T, H) * 0.02).to(torch.bfloat16)
            s["dx"], s["dweight"] = empty(T, H), empty(H, dtype=torch.float32)
        return s
    N = c["N"] * (2 if c.get("act") == "swiglu" else 1)      # rows of the weights
    if c["op"] == "act_grad":
        s["z"] = (normal(T, N) * 1.5).to(torch.bfloat16)
        s["do"] = (normal(T, c["N"]) * 0.02).to(torch.bfloat16)
        s["dz"], s["dbias"] = empty(T, N), empty(N, dtype=torch.float32)
        return s
    C = c["C"]
    s["x"] = normal(T, C).to(torch.bfloat16)
    s["w"] = (normal(N, C) / math.sqrt(C)).to(torch.bfloat16)
    if c["op"] == "linear":
        s["bias"] = normal(N) * 0.3 if c["bias"] else None
        s["res"] = normal(T, c["N"]).to(torch.bfloat16) if c["res"] else None
        s["out"] = empty(T, c["N"], dtype=torch.float32 if c["f32"] else torch.bfloat16)
        s["pre"] = empty(T, N) if c["pre"] else None
        return s
    s["dz"] = (normal(T, N) * 0.02).to(torch.bfloat16)
    s["dx"], s["dw"] = empty(T, C), empty(N, C, dtype=torch.float32)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "gate": _plain_gate, "linear": _plain_linear,
            "act_grad": _plain_act_grad, "lin_grad": _plain_lin_grad}[state["c"]["op"]](state)


def _run_own(s):
    from combine_moe_layout_03_amd import capi

    c, T = s["c"], s["c"]["T"]
    if c["op"] == "norm":
        H = c["H"]
        capi.moe_rms_norm(T, H, s["x"], s["res"], s["weight"], EPS, s["sum"], s["y"],
                          s.get("q"), s.get("qs"))
        got = {"y": s["y"]}
        if c["res"]:
            got["sum"] = s["sum"]
        if c["fp8"]:
            got["q"], got["scale"] = s["q"], s["qs"]
        if c["grad"]:
            capi.moe_rms_norm_grad(T, H, s["sum"] if c["res"] else s["x"], s["weight"], EPS,
                                   s["dy"], s["dsum"], s["dx"], s["dweight"], s["ws"])
            got["d_x"], got["d_weight"] = s["dx"], s["dweight"]
        return got
    if c["op"] == "gate":
        flags = ((GATE_SIGMOID if c["sigmoid"] else 0) | (GATE_RENORM if c["renorm"] else 0)
                 | (GATE_GROUP_SUM2 if c["sum2"] else 0))
        capi.moe_gate_grouped(T, c["E"], c["K"], c["G"], c["KG"], s["x"], s["bias"], s["idx"],
                              s["w"], flags, c["scale"])
        return {"idx": s["idx"], "weights": s["w"]}
    if c["op"] == "linear":
        flags = ACTS.index(c["act"]) | (LINEAR_F32 if c["f32"] else 0)
        capi.moe_linear(T, c["N"], c["C"], s["x"], s["w"], s["bias"], s["res"], s["out"],
                        s["pre"], flags, s["ws"])
        got = {"out": s["out"]}
        if c["pre"]:
            got["z"] = s["pre"]
        return got
    if c["op"] == "act_grad":
        capi.moe_linear_act_grad(T, c["N"], s["do"], s["z"], s["dz"], s["dbias"],
                                 ACTS.index(c["act"]), s["ws"])
        return {"d_z": s["dz"], "d_bias": s["dbias"]}
    capi.moe_linear_grad(T, c["N"], c["C"], s["dz"], s["x"], s["w"], s["dx"], s["dw"], s["ws"])
    return {"d_x": s["dx"], "d_w": s["dw"]}


def _plain_norm(s):
    c = s["c"]
    x = s["x"]
    if c["res"]:
        x = (x.float() + s["res"].float()).to(torch.bfloat16)
    v = x.float()
    rstd = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    n, w = v * rstd, s["weight"].float()
    y = n * w
    got = {"y": y.to(torch.bfloat16)}
    if c["res"]:
        got["sum"] = x
    if c["fp8"]:
        h = y.view(c["T"], -1, 128)
        got["scale"] = h.abs().amax(-1).clamp_min(1e-4) / FP8_MAX
        q = (h / got["scale"][..., None]).clamp(-FP8_MAX, FP8_MAX)
        got["q"] = q.view(c["T"], -1).to(torch.float8_e4m3fn)
    if c["grad"]:
        dy = s["dy"].float()
        g = dy * w
        d = rstd * (g - n * (g * n).mean(dim=1, keepdim=True)) + s["dsum"].float()
        got["d_x"] = d.to(torch.bfloat16)
        got["d_weight"] = (dy * n).sum(dim=0)
    return got


def _plain_gate(s):
    """In 64 bits: scores next to each other have to be told apart."""
    c = s["c"]
    T, E, K, G = c["T"], c["E"], c["K"], c["G"]
    x = s["x"].double()
    if c["sigmoid"]:
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
    choice = p if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        best = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values
        score = best[..., 0] + best[..., 1] if c["sum2"] else best[..., 0]
        order = torch.sort(score, dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, order[:, :c["KG"]], True)
        choice = torch.where(keep.repeat_interleave(E // G, dim=1), choice, -math.inf)
    idx = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :K]
    w = torch.gather(p, 1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"idx": idx, "weights": (w * c["scale"]).float()}


def _plain_linear(s):
    c = s["c"]
    z = torch.mm(s["x"].float(), s["w"].float().t())
    if c["bias"]:
        z = z + s["bias"]
    if c["act"] == "silu":
        h = z / (1.0 + torch.exp(-z))
    elif c["act"] == "gelu":
        h = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    elif c["act"] == "swiglu":
        a, u = z[:, :c["N"]], z[:, c["N"]:]
        h = a / (1.0 + torch.exp(-a)) * u
    else:
        h = z
    if c["res"]:
        h = h + s["res"].float()
    got = {"out": h if c["f32"] else h.to(torch.bfloat16)}
    if c["pre"]:
        got["z"] = z.to(torch.bfloat16)
    return got


def _plain_act_grad(s):
    c = s["c"]
    z, d = s["z"].float(), s["do"].float()
    if c["act"] == "gelu":
        slope = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        slope = slope + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        dz = d * slope
    else:
        a = z[:, :c["N"]]
        sg = 1.0 / (1.0 + torch.exp(-a))
        dz = d * (sg * (1.0 + a * (1.0 - sg)))
        if c["act"] == "swiglu":
            dz = torch.cat([dz * z[:, c["N"]:], d * a * sg], dim=1)
    return {"d_z": dz.to(torch.bfloat16), "d_bias": dz.sum(dim=0)}


def _plain_lin_grad(s):
    dz = s["dz"].float()
    return {"d_x": torch.mm(dz, s["w"].float()).to(torch.bfloat16),
            "d_w": torch.mm(dz.t().contiguous(), s["x"].float())}


# ---------------------------------------------------------------- 64 bits

def _e4m3(v):
    """Doubles -> the nearest E4M3 value (ties to even), saturating at 448."""
    m = v.abs().clamp(max=FP8_MAX)
    e = torch.floor(torch.log2(m.clamp_min(2.0 ** -20)))
    e = torch.where(torch.exp2(e) > m, e - 1, e)
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.copysign(torch.round(m / step) * step, v)


def _exact_norm(c, s):
    x = s["x"].double()
    if c["res"]:
        x = (x + s["res"].double()).float().to(torch.bfloat16).double()   # the sum as it is stored
    H = c["H"]
    got = {k: [] for k in ["y"] + ["sum"] * c["res"] + ["q", "scale"] * c["fp8"]
           + ["d_x"] * c["grad"]}
    dweight = torch.zeros(H, dtype=torch.float64, device="cuda")
    w = s["weight"].double()
    for at in torch.arange(c["T"], device="cuda").split(2048):
        v = x[at]
        length = torch.sqrt(v.square().sum(dim=1, keepdim=True) / H + EPS)
        n = v / length
        y = n * w
        got["y"].append(y)
        if c["res"]:
            got["sum"].append(v)
        if c["fp8"]:
            sc = y.view(len(at), -1, 128).abs().amax(-1).clamp_min(1e-4) / FP8_MAX
            got["scale"].append(sc)
            got["q"].append(_e4m3(y / sc.repeat_interleave(128, dim=1)))
        if c["grad"]:
            dy = s["dy"][at].double()
            along = (dy * w * n).sum(dim=1, keepdim=True) / H
            got["d_x"].append((dy * w - along * n) / length + s["dsum"][at].double())
            dweight += (dy * n).sum(dim=0)
    got = {k: torch.cat(v) for k, v in got.items()}
    if c["grad"]:
        got["d_weight"] = dweight
    return got


def _exact_gate(c, s):
    x = s["x"].double()
    T, E, K, G = c["T"], c["E"], c["K"], c["G"]
    p = torch.sigmoid(x) if c["sigmoid"] else torch.softmax(x, dim=1)
    b = torch.zeros(E, dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].double()
    ids = torch.arange(E, device="cuda")
    groups = torch.arange(G, device="cuda")
    idx = torch.empty(T, K, dtype=torch.int64, device="cuda")
    for t in range(0, T, 512):
        v = p[t:t + 512] + b
        if G > 1:  # groups with fewer than KG others before them stay
            top = torch.topk(v.view(-1, G, E // G), 2, dim=2).values
            gs = top.sum(dim=2) if c["sum2"] else top[..., 0]
            before = ((gs[:, None, :] > gs[:, :, None])
                      | ((gs[:, None, :] == gs[:, :, None]) & (groups[None, :] < groups[:, None])))
            off = (before.sum(-1) >= c["KG"])[:, ids // (E // G)]
            v = v.masked_fill(off, -math.inf)
        before = ((v[:, None, :] > v[:, :, None])
                  | ((v[:, None, :] == v[:, :, None]) & (ids[None, :] < ids[:, None]))).sum(-1)
        idx[t:t + 512] = torch.argsort(before, dim=1)[:, :K]
    w = torch.gather(p, 1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"idx": idx, "weights": w * c["scale"]}


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    if c["op"] == "gate":
        return _exact_gate(c, s)
    if c["op"] == "lin_grad":
        dz = s["dz"].double()
        return {"d_x": dz @ s["w"].double(), "d_w": dz.t().contiguous() @ s["x"].double()}
    if c["op"] == "linear":
        z = s["x"].double() @ s["w"].double().t().contiguous()
        if c["bias"]:
            z += s["bias"].double()
    else:
        z = s["z"].double().requires_grad_(True)
    with torch.set_grad_enabled(c["op"] == "act_grad"):
        if c["act"] == "swiglu":
            h = torch.nn.functional.silu(z[:, :c["N"]]) * z[:, c["N"]:]
        elif c["act"] == "none":
            h = z
        else:
            h = getattr(torch.nn.functional, c["act"])(z)
        if c["op"] == "act_grad":
            h.backward(s["do"].double())
            return {"d_z": z.grad, "d_bias": z.grad.sum(dim=0)}
    got = {"out": h + s["res"].double() if c["res"] else h}
    if c["pre"]:
        got["z"] = z
    return got
