"""The operators around the experts of a mixture-of-experts layer, as cases to measure.

Four families, each reached through the library's C-ABI binding (``own``) or
computed by elementary torch operations in 32 bits (the plain form):

* ``gate``          router logits -> top-k expert ids and weights, and the gradient;
* ``combine_grad``  gradient of the weighted combine: per receive row and per weight;
* ``gemm``          each expert's product of FP8 rows (a scale per 128 channels) with
                    its FP8 weights (a scale per 128 x 128 block), bf16 out;
* ``swiglu``        silu(gate) * up cast to FP8 (a scale per 128 channels) between an
                    expert's two products, and the activation's gradient.

Rows of expert e are ``row_start[e] ... row_start[e] + count[e]`` of a receive
buffer, as the contiguous and the low-latency layouts place them; all other
rows are left as they were.
"""
from __future__ import annotations

import math

import torch

own = False

FP8_MAX = 448.0
ROUND_SCALE, UE8M0, SCALE_ROWS = 1, 2, 4        # FP8 flags of the library
GATE_SIGMOID, GATE_RENORM = 2, 4                # router flags of the library
MAX_FLOPS = 3.8e12                              # the largest listed product
MAX_BYTES = 8.0e9


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a small batch: the router's launch latency
        dict(name="gate_16x256_bf16", op="gate", T=16, E=256, K=8, dtype="bf16", sigmoid=True,
             renorm=True, scale=2.5, grad=False, masked=0),
        # a training step's router, softmax over all experts
        dict(name="gate_8192x256_train", op="gate", T=8192, E=256, K=8, dtype="f32",
             sigmoid=False, renorm=False, scale=1.0, grad=True, masked=0),
        # the skewed batch's router, one of eight ranks taken out (its experts at -inf)
        dict(name="gate_4096x64_train", op="gate", T=4096, E=64, K=6, dtype="bf16",
             sigmoid=False, renorm=True, scale=1.0, grad=True, masked=8),
        # backward of the standard batch's combine
        dict(name="combine_grad_128x7168", op="combine_grad", T=128, H=7168, E=256, K=8, A=1,
             zipf=0.0, masked=0, neg=0.0),
        # the skewed batch, expert rows aligned to 16, some selections dropped, one rank masked
        dict(name="combine_grad_4096x4096", op="combine_grad", T=4096, H=4096, E=64, K=6, A=16,
             zipf=1.2, masked=1, neg=0.02),
        # a training batch
        dict(name="combine_grad_8192x7168", op="combine_grad", T=8192, H=7168, E=256, K=8, A=1,
             zipf=1.0, masked=0, neg=0.0),
        # first product of a decoding step: 16 tokens, every expert's rows in its stripe
        dict(name="gemm_ll16_7168x4096", op="gemm", ll=True, T=16, M=16, R=8, E=256, K=8, A=1,
             zipf=0.0, N=4096, C=7168, flags=0),
        # second product of a full low-latency batch, packed power-of-two scales by row
        dict(name="gemm_ll128_2048x7168", op="gemm", ll=True, T=128, M=128, R=8, E=256, K=8, A=1,
             zipf=0.0, N=7168, C=2048, flags=ROUND_SCALE | UE8M0 | SCALE_ROWS),
        # the skewed batch: from a few rows to thousands of an expert, ragged width
        dict(name="gemm_4096_skew_4096x2824", op="gemm", ll=False, T=4096, M=0, R=8, E=64, K=6,
             A=16, zipf=1.2, N=2824, C=4096, flags=SCALE_ROWS),
        # a prompt's or training batch's first product
        dict(name="gemm_8192_7168x4096", op="gemm", ll=False, T=8192, M=0, R=8, E=256, K=8, A=1,
             zipf=0.0, N=4096, C=7168, flags=SCALE_ROWS),
        # activation of a low-latency batch
        dict(name="swiglu_ll64_2048", op="swiglu", ll=True, T=64, M=64, R=8, E=256, K=8, A=1,
             zipf=0.0, I=2048, grad=False),
        # activation of a training batch, forward and backward
        dict(name="swiglu_8192_2048_train", op="swiglu", ll=False, T=8192, M=0, R=8, E=256, K=8,
             A=1, zipf=1.0, I=2048, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _routing(rng, c, most_t):
    E = c["E"]
    c["K"] = rng.choice([k for k in (1, 2, 4, 6, 8) if k <= E])
    c["T"] = _log(rng, 1, most_t)
    c["zipf"] = rng.choice([0.0, 1.0, 1.2])


def _segments(rng, c):
    """The layout half of a drawn case: padded stripes or contiguous rows."""
    c["ll"] = rng.random() < 0.5
    c["R"] = 8
    c["E"] = rng.choice([8, 16, 32, 64, 128, 256])
    _routing(rng, c, 512 if c["ll"] else 8192)
    c["M"] = min(512, c["T"] + rng.randrange(0, 17)) if c["ll"] else 0
    c["A"] = 1 if c["ll"] else rng.choice([1, 16, 128])


def draw(rng):
    op = rng.choice(["gate", "combine_grad", "gemm", "gemm", "swiglu"])
    while True:
        c = dict(op=op)
        if op == "gate":
            c["E"] = rng.choice([16, 60, 64, 128, 160, 256])
            c["K"] = rng.choice([1, 2, 4, 6, 8])
            c["T"] = _log(rng, 1, 8192)
            c["dtype"] = rng.choice(["f32", "bf16"])
            c["sigmoid"], c["renorm"] = rng.random() < 0.5, rng.random() < 0.5
            c["scale"] = rng.choice([1.0, 2.5])
            c["grad"] = rng.random() < 0.5
            c["masked"] = rng.choice([0, 0, c["E"] // 8])
        elif op == "combine_grad":
            c["E"] = rng.choice([16, 64, 256])
            _routing(rng, c, 8192)
            c["H"] = 8 * _log(rng, 32, 896)
            c["A"] = rng.choice([1, 16])
            c["masked"] = rng.choice([0, 1])
            c["neg"] = rng.choice([0.0, 0.05])
        elif op == "gemm":
            _segments(rng, c)
            c["N"] = 8 * _log(rng, 64, 896)
            words = rng.random() < 0.3
            c["C"] = 512 * rng.randrange(1, 15) if words else 128 * _log(rng, 2, 56)
            c["flags"] = (ROUND_SCALE | UE8M0) if words else rng.choice([0, ROUND_SCALE])
            if not c["ll"] or rng.random() < 0.5:
                c["flags"] |= SCALE_ROWS
        else:
            _segments(rng, c)
            c["I"] = 128 * _log(rng, 2, 32)
            c["grad"] = rng.random() < 0.5
        w = work(c)
        if w["flops"] <= MAX_FLOPS and w["bytes"] <= MAX_BYTES and _buffers(c) <= 6e9:
            return c


def _rows(c):
    """Rows of a case's receive buffer."""
    if c.get("ll"):
        return c["E"] * c["R"] * c["M"]
    return c["T"] * c["K"] + c["E"] * (c["A"] - 1)


def _buffers(c):
    """Bytes that bound a drawn case: what its state and its plain form hold."""
    if c["op"] == "gemm":
        most = c["T"] if c["zipf"] else min(c["T"], 2 * c["T"] * c["K"] // c["E"] + 32)
        return max(_rows(c) * (c["C"] + 2 * c["N"]), c["E"] * c["C"] * c["N"] * 0.75,
                   c["E"] * most * (c["C"] + c["N"]) * 1.0)
    if c["op"] == "swiglu":
        return _rows(c) * c["I"] * (9 if c["grad"] else 5)
    return 0


def work(case):
    c = case
    if c["op"] == "gate":
        el = 4 if c["dtype"] == "f32" else 2
        T, E, K = c["T"], c["E"], c["K"]
        b = T * E * el + T * K * 12
        if c["grad"]:
            b += T * K * 4 + T * E * el
        return {"bytes": b, "flops": 4 * T * E * (2 if c["grad"] else 1)}
    pairs = c["T"] * c["K"]
    if c["op"] == "combine_grad":
        n = pairs * (1 - c["neg"])
        return {"bytes": c["T"] * c["H"] * 2 + n * c["H"] * 4 + pairs * 12, "flops": 3 * n * c["H"]}
    if c["op"] == "gemm":
        E, N, C = c["E"], c["N"], c["C"]
        p = [1.0 / E] * E
        if c["zipf"]:
            p = [(i + 1) ** -c["zipf"] for i in range(E)]
            s = sum(p)
            p = [v / s for v in p]
        used = sum(1 - (1 - min(1.0, v * c["K"])) ** c["T"] for v in p)
        b = used * (N * C + ((N + 127) // 128) * (C // 128) * 4)
        b += pairs * (C + C // 128 * (1 if c["flags"] & UE8M0 else 4) + 2 * N)
        return {"bytes": b, "flops": 2 * pairs * N * C}
    I = c["I"]
    b = pairs * (4 * I + I + I // 128 * 4)
    if c["grad"]:
        b += pairs * (2 * I + 4 * I)
    return {"bytes": b, "flops": pairs * I * (16 if c["grad"] else 6)}


# ---------------------------------------------------------------- inputs

def _route(c, g):
    """topk ids [T, K] int64 (distinct in a row) and weights [T, K] float."""
    T, E, K = c["T"], c["E"], c["K"]
    keys = torch.rand(T, E, generator=g, device="cuda")
    if c["zipf"]:
        logp = -c["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        logp = logp[torch.randperm(E, generator=g, device="cuda")]
        keys = logp - torch.log(-torch.log(keys.clamp(1e-7, 1 - 1e-7)))
    idx = torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :K].contiguous()
    w = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), dim=1)
    if c.get("neg"):
        idx = torch.where(torch.rand(T, K, generator=g, device="cuda") < c["neg"], -1, idx)
    return idx, w


def _layout(c, idx):
    """count, offset [E + 1], slot [T, K]: stable slots, as the layout calls give them."""
    E = c["E"]
    flat = idx.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    n = torch.bincount(key, minlength=E + 1)
    first = torch.cumsum(n, 0) - n
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device="cuda") - first[key[order]]
    count = n[:E]
    if c.get("ll"):
        start = torch.arange(E + 1, device="cuda") * (c["R"] * c["M"])
    else:
        up = (count + c["A"] - 1) // c["A"] * c["A"]
        start = torch.cat([torch.zeros(1, dtype=up.dtype, device="cuda"), torch.cumsum(up, 0)])
    slot = torch.where(flat < 0, -1, start[key.clamp(max=E - 1)] + rank)
    return (count.to(torch.int32), start.to(torch.int32), slot.to(torch.int32).view(idx.shape))


def _cast_rows(x):
    """Rows -> (E4M3 codes, float scale per 128 channels)."""
    n, w = x.shape
    v = x.view(n, w // 128, 128)
    s = v.abs().amax(-1).clamp_min(1e-4) / FP8_MAX
    return (v / s[..., None]).view(n, w).to(torch.float8_e4m3fn), s


def _pow2_up(s):
    """The smallest power of two at or above each positive normal float."""
    b = s.view(torch.int32)
    return torch.where((b & 0x7FFFFF) != 0, (b & 0x7F800000) + 0x800000, b).view(torch.float32)


def _pack(s):
    """Power-of-two scales [n, G] -> int32 words [n, G / 4] of exponent bytes."""
    e = (s.contiguous().view(torch.int32) >> 23) & 255
    e = e.view(s.shape[0], -1, 4)
    return (e[..., 0] | e[..., 1] << 8 | e[..., 2] << 16 | e[..., 3] << 24).contiguous()


def _segment_plan(c, s, idx):
    s["count"], s["offset"], slot = _layout(c, idx)
    n = c["T"] * c["K"]
    live = torch.sort(slot.reshape(-1).long()).values      # the rows in use, expert by expert
    s["live"], s["live_n"] = live, n
    s["cap"] = max(int(s["count"].max()), 1)
    e = torch.searchsorted(s["offset"][:c["E"]].long().contiguous(), live, right=True) - 1
    # empty experts share their start with the next one: the last of them holds the row
    s["expert"] = e
    s["place"] = e * s["cap"] + live - s["offset"].long()[e]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c=c)
    dev = dict(device="cuda")
    if c["op"] == "gate":
        T, E, K = c["T"], c["E"], c["K"]
        x = torch.randn(T, E, generator=g, **dev) * 1.5
        if c["masked"]:
            lo = int(torch.randint(0, E - c["masked"] + 1, (1,), generator=g, **dev))
            x[:, lo:lo + c["masked"]] = -math.inf
        s["x"] = x if c["dtype"] == "f32" else x.to(torch.bfloat16)
        s["dw"] = torch.randn(T, K, generator=g, **dev)
        s["idx"] = torch.empty(T, K, dtype=torch.int64, **dev)
        s["w"] = torch.empty(T, K, **dev)
        s["dx"] = torch.empty_like(s["x"])
        return s
    idx, w = _route(c, g)
    if c["op"] == "combine_grad":
        T, H = c["T"], c["H"]
        rows = _rows(c)
        _, _, s["slot"] = _layout(c, idx)
        s["idx"], s["w"], s["rows"] = idx, w, rows
        s["do"] = (torch.randn(T, H, generator=g, **dev) * 0.02).to(torch.bfloat16)
        s["y"] = torch.randn(rows, H, generator=g, **dev).to(torch.bfloat16)
        # one row more than the buffer: where the plain form puts pairs without a row
        s["dy"] = torch.zeros(rows + 1, H, dtype=torch.bfloat16, **dev)
        s["dw"] = torch.empty(T, c["K"], **dev)
        s["mask"] = None
        if c["masked"]:
            s["mask"] = torch.zeros(8, dtype=torch.int32, **dev)
            s["mask"][int(torch.randint(0, 8, (1,), generator=g, **dev))] = 1
        return s
    _segment_plan(c, s, idx)
    rows, n, live, E = _rows(c), s["live_n"], s["live"], c["E"]
    if c["op"] == "gemm":
        N, C = c["N"], c["C"]
        G, B = C // 128, (N + 127) // 128
        a, sc = _cast_rows(torch.randn(n, C, generator=g, **dev)
                           * torch.exp(torch.randn(n, 1, generator=g, **dev) * 0.5))
        s["a"] = torch.zeros(rows, C, dtype=torch.uint8, **dev)
        s["a"][live] = a.view(torch.uint8)
        s["a"] = s["a"].view(torch.float8_e4m3fn)
        if c["flags"] & ROUND_SCALE:
            sc = _pow2_up(sc)
        if c["flags"] & UE8M0:
            sc = _pack(sc)
        full = torch.zeros(rows, sc.shape[1], dtype=sc.dtype, **dev)
        full[live] = sc
        if not c["flags"] & SCALE_ROWS:  # column-major in each expert's rows
            full = full.view(E, rows // E, -1).transpose(1, 2).contiguous()
        s["as"] = full
        s["b"] = torch.empty(E, N, C, dtype=torch.float8_e4m3fn, **dev)
        for e in range(0, E, 16):  # weights near a normal law fill the codes to about 4 sigma
            part = s["b"][e:e + 16]
            v = torch.randn(part.shape, generator=g, dtype=torch.float16, **dev)
            part.copy_(v.mul_(112).clamp_(-FP8_MAX, FP8_MAX))
        s["bs"] = (4.0 / FP8_MAX / math.sqrt(C)
                   * (0.8 + 0.4 * torch.rand(E, B, G, generator=g, **dev)))
        s["out"] = torch.zeros(rows, N, dtype=torch.bfloat16, **dev)
        return s
    I = c["I"]
    s["x"] = torch.zeros(rows, 2 * I, dtype=torch.bfloat16, **dev)
    s["x"][live] = torch.randn(n, 2 * I, generator=g, **dev).to(torch.bfloat16)
    s["q"] = torch.zeros(rows, I, dtype=torch.uint8, **dev)
    s["qs"] = torch.zeros(rows, I // 128, **dev)
    if c["grad"]:
        s["dh"] = torch.zeros(rows, I, dtype=torch.bfloat16, **dev)
        s["dh"][live] = (torch.randn(n, I, generator=g, **dev) * 0.02).to(torch.bfloat16)
        s["dx"] = torch.zeros(rows, 2 * I, dtype=torch.bfloat16, **dev)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return {"gate": _plain_gate, "combine_grad": _plain_combine_grad, "gemm": _plain_gemm,
            "swiglu": _plain_swiglu}[state["c"]["op"]](state)


def _run_own(s):
    from combine_moe_layout_03_amd import capi

    c = s["c"]
    if c["op"] == "gate":
        T, E, K = c["T"], c["E"], c["K"]
        flags = (GATE_SIGMOID if c["sigmoid"] else 0) | (GATE_RENORM if c["renorm"] else 0)
        capi.moe_gate(T, E, K, s["x"], s["idx"], s["w"], flags, c["scale"])
        if not c["grad"]:
            return {"idx": s["idx"], "weights": s["w"]}
        capi.moe_gate_grad(T, E, K, s["x"], s["idx"], s["dw"], s["dx"], flags, c["scale"])
        return {"idx": s["idx"], "weights": s["w"], "d_logits": s["dx"]}
    if c["op"] == "combine_grad":
        shape = capi.make_shape(c["T"], c["H"], c["E"], 8, c["K"], c["A"])
        dy = s["dy"][:s["rows"]]
        capi.moe_combine_grad(shape, s["do"], s["y"], s["rows"], s["slot"], s["w"], dy, s["dw"],
                              s["idx"] if c["masked"] else None, s["mask"])
        return {"d_y": dy, "d_weights": s["dw"]}
    if c["op"] == "gemm":
        capi.moe_grouped_gemm_fp8(c["E"], c["N"], c["C"], s["a"], s["as"], s["a"].shape[0],
                                  s["offset"], s["count"], s["b"], s["bs"], s["out"], c["flags"],
                                  max_count=c["T"])
        return {"out": s["out"]}
    capi.moe_swiglu_fp8(c["E"], c["I"], s["x"].shape[0], s["x"], s["offset"], s["count"], s["q"],
                        s["qs"])
    got = {"h": s["q"].view(torch.float8_e4m3fn), "scale": s["qs"]}
    if c["grad"]:
        capi.moe_swiglu_grad(c["E"], c["I"], s["x"].shape[0], s["x"], s["dh"], s["offset"],
                             s["count"], s["dx"])
        got["d_x"] = s["dx"]
    return got


def _plain_gate(s):
    c, K = s["c"], s["c"]["K"]
    x = s["x"].float()
    top, idx = torch.sort(x, dim=1, descending=True, stable=True)
    top, idx = top[:, :K], idx[:, :K]
    off = top == -math.inf                       # masked experts are never selected
    none = off.all(dim=1, keepdim=True)
    if c["sigmoid"]:
        z = torch.minimum(top, torch.zeros_like(top)) - torch.log1p(torch.exp(-top.abs()))
        z = torch.where(off, -math.inf, z)       # log sigmoid
        score = torch.exp(z)
    else:
        m = torch.where(none, 0.0, x.amax(dim=1, keepdim=True))
        score = torch.exp(top - m) / torch.exp(x - m).sum(dim=1, keepdim=True)
        z = top
    if c["renorm"]:
        zm = torch.where(none, 0.0, z.amax(dim=1, keepdim=True))
        ez = torch.exp(z - zm)
        score = ez / ez.sum(dim=1, keepdim=True)
    w = torch.where(off, 0.0, score * c["scale"])
    idx = torch.where(off, -1, idx)
    if not c["grad"]:
        return {"idx": idx, "weights": w}
    dw = torch.where(off, 0.0, s["dw"] * c["scale"])
    p = torch.where(off, 0.0, score)
    if c["renorm"]:
        d = p * (dw - (dw * p).sum(dim=1, keepdim=True))
        if c["sigmoid"]:
            d = d * torch.exp(-torch.clamp(top, min=0) - torch.log1p(torch.exp(-top.abs())))
        d = torch.where(off, 0.0, d)
        dx = torch.zeros_like(x).scatter_add(1, idx.clamp_min(0), d)
    elif c["sigmoid"]:
        d = torch.where(off, 0.0, dw * p * torch.exp(-torch.clamp(top, min=0)
                                                     - torch.log1p(torch.exp(-top.abs()))))
        dx = torch.zeros_like(x).scatter_add(1, idx.clamp_min(0), d)
    else:
        e = torch.exp(x - m)
        pe = e / e.sum(dim=1, keepdim=True)
        dx = -pe * (dw * p).sum(dim=1, keepdim=True)
        dx = dx.scatter_add(1, idx.clamp_min(0), dw * p)
    return {"idx": idx, "weights": w, "d_logits": dx.to(s["x"].dtype)}


def _plain_combine_grad(s):
    c = s["c"]
    slot = s["slot"].long()
    on = slot >= 0
    do = s["do"].float()[:, None, :]
    wt = s["w"]
    if c["masked"]:
        dead = s["mask"].bool()[(s["idx"].clamp_min(0) // (c["E"] // 8))]
        wt = torch.where(dead, 0.0, wt)
        live = on & ~dead
    else:
        live = on
    y = s["y"][slot.clamp_min(0)].float()
    dw = torch.where(live, (do * y).sum(-1), 0.0)
    g = (do * wt[..., None]).to(torch.bfloat16)
    if c["masked"]:
        g = torch.where(dead[..., None], 0.0, g)
    s["dy"][torch.where(on, slot, s["rows"]).reshape(-1)] = g.view(-1, c["H"])
    return {"d_y": s["dy"][:s["rows"]], "d_weights": dw}


def _row_scales(s):
    """The float scales [rows in use, C / 128] of a product's rows."""
    c, t = s["c"], s["as"]
    if not c["flags"] & SCALE_ROWS:
        t = t.transpose(1, 2).reshape(-1, t.shape[1])
    t = t[s["live"]]
    if c["flags"] & UE8M0:
        b = torch.stack([(t >> k) & 255 for k in (0, 8, 16, 24)], dim=-1).view(t.shape[0], -1)
        t = torch.exp2((b - 127).float())
    return t


def _plain_gemm(s):
    c = s["c"]
    E, N, C, cap = c["E"], c["N"], c["C"], s["cap"]
    a = s["a"].view(torch.uint8)[s["live"]].view(torch.float8_e4m3fn).float().view(-1, C // 128, 128)
    a = (a * _row_scales(s)[..., None]).view(-1, C)
    pad = torch.zeros(E * cap, C, device="cuda")
    pad[s["place"]] = a
    bs = s["bs"].repeat_interleave(128, dim=1)[:, :N]
    b = (s["b"].float().view(E, N, C // 128, 128) * bs[..., None]).view(E, N, C)
    o = torch.bmm(pad.view(E, cap, C), b.transpose(1, 2))
    s["out"][s["live"]] = o.view(E * cap, N)[s["place"]].to(torch.bfloat16)
    return {"out": s["out"]}


def _plain_swiglu(s):
    c, I = s["c"], s["c"]["I"]
    x = s["x"][s["live"]].float()
    g, u = x[:, :I], x[:, I:]
    sg = 1.0 / (1.0 + torch.exp(-g))
    h = (g * sg * u).view(-1, I // 128, 128)
    sc = h.abs().amax(-1).clamp_min(1e-4) / FP8_MAX
    q = (h / sc[..., None]).clamp(-FP8_MAX, FP8_MAX).view(-1, I).to(torch.float8_e4m3fn)
    s["q"][s["live"]] = q.view(torch.uint8)
    s["qs"][s["live"]] = sc
    got = {"h": s["q"].view(torch.float8_e4m3fn), "scale": s["qs"]}
    if c["grad"]:
        d = s["dh"][s["live"]].float()
        dg = d * u * sg * (1.0 + g * (1.0 - sg))
        s["dx"][s["live"]] = torch.cat([dg, d * g * sg], dim=1).to(torch.bfloat16)
        got["d_x"] = s["dx"]
    return got


# ---------------------------------------------------------------- 64 bits

def _e4m3(v):
    """Doubles -> the nearest E4M3 value (ties to even), saturating at 448."""
    m = v.abs().clamp(max=FP8_MAX)
    e = torch.floor(torch.log2(m.clamp_min(2.0 ** -20)))
    e = torch.where(torch.exp2(e) > m, e - 1, e)
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.copysign(torch.round(m / step) * step, v).clamp(-FP8_MAX, FP8_MAX)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "gate":
        x = s["x"].double()
        T, E = x.shape
        K = c["K"]
        # rank of each expert: how many come before it (a larger logit, or an equal one of lower id)
        ids = torch.arange(E, device="cuda")
        idx = torch.empty(T, K, dtype=torch.int64, device="cuda")
        for t in range(0, T, 1024):
            v = x[t:t + 1024]
            before = ((v[:, None, :] > v[:, :, None])
                      | ((v[:, None, :] == v[:, :, None]) & (ids[None, :] < ids[:, None]))).sum(-1)
            idx[t:t + 1024] = torch.argsort(before, dim=1)[:, :K]
        xx = x.clone().requires_grad_(True)
        with torch.enable_grad():
            f = torch.nn.functional.logsigmoid(xx) if c["sigmoid"] else xx
            sel = torch.gather(f, 1, idx)
            if c["renorm"]:
                w = torch.softmax(sel, dim=1)
            elif c["sigmoid"]:
                w = torch.exp(sel)
            else:
                w = torch.exp(sel - torch.logsumexp(f, dim=1, keepdim=True))
            w = w * c["scale"]
            if c["grad"]:
                w.backward(s["dw"].double())
        off = torch.gather(x, 1, idx) == -math.inf
        got = {"idx": torch.where(off, -1, idx), "weights": w.detach()}
        if c["grad"]:
            got["d_logits"] = xx.grad.nan_to_num(0.0)
        return got
    if c["op"] == "combine_grad":
        T, H, K = c["T"], c["H"], c["K"]
        dy = torch.zeros(s["rows"], H, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        do, slot = s["do"].double(), s["slot"].long()
        for k in range(K):
            w = s["w"][:, k].double()
            if c["masked"]:
                w = w * (1 - s["mask"][s["idx"][:, k].clamp_min(0) * 8 // c["E"]].double())
            t = torch.nonzero(slot[:, k] >= 0)[:, 0]
            r = slot[t, k]
            dy[r] = do[t] * w[t, None]
            dw[t, k] = (do[t] * s["y"][r].double()).sum(-1) * (w[t] != 0)
        return {"d_y": dy, "d_weights": dw}
    rows, start, count = _rows(c), s["offset"].tolist(), s["count"].tolist()
    if c["op"] == "gemm":
        N, C = c["N"], c["C"]
        out = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
        sc = torch.zeros(rows, C // 128, dtype=torch.float64, device="cuda")
        sc[s["live"]] = _row_scales(s).double()
        for e in range(c["E"]):
            if not count[e]:
                continue
            r = slice(start[e], start[e] + count[e])
            a = s["a"][r].double() * sc[r].repeat_interleave(128, dim=1)
            bs = s["bs"][e].double().repeat_interleave(128, dim=0)[:N]
            b = s["b"][e].double() * bs.repeat_interleave(128, dim=1)
            out[r] = a @ b.t().contiguous()
        return {"out": out}
    I = c["I"]
    hq = torch.zeros(rows, I, dtype=torch.float64, device="cuda")
    qs = torch.zeros(rows, I // 128, dtype=torch.float64, device="cuda")
    dx = torch.zeros(rows, 2 * I, dtype=torch.float64, device="cuda") if c["grad"] else None
    for at in s["live"].split(8192):
        x = s["x"][at].double()
        g, u = x[:, :I], x[:, I:]
        h = (torch.nn.functional.silu(g) * u).view(-1, I // 128, 128)
        sc = h.abs().amax(-1).clamp_min(1e-4) / FP8_MAX
        hq[at] = _e4m3((h / sc[..., None]).view(-1, I))
        qs[at] = sc
        if c["grad"]:
            d, sg = s["dh"][at].double(), torch.sigmoid(g)
            dx[at] = torch.cat([d * u * sg * (1 + g * (1 - sg)), d * g * sg], dim=1)
    got = {"h": hq, "scale": qs}
    if c["grad"]:
        got["d_x"] = dx
    return got
