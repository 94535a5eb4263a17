"""Plain 64-bit references of the operators around the experts, and the inputs
their tests share. Written from the definitions in moe_experts.h; nothing here
calls the library."""
from __future__ import annotations

import numpy as np
import torch

EPS24 = 2.0 ** -24  # half a float step, relative
HALF_BF16 = 2.0 ** -8


# ---- E4M3 ------------------------------------------------------------------

def e4m3_values(codes: np.ndarray) -> np.ndarray:
    """E4M3 codes (uint8) -> doubles."""
    t = torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn)
    return t.to(torch.float32).numpy().astype(np.float64)


def random_codes(rng, shape) -> np.ndarray:
    """Codes of a normal law that fills the range, no NaN."""
    v = np.clip(rng.standard_normal(shape, dtype=np.float32) * 112, -448, 448)
    return torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def product_bound(a: np.ndarray, b: np.ndarray, G: int) -> np.ndarray:
    """How far the matrix unit's sums of the products a[m, C] * b[n, C] (with
    their scales in them) may be from the exact ones.

    The instruction adds eight neighbouring channels at once, their products
    aligned to the largest exponent of the eight and cut off 13 bits below its
    binade (measured: 4096 + 1.265625 gives 4097, 4096 + 0.5625 gives 4096.5,
    65536 + 1.265625 gives 65536 inside one block of eight, and the exact sum
    across blocks). Each of the seven others so loses at most 2^-13 of the
    largest product. The 16 blocks of a group then add in float (16 half steps
    of their magnitudes, twice where a sum is cut instead of rounded), the
    scaling of a group costs 3 and the G groups G + 4."""
    ta, tb = (torch.from_numpy(np.abs(v)).to("cuda", torch.float32) for v in (a, b))
    m, C = ta.shape
    n = tb.shape[0]
    big = torch.empty(m, n, device="cuda", dtype=torch.float64)
    mag = torch.empty_like(big)
    step = max(1, (1 << 27) // (n * C))
    for i in range(0, m, step):
        p = (ta[i:i + step, None, :] * tb[None]).view(-1, n, C // 8, 8)
        big[i:i + step] = p.amax(-1).double().sum(-1)
        mag[i:i + step] = p.double().sum((-1, -2))
    # both sums of positive terms were made from float products: 2^-20 is ample
    out = 7 * 2.0 ** -13 * big + (2 * 16 + 3 + G + 4) * EPS24 * mag
    return (out * (1 + 2.0 ** -20)).cpu().numpy()


# ---- router ----------------------------------------------------------------

def gate_select(x: np.ndarray, K: int) -> np.ndarray:
    """ids [T, K]: larger logit first, equal ones by lower id, -1 where none is
    left; only finite logits can be selected."""
    T, E = x.shape
    key = np.where(np.isfinite(x), x, -np.inf)
    order = np.argsort(-key, axis=1, kind="stable")[:, :K]
    return np.where(np.isfinite(np.take_along_axis(key, order, 1)), order, -1).astype(np.int64)


def gate_weights(x: np.ndarray, ids: np.ndarray, sigmoid: bool, renorm: bool,
                 scale: float) -> np.ndarray:
    """Weights in 64 bits of the selected ids (-1, masked: 0)."""
    x = np.where(np.isfinite(x), x, -np.inf).astype(np.float64)
    sel = np.take_along_axis(x, np.maximum(ids, 0), 1)
    sel = np.where(ids < 0, -np.inf, sel)
    on = np.isfinite(sel)
    with np.errstate(all="ignore"):
        logsig = np.where(on, -np.logaddexp(0.0, -sel), -np.inf)
        z = logsig if sigmoid else sel
        if renorm:
            m = np.max(np.where(on, z, -np.inf), axis=1, keepdims=True)
            e = np.where(on, np.exp(z - np.where(np.isfinite(m), m, 0)), 0.0)
            s = e.sum(1, keepdims=True)
            p = np.where(on, e / np.where(s > 0, s, 1), 0.0)
        elif sigmoid:
            p = np.where(on, np.exp(logsig), 0.0)
        else:
            m = np.max(x, axis=1, keepdims=True)
            m = np.where(np.isfinite(m), m, 0)
            s = np.exp(x - m).sum(1, keepdims=True)
            p = np.where(on, np.exp(sel - m) / np.where(s > 0, s, 1), 0.0)
    return p * scale


def gate_grad(x: np.ndarray, ids: np.ndarray, dw: np.ndarray, sigmoid: bool, renorm: bool,
              scale: float) -> np.ndarray:
    T, E = x.shape
    p = gate_weights(x, ids, sigmoid, renorm, 1.0)
    xf = np.where(np.isfinite(x), x, -np.inf).astype(np.float64)
    sel = np.where(ids < 0, -np.inf, np.take_along_axis(xf, np.maximum(ids, 0), 1))
    on = np.isfinite(sel)
    d = np.where(on, dw.astype(np.float64) * scale, 0.0)
    dx = np.zeros((T, E))
    with np.errstate(all="ignore"):
        # sigmoid(-x) = 1 / (1 + exp(x)), 0 where exp overflows
        down = np.where(on, 1.0 / (1.0 + np.exp(np.where(on, sel, 0.0))), 0.0)
        if renorm:
            g = p * (d - (d * p).sum(1, keepdims=True))
            if sigmoid:
                g = g * down
        elif sigmoid:
            g = d * p * down
        else:
            m = np.max(xf, axis=1, keepdims=True)
            m = np.where(np.isfinite(m), m, 0)
            e = np.exp(xf - m)
            s = e.sum(1, keepdims=True)
            pe = e / np.where(s > 0, s, 1)
            dx -= pe * (d * p).sum(1, keepdims=True)
            g = d * p
    for k in range(ids.shape[1]):
        t = np.nonzero(on[:, k])[0]
        np.add.at(dx, (t, ids[t, k]), g[t, k])
    return dx


# ---- segments --------------------------------------------------------------

def lay_rows(counts, mode: str, per_expert: int = 0, align: int = 1, gap: int = 0):
    """(row_start, rows): contiguous segments (aligned, `gap` rows between them),
    or one at a place inside every expert's per_expert rows."""
    E = len(counts)
    if mode == "padded":
        src = (np.arange(E) * 7) % (per_expert - np.asarray(counts) + 1)
        return (np.arange(E) * per_expert + src).astype(np.int32), E * per_expert
    start, at = [], gap
    for c in counts:
        start.append(at)
        at += (c + align - 1) // align * align + gap
    return np.array(start, np.int32), max(at, 1)


def live_rows(start, counts):
    return np.concatenate([np.arange(s, s + c) for s, c in zip(start, counts)] +
                          [np.zeros(0, np.int64)]).astype(np.int64)


# ---- FP8 cast and activation -----------------------------------------------

def silu_mul(x: np.ndarray):
    """(gates, ups, sigmoid, h) in 64 bits of rows [n, 2I]."""
    x = x.astype(np.float64)
    I = x.shape[1] // 2
    g, u = x[:, :I], x[:, I:]
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return g, u, s, g * s * u
