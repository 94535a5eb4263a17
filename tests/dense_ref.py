"""Plain 64-bit references of the norm, the grouped router and the dense product,
and the bounds their tests share. Written from the definitions in moe_experts.h;
nothing here calls the library."""
from __future__ import annotations

import numpy as np
import torch

EPS24 = 2.0 ** -24  # half a float step, relative
HALF_BF16 = 2.0 ** -8
ACTS = ("none", "silu", "gelu", "swiglu")


def guarded(n, dtype, device, fill=float("nan"), pad=4096):
    """(the buffer, its first n elements): NaN behind them, which nothing may read
    into a result or overwrite."""
    b = torch.full((n + pad,), fill, device=device, dtype=dtype)
    return b, b[:n]


def guard_ok(b, n):
    return bool(torch.isnan(b[n:].float()).all())


# ---- router ----------------------------------------------------------------

def grouped_select(x, bias, K, G, KG, sigmoid, sum2):
    """(ids [T, K] int64, scores [T, E]) in doubles from the definition; x and bias
    numpy. Not finite but -infinity counts as masked."""
    T, E = x.shape
    x = np.where(np.isfinite(x), x, -np.inf).astype(np.float64)
    with np.errstate(all="ignore"):
        if sigmoid:
            s = 1.0 / (1.0 + np.exp(-x))
        else:
            top = np.max(x, axis=1, keepdims=True)
            e = np.exp(x - np.where(np.isfinite(top), top, 0.0))
            s = e / e.sum(1, keepdims=True)
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    ids = np.full((T, K), -1, np.int64)
    n = E // G
    for t in range(T):
        ok = [e for e in range(E) if np.isfinite(x[t, e]) and np.isfinite(b[e])]
        c = {e: s[t, e] + b[e] for e in ok}
        groups = {}
        for e in ok:
            groups.setdefault(e // n, []).append(c[e])
        score = {}
        for g, v in groups.items():
            v = sorted(v, reverse=True)
            score[g] = v[0] + v[1] if sum2 and len(v) > 1 else v[0]
        kept = set(sorted(score, key=lambda g: (-score[g], g))[:KG])
        order = sorted((e for e in ok if e // n in kept), key=lambda e: (-c[e], e))[:K]
        ids[t, :len(order)] = order
    return ids, s


def grouped_weights(x, ids, s, sigmoid, renorm, scale):
    """Weights of the selected experts; renormalised from the logits' own logarithms,
    which do not underflow."""
    x = np.where(np.isfinite(x), x, -np.inf).astype(np.float64)
    on = ids >= 0
    at = np.maximum(ids, 0)
    if renorm:
        z = np.take_along_axis(x, at, 1)
        if sigmoid:
            z = np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z)))
        z = np.where(on, z, -np.inf)
        top = np.max(z, axis=1, keepdims=True)
        e = np.exp(z - np.where(np.isfinite(top), top, 0.0))
        w = e / np.where(e.sum(1, keepdims=True) > 0, e.sum(1, keepdims=True), 1.0)
    else:
        w = np.take_along_axis(s, at, 1)
    return np.where(on, w * scale, 0.0)


# ---- dense product ---------------------------------------------------------

def dot_bound(a, b):
    """(a b^T, how far the matrix unit's float sums may be from it), doubles on the
    GPU; a [m, k], b [n, k].

    The unit adds eight neighbouring products at once, cut at the last bit of the
    largest one's float (at most 8 half steps of it, twice as it is cut), and then
    k / 8 such sums one after the other, each addition off by at most a whole float
    step of the magnitudes' sum. Partial sums of a split product add at most 64
    more."""
    a, b = a.double(), b.double()
    k = a.shape[1]
    mag = a.abs() @ b.abs().t().contiguous()
    return a @ b.t().contiguous(), (k / 8 + 16 + 64) * 2 * EPS24 * mag


def act64(z, act, N):
    """act(z) and the largest slope times |z|'s error, as a function: the value and
    |d act| per unit of error in each half."""
    if act == "none":
        return z, torch.ones_like(z), None
    if act == "swiglu":
        a, u = z[:, :N], z[:, N:]
        s = torch.sigmoid(a)
        return a * s * u, (s * (1 + a * (1 - s)) * u).abs(), (a * s).abs()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, (s * (1 + z * (1 - s))).abs(), None
    phi = torch.special.ndtr(z)
    return z * phi, (phi + z * torch.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)).abs(), None


def act_grad64(z, d, act, N):
    """d_z in doubles."""
    if act == "swiglu":
        a, u = z[:, :N], z[:, N:]
        s = torch.sigmoid(a)
        return torch.cat([d * u * s * (1 + a * (1 - s)), d * a * s], dim=1)
    if act == "silu":
        s = torch.sigmoid(z)
        return d * s * (1 + z * (1 - s))
    if act == "gelu":
        return d * (torch.special.ndtr(z) + z * torch.exp(-0.5 * z * z) / np.sqrt(2 * np.pi))
    return d
