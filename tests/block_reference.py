"""The block-scaled e4m3 rule, its products, the routing and the mixture of
experts on the CPU: codes and scales in the rule's own fp32 steps, everything
else in 64 bits from the definitions. Shares no code with the package."""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 128


def blocks_of(n):
    return -(-n // BLOCK)


def e4m3_values():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m / 8.0 * 2.0 ** -6)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


VALUES = e4m3_values()
STEPS = VALUES[:127]                                       # the magnitudes 0 .. 448, rising


def e4m3(v):
    """Nearest codes of finite v within +-448, ties to the even code, the sign kept."""
    a = np.abs(np.asarray(v, dtype=np.float64))
    hi = np.clip(np.searchsorted(STEPS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - STEPS[lo], STEPS[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | (np.signbit(v).astype(int) << 7)).astype(np.uint8)


def scale_of(a):
    """fp32 scale and factor of blocks whose largest magnitude is a (fp32 array)."""
    a = np.asarray(a, dtype=np.float32)
    live = ~(a < np.float32(2.0 ** -100))
    with np.errstate(all="ignore"):
        s, f = a / np.float32(448), np.float32(1) / a * np.float32(448)
        return np.where(live, s, np.float32(0)), np.where(live, f, np.float32(0))


def _blocked(x):
    m, k = x.shape
    return np.pad(x, ((0, 0), (0, -k % BLOCK))).reshape(m, -1, BLOCK)


def quant(x):
    """(codes [M, K], fp32 scales [M, blocks]) of finite fp32 rows."""
    b = _blocked(np.asarray(x, dtype=np.float32))
    s, inv = scale_of(np.abs(b).max(-1, keepdims=True))
    t = np.clip((b * inv).astype(np.float32), -448, 448)
    return e4m3(t).reshape(x.shape[0], -1)[:, :x.shape[1]], s[..., 0]


def dequant(q, s):
    return VALUES[q] * np.repeat(s.astype(np.float64), BLOCK, 1)[:, :q.shape[1]]


def quant_weight(w):
    """(codes [N, K], fp32 scales [N blocks, K blocks]) of a finite fp32 matrix."""
    n, k = w.shape
    p = np.pad(np.asarray(w, dtype=np.float32), ((0, -n % BLOCK), (0, -k % BLOCK)))
    p = p.reshape(blocks_of(n), BLOCK, blocks_of(k), BLOCK)
    s, inv = scale_of(np.abs(p).max((1, 3), keepdims=True))
    q = e4m3(np.clip((p * inv).astype(np.float32), -448, 448))
    return q.reshape(blocks_of(n) * BLOCK, -1)[:n, :k], s[:, 0, :, 0]


def weight(q, s):
    s = np.repeat(np.repeat(s.astype(np.float64), BLOCK, 0), BLOCK, 1)
    return VALUES[q] * s[:q.shape[0], :q.shape[1]]


def product(x, w, k_total=None):
    """Exact x @ w.T of dequantized rows, and a bound on what an fp32 kernel on the
    e4m3 matrix instruction may be off by.

    The instruction's own error is not documented; it is bounded here, as for
    the layer with a scale per row, by 2^-9 of each 64 products' largest
    magnitudes' product (measured: 2^-11.4 at most). fp32: every block's sum is
    multiplied by a rounded product of scales and added, in any order: at
    most (blocks + 4) roundings of 2^-24 of partial sums up to sum |x w|."""
    k = x.shape[1]
    p = np.pad(np.abs(x), ((0, 0), (0, -k % 64))).reshape(x.shape[0], -1, 64).max(-1)
    r = np.pad(np.abs(w), ((0, 0), (0, -k % 64))).reshape(w.shape[0], -1, 64).max(-1)
    mag = np.abs(x) @ np.abs(w).T
    return x @ w.T, 2.0 ** -9 * (p @ r.T) + (blocks_of(k) + 4) * 2.0 ** -23 * mag


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1 + np.exp(-v))


def gated(g, u, dg, du):
    """silu(g) * u and a bound on its error for g and u off by up to dg and du:
    |silu'| < 1.1; the kernel's own exponential, sum, reciprocal and products
    add (|g| * 2^-24 * 1.45 + 5 * 2^-23) relative."""
    h = silu(g) * u
    d = 1.1 * dg * (np.abs(u) + du) + (np.abs(silu(g)) + 1.1 * dg) * du
    return h, d + (np.abs(g) * 2.0 ** -23 + 5 * 2.0 ** -23) * np.abs(h)


def requant(h, dh):
    """(values, bound): h through the rule's codes. Where an element's error (and its
    block maximum's) can move it across a border between two codes, the bound
    holds the codes' distance."""
    b, d = _blocked(h), _blocked(dh)
    a = np.abs(b).max(-1, keepdims=True)
    # the maximum's own error: of any element that may be it
    da = (np.abs(b) + d).max(-1, keepdims=True) - a + np.where(np.abs(b) + d >= a - d, d, 0).max(-1, keepdims=True)
    live = a >= 2.0 ** -100
    safe = np.where(live, a, 1.0)
    f = np.where(live, 448.0 / safe, 0.0)
    rel = da / safe + 4 * 2.0 ** -24
    v = b * f
    dv = d * f * (1 + rel) + np.abs(v) * rel
    at = np.clip(v, -448, 448)
    lo = VALUES[e4m3(np.clip(v - dv, -448, 448))]
    hi = VALUES[e4m3(np.clip(v + dv, -448, 448))]
    val = VALUES[e4m3(at)]
    s = a / 448.0
    bound = np.maximum(np.abs(hi - val), np.abs(val - lo)) * s * (1 + rel) + np.abs(val) * s * rel
    m, k = h.shape
    return (val * s).reshape(m, -1)[:, :k], bound.reshape(m, -1)[:, :k]


def experts(x, ids, weights, gate_up, down):
    """(out, bound) of the mixture: x [T, K] dequantized rows, gate_up [E][2I, K] and
    down [E][K, I] dequantized weights, before the last rounding."""
    T, K = x.shape
    out, bound = np.zeros((T, K)), np.zeros((T, K))
    for e in range(len(gate_up)):
        tok, slot = np.nonzero(ids == e)
        if not len(tok):
            continue
        inner = gate_up[e].shape[0] // 2
        up, dup = product(x[tok], gate_up[e])
        h, dh = gated(up[:, :inner], up[:, inner:], dup[:, :inner], dup[:, inner:])
        hv, dhv = requant(h, dh)
        y, dy = product(hv, down[e])
        dy = dy * (1 + 2.0 ** -6) + dhv @ np.abs(down[e]).T      # (the product's own bound at moved codes too)
        w = weights[tok, slot].astype(np.float64)[:, None]
        np.add.at(out, tok, w * y)
        np.add.at(bound, tok, np.abs(w) * (dy + 2.0 ** -23 * (ids.shape[1] + 1) * (np.abs(y) + dy)))
    return out, bound


def route(logits, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_top=2, renormalize=True, scale=1.0):
    """(ids, weights in 64 bits) by the definition, a row at a time."""
    T, E = logits.shape
    ids, weights = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))
    for t in range(T):
        x = logits[t].astype(np.float64)
        out = np.isnan(x) | (x == -np.inf)
        s = np.zeros(E)
        if score == "softmax":
            if not out.all():
                top = x[~out].max()
                e = np.array([0.0 if o else 1.0 if v == top else np.exp(v - top) for v, o in zip(x, out)])
                s = e / e.sum()
        else:
            s = np.array([0.0 if o else 1 / (1 + np.exp(-v)) if v > -700 else 0.0 for v, o in zip(x, out)])
        c = s.copy()
        if bias is not None:
            b = bias.astype(np.float64)
            out = out | np.isnan(b) | (b == -np.inf)
            c = c + np.where(np.isnan(b), 0, b)
        c = np.where(out, -np.inf, c)
        if groups > 1:
            worth = []
            for g in c.reshape(groups, -1):
                live = np.sort(g[g > -np.inf])[::-1]
                worth.append(live[:group_top].sum() if len(live) else -np.inf)
            best = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            c = np.where(np.isin(np.arange(E) // (E // groups), best), c, -np.inf)
        order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -np.inf][:top_k]
        w = s[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        ids[t, :len(order)] = order
        weights[t, :len(order)] = w * scale
    return ids, weights


def as_torch(a, device):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)
