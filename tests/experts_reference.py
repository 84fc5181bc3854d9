"""Tight checks of the mixture of experts, on tests/block_reference.py's definitions: the codes that
its inner rows have, and how far outputs may be off in norm and elementwise.

The gated products have two forms (include/w8a8.h): exact products summed in fp32, up to 32 slots an
expert, and the e4m3 matrix instruction's beyond. The instruction is followed here step by step, so
that either form is held to what fp32 sums are off by: an inner element that is off by d crosses a
border between two codes with probability d over the codes' distance, and then moves by it."""
from __future__ import annotations

import numpy as np
import torch

from tests import block_reference as ref

EXACT_SLOTS = 32
GROUP, BITS = 8, 13              # of the instruction, see instruction_sums

# Error of a gate or up sum over its rms: 128 products of a block, then the blocks, are added in fp32,
# about 140 roundings of 2^-24 / sqrt(3) of partial sums that grow as the square root of their length:
# 2^-24 * sqrt(140 / 6) = 2^-21.7, taken as 2^-19.
SUMS = 2.0 ** -19


def is_exact(tokens, top_k, experts):
    return tokens * top_k // experts <= EXACT_SLOTS


def instruction_sums(x, w):
    """x @ w.T of e4m3 values [M, 128] and [N, 128] as v_mfma_scale_f32_16x16x128_f8f6f4 sums them on
    gfx950 (established on MI355X with products of chosen sizes and places; random codes then agree to
    fp32's rounding): of each 8 neighbouring products the bits below 2^-13 of the largest one's power of
    two are cut off, towards zero, and the 16 groups are added in fp32 (here: exactly)."""
    out = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    for k in range(0, ref.BLOCK, GROUP):
        a, b = x[:, None, k:k + GROUP], w[None, :, k:k + GROUP]
        p = a * b
        power = torch.frexp(a).exponent + torch.frexp(b).exponent - 2
        top = torch.where(p != 0, power, -100).amax(-1, keepdim=True)
        unit = torch.exp2((top - BITS).double())
        out += (torch.trunc(p / unit) * unit).sum(-1)
    return out


def instruction_product(xq, xs, wq, ws, device="cpu"):
    """block_reference.product's first result by the instruction: codes [M, K] and [N, K], their scales."""
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)
    pad = lambda q: to(ref._blocked(ref.VALUES[q]))
    x, w, total = pad(xq), pad(wq), 0
    sw = np.repeat(ws.astype(np.float64), ref.BLOCK, 0)[:len(wq)]
    for b in range(x.shape[1]):
        total = total + instruction_sums(x[:, b], w[:, b]) * torch.outer(to(xs[:, b].astype(np.float64)), to(sw[:, b]))
    return total.cpu().numpy()


def gated_sums(xq, xs, gate_up, scales, exact, device="cpu"):
    """The gate and up sums of rows (codes and scales) with an expert's weights (codes [2I, K], scales)."""
    inner, half = len(gate_up) // 2, len(scales) // 2
    both = ((gate_up[:inner], scales[:half]), (gate_up[inner:], scales[half:]))
    if exact:
        return [ref.dequant(xq, xs) @ ref.weight(*w).T for w in both]
    return [instruction_product(xq, xs, *w, device) for w in both]


def magnitudes(xq, xs, gate_up, scales):
    """Of the same sums, those of their products' magnitudes, and the root of those of their squares: the
    sums' rms, were the signs random."""
    inner, half, x = len(gate_up) // 2, len(scales) // 2, np.abs(ref.dequant(xq, xs))
    w = [np.abs(ref.weight(*p)) for p in ((gate_up[:inner], scales[:half]), (gate_up[inner:], scales[half:]))]
    return [x @ v.T for v in w], [np.sqrt((x ** 2) @ (v ** 2).T) for v in w]


def norm_limit(n):
    """Of the error of fp32 outputs over their norm, with n inner elements: an error d of a sum is one of
    about 2 * d of the element, whose codes lie 2^-4 of it apart or more, so that 2^5 * d cross a border,
    and move by 2^-3 at most. Four standard deviations of their number and four more are allowed, of n / 16
    elements: products of normal values spread the norm as fewer equal ones would (their fourth moment
    is 9 times the square of the second), tokens' weights differ. The down product's instruction adds, as
    SUMS of normal values, 2^-13 * sqrt(8 / 3) of a group's largest product at most: over the 16 groups of
    a block, whose largest product is about 5 of their rms, 2^-13 * 1.6 * 5 / sqrt(8) = 2^-11.5 at most."""
    n, p = n / 16, 2.0 ** 5 * SUMS
    return 2.0 ** -3 * np.sqrt(p + 4 * np.sqrt(p / n) + 4 / n) + 2.0 ** -11.5


def token_error(got, exact):
    """Root mean square over tokens of the error's norm over the token's."""
    got, exact = np.asarray(got, np.float64), np.asarray(exact, np.float64)
    own = np.linalg.norm(exact, axis=1)
    live = own > 0
    return np.sqrt(np.mean((np.linalg.norm(got - exact, axis=1)[live] / own[live]) ** 2))


def experts(x, ids, weights, parts, exact, inner_rows=None, device="cpu"):
    """(out, bound) of the mixture, as block_reference.experts, for rows x of floats and weights as codes
    and scales [gate_up, its scales, down, its scales] of each expert. inner_rows: what the values of the
    inner rows become on their way to the down product (the rule's codes by default).

    Bounds: a gate or up sum is off by 2^-23 of a partial sum at each of its additions, 128 of a block and
    then the blocks' with their scales' products; the down product by the instruction's 8 cut products of
    a group, each by less than 2^-13 of its largest, and the same additions."""
    xq, xs = ref.quant(x)
    K = x.shape[1]
    out, bound = np.zeros(x.shape), np.zeros(x.shape)
    for e in range(len(parts[0])):
        tok, slot = np.nonzero(ids == e)
        if not len(tok):
            continue
        gu, gs, dn, ds = (p[e] for p in parts)
        g, u = gated_sums(xq[tok], xs[tok], gu, gs, exact, device)
        dg, du = ((128 + ref.blocks_of(K) + 4) * 2.0 ** -23 * m for m in magnitudes(xq[tok], xs[tok], gu, gs)[0])
        h, dh = ref.gated(g, u, dg, du)
        hv, dhv = ref.requant(h, dh)
        if inner_rows is not None:
            hv = inner_rows(h)
        d = ref.weight(dn, ds)
        group = lambda a: np.abs(ref._blocked(a)).reshape(len(a), -1, GROUP).max(-1)
        dy = GROUP * 2.0 ** -BITS * (group(hv) @ group(d).T) + \
            (16 + ref.blocks_of(hv.shape[1]) + 4) * 2.0 ** -23 * (np.abs(hv) @ np.abs(d).T)
        dy = dy * (1 + 2.0 ** -3) + dhv @ np.abs(d).T        # (the product's own bound at moved codes too)
        y, w = hv @ d.T, weights[tok, slot].astype(np.float64)[:, None]
        # (more than 10 slots an expert: a slot's result waits as fp16, 2^-11 of it or 2^-38 of the scales' bound)
        s = np.repeat(np.abs(ds.astype(np.float64)), ref.BLOCK, 0)[:K]
        dy = dy + 2.0 ** -11 * (np.abs(y) + dy) + 2.0 ** -13 * (np.abs(ref._blocked(hv)).max(-1) / 448 @ s.T)
        np.add.at(out, tok, w * y)
        np.add.at(bound, tok, np.abs(w) * (dy + 2.0 ** -23 * (ids.shape[1] + 1) * (np.abs(y) + dy)))
    return out, bound


def inner_codes(h):
    """Codes and scales of inner rows by the rule in 64 bits, -0 as 0."""
    b = ref._blocked(h)
    a = np.abs(b).max(-1, keepdims=True)
    v = np.where(a >= 2.0 ** -100, b * 448 / np.where(a > 0, a, 1), 0)
    q = ref.e4m3(np.clip(v, -448, 448)).reshape(h.shape[0], -1)[:, :h.shape[1]]
    return np.where(q == 128, 0, q), a[..., 0] / 448


def codes_of(y, s):
    """The codes that rows y = code * scale, to within 2^-10 of them, stand for."""
    v = y / np.repeat(np.where(s > 0, s, 1), ref.BLOCK, 1)[:, :y.shape[1]]
    q = ref.e4m3(np.clip(v, -448, 448))
    assert (np.abs(ref.VALUES[q] - v) <= 2.0 ** -10 * np.abs(v)).all()
    return np.where(q == 128, 0, q)


def crossings(g, u, dg, du):
    """How many elements of inner rows silu(g) * u are expected to get another code where g and u have
    errors of standard deviations dg and du: the mean error (0.8 of its standard deviation, which holds the
    sums', the block maximum's and the fp32 steps' shares) over the codes' distance."""
    h = ref.silu(g) * u
    with np.errstate(over="ignore"):
        part = 1 / (1 + np.exp(-g))
    slope = part * (1 + g * (1 - part))
    off = np.sqrt((slope * u * dg) ** 2 + (ref.silu(g) * du) ** 2 + (h * 2.0 ** -22) ** 2)
    b, o = ref._blocked(h), ref._blocked(off)
    top = np.abs(b).argmax(-1)[..., None]
    most = np.maximum(np.abs(np.take_along_axis(b, top, -1)), 2.0 ** -100)
    o = np.sqrt(o ** 2 + (b * np.take_along_axis(o, top, -1) / most) ** 2)
    step = np.abs(b) * 448 / most
    step = 2.0 ** (np.floor(np.log2(np.maximum(step, 2.0 ** -6))) - 3)
    return float((0.8 * o * 448 / most / step).sum())


def diagonal(k, inner):
    """Codes and scales of a down weight [k, inner] that hands inner column j on as output column j, 448
    times: of each row of blocks only the diagonal one has a scale."""
    q, s = np.zeros((k, inner), np.uint8), np.zeros((ref.blocks_of(k), ref.blocks_of(inner)), np.float32)
    n = min(k, inner)
    q[np.arange(n), np.arange(n)] = 126
    s[np.arange(ref.blocks_of(n)), np.arange(ref.blocks_of(n))] = 1.0
    return q, s
