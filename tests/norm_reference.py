"""The norms and gated residuals around a layer in 64 bits, with a bound on
what fp32 arithmetic may differ by, element for element.

With u = 2^-24 and L = K/256 + 32 (no sum of K terms is a longer chain of
fp32 additions than that: at least 64 lanes of 8 elements or 256 of them
share a row, and trees join the rest), to first order:
  mean:      off by L u mean|v|, plus the mean of v's own error
  v - mean:  d = v_err + mean_err + u |v - mean|
  deviation: relative (L + 8) u + rms(d) / deviation
  n:         d / deviation + |n| * that
each later product and sum adds u of its result. Twice the sum covers the
second order."""
from __future__ import annotations

import torch

U = 2.0 ** -24


def norm(v, v_err, kind, eps, weight=None, bias=None, scale=None, shift=None):
    """(norm(v), bound) of float64 rows v [M, K] known within v_err; vectors as
    in ops.Norm, any float type."""
    M, K = v.shape
    L = K / 256 + 32
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    d = v - mean
    d_err = v_err + U * d.abs()
    if kind == "layer":
        d_err = d_err + L * U * v.abs().mean(-1, keepdim=True) + v_err.mean(-1, keepdim=True)
    dev = torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    n = d / dev
    rel = (L + 8) * U + torch.sqrt((d_err * d_err).mean(-1, keepdim=True)) / dev
    err = d_err / dev + n.abs() * rel
    rows = lambda t: t.double().reshape(-1, K).repeat_interleave(M // t.reshape(-1, K).shape[0], 0)  # noqa: E731
    for t, mul in ((weight, 0), (bias, None), (scale, 1), (shift, None)):
        if t is None:
            continue
        t = rows(t)
        if mul is None:
            n = n + t
            err = err + U * (n.abs() + t.abs())
        else:
            n = n * (t + mul)
            err = err * (t + mul).abs() + 3 * U * n.abs()
    return n, 2 * err


def residual(x, y, gate=None, post=None, residual_scale=1.0, branch_scale=1.0):
    """(r, bound) before r is rounded to its stored type; post: the arguments of
    norm() after its error."""
    x, b = x.double(), y.double()
    M, K = x.shape
    # the two factors reach the arithmetic as fp32
    residual_scale, branch_scale = (float(torch.tensor(s, dtype=torch.float32)) for s in (residual_scale, branch_scale))
    err = torch.zeros_like(b)
    if post is not None:
        b, err = norm(b, err, **post)
    if gate is not None:
        g = gate.double().reshape(-1, K)
        g = g.repeat_interleave(M // g.shape[0], 0)
        b, err = b * g, err * g.abs() + U * (b * g).abs()
    r = residual_scale * x + branch_scale * b
    return r, 2 * (abs(branch_scale) * err + 2 * U * ((residual_scale * x).abs() + (branch_scale * b).abs()))


def check_float(got, want, bound, dtype, what=""):
    """Within the bound and half a step of the stored type."""
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny * half
    got, want, bound = got.double().cpu(), want.cpu(), bound.cpu()
    off = (got - want).abs() - (bound + half * (want.abs() + bound) + tiny)
    assert torch.isfinite(got).all() and (off <= 0).all(), f"{what}: {(off > 0).sum()} of {off.numel()} outside"


def check_codes(codes, scales, want, bound, top, what=""):
    """int8 (top 127) or e4m3 (top 448) codes and row scales of want: the scale
    within its error, each code's value within half a step of the quotient."""
    want, bound = want.cpu(), bound.cpu()
    a = want.abs().amax(-1, keepdim=True)
    a_err = bound.amax(-1, keepdim=True)
    assert (a > 1e-20).all()
    s = scales.double().cpu().unsqueeze(-1)
    assert ((s - a / top).abs() <= a_err / top + 2 * U * a / top).all(), f"{what}: scales"
    q = want * top / a
    slack = top * (bound / a + want.abs() * a_err / (a * a)) * 1.01 + 4 * U * q.abs()
    v = (codes.to(torch.float64) if top == 127 else codes.view(torch.float8_e4m3fn).to(torch.float64)).cpu()
    half = torch.full_like(q, 0.5) if top == 127 else \
        torch.exp2(torch.floor(torch.log2((q.abs() + slack).clamp(min=2.0 ** -6))) - 4)
    off = (v - q).abs() - (half + slack)
    assert (off <= 0).all() and (v.abs() <= top).all(), f"{what}: {(off > 0).sum()} codes outside"
