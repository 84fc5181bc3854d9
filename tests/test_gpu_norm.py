"""The norms and gated residuals on the GPU against 64 bits, within the bounds
of norm_reference.py: every element type, widths from one element to rows too
long for registers, groups, odd pitches and starts, an updated stream in
place, and rows that are zero or not finite."""
from __future__ import annotations

import itertools

import pytest
import torch

from tests import norm_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w8a8_int8_dynamic_amd import _lib
    from w8a8_int8_dynamic_amd import ops as _ops
    assert _ops.device_supported(torch.cuda.current_device()), _lib.last_error()
    return _ops


def rows(m, k, seed, dtype=BF, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.where(torch.rand(k, generator=g) < 0.02, 12.0, 1.0)
    return ((x + mean) * 10.0 ** (torch.rand(m, 1, generator=g) * 2 - 1)).to(dtype).to(DEV)


def vec(k, seed, dtype, mean=0.0, groups=None, spread=0.3):
    g = torch.Generator().manual_seed(seed)
    return (mean + spread * torch.randn((k,) if groups is None else (groups, k), generator=g)).to(dtype).to(DEV)


def check_norm(ops, got, want, bound, dtype, kind, what):
    if kind == "same":
        ref.check_float(got, want, bound, dtype, what)
    else:
        assert got[0].dtype == (torch.int8 if kind == "int8" else torch.uint8) and got[1].dtype == F32
        ref.check_codes(*got, want, bound, 127 if kind == "int8" else 448, what)


def run_norm(ops, x, n, kind, **more):
    if kind == "same":
        return ops.norm(x, n, **more)
    return (ops.norm_quant_per_token if kind == "int8" else ops.fp8_norm_quant_per_token)(x, n)


WIDTHS = [1, 2, 7, 8, 9, 48, 63, 64, 65, 100, 511, 512, 513, 1000, 2048, 2056, 4096, 5001, 8192, 8200, 12288, 16400,
          33000]


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_widths(ops, kind, k):
    for m, dtype, out in ((1, BF, "same"), (5, HF, "int8"), (3, BF, "fp8"), (6, F32, "same"), (4, F32, "int8")):
        x = rows(m, k, 10 * k + m, dtype, mean=0.5)
        v = {"weight": vec(k, 1, dtype, 1.0), "bias": vec(k, 2, dtype) if m != 5 else None,
             "scale": vec(k, 3, F32), "shift": vec(k, 4, F32, 0.5)}
        n = ops.Norm(kind, eps=1e-5, **v)
        want, bound = ref.norm(x.double(), torch.zeros_like(x, dtype=torch.float64), kind, 1e-5, **v)
        check_norm(ops, run_norm(ops, x, n, out), want, bound, BF if dtype == F32 else dtype, out, f"{m} {dtype} {out}")


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("have", list(itertools.product([0, 1], repeat=4)))
def test_norm_vectors(ops, kind, have):
    """Each subset of weight, bias, scale and shift, in each type of vector."""
    m, k = 6, 264
    x = rows(m, k, 3)
    for vt, mt, groups in ((BF, F32, 2), (F32, HF, 3), (HF, BF, 6), (BF, BF, 1), (F32, F32, None)):
        v = {"weight": vec(k, 1, vt, 1.0), "bias": vec(k, 2, vt), "scale": vec(k, 3, mt, groups=groups),
             "shift": vec(k, 4, mt, groups=groups)}
        v = {a: t for (a, t), h in zip(v.items(), have) if h}
        want, bound = ref.norm(x.double(), torch.zeros(m, k, device=DEV, dtype=torch.float64), kind, 1e-6, **v)
        n = ops.Norm(kind, **v)
        for out in ("same", "int8", "fp8"):
            check_norm(ops, run_norm(ops, x, n, out), want, bound, BF, out, f"{vt} {mt} {groups} {out}")


def test_norm_many_rows_of_groups(ops):
    """Rows of several workgroups, groups that begin inside one, and modulation
    vectors that are columns of a wider tensor."""
    for m, k, groups in ((1029, 96, 3), (700, 520, 7), (2050, 64, 1025), (4099, 32, 1), (515, 4104, 5)):
        x = rows(m, k, m)
        both = vec(3 * k, 5, BF, groups=groups)
        v = {"scale": both[:, k:2 * k], "shift": both[:, 2 * k:]}
        want, bound = ref.norm(x.double(), torch.zeros(m, k, device=DEV, dtype=torch.float64), "layer", 1e-6, **v)
        for out in ("same", "int8", "fp8"):
            check_norm(ops, run_norm(ops, x, ops.Norm("layer", **v), out), want, bound, BF, out, f"{m} {k} {out}")


@pytest.mark.parametrize("dtype,stream", [(BF, BF), (HF, HF), (BF, F32), (HF, F32)])
@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("m,k", [(1, 64), (4, 4096), (6, 5001), (9, 100), (2, 16392), (3, 33001), (300, 72)])
def test_gated_residual(ops, dtype, stream, post, m, k):
    x, y = rows(m, k, 1, stream), rows(m, k, 2, dtype, mean=0.3)
    groups = 3 if m % 3 == 0 else None
    pn = None if post is None else {"kind": post, "eps": 1e-5, "weight": vec(k, 3, dtype, 1.0),
                                    "bias": vec(k, 4, dtype) if post == "layer" else None}
    for gate, scales in ((None, (1.0, 1.0)), (vec(k, 5, F32, groups=groups, spread=0.7), (0.9, 1.25)),
                         (vec(k, 6, dtype), (1.0, -0.5))):
        more = {"residual_scale": scales[0], "branch_scale": scales[1], "gate": gate}
        r, r_err = ref.residual(x, y, post=pn, **more)
        p = None if pn is None else ops.Norm(**pn)
        ref.check_float(ops.gated_residual(x, y, post=p, **more), r, r_err, stream, "r alone")
        for kind, out in (("rms", "same"), ("layer", "int8"), ("rms", "fp8")):
            v = {"scale": vec(k, 7, F32, groups=groups), "shift": vec(k, 8, F32, 0.5, groups=groups),
                 "weight": vec(k, 9, dtype, 1.0)}
            h, h_err = ref.norm(r, r_err, kind, 1e-6, **v)
            n = ops.Norm(kind, **v)
            if out == "same":
                got_r, got = ops.gated_residual_norm(x, y, n, post=p, **more)
                ref.check_float(got, h, h_err, dtype, "h")
            else:
                f = ops.gated_residual_norm_quant if out == "int8" else ops.fp8_gated_residual_norm_quant
                got_r, *got = f(x, y, n, post=p, **more)
                ref.check_codes(*got, h, h_err, 127 if out == "int8" else 448, "codes")
            ref.check_float(got_r, r, r_err, stream, "r")


@pytest.mark.parametrize("k", [96, 100, 4096, 33000])
def test_in_place_odd_rows_and_neighbours(ops, k):
    """r into x itself gives what r elsewhere gives; rows of odd pitch and start;
    what lies beside the outputs stays."""
    m = 5
    x, y = rows(m, k, 1), rows(m, k, 2)
    n, p = ops.Norm("layer", shift=vec(k, 3, F32)), ops.Norm("rms", weight=vec(k, 4, BF, 1.0))
    r, h = ops.gated_residual_norm(x, y, n, post=p, gate=vec(k, 5, BF))
    wx, wy = (torch.full((m, k + 7), 3.0, dtype=BF, device=DEV) for _ in range(2))
    wx[:, 3:3 + k], wy[:, 5:5 + k] = x, y
    r2, h2 = ops.gated_residual_norm(wx[:, 3:3 + k], wy[:, 5:5 + k], n, post=p, gate=vec(k, 5, BF),
                                     out=wx[:, 3:3 + k])
    assert r2.data_ptr() == wx[:, 3:].data_ptr() and torch.equal(r2, r) and torch.equal(h2, h)
    assert (wx[:, :3] == 3.0).all() and (wx[:, 3 + k:] == 3.0).all()
    x2 = x.clone()
    assert torch.equal(ops.gated_residual(x2, y, out=x2), ops.gated_residual(x, y))
    # vectors of odd start
    odd = torch.zeros(k + 1, dtype=BF, device=DEV)
    odd[1:] = vec(k, 4, BF, 1.0)
    assert torch.equal(ops.norm(x, ops.Norm("rms", weight=odd[1:])), ops.norm(x, p))


def test_fused_calls_agree(ops):
    """The norm in front and the norm behind a block are one arithmetic: with an
    fp32 stream that r fits exactly they agree bit for bit."""
    m, k = 37, 1000
    x, y = rows(m, k, 1).float(), torch.zeros(m, k, dtype=BF, device=DEV)
    n = ops.Norm("layer", weight=vec(k, 3, BF, 1.0), scale=vec(k, 4, F32), shift=vec(k, 5, F32))
    r, h = ops.gated_residual_norm(x, y, n)
    assert torch.equal(r, x) and torch.equal(h, ops.norm(x, n))
    _, q, s = ops.gated_residual_norm_quant(x, y, n)
    q2, s2 = ops.norm_quant_per_token(x, n)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("k", [96, 4096, 33000])
def test_zero_and_not_finite_rows(ops, k):
    """A row of zeros gives zeros (scale 0); one with NaN or an infinity is not
    finite and leaves its neighbours alone."""
    x = rows(4, k, 1)
    x[1] = 0
    good = ops.norm(x, ops.Norm("rms")).clone()
    assert (good[1] == 0).all()
    x[2, 5], x[3, k - 1] = float("nan"), float("inf")
    for kind in ("rms", "layer"):
        n = ops.Norm(kind)
        h = ops.norm(x, n)
        assert torch.isnan(h[2]).any() and not torch.isfinite(h[3]).all() and torch.isfinite(h[:2]).all()
        for f in (ops.norm_quant_per_token, ops.fp8_norm_quant_per_token):
            q, s = f(x, n)
            assert s[1] == 0 and (q[1] == 0).all() and torch.isfinite(s[:2]).all()
            assert not torch.isfinite(s[2]) and not torch.isfinite(s[3])
        r, q, s = ops.gated_residual_norm_quant(x, torch.zeros_like(x), n)
        assert torch.equal(r[:3], x[:3]) or torch.isnan(r[2, 5]) and not torch.isfinite(s[2:]).any()
    # one constant row under a layer norm with eps: zeros
    c = torch.full((2, k), 3.0, dtype=BF, device=DEV)
    assert (ops.norm(c, ops.Norm("layer")) == 0).all()


def test_empty(ops):
    x = torch.zeros(0, 64, dtype=BF, device=DEV)
    n = ops.Norm("rms", scale=vec(64, 1, F32))
    assert ops.norm(x, n).shape == (0, 64)
    q, s = ops.norm_quant_per_token(x, n)
    assert q.shape == (0, 64) and s.shape == (0,)
    assert [t.shape[0] for t in ops.gated_residual_norm_quant(x, x, n)] == [0, 0, 0]


def test_repeats_are_equal(ops):
    """No result depends on scheduling."""
    x, y = rows(700, 4104, 1), rows(700, 4104, 2)
    n, p = ops.Norm("layer", shift=vec(4104, 3, F32)), ops.Norm("rms")
    first = ops.gated_residual_norm_quant(x, y, n, post=p)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, ops.gated_residual_norm_quant(x, y, n, post=p)))


def test_refusals(ops):
    x, y = rows(6, 64, 1), rows(6, 64, 2)
    bad = [lambda: ops.norm(x, ops.Norm("batch")), lambda: ops.norm(x, ops.Norm(weight=vec(63, 1, BF))),
           lambda: ops.norm(x, ops.Norm(weight=vec(64, 1, BF, groups=2))),
           lambda: ops.norm(x, ops.Norm(scale=vec(64, 1, BF, groups=4))),
           lambda: ops.norm(x, ops.Norm(scale=vec(64, 1, BF, groups=2), shift=vec(64, 1, BF, groups=3))),
           lambda: ops.norm(x, ops.Norm(shift=vec(128, 1, BF)[::2])), lambda: ops.norm(x.t(), ops.Norm()),
           lambda: ops.norm(x, ops.Norm(weight=vec(64, 1, BF).cpu())),
           lambda: ops.gated_residual(x, y[:5]), lambda: ops.gated_residual(x, y, gate=vec(64, 1, BF, groups=4)),
           lambda: ops.gated_residual(x, y, post=ops.Norm(scale=vec(64, 1, BF))),
           lambda: ops.gated_residual(x, y, out=x[:3])]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    wrong = [lambda: ops.norm(x, ops.Norm(), out_dtype=HF), lambda: ops.norm(x.double(), ops.Norm()),
             lambda: ops.norm(x, ops.Norm(weight=vec(64, 1, BF), bias=vec(64, 1, F32))),
             lambda: ops.norm(x, ops.Norm(scale=vec(64, 1, BF), shift=vec(64, 1, F32))),
             lambda: ops.gated_residual(x.half(), y), lambda: ops.gated_residual(x, y.float())]
    for f in wrong:
        with pytest.raises(TypeError):
            f()
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(ops._lib.W8A8Error):
            ops.norm(x, ops.Norm(eps=eps))


def test_other_stream_and_graph(ops):
    m, k = 24, 4096
    n, p = ops.Norm("rms", scale=vec(k, 3, F32, groups=2), shift=vec(k, 4, F32, groups=2)), ops.Norm("layer")
    xs, y = [rows(m, k, 20 + i) for i in range(3)], rows(m, k, 2)
    call = lambda x: ops.gated_residual_norm_quant(x, y, n, post=p)  # noqa: E731
    want = [[t.clone() for t in call(x)] for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    static = xs[0].clone()
    with torch.cuda.stream(side):
        assert all(torch.equal(a, b) for a, b in zip(call(static), want[0]))
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = call(static)
    torch.cuda.synchronize()
    for i in (0, 1, 2, 1):
        static.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(call(xs[i]), want[i]))


@pytest.mark.parametrize("m,k", [(515, 4096), (600, 3000), (520, 8192), (513, 6000), (1100, 12288), (2050, 2048),
                                 (1030, 1500), (300, 16384), (1025, 16000)])
def test_many_wide_rows(ops, m, k):
    """Runs of several rows per workgroup in every row shape, whole and ragged,
    with groups that end inside a run."""
    groups = 5 if m % 5 == 0 else None
    x, y = rows(m, k, m), rows(m, k, m + 1)
    v = {"scale": vec(k, 3, F32, groups=groups), "shift": vec(k, 4, F32, 0.5, groups=groups)}
    z = torch.zeros(m, k, device=DEV, dtype=torch.float64)
    for kind in ("rms", "layer"):
        want, bound = ref.norm(x.double(), z, kind, 1e-6, **v)
        n = ops.Norm(kind, **v)
        for out in ("same", "int8", "fp8"):
            check_norm(ops, run_norm(ops, x, n, out), want, bound, BF, out, f"{kind} {out}")
    post = {"kind": "rms", "eps": 1e-6, "weight": vec(k, 6, BF, 1.0)}
    gate = vec(k, 5, BF, groups=groups, spread=0.7)
    r, err = ref.residual(x, y, gate=gate, post=post)
    h, h_err = ref.norm(r, err, "layer", 1e-6, **v)
    got_r, got_h = ops.gated_residual_norm(x, y, ops.Norm("layer", **v), gate=gate, post=ops.Norm(**post))
    ref.check_float(got_r, r, err, BF, "r")
    ref.check_float(got_h, h, h_err, BF, "h")
    assert torch.equal(ops.gated_residual(x, y, gate=gate, post=ops.Norm(**post)), got_r)


@pytest.mark.parametrize("m,k", [(6, 1536), (7, 1200), (5, 2500), (3, 5120), (7, 5001), (4, 6144), (9, 5200),
                                 (515, 5120), (700, 5001), (520, 1536), (514, 9001), (515, 10240), (2, 16001),
                                 (514, 12296), (3, 16384), (1024, 12296), (1025, 12296), (1030, 16384)])
def test_thread_counts(ops, m, k):
    """The row shapes in between, whole and ragged, few rows and many; the
    residual in place of the stream."""
    x, y = rows(m, k, m), rows(m, k, m + 1)
    v = {"scale": vec(k, 3, F32), "shift": vec(k, 4, F32, 0.5)}
    z = torch.zeros(m, k, device=DEV, dtype=torch.float64)
    for kind in ("rms", "layer"):
        want, bound = ref.norm(x.double(), z, kind, 1e-6, **v)
        for out in ("same", "int8", "fp8"):
            check_norm(ops, run_norm(ops, x, ops.Norm(kind, **v), out), want, bound, BF, out, f"{kind} {out}")
    post = {"kind": "layer", "eps": 1e-6, "weight": vec(k, 6, BF, 1.0)}
    for stream in (BF, F32):
        xs = x.to(stream)
        r, err = ref.residual(xs, y, post=post)
        h, h_err = ref.norm(r, err, "rms", 1e-6, **v)
        got_r, got_h = ops.gated_residual_norm(xs, y, ops.Norm("rms", **v), post=ops.Norm(**post))
        ref.check_float(got_r, r, err, stream, "r")
        ref.check_float(got_h, h, h_err, BF, "h")
        again, *codes = ops.gated_residual_norm_quant(xs, y, ops.Norm("rms", **v), post=ops.Norm(**post))
        ref.check_codes(*codes, h, h_err, 127, "codes")
        assert torch.equal(again, got_r)
        assert torch.equal(ops.gated_residual(xs, y, post=ops.Norm(**post), out=xs), got_r)


@pytest.mark.parametrize("k", [104, 33000])
def test_offsets_past_32_bits(ops, k):
    """Rows, modulation vectors and outputs billions of elements apart."""
    m, pitch = 5, (1 << 30) + 7
    big = torch.empty(m * pitch, dtype=BF, device=DEV)
    x, y = rows(m, k, 1), rows(m, k, 2)
    at = lambda i: big.as_strided((m, k), (pitch, 1), i * 40000)  # noqa: E731
    wx, wy, mod, out = (at(i) for i in range(4))
    wx.copy_(x)
    wy.copy_(y)
    mod.copy_(vec(k, 3, BF, groups=m))
    n = ops.Norm("layer", scale=mod, shift=mod)
    small = ops.Norm("layer", scale=mod.contiguous(), shift=mod.contiguous())
    assert torch.equal(ops.norm(wx, n), ops.norm(x, small))
    got = ops.gated_residual_norm_quant(wx, wy, n, gate=mod, out=out)
    want = ops.gated_residual_norm_quant(x, y, small, gate=mod.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_one_vector_each(ops):
    """As many groups as rows, and a gate that is one row for all."""
    m, k = 40, 520
    x, y = rows(m, k, 1, F32), rows(m, k, 2)
    v = {"scale": vec(k, 3, HF, groups=m), "shift": vec(k, 4, HF, 0.3, groups=m)}
    gate = vec(k, 5, F32, groups=1)
    r, err = ref.residual(x, y, gate=gate, residual_scale=0.5)
    h, h_err = ref.norm(r, err, "rms", 1e-6, **v)
    got_r, *codes = ops.gated_residual_norm_quant(x, y, ops.Norm("rms", **v), gate=gate, residual_scale=0.5)
    ref.check_float(got_r, r, err, F32, "r")
    ref.check_codes(*codes, h, h_err, 127, "codes")


@pytest.mark.parametrize("k", [1, 7, 8, 96, 1000, 4096, 12296, 16384, 33000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_mean_squares_below_the_normal_range(ops, dtype, k):
    """eps = 0 and rows of 2^-66 .. 2^-63, whose squares and their mean are fp32
    subnormals: norms of about one, whichever kernel the width picks.
    On top of the reference's bound: each of the K squares, and the mean, is
    rounded to a multiple of 2^-149, so the mean is off by at most 2^-150 for
    the squares and 2^-150 for itself; half of that, relative to the mean
    square, is the deviation's error and so the norm's (taken twice here)."""
    g = torch.Generator().manual_seed(k)
    sign = torch.where(torch.rand(4, k, generator=g) < 0.5, -1.0, 1.0)
    x = (sign * (1 + torch.rand(4, k, generator=g)) * 2.0 ** torch.tensor([[-66.0], [-65], [-64], [-64]]))
    x = x.to(dtype).to(DEV)
    z = torch.zeros(4, k, device=DEV, dtype=torch.float64)
    for kind in ("rms", "layer") if k > 1 else ("rms",):
        v = x.double()
        d = v - v.mean(-1, keepdim=True) if kind == "layer" else v
        low = 2.0 ** -149 / (d * d).mean(-1, keepdim=True)
        if kind == "layer":
            assert (low < 2.0 ** -8).all(), "rows of one value have no norm"
        want, bound = ref.norm(v, z, kind, 0.0)
        bound = bound + want.abs() * low
        n = ops.Norm(kind, eps=0.0)
        ref.check_float(ops.norm(x, n), want, bound, BF, kind)
        ref.check_codes(*ops.norm_quant_per_token(x, n), want, bound, 127, kind)
        ref.check_codes(*ops.fp8_norm_quant_per_token(x, n), want, bound, 448, kind)
        # the same rows as a branch whose norm goes into the stream
        y = x.bfloat16()
        p, err = ref.norm(y.double(), z, kind, 0.0)
        err = err + p.abs() * low * 1.1              # (y's mean square is x's but for its rounding to bf16)
        ref.check_float(ops.gated_residual(torch.ones_like(y), y, post=n), 1 + p, err + 2 * ref.U * (1 + p.abs()), BF,
                        "branch")


def test_no_rows_and_a_vector_for_each(ops):
    """A batch of no tokens whose modulation and gate come per token: [0, K]."""
    k = 64
    x, v = torch.zeros(0, k, dtype=BF, device=DEV), torch.zeros(0, k, device=DEV)
    n = ops.Norm("layer", scale=v, shift=v)
    assert ops.norm(x, n).shape == (0, k)
    q, s = ops.norm_quant_per_token(x, n)
    assert q.shape == (0, k) and s.shape == (0,)
    r, h = ops.gated_residual_norm(x, x, n, gate=v)
    assert r.shape == h.shape == (0, k)
    assert ops.gated_residual(x, x, gate=v).shape == (0, k)
    with pytest.raises(ValueError, match="rows"):
        ops.norm(torch.zeros(3, k, dtype=BF, device=DEV), n)
    with pytest.raises(ValueError):
        ops.norm(x, ops.Norm(scale=torch.zeros(0, k + 1, device=DEV)))


@pytest.mark.parametrize("k", [96, 100, 4096, 33000])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_beside_one_that_is_not_finite(ops, kind, k):
    """NaN and infinities stay in their rows: the others' results are, bit for
    bit, those of a call without them, of each entry point."""
    m = 9
    clean, y = rows(m, k, 1), rows(m, k, 2)
    x, yx = clean.clone(), y.clone()
    x[2, 5], x[4, k - 1], x[7, 0] = float("nan"), float("inf"), float("-inf")
    yx[5, k // 2] = float("nan")
    good, n, p = [0, 1, 3, 6, 8], ops.Norm(kind, scale=vec(k, 3, F32)), ops.Norm(kind)
    calls = [lambda a, b: (ops.norm(a, n),), lambda a, b: ops.norm_quant_per_token(a, n),
             lambda a, b: ops.fp8_norm_quant_per_token(a, n), lambda a, b: (ops.gated_residual(a, b, post=p),),
             lambda a, b: ops.gated_residual_norm(a, b, n, post=p), lambda a, b: ops.gated_residual_norm(a, b, n),
             lambda a, b: ops.gated_residual_norm_quant(a, b, n, post=p),
             lambda a, b: ops.fp8_gated_residual_norm_quant(a, b, n)]
    for i, f in enumerate(calls):
        for u, v in zip(f(x, yx), f(clean, y)):
            assert torch.equal(u[good], v[good]), i
    r, h = ops.gated_residual_norm(x, yx, n, post=p)
    assert all(not torch.isfinite(t[j]).all() for t in (r, h) for j in (2, 4, 5, 7))
    assert not torch.isfinite(ops.gated_residual_norm_quant(x, yx, n, post=p)[2][[2, 4, 5, 7]]).any()
