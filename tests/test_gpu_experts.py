"""Routing and the mixture of experts on the GPU against their definitions in 64 bits.

Ids are exact (scores, sums and choices are 64-bit on both sides, and random
logits give no two choices within their last bits but equal ones). Weights: one
rounding to fp32 of a 64-bit value, 2^-24 relative, and half the smallest
subnormal. Outputs keep the bound that tests/block_reference.py derives (where an
inner row's element lies so near a border between two codes that the products'
bound may move it across, that includes the codes' distance), and half a step of
the output's type."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import block_reference as ref
from tests.test_gpu_fp8_block import DEV, HALF, TINY, check, codes, dev, rows, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w8a8_int8_dynamic_amd import _lib
    from w8a8_int8_dynamic_amd import ops as _ops
    assert _ops.device_supported(torch.cuda.current_device()), _lib.last_error()
    return _ops


def same_route(ops, logits, what="", **how):
    bias = how.pop("bias", None)
    got_ids, got_w = ops.route_experts(logits.to(DEV), ops.Routing(bias=None if bias is None else bias.to(DEV), **how))
    ids, w = ref.route(logits.float().numpy(), bias=None if bias is None else bias.numpy(), **how)
    assert got_ids.dtype == torch.int32 and got_w.dtype == torch.float32
    assert np.array_equal(got_ids.cpu().numpy(), ids), what
    off = np.abs(got_w.double().cpu().numpy() - w)
    assert (off <= 2.0 ** -23 * np.abs(w) + 2.0 ** -149).all(), what


def logits_of(t, e, seed, dtype=torch.float32):
    return (2 * torch.randn(t, e, generator=torch.Generator().manual_seed(seed))).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 256, 8), (5, 8, 8), (33, 60, 6), (7, 64, 64), (9, 65, 3),
                                   (2, 1024, 16),
                                   (130, 160, 6)])
def test_route(ops, dtype, score, t, e, k):
    """Sixteen-bit logits have many equal ones in a row: ties go to the lowest index."""
    x = logits_of(t, e, t + e, dtype)
    bias = 0.1 * torch.randn(e, generator=torch.Generator().manual_seed(1))
    for b in (None, bias):
        for renormalize in (True, False):
            same_route(ops, x, f"{t} {e} {b is None}", top_k=k, score=score, bias=b, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("groups,top_groups,e", [(8, 4, 256), (2, 1, 16), (64, 3, 128), (4, 4, 60), (3, 2, 99),
                                                 (8, 1, 8)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_groups(ops, groups, top_groups, e, group_top):
    bias = 0.1 * torch.randn(e, generator=torch.Generator().manual_seed(1))
    k = min(6, e // groups * top_groups)
    for dtype in (torch.float32, torch.bfloat16):
        for score in ("softmax", "sigmoid"):
            for b in (None, bias):
                same_route(ops, logits_of(40, e, e, dtype), top_k=k, score=score, bias=b, groups=groups,
                           top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masks(ops, score, groups):
    """Rows whose mask leaves nothing, one or two experts, a group's worth; -infinity, NaN, the
    type's lowest value, +infinity; a bias that excludes."""
    e, inf = 32, float("inf")
    x = logits_of(12, e, 5)
    x[0] = -inf
    x[1] = float("nan")
    x[2] = -inf
    x[2, 17] = 0.3
    x[3, 1:31] = float("nan")
    x[4, 8:] = -inf
    x[5] = torch.finfo(torch.float32).min
    x[6] = torch.finfo(torch.float32).min
    x[6, 9] = 1.0
    x[7, [3, 30]] = inf
    x[8] = inf
    x[9] = 0.0
    x[10] = -200.0                                        # sigmoid: scores near e^-200
    x[10, 4] = -90.0
    x[11, ::2] = -inf
    bias = 0.1 * torch.randn(e, generator=torch.Generator().manual_seed(1))
    hard = bias.clone()
    hard[5], hard[6] = -inf, float("nan")
    for b in (None, bias, hard):
        for renormalize in (True, False):
            same_route(ops, x, f"{score} {groups} {b is None} {renormalize}", top_k=5, score=score, bias=b,
                       groups=groups, top_groups=max(1, groups - 1), renormalize=renormalize)


def test_route_strides_streams_and_graph(ops):
    wide = logits_of(50, 100, 3)
    how = ops.Routing(4, "sigmoid", renormalize=False)
    ids, w = ref.route(wide[::2, 10:70].numpy(), 4, "sigmoid", renormalize=False)
    x = wide.to(DEV)[::2, 10:70]
    got = ops.route_experts(x, how)
    assert np.array_equal(got[0].cpu().numpy(), ids)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    buf = x.contiguous()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = ops.route_experts(buf, how)
    for i in range(3):
        y = logits_of(25, 60, 40 + i).to(DEV)
        buf.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want = ops.route_experts(y, how)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    ids, w = ops.route_experts(x[:0], how)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def make(e, inner, k, seed):
    """Experts' weights as codes and scales, and dequantized."""
    gu, gs, dn, ds, gv, dv = [], [], [], [], [], []
    for i in range(e):
        gate, up, down = (weights(*s, seed + 10 * i + j) for j, s in enumerate(((inner, k), (inner, k), (k, inner))))
        gu.append(np.concatenate((gate[0], up[0])))
        gs.append(np.concatenate((gate[1], up[1])))
        dn.append(down[0])
        ds.append(down[1])
        gv.append(np.concatenate((ref.weight(*gate), ref.weight(*up))))
        dv.append(ref.weight(*down))
    return [np.stack(a) for a in (gu, gs, dn, ds)], gv, dv


def layer_of(parts, routing=None):
    from w8a8_int8_dynamic_amd import W8A8Experts
    return W8A8Experts.from_quantized(*(dev(p) for p in parts), routing=routing)


def choose(t, e, k, seed, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, e, generator=g) + skew * torch.randn(e, generator=g)
    v, i = x.topk(k, -1)
    return i.to(torch.int32), torch.softmax(v, -1)


CASES = [(1, 4, 1, 16, 16), (1, 8, 3, 272, 144), (5, 3, 2, 128, 128), (40, 6, 2, 400, 272), (150, 4, 3, 144, 80),
         (333, 5, 2, 528, 208), (64, 64, 4, 256, 128), (600, 2, 1, 160, 400), (700, 3, 2, 272, 144)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,e,top_k,k,inner", CASES)
def test_experts(ops, dtype, t, e, top_k, k, inner):
    parts, gv, dv = make(e, inner, k, t)
    layer = layer_of(parts)
    x = (rows(t, k, t + 1, torch.float32) * 0.3).to(dtype)
    ids, w = choose(t, e, top_k, 3, skew=1.0)
    xv = ref.dequant(*ref.quant(x.float().numpy()))
    exact, bound = ref.experts(xv, ids.numpy(), w.numpy(), gv, dv)
    y = layer(x.to(DEV), ids.to(DEV), w.to(DEV))
    assert y.dtype == dtype
    check(y, exact, bound, dtype, what=f"{t} {e}")
    # Over many elements the error's norm is far below the bound's. The instruction's error is 2^-16 of the
    # sums' rms as measured, 2^-13 with a margin of 8; of the inner elements, whose codes lie 2^-4 of their
    # value apart or more, such an error takes less than 2^-13 * 4 / 2^-4 = 2^-7 across a border, each by
    # 2^-3 at most: 2^-3 * 2^-3.5 = 2^-6.5 of the norm, and the output's half step.
    if t * inner >= 10000:
        off = np.linalg.norm(y.double().cpu().numpy() - exact) / np.linalg.norm(exact)
        assert off < 2.0 ** -6.5 + HALF[dtype], off
    assert torch.equal(layer(x.to(DEV), ids.to(DEV), w.to(DEV)), y)


@pytest.mark.parametrize("t,e,top_k,k,inner", [(48, 2, 1, 16, 16), (45, 3, 1, 128, 128), (90, 5, 2, 528, 208),
                                               (60, 4, 2, 640, 1040), (50, 2, 1, 1168, 144), (100, 8, 4, 272, 528),
                                               (64, 4, 1, 8208, 32), (30, 1, 1, 1040, 272), (130, 7, 2, 2064, 720)])
def test_experts_of_a_few_dozen_rows(ops, t, e, top_k, k, inner):
    parts, gv, dv = make(e, inner, k, t + 1)
    layer = layer_of(parts)
    for skew in (0.0, 1.5):
        x = (rows(t, k, t + 1, torch.float32) * 0.3).to(torch.bfloat16)
        ids, w = choose(t, e, top_k, 3, skew=skew)
        exact, bound = ref.experts(ref.dequant(*ref.quant(x.float().numpy())), ids.numpy(), w.numpy(), gv, dv)
        y = layer(x.to(DEV), ids.to(DEV), w.to(DEV))
        check(y, exact, bound, torch.bfloat16, what=f"{t} {e} {skew}")
        assert torch.equal(layer(x.to(DEV), ids.to(DEV), w.to(DEV)), y)


@pytest.mark.parametrize("t,e,top_k,k,inner", [(1200, 36, 6, 784, 784), (1000, 32, 3, 784, 912),
                                               (1500, 64, 2, 1040, 784)])
def test_experts_many_tiles(ops, t, e, top_k, k, inner):
    """About 200, 94 and 47 rows an expert, of uneven shares, in more tiles than the card holds at once."""
    parts, gv, dv = make(e, inner, k, t)
    layer = layer_of(parts)
    x = (rows(t, k, t + 1, torch.float32) * 0.3).to(torch.bfloat16)
    ids, w = choose(t, e, top_k, 5, skew=0.5)
    xv = ref.dequant(*ref.quant(x.float().numpy()))
    exact, bound = ref.experts(xv, ids.numpy(), w.numpy(), gv, dv)
    y = layer(x.to(DEV), ids.to(DEV), w.to(DEV))
    check(y, exact, bound, torch.bfloat16, what=f"{t} {e}")
    off = np.linalg.norm(y.double().cpu().numpy() - exact) / np.linalg.norm(exact)
    assert off < 2.0 ** -6.5 + HALF[torch.bfloat16], off          # (as in test_experts)
    assert torch.equal(layer(x.to(DEV), ids.to(DEV), w.to(DEV)), y)


@pytest.mark.parametrize("t", [6, 200])
def test_experts_any_ids(ops, t):
    """No expert (-1, or past the last), all slots one expert, the same expert twice, an order
    without any meaning; a token without experts is zero; fp32 rows."""
    e, top_k, k, inner = 5, 4, 272, 144
    parts, gv, dv = make(e, inner, k, 7)
    layer = layer_of(parts)
    x = (rows(t, k, 2, torch.float32) * 0.3).to(torch.bfloat16)
    xv = ref.dequant(*ref.quant(x.float().numpy()))
    r = np.random.default_rng(4)
    w = r.uniform(-1, 1, (t, top_k)).astype(np.float32)
    free = r.integers(-1, e + 1, (t, top_k)).astype(np.int32)
    free[1] = -1
    free[2] = [3, 3, 3, 0]
    free[3] = [2 ** 31 - 1, -2 ** 31, e, 1]
    for ids in (free, np.full((t, top_k), 2, np.int32), np.full((t, top_k), -1, np.int32)):
        exact, bound = ref.experts(xv, ids, w, gv, dv)
        y = layer(x.to(DEV), dev(ids), dev(w))
        check(y, exact, bound, torch.bfloat16)
        none = ((ids < 0) | (ids >= e)).all(1)
        assert (y.cpu()[torch.from_numpy(none)] == 0).all()
        f = ops.fp8_block_experts(x.float().to(DEV), dev(ids), dev(w), layer.gate_up, layer.gate_up_scale, layer.down,
                                  layer.down_scale, inner)
        assert f.dtype == torch.float32
        check(f, exact, bound, torch.float32)
        assert torch.equal(f.bfloat16(), y)


@pytest.mark.parametrize("t", [1, 20, 60, 500])
def test_experts_large_values(ops, t):
    """Inner rows up to about 1e36 and sums of scales past 2^103: results in fp32's range are there."""
    e, top_k, k, inner = 4, 2, 272, 144
    parts, gv, dv = make(e, inner, k, 15)
    layer = layer_of(parts)
    x = rows(t, k, 2, torch.float32).clamp(-4, 4) * 2.0 ** 58
    ids, w = choose(t, e, top_k, 5)
    exact, bound = ref.experts(ref.dequant(*ref.quant(x.numpy())), ids.numpy(), w.numpy(), gv, dv)
    assert np.abs(exact).max() < 2.0 ** 126
    y = ops.fp8_block_experts(x.to(DEV), ids.to(DEV), w.to(DEV), layer.gate_up, layer.gate_up_scale, layer.down,
                              layer.down_scale, inner)
    check(y, exact, bound, torch.float32)


@pytest.mark.parametrize("t", [3, 5000])
def test_experts_many_experts_and_choices(ops, t):
    """1024 experts of one block each way; 64 choices a token."""
    for e, top_k, k, inner in ((1024, 6, 128, 16), (70, 64, 144, 32)):
        t1 = min(t, 300) if top_k == 64 else t
        parts, gv, dv = make(e, inner, k, 17)
        layer = layer_of(parts)
        x = (rows(t1, k, t, torch.float32) * 0.3).to(torch.bfloat16)
        ids, w = choose(t1, e, top_k, 5)
        exact, bound = ref.experts(ref.dequant(*ref.quant(x.float().numpy())), ids.numpy(), w.numpy(), gv, dv)
        check(layer(x.to(DEV), ids.to(DEV), w.to(DEV)), exact, bound, torch.bfloat16, what=f"{e} experts")


def test_experts_passes(ops):
    """More than 65536 slots go in passes: the tokens of each have the values of a call that is
    one pass."""
    e, top_k, k, inner, t = 24, 4, 144, 48, 20000
    parts, _, _ = make(e, inner, k, 19)
    layer = layer_of(parts)
    x = (rows(t, k, 2, torch.float32) * 0.3).to(torch.bfloat16).to(DEV)
    ids, w = (v.to(DEV) for v in choose(t, e, top_k, 5))
    y, one = layer(x, ids, w), 65536 // top_k
    assert torch.equal(y[:one], layer(x[:one], ids[:one], w[:one]))
    assert torch.equal(y[t - one:], layer(x[t - one:], ids[t - one:], w[t - one:]))


@pytest.mark.parametrize("t", [1, 300, 5000])
def test_experts_weights_past_32_bits(ops, t):
    """The last of experts whose weights end past 4 GiB, by three paths."""
    e, k, inner = 264, 4096, 2048
    g, u, dn = (weights(*s, 23 + j) for j, s in enumerate(((inner, k), (inner, k), (k, inner))))
    gate_up = torch.zeros(e, 2 * inner, k, dtype=torch.uint8, device=DEV)
    gate_up[-1] = dev(np.concatenate((g[0], u[0])))
    down = torch.zeros(e, k, inner, dtype=torch.uint8, device=DEV)
    down[-1] = dev(dn[0])
    gs = torch.zeros(e, 2 * inner // 128, k // 128, device=DEV)
    gs[-1] = dev(np.concatenate((g[1], u[1])))
    ds = torch.zeros(e, k // 128, inner // 128, device=DEV)
    ds[-1] = dev(dn[1])
    from w8a8_int8_dynamic_amd import W8A8Experts
    layer = W8A8Experts.from_quantized(gate_up, gs, down, ds)
    assert layer.gate_up.numel() > 2 ** 32
    x = (rows(t, k, 2, torch.float32) * 0.1).to(torch.bfloat16)
    ids, w = torch.full((t, 1), e - 1, dtype=torch.int32), torch.ones(t, 1)
    y = layer(x.to(DEV), ids.to(DEV), w.to(DEV))
    some = [0, t // 2, t - 1]
    exact, bound = ref.experts(ref.dequant(*ref.quant(x[some].float().numpy())), np.zeros((3, 1), np.int32),
                               np.ones((3, 1), np.float32), [np.concatenate((ref.weight(*g), ref.weight(*u)))],
                               [ref.weight(*dn)])
    check(y[some], exact, bound, torch.bfloat16)


def test_rows_past_32_bits(ops):
    """Rows of logits, inputs and outputs 2 GiB apart."""
    far, t, e, top_k, k, inner = 2 ** 30, 5, 60, 3, 144, 48
    big = torch.empty(far * (t - 1) + 1024, dtype=torch.bfloat16, device=DEV)
    logits = logits_of(t, e, 1, torch.bfloat16)
    view = big.as_strided((t, e), (far, 1))
    view.copy_(logits)
    how = ops.Routing(top_k, score="sigmoid")
    want, got = ops.route_experts(logits.to(DEV), how), ops.route_experts(view, how)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    parts, _, _ = make(4, inner, k, 21)
    layer = layer_of(parts)
    x = (rows(t, k, 2, torch.float32) * 0.3).to(torch.bfloat16).to(DEV)
    view, out = big.as_strided((t, k), (far, 1)), big.as_strided((t, k), (far, 1), 512)
    view.copy_(x)
    for n, reps in ((t, 1), (t, 40)):
        ids, w = (v.to(DEV) for v in choose(t * reps, 4, 2, 5))
        ids, w = ids[:n], w[:n]
        args = (layer.gate_up, layer.gate_up_scale, layer.down, layer.down_scale, inner)
        ops.fp8_block_experts(view, ids, w, *args, out=out)
        assert torch.equal(out, ops.fp8_block_experts(x, ids, w, *args))


def test_experts_on_two_streams_at_once(ops):
    e, top_k, k, inner = 6, 2, 272, 144
    parts, _, _ = make(e, inner, k, 25)
    layer = layer_of(parts)
    streams, sets = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for n, t in enumerate((7, 400)):
        x = (rows(t, k, n, torch.float32) * 0.3).to(torch.bfloat16).to(DEV)
        ids, w = (v.to(DEV) for v in choose(t, e, top_k, n))
        sets.append((x, ids, w, layer(x, ids, w)))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n].append(layer(*sets[n][:3]))
    torch.cuda.synchronize()
    for n in range(2):
        assert all(torch.equal(y, sets[n][3]) for y in got[n])


def test_experts_rows_are_their_own(ops):
    """A token's result does not depend on the tokens beside it nor on which of them share its
    experts (within one path), and a token that is not finite harms no other."""
    e, top_k, k, inner, t = 4, 2, 272, 144, 300
    parts, _, _ = make(e, inner, k, 9)
    layer = layer_of(parts)
    x = (rows(t, k, 2, torch.float32) * 0.3).to(torch.bfloat16).to(DEV)
    ids, w = (v.to(DEV) for v in choose(t, e, top_k, 5))
    want = layer(x, ids, w)
    perm = torch.randperm(t, generator=torch.Generator().manual_seed(3)).to(DEV)
    assert torch.equal(layer(x[perm], ids[perm], w[perm]), want[perm])
    bad = x.clone()
    bad[17, 3] = float("nan")
    bad[150, 200] = float("inf")
    got = layer(bad, ids, w)
    others = [i for i in range(t) if i not in (17, 150)]
    assert torch.equal(got[others], want[others])
    assert got[17].isnan().all() and not got[150].isfinite().all()
    w2 = w.clone()
    w2[9] = float("nan")
    got = layer(x, ids, w2)
    assert got[9].isnan().all() and torch.equal(got[10:], want[10:]) and torch.equal(got[:9], want[:9])


def test_experts_strides_and_shapes(ops):
    e, top_k, k, inner, t = 3, 2, 160, 80, 24
    parts, _, _ = make(e, inner, k, 11)
    layer = layer_of(parts)
    x = (rows(t, k, 2, torch.float32) * 0.3).to(torch.bfloat16).to(DEV)
    ids, w = (v.to(DEV) for v in choose(t, e, top_k, 5))
    want = layer(x, ids, w)
    wide = torch.full((t, k + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    for at in (8, 5):
        wide[:, at:at + k] = x
        assert torch.equal(layer(wide[:, at:at + k], ids, w), want)
    assert torch.equal(layer(x, ids.t().contiguous().t(), w.t().contiguous().t()), want)
    got = layer(x.reshape(2, 3, 4, k), ids.reshape(2, 3, 4, 2), w.reshape(2, 3, 4, 2))
    assert torch.equal(got, want.reshape(2, 3, 4, k))
    for at in (8, 3):
        out = torch.full((t, k + 24), 7.0, dtype=torch.bfloat16, device=DEV)
        ops.fp8_block_experts(x, ids, w, layer.gate_up, layer.gate_up_scale, layer.down, layer.down_scale, inner,
                              out=out[:, at:at + k])
        assert torch.equal(out[:, at:at + k], want) and (out[:, :at] == 7).all() and (out[:, at + k:] == 7).all()
    assert layer(x[:0], ids[:0], w[:0]).shape == (0, k)


@pytest.mark.parametrize("t", [1, 5, 30, 400])
def test_together(ops, t):
    """A router, its experts and the residual stream as they run in a block: eager, on two streams at
    once, and captured and replayed with other tokens."""
    from w8a8_int8_dynamic_amd import W8A8Linear
    e, top_k, k, inner = 16, 4, 256, 144
    parts, gv, dv = make(e, inner, k, 13)
    g = torch.Generator().manual_seed(8)
    routing = ops.Routing(top_k, "sigmoid", bias=(0.1 * torch.randn(e, generator=g)).to(DEV), groups=4, top_groups=2,
                          scale=1.5)
    layer = layer_of(parts, routing)
    gate = (0.2 * torch.randn(e, k, generator=g)).to(DEV)
    shared = W8A8Linear.from_float((0.05 * torch.randn(k, k, generator=g)).to(DEV), scheme="fp8_block")
    norm = ops.Norm("rms")

    def block(x):
        h = ops.norm(x, norm)
        y = layer.forward_logits(h, h.float() @ gate.t()) + shared(h)
        return ops.gated_residual(x, y)

    xs = [rows(t, k, 30 + i).to(DEV) for i in range(4)]
    want = [block(x).clone() for x in xs]
    # the routed part by its definition
    h = ops.norm(xs[0], norm)
    logits = h.float() @ gate.t()
    ids, w = ref.route(logits.cpu().numpy(), top_k, "sigmoid", routing.bias.cpu().numpy(), 4, 2, scale=1.5)
    exact, bound = ref.experts(ref.dequant(*ref.quant(h.float().cpu().numpy())), ids, w.astype(np.float32), gv, dv)
    check(layer.forward_logits(h, logits), exact, bound, torch.bfloat16)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(block(xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(r, want[i]) for r in got[i])
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        y = block(x)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]), i
        assert torch.equal(block(xs[i]), want[i]), i


def test_no_tokens(ops):
    parts, _, _ = make(4, 48, 144, 27)
    layer = layer_of(parts, routing=ops.Routing(2))
    for lead in ((0,), (3, 0)):
        x = torch.empty(*lead, 144, dtype=torch.bfloat16, device=DEV)
        y = layer.forward_logits(x, torch.empty(*lead, 4, device=DEV))
        assert y.shape == x.shape and y.dtype == x.dtype


def test_from_float(ops):
    from w8a8_int8_dynamic_amd import W8A8Experts
    e, k, inner = 3, 272, 144
    g = torch.Generator().manual_seed(8)
    gate_up, down = torch.randn(e, 2 * inner, k, generator=g), torch.randn(e, k, inner, generator=g)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        layer = W8A8Experts.from_float(gate_up.to(dtype).to(DEV), down.to(dtype).to(DEV))
        q = [[ref.quant_weight(p.to(dtype).float().numpy()) for p in (a[:inner], a[inner:], b)]
             for a, b in zip(gate_up, down)]
        other = layer_of([np.stack([np.concatenate((p[0][i], p[1][i])) for p in q]) if j == 0 else
                          np.stack([p[2][i] for p in q]) for j, i in ((0, 0), (0, 1), (1, 0), (1, 1))])
        for name in ("gate_up", "gate_up_scale", "down", "down_scale"):
            assert torch.equal(getattr(layer, name), getattr(other, name)), name
        assert layer.inner == inner and layer.in_features == k and layer.experts == e


def test_python_refusals(ops):
    e, top_k, k, inner, t = 3, 2, 160, 80, 4
    parts, _, _ = make(e, inner, k, 11)
    layer = layer_of(parts)
    x = rows(t, k, 2).to(DEV)
    ids, w = (v.to(DEV) for v in choose(t, e, top_k, 5))
    layer(x, ids, w)
    for bad in ((x[:, :-16], ids, w), (x, ids[:-1], w[:-1]), (x, ids, w[:, :1]), (x, ids[0], w[0]), (x, ids.cpu(), w),
                (x, ids, w.cpu()), (x, ids[:, :0], w[:, :0])):
        with pytest.raises(ValueError):
            layer(*bad)
    for bad in ((x.float(), ids, w), (x, ids.long(), w), (x, ids, w.double())):
        with pytest.raises(TypeError):
            layer(*bad)
    with pytest.raises(ValueError, match="routing"):
        layer.forward_logits(x, torch.zeros(t, e, device=DEV))
    layer.routing = ops.Routing(2)
    with pytest.raises(ValueError, match="logits"):
        layer.forward_logits(x, torch.zeros(t, e + 1, device=DEV))
    logits = torch.zeros(t, 8, device=DEV)
    for how in (ops.Routing(9), ops.Routing(0), ops.Routing(2, groups=3), ops.Routing(2, groups=4, top_groups=5),
                ops.Routing(5, groups=2), ops.Routing(2, group_top=3), ops.Routing(2, scale=float("nan")),
                ops.Routing(2, "top"), ops.Routing(2, bias=torch.zeros(7, device=DEV)),
                ops.Routing(2, bias=torch.zeros(8)), ops.Routing(2, bias=torch.zeros(8, device=DEV).double())):
        with pytest.raises((ValueError, RuntimeError)):
            ops.route_experts(logits, how)
    with pytest.raises(RuntimeError):
        ops.route_experts(torch.zeros(2, 1025, device=DEV), ops.Routing(2))
    with pytest.raises(ValueError):
        layer_of([parts[0][:, :-16], parts[1], parts[2], parts[3]])
    with pytest.raises(ValueError):
        layer_of([parts[0], parts[1][:, :-1], parts[2], parts[3]])


def test_route_logits_of_any_strides(ops):
    """Rows that are one row of memory, overlap, or lie further apart are routed as their contiguous copies are."""
    from tests.test_fp8_block_cpu import overlapping_logits
    for name, x in overlapping_logits().items():
        print(name, flush=True)
        flat = torch.empty(0).set_(x.untyped_storage()).to(DEV)
        view = flat.as_strided(x.shape, x.stride(), x.storage_offset())
        for score in ("softmax", "sigmoid"):
            how = ops.Routing(min(4, x.shape[1]), score)
            got, want = ops.route_experts(view, how), ops.route_experts(x.contiguous().to(DEV), how)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), name


# Rows an expert on average, of each path but the slots alone: small tiles, rows cut at 64, 128-row and 256-row
# tiles; of uneven shares, so that tiles of every fill are met.
@pytest.mark.parametrize("rows_each", [6, 10, 11, 24, 32, 33, 40, 70, 100, 104, 105, 150])
def test_experts_rows_whatever_their_place(ops, rows_each):
    """A token's result depends neither on its place among its expert's rows nor on how many others the expert
    has, on every path: all tokens in other orders, and with the other half of the tokens elsewhere."""
    e, top_k, k, inner = 6, 2, 656, 272
    t = rows_each * e // top_k
    parts, _, _ = make(e, inner, k, 31)
    layer = layer_of(parts)
    x = (rows(t, k, 2, torch.float32) * 0.3).to(torch.bfloat16).to(DEV)
    ids, w = (v.to(DEV) for v in choose(t, e, top_k, 5, skew=0.7))
    counts = torch.bincount(ids.flatten().long().cpu(), minlength=e).tolist()
    print(counts, flush=True)
    want = layer(x, ids, w)
    g = torch.Generator().manual_seed(3)
    for _ in range(4):
        perm = torch.randperm(t, generator=g).to(DEV)
        assert torch.equal(layer(x[perm], ids[perm], w[perm]), want[perm])
    half = torch.arange(t, device=DEV) % 2 == 0
    for turn in range(1, e):
        other = torch.where(half.unsqueeze(1), ids, (ids + turn) % e)
        assert torch.equal(layer(x, other, w)[half], want[half])
    none = torch.where(half.unsqueeze(1), ids, -1)
    got = layer(x, none, w)
    assert torch.equal(got[half], want[half]) and (got[~half] == 0).all()
