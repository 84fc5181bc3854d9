"""The block-scaled e4m3 layer on the GPU against the rule in 64 bits.

Codes, scales, packed bytes and dequantized values are exact. Products keep the
bound that tests/block_reference.py derives; the bias adds one fp32 rounding
and the store half a step of the output's type (and half its smallest
subnormal)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import block_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 0.0}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w8a8_int8_dynamic_amd import _lib
    from w8a8_int8_dynamic_amd import ops as _ops
    assert _ops.device_supported(torch.cuda.current_device()), _lib.last_error()
    return _ops


def rows(m, k, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.where(torch.rand(k, generator=g) < 0.02, 20.0, 1.0)
    return (x * 10.0 ** (torch.rand(m, 1, generator=g) * 2 - 1)).to(dtype)


def codes(m, k, seed):
    """Random e4m3 codes (no NaN) whose products stay moderate, and scales."""
    r = np.random.default_rng(seed)
    q = r.integers(0, 256, (m, k), dtype=np.uint8)
    q[(q & 127) == 127] ^= 1
    return q, (2.0 ** r.uniform(-9, -5, (m, ref.blocks_of(k)))).astype(np.float32)


def weights(n, k, seed):
    q, _ = codes(n, k, seed)
    r = np.random.default_rng(seed + 1)
    return q, (2.0 ** r.uniform(-12, -8, (ref.blocks_of(n), ref.blocks_of(k)))).astype(np.float32)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check(got, exact, bound, dtype, bias=None, what=""):
    got = got.double().cpu().numpy()
    if bias is not None:
        exact = exact + bias.double().cpu().numpy()
        bound = bound + 2.0 ** -24 * (np.abs(exact) + bound)
    bound = bound + HALF[dtype] * (np.abs(exact) + bound) + TINY[dtype]
    ok = np.abs(got - exact) <= bound
    if dtype == torch.float16:
        ok |= np.isinf(got) & (np.abs(exact) + bound >= 65504)
    assert ok.all(), f"{what}: {(~ok).sum()} of {ok.size} outside, worst {(np.abs(got - exact) / bound)[~ok].max()}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,k", [(1, 16), (3, 128), (7, 144), (2, 4096), (65, 4112), (5, 12288), (1030, 272)])
def test_quant_and_dequant(ops, dtype, m, k):
    x = rows(m, k, m * 7 + k, dtype)
    x[0, : min(k, 5)] = 0.0
    q, s = ops.fp8_quant_per_block(x.to(DEV))
    want_q, want_s = ref.quant(x.float().numpy())
    assert q.dtype == torch.uint8 and s.shape == (m, ref.blocks_of(k))
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)
    exact = torch.from_numpy((ref.VALUES.astype(np.float32)[want_q] *
                              np.repeat(want_s, 128, 1)[:, :k]).astype(np.float32))
    for out in (torch.bfloat16, torch.float16, torch.float32):
        assert torch.equal(ops.fp8_block_dequant(q, s, out).cpu(), exact.to(out)), out


def test_quant_special_blocks(ops):
    """Blocks of zeros, below 2^-100, with a subnormal, an infinity or NaN: the rest of
    the row keeps its codes and scales."""
    x = rows(6, 512, 3, torch.float32)
    x[0, :128] = 0.0
    x[1, 128:256] = 2.0 ** -101
    x[2, 300] = float("inf")
    x[3, 511] = float("nan")
    x[4, 256:384] = 2.0 ** -100
    x[5, :] = -0.0
    q, s = (t.cpu().numpy() for t in ops.fp8_quant_per_block(x.to(DEV)))
    clean = x.clone()
    clean[2, 256:384] = 0
    clean[3, 384:] = 0
    want_q, want_s = ref.quant(clean.numpy())
    bad = np.zeros((6, 4), bool)
    bad[2, 2] = bad[3, 3] = True
    assert not np.isfinite(s[bad]).any()
    assert np.array_equal(s[~bad], want_s[~bad])
    keep = ~np.repeat(bad, 128, 1)
    assert np.array_equal(q[keep], want_q[keep])
    assert want_s[0, 0] == 0 and want_s[1, 1] == 0 and want_s[4, 2] > 0


def test_quant_strides_and_given_outputs(ops):
    wide = rows(9, 700, 4)
    x = wide.to(DEV)[:, 4:4 + 400]                         # rows off 16 bytes: copied
    y = wide.to(DEV)[:, 8:8 + 400][::2]
    for t, src in ((x, wide[:, 4:404]), (y, wide[::2, 8:408])):
        q, s = ops.fp8_quant_per_block(t)
        want = ref.quant(src.float().numpy())
        assert np.array_equal(q.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])
    qb = torch.full((9, 432), 7, dtype=torch.uint8, device=DEV)
    sb = torch.full((9, 8), 7.0, device=DEV)
    ops.fp8_quant_per_block(x, qb[:, :400], sb[:, 2:6])
    want = ref.quant(wide[:, 4:404].float().numpy())
    assert np.array_equal(qb[:, :400].cpu().numpy(), want[0]) and (qb[:, 400:] == 7).all()
    assert np.array_equal(sb[:, 2:6].cpu().numpy(), want[1]) and (sb[:, :2] == 7).all() and (sb[:, 6:] == 7).all()
    assert torch.equal(ops.fp8_block_dequant(qb[:, :400], sb[:, 2:6], torch.float32).cpu().double(),
                       torch.from_numpy(ref.VALUES.astype(np.float32)[want[0]] *
                                        np.repeat(want[1], 128, 1)[:, :400]).double())
    q, s = ops.fp8_quant_per_block(x[:0])
    assert q.shape == (0, 400) and s.shape == (0, 4) and ops.fp8_block_dequant(q, s).shape == (0, 400)


@pytest.mark.parametrize("n,k", [(1, 16), (16, 128), (130, 272), (257, 400), (48, 1040)])
def test_weights(ops, n, k):
    """The repack and its inverse, the online quantization of both types, and the layout."""
    q, _ = codes(n, k, n + k)
    packed = ops.fp8_block_prepack_weight(dev(q))
    assert np.array_equal(ops.fp8_block_unpack_weight(packed, n, k).cpu().numpy(), q)
    frag = packed.cpu().numpy().reshape(-(-n // 16), ref.blocks_of(k), 8, 16, 16)   # nb, kb, chunk, channel, byte
    padded = np.zeros((frag.shape[0] * 16, frag.shape[1] * 128), np.uint8)
    padded[:n, :k] = q
    assert np.array_equal(frag.transpose(0, 3, 1, 2, 4).reshape(padded.shape), padded)
    for dtype in (torch.float32, torch.bfloat16):
        w = rows(n, k, 5, dtype)
        got, ws = ops.fp8_block_quant_prepack_weight(w.to(DEV))
        want_q, want_s = ref.quant_weight(w.float().numpy())
        assert np.array_equal(ws.cpu().numpy(), want_s)
        assert np.array_equal(ops.fp8_block_unpack_weight(got, n, k).cpu().numpy(), want_q)
        assert torch.equal(got, ops.fp8_block_prepack_weight(dev(want_q)))


@pytest.mark.parametrize("inner,k", [(16, 16), (144, 272), (128, 128), (272, 400)])
def test_expert_weights(ops, inner, k):
    q = np.stack([codes(2 * inner, k, 10 + e)[0] for e in range(3)])
    packed = ops.fp8_block_prepack_weight(dev(q), gated=True)
    assert np.array_equal(ops.fp8_block_unpack_weight(packed, 2 * inner, k, gated=True, experts=3).cpu().numpy(), q)
    frag = packed.cpu().numpy().reshape(3, inner // 16, 2, ref.blocks_of(k), 8, 16, 16)
    back = frag.transpose(0, 2, 1, 5, 3, 4, 6).reshape(3, 2 * inner, -1)[..., :k]
    assert np.array_equal(back, q)
    w = torch.stack([rows(2 * inner, k, e, torch.float32) for e in range(3)])
    got, ws = ops.fp8_block_quant_prepack_weight(w.to(DEV), gated=True)
    halves = [[ref.quant_weight(h.numpy()) for h in (e[:inner], e[inner:])] for e in w]
    assert np.array_equal(ws.cpu().numpy(), np.stack([np.concatenate([h[1] for h in e]) for e in halves]))
    want = np.stack([np.concatenate([h[0] for h in e]) for e in halves])
    assert np.array_equal(ops.fp8_block_unpack_weight(got, 2 * inner, k, gated=True, experts=3).cpu().numpy(), want)
    plain = np.stack([codes(40, k, 20 + e)[0] for e in range(3)])
    packed = ops.fp8_block_prepack_weight(dev(plain))
    assert np.array_equal(ops.fp8_block_unpack_weight(packed, 40, k, experts=3).cpu().numpy(), plain)


SHAPES = [(1, 16, 16), (1, 300, 4112), (3, 40, 128), (16, 33, 400), (17, 129, 144), (65, 200, 1040), (130, 257, 272),
          (300, 520, 656), (257, 640, 128)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_every_tile(ops, m, n, k):
    xq, xs = codes(m, k, m + k)
    wq, ws = weights(n, k, n + k)
    exact, bound = ref.product(ref.dequant(xq, xs), ref.weight(wq, ws))
    packed = ops.fp8_block_prepack_weight(dev(wq))
    x, s, w = dev(xq), dev(xs), dev(ws)
    for tile in range(-1, ops.fp8_block_tile_count()):
        what = f"{m}x{n}x{k} {ops.fp8_block_tile_name(tile)}"
        print(what, flush=True)
        check(ops.fp8_block_scaled_mm(x, s, packed, w, n, out_dtype=torch.float32, tile=tile), exact, bound,
              torch.float32, what=what)
        for dtype in (torch.bfloat16, torch.float16):
            bias = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(dtype).to(DEV)
            check(ops.fp8_block_scaled_mm(x, s, packed, w, n, bias, dtype, tile=tile), exact, bound, dtype, bias, what)
            got = ops.fp8_block_scaled_mm(x, s, packed, w, n, None, dtype, tile=tile)
            check(got, exact, bound, dtype, what=what)


@pytest.mark.parametrize("m,n,k", [(70, 260, 8336), (3, 40, 131056)])
def test_product_long_rows(ops, m, n, k):
    """More than 64 blocks, and the most."""
    test_product_every_tile(ops, m, n, k)


def test_offsets_past_32_bits(ops):
    """More than 2^32 codes, and results 2 GiB apart: the last rows are those of a small call."""
    m, k = 270000, 16384
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    x[-3:] = rows(3, k, 1).to(DEV)
    q, s = ops.fp8_quant_per_block(x)
    q3, s3 = ops.fp8_quant_per_block(x[-3:].clone())
    assert q.numel() > 2 ** 32 and torch.equal(q[-3:], q3) and torch.equal(s[-3:], s3)
    assert torch.equal(ops.fp8_block_dequant(q, s)[-3:], ops.fp8_block_dequant(q3, s3))
    del x
    wq, ws = weights(80, k, 2)
    packed, w = ops.fp8_block_prepack_weight(dev(wq)), dev(ws)
    for tile in range(ops.fp8_block_tile_count()):
        got = ops.fp8_block_scaled_mm(q, s, packed, w, 80, tile=tile)
        assert torch.equal(got[-3:], ops.fp8_block_scaled_mm(q3, s3, packed, w, 80, tile=tile)), tile
    far = 2 ** 30
    out = torch.empty(far * 2 + 80, dtype=torch.bfloat16, device=DEV).as_strided((3, 80), (far, 1))
    for tile in range(ops.fp8_block_tile_count()):
        want = ops.fp8_block_scaled_mm(q3, s3, packed, w, 80, tile=tile)
        out.zero_()
        ops.fp8_block_scaled_mm(q3, s3, packed, w, 80, out=out, tile=tile)
        assert torch.equal(out, want), tile


@pytest.mark.parametrize("m,n,k", [(5, 70, 272), (140, 200, 400)])
def test_product_strides(ops, m, n, k):
    """Rows of codes, scales and outputs further apart than they are long; what lies
    between the outputs' rows stays."""
    xq, xs = codes(m, k, 1)
    wq, ws = weights(n, k, 2)
    exact, bound = ref.product(ref.dequant(xq, xs), ref.weight(wq, ws))
    packed, w = ops.fp8_block_prepack_weight(dev(wq)), dev(ws)
    xb = torch.full((m, k + 48), 0x7f, dtype=torch.uint8, device=DEV)
    xb[:, 16:16 + k] = dev(xq)
    sb = torch.full((m, xs.shape[1] + 3), float("nan"), device=DEV)
    sb[:, 1:1 + xs.shape[1]] = dev(xs)
    off = torch.full((m, k + 7), 0x7f, dtype=torch.uint8, device=DEV)
    off[:, 3:3 + k] = dev(xq)
    for x in (xb[:, 16:16 + k], off[:, 3:3 + k]):
        for ld, at in ((n + 8, 0), (n + 5, 3)):
            for tile in range(ops.fp8_block_tile_count()):
                out = torch.full((m, ld + at), 7.0, dtype=torch.bfloat16, device=DEV)
                ops.fp8_block_scaled_mm(x, sb[:, 1:1 + xs.shape[1]], packed, w, n, out=out[:, at:at + n], tile=tile)
                check(out[:, at:at + n], exact, bound, torch.bfloat16, what=f"tile {tile} ld {ld}")
                assert (out[:, :at] == 7).all() and (out[:, at + n:] == 7).all()


@pytest.mark.parametrize("k", [400, 656, 1040, 1168])
def test_product_many_tiles(ops, k):
    """More tiles than the card holds at once: rows have the values of smaller launches."""
    m, n, step = 4400, 4250, 320
    x, s = (dev(a) for a in codes(m, k, 7))
    wq, ws = weights(n, k, 8)
    packed, w = ops.fp8_block_prepack_weight(dev(wq)), dev(ws)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(9)).to(torch.float16).to(DEV)
    for tile in range(ops.fp8_block_tile_count()):
        print(ops.fp8_block_tile_name(tile), flush=True)
        for b, dtype in ((None, torch.float32), (None, torch.bfloat16), (bias, torch.float16)):
            got = ops.fp8_block_scaled_mm(x, s, packed, w, n, b, dtype, tile=tile)
            for at in range(0, m, step):
                want = ops.fp8_block_scaled_mm(x[at:at + step], s[at:at + step], packed, w, n, b, dtype, tile=tile)
                assert torch.equal(got[at:at + step], want), (tile, at)


def test_product_keeps_to_its_rows(ops):
    """A row of NaN scales or NaN codes, or zero rows, changes no other row; zero
    weight blocks give zeros."""
    m, n, k = 70, 150, 528
    xq, xs = codes(m, k, 3)
    wq, ws = weights(n, k, 4)
    packed = ops.fp8_block_prepack_weight(dev(wq))
    want = [ops.fp8_block_scaled_mm(dev(xq), dev(xs), packed, dev(ws), n, tile=t)
            for t in range(ops.fp8_block_tile_count())]
    xs2, xq2 = xs.copy(), xq.copy()
    xs2[5, 1] = np.nan
    xs2[20] = 0
    xs2[33, 0] = np.inf
    xq2[69] = 0x7f
    others = [i for i in range(m) if i not in (5, 20, 33, 69)]
    for t, w in enumerate(want):
        got = ops.fp8_block_scaled_mm(dev(xq2), dev(xs2), packed, dev(ws), n, tile=t)
        assert torch.equal(got[others], w[others]), t
        assert got[5].isnan().all() and (got[20] == 0).all() and not got[33].isfinite().any() and got[69].isnan().all()


def test_layer(ops):
    """The layer is quant and product; N-D inputs keep their shape; both types; M = 0."""
    from w8a8_int8_dynamic_amd import W8A8Linear, quantize_linear_layers
    n, k = 200, 1040
    w = rows(n, k, 1, torch.float32) * 0.05
    b = torch.randn(n, generator=torch.Generator().manual_seed(2))
    layer = W8A8Linear.from_float(w.to(DEV), b.to(DEV), scheme="fp8_block")
    wq, ws = ref.quant_weight(w.numpy())
    again = W8A8Linear.from_quantized(dev(wq).view(torch.float8_e4m3fn), dev(ws), b.to(DEV), scheme="fp8_block")
    assert torch.equal(layer.w_packed, again.w_packed) and torch.equal(layer.w_scale, again.w_scale)
    for m in (1, 5, 64, 200):
        for dtype in (torch.bfloat16, torch.float16):
            x = rows(m, k, m, dtype)
            exact, bound = ref.product(ref.dequant(*ref.quant(x.float().numpy())), ref.weight(wq, ws))
            y = layer(x.to(DEV))
            assert y.dtype == dtype
            check(y, exact, bound, dtype, b.to(dtype), f"m {m}")
            assert torch.equal(again(x.to(DEV)), y)
            assert torch.equal(layer.forward_quantized(*ops.fp8_quant_per_block(x.to(DEV)), out_dtype=dtype), y)
            out, q, s = ops.fp8_block_quant_scaled_mm(x.to(DEV), layer.w_packed, layer.w_scale, n,
                                                      layer.bias if dtype == torch.bfloat16 else layer.bias_f16)
            assert torch.equal(out, y)
            want_q, want_s = ref.quant(x.float().numpy())
            assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)
    x = rows(12, k, 9)
    assert torch.equal(layer(x.to(DEV).reshape(3, 4, k)), layer(x.to(DEV)).reshape(3, 4, n))
    assert torch.equal(layer(x.t().contiguous().t().to(DEV)), layer(x.to(DEV)))
    assert layer(x[:0].to(DEV)).shape == (0, n)
    lin = torch.nn.Linear(k, n).to(DEV)
    net = quantize_linear_layers(torch.nn.Sequential(lin), method="fp8_block")
    assert net[0].scheme == "fp8_block"
    assert torch.equal(net[0].w_packed, ops.fp8_block_quant_prepack_weight(lin.weight.detach())[0])


def test_layer_beats_a_scale_per_row_on_outliers(ops):
    """What the finer scales are for: with one column in a block far above the rest, the
    other blocks keep their precision."""
    from w8a8_int8_dynamic_amd import W8A8Linear
    n, k = 64, 1024
    g = torch.Generator().manual_seed(1)
    x = torch.randn(32, k, generator=g)
    x[:, 7] = 2e6
    w = torch.randn(n, k, generator=g) * 0.02
    w[:, 7] = 0.0                                          # the outlier itself meets no weight
    xb = x.bfloat16().to(DEV)
    exact = xb.double() @ w.double().to(DEV).t()

    def off(scheme):
        y = W8A8Linear.from_float(w.to(DEV), scheme=scheme)(xb).double()
        return ((y - exact).norm() / exact.norm()).item()

    # One scale per row: the smallest code stands for 2e6 / 448 * 2^-9 = 8.7, twice what any other element
    # reaches, so everything is lost. Per block: 1 of 8 blocks is, sqrt(1/8) = 0.35 of the norm, and the
    # others' codes and the weights' are 2^-4 / sqrt(3) off at most each, 0.05 together.
    assert off("fp8_block") < 0.45 < 0.95 < off("fp8")


@pytest.mark.parametrize("m", [1, 40, 300])
def test_other_stream_and_graph(ops, m):
    from w8a8_int8_dynamic_amd import W8A8Linear
    n, k = 264, 656
    layer = W8A8Linear.from_float((rows(n, k, 1, torch.float32) * 0.05).to(DEV), scheme="fp8_block")
    xs = [rows(m, k, 20 + i).to(DEV) for i in range(4)]
    want = [layer(x).clone() for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [layer(x) for x in xs]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = layer(x)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]), i
        assert torch.equal(layer(xs[i]), want[i])


def test_python_refusals(ops):
    from w8a8_int8_dynamic_amd import W8A8Linear
    m, n, k = 4, 136, 272
    xq, xs = (dev(t) for t in codes(m, k, 1))
    wq, ws = (dev(t) for t in weights(n, k, 2))
    packed = ops.fp8_block_prepack_weight(wq)
    mm = lambda **a: ops.fp8_block_scaled_mm(a.get("xq", xq), a.get("xs", xs), a.get("p", packed), a.get("ws", ws),
                                             a.get("n", n), a.get("bias"), a.get("dtype", torch.bfloat16),
                                             a.get("out"), a.get("tile", -1))
    mm()
    for bad in (dict(xq=xq[:, :-8]), dict(xs=xs[:, :-1]), dict(xs=xs[:-1]), dict(p=packed[:-1]), dict(ws=ws[:, :-1]),
                dict(ws=ws.t().contiguous().t()), dict(n=n + 100), dict(n=0), dict(bias=torch.zeros(n, device=DEV)),
                dict(bias=torch.zeros(n + 1, dtype=torch.bfloat16, device=DEV)),
                dict(bias=torch.zeros(n, dtype=torch.float32, device=DEV), dtype=torch.float32),
                dict(out=torch.zeros(m, n + 1, dtype=torch.bfloat16, device=DEV)), dict(ws=ws.cpu()),
                dict(xs=xs.cpu()), dict(p=packed.cpu())):
        with pytest.raises((ValueError, TypeError)):
            mm(**bad)
    for bad in (dict(dtype=torch.float64), dict(xq=xq.int()), dict(xs=xs.double())):
        with pytest.raises(TypeError):
            mm(**bad)
    with pytest.raises(Exception, match="tile"):
        mm(tile=ops.fp8_block_tile_count())
    with pytest.raises(ValueError, match="multiple"):
        ops.fp8_quant_per_block(torch.zeros(2, 24, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        ops.fp8_block_prepack_weight(wq, gated=True)        # 136 rows: no two halves of whole fragments
    with pytest.raises(ValueError, match="shape"):
        W8A8Linear.from_quantized(wq, ws[:, :-1], scheme="fp8_block")
    with pytest.raises(ValueError, match="finite"):
        W8A8Linear.from_quantized(wq, ws * float("inf"), scheme="fp8_block")
    layer = W8A8Linear.from_quantized(wq, ws, scheme="fp8_block")
    with pytest.raises(TypeError):
        layer(torch.zeros(2, k, device=DEV))
    with pytest.raises(ValueError):
        layer(torch.zeros(2, k + 16, dtype=torch.bfloat16, device=DEV))


def test_weights_of_any_strides(ops):
    """Rows that are one row of memory, overlap, or lie further apart: packed as their contiguous copies are."""
    from tests.test_fp8_block_cpu import overlapping_weights
    for name, w in overlapping_weights().items():
        print(name, flush=True)
        full = w.contiguous().to(DEV)
        for dtype in (torch.uint8, torch.float32, torch.bfloat16):
            flat = torch.empty(0, dtype=torch.float32).set_(w.untyped_storage()).to(dtype).to(DEV)
            view = flat.as_strided(w.shape, w.stride(), w.storage_offset())
            assert torch.equal(view.float(), full)
            for gated in (False, True) if w.shape[-2] == 32 else (False,):
                if dtype == torch.uint8:
                    assert torch.equal(ops.fp8_block_prepack_weight(view, gated),
                                       ops.fp8_block_prepack_weight(full.to(dtype), gated))
                else:
                    got = ops.fp8_block_quant_prepack_weight(view, gated)
                    want = ops.fp8_block_quant_prepack_weight(full.to(dtype), gated)
                    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
