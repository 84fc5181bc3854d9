"""The microscaled 4-bit layer on the GPU against the rule in 64 bits.

Codes, scale bytes, packed bytes and dequantized values are exact. Products:
a block's 32 products of e2m1 values are whole multiples of a quarter of its
scales and their sum is exact in fp32, so only the additions across blocks
round, at most K/32 of them (K/64 by the instruction's own two blocks, in any
order), each by less than 2^-23 of a partial sum that is at most S = sum |x w|:
    |acc - exact| <= (K/32 + 1) * 2^-23 * S
The bias adds one fp32 rounding, 2^-24 of the result, and the store half a
step of the output's type (and half its smallest subnormal)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import fp4_reference as ref

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


def codes(m, k, seed, spread=6):
    """Random codes and scale bytes within `spread` powers of two of each other."""
    r = np.random.default_rng(seed)
    return (r.integers(0, 256, (m, k // 2), dtype=np.uint8),
            r.integers(127 - spread, 128 + spread, (m, k // 32), dtype=np.uint8))


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check(got, exact, mag, k, dtype, bias=None, what=""):
    got = got.double().cpu().numpy()
    bound = (k / 32 + 1) * 2.0 ** -23 * mag
    if bias is not None:
        exact = exact + bias.double().cpu().numpy()
        bound = bound + 2.0 ** -24 * (np.abs(exact) + bound)
    bound = bound + HALF[dtype] * (np.abs(exact) + bound) + TINY[dtype]
    nan = np.isnan(exact)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    top = torch.finfo(dtype).max
    over = ~nan & (np.abs(exact) - bound > top * (1 + HALF[dtype]))
    assert np.isinf(got[over]).all(), what
    ok = nan | over | (np.abs(got - exact) <= bound) | (np.isinf(got) & (np.abs(exact) + bound >= top))
    assert ok.all(), f"{what}: {(~ok).sum()} of {ok.size} outside, worst {np.nanmax((np.abs(got - exact) / bound)[~ok])}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,k", [(1, 32), (3, 64), (7, 96), (2, 4096), (65, 4128), (5, 12288), (1030, 160)])
def test_quant(ops, dtype, m, k):
    x = rows(m, k, 100 + m + k, dtype)
    xq, xs = ops.fp4_quant_per_block(x.to(DEV))
    q, s = ref.quant(x.double().numpy())
    assert np.array_equal(xs.cpu().numpy(), s) and np.array_equal(xq.cpu().numpy(), q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quant_every_pattern(ops, dtype):
    """Every 16-bit pattern (for fp32 those of bf16 and random ones) next to
    maxima that put it at every place of the grid: ties, subnormals, signed
    zeros, infinities and NaN."""
    bits = torch.arange(65536, dtype=torch.int32)
    if dtype == torch.float32:
        x = torch.cat(((bits << 16).view(torch.float32),
                       torch.randint(-2 ** 31, 2 ** 31 - 1, (65536,), generator=torch.Generator().manual_seed(1),
                                     dtype=torch.int32).view(torch.float32)))
    else:
        x = bits.to(torch.int16).view(dtype)
    x = torch.stack([x.reshape(-1, 32)] + [torch.where(torch.arange(32) == 5, t * x.reshape(-1, 32)[:, :1].float(),
                                                      x.reshape(-1, 32).float()).to(dtype)
                                           for t in (2.0, 8.0, 12.0, 100.0)]).reshape(-1, 64).contiguous()
    xq, xs = ops.fp4_quant_per_block(x.to(DEV))
    with np.errstate(invalid="ignore", over="ignore"):
        q, s = ref.quant(x.double().numpy())
    assert np.array_equal(xs.cpu().numpy(), s)
    assert np.array_equal(xq.cpu().numpy(), q)
    # and back: exact in bf16 and fp32, NaN where the block holds one
    for back in (torch.bfloat16, torch.float32):
        got = ops.fp4_dequant(xq, xs, back).double().cpu().numpy()
        assert np.array_equal(got, ref.dequant(q, s), equal_nan=True)


def test_dequant_rounds_once(ops):
    """fp16: overflow gives infinity, small values fp16 subnormals, nearest even;
    every scale byte in fp32."""
    q = np.tile(np.arange(256, dtype=np.uint8), (256, 1))[:, :256]
    s = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 16))
    want = ref.dequant(q, s)
    with np.errstate(over="ignore"):
        for dtype, to in ((torch.float16, np.float16), (torch.float32, np.float32)):
            got = ops.fp4_dequant(dev(q), dev(s), dtype).cpu().numpy()
            assert np.array_equal(got, want.astype(to), equal_nan=True)


def test_quant_strided_and_untouched(ops):
    """Rows inside wider buffers: the columns beside them stay as they were."""
    x = rows(9, 96, 7)
    wide = torch.zeros(9, 200, dtype=torch.bfloat16, device=DEV)
    wide[:, 8:104] = x.to(DEV)
    xq = torch.full((9, 96), 0xAA, dtype=torch.uint8, device=DEV)
    xs = torch.full((9, 16), 0xAA, dtype=torch.uint8, device=DEV)
    ops.fp4_quant_per_block(wide[:, 8:104], xq[:, :48], xs[:, :3])
    q, s = ref.quant(x.double().numpy())
    assert np.array_equal(xq[:, :48].cpu().numpy(), q) and np.array_equal(xs[:, :3].cpu().numpy(), s)
    assert (xq[:, 48:] == 0xAA).all() and (xs[:, 3:] == 0xAA).all()
    # an odd start and pitch are copied into aligned rows first
    odd = torch.zeros(9, 101, dtype=torch.bfloat16, device=DEV)
    odd[:, 5:] = x.to(DEV)
    xq2, xs2 = ops.fp4_quant_per_block(odd[:, 5:])
    assert np.array_equal(xq2.cpu().numpy(), q) and np.array_equal(xs2.cpu().numpy(), s)


def packed_reference(q, s):
    N, half = q.shape
    K = 2 * half
    nb, kb, ch = -(-N // 16), -(-K // 128), -(-K // 512)
    p = np.zeros((nb * 16, kb * 64), np.uint8)
    p[:N, :half] = q
    sp = np.full((nb * 16, ch * 16), 127, np.uint8)
    sp[:N, :K // 32] = s
    return (p.reshape(nb, 16, kb, 4, 16).transpose(0, 2, 3, 1, 4).reshape(-1),
            sp.reshape(nb, 16, ch, 16).transpose(0, 2, 1, 3).reshape(-1))


@pytest.mark.parametrize("n,k", [(1, 32), (16, 128), (17, 160), (100, 544), (33, 4128)])
def test_prepack(ops, n, k):
    for dtype in (torch.bfloat16, torch.float32):
        w = rows(n, k, n + k, dtype)
        q, s = ref.quant(w.double().numpy())
        p, sp = packed_reference(q, s)
        for a, b in (ops.fp4_quant_prepack_weight(w.to(DEV)), ops.fp4_prepack_weight(dev(q), dev(s))):
            assert np.array_equal(a.cpu().numpy(), p) and np.array_equal(b.cpu().numpy(), sp)
            q2, s2 = ops.fp4_unpack_weight(a, b, n, k)
            assert np.array_equal(q2.cpu().numpy(), q) and np.array_equal(s2.cpu().numpy(), s)


SHAPES = [(1, 1, 32), (1, 16, 32), (1, 300, 4096), (2, 48, 96), (5, 65, 160), (16, 128, 512), (17, 1111, 544),
          (33, 200, 4128), (64, 64, 128), (77, 129, 1056), (128, 192, 640), (200, 300, 2080), (257, 513, 1152),
          (300, 260, 8192)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_every_tile(ops, m, n, k):
    xq, xs = codes(m, k, m * n)
    wq, ws = codes(n, k, m * n + 1)
    exact, mag = ref.product(ref.dequant(xq, xs), ref.dequant(wq, ws))
    packed = ops.fp4_prepack_weight(dev(wq), dev(ws))
    g = torch.Generator().manual_seed(3)
    for tile in range(-1, ops.fp4_tile_count()):
        for dtype, with_bias in ((torch.bfloat16, False), (torch.float16, True), (torch.bfloat16, True),
                                 (torch.float32, False)):
            bias = (torch.randn(n, generator=g) * 30).to(dtype).to(DEV) if with_bias else None
            got = ops.fp4_scaled_mm(dev(xq), dev(xs), *packed, n, bias, out_dtype=dtype, tile=tile)
            check(got, exact, mag, k, dtype, bias, f"tile {tile} {dtype}")


@pytest.mark.parametrize("m,n,k", [(3, 50, 160), (40, 100, 544), (300, 260, 1056)])
def test_product_nan_blocks_and_garbage_beside_rows(ops, m, n, k):
    """A NaN block of a row or channel gives NaN exactly in its outputs; what
    lies behind the rows' codes and scales has no effect; the columns beside
    the output stay as they were."""
    xq, xs = codes(m, k, 1)
    wq, ws = codes(n, k, 2)
    xs[1, -1] = xs[m - 1, 0] = 255
    ws[n // 2, 1] = 255
    exact, mag = ref.product(ref.dequant(xq, xs), ref.dequant(wq, ws))
    assert np.isnan(exact).any() and not np.isnan(exact).all()
    packed = ops.fp4_prepack_weight(dev(wq), dev(ws))
    xqw = torch.full((m, k // 2 + 32), 0xFF, dtype=torch.uint8, device=DEV)
    xsw = torch.full((m, -(-(k // 32) // 16) * 16 + 16), 0xFF, dtype=torch.uint8, device=DEV)
    xqw[:, :k // 2], xsw[:, :k // 32] = dev(xq), dev(xs)
    for tile in range(-1, ops.fp4_tile_count()):
        out = torch.full((m, n + 9), 5.0, dtype=torch.bfloat16, device=DEV)
        ops.fp4_scaled_mm(xqw[:, :k // 2], xsw[:, :k // 32], *packed, n, out=out[:, :n], tile=tile)
        check(out[:, :n], exact, mag, k, torch.bfloat16, what=f"tile {tile}")
        assert (out[:, n:] == 5.0).all()


def test_product_scale_extremes(ops):
    """Scale bytes whose product leaves fp32's range: large sums give infinity,
    and opposite extremes cancel exactly."""
    q = np.full((2, 32), 0x22, np.uint8)                  # ones
    wp = {b: ops.fp4_prepack_weight(dev(q), dev(np.full((2, 2), b, np.uint8))) for b in (0, 127, 254)}
    for tile in range(-1, ops.fp4_tile_count()):
        for xb, wb, want in ((254, 0, 64.0), (0, 254, 64.0), (127, 127, 64.0), (254, 254, np.inf),
                             (254, 127, np.inf), (0, 127, 64.0 * 2.0 ** -127)):
            xs = dev(np.full((2, 2), xb, np.uint8))
            got = ops.fp4_scaled_mm(dev(q), xs, *wp[wb], 2, out_dtype=torch.float32, tile=tile).cpu().numpy()
            assert (got == np.float32(want)).all(), (tile, xb, wb, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1, 64, 4096), (2, 100, 160), (7, 333, 4128), (16, 48, 544), (33, 129, 96),
                                   (130, 257, 2080)])
def test_quant_scaled_mm(ops, dtype, m, n, k):
    """The one call gives the two calls' codes and product."""
    x = rows(m, k, m + n, dtype)
    wq, ws = codes(n, k, 5)
    packed = ops.fp4_prepack_weight(dev(wq), dev(ws))
    q, s = ref.quant(x.double().numpy())
    exact, mag = ref.product(ref.dequant(q, s), ref.dequant(wq, ws))
    for tile in range(-1, ops.fp4_tile_count()):
        out_dtype = torch.bfloat16 if dtype == torch.float32 else dtype
        out, xq, xs = ops.fp4_quant_scaled_mm(x.to(DEV), *packed, n, tile=tile)
        assert out.dtype == out_dtype
        assert np.array_equal(xq.cpu().numpy(), q) and np.array_equal(xs.cpu().numpy(), s), tile
        check(out, exact, mag, k, out_dtype, what=f"tile {tile}")


def test_empty_rows(ops):
    packed = ops.fp4_quant_prepack_weight(rows(16, 64, 1).to(DEV))
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    out, xq, xs = ops.fp4_quant_scaled_mm(x, *packed, 16)
    assert out.shape == (0, 16) and xq.shape == (0, 32) and xs.shape == (0, 2)
    assert ops.fp4_dequant(xq, xs).shape == (0, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer(ops, dtype):
    """from_float and from_quantized give one layer; inputs of any rank."""
    from w8a8_int8_dynamic_amd import W8A8Linear
    w, b = rows(96, 160, 11, torch.float32), torch.randn(96, generator=torch.Generator().manual_seed(2))
    layer = W8A8Linear.from_float(w.to(DEV), b.to(DEV), scheme="fp4")
    q, s = ref.quant(w.double().numpy())
    other = W8A8Linear.from_quantized(dev(q), dev(s), b.to(DEV), scheme="fp4")
    x = rows(6, 160, 12, dtype).reshape(2, 3, 160).to(DEV)
    out = layer(x)
    assert out.shape == (2, 3, 96) and out.dtype == dtype and torch.equal(out, other(x))
    xq, xs = ref.quant(x.double().cpu().numpy().reshape(6, 160))
    exact, mag = ref.product(ref.dequant(xq, xs), ref.dequant(q, s))
    check(out.reshape(6, 96), exact, mag, 160, dtype, b.to(dtype), "layer")
    with pytest.raises(TypeError):
        layer(x.float())
    bad = w.clone()
    bad[3, 40] = float("nan")
    with pytest.raises(ValueError, match="finite"):
        W8A8Linear.from_float(bad.to(DEV), scheme="fp4")
    with pytest.raises(ValueError, match="multiple of 32"):
        W8A8Linear.from_float(w[:, :48].to(DEV), scheme="fp4")


def test_convert(ops):
    from w8a8_int8_dynamic_amd import W8A8Linear, quantize_linear_layers
    torch.manual_seed(0)
    m = torch.nn.Sequential(torch.nn.Linear(64, 96), torch.nn.GELU(), torch.nn.Linear(96, 32)).to(DEV, torch.bfloat16)
    quantize_linear_layers(m, method="fp4")
    assert isinstance(m[0], W8A8Linear) and m[0].scheme == m[2].scheme == "fp4"
    assert m(torch.randn(5, 64, device=DEV, dtype=torch.bfloat16)).shape == (5, 32)
    with pytest.raises(ValueError, match="32"):
        quantize_linear_layers(torch.nn.Linear(48, 32).to(DEV), method="fp4")


def test_refusals(ops):
    xq, xs = (dev(a) for a in codes(4, 64, 1))
    packed = ops.fp4_prepack_weight(xq, xs)
    with pytest.raises(ValueError, match="xs"):
        ops.fp4_scaled_mm(xq, xs[:, :1], *packed, 4)
    with pytest.raises(ValueError, match="packed"):
        ops.fp4_scaled_mm(xq, xs, *packed, 17)
    with pytest.raises(ValueError, match="bias"):
        ops.fp4_scaled_mm(xq, xs, *packed, 4, bias=torch.zeros(4, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError, match="bias"):
        ops.fp4_scaled_mm(xq, xs, *packed, 4, bias=torch.zeros(4, device=DEV), out_dtype=torch.float32)
    with pytest.raises(TypeError):
        ops.fp4_scaled_mm(xq, xs, *packed, 4, out_dtype=torch.int32)
    with pytest.raises(ValueError, match="multiple of 32"):
        ops.fp4_quant_per_block(torch.zeros(2, 40, device=DEV))
    with pytest.raises(ops._lib.W8A8Error):
        ops.fp4_scaled_mm(xq, xs, *packed, 4, tile=ops.fp4_tile_count())


@pytest.mark.parametrize("m", [1, 20, 300])
def test_other_stream_and_graph(ops, m):
    """On a side stream, and captured: every replay gives the eager result, with
    eager work between them."""
    n, k = 200, 1056
    packed = ops.fp4_quant_prepack_weight(rows(n, k, 1).to(DEV))
    xs = [rows(m, k, 20 + i).to(DEV) for i in range(3)]
    want = [ops.fp4_quant_scaled_mm(x, *packed, n)[0].clone() for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    static = xs[0].clone()
    with torch.cuda.stream(side):
        assert torch.equal(ops.fp4_quant_scaled_mm(static, *packed, n)[0], want[0])
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = ops.fp4_quant_scaled_mm(static, *packed, n)[0]
    torch.cuda.synchronize()
    for i in (0, 1, 2, 1):
        static.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
        assert torch.equal(ops.fp4_quant_scaled_mm(xs[i], *packed, n)[0], want[i])


@pytest.mark.parametrize("m", [2, 40])
def test_longest_k(ops, m):
    """The largest K: every tile's chunk and block offsets at their limits."""
    n, k = 24, ops._lib.W8A8_FP4_MAX_K
    xq, xs = codes(m, k, 1)
    wq, ws = codes(n, k, 2)
    exact, mag = ref.product(ref.dequant(xq, xs), ref.dequant(wq, ws))
    packed = ops.fp4_prepack_weight(dev(wq), dev(ws))
    for tile in range(-1, ops.fp4_tile_count()):
        got = ops.fp4_scaled_mm(dev(xq), dev(xs), *packed, n, tile=tile)
        check(got, exact, mag, k, torch.bfloat16, what=f"tile {tile}")
    x = rows(m, k, 3)
    out, q, s = ops.fp4_quant_scaled_mm(x.to(DEV), *packed, n)
    want = ref.quant(x.double().numpy())
    assert np.array_equal(q.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])
    exact, mag = ref.product(ref.dequant(*want), ref.dequant(wq, ws))
    check(out, exact, mag, k, torch.bfloat16, what="quant")


def test_offsets_past_32_bits(ops):
    """Rows whose pitch puts the last of them billions of elements behind the
    first: rows of floats, codes, scales and outputs."""
    k, n = 544, 40
    wq, ws = codes(n, k, 2)
    packed = ops.fp4_prepack_weight(dev(wq), dev(ws))
    m, pitch = 5, (1 << 30) + 64
    x = rows(m, k, 3)
    big = torch.empty(m * pitch, dtype=torch.bfloat16, device=DEV)
    wide = big.as_strided((m, k), (pitch, 1))
    wide.copy_(x)
    want = ref.quant(x.double().numpy())
    exact, mag = ref.product(ref.dequant(*want), ref.dequant(wq, ws))
    for tile in range(-1, ops.fp4_tile_count()):
        out = big.as_strided((m, n), (pitch, 1), 4096)
        _, q, s = ops.fp4_quant_scaled_mm(wide, *packed, n, out=out, tile=tile)
        assert np.array_equal(q.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])
        check(out, exact, mag, k, torch.bfloat16, what=f"tile {tile}")
    del big, wide, out
    # codes and scales at the largest pitch the product takes, past 2^32 bytes
    m, pitch = 1030, ops._lib.W8A8_MAX_LDQ
    xq, xs = codes(m, k, 5)
    bytes_ = torch.empty(m * pitch, dtype=torch.uint8, device=DEV)
    q, s = bytes_.as_strided((m, k // 2), (pitch, 1)), bytes_.as_strided((m, k // 32), (pitch, 1), 1024)
    q.copy_(dev(xq))
    s.copy_(dev(xs))
    exact, mag = ref.product(ref.dequant(xq, xs), ref.dequant(wq, ws))
    for tile in range(-1, ops.fp4_tile_count()):
        check(ops.fp4_scaled_mm(q, s, *packed, n, tile=tile), exact, mag, k, torch.bfloat16, what=f"tile {tile}")
    assert np.array_equal(ops.fp4_dequant(q, s, torch.float32).cpu().numpy(), ref.dequant(xq, xs).astype(np.float32))


@pytest.mark.parametrize("m,n,k", [(1, 20, 16384), (1, 20, 16416), (2, 20, 8192), (2, 20, 8224), (3, 40, 4096),
                                   (4, 40, 4096), (4, 40, 4128), (5, 40, 4096), (16, 20, 1024), (16, 20, 1056),
                                   (17, 33, 1024), (40, 100, 992), (100, 300, 64), (250, 20, 736), (16, 20, 32)])
def test_quant_inside_the_product_and_beside_it(ops, m, n, k):
    """Either side of where the rows are too many to be quantized in the same
    launch."""
    x = rows(m, k, m + k)
    wq, ws = codes(n, k, 5)
    packed = ops.fp4_prepack_weight(dev(wq), dev(ws))
    want = ref.quant(x.double().numpy())
    exact, mag = ref.product(ref.dequant(*want), ref.dequant(wq, ws))
    for dtype in (torch.bfloat16, torch.float32):
        out, q, s = ops.fp4_quant_scaled_mm(x.to(dtype).to(DEV), *packed, n)
        assert np.array_equal(q.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])
        check(out, exact, mag, k, torch.bfloat16)


def test_rows_that_hold_nan_next_to_others(ops):
    """A NaN or infinity reaches the outputs of its row alone, quantized in the
    product's launch or before it; a row of zeros gives the bias."""
    n, k = 33, 1056
    packed = ops.fp4_quant_prepack_weight(rows(n, k, 1).to(DEV))
    bias = torch.randn(n, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    for m in (4, 24):
        x = rows(m, k, 2)
        x[0, 7], x[2, k - 1], x[3] = float("nan"), float("inf"), 0
        out, _, s = ops.fp4_quant_scaled_mm(x.to(DEV), *packed, n, bias)
        assert torch.isnan(out[0]).all() and torch.isnan(out[2]).all() and torch.isfinite(out[1]).all()
        assert torch.equal(out[3], bias) and s[0, 0] == 255 and s[2, -1] == 255 and (s[3] == 0).all()


def test_layer_checks_its_bias_at_each_call(ops):
    """A bias whose type, length, stride or device is not what the kernels read is
    refused, as by the other schemes: after a cast of the layer's floats (the
    codes stay as they are) and after an assignment."""
    from w8a8_int8_dynamic_amd import W8A8Linear
    n, k = 96, 160
    w, b = rows(n, k, 11, torch.float32).to(DEV), torch.randn(n, generator=torch.Generator().manual_seed(2)).to(DEV)
    make = lambda: W8A8Linear.from_float(w, b, scheme="fp4")  # noqa: E731
    x = {dtype: rows(6, k, 12, dtype).to(DEV) for dtype in (torch.bfloat16, torch.float16)}
    want = {dtype: make()(t) for dtype, t in x.items()}
    for cast, good in (("float", None), ("half", torch.float16), ("bfloat16", torch.bfloat16), ("double", None)):
        layer = getattr(make(), cast)()
        for dtype, t in x.items():
            if dtype == good:
                assert torch.equal(layer(t), want[dtype]), cast
            else:
                with pytest.raises(ValueError, match="bias"):
                    layer(t)
    bf = b.bfloat16()
    for bad in (bf[:-1], bf[:1], torch.cat((bf, bf)), torch.cat((bf, bf))[::2], bf[None], bf.cpu(), b):
        layer = make()
        layer.bias = bad
        with pytest.raises(ValueError, match="bias|device"):
            layer(x[torch.bfloat16])
    layer = make()
    layer.bias = torch.nn.Parameter(bf)
    assert torch.equal(layer(x[torch.bfloat16]), want[torch.bfloat16])
    layer.bias = None
    out = layer(x[torch.bfloat16])
    assert torch.equal(out, W8A8Linear.from_float(w, scheme="fp4")(x[torch.bfloat16]))
