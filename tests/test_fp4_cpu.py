"""The 4-bit entry points' argument checks on the host (no kernel runs: a bad
argument returns before the device is touched, and a good call on a machine
without a GPU fails with W8A8_ERR_DEVICE), the reference rule on values
worked out by hand, and the layer's refusals."""
from __future__ import annotations

import os
import subprocess

import numpy as np
import pytest
import torch

from tests import fp4_reference as ref
from tests.test_abi_cpu import A, ALIGN, DEVICE, HEADER, L, MODE, NULL, OK, SHAPE
from w8a8_int8_dynamic_amd import W8A8Linear, _lib, ops, quantize_linear_layers
from w8a8_int8_dynamic_amd.build import CSRC, hipcc

NO_GPU = not torch.cuda.is_available()


def quant(x=A, t=0, M=4, K=64, ldx=64, q=A, ldq=32, s=A, lds=2):
    return L.fp4_quant_per_block(x, t, M, K, ldx, q, ldq, s, lds, None)


def mm(xq=A, ldq=32, xs=A, lds=16, wp=A, sp=A, bias=None, M=4, N=16, K=64, mode=0, out=A, ldo=16, tile=-1):
    return L.fp4_scaled_mm_tile(xq, ldq, xs, lds, wp, sp, bias, M, N, K, mode, out, ldo, None, tile)


def qmm(x=A, t=0, ldx=64, xq=A, ldq=32, xs=A, lds=16, wp=A, sp=A, bias=None, M=4, N=16, K=64, mode=0, out=A,
        ldo=16, tile=-1):
    return L.fp4_quant_scaled_mm_tile(x, t, ldx, xq, ldq, xs, lds, wp, sp, bias, M, N, K, mode, out, ldo, None,
                                      tile)


def test_quant_checks():
    assert quant(t=3) == MODE and quant(t=-1) == MODE
    assert quant(M=-1) == SHAPE and quant(K=0, ldx=0) == SHAPE and quant(K=48) == SHAPE
    assert quant(ldx=63) == SHAPE and quant(ldq=31) == SHAPE and quant(lds=1) == SHAPE
    assert quant(M=0, x=None, q=None, s=None) == OK
    assert quant(x=None) == NULL and quant(q=None) == NULL and quant(s=None) == NULL
    assert quant(x=A + 8) == ALIGN and quant(ldx=68) == ALIGN and quant(t=1, ldx=66) == ALIGN
    assert quant(q=A + 2) == ALIGN and quant(ldq=34) == ALIGN
    d = lambda **k: L.fp4_dequant(k.get("q", A), k.get("ldq", 32), k.get("s", A), k.get("lds", 2), k.get("M", 4),
                                  k.get("K", 64), k.get("t", 0), k.get("o", A), k.get("ldo", 64), None)
    assert d(t=7) == MODE and d(K=16) == SHAPE and d(ldo=32) == SHAPE and d(o=None) == NULL
    assert d(o=A + 4) == ALIGN and d(q=A + 1) == ALIGN and d(M=0, o=None, q=None, s=None) == OK
    if NO_GPU:
        assert quant(s=A + 1) == DEVICE and quant(t=1, ldx=68) == DEVICE and d() == DEVICE


def test_pack_checks():
    assert L.fp4_prepack_weight_bytes(16, 128) == 1024 and L.fp4_prepack_weight_bytes(17, 160) == 32 * 128
    assert L.fp4_prepack_scale_bytes(16, 128) == 256 and L.fp4_prepack_scale_bytes(17, 544) == 2 * 2 * 256
    for f in (L.fp4_prepack_weight_bytes, L.fp4_prepack_scale_bytes):
        assert f(0, 64) == 0 and f(16, 0) == 0 and f(16, 48) == 0 and f(2 ** 31, 64) == 0
    p = lambda **k: L.fp4_prepack_weight(k.get("q", A), k.get("ldq", 32), k.get("s", A), k.get("lds", 2),
                                         k.get("N", 4), k.get("K", 64), k.get("p", A), k.get("sp", A), None)
    u = lambda **k: L.fp4_unpack_weight(k.get("p", A), k.get("sp", A), k.get("N", 4), k.get("K", 64),
                                        k.get("q", A), k.get("ldq", 32), k.get("s", A), k.get("lds", 2), None)
    for f in (p, u):
        assert f(N=0) == SHAPE and f(K=40) == SHAPE and f(ldq=31) == SHAPE and f(lds=1) == SHAPE
        assert f(q=None) == NULL and f(s=None) == NULL and f(p=None) == NULL and f(sp=None) == NULL
        assert f(p=A + 8) == ALIGN and f(sp=A + 4) == ALIGN
        if NO_GPU:
            assert f(q=A + 1, s=A + 1) == DEVICE
    o = lambda **k: L.fp4_quant_prepack_weight(k.get("w", A), k.get("t", 1), k.get("N", 4), k.get("K", 64),
                                               k.get("ldw", 64), k.get("p", A), k.get("sp", A), None)
    assert o(t=2) == MODE and o(N=0) == SHAPE and o(K=33) == SHAPE and o(ldw=63) == SHAPE
    assert o(w=None) == NULL and o(sp=None) == NULL and o(w=A + 8) == ALIGN and o(ldw=68) == ALIGN
    assert o(t=0, ldw=66) == ALIGN
    if NO_GPU:
        assert o() == DEVICE and o(t=0, ldw=68) == DEVICE


def test_mm_checks():
    for f in (mm, qmm):
        assert f(mode=3) == MODE and f(mode=-1) == MODE and f(tile=-2) == MODE
        assert f(tile=L.w8a8_fp4_tile_count()) == MODE
        assert f(M=-1) == SHAPE and f(N=0) == SHAPE and f(K=16) == SHAPE and f(K=72) == SHAPE
        assert f(ldq=16) == SHAPE and f(lds=1) == SHAPE and f(ldo=15) == SHAPE
        big = _lib.W8A8_FP4_MAX_K + 32
        assert f(K=big, ldq=big, lds=big, **({"ldx": big} if f is qmm else {})) == SHAPE
        assert f(ldq=_lib.W8A8_MAX_LDQ + 16) == SHAPE and f(lds=_lib.W8A8_MAX_LDQ + 16) == SHAPE
        assert f(xq=None) == NULL and f(xs=None) == NULL and f(wp=None) == NULL
        assert f(sp=None) == NULL and f(out=None) == NULL
        assert f(xq=A + 8) == ALIGN and f(ldq=40) == ALIGN and f(wp=A + 8) == ALIGN and f(sp=A + 8) == ALIGN
        assert f(xs=A + 4) == ALIGN and f(lds=20) == ALIGN
        assert f(out=A + 1) == ALIGN and f(out=A + 2, mode=1) == ALIGN and f(bias=A + 1) == ALIGN
        n = 2 ** 31 - 1
        assert f(M=n, N=n, ldo=n) == SHAPE                  # no launch holds that many tiles
        none = dict(xq=None, xs=None, wp=None, sp=None, out=None)
        assert f(M=0, **none, **({"x": None} if f is qmm else {})) == OK
        if NO_GPU:
            assert f() == DEVICE and f(mode=1, bias=A + 1) == DEVICE and f(mode=2, bias=A) == DEVICE
    assert qmm(t=5) == MODE and qmm(ldx=63) == SHAPE and qmm(x=None) == NULL
    assert qmm(x=A + 8) == ALIGN and qmm(ldx=68) == ALIGN


def test_constants_and_tiles():
    text = open(HEADER).read()
    assert f"#define W8A8_FP4_MAX_K {_lib.W8A8_FP4_MAX_K}" in text
    n = ops.fp4_tile_count()
    names = [ops.fp4_tile_name(i) for i in range(n)]
    assert n >= 1 and len(set(names)) == n and all(names) and ops.fp4_tile_name(n) == ""
    for shape in [(1, 16, 32), (1, 12288, 4096), (512, 12288, 4096), (8192, 4096, 12288)]:
        assert 0 <= ops.fp4_tile_auto(*shape) < n


def test_reference_rule_by_hand():
    x = np.zeros((1, 64))
    # a = 6: floor(log2 6) = 2, scale 2^0: ties 0.25 -> 0, 0.75 -> 1, 1.25 -> 1,
    # 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4; -0 keeps its sign
    x[0, :11] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.0, -1.5, -5.0001]
    x[0, 32] = 7.9                                         # over 6: saturates
    q, s = ref.quant(x)
    v = ref.dequant(q, s)
    assert list(s[0]) == [127, 127]
    assert list(v[0, :11]) == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1.5, -6] and np.signbit(v[0, 8]) and v[0, 32] == 6
    assert q[0, 0] == 0x07 and q[0, 4] == 0xB8             # even element in the low nibble
    y = np.zeros((1, 96))
    y[0, 0], y[0, 33], y[0, 64] = 2.0 ** -140, np.nan, 2.0 ** 127
    q, s = ref.quant(y)
    assert list(s[0]) == [0, 255, 252] and q[0, 0] == 0 and not q[0, 16:32].any()
    assert np.isnan(ref.dequant(q, s)[0, 32:64]).all() and ref.dequant(q, s)[0, 64] == 2.0 ** 127


def test_refusals():
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        ops.fp4_quant_per_block(cpu)
    with pytest.raises(TypeError):
        ops.fp4_quant_per_block(cpu.double())
    with pytest.raises(ValueError, match="scheme"):
        W8A8Linear(torch.zeros(1), torch.zeros(1), 1, 32, scheme="fp5")
    with pytest.raises(ValueError, match="scheme"):
        W8A8Linear.from_quantized(torch.zeros(1, 16), torch.zeros(1), scheme="fp8")
    with pytest.raises(ValueError, match="GPU"):
        quantize_linear_layers(torch.nn.Linear(64, 64), method="fp4")


@pytest.mark.parametrize("scheme", ["int8", "fp8", "fp4"])
def test_layer_refuses_a_bias_of_another_shape(scheme):
    """The kernels read out_features elements of the bias, so the layer is not
    built on any other number of them."""
    packed = torch.zeros(16 * 64, dtype=torch.uint8)
    scale = torch.zeros(256, dtype=torch.uint8) if scheme == "fp4" else torch.zeros(16)
    for shape in ((), (1,), (15,), (17,), (1, 16), (16, 1)):
        with pytest.raises(ValueError, match="bias"):
            W8A8Linear(packed, scale, 16, 64, torch.zeros(shape), scheme)
    layer = W8A8Linear(packed, scale, 16, 64, torch.zeros(32)[::2], scheme)
    assert layer.bias.shape == (16,) and layer.bias.is_contiguous() and layer.bias_f16.is_contiguous()


def test_tiles_that_the_scale_rings_do_not_fit_are_not_compiled(tmp_path):
    """With two k-groups the second chunk of channel scales is loaded three steps
    ahead of the loop, so a tile that begins later must not compile."""
    for tile, fits in (("64, 64, 1, 2, 2, 3, 3", True), ("64, 64, 1, 2, 2, 1, 3", False),
                       ("64, 64, 2, 2, 1, 1, 3", True)):
        src = tmp_path / "tile.hip"
        src.write_text('#include "mm_kernel.hpp"\nnamespace w8a8 { namespace {\n'
                       f"static_assert(sizeof(Tile<{tile}>) > 0);\n}} }}\n")
        r = subprocess.run([hipcc(), "--cuda-host-only", "--offload-arch=gfx950", "-std=c++17", "-fsyntax-only", f"-I{CSRC}",
                            "-I" + os.path.dirname(HEADER), str(src)], capture_output=True, text=True)
        assert (r.returncode == 0) == fits, (tile, r.stderr[-2000:])
        assert fits or "scales" in r.stderr, r.stderr[-2000:]
