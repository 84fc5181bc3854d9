"""The 4-bit layer, the norms and the gated residuals together, as a block of a
diffusion or language model uses them: norm to codes, a quantized layer on the
codes, its output back into the stream with the next norm, a 4-bit feed-forward.
Each step is held to the 64-bit reference on the step before; the whole block,
replayed from a graph, to its own eager run."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import fp4_reference as fp4
from tests import norm_reference as ref
from tests.test_gpu_fp4 import check

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(k, seed, dtype):
    from w8a8_int8_dynamic_amd import W8A8Linear
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = {"attn": r(k, k) * 0.05, "up": r(2 * k, k) * 0.05, "down": r(k, 2 * k) * 0.05}
    b = {n: 0.1 * r(t.shape[0]) for n, t in w.items()}
    layers = {"int8": W8A8Linear.from_float(w["attn"].to(DEV), b["attn"].to(DEV)),
              "fp8": W8A8Linear.from_float(w["attn"].to(DEV), b["attn"].to(DEV), scheme="fp8"),
              "up": W8A8Linear.from_float(w["up"].to(DEV), b["up"].to(DEV), scheme="fp4"),
              "down": W8A8Linear.from_float(w["down"].to(DEV), b["down"].to(DEV), scheme="fp4")}
    return layers, w, b, (r(1, k) * 0.1 + 1).to(dtype).to(DEV)[0]


def block(ops, layers, x, mod, post, code):
    """(r1, h1, up, r2) of one block; mod: [G, 6, K] as a model's projection gives it."""
    quant = ops.norm_quant_per_token if code == "int8" else ops.fp8_norm_quant_per_token
    xq, xs = quant(x, ops.Norm("layer", scale=mod[:, 0], shift=mod[:, 1]))
    a = layers[code].forward_quantized(xq, xs, out_dtype=x.dtype)
    r1, h1 = ops.gated_residual_norm(x, a, ops.Norm("layer", scale=mod[:, 3], shift=mod[:, 4]), gate=mod[:, 2],
                                     post=ops.Norm("rms", weight=post))
    up = layers["up"](h1)
    down = layers["down"](torch.nn.functional.gelu(up, approximate="tanh"))
    r2 = ops.gated_residual(r1, down, gate=mod[:, 5], post=ops.Norm("rms", weight=post))
    return a, r1, h1, up, down, r2


@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, "int8"), (torch.bfloat16, "fp8"), (torch.float16, "int8")])
@pytest.mark.parametrize("images,tokens", [(1, 1), (2, 33), (3, 100)])
def test_block(dtype, code, images, tokens):
    from w8a8_int8_dynamic_amd import ops
    k = 256
    layers, w, b, post = make(k, 5, dtype)
    g = torch.Generator().manual_seed(images)
    x = (torch.randn(images * tokens, k, generator=g) * 2).to(dtype).to(DEV)
    mod = (0.3 * torch.randn(images, 6, k, generator=g)).to(DEV)
    a, r1, h1, up, down, r2 = block(ops, layers, x, mod, post, code)
    # the layer on the norm's codes is the two steps on their own
    n = ops.Norm("layer", scale=mod[:, 0].contiguous(), shift=mod[:, 1].contiguous())
    quant = ops.norm_quant_per_token if code == "int8" else ops.fp8_norm_quant_per_token
    h, err = ref.norm(x.double(), torch.zeros_like(x, dtype=torch.float64), "layer", 1e-6,
                      scale=mod[:, 0], shift=mod[:, 1])
    codes = quant(x, n)
    ref.check_codes(*codes, h, err, 127 if code == "int8" else 448, "first norm")
    assert torch.equal(layers[code].forward_quantized(*codes, out_dtype=dtype), a)
    p = {"kind": "rms", "eps": 1e-6, "weight": post}
    want, err = ref.residual(x, a, gate=mod[:, 2], post=p)
    ref.check_float(r1, want, err, dtype, "r1")
    h, h_err = ref.norm(want, err, "layer", 1e-6, scale=mod[:, 3], shift=mod[:, 4])
    ref.check_float(h1, h, h_err, dtype, "h1")
    for name, xin, got in (("up", h1, up), ("down", torch.nn.functional.gelu(up, approximate="tanh"), down)):
        xq = fp4.dequant(*fp4.quant(xin.double().cpu().numpy()))
        wq = fp4.dequant(*fp4.quant(w[name].double().numpy()))
        exact, mag = fp4.product(xq, wq)
        check(got, exact, mag, xin.shape[1], dtype, b[name].to(dtype), name)
    want, err = ref.residual(r1, down, gate=mod[:, 5], post=p)
    ref.check_float(r2, want, err, dtype, "r2")
    assert np.isfinite(r2.float().cpu().numpy()).all()


def test_block_replayed():
    """Captured once and replayed on new inputs, with eager work in between."""
    from w8a8_int8_dynamic_amd import ops
    k, rows = 256, 48
    layers, _, _, post = make(k, 6, torch.bfloat16)
    g = torch.Generator().manual_seed(1)
    xs = [(torch.randn(rows, k, generator=g) * 2).bfloat16().to(DEV) for _ in range(3)]
    mod = (0.3 * torch.randn(2, 6, k, generator=g)).to(DEV)
    want = [[t.clone() for t in block(ops, layers, x, mod, post, "int8")] for x in xs]
    static = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(ops, layers, static, mod, post, "int8")
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = block(ops, layers, static, mod, post, "int8")
    torch.cuda.synchronize()
    for i in (0, 1, 2, 0, 2):
        static.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want[i])), i
        again = block(ops, layers, xs[i], mod, post, "int8")
        assert all(torch.equal(u, v) for u, v in zip(again, want[i])), i


def test_calls_at_once_on_two_streams():
    """Calls that overlap share nothing: each stream's results are its own."""
    from w8a8_int8_dynamic_amd import ops
    k, rows = 512, 200
    layers, _, _, post = make(k, 7, torch.bfloat16)
    g = torch.Generator().manual_seed(2)
    xs = [(torch.randn(rows, k, generator=g) * 2).bfloat16().to(DEV) for _ in range(2)]
    mod = (0.3 * torch.randn(2, 6, k, generator=g)).to(DEV)
    want = [[t.clone() for t in block(ops, layers, x, mod, post, "fp8")] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(block(ops, layers, xs[i], mod, post, "fp8"))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(u, v) for u, v in zip(r, want[i]))


@pytest.mark.parametrize("scheme", ["int8", "fp8", "fp4"])
@pytest.mark.parametrize("m", [1, 70])
def test_forward_quantized(scheme, m):
    """A layer on codes made beside it is the layer on the floats, in both
    output types; several streams at once give what one gives."""
    from w8a8_int8_dynamic_amd import W8A8Linear, ops
    n, k = 200, 1056
    g = torch.Generator().manual_seed(3)
    lin = W8A8Linear.from_float((0.05 * torch.randn(n, k, generator=g)).to(DEV),
                                torch.randn(n, generator=g).to(DEV), scheme=scheme)
    quant = {"int8": ops.quant_per_token, "fp8": ops.fp8_quant_per_token, "fp4": ops.fp4_quant_per_block}[scheme]
    for dtype in (torch.bfloat16, torch.float16):
        if scheme == "fp8" and dtype == torch.float16:
            continue
        x = torch.randn(m, k, generator=g).to(dtype).to(DEV)
        assert torch.equal(lin.forward_quantized(*quant(x), out_dtype=dtype), lin(x))
    codes = quant(torch.randn(m, k, generator=g).bfloat16().to(DEV))
    want = lin.forward_quantized(*codes)
    half = lin.forward_quantized(*codes, out_dtype=torch.float16)
    # one sum rounded to either type (bias too): each within its half steps
    top = want.float().abs().max().item()
    assert (want.float() - half.float()).abs().max().item() <= top * (2 ** -7 + 2 ** -10) + 4 * (2 ** -8 + 2 ** -11)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(lin.forward_quantized(*codes))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got)
    for bad in ((codes[0][:, :-16], codes[1]), (codes[0].cpu(), codes[1])):
        with pytest.raises((ValueError, TypeError)):
            lin.forward_quantized(*bad)
    with pytest.raises(TypeError):
        lin.forward_quantized(*codes, out_dtype=torch.float32)
