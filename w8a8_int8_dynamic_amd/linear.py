"""W8A8Linear: a linear layer whose forward pass runs the W8A8 int8-dynamic path.

Shape handling follows the page "Diffusion Quantization Reference": its GGUF
rules flatten N-D activations around the matmul and restore the shape, and
its "Common Failures" table lists an output rank collapsing from 3-D to 2-D
as a bug. Inputs [..., K] are viewed as [M, K] (no copy when the last
dimension is contiguous) and outputs come back as [..., N].
"""
from __future__ import annotations

import fnmatch
from typing import Optional, Sequence

import torch

from . import ops

__all__ = ["W8A8Linear", "quantize_linear_layers"]


def _codes(wq: torch.Tensor) -> torch.Tensor:
    """e4m3 codes as uint8."""
    return wq.view(torch.uint8) if wq.dtype == torch.float8_e4m3fn else wq


def _block_scales(ws: torch.Tensor, shape: Sequence[int]) -> torch.Tensor:
    """Block scales [*shape] as contiguous fp32, checked."""
    if ws.shape != tuple(shape):
        raise ValueError(f"weight scales must have shape {tuple(shape)}, got {tuple(ws.shape)}")
    ws = ws.to(torch.float32).contiguous()
    if not torch.isfinite(ws).all():                   # (fp64 scales may lie past fp32's range)
        raise ValueError("weight scales must be finite")
    return ws


class W8A8Linear(torch.nn.Module):
    """y = q(x) @ q(W)^T * x_scale * w_scale (+ bias), in x's type.

    scheme "int8" (the default): int8 codes, bf16 or fp16 activations.
    scheme "fp8": the e4m3 twin (page "Online Quantization": FP8 W8A8 with
    dynamic per-token activation scales), bf16 activations.
    scheme "fp4": weights and activations in microscaled 4-bit floating point
    (MX FP4: e2m1 codes, a power-of-two scale per 32 elements along K), bf16 or
    fp16 activations; in_features a multiple of 32.
    scheme "fp8_block": e4m3 with an fp32 scale per 128 elements of an activation
    row and per 128 x 128 block of the weight, bf16 or fp16 activations.

    Build with ``from_float`` (online weight quantization on the GPU, written
    straight into the load-time layout) or ``from_quantized`` (weights and
    scales already made offline: int8 and fp32, or for "fp4" the uint8 codes
    [N, K/2] and scale bytes [N, K/32] of ops.fp4_quant_per_block, or for
    "fp8_block" e4m3 codes [N, K] as uint8 or float8_e4m3fn and fp32 scales
    [ceil(N/128), ceil(K/128)]).
    """

    def __init__(self, w_packed: torch.Tensor, w_scale: torch.Tensor, out_features: int,
                 in_features: int, bias: Optional[torch.Tensor] = None, scheme: str = "int8"):
        super().__init__()
        if scheme not in ("int8", "fp8", "fp4", "fp8_block"):
            raise ValueError(f"scheme must be 'int8', 'fp8', 'fp4' or 'fp8_block', got {scheme!r}")
        if bias is not None and bias.shape != (out_features,):
            raise ValueError(f"bias must have shape {(out_features,)}, got {tuple(bias.shape)}")
        self.scheme = scheme
        self.in_features = in_features
        self.out_features = out_features
        self.register_buffer("w_packed", w_packed)
        self.register_buffer("w_scale", w_scale)
        # The bias in each output type, rounded once from what was given.
        self.register_buffer("bias", None if bias is None else bias.to(torch.bfloat16).contiguous())
        self.register_buffer("bias_f16", None if bias is None else bias.to(torch.float16).contiguous())
        # The layer's own workspace for decode-shaped calls (a handful of
        # tokens against a weight with few column blocks), allocated once
        # here so that forward never allocates it.
        self.register_buffer(
            "workspace",
            ops.new_workspace(out_features, in_features, device=w_packed.device)
            if scheme == "int8" and w_packed.is_cuda else None,
            persistent=False)

    @classmethod
    def from_quantized(cls, wq: torch.Tensor, w_scale: torch.Tensor,
                       bias: Optional[torch.Tensor] = None, scheme: str = "int8") -> "W8A8Linear":
        if scheme not in ("int8", "fp4", "fp8_block"):
            raise ValueError(f"scheme must be 'int8', 'fp4' or 'fp8_block', got {scheme!r}")
        N, K = wq.shape
        if scheme == "fp8_block":
            w_scale = _block_scales(w_scale, (-(-N // 128), -(-K // 128)))
            return cls(ops.fp8_block_prepack_weight(_codes(wq)), w_scale, N, K, bias, scheme)
        if scheme == "fp4":
            if (w_scale == 255).any():
                raise ValueError("weight scales must be finite")
            packed = ops.fp4_prepack_weight(wq.contiguous(), w_scale.contiguous())
            return cls(*packed, N, 2 * K, bias, scheme)
        if not torch.isfinite(w_scale).all():
            raise ValueError("weight scales must be finite")
        packed = ops.prepack_weight(wq.contiguous())
        return cls(packed, w_scale.to(torch.float32).contiguous(), N, K, bias)

    @classmethod
    def from_float(cls, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   scheme: str = "int8") -> "W8A8Linear":
        """bf16 and fp32 weights are quantized as they are. Other float types
        are converted to fp32 first: exact for fp16, rounded for fp64 (the
        quant rule works on fp32 values)."""
        w = weight if weight.dtype in (torch.bfloat16, torch.float32) else weight.to(torch.float32)
        N, K = w.shape
        if scheme == "fp4":
            packed, ws = ops.fp4_quant_prepack_weight(w.contiguous())
            if (ws == 255).any():
                raise ValueError("weight scales must be finite")
            return cls(packed, ws, N, K, bias, scheme)
        if scheme == "fp8_block":
            packed, ws = ops.fp8_block_quant_prepack_weight(w.contiguous())
            return cls(packed, _block_scales(ws, ws.shape), N, K, bias, scheme)
        quant = ops.fp8_quant_prepack_weight if scheme == "fp8" else ops.quant_prepack_weight
        packed, ws = quant(w.contiguous())
        if not torch.isfinite(ws).all():
            raise ValueError("weight scales must be finite")
        return cls(packed, ws, N, K, bias, scheme)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected last dimension {self.in_features}, got {x.shape[-1]}")
        lead = x.shape[:-1]
        x2 = x if x.dim() == 2 else x.reshape(-1, self.in_features)
        if x2.stride(-1) != 1:
            x2 = x2.contiguous()
        # The quant and the scaled matmul, as one library call; the output (and
        # bias) type is x's.
        if self.scheme == "fp4" or self.scheme == "fp8_block":
            dtype = x2.dtype
            if dtype != torch.bfloat16 and dtype != torch.float16:
                raise TypeError(f"the {self.scheme} scheme takes bfloat16 or float16 activations, got {dtype}")
            name = "bias_f16" if dtype == torch.float16 else "bias"
            try:
                # (a Module's own lookup of a buffer costs about 0.4 us)
                b = self._buffers
                args = b["w_packed"], b["w_scale"], self.out_features, b[name]
            except KeyError:                           # one of them was replaced by a Parameter
                args = self.w_packed, self.w_scale, self.out_features, getattr(self, name)
            out = (ops._fp4_linear if self.scheme == "fp4" else ops._fp8_block_linear)(x2, *args)
            return out if x2 is x else out.reshape(*lead, self.out_features)
        bias = self.bias_f16 if x2.dtype == torch.float16 else self.bias
        if self.scheme == "fp8":
            if x2.dtype != torch.bfloat16:
                raise TypeError(f"the fp8 scheme takes bfloat16 activations, got {x2.dtype}")
            out, _, _ = ops.fp8_quant_scaled_mm(x2, self.w_packed, self.w_scale,
                                                self.out_features, bias)
        else:
            wsp = self.workspace if x2.dtype == torch.bfloat16 else None
            out, _, _ = ops.quant_scaled_mm(x2, self.w_packed, self.w_scale, self.out_features,
                                            bias, workspace=wsp)
        return out.reshape(*lead, self.out_features)

    def forward_quantized(self, xq: torch.Tensor, xs: torch.Tensor,
                          out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """The layer's product alone, for activations quantized elsewhere (by the
        ops that end in quant_per_token for "int8" and "fp8", by
        fp4_quant_per_block for "fp4", by fp8_quant_per_block for "fp8_block"): codes [M, K] (fp4: [M, K/2]) and their
        scales to [M, N] in out_dtype (bf16 or fp16). It uses no workspace of the
        layer, so calls on several streams may run at once; ops.scaled_mm takes
        one for a split of K at few rows (scheme "int8")."""
        if out_dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"out_dtype must be bfloat16 or float16, got {out_dtype}")
        K = xq.shape[-1] * (2 if self.scheme == "fp4" else 1)
        if K != self.in_features:
            raise ValueError(f"expected codes of {self.in_features} elements, got {K}")
        bias = self.bias_f16 if out_dtype == torch.float16 else self.bias
        if self.scheme == "fp4":
            return ops.fp4_scaled_mm(xq, xs, self.w_packed, self.w_scale, self.out_features, bias, out_dtype)
        if self.scheme == "fp8_block":
            return ops.fp8_block_scaled_mm(xq, xs, self.w_packed, self.w_scale, self.out_features, bias, out_dtype)
        if self.scheme == "fp8":
            return ops.fp8_scaled_mm(xq, xs, self.w_packed, self.w_scale, self.out_features, bias, out_dtype)
        return ops.scaled_mm(xq, xs, self.w_packed, self.w_scale, self.out_features, bias, out_dtype)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, scheme={self.scheme}")


def quantize_linear_layers(module: torch.nn.Module, method: str = "int8",
                           activation_scheme: str = "dynamic",
                           ignored_layers: Sequence[str] = ()) -> torch.nn.Module:
    """Replace the torch.nn.Linear layers of `module` by W8A8Linear layers.

    The selection follows the page "Online Quantization" (Parameters table):
    `method` is "int8", "fp8", "fp4" or "fp8_block"; `activation_scheme` must be "dynamic"
    (activation scales computed at run time, the only scheme implemented);
    `ignored_layers` holds name patterns of layers to keep in their float
    type. A layer is kept when its qualified name (as in
    module.named_modules()) matches a pattern by fnmatch or contains it.
    Weights are quantized online on their device (W8A8Linear.from_float).
    Anything the path cannot run raises ValueError naming the layer: a layer
    on the CPU, or in_features not a multiple of 16 (32 for "fp4"). Returns
    `module`, or the replacement when `module` is itself a Linear."""
    if method not in ("int8", "fp8", "fp4", "fp8_block"):
        raise ValueError(f"method must be 'int8', 'fp8', 'fp4' or 'fp8_block', got {method!r}")
    if activation_scheme != "dynamic":
        raise ValueError(f"only activation_scheme='dynamic' is implemented, got {activation_scheme!r}")
    patterns = [p for p in ignored_layers if p]
    step = 32 if method == "fp4" else 16

    def kept(name: str) -> bool:
        return any(fnmatch.fnmatchcase(name, p) or p in name for p in patterns)

    def convert(name: str, lin: torch.nn.Linear) -> W8A8Linear:
        if not lin.weight.is_cuda:
            raise ValueError(f"layer {name!r} is on {lin.weight.device}; move the model to the GPU first")
        if lin.in_features % step != 0:
            raise ValueError(f"layer {name!r}: in_features {lin.in_features} is not a multiple of {step}")
        bias = None if lin.bias is None else lin.bias.detach()
        return W8A8Linear.from_float(lin.weight.detach(), bias, scheme=method)

    if isinstance(module, torch.nn.Linear):
        return module if kept("") else convert("", module)
    for parent_name, parent in list(module.named_modules()):
        for child_name, child in list(parent.named_children()):
            name = f"{parent_name}.{child_name}" if parent_name else child_name
            if isinstance(child, torch.nn.Linear) and not kept(name):
                setattr(parent, child_name, convert(name, child))
    return module
