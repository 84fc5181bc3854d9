"""W8A8Experts: a mixture of experts whose products run the block-scaled e4m3 path.

The routed counterpart of W8A8Linear's scheme "fp8_block": every expert is a
gated feed-forward block (gate and up products, silu, down product) with e4m3
weights, and each token's rows go through the experts that its router chose.
Inputs [..., K] are viewed as [T, K] and come back in their shape.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import ops
from .linear import _block_scales, _codes

__all__ = ["W8A8Experts"]


class W8A8Experts(torch.nn.Module):
    """y[t] = sum over j of weights[t, j] * down_e(silu(gate_e x[t]) * up_e x[t]), e = ids[t, j].

    Build with ``from_float`` (online quantization on the GPU) or
    ``from_quantized`` (e4m3 codes as uint8 or float8_e4m3fn, and fp32 scales of
    128 x 128 blocks). gate_up is [E, 2 * inner, K], an expert's gate rows, then
    its up rows; down is [E, K, inner]. K and inner are multiples of 16.

    forward takes the experts of each token and their weights; with ``routing``
    (an ops.Routing) forward_logits takes the router's logits. It runs forward
    only, and uses no workspace of the layer, so calls on several streams may
    run at once.
    """

    def __init__(self, gate_up: torch.Tensor, gate_up_scale: torch.Tensor, down: torch.Tensor,
                 down_scale: torch.Tensor, inner: int, in_features: int, routing: Optional[ops.Routing] = None):
        super().__init__()
        self.in_features = in_features
        self.inner = inner
        self.experts = gate_up_scale.shape[0]
        self.register_buffer("gate_up", gate_up)
        self.register_buffer("gate_up_scale", gate_up_scale)
        self.register_buffer("down", down)
        self.register_buffer("down_scale", down_scale)
        self.routing = routing

    @staticmethod
    def _shapes(gate_up: torch.Tensor, down: torch.Tensor):
        if gate_up.dim() != 3 or down.dim() != 3 or gate_up.shape[1] % 2 != 0 or \
                down.shape != (gate_up.shape[0], gate_up.shape[2], gate_up.shape[1] // 2):
            raise ValueError(f"gate_up [E, 2 * inner, K] and down [E, K, inner] do not belong together: "
                             f"{tuple(gate_up.shape)} and {tuple(down.shape)}")
        E, both, K = gate_up.shape
        if both // 2 % 16 != 0 or K % 16 != 0:
            raise ValueError(f"inner and K must be multiples of 16, got {both // 2} and {K}")
        return E, both // 2, K

    @classmethod
    def from_quantized(cls, gate_up: torch.Tensor, gate_up_scale: torch.Tensor, down: torch.Tensor,
                       down_scale: torch.Tensor, routing: Optional[ops.Routing] = None) -> "W8A8Experts":
        """gate_up_scale [E, 2*ceil(inner/128), ceil(K/128)], the gate's blocks, then the
        up's; down_scale [E, ceil(K/128), ceil(inner/128)]."""
        E, inner, K = cls._shapes(gate_up, down)
        k, i = -(-K // 128), -(-inner // 128)
        return cls(ops.fp8_block_prepack_weight(_codes(gate_up), gated=True),
                   _block_scales(gate_up_scale, (E, 2 * i, k)), ops.fp8_block_prepack_weight(_codes(down)),
                   _block_scales(down_scale, (E, k, i)), inner, K, routing)

    @classmethod
    def from_float(cls, gate_up: torch.Tensor, down: torch.Tensor,
                   routing: Optional[ops.Routing] = None) -> "W8A8Experts":
        """bf16 and fp32 weights are quantized as they are, other float types by way of fp32."""
        E, inner, K = cls._shapes(gate_up, down)

        def quant(w, gated):
            w = w if w.dtype in (torch.bfloat16, torch.float32) else w.to(torch.float32)
            packed, ws = ops.fp8_block_quant_prepack_weight(w, gated)
            return packed, _block_scales(ws, ws.shape)

        return cls(*quant(gate_up, True), *quant(down, False), inner, K, routing)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor) -> torch.Tensor:
        """x [..., K] (bf16 or fp16), ids int32 and weights fp32 [..., top_k], or of the flattened
        tokens [T, top_k] (an id outside [0, E) stands for no expert) -> [..., K] in x's type."""
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected last dimension {self.in_features}, got {x.shape[-1]}")
        if x.dtype != torch.bfloat16 and x.dtype != torch.float16:
            raise TypeError(f"x must be bfloat16 or float16, got {x.dtype}")
        flat = x.dim() == 2
        x2 = x if flat else x.reshape(-1, self.in_features)
        if x2.stride(-1) != 1:
            x2 = x2.contiguous()
        if not flat:
            if ids.shape != weights.shape or (ids.shape[:-1] != x.shape[:-1] and ids.dim() != 2):
                raise ValueError(f"ids and weights must be [..., top_k] beside x {tuple(x.shape)}, got "
                                 f"{tuple(ids.shape)} and {tuple(weights.shape)}")
            ids, weights = ids.reshape(-1, ids.shape[-1]), weights.reshape(-1, weights.shape[-1])
        y = ops.fp8_block_experts(x2, ids, weights, self.gate_up, self.gate_up_scale, self.down, self.down_scale,
                                  self.inner)
        return y if flat else y.reshape(x.shape)

    def forward_logits(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """The same by the router's logits [..., E] (bf16, fp16 or fp32) and the layer's routing."""
        if self.routing is None:
            raise ValueError("the layer has no routing")
        if logits.shape[-1] != self.experts or logits.shape[:-1] != x.shape[:-1]:
            raise ValueError(f"logits must be {(*x.shape[:-1], self.experts)}, got {tuple(logits.shape)}")
        logits = logits.reshape(-1, self.experts)
        ids, weights = ops.route_experts(logits if logits.stride(-1) == 1 else logits.contiguous(), self.routing)
        shape = (*x.shape[:-1], self.routing.top_k)
        return self.forward(x, ids.reshape(shape), weights.reshape(shape))

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, inner={self.inner}, experts={self.experts}"
