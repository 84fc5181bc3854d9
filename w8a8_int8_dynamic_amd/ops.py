"""Torch-tensor wrappers over the libw8a8 C ABI (argument marshalling only).

Every step of the layer runs in the HIP kernels; these functions only check
dtypes and devices, allocate outputs with torch, and pass raw device
pointers, leading dimensions and torch's current HIP stream to the library.
Tensors must be on a CUDA (HIP) device; the last dimension must be
contiguous (stride 1); the row stride becomes the leading dimension.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import W8A8_OUT_BF16, W8A8_OUT_F16, W8A8_OUT_I32, call

__all__ = ["quant_per_token", "quant_per_channel", "prepack_weight", "quant_prepack_weight", "unpack_weight",
           "prepack_weight_bytes", "scaled_mm", "quant_scaled_mm", "tile_count", "tile_name",
           "workspace_bytes", "new_workspace",
           "tile_auto", "device_supported", "fp8_quant_per_token", "fp8_quant_per_channel",
           "fp8_quant_prepack_weight", "fp8_scaled_mm", "fp8_quant_scaled_mm", "fp8_tile_count",
           "fp4_quant_per_block", "fp4_dequant", "fp4_prepack_weight", "fp4_quant_prepack_weight",
           "fp4_unpack_weight", "fp4_scaled_mm", "fp4_quant_scaled_mm", "fp4_tile_count", "fp4_tile_name",
           "fp4_tile_auto", "fp8_quant_per_block", "fp8_block_dequant", "fp8_block_prepack_weight",
           "fp8_block_quant_prepack_weight", "fp8_block_unpack_weight", "fp8_block_scaled_mm",
           "fp8_block_quant_scaled_mm", "fp8_block_tile_count", "fp8_block_tile_name", "fp8_block_tile_auto",
           "Routing", "route_experts", "fp8_block_experts", "Norm", "norm",
           "norm_quant_per_token", "fp8_norm_quant_per_token", "gated_residual",
           "gated_residual_norm", "gated_residual_norm_quant", "fp8_gated_residual_norm_quant"]


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _matrix(t: torch.Tensor, name: str, dtype: torch.dtype) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return t


def _ld(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _vector(t: Optional[torch.Tensor], n: int, name: str, dtype: torch.dtype):
    if t is None:
        return None
    if not t.is_cuda or t.dtype != dtype or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous {dtype} device vector of length {n}")
    return t


def _same_device(ref: torch.Tensor, *others: Optional[torch.Tensor]) -> None:
    for t in others:
        if t is not None and t.device != ref.device:
            raise ValueError(f"all tensors must be on {ref.device}, got one on {t.device}")


def _packed(w_packed: torch.Tensor, N: int, K: int) -> None:
    if not w_packed.is_cuda or w_packed.dtype != torch.uint8 or \
            w_packed.numel() < prepack_weight_bytes(N, K):
        raise ValueError("w_packed must be a uint8 device buffer of the packed layout (N, K)")


def _round_up(a: int, b: int) -> int:
    return -(-a // b) * b


def _rows_aligned(t: torch.Tensor, elems: int) -> torch.Tensor:
    """t itself when its rows start on 16-byte boundaries (row stride a multiple of
    ``elems``), else a copy into a row-padded buffer, viewed back to t's shape."""
    if t.data_ptr() % 16 == 0 and _ld(t) % elems == 0:
        return t
    M, K = t.shape
    buf = torch.empty((M, _round_up(K, elems)), dtype=t.dtype, device=t.device)
    buf[:, :K].copy_(t)
    return buf[:, :K]


def _codes(M: int, K: int, device) -> torch.Tensor:
    """int8 [M, K] view of a buffer whose rows are padded to 16 bytes, the row
    stride int8_scaled_mm requires."""
    return torch.empty((M, _round_up(K, 16)), dtype=torch.int8, device=device)[:, :K]


_ACT_ENTRY = {torch.bfloat16: "", torch.float16: "_f16"}
_OUT_MODE = {torch.bfloat16: W8A8_OUT_BF16, torch.float16: W8A8_OUT_F16, torch.int32: W8A8_OUT_I32}


def _act_dtype(x: torch.Tensor) -> torch.dtype:
    if x.dtype not in _ACT_ENTRY:
        raise TypeError(f"x must be bfloat16 or float16, got {x.dtype}")
    return x.dtype


def _out_mode(out_dtype: torch.dtype) -> int:
    if out_dtype not in _OUT_MODE:
        raise TypeError("out_dtype must be torch.bfloat16, torch.float16 or torch.int32")
    return _OUT_MODE[out_dtype]


def quant_per_token(x: torch.Tensor, xq: Optional[torch.Tensor] = None,
                    xs: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-token dynamic quantization of bf16 or fp16 x [M, K] -> (int8 [M, K], fp32 [M])."""
    _matrix(x, "x", _act_dtype(x))
    M, K = x.shape
    x = _rows_aligned(x, 8)
    if xq is None:
        xq = _codes(M, K, x.device)
    if xs is None:
        xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _matrix(xq, "xq", torch.int8)
    if xq.shape != (M, K):
        raise ValueError(f"xq must have shape {(M, K)}")
    _vector(xs, M, "xs", torch.float32)
    _same_device(x, xq, xs)
    with torch.cuda.device(x.device):
        call("int8_quant_per_token" + _ACT_ENTRY[x.dtype], x.data_ptr(), M, K, _ld(x),
             xq.data_ptr(), _ld(xq), xs.data_ptr(), _stream(x))
    return xq, xs


def quant_per_channel(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-output-channel quantization of fp32 w [N, K] -> (int8 [N, K], fp32 [N])."""
    _matrix(w, "w", torch.float32)
    N, K = w.shape
    w = _rows_aligned(w, 4)
    wq = _codes(N, K, w.device)
    ws = torch.empty((N,), dtype=torch.float32, device=w.device)
    with torch.cuda.device(w.device):
        call("int8_quant_per_channel", w.data_ptr(), N, K, _ld(w), wq.data_ptr(), _ld(wq),
             ws.data_ptr(), _stream(w))
    return wq, ws


def prepack_weight_bytes(N: int, K: int) -> int:
    n = _lib.lib().int8_prepack_weight_bytes(N, K)
    if n == 0:
        raise ValueError(f"no prepacked size for N={N}, K={K}")
    return n


def prepack_weight(wq: torch.Tensor) -> torch.Tensor:
    """Repack int8 wq [N, K] into the fragment layout int8_scaled_mm reads (uint8 bytes)."""
    _matrix(wq, "wq", torch.int8)
    N, K = wq.shape
    packed = torch.empty((prepack_weight_bytes(N, K),), dtype=torch.uint8, device=wq.device)
    with torch.cuda.device(wq.device):
        call("int8_prepack_weight", wq.data_ptr(), N, K, _ld(wq), packed.data_ptr(), _stream(wq))
    return packed


def quant_prepack_weight(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Online per-output-channel quantization of a bf16 or fp32 weight [N, K],
    written straight into the prepacked layout: (packed uint8 bytes, fp32 [N]).
    The same bytes and scales as prepack_weight(quant_per_channel(w))."""
    if w.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"w must be bfloat16 or float32, got {w.dtype}")
    _matrix(w, "w", w.dtype)
    N, K = w.shape
    f32 = w.dtype == torch.float32
    w = _rows_aligned(w, 4 if f32 else 8)
    packed = torch.empty((prepack_weight_bytes(N, K),), dtype=torch.uint8, device=w.device)
    ws = torch.empty((N,), dtype=torch.float32, device=w.device)
    with torch.cuda.device(w.device):
        call("int8_quant_prepack_weight", w.data_ptr(), 0 if f32 else 1, N, K, _ld(w),
             packed.data_ptr(), ws.data_ptr(), _stream(w))
    return packed, ws


def unpack_weight(packed: torch.Tensor, N: int, K: int) -> torch.Tensor:
    """Inverse of prepack_weight: int8 [N, K]."""
    if not packed.is_cuda or packed.dtype != torch.uint8 or packed.numel() < prepack_weight_bytes(N, K):
        raise ValueError("packed must be a uint8 device buffer from prepack_weight")
    wq = torch.empty((N, K), dtype=torch.int8, device=packed.device)
    with torch.cuda.device(packed.device):
        call("int8_unpack_weight", packed.data_ptr(), N, K, wq.data_ptr(), K, _stream(packed))
    return wq


def workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes of workspace the split of K uses for an M x N x K product (0: none)."""
    return int(_lib.lib().int8_scaled_mm_workspace_bytes(M, N, K))


def new_workspace(N: int, K: int, max_rows: int = 32, device=None) -> Optional[torch.Tensor]:
    """A zeroed workspace large enough for every M up to max_rows against an
    N x K weight (None when no such shape splits K). Give each stream (or
    each concurrently replayed graph) its own."""
    need = max(workspace_bytes(m, N, K) for m in range(1, max_rows + 1))
    if need == 0:
        return None
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return torch.zeros((need,), dtype=torch.uint8, device=device)


def _workspace(workspace: Optional[torch.Tensor]):
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def scaled_mm(xq: torch.Tensor, xs: Optional[torch.Tensor], w_packed: torch.Tensor,
              ws: Optional[torch.Tensor], N: int, bias: Optional[torch.Tensor] = None,
              out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
              tile: int = -1, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[m, n] = acc * xs[m] * ws[n] (+ bias[n]) rounded to out_dtype (bf16 or fp16;
    the bias in the same type), or the int32 accumulators when out_dtype=int32.
    With a workspace (from new_workspace; automatic tile only) decode-shaped
    products may split K over workgroups; results are bit-identical."""
    _matrix(xq, "xq", torch.int8)
    M, K = xq.shape
    mode = _out_mode(out_dtype)
    if mode != W8A8_OUT_I32:
        _vector(xs, M, "xs", torch.float32)
        _vector(ws, N, "ws", torch.float32)
        _vector(bias, N, "bias", out_dtype)
    _packed(w_packed, N, K)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    _matrix(out, "out", out_dtype)
    if out.shape != (M, N):
        raise ValueError(f"out must have shape {(M, N)}")

    def ptr(t):
        return None if t is None or mode == W8A8_OUT_I32 else t.data_ptr()

    _same_device(xq, w_packed, out, *((xs, ws, bias) if mode != W8A8_OUT_I32 else ()))
    if workspace is not None:
        if tile != -1:
            raise ValueError("a workspace goes with the automatic tile (tile=-1)")
        _same_device(xq, workspace)
        wp, wb = _workspace(workspace)
        with torch.cuda.device(xq.device):
            call("int8_scaled_mm_ws", xq.data_ptr(), _ld(xq), ptr(xs), w_packed.data_ptr(), ptr(ws),
                 ptr(bias), M, N, K, mode, out.data_ptr(), _ld(out), wp, wb, _stream(xq))
        return out
    with torch.cuda.device(xq.device):
        call("int8_scaled_mm_tile", xq.data_ptr(), _ld(xq), ptr(xs), w_packed.data_ptr(), ptr(ws),
             ptr(bias), M, N, K, mode, out.data_ptr(), _ld(out), _stream(xq), tile)
    return out


def quant_scaled_mm(x: torch.Tensor, w_packed: torch.Tensor, ws: Optional[torch.Tensor], N: int,
                    bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                    out: Optional[torch.Tensor] = None, tile: int = -1,
                    xq: Optional[torch.Tensor] = None, xs: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Per-token quant of bf16 or fp16 x [M, K] and the scaled matmul in one call.

    out_dtype defaults to x's type. Returns (out, xq, xs): out as scaled_mm
    returns it, and the int8 codes and fp32 scales the quant produced
    (bit-identical to quant_per_token). A workspace (bf16 x, automatic tile)
    lets decode-shaped products split K, as in scaled_mm."""
    _matrix(x, "x", _act_dtype(x))
    if out_dtype is None:
        out_dtype = x.dtype
    M, K = x.shape
    x = _rows_aligned(x, 8)
    mode = _out_mode(out_dtype)
    if mode != W8A8_OUT_I32:
        _vector(ws, N, "ws", torch.float32)
        _vector(bias, N, "bias", out_dtype)
    _packed(w_packed, N, K)
    if xq is None:
        xq = _codes(M, K, x.device)
    if xs is None:
        xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _matrix(xq, "xq", torch.int8)
    if xq.shape != (M, K):
        raise ValueError(f"xq must have shape {(M, K)}")
    _vector(xs, M, "xs", torch.float32)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _matrix(out, "out", out_dtype)
    if out.shape != (M, N):
        raise ValueError(f"out must have shape {(M, N)}")

    def ptr(t):
        return None if t is None or mode == W8A8_OUT_I32 else t.data_ptr()

    _same_device(x, w_packed, xq, xs, out, *((ws, bias) if mode != W8A8_OUT_I32 else ()))
    if workspace is not None:
        if tile != -1 or x.dtype != torch.bfloat16:
            raise ValueError("a workspace goes with bf16 activations and the automatic tile")
        _same_device(x, workspace)
        wp, wb = _workspace(workspace)
        with torch.cuda.device(x.device):
            call("int8_quant_scaled_mm_ws", x.data_ptr(), _ld(x), xq.data_ptr(), _ld(xq),
                 xs.data_ptr(), w_packed.data_ptr(), ptr(ws), ptr(bias), M, N, K, mode,
                 out.data_ptr(), _ld(out), wp, wb, _stream(x))
        return out, xq, xs
    with torch.cuda.device(x.device):
        call("int8_quant_scaled_mm" + _ACT_ENTRY[x.dtype] + "_tile", x.data_ptr(), _ld(x),
             xq.data_ptr(), _ld(xq), xs.data_ptr(), w_packed.data_ptr(), ptr(ws), ptr(bias), M,
             N, K, mode, out.data_ptr(), _ld(out), _stream(x), tile)
    return out, xq, xs


# ---- the FP8 (e4m3) twin ------------------------------------------------
_FP8_OUT_MODE = {torch.bfloat16: W8A8_OUT_BF16, torch.float16: W8A8_OUT_F16,
                 torch.float32: W8A8_OUT_I32}


def _fp8_codes(M: int, K: int, device) -> torch.Tensor:
    return torch.empty((M, _round_up(K, 16)), dtype=torch.uint8, device=device)[:, :K]


def fp8_quant_per_token(x: torch.Tensor, xq: Optional[torch.Tensor] = None,
                        xs: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-token dynamic e4m3 quantization of bf16 x [M, K] -> (uint8 codes [M, K], fp32 [M])."""
    _matrix(x, "x", torch.bfloat16)
    M, K = x.shape
    x = _rows_aligned(x, 8)
    xq = _fp8_codes(M, K, x.device) if xq is None else xq
    xs = torch.empty((M,), dtype=torch.float32, device=x.device) if xs is None else xs
    _matrix(xq, "xq", torch.uint8)
    if xq.shape != (M, K):
        raise ValueError(f"xq must have shape {(M, K)}")
    _vector(xs, M, "xs", torch.float32)
    _same_device(x, xq, xs)
    with torch.cuda.device(x.device):
        call("fp8_quant_per_token", x.data_ptr(), M, K, _ld(x), xq.data_ptr(), _ld(xq),
             xs.data_ptr(), _stream(x))
    return xq, xs


def fp8_quant_per_channel(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-output-channel e4m3 quantization of fp32 w [N, K] -> (uint8 [N, K], fp32 [N])."""
    _matrix(w, "w", torch.float32)
    N, K = w.shape
    w = _rows_aligned(w, 4)
    wq = _fp8_codes(N, K, w.device)
    ws = torch.empty((N,), dtype=torch.float32, device=w.device)
    with torch.cuda.device(w.device):
        call("fp8_quant_per_channel", w.data_ptr(), N, K, _ld(w), wq.data_ptr(), _ld(wq),
             ws.data_ptr(), _stream(w))
    return wq, ws


def fp8_quant_prepack_weight(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Online e4m3 quantization of a bf16 or fp32 weight [N, K] into the packed layout."""
    if w.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"w must be bfloat16 or float32, got {w.dtype}")
    _matrix(w, "w", w.dtype)
    N, K = w.shape
    f32 = w.dtype == torch.float32
    w = _rows_aligned(w, 4 if f32 else 8)
    packed = torch.empty((prepack_weight_bytes(N, K),), dtype=torch.uint8, device=w.device)
    ws = torch.empty((N,), dtype=torch.float32, device=w.device)
    with torch.cuda.device(w.device):
        call("fp8_quant_prepack_weight", w.data_ptr(), 0 if f32 else 1, N, K, _ld(w),
             packed.data_ptr(), ws.data_ptr(), _stream(w))
    return packed, ws


def fp8_scaled_mm(xq: torch.Tensor, xs: Optional[torch.Tensor], w_packed: torch.Tensor,
                  ws: Optional[torch.Tensor], N: int, bias: Optional[torch.Tensor] = None,
                  out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                  tile: int = -1) -> torch.Tensor:
    """The e4m3 twin of scaled_mm: xq uint8 e4m3 codes; out_dtype bf16 or fp16 (bias
    of that type), or float32 for the raw fp32 accumulators."""
    _matrix(xq, "xq", torch.uint8)
    M, K = xq.shape
    if out_dtype not in _FP8_OUT_MODE:
        raise TypeError("out_dtype must be torch.bfloat16, torch.float16 or torch.float32")
    mode = _FP8_OUT_MODE[out_dtype]
    if mode != W8A8_OUT_I32:
        _vector(xs, M, "xs", torch.float32)
        _vector(ws, N, "ws", torch.float32)
        _vector(bias, N, "bias", out_dtype)
    _packed(w_packed, N, K)
    out = torch.empty((M, N), dtype=out_dtype, device=xq.device) if out is None else out
    _matrix(out, "out", out_dtype)
    if out.shape != (M, N):
        raise ValueError(f"out must have shape {(M, N)}")

    def ptr(t):
        return None if t is None or mode == W8A8_OUT_I32 else t.data_ptr()

    _same_device(xq, w_packed, out, *((xs, ws, bias) if mode != W8A8_OUT_I32 else ()))
    with torch.cuda.device(xq.device):
        call("fp8_scaled_mm_tile", xq.data_ptr(), _ld(xq), ptr(xs), w_packed.data_ptr(), ptr(ws),
             ptr(bias), M, N, K, mode, out.data_ptr(), _ld(out), _stream(xq), tile)
    return out


def fp8_quant_scaled_mm(x: torch.Tensor, w_packed: torch.Tensor, ws: Optional[torch.Tensor],
                        N: int, bias: Optional[torch.Tensor] = None,
                        out_dtype: torch.dtype = torch.bfloat16,
                        out: Optional[torch.Tensor] = None, tile: int = -1,
                        xq: Optional[torch.Tensor] = None, xs: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """e4m3 per-token quant of bf16 x and the e4m3 scaled matmul: (out, xq, xs).
    out_dtype bf16 or fp16, or float32 for the raw fp32 accumulators."""
    _matrix(x, "x", torch.bfloat16)
    M, K = x.shape
    x = _rows_aligned(x, 8)
    if out_dtype not in _FP8_OUT_MODE:
        raise TypeError("out_dtype must be torch.bfloat16, torch.float16 or torch.float32")
    mode = _FP8_OUT_MODE[out_dtype]
    if mode != W8A8_OUT_I32:
        _vector(ws, N, "ws", torch.float32)
        _vector(bias, N, "bias", out_dtype)
    _packed(w_packed, N, K)
    xq = _fp8_codes(M, K, x.device) if xq is None else xq
    xs = torch.empty((M,), dtype=torch.float32, device=x.device) if xs is None else xs
    _matrix(xq, "xq", torch.uint8)
    if xq.shape != (M, K):
        raise ValueError(f"xq must have shape {(M, K)}")
    _vector(xs, M, "xs", torch.float32)
    out = torch.empty((M, N), dtype=out_dtype, device=x.device) if out is None else out
    _matrix(out, "out", out_dtype)
    if out.shape != (M, N):
        raise ValueError(f"out must have shape {(M, N)}")

    def ptr(t):
        return None if t is None or mode == W8A8_OUT_I32 else t.data_ptr()

    _same_device(x, w_packed, xq, xs, out, *((ws, bias) if mode != W8A8_OUT_I32 else ()))
    with torch.cuda.device(x.device):
        call("fp8_quant_scaled_mm_tile", x.data_ptr(), _ld(x), xq.data_ptr(), _ld(xq),
             xs.data_ptr(), w_packed.data_ptr(), ptr(ws), ptr(bias), M, N, K, mode,
             out.data_ptr(), _ld(out), _stream(x), tile)
    return out, xq, xs


# ---- the microscaled 4-bit (MX FP4) layer ---------------------------------
_DTYPE = {torch.bfloat16: _lib.W8A8_T_BF16, torch.float16: _lib.W8A8_T_F16, torch.float32: _lib.W8A8_T_F32}
_FP4_BLOCK = 32
_entry = {}
# (absent where torch has no GPU support, as every tensor they are called for)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run(x: torch.Tensor, name: str, *args, tile: Tuple[int, ...] = ()) -> None:
    """Call entry point ``name`` with args, x's current stream and tile (behind
    it, where the entry point has one), on x's device.
    (The device is only switched when it is not the current one, and the
    stream is asked for by its handle: a call of a small kernel is short.)"""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(_lib.lib(), name)
    device = x.get_device()
    if device == _current_device():
        rc = fn(*args, _raw_stream(device), *tile)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(device), *tile)
    if rc:
        raise _lib.W8A8Error(rc, name, _lib.last_error())


def _fp4_k(K: int) -> int:
    if K < _FP4_BLOCK or K % _FP4_BLOCK != 0:
        raise ValueError(f"K must be a multiple of {_FP4_BLOCK}, got {K}")
    return K


def _scale_bytes(M: int, n: int, ref: torch.Tensor) -> torch.Tensor:
    """uint8 [M, n] whose rows start on, and are readable to, 16-byte boundaries."""
    if n % 16 == 0:
        return ref.new_empty((M, n), dtype=torch.uint8)
    return ref.new_empty((M, _round_up(n, 16)), dtype=torch.uint8)[:, :n]


def _fp4_rows(xq: torch.Tensor, xs: torch.Tensor) -> Tuple[int, int]:
    """(M, K) of 4-bit codes [M, K/2] and their scale bytes [M, K/32]."""
    _matrix(xq, "xq", torch.uint8)
    _matrix(xs, "xs", torch.uint8)
    M, half = xq.shape
    K = _fp4_k(2 * half)
    if xs.shape != (M, K // _FP4_BLOCK):
        raise ValueError(f"xs must have shape {(M, K // _FP4_BLOCK)}, got {tuple(xs.shape)}")
    if xs.get_device() != xq.get_device():
        _same_device(xq, xs)
    return M, K


def _scale_rows(xs: torch.Tensor) -> torch.Tensor:
    """xs itself when its rows start on 16-byte boundaries and the last one can
    be read to a whole 16 bytes, else a copy into a row-padded buffer."""
    M, n = xs.shape
    ld = _ldp(xs)
    if xs.data_ptr() % 16 == 0 and ld % 16 == 0 and ld >= n and \
            xs.untyped_storage().nbytes() - xs.storage_offset() >= M * ld:
        return xs
    buf = _scale_bytes(M, n, xs)
    buf.copy_(xs)
    return buf


def _ldp(t: torch.Tensor) -> int:
    """Row pitch of byte rows (a single row's: its length to a whole 16 bytes)."""
    return t.stride(0) if t.shape[0] > 1 else _round_up(t.shape[1], 16)


def _float_rows(x: torch.Tensor, name: str) -> Tuple[int, int, int, int]:
    """(element type, M, K, row pitch) of rows x [M, K] of floats."""
    t = _DTYPE.get(x.dtype)
    if t is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {x.dtype}")
    if not x.is_cuda or x.dim() != 2:
        _matrix(x, name, x.dtype)
    M, K = x.shape
    ld, step = x.stride()
    if step != 1 and K > 1:
        _matrix(x, name, x.dtype)
    return t, M, K, (ld if M > 1 else K)


def _vector_rows(x: torch.Tensor, t: int, ld: int) -> Tuple[torch.Tensor, int]:
    """x and its pitch as _rows_aligned gives them: rows on 16-byte boundaries."""
    step = 4 if t == _lib.W8A8_T_F32 else 8
    if x.data_ptr() % 16 == 0 and ld % step == 0:
        return x, ld
    x = _rows_aligned(x, step)
    return x, _ld(x)


def fp4_quant_per_block(x: torch.Tensor, xq: Optional[torch.Tensor] = None,
                        xs: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """MX FP4 quantization of bf16, fp16 or fp32 x [M, K] (K a multiple of 32):
    (uint8 codes [M, K/2], the even element in the low nibble; uint8 scale
    bytes [M, K/32], one power of two per 32 elements)."""
    t, M, K, ld = _float_rows(x, "x")
    _fp4_k(K)
    x, ld = _vector_rows(x, t, ld)
    ldq, lds = K // 2, _round_up(K // _FP4_BLOCK, 16)
    own = xq is None and xs is None
    xq = x.new_empty((M, ldq), dtype=torch.uint8) if xq is None else xq
    xs = _scale_bytes(M, K // _FP4_BLOCK, x) if xs is None else xs
    if not own:
        if _fp4_rows(xq, xs) != (M, K):
            raise ValueError(f"xq must have shape {(M, K // 2)}")
        _same_device(x, xq)
        ldq, lds = _ld(xq), _ld(xs)
    _run(x, "fp4_quant_per_block", x.data_ptr(), t, M, K, ld, xq.data_ptr(), ldq, xs.data_ptr(), lds)
    return xq, xs


def fp4_dequant(xq: torch.Tensor, xs: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values [M, K] that 4-bit codes and scale bytes stand for, rounded
    once to dtype (bf16 and fp32: exact)."""
    if dtype not in _DTYPE:
        raise TypeError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    M, K = _fp4_rows(xq, xs)
    if xq.data_ptr() % 4 != 0 or _ld(xq) % 4 != 0:
        xq = _rows_aligned(xq, 16)
    out = xq.new_empty((M, K), dtype=dtype)
    _run(xq, "fp4_dequant", xq.data_ptr(), _ld(xq), xs.data_ptr(), _ld(xs), M, K, _DTYPE[dtype], out.data_ptr(), K)
    return out


def _fp4_packed(N: int, K: int, device) -> Tuple[torch.Tensor, torch.Tensor]:
    L = _lib.lib()
    w, s = L.fp4_prepack_weight_bytes(N, K), L.fp4_prepack_scale_bytes(N, K)
    if w == 0 or s == 0:
        raise ValueError(f"no packed size for N={N}, K={K}")
    return (torch.empty((w,), dtype=torch.uint8, device=device),
            torch.empty((s,), dtype=torch.uint8, device=device))


def _check_fp4_packed(w_packed: torch.Tensor, s_packed: torch.Tensor, N: int, K: int, ref: torch.Tensor) -> None:
    """The packed buffers of a weight [N, K] (fp4_prepack_weight_bytes and
    fp4_prepack_scale_bytes of include/w8a8.h), on ref's device."""
    if N < 1:
        raise ValueError(f"N must be at least 1, got {N}")
    rows = _round_up(N, 16)

    device = ref.get_device()
    if device < 0 or w_packed.get_device() != device or s_packed.get_device() != device:
        raise ValueError(f"all tensors must be on one GPU, and x is on {ref.device}")
    if w_packed.dtype != torch.uint8 or s_packed.dtype != torch.uint8 or \
            w_packed.numel() < rows * ((K + 127) // 128 * 64) or s_packed.numel() < rows * ((K + 511) // 512 * 16) or \
            not w_packed.is_contiguous() or not s_packed.is_contiguous():
        raise ValueError("w_packed and s_packed must be uint8 device buffers of the packed layout (N, K)")


def fp4_prepack_weight(wq: torch.Tensor, ws: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Repack a weight quantized before, codes [N, K/2] and scale bytes
    [N, K/32], into the two buffers that fp4_scaled_mm reads."""
    N, K = _fp4_rows(wq, ws)
    packed, spacked = _fp4_packed(N, K, wq.device)
    _run(wq, "fp4_prepack_weight", wq.data_ptr(), _ld(wq), ws.data_ptr(), _ld(ws), N, K, packed.data_ptr(),
         spacked.data_ptr())
    return packed, spacked


def fp4_quant_prepack_weight(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Online MX FP4 quantization of a bf16 or fp32 weight [N, K] into the packed
    buffers: the same bytes as fp4_prepack_weight(*fp4_quant_per_block(w))."""
    if w.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"w must be bfloat16 or float32, got {w.dtype}")
    _matrix(w, "w", w.dtype)
    N, K = w.shape[0], _fp4_k(w.shape[1])
    f32 = w.dtype == torch.float32
    w = _rows_aligned(w, 4 if f32 else 8)
    packed, spacked = _fp4_packed(N, K, w.device)
    _run(w, "fp4_quant_prepack_weight", w.data_ptr(), 0 if f32 else 1, N, K, _ld(w), packed.data_ptr(),
         spacked.data_ptr())
    return packed, spacked


def fp4_unpack_weight(w_packed: torch.Tensor, s_packed: torch.Tensor, N: int, K: int
                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Inverse of fp4_prepack_weight: codes [N, K/2] and scale bytes [N, K/32]."""
    _check_fp4_packed(w_packed, s_packed, N, _fp4_k(K), w_packed)
    wq = torch.empty((N, K // 2), dtype=torch.uint8, device=w_packed.device)
    ws = torch.empty((N, K // _FP4_BLOCK), dtype=torch.uint8, device=w_packed.device)
    _run(w_packed, "fp4_unpack_weight", w_packed.data_ptr(), s_packed.data_ptr(), N, K, wq.data_ptr(), K // 2,
         ws.data_ptr(), K // _FP4_BLOCK)
    return wq, ws


def _fp4_out(M: int, N: int, bias, out_dtype, out, x: torch.Tensor):
    """(mode, out), with bias and out checked."""
    mode = _FP8_OUT_MODE.get(out_dtype)
    if mode is None:
        raise TypeError("out_dtype must be torch.bfloat16, torch.float16 or torch.float32")
    if bias is not None:
        if mode == W8A8_OUT_I32:
            raise ValueError("out_dtype=torch.float32 gives the raw sums: bias must be None")
        _vector(bias, N, "bias", out_dtype)
        _same_device(x, bias)
    if out is None:
        return mode, x.new_empty((M, N), dtype=out_dtype)
    _matrix(out, "out", out_dtype)
    if out.shape != (M, N):
        raise ValueError(f"out must have shape {(M, N)}")
    _same_device(x, out)
    return mode, out


def fp4_scaled_mm(xq: torch.Tensor, xs: torch.Tensor, w_packed: torch.Tensor, s_packed: torch.Tensor,
                  N: int, bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                  out: Optional[torch.Tensor] = None, tile: int = -1) -> torch.Tensor:
    """The product [M, N] of MX FP4 rows (codes xq [M, K/2], scale bytes xs
    [M, K/32]) with a packed weight, plus bias, rounded to out_dtype (bf16 or
    fp16; the bias in the same type), or the raw fp32 sums."""
    M, K = _fp4_rows(xq, xs)
    _check_fp4_packed(w_packed, s_packed, N, K, xq)
    mode, out = _fp4_out(M, N, bias, out_dtype, out, xq)
    xq, xs = _rows_aligned(xq, 16), _scale_rows(xs)
    _run(xq, "fp4_scaled_mm_tile", xq.data_ptr(), _ld(xq), xs.data_ptr(), _ldp(xs), w_packed.data_ptr(),
         s_packed.data_ptr(), None if bias is None else bias.data_ptr(), M, N, K, mode, out.data_ptr(), _ld(out),
         tile=(tile,))
    return out


def fp4_quant_scaled_mm(x: torch.Tensor, w_packed: torch.Tensor, s_packed: torch.Tensor, N: int,
                        bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                        out: Optional[torch.Tensor] = None, tile: int = -1
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """fp4_quant_per_block of x [M, K] and fp4_scaled_mm in one call: (out, xq,
    xs). out_dtype defaults to x's type, bf16 for fp32 x."""
    t, M, K, ld = _float_rows(x, "x")
    _fp4_k(K)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if t == _lib.W8A8_T_F32 else x.dtype
    _check_fp4_packed(w_packed, s_packed, N, K, x)
    mode, out = _fp4_out(M, N, bias, out_dtype, out, x)
    x, ld = _vector_rows(x, t, ld)
    xq = x.new_empty((M, K // 2), dtype=torch.uint8)
    xs = _scale_bytes(M, K // _FP4_BLOCK, x)
    _run(x, "fp4_quant_scaled_mm_tile", x.data_ptr(), t, ld, xq.data_ptr(), K // 2, xs.data_ptr(), _ldp(xs),
         w_packed.data_ptr(), s_packed.data_ptr(), None if bias is None else bias.data_ptr(), M, N, K, mode,
         out.data_ptr(), _ld(out), tile=(tile,))
    return out, xq, xs


def _fp4_linear(x: torch.Tensor, w_packed: torch.Tensor, s_packed: torch.Tensor, N: int,
                bias: Optional[torch.Tensor]) -> torch.Tensor:
    """fp4_quant_scaled_mm's out alone, for a layer (which has no use for the codes:
    they go through one buffer)."""
    t, M, K, ld = _float_rows(x, "x")
    _check_fp4_packed(w_packed, s_packed, N, K, x)
    if bias is not None and (bias.dtype != x.dtype or bias.size() != (N,) or not bias.is_contiguous() or
                             bias.get_device() != x.get_device()):
        _vector(bias, N, "bias", x.dtype)
        _same_device(x, bias)
    x, ld = _vector_rows(x, t, ld)
    out = x.new_empty((M, N))
    lds = _round_up(K // _FP4_BLOCK, 16)
    xq = x.new_empty((M * (K // 2 + lds),), dtype=torch.uint8)
    at = xq.data_ptr()
    _run(x, "fp4_quant_scaled_mm", x.data_ptr(), t, ld, at, K // 2, at + M * (K // 2), lds, w_packed.data_ptr(),
         s_packed.data_ptr(), None if bias is None else bias.data_ptr(), M, N, K, _OUT_MODE[x.dtype],
         out.data_ptr(), N)
    return out


def fp4_tile_count() -> int:
    return _lib.lib().w8a8_fp4_tile_count()


def fp4_tile_name(tile: int) -> str:
    return _lib.lib().w8a8_fp4_tile_name(tile).decode()


def fp4_tile_auto(M: int, N: int, K: int) -> int:
    return _lib.lib().w8a8_fp4_tile_auto(M, N, K)


# ---- the block-scaled 8-bit (e4m3) layer ----------------------------------
_SCALE_BLOCK = 128


def _blocks_of(n: int) -> int:
    return -(-n // _SCALE_BLOCK)


def _block_k(K: int) -> int:
    if K < 16 or K > _lib.W8A8_MAX_K or K % 16 != 0:
        raise ValueError(f"K must be a multiple of 16 in [16, {_lib.W8A8_MAX_K}], got {K}")
    return K


def _block_rows(xq: torch.Tensor, xs: torch.Tensor) -> Tuple[int, int]:
    """(M, K) of e4m3 codes [M, K] and their scales [M, ceil(K/128)]."""
    _matrix(xq, "xq", torch.uint8)
    _matrix(xs, "xs", torch.float32)
    M, K = xq.shape
    if xs.shape != (M, _blocks_of(_block_k(K))):
        raise ValueError(f"xs must have shape {(M, _blocks_of(K))}, got {tuple(xs.shape)}")
    if xs.get_device() != xq.get_device():
        _same_device(xq, xs)
    return M, K


def _block_scale_buffer(M: int, n: int, ref: torch.Tensor) -> torch.Tensor:
    """fp32 [M, n] whose rows start on, and are readable to, 16-byte boundaries."""
    if n % 4 == 0:
        return ref.new_empty((M, n), dtype=torch.float32)
    return ref.new_empty((M, _round_up(n, 4)), dtype=torch.float32)[:, :n]


def _block_scale_rows_of(xs: torch.Tensor) -> Tuple[torch.Tensor, int]:
    """xs and its pitch when its rows start on 16-byte boundaries and the last one can
    be read to a whole 16 bytes, else those of a copy into a row-padded buffer."""
    M, n = xs.shape
    ld = xs.stride(0) if M > 1 else _round_up(n, 4)
    if xs.data_ptr() % 16 == 0 and ld % 4 == 0 and ld >= n and \
            xs.untyped_storage().nbytes() // 4 - xs.storage_offset() >= M * ld:
        return xs, ld
    buf = _block_scale_buffer(M, n, xs)
    buf.copy_(xs)
    return buf, _round_up(n, 4)


def fp8_quant_per_block(x: torch.Tensor, xq: Optional[torch.Tensor] = None,
                        xs: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Block-scaled quantization of bf16, fp16 or fp32 x [M, K] (K a multiple of
    16): (uint8 e4m3 codes [M, K], fp32 scales [M, ceil(K/128)], one per 128
    elements)."""
    t, M, K, ld = _float_rows(x, "x")
    _block_k(K)
    x, ld = _vector_rows(x, t, ld)
    ldq, lds = K, _round_up(_blocks_of(K), 4)
    own = xq is None and xs is None
    xq = x.new_empty((M, K), dtype=torch.uint8) if xq is None else xq
    xs = _block_scale_buffer(M, _blocks_of(K), x) if xs is None else xs
    if not own:
        if _block_rows(xq, xs) != (M, K):
            raise ValueError(f"xq must have shape {(M, K)}")
        _same_device(x, xq)
        ldq, lds = _ld(xq), _ld(xs)
    _run(x, "fp8_quant_per_block", x.data_ptr(), t, M, K, ld, xq.data_ptr(), ldq, xs.data_ptr(), lds)
    return xq, xs


def fp8_block_dequant(xq: torch.Tensor, xs: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values [M, K] that e4m3 codes and block scales stand for: code * scale in fp32, rounded to dtype."""
    if dtype not in _DTYPE:
        raise TypeError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    M, K = _block_rows(xq, xs)
    at, ld = xq.data_ptr(), xq.stride(0) if M > 1 else K
    if at % 8 != 0 or ld % 8 != 0:
        xq = _rows_aligned(xq, 16)
        at, ld = xq.data_ptr(), _ld(xq)
    out = xq.new_empty((M, K), dtype=dtype)
    _run(xq, "fp8_block_dequant", at, ld, xs.data_ptr(), xs.stride(0) if M > 1 else xs.shape[1], M, K,
         _DTYPE[dtype], out.data_ptr(), K)
    return out


def _matrices(w: torch.Tensor) -> Tuple[torch.Tensor, int]:
    """w [N, K] or [E, N, K] and the pitch of its rows, one matrix behind the other; a
    copy where the strides are no such pitch, or rows overlap (those of an expanded
    tensor are one row of memory)."""
    N, K = w.shape[-2:]
    E = w.shape[0] if w.dim() == 3 else 1
    ld = w.stride(-2) if N > 1 else w.stride(0) if E > 1 else K
    if w.stride(-1) != 1 or ld < K or (E > 1 and w.stride(0) != N * ld):
        return w.clone(memory_format=torch.contiguous_format), K
    return w, ld


def _block_weights(w: torch.Tensor, name: str, gated: bool) -> Tuple[torch.Tensor, int, int, int, int]:
    """(w, its row pitch, E, N, K) of a weight [N, K], or of experts' weights [E, N, K]."""
    if not w.is_cuda:
        raise ValueError(f"{name} must be a device tensor, got {w.device}")
    if w.dim() not in (2, 3):
        raise ValueError(f"{name} must be [N, K] or [E, N, K], got shape {tuple(w.shape)}")
    N, K = w.shape[-2:]
    E = w.shape[0] if w.dim() == 3 else 1
    _block_k(K)
    if N < 1 or E < 1 or (gated and N % 32 != 0):
        raise ValueError(f"{name}: no packed form of shape {tuple(w.shape)}"
                         f"{' (gated: N must be a multiple of 32)' if gated else ''}")
    w, ld = _matrices(w)
    return w, ld, E, N, K


def _block_packed(E: int, N: int, K: int, ref: torch.Tensor) -> torch.Tensor:
    n = _lib.lib().fp8_block_prepack_weight_bytes(E, N, K)
    if n == 0:
        raise ValueError(f"no packed size for E={E}, N={N}, K={K}")
    return ref.new_empty((n,), dtype=torch.uint8)


def _block_scale_rows(N: int, gated: bool) -> int:
    return 2 * _blocks_of(N // 2) if gated else _blocks_of(N)


def fp8_block_prepack_weight(wq: torch.Tensor, gated: bool = False) -> torch.Tensor:
    """Repack e4m3 codes [N, K] (uint8), or [E, N, K] of experts, into the layout
    that fp8_block_scaled_mm reads. gated: a matrix holds the gate rows, then
    as many up rows (the first weight of fp8_block_experts)."""
    if wq.dtype != torch.uint8:
        raise TypeError(f"wq must be torch.uint8, got {wq.dtype}")
    wq, ld, E, N, K = _block_weights(wq, "wq", gated)
    packed = _block_packed(E, N, K, wq)
    _run(wq, "fp8_block_prepack_weight", wq.data_ptr(), ld, E, N, K, int(gated), packed.data_ptr())
    return packed


def fp8_block_quant_prepack_weight(w: torch.Tensor, gated: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Online quantization of a bf16 or fp32 weight [N, K] ([E, N, K]) in blocks of
    128 x 128: (packed codes, fp32 scales [ceil(N/128), ceil(K/128)]; of each
    expert, and of a gated weight [2*ceil(N/2/128), ceil(K/128)])."""
    if w.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"w must be bfloat16 or float32, got {w.dtype}")
    w, ld, E, N, K = _block_weights(w, "w", gated)
    f32 = w.dtype == torch.float32
    if w.data_ptr() % 16 != 0 or ld % (4 if f32 else 8) != 0:
        w, ld = w.clone(memory_format=torch.contiguous_format), K
    packed = _block_packed(E, N, K, w)
    shape = (_block_scale_rows(N, gated), _blocks_of(K))
    ws = w.new_empty(shape if w.dim() == 2 else (E, *shape), dtype=torch.float32)
    _run(w, "fp8_block_quant_prepack_weight", w.data_ptr(), 0 if f32 else 1, ld, E, N, K, int(gated),
         packed.data_ptr(), ws.data_ptr())
    return packed, ws


def _check_block_packed(w_packed: torch.Tensor, ws: torch.Tensor, N: int, K: int, ref: torch.Tensor) -> None:
    """The packed buffer and scales of a weight [N, K], on ref's device."""
    if N < 1:
        raise ValueError(f"N must be at least 1, got {N}")
    device = ref.get_device()
    if device < 0 or w_packed.get_device() != device or ws.get_device() != device:
        raise ValueError(f"all tensors must be on one GPU, and x is on {ref.device}")
    if w_packed.dtype != torch.uint8 or w_packed.numel() < _round_up(N, 16) * _round_up(K, 128) or \
            not w_packed.is_contiguous():
        raise ValueError("w_packed must be a uint8 device buffer of the packed layout (N, K)")
    if ws.dtype != torch.float32 or ws.shape != (_blocks_of(N), _blocks_of(K)) or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous fp32 {(_blocks_of(N), _blocks_of(K))}, got {ws.dtype} "
                         f"{tuple(ws.shape)}")


def fp8_block_unpack_weight(w_packed: torch.Tensor, N: int, K: int, gated: bool = False,
                            experts: Optional[int] = None) -> torch.Tensor:
    """Inverse of fp8_block_prepack_weight: codes [N, K], or [experts, N, K]."""
    E = 1 if experts is None else experts
    n = _lib.lib().fp8_block_prepack_weight_bytes(E, N, _block_k(K))
    if n == 0 or (gated and N % 32 != 0):
        raise ValueError(f"no packed size for E={E}, N={N}, K={K}")
    if not w_packed.is_cuda or w_packed.dtype != torch.uint8 or w_packed.numel() < n or not w_packed.is_contiguous():
        raise ValueError("w_packed must be a uint8 device buffer of the packed layout (N, K)")
    wq = w_packed.new_empty((N, K) if experts is None else (E, N, K))
    _run(w_packed, "fp8_block_unpack_weight", w_packed.data_ptr(), E, N, K, int(gated), wq.data_ptr(), K)
    return wq


def fp8_block_scaled_mm(xq: torch.Tensor, xs: torch.Tensor, w_packed: torch.Tensor, ws: torch.Tensor, N: int,
                        bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                        out: Optional[torch.Tensor] = None, tile: int = -1) -> torch.Tensor:
    """The product [M, N] of block-scaled rows (e4m3 codes xq [M, K], scales xs
    [M, ceil(K/128)]) with a packed weight and its scales ws [ceil(N/128),
    ceil(K/128)], plus bias, rounded to out_dtype (bf16 or fp16; the bias in the
    same type), or the raw fp32 sums."""
    M, K = _block_rows(xq, xs)
    _check_block_packed(w_packed, ws, N, K, xq)
    mode, out = _fp4_out(M, N, bias, out_dtype, out, xq)
    xq, (xs, lds) = _rows_aligned(xq, 16), _block_scale_rows_of(xs)
    _run(xq, "fp8_block_scaled_mm_tile", xq.data_ptr(), _ld(xq), xs.data_ptr(), lds, w_packed.data_ptr(),
         ws.data_ptr(), None if bias is None else bias.data_ptr(), M, N, K, mode, out.data_ptr(), _ld(out),
         tile=(tile,))
    return out


def fp8_block_quant_scaled_mm(x: torch.Tensor, w_packed: torch.Tensor, ws: torch.Tensor, N: int,
                              bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                              out: Optional[torch.Tensor] = None, tile: int = -1
                              ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """fp8_quant_per_block of x [M, K] and fp8_block_scaled_mm in one call: (out,
    xq, xs). out_dtype defaults to x's type, bf16 for fp32 x."""
    t, M, K, ld = _float_rows(x, "x")
    _block_k(K)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if t == _lib.W8A8_T_F32 else x.dtype
    _check_block_packed(w_packed, ws, N, K, x)
    mode, out = _fp4_out(M, N, bias, out_dtype, out, x)
    x, ld = _vector_rows(x, t, ld)
    xq = x.new_empty((M, K), dtype=torch.uint8)
    xs = _block_scale_buffer(M, _blocks_of(K), x)
    lds = _round_up(_blocks_of(K), 4)
    _run(x, "fp8_block_quant_scaled_mm_tile", x.data_ptr(), t, ld, xq.data_ptr(), K, xs.data_ptr(), lds,
         w_packed.data_ptr(), ws.data_ptr(), None if bias is None else bias.data_ptr(), M, N, K, mode, out.data_ptr(),
         _ld(out), tile=(tile,))
    return out, xq, xs


def _fp8_block_linear(x: torch.Tensor, w_packed: torch.Tensor, ws: torch.Tensor, N: int,
                      bias: Optional[torch.Tensor]) -> torch.Tensor:
    """fp8_block_quant_scaled_mm's out alone, for a layer (which has no use for the
    codes: they go through one buffer)."""
    t, M, K, ld = _float_rows(x, "x")
    _check_block_packed(w_packed, ws, N, K, x)
    if bias is not None and (bias.dtype != x.dtype or bias.size() != (N,) or not bias.is_contiguous() or
                             bias.get_device() != x.get_device()):
        _vector(bias, N, "bias", x.dtype)
        _same_device(x, bias)
    x, ld = _vector_rows(x, t, ld)
    out = x.new_empty((M, N))
    lds = _round_up(_blocks_of(K), 4)
    xq = x.new_empty((M * (K + 4 * lds),), dtype=torch.uint8)
    at = xq.data_ptr()
    _run(x, "fp8_block_quant_scaled_mm", x.data_ptr(), t, ld, at, K, at + M * K, lds, w_packed.data_ptr(),
         ws.data_ptr(), None if bias is None else bias.data_ptr(), M, N, K, _OUT_MODE[x.dtype], out.data_ptr(), N)
    return out


def fp8_block_tile_count() -> int:
    return _lib.lib().w8a8_fp8_block_tile_count()


def fp8_block_tile_name(tile: int) -> str:
    return _lib.lib().w8a8_fp8_block_tile_name(tile).decode()


def fp8_block_tile_auto(M: int, N: int, K: int) -> int:
    return _lib.lib().w8a8_fp8_block_tile_auto(M, N, K)


# ---- a mixture of experts -------------------------------------------------
@dataclass(eq=False)
class Routing:
    """How a router's logits choose top_k experts for each token:

        score  = softmax(logits) or sigmoid(logits)             score "softmax" or "sigmoid"
        choice = score + bias                                   bias fp32 [E] or None
        groups > 1: the experts stand in equal groups; a group's worth is the sum
        of its group_top (1 or 2) largest choices; the top_groups best stay
        ids = the top_k best choices, best first, ties to the lowest index
        weights = their scores, over their sum (renormalize), times scale

    Experts whose logit (or bias) is NaN or -infinity are left out; a row with
    fewer than top_k left ends in ids -1 with weight 0."""
    top_k: int
    score: str = "softmax"
    bias: Optional[torch.Tensor] = None
    groups: int = 1
    top_groups: int = 1
    group_top: int = 2
    renormalize: bool = True
    scale: float = 1.0


_SCORE = {"softmax": _lib.W8A8_SCORE_SOFTMAX, "sigmoid": _lib.W8A8_SCORE_SIGMOID}


def route_experts(logits: torch.Tensor, routing: Routing) -> Tuple[torch.Tensor, torch.Tensor]:
    """The experts of each token by its logits [T, E] (bf16, fp16 or fp32; E up to
    1024): (int32 ids [T, top_k], fp32 weights [T, top_k])."""
    t, T, E, ld = _float_rows(logits, "logits")
    r = routing
    score = _SCORE.get(r.score)
    if score is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {r.score!r}")
    bias = r.bias
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (E,) or not bias.is_contiguous() or
                             bias.get_device() != logits.get_device()):
        raise ValueError(f"bias must be contiguous fp32 [{E}] on {logits.device}")
    if r.top_k < 1:
        raise ValueError(f"top_k must be at least 1, got {r.top_k}")
    if ld < E:                                         # rows overlap, as those of an expanded tensor do
        logits, ld = logits.contiguous(), E
    ids = logits.new_empty((T, r.top_k), dtype=torch.int32)
    weights = logits.new_empty((T, r.top_k), dtype=torch.float32)
    how = _lib.ROUTING_STRUCT.pack(0 if bias is None else bias.data_ptr(), score, r.top_k, r.groups, r.top_groups,
                                   r.group_top, int(r.renormalize), r.scale)
    _run(logits, "route_experts", logits.data_ptr(), t, ld, T, E, how, ids.data_ptr(), weights.data_ptr())
    return ids, weights


def fp8_block_experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate_up: torch.Tensor,
                      gate_up_scale: torch.Tensor, down: torch.Tensor, down_scale: torch.Tensor, inner: int,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A mixture of experts over tokens x [T, K] (bf16, fp16 or fp32), in x's type:

        out[t] = sum over j of weights[t, j] * down_e(silu(gate_e x[t]) * up_e x[t]),   e = ids[t, j]

    ids int32 and weights fp32 [T, top_k] (route_experts' results); an id outside
    [0, E) stands for no expert. gate_up: fp8_block_prepack_weight of codes
    [E, 2 * inner, K] (gated), gate_up_scale [E, 2*ceil(inner/128), ceil(K/128)];
    down: of codes [E, K, inner], down_scale [E, ceil(K/128), ceil(inner/128)].
    x and the inner rows pass through fp8_quant_per_block's codes."""
    t, T, K, ld = _float_rows(x, "x")
    device = x.get_device()
    _block_k(K)
    _block_k(inner)
    if ids.dim() != 2 or ids.shape[0] != T or weights.shape != ids.shape:
        raise ValueError(f"ids and weights must be [{T}, top_k], got {tuple(ids.shape)} and {tuple(weights.shape)}")
    if ids.dtype != torch.int32 or weights.dtype != torch.float32:
        raise TypeError(f"ids must be int32 and weights fp32, got {ids.dtype} and {weights.dtype}")
    for name, s in (("gate_up_scale", gate_up_scale), ("down_scale", down_scale)):
        if s.dtype != torch.float32 or s.dim() != 3 or not s.is_contiguous():
            raise ValueError(f"{name} must be contiguous fp32 [E, rows, blocks]")
    E = gate_up_scale.shape[0]
    if E < 1 or gate_up_scale.shape[1:] != (2 * _blocks_of(inner), _blocks_of(K)) or \
            down_scale.shape != (E, _blocks_of(K), _blocks_of(inner)):
        raise ValueError(f"scales {tuple(gate_up_scale.shape)} and {tuple(down_scale.shape)} do not belong to "
                         f"experts of K={K}, inner={inner}")
    for name, w, least in (("gate_up", gate_up, 2 * inner * _round_up(K, 128)),
                           ("down", down, K * _round_up(inner, 128))):
        if w.dtype != torch.uint8 or w.numel() < E * least or not w.is_contiguous():
            raise ValueError(f"{name} must be a uint8 device buffer of the packed layout")
    for o in (ids, weights, gate_up, gate_up_scale, down, down_scale):
        if o.get_device() != device:
            _same_device(x, o)
    ids, weights = ids.contiguous(), weights.contiguous()
    x, ld = _vector_rows(x, t, ld)
    if out is None:
        out = r = x.new_empty((T, K))
    else:
        _matrix(out, "out", x.dtype)
        if out.shape != (T, K):
            raise ValueError(f"out must have shape {(T, K)}")
        _same_device(x, out)
        step = 4 if t == _lib.W8A8_T_F32 else 8
        r = out if out.data_ptr() % 16 == 0 and _ld(out) % step == 0 else x.new_empty((T, K))
    top_k = ids.shape[1]
    need = _lib.lib().fp8_block_experts_workspace_bytes(T, K, inner, E, top_k)
    if need == 0 and T > 0:
        raise ValueError(f"out of range: {T} tokens, {E} experts, top_k {top_k}")
    work = x.new_empty((need,), dtype=torch.uint8)
    layer = _lib.EXPERTS_STRUCT.pack(gate_up.data_ptr(), gate_up_scale.data_ptr(), down.data_ptr(),
                                     down_scale.data_ptr(), K, inner, E)
    _run(x, "fp8_block_experts", layer, x.data_ptr(), t, ld, T, ids.data_ptr(), weights.data_ptr(), top_k,
         r.data_ptr(), _ld(r), work.data_ptr(), need)
    if r is not out:
        out.copy_(r)
    return out


def fp8_tile_count() -> int:
    return _lib.lib().w8a8_fp8_tile_count()


def tile_count() -> int:
    return _lib.lib().w8a8_mm_tile_count()


def tile_name(tile: int) -> str:
    return _lib.lib().w8a8_mm_tile_name(tile).decode()


def tile_auto(M: int, N: int, K: int) -> int:
    return _lib.lib().w8a8_mm_tile_auto(M, N, K)


def device_supported(device: int = 0) -> bool:
    return bool(_lib.lib().w8a8_device_supported(device))


# ---- norms around a layer -------------------------------------------------
@dataclass(eq=False)
class Norm:
    """A norm over the last dimension and its vectors:

        n(v) = v / sqrt(mean(v^2) + eps)                        kind "rms"
        n(v) = (v - mean(v)) / sqrt(var(v) + eps)               kind "layer"
        (n(v) * weight + bias) * (1 + scale) + shift

    weight, bias: [K]. scale, shift: [K], or [G, K] for rows in G equal groups
    (row m of M takes vector m // (M // G): images of a batch, or tokens with
    a vector each). bf16, fp16 or fp32, weight and bias in one type, scale and
    shift in one type; the last dimension contiguous."""
    kind: str = "rms"
    weight: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None
    scale: Optional[torch.Tensor] = None
    shift: Optional[torch.Tensor] = None
    eps: float = 1e-6


_NORM_KIND = {"rms": _lib.W8A8_NORM_RMS, "layer": _lib.W8A8_NORM_LAYER}
_CODE_TYPE = {_lib.W8A8_NORM_OUT_INT8: torch.int8, _lib.W8A8_NORM_OUT_FP8: torch.uint8}


def _groups(t: torch.Tensor, M: int, K: int, ref: torch.Tensor, name: str) -> Tuple[int, int]:
    """(groups, leading dimension) of a vector per group, [K] or [G, K]."""
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    shape = t.shape
    if len(shape) not in (1, 2) or shape[-1] != K or (K > 1 and t.stride(-1) != 1) or \
            t.get_device() != ref.get_device():
        raise ValueError(f"{name} must be [{K}] or [G, {K}] on {ref.device} with a contiguous last dimension")
    if len(shape) == 1:
        return 1, K
    G = shape[0]
    if M == 0:                                         # any number of groups, as none has a row
        return 1, K
    if G < 1 or M % G != 0:
        raise ValueError(f"{M} rows do not split into the {G} rows of {name}")
    return G, (t.stride(0) if G > 1 else K)


def _norm_struct(n: Norm, M: int, K: int, ref: torch.Tensor) -> bytes:
    """The w8a8_norm_t of n for rows [M, K]."""
    kind = _NORM_KIND.get(n.kind)
    if kind is None:
        raise ValueError(f"kind must be 'rms' or 'layer', got {n.kind!r}")
    weight = bias = scale = shift = ld_scale = ld_shift = vec = mod = 0
    groups = 1
    if n.weight is not None or n.bias is not None:
        for name, t in (("weight", n.weight), ("bias", n.bias)):
            if t is not None:
                if t.dim() != 1:
                    raise ValueError(f"{name} must be [{K}], got shape {tuple(t.shape)}")
                _groups(t, M, K, ref, name)
        if n.weight is not None:
            weight, vec = n.weight.data_ptr(), _DTYPE[n.weight.dtype]
        if n.bias is not None:
            bias, kind_of = n.bias.data_ptr(), _DTYPE[n.bias.dtype]
            if weight and kind_of != vec:
                raise TypeError("weight and bias must have one type")
            vec = kind_of
    if n.scale is not None:
        groups, ld_scale = _groups(n.scale, M, K, ref, "scale")
        scale, mod = n.scale.data_ptr(), _DTYPE[n.scale.dtype]
    if n.shift is not None:
        G, ld_shift = _groups(n.shift, M, K, ref, "shift")
        if n.scale is not None:
            if G != groups:
                raise ValueError("scale and shift must have the same number of rows")
            if n.scale.dtype != n.shift.dtype:
                raise TypeError("scale and shift must have one type")
        groups, shift, mod = G, n.shift.data_ptr(), _DTYPE[n.shift.dtype]
    return _lib.NORM_STRUCT.pack(kind, n.eps, weight, bias, scale, shift, ld_scale, ld_shift, groups, vec, mod)


def _norm_out(M: int, K: int, act: torch.dtype, kind: int, x: torch.Tensor):
    """(out, its leading dimension, scales or None) of a norm."""
    if kind == _lib.W8A8_NORM_OUT_16:
        return x.new_empty((M, K), dtype=act), K, None
    ld = _round_up(K, 16)
    codes = x.new_empty((M, ld), dtype=_CODE_TYPE[kind])
    return codes if ld == K else codes[:, :K], ld, x.new_empty((M,), dtype=torch.float32)


def _norm_call(x: torch.Tensor, norm: Norm, kind: int, out_dtype: Optional[torch.dtype]):
    t, M, K, ldx = _float_rows(x, "x")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if t == _lib.W8A8_T_F32 else x.dtype
    elif out_dtype not in _ACT_ENTRY or (t != _lib.W8A8_T_F32 and out_dtype != x.dtype):
        raise TypeError(f"out_dtype must be {'bfloat16 or float16' if t == _lib.W8A8_T_F32 else x.dtype}")
    n = _norm_struct(norm, M, K, x)
    out, ld, scales = _norm_out(M, K, out_dtype, kind, x)
    _run(x, "norm_rows", x.data_ptr(), t, M, K, ldx, n, _DTYPE[out_dtype], kind, out.data_ptr(), ld,
         None if scales is None else scales.data_ptr())
    return out, scales


def norm(x: torch.Tensor, norm: Norm, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """The norm of each row of x [M, K] (bf16, fp16 or fp32) in x's type; of fp32
    x in out_dtype (bf16, the default, or fp16)."""
    return _norm_call(x, norm, _lib.W8A8_NORM_OUT_16, out_dtype)[0]


def norm_quant_per_token(x: torch.Tensor, norm: Norm) -> Tuple[torch.Tensor, torch.Tensor]:
    """The norm of each row of x [M, K] as int8 codes and fp32 scales [M], the
    operands of scaled_mm: quant_per_token's rule on the fp32 norm."""
    return _norm_call(x, norm, _lib.W8A8_NORM_OUT_INT8, None)


def fp8_norm_quant_per_token(x: torch.Tensor, norm: Norm) -> Tuple[torch.Tensor, torch.Tensor]:
    """The e4m3 twin of norm_quant_per_token: uint8 e4m3 codes and fp32 scales."""
    return _norm_call(x, norm, _lib.W8A8_NORM_OUT_FP8, None)


def _residual_call(x: torch.Tensor, y: torch.Tensor, norm: Optional[Norm], kind: int,
                   gate: Optional[torch.Tensor], post: Optional[Norm], residual_scale: float,
                   branch_scale: float, out: Optional[torch.Tensor]):
    _matrix(y, "y", _act_dtype(y))
    if x.dtype != y.dtype and x.dtype != torch.float32:
        raise TypeError(f"x must be {y.dtype} (y's type) or float32, got {x.dtype}")
    t, M, K, ldx = _float_rows(x, "x")
    if y.shape != (M, K):
        raise ValueError(f"y must have shape {(M, K)}, got {tuple(y.shape)}")
    if y.get_device() != x.get_device():
        _same_device(x, y)
    if out is None:
        r, ldr = x.new_empty((M, K)), K
    else:
        r = _matrix(out, "out", x.dtype)
        if r.shape != (M, K):
            raise ValueError(f"out must have shape {(M, K)}")
        _same_device(x, r)
        ldr = _ld(r)
    groups, ld_gate, gate_ptr, gate_dtype = 1, 0, 0, 0
    if gate is not None:
        groups, ld_gate = _groups(gate, M, K, x, "gate")
        gate_ptr, gate_dtype = gate.data_ptr(), _DTYPE[gate.dtype]
    p = n = None
    if post is not None:
        if post.scale is not None or post.shift is not None:
            raise ValueError("post takes no scale or shift: the gate multiplies its result")
        p = _norm_struct(post, M, K, x)
    h, ld, hs = None, 0, None
    if norm is not None:
        n = _norm_struct(norm, M, K, x)
        h, ld, hs = _norm_out(M, K, y.dtype, kind, x)
    res = _lib.RESIDUAL_STRUCT.pack(x.data_ptr(), y.data_ptr(), r.data_ptr(), ldx, y.stride(0) if M > 1 else K, ldr,
                                    gate_ptr, ld_gate, groups, residual_scale, branch_scale, t, _DTYPE[y.dtype],
                                    gate_dtype)
    _run(x, "gated_residual_rows", res, p, M, K, n, kind, None if h is None else h.data_ptr(), ld,
         None if hs is None else hs.data_ptr())
    return r, h, hs


def gated_residual(x: torch.Tensor, y: torch.Tensor, gate: Optional[torch.Tensor] = None,
                   post: Optional[Norm] = None, residual_scale: float = 1.0, branch_scale: float = 1.0,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A block's output y [M, K] (bf16 or fp16) back into the residual stream x
    (y's type or fp32): residual_scale * x + branch_scale * gate * post(y), in
    x's type. gate: [K] or [G, K] as a Norm's scale (None: 1). post: a Norm
    with weight and bias, or None (y itself). out may be x itself; otherwise it
    shares no memory with the other tensors."""
    return _residual_call(x, y, None, _lib.W8A8_NORM_OUT_16, gate, post, residual_scale, branch_scale, out)[0]


def gated_residual_norm(x: torch.Tensor, y: torch.Tensor, norm: Norm, gate: Optional[torch.Tensor] = None,
                        post: Optional[Norm] = None, residual_scale: float = 1.0, branch_scale: float = 1.0,
                        out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """gated_residual and the next block's norm in one pass: (r, norm(r) in y's
    type). The norm sees r before its rounding to x's type."""
    return _residual_call(x, y, norm, _lib.W8A8_NORM_OUT_16, gate, post, residual_scale, branch_scale, out)[:2]


def gated_residual_norm_quant(x: torch.Tensor, y: torch.Tensor, norm: Norm,
                              gate: Optional[torch.Tensor] = None, post: Optional[Norm] = None,
                              residual_scale: float = 1.0, branch_scale: float = 1.0,
                              out: Optional[torch.Tensor] = None
                              ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """gated_residual_norm with the norm as int8 codes and fp32 scales, the
    operands of scaled_mm: (r, codes, scales)."""
    return _residual_call(x, y, norm, _lib.W8A8_NORM_OUT_INT8, gate, post, residual_scale, branch_scale, out)


def fp8_gated_residual_norm_quant(x: torch.Tensor, y: torch.Tensor, norm: Norm,
                                  gate: Optional[torch.Tensor] = None, post: Optional[Norm] = None,
                                  residual_scale: float = 1.0, branch_scale: float = 1.0,
                                  out: Optional[torch.Tensor] = None
                                  ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The e4m3 twin of gated_residual_norm_quant: (r, uint8 e4m3 codes, scales)."""
    return _residual_call(x, y, norm, _lib.W8A8_NORM_OUT_FP8, gate, post, residual_scale, branch_scale, out)
