"""How near the mixture of experts comes to its definition in 64 bits, on every path: the codes of
its inner rows one by one, and outputs in norm and by tests/experts_reference.py's bounds.
tests/test_experts_accuracy_cpu.py shows what these checks tell apart."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import block_reference as ref
from tests import experts_reference as tight
from tests.test_experts_accuracy_cpu import CASES, INNER_CASES, case_of, inner_case_of, make, rows
from tests.test_gpu_fp8_block import DEV, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w8a8_int8_dynamic_amd import _lib
    from w8a8_int8_dynamic_amd import ops as _ops
    assert _ops.device_supported(torch.cuda.current_device()), _lib.last_error()
    return _ops


def layer_of(parts):
    from w8a8_int8_dynamic_amd import W8A8Experts
    return W8A8Experts.from_quantized(*(dev(p) for p in parts))


def outputs(ops, layer, x, ids, w):
    """In fp32, of 16-bit x; those in x's type are that rounded once."""
    args = x.to(DEV), dev(ids), dev(w)
    f = ops.fp8_block_experts(args[0].float(), *args[1:], layer.gate_up, layer.gate_up_scale, layer.down,
                              layer.down_scale, layer.inner)
    assert torch.equal(layer(*args), f.to(x.dtype))
    return f.double().cpu().numpy()


def values(kind, n, k, r):
    """Codes of rows that are random codes, normal values, or normal values with some columns 20 times as large."""
    if kind == "codes":
        q = r.integers(0, 256, (n, k), dtype=np.uint8)
        return np.where((q & 127) == 127, q ^ 1, q).astype(np.uint8)
    return ref.quant(r.standard_normal((n, k)) * np.where(r.random(k) < (0.02 if kind == "outliers" else 0), 20, 1))[0]


@pytest.mark.parametrize("kind", ["codes", "normal", "outliers"])
def test_instruction(ops, kind):
    """Sums of every tile are the instruction's as tests/experts_reference.py follows it, to fp32's rounding
    of their 16 groups a block, the blocks and the scales' products; and so far from exact ones as csrc/
    fp8_block_device.hpp says."""
    m, n, k = 70, 144, 656
    r = np.random.default_rng(9)
    xq, wq = values(kind, m, k, r), values("codes" if kind == "codes" else "normal", n, k, r)
    xs = (2.0 ** r.uniform(-9, -5, (m, ref.blocks_of(k)))).astype(np.float32)
    ws = (2.0 ** r.uniform(-12, -8, (ref.blocks_of(n), ref.blocks_of(k)))).astype(np.float32)
    want, x, w = tight.instruction_product(xq, xs, wq, ws, DEV), ref.dequant(xq, xs), ref.weight(wq, ws)
    bound = (16 + ref.blocks_of(k) + 4) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    packed = ops.fp8_block_prepack_weight(dev(wq))
    for tile in range(ops.fp8_block_tile_count()):
        y = ops.fp8_block_scaled_mm(dev(xq), dev(xs), packed, dev(ws), n, out_dtype=torch.float32, tile=tile)
        assert (np.abs(y.double().cpu().numpy() - want) <= bound).all(), ops.fp8_block_tile_name(tile)
    off = np.sqrt(np.mean((want - x @ w.T) ** 2 / ((x ** 2) @ (w ** 2).T)))
    print(f"{kind}: {off:.2g} of the sums' rms", flush=True)
    assert off < 2.0 ** -13


def held(y, x, ids, w, parts, exact):
    """Outputs y are near enough to the definition, in norm and elementwise."""
    want, bound = tight.experts(x.float().numpy(), ids, w, parts, exact, device=DEV)
    off, limit = tight.token_error(y, want), tight.norm_limit(ids.size * (parts[0].shape[1] // 2))
    print(f"off by {off:.2g} of {limit:.2g}, of the bound {(np.abs(y - want) / np.maximum(bound, 1e-300)).max():.2g}",
          flush=True)
    assert off <= limit and (np.abs(y - want) <= bound).all()
    assert (y[((ids < 0) | (ids >= len(parts[0]))).all(1)] == 0).all()


@pytest.mark.parametrize("t,e,sets", INNER_CASES)
def test_inner_codes(ops, t, e, sets):
    """The inner rows' codes, handed through a diagonal down weight: as many differ from those of the form's
    sums in 64 bits as fp32 sums explain, four standard deviations of that and four more at most."""
    parts, xs, ids, w = inner_case_of(t, e, sets)
    layer, exact = layer_of(parts), tight.is_exact(t, 1, e)
    differ = total = expected = 0
    for x, i in zip(xs, ids):
        y = outputs(ops, layer, x, i, w)
        assert (y[:, layer.inner:] == 0).all()
        for n in range(e):
            mine = i[:, 0] == n
            if not mine.any():
                continue
            xq, s = ref.quant(x.float().numpy()[mine])
            gu = parts[0][n], parts[1][n]
            g, u = tight.gated_sums(xq, s, *gu, exact, DEV)
            q, s_h = tight.inner_codes(ref.silu(g) * u)
            differ += (tight.codes_of(y[mine, :layer.inner] / 448, s_h) != q).sum()
            total += q.size
            expected += tight.crossings(g, u, *(tight.SUMS * m for m in tight.magnitudes(xq, s, *gu)[1]))
    print(f"{differ} of {total} differ, {expected:.1f} expected at most", flush=True)
    assert total >= 100000 and differ <= expected + 4 * np.sqrt(expected) + 4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("name", list(CASES))
def test_outputs(ops, name, dtype):
    parts, x, ids, w = case_of(name, dtype)
    t, e, top_k = CASES[name][:3]
    held(outputs(ops, layer_of(parts), x, ids, w), x, ids, w, parts, tight.is_exact(t, top_k, e))


def test_outputs_of_single_tokens(ops):
    """Slots alone, without a plan, one to four tokens a call."""
    parts, x, ids, w = case_of("few rows", torch.bfloat16)
    layer, y, at = layer_of(parts), [], 0
    while at < len(ids):
        n = 1 + at % 4
        y.append(outputs(ops, layer, x[at:at + n], ids[at:at + n], w[at:at + n]))
        at += n
    held(np.concatenate(y), x, ids, w, parts, True)


def test_outputs_of_several_passes(ops):
    """More than 65536 slots: 500 of the tokens, from every pass."""
    parts, x, ids, w = case_of("many rows", torch.bfloat16)
    times = 70000 // ids.size + 1
    g = np.random.default_rng(5)
    order = g.permutation(len(ids) * times) % len(ids)
    y = outputs(ops, layer_of(parts), x[order], ids[order], w[order])
    some = g.permutation(len(order))[:500]
    held(y[some], x[order[some]], ids[order[some]], w[order[some]], parts, False)


@pytest.mark.parametrize("name", ["few rows", "some rows", "a dozen rows", "dozens of rows", "many rows"])
def test_outputs_of_any_ids(ops, name):
    """Slots without an expert, the same expert twice, all slots one expert."""
    parts, x, ids, w = case_of(name, torch.bfloat16)
    t, e, top_k = CASES[name][:3]
    layer, g = layer_of(parts), np.random.default_rng(6)
    free = g.integers(-1, e + 1, ids.shape).astype(np.int32)
    free[:3] = -1
    for i in (free, np.repeat(ids[:, :1], top_k, 1), np.full_like(ids, e - 1)):
        held(outputs(ops, layer, x, i, w), x, i, w, parts, tight.is_exact(t, top_k, e))


@pytest.mark.parametrize("name", ["few rows", "some rows", "a dozen rows", "dozens of rows", "many rows"])
def test_outputs_of_large_values(ops, name):
    """Inner rows up to about 1e36."""
    parts, x, ids, w = case_of(name, torch.bfloat16)
    t, e, top_k = CASES[name][:3]
    layer = layer_of(parts)
    x = x.float().clamp(-4, 4) * 2.0 ** 58
    y = ops.fp8_block_experts(x.to(DEV), dev(ids), dev(w), layer.gate_up, layer.gate_up_scale, layer.down,
                              layer.down_scale, layer.inner).double().cpu().numpy()
    assert np.abs(y).max() > 2.0 ** 100
    held(y, x, ids, w, parts, tight.is_exact(t, top_k, e))


@pytest.mark.parametrize("t,skew", [(10, 9.0), (80, 9.0), (160, 4.0)])
def test_outputs_of_concentrated_choices(ops, t, skew):
    """Few rows an expert on average, nearly all of them one expert's: many row tiles of that one on the
    small-M tiles, and beside them experts with a row or none."""
    e, top_k, k, inner = 64, 4, 400, 208
    parts, x, ids, w = case_of((t, e, top_k, k, inner), torch.bfloat16, skew)
    counts = np.bincount(ids.flatten(), minlength=e)
    assert counts.max() >= 0.9 * t and (counts == 0).any()
    layer = layer_of(parts)
    for i in (ids, np.zeros_like(ids), np.full_like(ids, e - 1)):
        held(outputs(ops, layer, x, i, w), x, i, w, parts, True)


@pytest.mark.parametrize("t", [1, 300, 5000, 9000, 30000])
def test_outputs_of_weights_past_32_bits(ops, t):
    """All tokens to the last of 264 experts, whose weights end past 4 GiB, on each path; three tokens' outputs."""
    from w8a8_int8_dynamic_amd import W8A8Experts
    e, k, inner = 264, 4096, 2048
    r = np.random.default_rng(t)
    one = make(1, inner, k, r)
    parts = [torch.zeros(e, *p.shape[1:], dtype=torch.from_numpy(p).dtype, device=DEV) for p in one]
    for p, last in zip(parts, one):
        p[-1] = dev(last[0])
    layer = W8A8Experts.from_quantized(*parts)
    assert layer.gate_up.numel() > 2 ** 32
    x = torch.from_numpy(rows(t, k, r).astype(np.float32)).to(torch.bfloat16)
    y = outputs(ops, layer, x, np.full((t, 1), e - 1, np.int32), np.ones((t, 1), np.float32))
    some = [0, t // 2, t - 1]
    held(y[some], x[some], np.zeros((3, 1), np.int32), np.ones((3, 1), np.float32), one, tight.is_exact(t, 1, e))
