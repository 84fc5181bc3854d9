"""The block-scaled layer's, routing's and experts' argument checks on the host (no kernel
runs: a bad argument returns before the device is touched, and a good call on a
machine without a GPU fails with W8A8_ERR_DEVICE), and the reference rules on values
worked out by hand."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from tests import block_reference as ref
from tests.test_abi_cpu import A, ALIGN, DEVICE, L, MODE, NULL, OK, SHAPE
from w8a8_int8_dynamic_amd import W8A8Experts, W8A8Linear, _lib, ops, quantize_linear_layers

NO_GPU = not torch.cuda.is_available()
BIG = _lib.W8A8_MAX_K + 16


def quant(x=A, t=0, M=4, K=144, ldx=144, q=A, ldq=144, s=A, lds=2):
    return L.fp8_quant_per_block(x, t, M, K, ldx, q, ldq, s, lds, None)


def dequant(q=A, ldq=144, s=A, lds=2, M=4, K=144, t=0, o=A, ldo=144):
    return L.fp8_block_dequant(q, ldq, s, lds, M, K, t, o, ldo, None)


def mm(xq=A, ldq=144, xs=A, lds=4, wp=A, ws=A, bias=None, M=4, N=16, K=144, mode=0, out=A, ldo=16, tile=-1):
    return L.fp8_block_scaled_mm_tile(xq, ldq, xs, lds, wp, ws, bias, M, N, K, mode, out, ldo, None, tile)


def qmm(x=A, t=0, ldx=144, xq=A, ldq=144, xs=A, lds=4, wp=A, ws=A, bias=None, M=4, N=16, K=144, mode=0, out=A,
        ldo=16, tile=-1):
    return L.fp8_block_quant_scaled_mm_tile(x, t, ldx, xq, ldq, xs, lds, wp, ws, bias, M, N, K, mode, out, ldo, None,
                                            tile)


def test_quant_checks():
    for f, rows in ((quant, "x"), (dequant, "o")):
        assert f(t=3) == MODE and f(t=-1) == MODE
        assert f(M=-1) == SHAPE and f(K=8) == SHAPE and f(K=136) == SHAPE and f(M=2 ** 31) == SHAPE
        assert f(K=BIG, ldq=BIG, lds=BIG, **{"ld" + rows: BIG}) == SHAPE
        assert f(**{"ld" + rows: 143}) == SHAPE and f(ldq=143) == SHAPE and f(lds=1) == SHAPE
        assert f(M=0, q=None, s=None, **{rows: None}) == OK
        assert f(q=None) == NULL and f(s=None) == NULL and f(**{rows: None}) == NULL
        assert f(**{rows: A + 8}) == ALIGN and f(**{"ld" + rows: 148}) == ALIGN
        assert f(t=1, **{"ld" + rows: 146}) == ALIGN
        assert f(q=A + 4) == ALIGN and f(ldq=148) == ALIGN and f(s=A + 2) == ALIGN
        if NO_GPU:
            assert f() == DEVICE and f(t=1, **{"ld" + rows: 148}) == DEVICE


def test_pack_checks():
    size = L.fp8_block_prepack_weight_bytes
    assert size(1, 16, 128) == 2048 and size(3, 17, 144) == 3 * 32 * 256
    assert size(0, 16, 128) == size(1, 0, 128) == size(1, 16, 8) == size(1, 16, 24) == size(1, 2 ** 31, 16) == 0
    assert size(1, 16, BIG) == 0 and size(2 ** 62, 16, 128) == 0
    p = lambda q=A, ldq=144, E=1, N=32, K=144, gated=0, p=A: L.fp8_block_prepack_weight(q, ldq, E, N, K, gated, p, None)
    u = lambda q=A, ldq=144, E=1, N=32, K=144, gated=0, p=A: L.fp8_block_unpack_weight(p, E, N, K, gated, q, ldq, None)
    o = lambda q=A, t=1, ldq=144, E=1, N=32, K=144, gated=0, p=A, s=A: L.fp8_block_quant_prepack_weight(
        q, t, ldq, E, N, K, gated, p, s, None)
    for f in (p, u, o):
        assert f(N=0) == SHAPE and f(E=0) == SHAPE and f(K=24) == SHAPE and f(ldq=143) == SHAPE
        assert f(N=16, gated=1) == SHAPE and f(E=2 ** 60) == SHAPE
        assert f(q=None) == NULL and f(p=None) == NULL and f(p=A + 8) == ALIGN
        if NO_GPU:
            assert f() == DEVICE and f(gated=1, E=4) == DEVICE
    assert o(t=2) == MODE and o(s=None) == NULL and o(q=A + 8) == ALIGN and o(ldq=148) == ALIGN and o(s=A + 2) == ALIGN
    assert o(t=0, ldq=146) == ALIGN


def test_mm_checks():
    for f in (mm, qmm):
        assert f(mode=3) == MODE and f(mode=-1) == MODE and f(tile=-2) == MODE
        assert f(tile=L.w8a8_fp8_block_tile_count()) == MODE
        assert f(M=-1) == SHAPE and f(N=0) == SHAPE and f(K=8) == SHAPE and f(K=136) == SHAPE
        assert f(ldq=128) == SHAPE and f(lds=1) == SHAPE and f(ldo=15) == SHAPE
        assert f(K=BIG, ldq=BIG, lds=BIG, **({"ldx": BIG} if f is qmm else {})) == SHAPE
        assert f(ldq=_lib.W8A8_MAX_LDQ + 16) == SHAPE and f(lds=_lib.W8A8_MAX_LDQ // 4 + 4) == SHAPE
        for name in ("xq", "xs", "wp", "ws", "out"):
            assert f(**{name: None}) == NULL, name
        assert f(xq=A + 8) == ALIGN and f(ldq=152) == ALIGN and f(wp=A + 8) == ALIGN and f(ws=A + 2) == ALIGN
        assert f(xs=A + 4) == ALIGN and f(lds=6) == ALIGN and f(out=A + 1) == ALIGN
        assert f(out=A + 2, mode=1) == ALIGN and f(bias=A + 1) == ALIGN
        n = 2 ** 31 - 1
        assert f(M=n, N=n, ldo=n) == SHAPE                  # no launch holds that many tiles
        none = dict(xq=None, xs=None, wp=None, ws=None, out=None)
        assert f(M=0, **none, **({"x": None} if f is qmm else {})) == OK
        if NO_GPU:
            assert f() == DEVICE and f(mode=1, bias=A + 1) == DEVICE and f(mode=2, bias=A) == DEVICE
    assert qmm(t=5) == MODE and qmm(ldx=143) == SHAPE and qmm(x=None) == NULL
    assert qmm(x=A + 8) == ALIGN and qmm(ldx=148) == ALIGN


def test_tiles():
    n = ops.fp8_block_tile_count()
    names = [ops.fp8_block_tile_name(i) for i in range(n)]
    assert n >= 1 and len(set(names)) == n and all(names) and ops.fp8_block_tile_name(n) == ""
    for shape in [(1, 16, 16), (1, 12288, 4096), (512, 12288, 4096), (8192, 4096, 12288)]:
        assert 0 <= ops.fp8_block_tile_auto(*shape) < n


def route(x=A, t=1, ld=16, T=4, E=16, bias=None, score=0, k=2, groups=1, top=1, group_top=2, renorm=1, scale=1.0, ids=A,
          w=A):
    how = _lib.ROUTING_STRUCT.pack(bias or 0, score, k, groups, top, group_top, renorm, scale)
    return L.route_experts(x, t, ld, T, E, how, ids, w, None)


def test_route_checks():
    assert L.route_experts(A, 1, 16, 4, 16, None, A, A, None) == NULL
    assert route(t=3) == MODE and route(score=2) == MODE and route(score=-1) == MODE
    assert route(T=-1) == SHAPE and route(E=0) == SHAPE and route(E=1025, ld=1025) == SHAPE and route(ld=15) == SHAPE
    assert route(k=0) == SHAPE and route(k=17) == SHAPE and route(k=65, E=128, ld=128) == SHAPE
    assert route(groups=0) == SHAPE and route(groups=3) == SHAPE and route(groups=4, top=5) == SHAPE
    assert route(groups=4, top=0) == SHAPE and route(groups=128, E=128, ld=128) == SHAPE
    assert route(groups=8, top=1, k=3) == SHAPE and route(group_top=0) == SHAPE and route(group_top=3) == SHAPE
    assert route(scale=math.nan) == SHAPE and route(scale=math.inf) == SHAPE
    assert route(T=0, x=None, ids=None, w=None) == OK
    assert route(x=None) == NULL and route(ids=None) == NULL and route(w=None) == NULL
    assert route(x=A + 2) == ALIGN and route(t=0, x=A + 1) == ALIGN and route(bias=A + 2) == ALIGN
    assert route(ids=A + 2) == ALIGN and route(w=A + 2) == ALIGN
    if NO_GPU:
        assert route() == DEVICE and route(t=0, x=A + 2, bias=A, groups=4, top=2, score=1) == DEVICE


def experts(gu=A, gs=A, dn=A, ds=A, K=144, inner=80, E=4, x=A, t=0, ldx=144, T=4, ids=A, w=A, k=2, out=A, ldo=144,
            work=A, size=1 << 40):
    layer = _lib.EXPERTS_STRUCT.pack(gu or 0, gs or 0, dn or 0, ds or 0, K, inner, E)
    return L.fp8_block_experts(layer, x, t, ldx, T, ids, w, k, out, ldo, work, size, None)


def test_experts_checks():
    assert L.fp8_block_experts(None, A, 0, 144, 4, A, A, 2, A, 144, A, 1 << 40, None) == NULL
    assert experts(t=3) == MODE
    for bad in (dict(T=-1), dict(K=136, ldx=136, ldo=136), dict(K=0), dict(inner=8), dict(inner=24), dict(E=0),
                dict(E=1025),
                dict(k=0), dict(k=65), dict(K=BIG, ldx=BIG, ldo=BIG), dict(inner=BIG), dict(ldx=143), dict(ldo=143),
                dict(T=2 ** 31)):
        assert experts(**bad) == SHAPE, bad
    assert experts(T=0, x=None, ids=None, w=None, out=None, work=None) == OK
    for name in ("gu", "gs", "dn", "ds", "x", "ids", "w", "out", "work"):
        assert experts(**{name: None}) == NULL, name
    for bad in (dict(x=A + 8), dict(ldx=148), dict(out=A + 8), dict(ldo=148), dict(t=1, ldx=146), dict(gu=A + 8),
                dict(dn=A + 8), dict(work=A + 128), dict(ids=A + 2), dict(w=A + 2), dict(gs=A + 2), dict(ds=A + 2)):
        assert experts(**bad) == ALIGN, bad
    most = _lib.W8A8_MAX_K
    # The largest layer's launches all fit: a pass of up to 65536 slots and 2^30 codes, its rows twice.
    for t, k in ((8192, 1), (2 ** 31 - 1, 64)):
        size = L.fp8_block_experts_workspace_bytes(t, most, most, 1024, k)
        assert 0 < size < 65536 * most * 8, (t, k)
    need = L.fp8_block_experts_workspace_bytes(4, 144, 80, 4, 2)
    assert need > 0 and experts(size=need - 1) == SHAPE
    assert L.fp8_block_experts_workspace_bytes(4, 136, 80, 4, 2) == 0
    assert L.fp8_block_experts_workspace_bytes(4, 144, 80, 1025, 2) == 0
    # the workspace stays bounded: long inputs go in passes
    assert L.fp8_block_experts_workspace_bytes(2 ** 30, 4096, 1024, 64, 8) == \
        L.fp8_block_experts_workspace_bytes(2 ** 20, 4096, 1024, 64, 8) < 4 << 30
    if NO_GPU:
        assert experts(size=need) == DEVICE and experts(t=1, ldx=148, ldo=148) == DEVICE


def test_reference_rule_by_hand():
    x = np.zeros((1, 144), np.float32)
    x[0, :7] = [448, 17, 18, 19, -25, 2.0 ** -10, -0.0]    # factor 1: 17 -> 16, 19 -> 20 (ties to even), -25 -> -24
    x[0, 130] = 7.0                                        # a block of its own: factor 64
    q, s = ref.quant(x)
    assert list(s[0]) == [1.0, 7.0 / 448]
    assert list(ref.VALUES[q[0, :7]]) == [448, 16, 18, 20, -24, 0, 0] and q[0, 6] == 0x80
    assert ref.VALUES[q[0, 130]] == 448
    # against torch's conversion, every fp16 value within the range
    v = np.arange(65536, dtype=np.uint16).view(np.float16).astype(np.float32)
    v = v[np.isfinite(v) & (np.abs(v) <= 448)]
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3(v), want)


def test_reference_requant_bound():
    """Elements far from a border keep their code and a small bound, elements at one get the codes' distance."""
    h = np.full((1, 128), 17.0)
    h[0, 0], h[0, 1] = 448.0, 16.5
    val, bound = ref.requant(h, np.full_like(h, 1e-4))
    assert val[0, 0] == 448 and val[0, 1] == 16 and bound[0, 1] < 0.01 and 1.9 < bound[0, 2] < 2.1


def test_reference_routing_by_hand():
    x = np.array([[0.0, 2.0, 1.0, 2.0]])
    ids, w = ref.route(x, 2)
    assert list(ids[0]) == [1, 3] and np.allclose(w, 0.5)
    ids, w = ref.route(x, 2, "sigmoid", bias=np.array([9.0, 0, 0, 0.1]), renormalize=False, scale=2.0)
    assert list(ids[0]) == [0, 3] and np.allclose(w[0], [1.0, 2 / (1 + np.exp(-2.0))])
    ids, _ = ref.route(x, 1, groups=2, top_groups=1, group_top=2)
    assert list(ids[0]) == [3]
    ids, w = ref.route(np.array([[-np.inf, np.nan, 5.0, -np.inf]]), 2)
    assert list(ids[0]) == [2, -1] and list(w[0]) == [1, 0]


def test_refusals():
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        ops.fp8_quant_per_block(cpu)
    with pytest.raises(ValueError, match="device tensor"):
        ops.fp8_block_prepack_weight(torch.zeros(16, 64, dtype=torch.uint8))
    with pytest.raises(TypeError):
        ops.fp8_block_prepack_weight(torch.zeros(16, 64))
    with pytest.raises(ValueError, match="device tensor"):
        ops.route_experts(torch.zeros(4, 8), ops.Routing(2))
    with pytest.raises(ValueError, match="GPU"):
        quantize_linear_layers(torch.nn.Linear(64, 64), method="fp8_block")
    with pytest.raises(ValueError, match="multiples of 16"):
        W8A8Experts.from_float(torch.zeros(2, 16, 64), torch.zeros(2, 64, 8))
    with pytest.raises(ValueError, match="belong together"):
        W8A8Experts.from_float(torch.zeros(2, 64, 64), torch.zeros(2, 64, 16))
    packed = torch.zeros(16 * 128, dtype=torch.uint8)
    for shape in ((), (1,), (17,), (1, 16)):
        with pytest.raises(ValueError, match="bias"):
            W8A8Linear(packed, torch.zeros(1, 1), 16, 64, torch.zeros(shape), "fp8_block")


def overlapping_weights(k=48):
    """Weights [N, K] and [E, N, K] whose rows lie anywhere but one pitch apart, by name."""
    base = torch.arange(8 * 32 * k, dtype=torch.float32).remainder(251)
    row = base[:k].view(1, k)
    return {
        "one row expanded": row.expand(32, k),
        "one row expanded to experts": row.view(1, 1, k).expand(3, 32, k),
        "one matrix expanded to experts": base[:32 * k].view(1, 32, k).expand(3, 32, k),
        "an expert's row expanded": base[:3 * k].view(3, 1, k).expand(3, 32, k),
        "sliding window": base.as_strided((32, k), (16, 1)),
        "sliding windows of experts": base.as_strided((3, 32, k), (32 * 16, 16, 1)),
        "experts of one row, overlapping": base.as_strided((3, 1, k), (16, 1, 1)),
        "experts of one row, apart": base.as_strided((3, 1, k), (64, 7, 1)),
        "experts of one row, the same": row.view(1, 1, k).expand(3, 1, k),
        "one row": base.as_strided((1, k), (3, 1)),
        "one expert": base.as_strided((1, 32, k), (5, k + 16, 1)),
        "pitch": base.as_strided((32, k), (k + 16, 1)),
        "pitch of experts": base.as_strided((3, 32, k), (32 * (k + 16), k + 16, 1)),
        "gaps between experts": base.as_strided((3, 32, k), (32 * k + 16, k, 1)),
        "columns": base[:32 * k].view(k, 32).t(),
    }


@pytest.mark.parametrize("name", list(overlapping_weights()))
def test_weight_pitch(name):
    """The pitch that a weight is handed over with leads to its own elements, inside its own memory."""
    w = overlapping_weights()[name]
    m, ld = ops._matrices(w)
    n, k = w.shape[-2:]
    rows = w.numel() // k
    assert ld >= k and (rows - 1) * ld + k <= m.untyped_storage().nbytes() // 4 - m.storage_offset()
    assert torch.equal(m.as_strided((rows, k), (ld, 1)), w.reshape(rows, k))
    assert (m is w) == (name in ("one row", "one expert", "pitch", "pitch of experts", "experts of one row, apart"))


def overlapping_logits(e=24):
    """Logits [8, e] whose rows are one row of memory, overlap, or lie further apart, by name."""
    base = torch.randn(8 * 64, generator=torch.Generator().manual_seed(5))
    return {"expanded": base[:e].expand(8, e), "overlapping": base.as_strided((8, e), (e - 1, 1)),
            "pitch": base.as_strided((8, e), (e + 8, 1)), "contiguous": base[:8 * e].view(8, e),
            "one": base.as_strided((1, e), (3, 1)), "one expert": base[:1].expand(8, 1),
            "one expert, apart": base.as_strided((8, 1), (5, 7))}


@pytest.mark.parametrize("name", list(overlapping_logits()))
def test_logits_pitch(name, monkeypatch):
    """The pitch that logits are handed over with leads to their own elements, inside their own memory."""
    x = overlapping_logits()[name]
    calls = []
    monkeypatch.setattr(ops, "_float_rows", lambda t, _: (1, *t.shape, t.stride(0) if t.shape[0] > 1 else t.shape[1]))
    monkeypatch.setattr(ops, "_run", lambda t, entry, at, kind, ld, *rest: calls.append((t, entry, at, ld)))
    ops.route_experts(x, ops.Routing(1))
    (t, entry, at, ld), = calls
    assert entry == "route_experts" and at == t.data_ptr() and ld >= x.shape[1]
    assert (t.shape[0] - 1) * ld + t.shape[1] <= t.untyped_storage().nbytes() // 4 - t.storage_offset()
    assert torch.equal(t.as_strided(t.shape, (ld, 1)), x)


def test_routing_divides_by_a_product():
    """csrc/routing.hip's group of an expert, expert * ceil(2^20 / size) >> 20, is expert / size for every size of a
    group and every expert that a lane may hold."""
    expert = np.arange(1024, dtype=np.uint32)
    for size in range(1, 1025):
        inverse = np.uint32(((1 << 20) + size - 1) // size)
        assert np.array_equal((expert * inverse) >> np.uint32(20), expert // size), size


def test_block_scales_are_checked_as_fp32():
    from w8a8_int8_dynamic_amd.linear import _block_scales
    for bad in (torch.full((1, 2), 1e39, dtype=torch.float64), torch.full((1, 2), float("nan")),
                torch.full((1, 2), float("inf"), dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="finite"):
            _block_scales(bad, (1, 2))
    with pytest.raises(ValueError, match="shape"):
        _block_scales(torch.ones(2, 1), (1, 2))
    for dtype in (torch.float64, torch.bfloat16):
        ws = _block_scales(torch.full((2, 3), 0.5, dtype=dtype).t(), (3, 2))
        assert ws.dtype == torch.float32 and ws.is_contiguous() and (ws == 0.5).all()


def test_experts_forward_takes_ids_of_its_tokens(monkeypatch):
    """ids and weights stand beside x's leading dimensions, or are of the flattened tokens; others are
    refused, also where they hold as many tokens."""
    got = []
    monkeypatch.setattr(ops, "fp8_block_experts", lambda x, ids, w, *_: got.append((ids, w)) or x)
    part = torch.zeros(1)
    layer = W8A8Experts(part, torch.zeros(4, 1, 1), part, part, 16, 48)
    x = torch.zeros(2, 3, 48, dtype=torch.bfloat16)
    ids = torch.arange(12, dtype=torch.int32).view(2, 3, 2)
    w = ids.float()
    for i, v in ((ids, w), (ids.view(6, 2), w.view(6, 2))):
        assert layer(x, i, v).shape == x.shape
        assert torch.equal(got[-1][0], ids.view(6, 2)) and torch.equal(got[-1][1], w.view(6, 2))
    assert layer(x[0, 0], ids[0, 0], w[0, 0]).shape == (48,) and got[-1][0].shape == (1, 2)
    before = len(got)
    for i, v in ((ids.view(3, 2, 2), w.view(3, 2, 2)), (ids, w.view(3, 2, 2)), (ids, w.view(6, 2)),
                 (ids.view(1, 6, 2), w.view(1, 6, 2)), (ids.flatten(), w.flatten())):
        with pytest.raises(ValueError, match="ids and weights"):
            layer(x, i, v)
    assert len(got) == before
