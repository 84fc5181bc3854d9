"""What the accuracy checks of the experts tell apart (tests/test_gpu_experts_accuracy.py runs them
on the GPU): on the same inputs, outputs with a known mistake fail them, and outputs as an error-free
kernel would give them pass."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import block_reference as ref
from tests import experts_reference as tight


def codes(n, k, r):
    q = r.integers(0, 256, (n, k), dtype=np.uint8)
    q[(q & 127) == 127] ^= 1
    return q


def weight(n, k, r):
    return codes(n, k, r), (2.0 ** r.uniform(-12, -8, (ref.blocks_of(n), ref.blocks_of(k)))).astype(np.float32)


def rows(t, k, r):
    """Normal values, one column in fifty 20 times as large, row magnitudes over a factor of 100."""
    x = r.standard_normal((t, k)) * np.where(r.random(k) < 0.02, 20.0, 1.0)
    return 0.3 * x * 10.0 ** (2 * r.random((t, 1)) - 1)


def chosen(t, e, top_k, r, skew):
    x = r.standard_normal((t, e)) + skew * r.standard_normal(e)
    ids = np.argsort(-x, 1)[:, :top_k].astype(np.int32)
    w = np.exp(np.take_along_axis(x, ids, 1))
    return ids, (w / w.sum(1, keepdims=True)).astype(np.float32)


def make(e, inner, k, r, diagonal=False):
    """Codes and scales of experts: [gate_up, its scales, down, its scales]."""
    parts = ([], [], [], [])
    for _ in range(e):
        gate, up = weight(inner, k, r), weight(inner, k, r)
        down = tight.diagonal(k, inner) if diagonal else weight(k, inner, r)
        for p, v in zip(parts, (np.concatenate((gate[0], up[0])), np.concatenate((gate[1], up[1])), *down)):
            p.append(v)
    return [np.stack(p) for p in parts]


# tokens, experts, choices, K, inner: of each path (slots alone are the first one's tokens in small calls)
CASES = {
    "few rows": (40, 12, 3, 528, 400),                     # small-M tiles, 16 x 32
    "some rows": (150, 64, 4, 272, 400),                   # small-M tiles
    "long rows, few": (24, 16, 2, 2064, 656),
    "a dozen rows": (70, 8, 2, 272, 528),                  # rows cut at 64
    "two dozen rows": (100, 8, 2, 656, 400),
    "a popular expert": (180, 24, 4, 400, 272),
    "long rows, two dozen": (50, 2, 1, 4112, 528),
    "dozens of rows": (160, 8, 2, 656, 400),               # 128-row tiles
    "a hundred rows": (300, 9, 3, 400, 272),
    "many rows": (400, 6, 2, 656, 272),                    # 256-row tiles
    "long rows, many": (260, 2, 1, 2064, 272),
    "1024 experts": (300, 1024, 6, 256, 48),
    "64 choices, few rows": (10, 70, 64, 272, 80),
    "64 choices": (150, 70, 64, 144, 48),
}


def case_of(name, dtype, skew=1.0):
    t, e, top_k, k, inner = CASES[name] if isinstance(name, str) else name
    r = np.random.default_rng(t + e + k + inner)
    parts = make(e, inner, k, r)
    return (parts, torch.from_numpy(rows(t, k, r).astype(np.float32)).to(dtype), *chosen(t, e, top_k, r, skew))


# tokens of a call, experts, calls: one choice a token; K 784, inner 656
INNER_CASES = [(1, 8, 160), (4, 8, 40), (40, 8, 4), (80, 8, 2), (88, 8, 2), (120, 5, 2), (160, 5, 1), (165, 5, 1),
               (260, 4, 1), (312, 3, 1), (315, 3, 1), (320, 2, 1)]


def inner_case_of(t, e, sets):
    r = np.random.default_rng(t + e)
    k, inner = 784, 656
    parts = make(e, inner, k, r, diagonal=True)
    xs, ids = [], []
    for _ in range(sets):
        xs.append(torch.from_numpy(rows(t, k, r).astype(np.float32)).to(torch.bfloat16))
        ids.append(chosen(t, e, 1, r, 0.7)[0])
    return parts, xs, ids, np.ones((t, 1), np.float32)


def test_inner_codes_tell_the_forms_apart():
    """Sums with fp32's errors get the codes that the check allows for; the instruction's sums where exact
    ones belong, exact ones where the instruction's do, and errors of 2^-16 do not."""
    (gu, gs, _, _), xs, ids, _ = inner_case_of(160, 5, 1)
    r = np.random.default_rng(3)
    differ, expected = {}, 0.0
    for n in range(5):
        xq, s = ref.quant(xs[0].float().numpy()[ids[0][:, 0] == n])
        sums = {exact: tight.gated_sums(xq, s, gu[n], gs[n], exact) for exact in (True, False)}
        rms = tight.magnitudes(xq, s, gu[n], gs[n])[1]
        sums["fp32"], sums["coarse"] = ([v + rel * m * r.standard_normal(v.shape) for v, m in zip(sums[True], rms)]
                                        for rel in (2.0 ** -21.7, 2.0 ** -16))
        q = {what: tight.inner_codes(ref.silu(g) * u)[0] for what, (g, u) in sums.items()}
        for what in q:
            differ[what] = differ.get(what, 0) + (q[what] != q[True]).sum()
        expected += tight.crossings(*sums[True], *(tight.SUMS * m for m in rms))
    limit = expected + 4 * np.sqrt(expected) + 4
    print(differ, limit)
    assert differ["fp32"] <= limit and min(differ["coarse"], differ[False]) > 2 * limit


def test_instruction_by_hand():
    x, w = np.zeros((1, 128)), np.zeros((3, 128))
    x[0, 0], w[0, 0], w[1, 0] = 256.0, 256.0, 256.0        # 2^16: of its 7 neighbours multiples of 8 stay
    x[0, 7], w[0, 7] = 1.875, 15.0                         # 28.125 -> 24
    x[0, 8], w[1, 8] = 1.875, -15.0                        # the next group's own largest: whole
    w[2, 7] = -1.875
    assert tight.instruction_sums(torch.from_numpy(x), torch.from_numpy(w)).tolist() == \
        [[65536 + 24.0, 65536 - 28.125, -3.515625]]


def test_diagonal_hands_codes_on():
    r = np.random.default_rng(5)
    gu, gs, _, _ = (p[0] for p in make(1, 272, 144, r))
    g, u = tight.gated_sums(*ref.quant(rows(20, 144, r)), gu, gs, True)
    h = ref.silu(g) * u
    q, s = tight.inner_codes(h)
    y = ref.requant(h, 0 * h)[0] @ ref.weight(*tight.diagonal(400, 272)).T
    assert y.shape == (20, 400) and (y[:, 272:] == 0).all()
    assert np.array_equal(tight.codes_of(y[:, :272] / 448, s), q)
    q2, s2 = ref.quant(h.astype(np.float32))
    assert (np.where(q2 == 128, 0, q2) == q).mean() > 0.9999 and np.allclose(s2, s, rtol=1e-6)


@pytest.mark.parametrize("name", list(CASES))
def test_outputs_with_mistakes_are_told_apart(name):
    """Inner rows that never pass through codes, a gain of 5 % on them, two experts' weights of a token
    exchanged, gate and up exchanged: each is off by more than the norm check lets pass."""
    parts, x, ids, w = case_of(name, torch.bfloat16)
    t, e, top_k, _, inner = CASES[name]
    x, exact, limit = x.float().numpy(), tight.is_exact(t, top_k, e), tight.norm_limit(t * top_k * inner)
    run = lambda **a: tight.experts(x, ids, a.get("w", w), a.get("parts", parts), True, a.get("inner"))
    want, bound = run()
    half = parts[1].shape[1] // 2
    wrong = {"no codes": run(inner=lambda h: h)[0], "gain": run(inner=lambda h: 1.05 * ref.requant(h, 0 * h)[0])[0],
             "swapped halves": run(parts=[np.roll(parts[0], inner, 1), np.roll(parts[1], half, 1), *parts[2:]])[0]}
    if top_k > 1:
        wrong["weights"] = run(w=w[:, ::-1])[0]
    for what, y in wrong.items():
        off = tight.token_error(y, want)
        print(what, off, limit)
        assert off > 2 * limit, what
    # and the elementwise bound says something about nearly every element
    assert (np.abs(want) > 4 * bound).mean() > 0.8
    assert (np.abs(wrong["gain"] - want) > bound).mean() > 0.1
