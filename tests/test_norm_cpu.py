"""The norm entry points' argument checks on the host (nothing is launched),
and the 64-bit reference on values worked out by hand."""
from __future__ import annotations

import os
import subprocess

import pytest
import torch

from tests import norm_reference as ref
from tests.test_abi_cpu import A, ALIGN, DEVICE, HEADER, L, MODE, NULL, OK, SHAPE
from w8a8_int8_dynamic_amd import _lib, ops

NO_GPU = not torch.cuda.is_available()


def ns(kind=0, eps=1e-6, weight=0, bias=0, scale=0, shift=0, ld_scale=64, ld_shift=64, groups=1, vec_dtype=0,
       mod_dtype=0):
    return _lib.NORM_STRUCT.pack(kind, eps, weight, bias, scale, shift, ld_scale, ld_shift, groups, vec_dtype,
                                 mod_dtype)


def rows(n=None, x=A, t=0, M=4, K=64, ldx=64, act=0, kind=0, out=A, ldo=64, s=A):
    n = ns() if n is None else n
    return L.norm_rows(x, t, M, K, ldx, n, act, kind, out, ldo, s, None)


def res(n=None, post=None, M=4, K=64, kind=0, out=A, ldo=64, s=A, x=A, y=A, r=A, ldx=64, ldy=64, ldr=64, gate=0,
        ld_gate=64, gate_groups=1, x_dtype=0, y_dtype=0, gate_dtype=0):
    b = _lib.RESIDUAL_STRUCT.pack(x or 0, y or 0, r or 0, ldx, ldy, ldr, gate, ld_gate, gate_groups, 1.0, 1.0,
                                  x_dtype, y_dtype, gate_dtype)
    return L.gated_residual_rows(b, post, M, K, n, kind, out, ldo, s, None)


def test_norm_rows_checks():
    assert rows(t=3) == MODE and rows(act=1) == MODE and rows(t=0, act=2) == MODE and rows(t=2, act=0) == MODE
    assert rows(kind=3) == MODE and rows(kind=-1) == MODE
    assert rows(M=-1) == SHAPE and rows(K=0) == SHAPE and rows(ldx=63) == SHAPE and rows(ldo=63) == SHAPE
    assert rows(x=None) == NULL and rows(out=None) == NULL and rows(kind=1, s=None) == NULL
    assert L.norm_rows(A, 0, 4, 64, 64, None, 0, 0, A, 64, A, None) == NULL
    assert rows(x=A + 1) == ALIGN and rows(t=1, x=A + 2) == ALIGN and rows(out=A + 1) == ALIGN
    assert rows(kind=1, out=A + 4) == ALIGN and rows(kind=1, ldo=68) == ALIGN and rows(kind=2, s=A + 2) == ALIGN
    assert rows(M=0, x=None, out=None) == OK
    if NO_GPU:
        assert rows(x=A + 2, ldx=65, ldo=67) == DEVICE and rows(t=1, act=2) == DEVICE and rows(kind=2) == DEVICE


def test_norm_struct_checks():
    for f in (lambda n: rows(n=n), lambda n: res(n=n)):
        assert f(ns(kind=2)) == MODE
        for eps in (-1.0, float("nan"), float("inf")):
            assert f(ns(eps=eps)) == SHAPE
        assert f(ns(weight=A, vec_dtype=3)) == MODE and f(ns(scale=A, mod_dtype=-1)) == MODE
        assert f(ns(scale=A, groups=3)) == SHAPE and f(ns(shift=A, groups=0)) == SHAPE
        assert f(ns(scale=A, groups=2, ld_scale=63)) == SHAPE and f(ns(shift=A, groups=4, ld_shift=0)) == SHAPE
        assert f(ns(weight=A + 1)) == ALIGN and f(ns(bias=A + 2, vec_dtype=1)) == ALIGN
        assert f(ns(scale=A + 1)) == ALIGN and f(ns(shift=A + 2, mod_dtype=1)) == ALIGN
        if NO_GPU:
            assert f(ns(scale=A, ld_scale=0)) == DEVICE and f(ns(shift=A, groups=4)) == DEVICE


def test_residual_checks():
    assert L.gated_residual_rows(None, None, 4, 64, None, 0, A, 64, A, None) == NULL
    assert res(x_dtype=3) == MODE and res(y_dtype=1) == MODE and res(x_dtype=2) == MODE
    assert res(M=-1) == SHAPE and res(K=0) == SHAPE
    assert res(ldx=63) == SHAPE and res(ldy=63) == SHAPE and res(ldr=63) == SHAPE
    assert res(x=None) == NULL and res(y=None) == NULL and res(r=None) == NULL
    assert res(x=A + 1) == ALIGN and res(y=A + 1) == ALIGN and res(x_dtype=1, r=A + 2) == ALIGN
    assert res(gate=A, gate_dtype=5) == MODE and res(gate=A, gate_groups=3) == SHAPE
    assert res(gate=A, gate_groups=2, ld_gate=63) == SHAPE and res(gate=A, gate_groups=0) == SHAPE
    assert res(gate=A + 2, gate_dtype=1) == ALIGN
    assert res(post=ns(scale=A)) == MODE                          # a branch's norm has no modulation
    assert res(post=ns(kind=7)) == MODE
    assert res(n=ns(), out=None) == NULL and res(n=ns(), ldo=0) == SHAPE and res(n=ns(), kind=9) == MODE
    assert res(M=0, x=None, y=None, r=None) == OK
    if NO_GPU:
        assert res(out=None, ldo=0) == DEVICE and res(x_dtype=1, y_dtype=2, n=ns(), kind=1) == DEVICE
        assert res(post=ns(weight=A), gate=A, gate_groups=4) == DEVICE


def test_structs_match_the_header(tmp_path):
    """The binding packs the structures in the C layout: a C program prints it."""
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "w8a8.h"\nint main(void) { printf("%zu %zu %zu %zu\\n", '
                   "sizeof(w8a8_norm_t), offsetof(w8a8_norm_t, mod_dtype), sizeof(w8a8_residual_t), "
                   "offsetof(w8a8_residual_t, gate_dtype)); return 0; }")
    subprocess.run(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()
    n = _lib.NORM_STRUCT.pack(*range(10), 77)
    r = _lib.RESIDUAL_STRUCT.pack(*range(13), 78)
    assert [int(v) for v in got] == [len(n), n.index(b"\x4d"), len(r), r.index(b"\x4e")]


def test_host_tensors_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        ops.norm(x, ops.Norm())
    with pytest.raises(ValueError, match="device tensor"):
        ops.gated_residual(x, x)


def test_reference_by_hand():
    x = torch.tensor([[3.0, 4.0], [1.0, 1.0]], dtype=torch.float64)
    z = torch.zeros_like(x)
    n, err = ref.norm(x, z, "rms", 0.0)
    assert torch.allclose(n, torch.tensor([[3 / 12.5 ** 0.5, 4 / 12.5 ** 0.5], [1.0, 1.0]], dtype=torch.float64))
    assert (err > 0).all() and (err < 1e-4).all()
    n, _ = ref.norm(x, z, "layer", 0.25, weight=torch.tensor([2.0, 4.0]), bias=torch.tensor([1.0, 0.0]),
                    scale=torch.tensor([[1.0, 0.0], [0.0, 0.0]]), shift=torch.tensor([0.5, 0.0]))
    s = 0.5 / 0.5 ** 0.5
    assert torch.allclose(n, torch.tensor([[(-2 * s + 1) * 2 + 0.5, 4 * s], [1.5, 0.0]], dtype=torch.float64))
    r, _ = ref.residual(x, torch.ones_like(x), gate=torch.tensor([2.0, 0.0]), residual_scale=0.5, branch_scale=3.0)
    assert r.tolist() == [[7.5, 2.0], [6.5, 0.5]]


def test_groups_of_no_rows():
    """No rows split into any number of groups, none among them."""
    ref_rows = torch.zeros(0, 64, dtype=torch.bfloat16)
    for G in (0, 1, 5):
        groups, ld = ops._groups(torch.zeros(G, 64), 0, 64, ref_rows, "scale")
        assert groups >= 1 and ld >= 64
    with pytest.raises(ValueError, match="rows"):
        ops._groups(torch.zeros(0, 64), 4, 64, torch.zeros(4, 64), "scale")
    with pytest.raises(ValueError):
        ops._groups(torch.zeros(0, 63), 0, 64, ref_rows, "scale")
