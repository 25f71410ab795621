"""Host-side checks of the layers (include/z1_layers.h): symbols, structures,
refusals of the C ABI and of the binding.  No GPU needed: every case is decided
before any device work."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from layer_refs import keep_mask, philox
from mixed_precision_zero_amd import binding as B
from mixed_precision_zero_amd import layers as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAN, INF = float("nan"), float("inf")


def test_every_declared_symbol_is_exported():
    text = open(os.path.join(ROOT, "include", "z1_layers.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(z1_[a-z_0-9]+)\s*\(", text))
    assert names == set(L.EXPORTS)
    for name in names:
        assert hasattr(B.lib, name)
    assert L.z1_layers_abi_version() == 1


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "z1_layers.h"\nint main(void) { z1_linear_args a; z1_qk_args b; (void)a; (void)b; '
                   'return Z1_LAYERS_ABI_VERSION - 1; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src),
                    "-o", str(tmp_path / "t.o")], check=True)


def test_structures_match_the_header(tmp_path):
    """Sizes and the last members' offsets of the ctypes structures against the C
    compiler's."""
    names = {"z1_drop": (L.Drop, "p"), "z1_dropout_args": (L.DropoutArgs, "reserved"), "z1_linear_args": (L.LinearArgs, "act"),
             "z1_linear_dz_args": (L.LinearDzArgs, "reserved"), "z1_linear_grad_args": (L.LinearGradArgs, "reserved"),
             "z1_heads": (L.Heads, "dout_head"), "z1_qk_args": (L.QkArgs, "accumulate")}
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "z1_layers.h"\nint main(void) { printf("' + "%d " * (2 * len(names))
                   + '", ' + ", ".join(f"(int)sizeof({n}), (int)offsetof({n}, {f})" for n, (_, f) in names.items()) + "); return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    want = [x for s, f in names.values() for x in (ctypes.sizeof(s), getattr(s, f).offset)]
    assert [int(x) for x in got] == want


def test_the_generator_against_its_published_vectors():
    """Philox4x32-10's known answers (the authors' test vectors), for the oracle
    that the GPU's masks are compared with."""
    for c, k, want in (((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
                       ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
                       ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
                        (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(int(x) for x in philox(c, k)) == want
    assert keep_mask(3, 11, 1, 2, 0.0).all() and not keep_mask(3, 11, 1, 2, 1.0).any()
    # element (r, c) takes half c mod 2 of word (c mod 8) / 2 of the block's counter
    w = [int(x) for x in philox((1, 2, 5, 6), (3, 4))]
    mask = keep_mask(3, 16, 3 + (4 << 32), 5 + (6 << 32), 0.5)
    assert [bool(x) for x in mask[2, 8:]] == [(w[j // 2] >> 16 * (j % 2)) & 0xffff >= 32768 for j in range(8)]


def dropout_args(**over):
    a = L.DropoutArgs(10, 20, 0x1000, 0x2000, 0x3000, 20, 20, 20, L.Drop(0x4000, 0, 0.5), 1, 0)
    for k, v in over.items():
        setattr(a.drop if k in ("rng", "offset", "p") else a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), B.Z1_EINVAL), (dict(rows=1 << 31), B.Z1_EINVAL), (dict(cols=0), B.Z1_EINVAL), (dict(cols=(1 << 24) + 1), B.Z1_EINVAL),
    (dict(x=None), B.Z1_EINVAL), (dict(y=None), B.Z1_EINVAL), (dict(ld_x=19), B.Z1_EINVAL), (dict(ld_y=19), B.Z1_EINVAL),
    (dict(ld_residual=19), B.Z1_EINVAL), (dict(dtype=3), B.Z1_EINVAL), (dict(dtype=-1), B.Z1_EINVAL), (dict(reserved=1), B.Z1_EINVAL),
    (dict(p=-0.1), B.Z1_EINVAL), (dict(p=1.1), B.Z1_EINVAL), (dict(p=NAN), B.Z1_EINVAL), (dict(x=0x1001), B.Z1_EALIGN),
    (dict(y=0x3001), B.Z1_EALIGN), (dict(residual=0x2001), B.Z1_EALIGN), (dict(rng=0x4004), B.Z1_EALIGN),
    (dict(y=0x1000, ld_y=24), B.Z1_EINVAL), (dict(y=0x2000, ld_y=24), B.Z1_EINVAL), (dict(dtype=0, x=0x1002), B.Z1_EALIGN)])
def test_dropout_refuses(over, status):
    assert B.lib.z1_dropout(ctypes.byref(dropout_args(**over)), None) == status


def linear_args(**over):
    a = L.LinearArgs(10, 32, 48, 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 0x70000, 32, 32, 48, 48, 48, 48,
                     L.Drop(0x80000, 0, 0.5), 1, 4)
    for k, v in over.items():
        setattr(a.drop if k in ("rng", "offset", "p") else a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), B.Z1_EINVAL), (dict(rows=(1 << 30) + 1), B.Z1_EINVAL), (dict(in_=0), B.Z1_EINVAL), (dict(out=0), B.Z1_EINVAL),
    (dict(in_=(1 << 20) + 1, ld_x=1 << 20, ld_weight=1 << 20), B.Z1_EINVAL), (dict(out=(1 << 20) + 1), B.Z1_EINVAL),
    (dict(x=None), B.Z1_EINVAL), (dict(weight=None), B.Z1_EINVAL), (dict(y=None), B.Z1_EINVAL), (dict(ld_x=31), B.Z1_EINVAL),
    (dict(ld_weight=31), B.Z1_EINVAL), (dict(ld_x=1 << 21), B.Z1_EINVAL), (dict(ld_weight=1 << 21), B.Z1_EINVAL),
    (dict(ld_y=47), B.Z1_EINVAL), (dict(ld_pre=47), B.Z1_EINVAL), (dict(ld_mul=47), B.Z1_EINVAL), (dict(ld_residual=47), B.Z1_EINVAL),
    (dict(dtype=3), B.Z1_EINVAL), (dict(act=6), B.Z1_EINVAL), (dict(act=-1), B.Z1_EINVAL), (dict(p=2.0), B.Z1_EINVAL),
    (dict(x=0x10001), B.Z1_EALIGN), (dict(weight=0x20001), B.Z1_EALIGN), (dict(bias=0x30001), B.Z1_EALIGN),
    (dict(mul=0x40001), B.Z1_EALIGN), (dict(residual=0x50001), B.Z1_EALIGN), (dict(pre=0x60001), B.Z1_EALIGN),
    (dict(y=0x70001), B.Z1_EALIGN), (dict(rng=0x80001), B.Z1_EALIGN), (dict(y=0x50000, ld_y=64), B.Z1_EINVAL),
    (dict(y=0x40000, ld_y=64), B.Z1_EINVAL)])
def test_linear_refuses(over, status):
    a = linear_args(**over)
    assert B.lib.z1_linear(ctypes.byref(a), 0x90000, 1 << 30, None) == status


def dz_args(**over):
    a = L.LinearDzArgs(10, 48, 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 48, 48, 48, 48, 48, L.Drop(0x80000, 0, 0.5), 1, 4,
                       0, 0)
    for k, v in over.items():
        setattr(a.drop if k in ("rng", "offset", "p") else a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), B.Z1_EINVAL), (dict(rows=(1 << 30) + 1), B.Z1_EINVAL), (dict(out=0), B.Z1_EINVAL), (dict(dy=None), B.Z1_EINVAL),
    (dict(pre=None), B.Z1_EINVAL), (dict(act=0, pre=None), B.Z1_EINVAL), (dict(dz=None, dmul=None, dbias=None), B.Z1_EINVAL),
    (dict(ld_dy=47), B.Z1_EINVAL), (dict(ld_pre=47), B.Z1_EINVAL), (dict(ld_mul=47), B.Z1_EINVAL), (dict(ld_dz=47), B.Z1_EINVAL),
    (dict(ld_dmul=47), B.Z1_EINVAL), (dict(dtype=3), B.Z1_EINVAL), (dict(act=6), B.Z1_EINVAL), (dict(accumulate=2), B.Z1_EINVAL),
    (dict(reserved=1), B.Z1_EINVAL), (dict(p=NAN), B.Z1_EINVAL), (dict(dz=0x10000, ld_dz=64), B.Z1_EINVAL),
    (dict(dz=0x20000, ld_dz=64), B.Z1_EINVAL), (dict(dz=0x30000, ld_dz=64), B.Z1_EINVAL), (dict(dmul=0x40000), B.Z1_EINVAL),
    (dict(dmul=0x10000), B.Z1_EINVAL), (dict(dmul=0x30000, ld_dmul=64), B.Z1_EINVAL), (dict(dy=0x10001), B.Z1_EALIGN),
    (dict(dz=0x40001), B.Z1_EALIGN), (dict(dbias=0x60002), B.Z1_EALIGN), (dict(rng=0x80002), B.Z1_EALIGN)])
def test_linear_dz_refuses(over, status):
    assert B.lib.z1_linear_dz(ctypes.byref(dz_args(**over)), 0x90000, 1 << 30, None) == status


def grad_args(**over):
    a = L.LinearGradArgs(10, 32, 48, 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 48, 32, 32, 32, 32, 32, 1, 0, 1, 0)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), B.Z1_EINVAL), (dict(in_=0), B.Z1_EINVAL), (dict(out=0), B.Z1_EINVAL), (dict(dz=None), B.Z1_EINVAL),
    (dict(x=None), B.Z1_EINVAL), (dict(weight=None), B.Z1_EINVAL), (dict(dx=None, dweight=None), B.Z1_EINVAL),
    (dict(ld_dz=47), B.Z1_EINVAL), (dict(ld_x=31), B.Z1_EINVAL), (dict(ld_weight=31), B.Z1_EINVAL), (dict(ld_add=31), B.Z1_EINVAL),
    (dict(ld_dx=31), B.Z1_EINVAL), (dict(ld_dweight=31), B.Z1_EINVAL), (dict(ld_dz=1 << 21), B.Z1_EINVAL), (dict(dtype=3), B.Z1_EINVAL),
    (dict(dweight_dtype=2, accumulate=0), B.Z1_EINVAL), (dict(dweight_dtype=1), B.Z1_EINVAL), (dict(accumulate=2), B.Z1_EINVAL),
    (dict(reserved=1), B.Z1_EINVAL), (dict(dx=0x40000, ld_dx=40), B.Z1_EINVAL), (dict(dz=0x10001), B.Z1_EALIGN),
    (dict(x=0x20001), B.Z1_EALIGN), (dict(weight=0x30001), B.Z1_EALIGN), (dict(add=0x40001), B.Z1_EALIGN), (dict(dx=0x50001), B.Z1_EALIGN),
    (dict(dweight=0x60002), B.Z1_EALIGN)])
def test_linear_grad_refuses(over, status):
    assert B.lib.z1_linear_grad(ctypes.byref(grad_args(**over)), 0x90000, 1 << 30, None) == status


def qk_args(**over):
    h = lambda b: L.Heads(4, b, b + 0x10000, b + 0x20000, b + 0x30000, b + 0x40000, 256, 64, 256, 64, 256, 64)  # noqa: E731
    a = L.QkArgs(10, 64, 32, h(0x100000), h(0x200000), 0x300000, 0x310000, 1e-6, 0, 1, 0, 0)
    for k, v in over.items():
        if k.startswith("q_"):
            setattr(a.q, k[2:], v)
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), B.Z1_EINVAL), (dict(tokens=1 << 31), B.Z1_EINVAL), (dict(dim=0), B.Z1_EINVAL), (dict(dim=513), B.Z1_EINVAL),
    (dict(n_freq=-1), B.Z1_EINVAL), (dict(n_freq=33), B.Z1_EINVAL), (dict(eps=-1.0), B.Z1_EINVAL), (dict(eps=NAN), B.Z1_EINVAL),
    (dict(eps=INF), B.Z1_EINVAL), (dict(dtype=3), B.Z1_EINVAL), (dict(position_type=2), B.Z1_EINVAL), (dict(interleaved=2), B.Z1_EINVAL),
    (dict(accumulate=2), B.Z1_EINVAL), (dict(positions=None), B.Z1_EINVAL), (dict(inv_freq=None), B.Z1_EINVAL),
    (dict(q_heads=-1), B.Z1_EINVAL), (dict(q_heads=(1 << 16) + 1), B.Z1_EINVAL), (dict(q_x=None), B.Z1_EINVAL), (dict(q_out=None), B.Z1_EINVAL),
    (dict(q_x=0x100001), B.Z1_EALIGN), (dict(q_out=0x110001), B.Z1_EALIGN), (dict(q_weight=0x130001), B.Z1_EALIGN),
    (dict(positions=0x300004), B.Z1_EALIGN), (dict(inv_freq=0x310004), B.Z1_EALIGN)])
def test_qk_refuses(grad, over, status):
    a = qk_args(**over)
    got = B.lib.z1_qk_norm_rope_grad(ctypes.byref(a), 0x90000, 1 << 30, None) if grad else B.lib.z1_qk_norm_rope(ctypes.byref(a), None)
    assert got == status


def test_qk_gradient_refuses():
    for over, status in ((dict(q_dout=None), B.Z1_EINVAL), (dict(q_weight=None), B.Z1_EINVAL), (dict(q_dweight=0x140002), B.Z1_EALIGN),
                         (dict(q_dout=0x120001), B.Z1_EALIGN)):
        assert B.lib.z1_qk_norm_rope_grad(ctypes.byref(qk_args(**over)), 0x90000, 1 << 30, None) == status
    need = L.z1_qk_norm_rope_grad_workspace(10, 4, 4, 64)
    assert B.lib.z1_qk_norm_rope_grad(ctypes.byref(qk_args()), 0x90000, need - 1, None) == B.Z1_EINVAL
    assert B.lib.z1_qk_norm_rope_grad(ctypes.byref(qk_args()), None, need, None) == B.Z1_EINVAL
    assert B.lib.z1_qk_norm_rope_grad(ctypes.byref(qk_args()), 0x90004, need, None) == B.Z1_EALIGN


def test_null_arguments():
    n = ctypes.c_int64()
    for f, args in (("z1_dropout", (None, None)), ("z1_linear", (None, None, 0, None)), ("z1_linear_dz", (None, None, 0, None)),
                    ("z1_linear_grad", (None, None, 0, None)), ("z1_qk_norm_rope", (None, None)),
                    ("z1_qk_norm_rope_grad", (None, None, 0, None)), ("z1_linear_workspace", (None, ctypes.byref(n))),
                    ("z1_linear_workspace", (ctypes.byref(linear_args()), None)), ("z1_linear_dz_workspace", (1, 1, None)),
                    ("z1_linear_grad_workspace", (None, ctypes.byref(n))), ("z1_qk_norm_rope_grad_workspace", (1, 1, 1, 1, None)),
                    ("z1_qk_norm_rope_grad_workspace", (1, 1, 1, 513, ctypes.byref(n)))):
        assert getattr(B.lib, f)(*args) == B.Z1_EINVAL, f


def ptr_args(rows, inner, outer, dtype=1, x=0x10000, w=0x20000, ld_x=None, ld_w=None):
    return L.LinearArgs(rows=rows, in_=inner, out=outer, x=x, weight=w, ld_x=ld_x or inner, ld_weight=ld_w or inner, dtype=dtype)


def need_of(a):
    n = ctypes.c_int64(-1)
    assert B.lib.z1_linear_workspace(ctypes.byref(a), ctypes.byref(n)) == B.Z1_OK
    return n.value


def test_workspace_of_a_product():
    """Whole 16-byte rows need none but for a split; others a copy of the operand."""
    assert need_of(ptr_args(4096, 4096, 4096)) == 0
    odd = need_of(ptr_args(4096, 4095, 4096))
    assert odd == 2 * 4096 * 4096 * 2
    assert need_of(ptr_args(4096, 4096, 4096, x=0x10002)) == 4096 * 4096 * 2
    assert need_of(ptr_args(4096, 4096, 4096, ld_w=4097)) == 4096 * 4096 * 2
    assert need_of(ptr_args(4096, 4094, 4096, dtype=0)) == 2 * 4096 * 4096 * 4
    # too small a workspace, or one that is not there
    a = linear_args(in_=31, ld_x=31, ld_weight=31)
    n = need_of(a)
    assert n > 0
    assert B.lib.z1_linear(ctypes.byref(a), 0x90000, n - 1, None) == B.Z1_EINVAL
    assert B.lib.z1_linear(ctypes.byref(a), None, n, None) == B.Z1_EINVAL
    assert B.lib.z1_linear(ctypes.byref(a), 0x90008, n, None) == B.Z1_EALIGN


def test_workspace_of_the_gradients():
    n = ctypes.c_int64()
    assert B.lib.z1_linear_grad_workspace(ctypes.byref(grad_args(rows=4096, in_=4096, out=4096, ld_dz=4096, ld_x=4096, ld_weight=4096)),
                                          ctypes.byref(n)) == B.Z1_OK and n.value == 0
    a = grad_args(rows=4096, in_=4096, out=4095, ld_dz=4095, ld_x=4096, ld_weight=4096)
    assert B.lib.z1_linear_grad_workspace(ctypes.byref(a), ctypes.byref(n)) == B.Z1_OK and n.value == 4096 * 4096 * 2
    a = grad_args(out=47, ld_dz=47)
    assert B.lib.z1_linear_grad_workspace(ctypes.byref(a), ctypes.byref(n)) == B.Z1_OK and n.value > 0
    assert B.lib.z1_linear_grad(ctypes.byref(a), 0x90000, n.value - 1, None) == B.Z1_EINVAL
    assert B.lib.z1_linear_grad(ctypes.byref(a), 0x90004, n.value, None) == B.Z1_EALIGN
    a = dz_args()
    assert B.lib.z1_linear_dz(ctypes.byref(a), None, 0, None) == B.Z1_EINVAL
    assert B.lib.z1_linear_dz(ctypes.byref(a), 0x90004, 1 << 20, None) == B.Z1_EALIGN


def m(*shape, t=torch.bfloat16):
    return torch.zeros(*shape, dtype=t)


@pytest.mark.parametrize("call,error", [
    (lambda: L.z1_linear(m(4, 8), m(6, 9), m(4, 6)), ValueError),
    (lambda: L.z1_linear(m(4, 8), m(6, 8, t=torch.float16), m(4, 6)), TypeError),
    (lambda: L.z1_linear(m(4, 8, t=torch.float64), m(6, 8, t=torch.float64), m(4, 6, t=torch.float64)), TypeError),
    (lambda: L.z1_linear(m(4, 8), m(6, 8), m(4, 7)), ValueError),
    (lambda: L.z1_linear(m(4, 8), m(6, 8), m(6, 4).t()), ValueError),
    (lambda: L.z1_linear(m(4, 8), m(6, 8), m(4, 6), act="tanh"), ValueError),
    (lambda: L.z1_linear(m(4, 8), m(6, 8), m(4, 6), bias=m(5)), ValueError),
    (lambda: L.z1_linear(m(4, 8), m(6, 8), m(4, 6), residual=m(4, 6, t=torch.float32)), TypeError),
    (lambda: L.z1_linear(m(4, 8), m(6, 8), m(4, 6)), ValueError),                       # not on a GPU
    (lambda: L.z1_linear(m(4, 8), m(6, 8), m(1, 6).expand(4, 6)), ValueError),
    (lambda: L.z1_linear(m(4, 8), m(6, 8), m(4, 6), dropout=L.Dropout(m(2), 0.5)), TypeError),
    (lambda: L.z1_linear(m(4, 8), m(6, 8), m(4, 6), workspace=b"x"), TypeError),
    (lambda: L.z1_linear_dz(m(4, 6), m(4, 5)), ValueError),
    (lambda: L.z1_linear_dz(m(4, 6), dbias=m(6)), TypeError),
    (lambda: L.z1_linear_grad(m(4, 6), None, None, dx=m(4, 8)), ValueError),
    (lambda: L.z1_linear_grad(m(4, 6), m(4, 8), m(6, 8)), ValueError),
    (lambda: L.z1_linear_grad(m(4, 6), m(5, 8), m(6, 8), dx=m(4, 8)), ValueError),
    (lambda: L.z1_linear_grad(m(4, 6), m(4, 8), m(6, 8), dweight=m(6, 8, t=torch.float16)), TypeError),
    (lambda: L.z1_dropout(m(4, 6), m(4, 5), L.Dropout(m(2, t=torch.int64), 0.5)), ValueError),
    (lambda: L.z1_dropout(m(4, 6), m(4, 6), L.Dropout(m(1, t=torch.int64), 0.5)), ValueError),
    (lambda: L.z1_qk_norm_rope(m(4, 2, 8), None, m(4, 2, 7), None, m(4, t=torch.int64), m(4, t=torch.float64)), ValueError),
    (lambda: L.z1_qk_norm_rope(m(4, 2, 8), None, m(4, 2, 8), None, m(5, t=torch.int64), m(4, t=torch.float64)), ValueError),
    (lambda: L.z1_qk_norm_rope(m(4, 2, 8), None, m(4, 2, 8), None, m(4, t=torch.int64), m(4)), TypeError),
    (lambda: L.z1_qk_norm_rope(m(4, 2, 8), None, m(4, 2, 8), None, m(4), m(4, t=torch.float64)), TypeError),
    (lambda: L.z1_qk_norm_rope(m(4, 2, 8), None, m(4, 1, 8).expand(4, 2, 8), None, m(4, t=torch.int64), m(4, t=torch.float64)), ValueError),
    (lambda: L.z1_qk_norm_rope(m(4, 8, 2).transpose(1, 2), None, m(4, 2, 8), None, m(4, t=torch.int64), m(4, t=torch.float64)), ValueError),
    (lambda: L.z1_qk_norm_rope(m(4, 2, 8), m(3, 2, 8), m(4, 2, 8), m(3, 2, 8), m(4, t=torch.int64), m(4, t=torch.float64)), ValueError),
])
def test_binding_refuses(call, error):
    with pytest.raises(error):
        call()


def test_weight_of_the_gradient_without_a_norm():
    """A dweight without a weight is refused before any device work."""
    a = qk_args(q_weight=None)
    assert B.lib.z1_qk_norm_rope_grad(ctypes.byref(a), 0x90000, 1 << 30, None) == B.Z1_EINVAL
    a = qk_args(q_weight=None, q_dweight=None, q_x=0x100001)
    assert B.lib.z1_qk_norm_rope_grad(ctypes.byref(a), 0x90000, 1 << 30, None) == B.Z1_EALIGN


@pytest.mark.parametrize("over", [dict(y=0x10000), dict(y=0x20000), dict(y=0x30000), dict(y=0x60000), dict(pre=0x10000), dict(pre=0x20000),
                                  dict(pre=0x30000), dict(pre=0x40000), dict(pre=0x50000)])
def test_linear_refuses_outputs_over_other_buffers(over):
    assert B.lib.z1_linear(ctypes.byref(linear_args(**over)), 0x90000, 1 << 30, None) == B.Z1_EINVAL


@pytest.mark.parametrize("over", [dict(dx=0x10000), dict(dx=0x20000), dict(dx=0x30000), dict(dx=0x60000), dict(dweight=0x10000),
                                  dict(dweight=0x20000), dict(dweight=0x30000), dict(dweight=0x40000)])
def test_linear_grad_refuses_outputs_over_other_buffers(over):
    assert B.lib.z1_linear_grad(ctypes.byref(grad_args(**over)), 0x90000, 1 << 30, None) == B.Z1_EINVAL


@pytest.mark.parametrize("grad", [False, True])
def test_qk_refuses_outputs_over_other_buffers(grad):
    overs = [dict(q_out=0x100000, q_out_token=512), dict(q_out=0x100000, q_out_head=128), dict(q_out=0x210000), dict(q_out=0x200000)]
    if grad:   # dout, of the same kind with other strides and of the other kind; one dweight for both
        overs += [dict(q_out=0x120000, q_out_token=512), dict(q_out=0x220000), dict(q_dweight=0x240000)]
    for over in overs:
        a = qk_args(**over)
        got = B.lib.z1_qk_norm_rope_grad(ctypes.byref(a), 0x90000, 1 << 30, None) if grad else B.lib.z1_qk_norm_rope(ctypes.byref(a), None)
        assert got == B.Z1_EINVAL, over
