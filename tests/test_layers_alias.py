"""Outputs of the layers that are another buffer of the call at the same address: refused
but for the pairs that include/z1_layers.h names.  No GPU needed: a pointer beside them is
misaligned, so that a call that is not refused for its buffers ends with Z1_EALIGN, not with
the Z1_EINVAL that a machine without a GPU gives to any."""
import ctypes

import pytest

from mixed_precision_zero_amd import binding as B
from mixed_precision_zero_amd import layers as L
from test_layers_host import dropout_args, dz_args, grad_args, linear_args, qk_args

WORK, RNG = 0x90000, 0x80000   # of the arguments below


# of each call a pointer that is misaligned, and another one where the first is in question
ODD = {"z1_dropout": ("x", 0x1001, "residual", 0x2001), "z1_linear": ("bias", 0x30001, "x", 0x10001),
       "z1_linear_dz": ("mul", 0x30001, "pre", 0x20001), "z1_linear_grad": ("add", 0x40001, "dz", 0x10001),
       "z1_qk_norm_rope": ("positions", 0x300004, "inv_freq", 0x310004), "z1_qk_norm_rope_grad": ("positions", 0x300004, "inv_freq", 0x310004)}
MAKE = {"z1_dropout": dropout_args, "z1_linear": linear_args, "z1_linear_dz": dz_args, "z1_linear_grad": grad_args,
        "z1_qk_norm_rope": qk_args, "z1_qk_norm_rope_grad": qk_args}


def status(call, over, keys={}):
    first, at, second, instead = ODD[call]
    address = {"mul": 0x30000, "x": 0x1000 if call == "z1_dropout" else 0x10000, "bias": 0x30000, "add": 0x40000, "positions": 0x300000}
    taken = first in over or address[first] in list(over.values()) + list(keys.values())
    a = MAKE[call](**{**over, **({second: instead} if taken else {first: at})})
    for k, v in keys.items():
        setattr(a.k, k, v)
    work = () if call in ("z1_dropout", "z1_qk_norm_rope") else (WORK, 1 << 30)
    return getattr(B.lib, call)(ctypes.byref(a), *work, None)


def refused(call, over, keys={}):
    return status(call, over, keys) == B.Z1_EINVAL


@pytest.mark.parametrize("call", MAKE)
def test_apart_they_are_not(call):
    assert status(call, {}) == B.Z1_EALIGN


@pytest.mark.parametrize("call,over", [
    ("z1_dropout", dict(y=0x2000)), ("z1_linear", dict(y=0x40000)), ("z1_linear", dict(y=0x50000)), ("z1_linear", dict(mul=0x50000)),
    ("z1_linear_dz", dict(dz=0x10000)), ("z1_linear_dz", dict(dz=0x20000)), ("z1_linear_dz", dict(dmul=0x20000)),
    ("z1_linear_grad", dict(add=0x50000)), ("z1_linear", dict(residual=None, y=0x40000)),
    ("z1_qk_norm_rope", dict(q_out=0x100000)), ("z1_qk_norm_rope_grad", dict(q_out=0x100000)), ("z1_qk_norm_rope_grad", dict(q_out=0x120000)),
    ("z1_qk_norm_rope_grad", dict(q_weight=0x230000))])
def test_the_pairs_that_may_be_one_are_not(call, over):
    assert status(call, over) == B.Z1_EALIGN


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("over", [dict(dbias=0x10000), dict(dbias=0x20000), dict(dbias=0x30000), dict(dbias=0x40000), dict(dbias=0x50000),
                                  dict(dbias=RNG), dict(dz=RNG), dict(dmul=RNG), dict(dbias=WORK), dict(dz=WORK), dict(dmul=WORK)])
def test_linear_dz(over, dtype):
    assert refused("z1_linear_dz", dict(dtype=dtype, **over))


def test_linear_dz_over_its_inputs_workspace():
    for name in ("dy", "pre", "mul"):
        assert refused("z1_linear_dz", {name: WORK}), name


@pytest.mark.parametrize("over", [dict(y=RNG), dict(pre=RNG)])
def test_linear(over):
    assert refused("z1_linear", over)


@pytest.mark.parametrize("name", ["x", "weight", "bias", "mul", "residual", "pre", "y", "rng"])
def test_linear_over_its_workspace(name):
    """Rows of 31 elements are copied, so there is one."""
    assert refused("z1_linear", {"in_": 31, "ld_x": 31, "ld_weight": 31, name: WORK})


@pytest.mark.parametrize("name", ["dz", "x", "weight", "add", "dx", "dweight"])
def test_linear_grad_over_its_workspace(name):
    assert refused("z1_linear_grad", {"out": 47, "ld_dz": 47, name: WORK})


def test_dropout():
    for over in (dict(y=0x4000), dict(y=0x4000, residual=None)):
        assert refused("z1_dropout", over)


# the arguments of qk_args: for queries x 0x100000, out 0x110000, dout 0x120000, weight 0x130000,
# dweight 0x140000, for keys the same from 0x200000; positions 0x300000, frequencies 0x310000
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("over", [dict(q_out=0x130000), dict(q_out=0x230000), dict(q_out=0x300000), dict(q_out=0x310000)])
def test_heads(grad, over):
    assert refused("z1_qk_norm_rope_grad" if grad else "z1_qk_norm_rope", over)


@pytest.mark.parametrize("over", [dict(q_out=0x140000), dict(q_out=0x240000), dict(q_out=WORK), dict(q_x=WORK), dict(q_dout=WORK),
                                  dict(q_weight=WORK), dict(q_dweight=WORK), dict(positions=WORK), dict(inv_freq=WORK)]
                         + [dict(q_dweight=x) for x in (0x100000, 0x110000, 0x120000, 0x130000, 0x200000, 0x210000, 0x220000, 0x230000,
                                                        0x300000, 0x310000)])
def test_gradient_of_heads(over):
    assert refused("z1_qk_norm_rope_grad", over)


@pytest.mark.parametrize("keys", [dict(out=0x230000), dict(out=0x130000), dict(out=0x140000), dict(dweight=0x230000), dict(dweight=0x130000),
                                  dict(dweight=0x100000), dict(dweight=0x110000), dict(weight=WORK)])
def test_the_keys_too(keys):
    assert refused("z1_qk_norm_rope_grad", {}, keys)
    if "out" in keys and keys["out"] != 0x140000:
        assert refused("z1_qk_norm_rope", {}, keys)
