"""Sizes at the ends of z1_linear's documented range: every product that is accepted runs
on a grid that a launch can hold, 2^32 - 1 threads in x, and the others are refused (no
GPU needed: the choice is made on the host, the refusals before any device work)."""
import ctypes

import pytest

from mixed_precision_zero_amd import binding as B
from mixed_precision_zero_amd import layers as L
from test_linear_tiles import choice  # noqa: F401  (a fixture)


@pytest.mark.parametrize("fp32", [False, True])
def test_every_grid_can_be_launched(choice, fp32):  # noqa: F811
    # shallow products of many rows, whose tiles of 64 are too many
    thin = [(72, 2 ** 29 + 100, 16), (16, 2 ** 30, 16), (128, 2 ** 29, 8), (8, 2 ** 30, 8), (65, 2 ** 30 - 63, 1), (1, 2 ** 30, 1),
            (129, 2 ** 29, 24), (64, 2 ** 30 - 64, 16)]
    deep = [(8, 8, 2 ** 30), (64, 64, 2 ** 30), (1, 130, 2 ** 30), (1448, 1448, 2 ** 28)]
    products = [s + (fp32,) for p in thin + deep for s in (p, (p[1], p[0], p[2]))]
    for (p, q, d, f), (tile, splits, piece) in zip(products, choice(products)):
        assert tile in (64, 128, 256) and not (f and tile == 256)
        assert -(-p // tile) * -(-q // tile) * splits * 256 < 2 ** 32, (p, q, d, tile, splits)
        assert piece > 0 and piece % 128 == 0 and splits * piece >= d * (4 if f else 2)


def test_the_choice_is_as_before_where_a_launch_holds_it(choice):  # noqa: F811
    assert choice([(64, 2 ** 30 - 64, 16, False), (72, 2 ** 29 + 100, 16, False)]) == [(64, 1, 128), (128, 1, 128)]


def test_what_no_launch_can_hold_is_refused():
    n = ctypes.c_int64()
    far = dict(x=0x10000, weight=0x20000, dtype=1)
    for rows, inner, outer, status in ((2 ** 30, 16, 16, B.Z1_OK), (2 ** 29 + 100, 16, 72, B.Z1_OK), (2 ** 30, 8, 2 ** 20, B.Z1_EINVAL),
                                       (2 ** 30, 2 ** 20, 2 ** 20, B.Z1_EINVAL)):
        a = L.LinearArgs(rows=rows, in_=inner, out=outer, ld_x=inner, ld_weight=inner, **far)
        assert B.lib.z1_linear_workspace(ctypes.byref(a), ctypes.byref(n)) == status, (rows, inner, outer)
    a = L.LinearArgs(rows=2 ** 30, in_=8, out=2 ** 20, ld_x=8, ld_weight=8, y=0x30000, ld_y=2 ** 20, **far)
    assert B.lib.z1_linear(ctypes.byref(a), None, 0, None) == B.Z1_EINVAL
    a = L.LinearGradArgs(rows=2 ** 30, in_=2 ** 20, out=8, dz=0x40000, dx=0x50000, ld_dz=8, ld_x=2 ** 20, ld_weight=2 ** 20, ld_dx=2 ** 20,
                         **far)
    assert B.lib.z1_linear_grad_workspace(ctypes.byref(a), ctypes.byref(n)) == B.Z1_EINVAL
    assert B.lib.z1_linear_grad(ctypes.byref(a), 0x60000, 1 << 40, None) == B.Z1_EINVAL
