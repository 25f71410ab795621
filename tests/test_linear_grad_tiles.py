"""Which kernels the gradients' products of the GPU tests run on (no GPU needed): the
choice is made on the host from the sizes alone (csrc/z1_linear_tile.h), and a new
estimate must not leave a kernel without a test.  Asked of each gradient and type by
itself, as each is a kernel of its own."""
import pytest

from linear_grad_cases import cases, shape_of
from linear_cases import forms
from test_linear_tiles import choice  # noqa: F401  (a fixture)

RING = {64: 3, 128: 3, 256: 6}   # 256: P has two slots and Q three


def test_the_cases_run_on_the_side_they_are_named_for(choice):  # noqa: F811
    listed = list(cases())
    for (form, kind, side, split, s), (tile, splits, _) in zip(listed, choice([s + (k == "f32",) for _, k, _, _, s in listed])):
        assert (tile, splits > 1) == (side, split), (form, kind, s, tile, splits)
        assert forms(shape_of(form, *s))[form] == s


@pytest.mark.parametrize("form", [1, 2])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_every_kernel_of_a_gradient_is_reached(choice, form, kind):  # noqa: F811
    mine = [(s, split) for f, k, _, split, s in cases() if (f, k) == (form, kind)]
    reached = {(t, n > 1) for t, n, _ in choice([s + (kind == "f32",) for s, _ in mine])}
    assert reached == {(t, split) for t in ((64, 128) if kind == "f32" else (64, 128, 256)) for split in (False, True)}, reached


@pytest.mark.parametrize("form", [1, 2])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("side", [64, 128, 256])
def test_the_rings_are_walked_to_every_remainder_and_edges_lie_on_every_side(choice, form, kind, side):  # noqa: F811
    if (kind, side) == ("f32", 256):
        pytest.skip("fp32 has no such tiles")
    mine = [s for f, k, _, _, s in cases() if (f, k) == (form, kind)]
    counts, edges = set(), 0
    for s, (tile, splits, _) in zip(mine, choice([s + (kind == "f32",) for s in mine])):
        if (tile, splits) == (side, 1):
            counts.add(-(-s[2] * (4 if kind == "f32" else 2) // 128) % RING[side])
            edges += all(x % 8 for x in s[:2]) and s[2] % 4 != 0
    assert counts == set(range(RING[side])) and edges > 0, (counts, edges)
