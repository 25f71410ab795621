"""Which kernels the products of the GPU tests run on (no GPU needed): the choice is
made on the host from the sizes alone (csrc/z1_linear_tile.h), and a new estimate must
not leave a kernel without a test."""
import os
import subprocess

import pytest

from linear_cases import EDGES, LARGE, PANELS, SPLIT, forms

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include "z1_linear_tile.h"
int main(int argc, char **argv)
{
    for (int i = 1; i + 3 < argc; i += 4) {
        const int fp32 = atoi(argv[i + 3]);
        const long long bytes = atoll(argv[i + 2]) * (fp32 ? 4 : 2);
        const z1::ops::TileChoice c = z1::ops::pick_product(atoll(argv[i]), atoll(argv[i + 1]), bytes, fp32 != 0);
        printf("%d %d %d\n", c.tile, c.splits, c.piece);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    """list of (P, Q, depth, fp32) -> list of (tile, splits, bytes of a piece)"""
    at = tmp_path_factory.mktemp("tile")
    (at / "t.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "mixed_precision_zero_amd", "csrc"),
                    str(at / "t.cpp"), "-o", str(at / "t")], check=True)

    def ask(products):
        args = [str(int(x)) for p in products for x in p]
        out = subprocess.run([str(at / "t")] + args, capture_output=True, text=True, check=True).stdout.split()
        return [tuple(int(x) for x in out[i:i + 3]) for i in range(0, len(out), 3)]

    return ask


def test_the_gpu_tests_reach_every_kernel(choice):
    for form in range(3):
        for fp32 in (False, True):
            products = [forms(s)[form] + (fp32,) for kind, s in PANELS + SPLIT + LARGE if (kind == "f32") == fp32]
            reached = {(t, s > 1) for t, s, _ in choice(products)}
            assert {(64, False), (64, True)} <= reached, (form, fp32, reached)
            if form == 0:
                assert reached == {(t, s) for t in ((64, 128) if fp32 else (64, 128, 256)) for s in (False, True)}, (fp32, reached)


def test_the_rings_are_walked_to_every_remainder(choice):
    for side, ring, kind in ((64, 3, "bf16"), (128, 3, "f16"), (256, 6, "bf16")):
        counts = set()
        for k, s in PANELS:
            p, q, depth = forms(s)[0]
            if k == kind and choice([(p, q, depth, False)])[0][0] == side:
                counts.add(-(-depth * 2 // 128) % ring)
        assert counts == set(range(ring)), (side, counts)


def test_pieces_cover_the_depth(choice):
    products = [(p, q, d, f) for p in (1, 8, 100, 1000, 8184) for q in (1, 72, 500, 4096) for d in (1, 63, 64, 1000, 8192, 200000)
                for f in (False, True)]
    for (p, q, d, f), (tile, splits, piece) in zip(products, choice(products)):
        size = d * (4 if f else 2)
        assert tile in (64, 128, 256) and not (f and tile == 256)
        assert piece % 128 == 0 and splits * piece >= size and (splits - 1) * piece < size


def test_the_edges_lie_on_every_tile_side(choice):
    for side, kind, s in EDGES:
        p, q, depth = forms(s)[0]
        assert choice([(p, q, depth, kind == "f32")])[0][:2] == (side, 1), (side, kind, s)
