"""Which of Muon's kernels the lists of the GPU tests run on (no GPU needed):
the choice is made on the host from the sizes alone (csrc/z1_muon_tile.h), and a
new estimate must not leave a kernel without a test."""
import os
import subprocess

import pytest

from muon_cases import LARGE, SMALL, TILED

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <vector>
#include "z1_muon_tile.h"
using namespace z1::ops;
int main(int argc, char **argv)
{
    std::vector<int64_t> rows, cols;
    int n_small = 0;
    const int passes = atoi(argv[1]);   // 3: wide products, which one workgroup does not take
    for (int i = 2; i + 1 < argc; i += 2) {
        const int64_t r = atoll(argv[i]), c = atoll(argv[i + 1]);
        if (passes == 1 && muon_small(pad_to(std::min(r, c), 32), pad_to(std::max(r, c), 32))) {
            ++n_small;
        } else {
            rows.push_back(r);
            cols.push_back(c);
        }
    }
    const int n = (int)rows.size();
    int tile[3];
    int64_t whole = 64, tiles = 0, panels = INT64_MAX;
    for (int p = 0; p < 3; ++p) {
        tile[p] = pick_tile(p, n, rows.data(), cols.data(), passes);
        whole = std::max<int64_t>(whole, tile[p]);
    }
    for (int i = 0; i < n; ++i) {
        const int64_t q = pad_to(std::min(rows[i], cols[i]), whole) / tile[0];
        tiles += q * (q + 1) / 2;
        panels = std::min(panels, pad_to(std::max(rows[i], cols[i]), whole) / 32);
    }
    printf("%d %d %d %d %d", n_small, tile[0], tile[1], tile[2], (int)gram_splits(tile[0], tiles, panels));
    return 0;
}
"""


@pytest.fixture(scope="module")
def kernels_of(tmp_path_factory):
    """list of (rows, cols) -> (matrices one workgroup takes, the three
    products' tile sides, pieces of X X^T)"""
    at = tmp_path_factory.mktemp("tile")
    (at / "t.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "mixed_precision_zero_amd", "csrc"), str(at / "t.cpp"), "-o", str(at / "t")],
                   check=True)

    def ask(shapes, passes=1):
        out = subprocess.run([str(at / "t"), str(passes)] + [str(x) for s in shapes for x in s], capture_output=True, text=True,
                             check=True).stdout.split()
        small, a, b, c, splits = map(int, out)
        return small, (a, b, c), splits

    return ask


def test_the_large_lists_reach_every_tile_side_of_every_product(kernels_of):
    for passes in (1, 3):
        sides = [kernels_of(s, passes)[1] for s in LARGE]
        for product in range(3):
            assert {t[product] for t in sides} == {64, 128, 256}, (product, sides)
        # one of them on 256 throughout, wide and tall
        assert sides[-2] == sides[-1] == (256, 256, 256)
    assert all(kernels_of(s)[0] == 0 for s in LARGE)


def test_the_tiled_lists_are_tiled_and_the_small_ones_are_not(kernels_of):
    for s in TILED:
        small, tiles, _ = kernels_of(s)
        assert small == 0 and tiles[0] == 64, s
    for passes in (1, 3):
        assert [kernels_of(s, passes)[2] > 1 for s in TILED[-2:]] == [True, True]
        assert kernels_of([(1, 300)], passes)[1] == (64, 64, 64)
    for s in SMALL:
        assert kernels_of(s)[0] == len(s), s


def test_choices_for_sizes_at_the_borders(kernels_of):
    assert kernels_of([]) == (0, (64, 64, 64), 1)
    # one workgroup's LDS: 128 x 160 and 64 x 512 fit, a block more does not
    for fits, more in (((128, 160), (128, 161)), ((64, 512), (65, 512)), ((160, 128), (161, 128))):
        assert kernels_of([fits])[0] == 1 and kernels_of([more])[0] == 0
    # many equal matrices fill the GPU with large tiles, few do not
    assert kernels_of([(2048, 2048)])[1] == (64, 64, 64)
    assert kernels_of([(2048, 2048)] * 24)[1] == (256, 256, 256)
