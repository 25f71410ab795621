"""The sharing out of matrices over ranks (no GPU needed)."""
import math

import pytest

from mixed_precision_zero_amd.muon import assign_matrices, rms_lr_scale
from mixed_precision_zero_amd import workloads as W


def cost(s):
    m, n = sorted(s)
    return 3 * m * m * n + m ** 3


@pytest.mark.parametrize("name", ["smollm135m", "llama1p7b", "llama7b"])
@pytest.mark.parametrize("D", [1, 2, 7, 8])
def test_every_matrix_has_one_owner_and_the_load_is_even(name, D):
    shapes = [s for s in W.WORKLOADS[name].shapes[1:] if len(s) == 2 and s[0] != W.WORKLOADS[name].shapes[0][0]]
    owner = assign_matrices(shapes, D)
    assert len(owner) == len(shapes) and set(owner) <= set(range(D))
    load = [sum(cost(s) for s, o in zip(shapes, owner) if o == r) for r in range(D)]
    assert sum(load) == sum(cost(s) for s in shapes)
    # largest first to the least loaded: at most one matrix over the mean
    assert max(load) <= sum(load) / D + max(cost(s) for s in shapes)
    assert owner == assign_matrices(shapes, D)


def test_small_lists_and_refusals():
    assert assign_matrices([], 3) == []
    assert assign_matrices([(4, 4)] * 3, 8) == [0, 1, 2]
    assert assign_matrices([(2, 2), (9, 9), (2, 2)], 2) == [1, 0, 1]
    with pytest.raises(ValueError):
        assign_matrices([(4,)], 2)
    with pytest.raises(ValueError):
        assign_matrices([(4, 4)], 0)
    assert rms_lr_scale([(4, 9), (16, 1)]) == [0.2 * 3, 0.2 * 4]
    assert math.isclose(rms_lr_scale([(100, 100)], rms=1.0)[0], 10.0)
