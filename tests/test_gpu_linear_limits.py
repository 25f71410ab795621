"""z1_linear_dz where values are not finite: dropped elements.  Everything is exact."""
import pytest
import torch

from layer_refs import TYPES, keep_mask, placed
from mixed_precision_zero_amd import layers as L

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "relu2")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rng(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("rows,outer,layout,p", [(1, 40, "plain", 0.5), (63, 75, "odd", 0.25), (200, 264, "ld", 0.5), (9, 24, "plain", 1.0)])
def test_what_is_dropped_is_zero_in_the_gradient_too(kind, name, rows, outer, layout, p):
    """A dropped element adds nothing to y, so whatever dy, pre and mul hold there, its dz
    and dmul are 0 and dbias is what finite values leave."""
    t = TYPES[kind]
    g = torch.Generator().manual_seed(rows + outer)
    clean = [torch.randn(rows, outer, generator=g).to(t) for _ in range(3)]
    kept = keep_mask(rows, outer, 21, 34 + 2, p)
    poison = torch.tensor([INF, -INF, NAN])[torch.arange(rows * outer).view(rows, outer) % 3].to(t)
    spoiled = [torch.where(kept, v, poison.roll(i, 1)) for i, v in enumerate(clean)]
    d = L.Dropout(rng(21, 34), p, 2)
    ws = torch.empty(L.z1_linear_dz_workspace(rows, outer), dtype=torch.uint8, device="cuda")

    def run(dy, pre, mul):
        dz, dmul = (torch.full((rows, outer), NAN, dtype=t, device="cuda") for _ in range(2))
        db = torch.full((outer,), NAN, device="cuda")
        L.z1_linear_dz(*(placed(v, layout)[0] for v in (dy,)), dz, act=name, pre=placed(pre, layout)[0], mul=placed(mul, layout)[0],
                       dmul=dmul, dbias=db, dropout=d, workspace=ws)
        return dz.cpu(), dmul.cpu(), db.cpu()

    want, got = run(*clean), run(*spoiled)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert bool((got[0][~kept] == 0).all()) and bool((got[1][~kept] == 0).all())
