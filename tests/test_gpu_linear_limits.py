"""z1_linear and z1_linear_dz where values are not finite: dropped elements, and
activations and slopes at their limits.  Everything is exact."""
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


# act and act' at -inf and +inf, their limits
LIMITS = {"none": ((-INF, INF), (1.0, 1.0)), "relu": ((0.0, INF), (0.0, 1.0)), "gelu": ((0.0, INF), (0.0, 1.0)),
          "gelu_tanh": ((0.0, INF), (0.0, 1.0)), "silu": ((0.0, INF), (0.0, 1.0)), "relu2": ((0.0, INF), (0.0, INF))}


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("name", ACTS)
def test_the_gradient_at_infinities(kind, name):
    t = TYPES[kind]
    value, slope = LIMITS[name]
    z = torch.tensor([[-INF, INF]]).to(t).repeat(5, 6)
    dz, dm = (torch.empty_like(z, device="cuda") for _ in range(2))
    L.z1_linear_dz(torch.ones_like(z, device="cuda"), dz, act=name, pre=z.cuda(), dmul=dm)
    assert torch.equal(dm.cpu().float(), torch.tensor([value]).repeat(5, 6))
    assert torch.equal(dz.cpu().float(), torch.tensor([slope]).repeat(5, 6))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("name", ("gelu", "gelu_tanh", "silu"))
def test_not_a_number_stays_one(kind, name):
    z = torch.full((3, 20), NAN, dtype=TYPES[kind], device="cuda")
    dz, dm = torch.zeros_like(z), torch.zeros_like(z)
    L.z1_linear_dz(torch.ones_like(z), dz, act=name, pre=z, dmul=dm)
    assert bool(torch.isnan(dz).all()) and bool(torch.isnan(dm).all())
    y = torch.zeros_like(z)
    L.z1_linear(z[:, :8].contiguous(), torch.ones(20, 8, dtype=TYPES[kind], device="cuda"), y, act=name)
    assert bool(torch.isnan(y).all())


@pytest.mark.parametrize("name", ("gelu", "gelu_tanh", "silu"))
@pytest.mark.parametrize("rows", [3, 70])
def test_a_pre_past_fp16(name, rows):
    """z = -71680 is -inf in fp16's pre; y is 0 from the unrounded z, and so are its gradients."""
    x = torch.full((rows, 8), 128.0, dtype=torch.float16, device="cuda")
    w = torch.full((16, 8), -70.0, dtype=torch.float16, device="cuda")
    y, pre, dz = (torch.full((rows, 16), NAN, dtype=torch.float16, device="cuda") for _ in range(3))
    ws = torch.empty(max(L.z1_linear_workspace(x, w), L.z1_linear_dz_workspace(rows, 16), L.z1_linear_grad_workspace(dz, x, w)),
                     dtype=torch.uint8, device="cuda")
    L.z1_linear(x, w, y, act=name, pre=pre, workspace=ws)
    dm, db, dx, dw = torch.empty_like(y), torch.empty(16, device="cuda"), torch.empty_like(x), torch.empty(16, 8, device="cuda")
    L.z1_linear_dz(torch.ones_like(y), dz, act=name, pre=pre, mul=torch.full_like(y, 3.0), dmul=dm, dbias=db, workspace=ws)
    L.z1_linear_grad(dz, x, w, dx=dx, dweight=dw, workspace=ws)
    assert bool((pre == -INF).all())
    for v in (y, dz, dm, db, dx, dw):
        assert bool((v == 0).all())
