"""z1_linear and z1_linear_grad on every tile side, split and not, at every remainder of
the rings of panels, against the products in 64 bits.  Tolerances as in
test_gpu_linear.py: (depth + 9) 2^-24 of the sum of magnitudes and half a step; a split
adds one rounding a piece, which the depth's count already holds."""
import pytest
import torch

from layer_refs import TYPES, U32, half_step, keep_mask, tiny
from linear_cases import EDGES, LARGE, PANELS, SPLIT
from mixed_precision_zero_amd import layers as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def near(got, want, size, depth, t, what):
    tol = (depth + 9) * U32 * size + half_step(t) * want.abs() * (1 + 2.0 ** -8) + tiny(t)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


def ident(case):
    return f"{case[0]}-{'x'.join(str(x) for x in case[1])}"


@pytest.mark.parametrize("case", PANELS + LARGE, ids=ident)
def test_three_products(case):
    kind, (rows, inner, outer) = case
    t = TYPES[kind]
    g = torch.Generator(device="cuda").manual_seed(rows + inner + outer)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    x, w, dz, b, r = rand(rows, inner), rand(outer, inner), rand(rows, outer), rand(outer), rand(rows, outer)
    y, pre, dx = torch.full_like(dz, float("nan")), torch.full_like(dz, float("nan")), torch.full_like(x, float("nan"))
    acc = torch.randn(outer, inner, generator=g, device="cuda")
    dw, slot = acc.clone(), torch.full_like(w, float("nan"))
    ws = torch.empty(max(L.z1_linear_workspace(x, w), L.z1_linear_grad_workspace(dz, x, w)), dtype=torch.uint8, device="cuda")
    L.z1_linear(x, w, y, bias=b, act="relu", residual=r, pre=pre, workspace=ws)
    L.z1_linear_grad(dz, x, w, dx=dx, dweight=dw, accumulate=True, workspace=ws)
    L.z1_linear_grad(dz, x, None, dweight=slot, workspace=ws)
    xd, wd, zd = x.double(), w.double(), dz.double()
    z, size = xd @ wd.t() + b.double(), xd.abs() @ wd.abs().t() + b.double().abs()
    near(pre, z, size, inner, t, "pre")
    near(y, z.clamp(min=0) + r.double(), size + r.double().abs(), inner + 1, t, "y")
    del z, size
    near(dx, zd @ wd, zd.abs() @ wd.abs(), outer, t, "dx")
    product, size = zd.t() @ xd, zd.abs().t() @ xd.abs()
    near(dw, product + acc.double(), size + acc.double().abs(), rows + 1, torch.float32, "dweight")
    near(slot, product, size, rows, t, "slot")


@pytest.mark.parametrize("case", SPLIT, ids=ident)
def test_deep_products_in_pieces(case):
    """x W', and the two gradients whose products have the same sizes."""
    kind, (q, depth, p) = case
    t = TYPES[kind]
    g = torch.Generator(device="cuda").manual_seed(q + depth + p)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731

    def workspace(n):
        assert n > 0
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    a, b = rand(q, depth), rand(p, depth)
    want, size = a.double() @ b.double().t(), a.double().abs() @ b.double().abs().t()
    y = torch.full((q, p), float("nan"), device="cuda", dtype=t)
    bias = rand(p)
    L.z1_linear(a, b, y, bias=bias, workspace=workspace(L.z1_linear_workspace(a, b)))
    near(y, want + bias.double(), size + bias.double().abs(), depth, t, "x W'")
    bt = b.t().contiguous()                                   # a weight of [depth, p]: dz W
    dx, add = torch.full_like(y, float("nan")), rand(q, p)
    x = torch.zeros(q, p, device="cuda", dtype=t)
    L.z1_linear_grad(a, None, bt, dx=dx, add=add, workspace=workspace(L.z1_linear_grad_workspace(a, x, bt)))
    near(dx, want + add.double(), size + add.double().abs(), depth + 1, t, "dz W")
    at = a.t().contiguous()                                   # dz of [depth, q], x of [depth, p]
    dw = torch.full((q, p), 2.0, device="cuda")
    ws = workspace(L.z1_linear_grad_workspace(at, bt, torch.zeros(q, p, device="cuda", dtype=t)))
    L.z1_linear_grad(at, bt, None, dweight=dw, accumulate=True, workspace=ws)
    near(dw, want + 2.0, size + 2.0, depth + 1, torch.float32, "dz' x")
    again = torch.full((q, p), 2.0, device="cuda")
    L.z1_linear_grad(at, bt, None, dweight=again, accumulate=True, workspace=ws)
    assert torch.equal(dw, again)


@pytest.mark.parametrize("side,kind,shape", EDGES)
@pytest.mark.parametrize("what", ["", "residual", "bias", "pre drop", "mul", "mul residual bias drop", "relu", "relu mul residual"])
def test_forms_of_the_epilogue(side, kind, shape, what):
    """What an epilogue may have to do chooses its form; rows and edges of each on every
    tile side.  y adds at most three roundings to z's, and the drop's scale one."""
    rows, inner, outer = shape
    t, what = TYPES[kind], what.split()
    g = torch.Generator(device="cuda").manual_seed(rows + inner + outer)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    x, w, b, m, r = rand(rows, inner), rand(outer, inner), rand(outer), rand(rows, outer), rand(rows, outer)
    y, pre = torch.full_like(r, float("nan")), torch.full_like(r, float("nan"))
    given = dict(bias=b, mul=m, residual=r, pre=pre, dropout=L.Dropout(torch.tensor([3, 5], device="cuda"), 0.25, 1))
    L.z1_linear(x, w, y, act="relu" if "relu" in what else "none",
                workspace=torch.empty(L.z1_linear_workspace(x, w), dtype=torch.uint8, device="cuda"),
                **{k: v for k, v in given.items() if k in what or (k == "dropout" and "drop" in what)})
    z, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    if "bias" in what:
        z, size = z + b.double(), size + b.double().abs()
    if "pre" in what:
        near(pre, z, size, inner, t, "pre")
    z = z.clamp(min=0) if "relu" in what else z
    if "mul" in what:
        z, size = z * m.double(), size * m.double().abs()
    if "drop" in what:
        kept = keep_mask(rows, outer, 3, 5 + 1, 0.25).cuda()
        z, size = torch.where(kept, z / 0.75, torch.zeros_like(z)), size / 0.75
    if "residual" in what:
        z, size = z + r.double(), size + r.double().abs()
    near(y, z, size, inner + 4, t, "y")
