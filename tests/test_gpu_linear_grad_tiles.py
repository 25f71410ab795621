"""z1_linear_grad on every kernel of either gradient: each type and tile side, split and
not, every remainder of the rings of panels, odd edges; dx with and without add and over
it, dweight written and added in fp32 and written to a slot of the type.  Against the
products in 64 bits, tolerances as in test_gpu_linear.py: (depth + 9) 2^-24 of the sum of
magnitudes and half a step; what is added is one term more."""
import pytest
import torch

from layer_refs import TYPES, U32, half_step, placed, tiny, untouched
from linear_grad_cases import cases, shape_of
from mixed_precision_zero_amd import layers as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def near(got, want, size, depth, t, what):
    tol = (depth + 9) * U32 * size + tiny(t)
    if t != torch.float32:
        tol += half_step(t) * want.abs() * (1 + 2.0 ** -8)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


def ident(case):
    form, kind, side, split, s = case
    return f"{('dx', 'dw')[form - 1]}-{kind}-{side}{'-split' if split else ''}-{'x'.join(str(x) for x in s)}"


def on_gpu(g, t, rows, cols, layout):
    m, _ = placed(torch.zeros(1, 1, dtype=t).expand(rows, cols), layout)
    return m.copy_(torch.randn(rows, cols, generator=g, device="cuda"))


@pytest.mark.parametrize("case", list(cases()), ids=ident)
def test_gradient(case):
    form, kind, _, _, (p, q, depth) = case
    rows, inner, outer = shape_of(form, p, q, depth)
    t = TYPES[kind]
    layout = "odd" if depth % 8 else "plain"
    g = torch.Generator(device="cuda").manual_seed(p + q + depth)
    dz = on_gpu(g, t, rows, outer, layout)
    if form == 1:
        w, add = on_gpu(g, t, outer, inner, layout), on_gpu(g, t, rows, inner, layout)
        x = torch.empty(rows, inner, dtype=t, device="cuda")
        ws = torch.empty(L.z1_linear_grad_workspace(dz, x, w), dtype=torch.uint8, device="cuda")
        want, size = dz.double() @ w.double(), dz.double().abs() @ w.double().abs()
        for given in (None, add):
            dx, buf = placed(torch.zeros(1, 1, dtype=t).expand(rows, inner), layout)
            dx.fill_(float("nan"))
            L.z1_linear_grad(dz, None, w, dx=dx, add=given, workspace=ws)
            near(dx, want if given is None else want + add.double(), size if given is None else size + add.double().abs(), depth, t, "dx")
            assert untouched(dx, buf)
        L.z1_linear_grad(dz, None, w, dx=add, add=add, workspace=ws)
        assert torch.equal(add, dx)
        return
    x = on_gpu(g, t, rows, inner, layout)
    ws = torch.empty(L.z1_linear_grad_workspace(dz, x, torch.empty(outer, inner, dtype=t, device="cuda")), dtype=torch.uint8, device="cuda")
    want, size = dz.double().t() @ x.double(), dz.double().abs().t() @ x.double().abs()
    for to, accumulate in ((torch.float32, True), (torch.float32, False), (t, False)):
        dw, buf = placed(torch.zeros(1, 1, dtype=to).expand(outer, inner), layout)
        old = torch.randn(outer, inner, generator=g, device="cuda") if accumulate else torch.full((outer, inner), float("nan"), device="cuda")
        dw.copy_(old)
        L.z1_linear_grad(dz, x, None, dweight=dw, accumulate=accumulate, workspace=ws)
        near(dw, want + old.double() if accumulate else want, size + old.double().abs() if accumulate else size, depth, to, "dweight")
        assert untouched(dw, buf)
