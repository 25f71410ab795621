"""Muon's tiled kernels (products of 64, 128 and 256 a side) against the
definition in binary64, at sizes that reach each of them
(tests/test_muon_kernels.py), and the corners of test_gpu_muon.py on the tiled
path.

Tolerances are those counted in test_gpu_muon.py: 7.3e-3 of the 2-norm for five
steps, sqrt(steps / 5) times that for more, and 2^-8 for a bf16 output.  Because
one wrong tile of a large matrix hardly shows in its norm, every 32 x 32 block
is held to it too.  There the errors of single elements count, which spread as
the sum of many independent roundings: 3 times the tolerance at the matrix's
mean size, for matrices whose blocks are all alike (gaussian)."""
import math

import pytest
import torch

from mixed_precision_zero_amd import ops as O
from muon_cases import LARGE, SMALL, TILED
from test_gpu_muon import matrix, orthogonal, rel

pytestmark = pytest.mark.gpu
TOL = 7.3e-3
HALF = 2.0 ** -8     # bf16, half a step


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def blocks(x):
    """Square sums over 32 x 32 blocks, and the blocks' element counts."""
    def total(y):
        y = torch.nn.functional.pad(y, (0, -y.shape[1] % 32, 0, -y.shape[0] % 32))
        return y.view(y.shape[0] // 32, 32, y.shape[1] // 32, 32).sum((1, 3))
    return total(x.double().square()), total(torch.ones_like(x, dtype=torch.float64))


def check(got, want, tol, by_block=True):
    assert rel(got, want) <= tol, rel(got, want)
    if by_block:
        err, count = blocks(got.double() - want)
        size = float(want.norm()) / math.sqrt(want.numel())
        worst = float((err.sqrt() / (count.sqrt() * size)).max())
        assert worst <= 3 * tol, worst


def place(x, shift, dtype=None):
    """x in memory that begins `shift` elements after an aligned address."""
    dtype = dtype or x.dtype
    return torch.empty(x.numel() + 8, device="cuda", dtype=dtype)[shift:shift + x.numel()].view(x.shape).copy_(x)


class Step:
    """A handle for steps, its buffers and their binary64 counterparts."""

    def __init__(self, shapes, dtype=torch.float32, shift=0, zero=False, spectrum="gauss", **kw):
        self.shapes = shapes
        self.grads = [place(matrix(s, 3 * i + s[0], spectrum).to(dtype), shift) for i, s in enumerate(shapes)]
        self.momentum = [place(torch.zeros(s, device="cuda"), shift) for s in shapes]
        self.master = [place(matrix(s, 70 + i) * (0.0 if zero else 20.0), shift) for i, s in enumerate(shapes)]
        self.weights = [place(torch.zeros(s, device="cuda", dtype=torch.bfloat16), shift) for s in shapes]
        self.muon = O.z1_muon_create(shapes, self.grads, momentum=self.momentum, master=self.master,
                                     weights=self.weights, **kw)

    def __call__(self, **hp):
        O.z1_muon_step(self.muon, **hp)
        torch.cuda.synchronize()
        for p, w in zip(self.master, self.weights):
            assert torch.equal(w, p.to(torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shapes", LARGE, ids=str)
def test_large_orthogonalize(shapes, dtype):
    gs = [matrix(s, 5 * i + s[0]).to(dtype) for i, s in enumerate(shapes)]
    out = [torch.full(s, float("nan"), device="cuda", dtype=torch.bfloat16) for s in shapes]
    m = O.z1_muon_create(shapes, gs, ortho=out)
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    for g, o in zip(gs, out):
        check(o, orthogonal(g), TOL + HALF)
    first = [o.clone() for o in out]
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    m.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shapes", LARGE + TILED, ids=str)
def test_step_writes_the_whole_update(shapes, dtype):
    """From a zero master with lr 1 the master is -O itself; a second step adds
    momentum, decay and clipping."""
    st = Step(shapes, dtype, zero=True)
    st(lr=1.0, momentum=0.0)
    for g, p, mo in zip(st.grads, st.master, st.momentum):
        assert torch.equal(mo, g.float())
        check(-p, orthogonal(g), TOL)
    S = torch.tensor([1e-2], dtype=torch.float64, device="cuda")
    c = 0.05 / (0.1 + 1e-6)
    was = [p.double() for p in st.master]
    st(lr=0.5, momentum=0.9, weight_decay=0.25, clip=0.05, d_S=S)
    for g, p, mo, w in zip(st.grads, st.master, st.momentum, was):
        # the clip factor, its product with g, 0.9 mom + cg: four roundings
        mom = 0.9 * g.double() + c * g.double()
        assert rel(mo, mom) <= 4 * 2.0 ** -24
        step = (w * (1 - 0.5 * 0.25) - p.double()) / 0.5
        want = orthogonal(c * g.double() + 0.9 * mom)
        check(step, want, TOL + 2.0 ** -23 * 2 * float(w.norm() / want.norm()))
    st.muon.close()


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shapes", TILED + SMALL + [[(2047, 2049), (2049, 2047)] * 2], ids=str)
def test_unaligned_buffers_and_their_weights(shapes, dtype, shift):
    st = Step(shapes, dtype, shift, zero=True)
    st(lr=1.0, momentum=0.0)
    for s, g, p, mo in zip(shapes, st.grads, st.master, st.momentum):
        assert torch.equal(mo, g.float())
        few = min(s) < 16
        check(-p, orthogonal(g), 5.2e-2 if few else TOL, by_block=not few)
    st.muon.close()
    out = [place(torch.zeros(s, device="cuda", dtype=torch.bfloat16), shift) for s in shapes]
    m = O.z1_muon_create(shapes, st.grads, ortho=out)
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    for o, p in zip(out, st.master):
        assert torch.equal(o, (-p).to(torch.bfloat16))     # the same iteration
    m.close()


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shapes", [TILED[4], [(96, 200), (300, 130), (33, 7), (1030, 300)]], ids=str)
def test_steps_on_bf16_gradients(shapes, nesterov):
    """Three clipped steps with per-matrix scales, as test_gpu_muon.py does with
    fp32 gradients."""
    lr_s, wd_s = [0.2 * math.sqrt(max(s)) for s in shapes], [1.0, 0.0, 2.0, 1.0]
    st = Step(shapes, torch.bfloat16, lr_scale=lr_s, wd_scale=wd_s)
    rm, rp = [x.double() for x in st.momentum], [x.double() for x in st.master]
    S, c, lr = torch.tensor([4.0], dtype=torch.float64, device="cuda"), 0.5 / (2.0 + 1e-6), 2e-3
    for step in range(3):
        st(lr=lr, momentum=0.9, weight_decay=0.1, nesterov=nesterov, clip=0.5, d_S=S)
        for i, s in enumerate(shapes):
            g = c * st.grads[i].double()
            rm[i] = 0.9 * rm[i] + g
            q = orthogonal(g + 0.9 * rm[i] if nesterov else rm[i])
            rp[i] = rp[i] * (1 - lr * 0.1 * wd_s[i]) - lr * lr_s[i] * q
            assert rel(st.momentum[i], rm[i]) <= 4 * (step + 1) * 2.0 ** -24
            tol = (TOL if min(s) >= 16 else 5.2e-2) * lr * lr_s[i] * float(q.norm())
            off = float((st.master[i].double() - rp[i]).norm())
            assert off <= (step + 1) * (tol + 2.0 ** -23 * float(rp[i].norm())), (i, step)
    st.muon.close()


@pytest.mark.parametrize("coeffs,steps", [((1.5, -0.5, 0.0), 12), ((2.0, -1.5, 0.5), 9), (O.MUON_COEFFS, 1),
                                          (O.MUON_COEFFS, 2), (O.MUON_COEFFS, 4), (O.MUON_COEFFS, 6)], ids=str)
@pytest.mark.parametrize("shapes", TILED, ids=str)
def test_tiled_steps_and_coefficients(shapes, coeffs, steps):
    gs = [matrix(s, i) for i, s in enumerate(shapes)]
    out = [torch.full(s, float("nan"), device="cuda", dtype=torch.bfloat16) for s in shapes]
    m = O.z1_muon_create(shapes, gs, ortho=out, ns_steps=steps, coeffs=coeffs)
    for again in range(2):
        O.z1_muon_orthogonalize(m)
        torch.cuda.synchronize()
        for g, o in zip(gs, out):
            check(o, orthogonal(g, steps, coeffs), math.sqrt(max(1.0, steps / 5)) * TOL + HALF)
    m.close()


@pytest.mark.parametrize("steps", [1, 2, 5])
@pytest.mark.parametrize("shapes", [TILED[4], [(170, 4100)] * 4, [(1601, 150)] * 4], ids=str)
def test_tiled_zero_and_nonfinite_stay_in_their_matrix(shapes, steps):
    gs = [matrix(s, i) for i, s in enumerate(shapes)]
    clean = [g.clone() for g in gs]
    gs[0].zero_()
    gs[1][3, 5] = float("nan")
    gs[2][0, 0] = float("inf")
    out = [torch.full(s, 7.0, device="cuda", dtype=torch.bfloat16) for s in shapes]
    m = O.z1_muon_create(shapes, gs, ortho=out, ns_steps=steps)
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    assert (out[0] == 0).all() and torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
    check(out[3], orthogonal(gs[3], steps), TOL + HALF)
    for g, x in zip(gs, clean):      # nothing of it stays in the workspace
        g.copy_(x)
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    for g, o in zip(gs, out):
        check(o, orthogonal(g, steps), TOL + HALF)
    m.close()


@pytest.mark.parametrize("shapes", [[(257, 259)], [(1030, 300)]], ids=str)
@pytest.mark.parametrize("factor", [1e-30, 1e-12, 1e20, 1e37])
def test_tiled_scale_of_the_gradient_does_not_matter(shapes, factor):
    g = (matrix(shapes[0], 1) * 1e3).clamp(-3, 3) * factor
    out = torch.zeros(shapes[0], device="cuda", dtype=torch.bfloat16)
    m = O.z1_muon_create(shapes, [g], ortho=[out], eps=0.0)
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    check(out, orthogonal(g, eps=0.0), TOL + HALF)
    m.close()


@pytest.mark.parametrize("shapes", [[(257, 259)], [(170, 4100)], [(2048, 2048)] * 4], ids=str)
def test_tiled_eps_counts(shapes):
    """One linear step: O = U / (|U| + eps), to the rounding of the output (and
    of the products, which add 0 here)."""
    gs = [matrix(s, 3 + i) for i, s in enumerate(shapes)]
    eps = float(gs[0].norm())
    out = [torch.zeros(s, device="cuda", dtype=torch.bfloat16) for s in shapes]
    m = O.z1_muon_create(shapes, gs, ortho=out, eps=eps, ns_steps=1, coeffs=(1.0, 0.0, 0.0))
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    for g, o in zip(gs, out):
        check(o, g.double() / (g.double().norm() + eps), HALF)
    m.close()


def test_a_low_rank_gradient_on_large_tiles():
    """Few strong directions over a floor of 1%: the remainder of X is carried
    through the 256 tiles."""
    shapes = [(4001, 9003)]
    st = Step(shapes, zero=True, spectrum="lowrank")
    st(lr=1.0, momentum=0.0)
    check(-st.master[0], orthogonal(st.grads[0]), TOL, by_block=False)
    st.muon.close()


def wide_tol(shape):
    """Wide products: the operands keep 22 bits (2^-22 off, and as much again
    for the product left out), and 3 K / 16 products are added in fp32 (2^-24
    each, in squares).  The amplification over five steps is that counted in
    test_gpu_muon.py, 26 / sqrt(3) in squares and 5 * 21 in a plain sum."""
    off = math.sqrt(2.0) * 2.0 ** -22 + math.sqrt(3 * max(max(shape), 64) / 16) * 2.0 ** -24
    return (26 / math.sqrt(3) if min(shape) >= 16 else 105) * off


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shapes", LARGE + TILED + SMALL + [[(2, 3), (96, 200), (5, 1)]], ids=str)
def test_wide_products(shapes, dtype):
    """A step from a zero master is -O itself; the orthogonalisation is that,
    rounded, and repeats its bits."""
    st = Step(shapes, dtype, zero=True, wide=True)
    st(lr=1.0, momentum=0.0)
    for s, g, p in zip(shapes, st.grads, st.master):
        check(-p, orthogonal(g), wide_tol(s), by_block=min(s) >= 16)
    st.muon.close()
    out = [torch.full(s, float("nan"), device="cuda", dtype=torch.bfloat16) for s in shapes]
    m = O.z1_muon_create(shapes, st.grads, ortho=out, wide=True)
    for again in range(2):
        O.z1_muon_orthogonalize(m)
        torch.cuda.synchronize()
        for o, p in zip(out, st.master):
            assert torch.equal(o, (-p).to(torch.bfloat16))
            o.fill_(7.0)
    m.close()


@pytest.mark.parametrize("shapes", [[(64, 96)], [(300, 1030)], [(2048, 2048)] * 4, [(4001, 9003)]], ids=str)
def test_wide_low_rank(shapes):
    st = Step(shapes, zero=True, spectrum="lowrank", wide=True)
    st(lr=1.0, momentum=0.0)
    for s, g, p in zip(shapes, st.grads, st.master):
        check(-p, orthogonal(g), wide_tol(s), by_block=False)
    st.muon.close()


@pytest.mark.parametrize("coeffs,steps", [((1.5, -0.5, 0.0), 12), (O.MUON_COEFFS, 1), (O.MUON_COEFFS, 2)], ids=str)
@pytest.mark.parametrize("shift", [0, 1])
def test_wide_steps_and_buffers(coeffs, steps, shift):
    shapes = TILED[4] + [(64, 96)]
    st = Step(shapes, torch.float32, shift, zero=True, wide=True, coeffs=coeffs, ns_steps=steps)
    st(lr=1.0, momentum=0.0)
    for s, g, p in zip(shapes, st.grads, st.master):
        check(-p, orthogonal(g, steps, coeffs), math.sqrt(max(1.0, steps / 5)) * wide_tol(s))
    st.muon.close()


@pytest.mark.parametrize("shapes", [TILED[4], [(170, 4100)] * 4], ids=str)
def test_wide_zero_and_nonfinite_stay_in_their_matrix(shapes):
    st = Step(shapes, zero=True, wide=True)
    clean = [g.clone() for g in st.grads]
    st.grads[0].zero_()
    st.grads[1][3, 5] = float("nan")
    st.grads[2][0, 0] = float("inf")
    O.z1_muon_step(st.muon, lr=1.0, momentum=0.0)
    torch.cuda.synchronize()
    assert (st.master[0] == 0).all() and torch.isnan(st.master[1]).all() and torch.isnan(st.master[2]).all()
    check(-st.master[3], orthogonal(st.grads[3]), wide_tol(shapes[3]))
    for g, x, mo, p in zip(st.grads, clean, st.momentum, st.master):
        g.copy_(x)
        mo.zero_()
        p.zero_()
    st(lr=1.0, momentum=0.0)
    for s, g, p in zip(shapes, st.grads, st.master):
        check(-p, orthogonal(g), wide_tol(s))
    st.muon.close()


def test_wide_in_a_graph_and_on_another_stream():
    shapes = [(300, 200), (128, 512), (170, 4100)]
    gs = [matrix(s, i) for i, s in enumerate(shapes)]
    out = [torch.zeros(s, device="cuda", dtype=torch.bfloat16) for s in shapes]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m = O.z1_muon_create(shapes, gs, ortho=out, wide=True, stream=s)
    O.z1_muon_orthogonalize(m, stream=s)
    s.synchronize()
    first = [o.clone() for o in out]
    for g, o in zip(gs, out):
        check(o, orthogonal(g), HALF + 1e-4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O.z1_muon_orthogonalize(m)
    for k in range(4):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, out)), k
        O.z1_muon_orthogonalize(m)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, out)), k
    m.close()


def test_wide_through_muon_step_and_an_empty_list():
    from mixed_precision_zero_amd.muon import MuonStep
    shapes = [(64, 96), (300, 130)]
    st = MuonStep(shapes, 1, wide=True)
    g = torch.Generator(device="cuda").manual_seed(0)
    for t in st.grads[0]:
        t.copy_(torch.randn(t.shape, generator=g, device="cuda") * 1e-3)
    st.step(lr=1.0, momentum=0.0)
    torch.cuda.synchronize()
    for s, t, p in zip(shapes, st.grads[0], st.views(st.master)):
        check(-p, orthogonal(t), wide_tol(s))
    st.close()
    m = O.z1_muon_create([], [], ortho=[], wide=True)
    O.z1_muon_orthogonalize(m)
    m.close()
