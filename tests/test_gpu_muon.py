"""z1_muon_step and z1_muon_orthogonalize against the definition in binary64.

Tolerance of the orthogonalised matrix O (relative, 2-norm over all elements).
One step X <- a X + B X, B = b A + c A A, rounds the operands X, A and B to
fp16, u = 2^-11 relative.  With |A| <= 1.446, |B| <= 2.81, |b| = 4.775 and
c = 2.0315 a rounding of X, of B and of A reaches the new X with at most 2.81,
2.81, |b| 1.446 = 6.9 and 2 c 1.446^2 = 8.5 times its size.  Roundings are
spread evenly within half a step, so their root mean square is u / sqrt(3) and
five steps add up in squares: sqrt(5 (2 * 2.81^2 + 6.9^2 + 8.5^2)) u / sqrt(3)
= 7.3e-3.  Where a matrix has few elements (one side below 16) the roundings do
not average, and the bound is the plain sum, 5 * 21 u = 5.2e-2.  The bf16
output adds 2^-8."""
import math

import pytest
import torch

from mixed_precision_zero_amd import binding as B
from mixed_precision_zero_amd import ops as O

pytestmark = pytest.mark.gpu
A_, B_, C_ = O.MUON_COEFFS


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def tol(shape):
    return (7.3e-3 if min(shape) >= 16 else 5.2e-2) + 2.0 ** -8


def rel(x, y):
    return float((x.double() - y).norm() / y.norm()) if float(y.norm()) else float(x.double().norm())


def orthogonal(u, steps=5, coeffs=(A_, B_, C_), eps=1e-7):
    a, b, c = coeffs
    x = u.double()
    flip = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if flip else x
    x = x / (x.norm() + eps)
    for _ in range(steps):
        g = x @ x.t()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.t() if flip else x


def matrix(shape, seed, spectrum="gauss"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    if spectrum == "lowrank":
        u = torch.randn(shape[0], 4, generator=g, device="cuda")
        x = 0.01 * x + u @ torch.randn(4, shape[1], generator=g, device="cuda")
    return x * 1e-3


SHAPES = [[(1, 1)], [(1, 300)], [(300, 1)], [(2, 3)], [(64, 64)], [(65, 129)], [(200, 72)], [(64, 512)], [(33, 1000)], [(96, 288)], [(160, 128)], [(161, 128)], [(1024, 32)],
          [(512, 1000), (64, 64), (1000, 512), (1, 5)], [(127, 128), (128, 127)],
          [(2304, 700)], [(170, 4100)], [(200, 3000), (8000, 70)], [(150, 1600), (64, 64)], [(2048, 2048), (2048, 2048)], [(2100, 5000)]]


@pytest.mark.parametrize("spectrum", ["gauss", "lowrank"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shapes", SHAPES, ids=str)
def test_orthogonalize(shapes, dtype, spectrum):
    gs = [matrix(s, 7 * i + s[0], spectrum).to(dtype) for i, s in enumerate(shapes)]
    out = [torch.full(s, float("nan"), device="cuda", dtype=torch.bfloat16) for s in shapes]
    m = O.z1_muon_create(shapes, gs, ortho=out)
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    for s, g, o in zip(shapes, gs, out):
        assert rel(o, orthogonal(g)) <= tol(s), s
    first = [o.clone() for o in out]
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    m.close()


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("clip", [0.0, 0.5, 1e9])
def test_step(nesterov, clip):
    shapes = [(96, 200), (576, 192), (33, 7), (256, 256)]
    hp = dict(lr=2e-3, momentum=0.9, weight_decay=0.1, nesterov=nesterov, clip=clip)
    lr_s, wd_s = [0.2 * math.sqrt(max(s)) for s in shapes], [1.0, 0.0, 2.0, 1.0]
    gs = [matrix(s, i) for i, s in enumerate(shapes)]
    mom = [torch.zeros(s, device="cuda") for s in shapes]
    master = [matrix(s, 50 + i) * 20 for i, s in enumerate(shapes)]
    w = [torch.zeros(s, device="cuda", dtype=torch.bfloat16) for s in shapes]
    S = torch.tensor([4.0], dtype=torch.float64, device="cuda")
    rm, rp = [x.double() for x in mom], [x.double() for x in master]
    m = O.z1_muon_create(shapes, gs, momentum=mom, master=master, weights=w, lr_scale=lr_s, wd_scale=wd_s)
    for step in range(3):
        O.z1_muon_step(m, d_S=S, **hp)
        torch.cuda.synchronize()
        c = min(1.0, clip / (2.0 + 1e-6)) if clip > 0 else 1.0
        for i, s in enumerate(shapes):
            g = c * gs[i].double()
            rm[i] = 0.9 * rm[i] + g
            q = orthogonal(g + 0.9 * rm[i] if nesterov else rm[i])
            rp[i] = rp[i] * (1 - hp["lr"] * 0.1 * wd_s[i]) - hp["lr"] * lr_s[i] * q
            # fp32 momentum: three roundings a step, halved sizes ahead
            assert rel(mom[i], rm[i]) <= 4 * (step + 1) * 2.0 ** -24
            off = (master[i].double() - rp[i]).norm()
            step_norm = hp["lr"] * lr_s[i] * q.norm()
            assert off <= (step + 1) * (tol(s) * step_norm + 2.0 ** -23 * rp[i].norm()), (i, step)
            assert torch.equal(w[i], master[i].to(torch.bfloat16))
        gs[0].mul_(0.5)   # bound buffers are read anew each step
    m.close()


def test_zero_and_nonfinite_stay_in_their_matrix():
    shapes = [(64, 96), (64, 96), (64, 96), (80, 64)]
    gs = [matrix(s, i) for i, s in enumerate(shapes)]
    gs[0].zero_()
    gs[1][3, 5] = float("nan")
    gs[2][0, 0] = float("inf")
    out = [torch.zeros(s, device="cuda", dtype=torch.bfloat16) for s in shapes]
    m = O.z1_muon_create(shapes, gs, ortho=out)
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    assert (out[0] == 0).all()
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
    assert rel(out[3], orthogonal(gs[3])) <= tol(shapes[3])
    for g in gs[:3]:      # nothing of it stays in the workspace
        g.copy_(matrix((64, 96), 9))
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    for i in range(3):
        assert rel(out[i], orthogonal(gs[i])) <= tol(shapes[i])


@pytest.mark.parametrize("factor", [1e-30, 1e-12, 1e20, 1e37])
def test_scale_of_the_gradient_does_not_matter(factor):
    g = (matrix((96, 128), 1) * 1e3).clamp(-3, 3) * factor
    out = torch.zeros(96, 128, device="cuda", dtype=torch.bfloat16)
    m = O.z1_muon_create([(96, 128)], [g], ortho=[out], eps=0.0)
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    assert rel(out, orthogonal(g, eps=0.0)) <= tol((96, 128))


def test_eps_counts():
    g = matrix((64, 64), 3)
    eps = float(g.norm())
    out = torch.zeros(64, 64, device="cuda", dtype=torch.bfloat16)
    m = O.z1_muon_create([(64, 64)], [g], ortho=[out], eps=eps, ns_steps=1, coeffs=(1.0, 0.0, 0.0))
    O.z1_muon_orthogonalize(m)
    torch.cuda.synchronize()
    assert rel(out, g.double() / (2 * eps)) <= 2.0 ** -8


def test_other_coefficients_and_steps():
    g = matrix((100, 140), 3)
    out = torch.zeros(100, 140, device="cuda", dtype=torch.bfloat16)
    for coeffs, steps in (((1.5, -0.5, 0.0), 12), ((2.0, -1.5, 0.5), 9), (O.MUON_COEFFS, 1), (O.MUON_COEFFS, 2)):
        m = O.z1_muon_create([(100, 140)], [g], ortho=[out], ns_steps=steps, coeffs=coeffs)
        O.z1_muon_orthogonalize(m)
        torch.cuda.synchronize()
        assert rel(out, orthogonal(g, steps, coeffs)) <= math.sqrt(max(1.0, steps / 5)) * 7.3e-3 + 2.0 ** -8


def test_unaligned_matrices():
    shapes = [(70, 90), (90, 70)]
    for shift in (1, 2, 3):
        place = lambda x, t: torch.empty(x.numel() + 8, device="cuda", dtype=t)[shift:shift + x.numel()].view(x.shape)  # noqa: E731
        src = [matrix(s, i) for i, s in enumerate(shapes)]
        gs = [place(x, torch.float32).copy_(x) for x in src]
        mom = [place(x, torch.float32).zero_() for x in src]
        master = [place(x, torch.float32).zero_() for x in src]
        w = [place(x, torch.bfloat16) for x in src]
        m = O.z1_muon_create(shapes, gs, momentum=mom, master=master, weights=w)
        O.z1_muon_step(m, lr=1.0, momentum=0.0)
        torch.cuda.synchronize()
        for s, g, p, mo in zip(shapes, src, master, mom):
            assert torch.equal(mo, g)
            assert rel(-p, orthogonal(g)) <= tol(s)


def test_state_errors_and_empty_list():
    g, o = matrix((8, 8), 0), torch.zeros(8, 8, device="cuda", dtype=torch.bfloat16)
    m = O.z1_muon_create([(8, 8)], [g], ortho=[o])
    with pytest.raises(B.Z1Error) as e:
        O.z1_muon_step(m, lr=1e-3)
    assert e.value.status == B.Z1_ESTATE
    p = torch.zeros(8, 8, device="cuda")
    m = O.z1_muon_create([(8, 8)], [g], momentum=[p], master=[p.clone()], weights=[o])
    with pytest.raises(B.Z1Error) as e:
        O.z1_muon_orthogonalize(m)
    assert e.value.status == B.Z1_ESTATE
    for bad in (dict(lr=float("nan")), dict(lr=1.0, momentum=1.0), dict(lr=1.0, momentum=-0.1),
                dict(lr=1.0, weight_decay=-1.0), dict(lr=1.0, clip=1.0)):
        with pytest.raises(B.Z1Error) as e:
            O.z1_muon_step(m, **bad)
        assert e.value.status == B.Z1_EINVAL
    m = O.z1_muon_create([], [], ortho=[])
    O.z1_muon_orthogonalize(m)
    m.close()


def test_other_stream_and_graph():
    shapes = [(300, 200), (128, 512)]
    gs = [matrix(s, i) for i, s in enumerate(shapes)]
    want = [orthogonal(g) for g in gs]
    out = [torch.zeros(s, device="cuda", dtype=torch.bfloat16) for s in shapes]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m = O.z1_muon_create(shapes, gs, ortho=out, stream=s)
    O.z1_muon_orthogonalize(m, stream=s)
    s.synchronize()
    assert all(rel(o, q) <= tol(sh) for o, q, sh in zip(out, want, shapes))
    first = [o.clone() for o in out]
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


def test_orthogonal_rows():
    """What the operator is for: singular values near 1 (the iteration's own
    band is about 0.68 to 1.13 after five steps; a gaussian has some that start
    too small for it)."""
    g = matrix((128, 1024), 5)
    out = torch.zeros(128, 1024, device="cuda", dtype=torch.bfloat16)
    O.z1_muon_orthogonalize(O.z1_muon_create([(128, 1024)], [g], ortho=[out]))
    s = torch.linalg.svdvals(out.double().cpu())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.25
