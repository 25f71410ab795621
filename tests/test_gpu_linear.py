"""z1_linear, z1_linear_dz and z1_linear_grad against their definitions in 64 bits.

Tolerances.  A product of depth K sums exact products (fp16 and bf16 operands) or
products rounded once (fp32) in fp32: at most K + 8 roundings of 2^-24 of the sum
of the magnitudes S = sum |x w|, whatever the order; the bias is one more.  The
result is rounded once to its type: half a step.  An activation multiplies an
error by at most 1.2 (its largest slope: GELU 1.13, its tanh form 1.13, SILU 1.1;
RELU2 by 2 |z|), and its own evaluation in fp32 (exponential, reciprocal, erfc: a
few units in the last place, the exponent's argument rounded at its size) is off
by at most 2^-20 of max(1, |z|)^2."""
import pytest
import torch

from layer_refs import TYPES, U32, act, drop, half_step, near, placed, tiny, untouched
from mixed_precision_zero_amd import layers as L

pytestmark = pytest.mark.gpu
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "relu2")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rand(g, *shape, t=torch.float32, by=1.0):
    return (torch.randn(*shape, generator=g) * by).to(t)


def workspace(n):
    """Just as large as asked, in the middle of a guarded buffer."""
    buf = torch.full((n + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    return buf[256:256 + n], buf


def guards(buf, n):
    return bool((buf[:256] == 0x5a).all()) and bool((buf[256 + n:] == 0x5a).all())


def rng(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def epilogue_tol(z, dz, name, scale=1.0):
    """How far act(z) may be off where z is off by dz."""
    slope = 1.2 if name != "relu2" else 2 * z.abs() + 2 * dz
    own = 0.0 if name in ("none", "relu") else 2.0 ** -20 * z.abs().clamp(min=1) ** 2
    return (slope * dz + own) * scale


def check_linear(t, rows, inner, outer, name="none", bias=False, mul=False, residual=False, pre=False, p=0.0, layout="plain", seed=0):
    g = torch.Generator().manual_seed(seed)
    x, w = rand(g, rows, inner, t=t), rand(g, outer, inner, t=t, by=inner ** -0.5)
    b = rand(g, outer, t=t) if bias else None
    m, r = (rand(g, rows, outer, t=t) if on else None for on in (mul, residual))
    z = x.double() @ w.double().t() + (b.double() if bias else 0.0)
    dz = (inner + 9) * U32 * (x.double().abs() @ w.double().abs().t() + (b.double().abs() if bias else 0.0))
    y, dy = act(z, name)[0], epilogue_tol(z, dz, name)
    if mul:
        y, dy = y * m.double(), dy * m.double().abs() + U32 * (y * m.double()).abs()
    y = drop(y, 1234567890123, 77 + 3, p)
    dy = dy / (1 - p) + 2 * U32 * y.abs() if p else dy
    if residual:
        y, dy = y + r.double(), dy + U32 * (y + r.double()).abs()
    at = lambda v: placed(v, layout)[0] if v is not None else None  # noqa: E731
    gx, gw, gm, gr = at(x), at(w), at(m), at(r)
    out, out_buf = placed(torch.zeros(rows, outer, dtype=t), layout)
    kept, kept_buf = placed(torch.zeros(rows, outer, dtype=t), layout) if pre else (None, None)
    n = L.z1_linear_workspace(gx, gw)
    ws, ws_buf = workspace(n)
    d = L.Dropout(rng(1234567890123, 77), p, 3) if p else None
    L.z1_linear(gx, gw, out, bias=b.cuda() if bias else None, act=name, mul=gm, residual=gr, pre=kept, dropout=d, workspace=ws)
    torch.cuda.synchronize()
    near(out, y, dy + half_step(t) * y.abs() * (1 + 2.0 ** -8) + tiny(t), "y")
    if pre:
        near(kept, z, dz + half_step(t) * z.abs() * (1 + 2.0 ** -8) + tiny(t), "pre")
    assert untouched(out, out_buf) and (not pre or untouched(kept, kept_buf)) and guards(ws_buf, n)
    return out


SHAPES = [(1, 1, 1), (1, 8, 16), (1, 333, 77), (2, 2048, 64), (3, 5, 7), (5, 64, 1), (16, 513, 33), (17, 96, 130), (31, 8, 65),
          (64, 64, 64), (65, 32, 63), (100, 100, 100), (129, 1000, 257), (200, 24, 1537), (333, 40, 511), (257, 2056, 96)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_product(kind, shape):
    check_linear(TYPES[kind], *shape, seed=sum(shape))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", [(1, 333, 77), (7, 512, 40), (70, 129, 200), (130, 256, 136)])
@pytest.mark.parametrize("layout", ["ld", "odd"])
def test_product_of_other_layouts(kind, shape, layout):
    check_linear(TYPES[kind], *shape, layout=layout, bias=True, residual=True, pre=True, mul=True, name="silu")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("rows,inner,outer", [(1, 72, 40), (9, 64, 37), (70, 600, 75), (128, 32, 264)])
def test_epilogue(kind, name, rows, inner, outer):
    check_linear(TYPES[kind], rows, inner, outer, name=name, bias=True, pre=name != "none", mul=name in ("silu", "gelu"),
                 residual=name in ("gelu", "none"), p=0.25 if name in ("relu", "gelu") else 0.0)


@pytest.mark.parametrize("kind,shape", [("bf16", (2500, 130, 4200)), ("f16", (4100, 72, 2600)), ("f32", (1700, 100, 2100)),
                                        ("bf16", (4096, 320, 2816)), ("f16", (1, 70000, 24)), ("bf16", (33, 30000, 96))])
def test_large_products(kind, shape):
    """Every tile side, deep and shallow, edges in both directions."""
    check_linear(TYPES[kind], *shape, bias=True, residual=True, p=0.1)


def test_no_rows():
    for t in TYPES.values():
        x, w, y = (torch.empty(s, dtype=t, device="cuda") for s in ((0, 8), (4, 8), (0, 4)))
        L.z1_linear(x, w, y)
        dw = torch.full((4, 8), 3.0, device="cuda")
        L.z1_linear_grad(y, x, w, dx=x, dweight=dw, accumulate=True, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
        assert bool((dw == 3.0).all())
        L.z1_linear_grad(y, x, w, dweight=dw, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
        assert bool((dw == 0.0).all())
        db = torch.full((4,), 2.0, device="cuda")
        L.z1_linear_dz(y, dbias=db, accumulate=True)
        assert bool((db == 2.0).all())
        L.z1_linear_dz(y, dbias=db)
        assert bool((db == 0.0).all())


@pytest.mark.parametrize("kind", TYPES)
def test_y_over_residual_or_mul(kind):
    t = TYPES[kind]
    g = torch.Generator().manual_seed(3)
    for rows, inner, outer in ((1, 64, 48), (70, 520, 75), (300, 64, 264)):
        x, w, r = rand(g, rows, inner, t=t).cuda(), rand(g, outer, inner, t=t, by=0.1).cuda(), rand(g, rows, outer, t=t).cuda()
        ws = torch.empty(L.z1_linear_workspace(x, w), dtype=torch.uint8, device="cuda")
        for name in ("residual", "mul"):
            apart, over = torch.empty_like(r), r.clone()
            L.z1_linear(x, w, apart, act="silu", workspace=ws, **{name: r})
            L.z1_linear(x, w, over, act="silu", workspace=ws, **{name: over})
            assert torch.equal(apart, over)


@pytest.mark.parametrize("kind", TYPES)
def test_what_is_not_finite_stays_in_its_row_and_column(kind):
    t = TYPES[kind]
    for rows, inner, outer in ((1, 40, 24), (20, 333, 40), (90, 64, 70)):
        x, w = torch.ones(rows, inner, dtype=t), torch.ones(outer, inner, dtype=t)
        x[rows - 1, inner - 1], w[outer - 1, 0] = float("inf"), float("nan")
        gx, gw = placed(x, "odd")[0], placed(w, "odd")[0]
        y = torch.empty(rows, outer, dtype=t, device="cuda")
        L.z1_linear(gx, gw, y, workspace=torch.empty(L.z1_linear_workspace(gx, gw), dtype=torch.uint8, device="cuda"))
        want = torch.full((rows, outer), float(inner), dtype=torch.float64)
        want[rows - 1] = float("inf")
        want[:, outer - 1] = float("nan")
        near(y, want, half_step(t) * want.abs().nan_to_num(posinf=0.0), "y")
        # dropped elements are zero whatever they were
        d = L.Dropout(rng(5, 6), 1.0)
        L.z1_linear(gx, gw, y, dropout=d, workspace=torch.empty(L.z1_linear_workspace(gx, gw), dtype=torch.uint8, device="cuda"))
        assert bool((y == 0).all())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("rows,outer,layout", [(1, 1, "plain"), (1, 40, "plain"), (63, 75, "plain"), (200, 264, "ld"), (77, 33, "odd"), (1000, 520, "plain")])
def test_gradient_through_the_epilogue(kind, name, rows, outer, layout):
    """The slope is off by at most 2^-20 max(1, |z|)^2 (as the activation above);
    dbias sums `rows` terms: rows + 8 roundings of the magnitudes' sum, and each
    term's own error."""
    t = TYPES[kind]
    g = torch.Generator().manual_seed(rows + outer)
    mul, p = name != "relu", 0.5 if name in ("none", "silu") else 0.0
    dy, z, m = rand(g, rows, outer, t=t), rand(g, rows, outer, t=t, by=2.0), rand(g, rows, outer, t=t)
    z[0, 0] = 0.0
    up, slope = act(z.double(), name)
    gr = drop(dy.double(), 99, 2 ** 40 + 1, p)
    dmul, dz = gr * up, gr * (m.double() if mul else 1.0) * slope
    own = (2.0 ** -20 * z.double().abs().clamp(min=1) ** 2 if name not in ("none", "relu") else torch.zeros_like(dz)) + 4 * U32 * slope.abs()
    e_mul = gr.abs() * (2.0 ** -20 * z.double().abs().clamp(min=1) ** 2 + 4 * U32 * up.abs())
    e_dz = gr.abs() * (m.double().abs() if mul else 1.0) * own
    at = lambda v: placed(v, layout)[0]  # noqa: E731
    out, out_buf = placed(torch.zeros_like(dy), layout)
    om, om_buf = placed(torch.zeros_like(dy), layout)
    db = torch.full((outer,), 0.5, device="cuda")
    n = L.z1_linear_dz_workspace(rows, outer)
    ws, ws_buf = workspace(n)
    d = L.Dropout(rng(99, 2 ** 40), p, 1) if p else None
    L.z1_linear_dz(at(dy), out, act=name, pre=at(z), mul=at(m) if mul else None, dmul=om, dbias=db, accumulate=True, dropout=d, workspace=ws)
    torch.cuda.synchronize()
    near(out, dz, e_dz + half_step(t) * dz.abs() * (1 + 2.0 ** -8) + tiny(t), "dz")
    near(om, dmul, e_mul + half_step(t) * dmul.abs() * (1 + 2.0 ** -8) + tiny(t), "dmul")
    near(db, dz.sum(0) + 0.5, e_dz.sum(0) + (rows + 9) * U32 * (dz.abs().sum(0) + 0.5), "dbias")
    assert untouched(out, out_buf) and untouched(om, om_buf) and guards(ws_buf, n)
    # written, and over its own inputs
    first = db.clone()
    a, b = at(dy), at(z)
    L.z1_linear_dz(a, a, act=name, pre=b, mul=at(m) if mul else None, dmul=b, dbias=db, dropout=d, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(a, out) and torch.equal(b, om)
    near(db, first.double().cpu() - 0.5, 2 * U32 * (first.double().cpu().abs() + 1), "dbias written")


def test_dbias_alone_and_dz_alone():
    g = torch.Generator().manual_seed(0)
    dy = rand(g, 300, 130, t=torch.bfloat16)
    db = torch.empty(130, device="cuda")
    ws = torch.empty(L.z1_linear_dz_workspace(300, 130), dtype=torch.uint8, device="cuda")
    L.z1_linear_dz(dy.cuda(), dbias=db, workspace=ws)
    near(db, dy.double().sum(0), 308 * U32 * dy.double().abs().sum(0), "dbias")
    dz = torch.empty(300, 130, dtype=torch.bfloat16, device="cuda")
    L.z1_linear_dz(dy.cuda(), dz, act="relu", pre=dy.cuda())
    assert torch.equal(dz.cpu(), torch.where(dy > 0, dy, torch.zeros_like(dy)))


def check_grad(t, rows, inner, outer, layout="plain", dw_type=torch.float32, accumulate=False, add=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    dz, x, w = rand(g, rows, outer, t=t), rand(g, rows, inner, t=t), rand(g, outer, inner, t=t, by=outer ** -0.5)
    r = rand(g, rows, inner, t=t) if add else None
    old = rand(g, outer, inner, t=dw_type)
    want_x = dz.double() @ w.double() + (r.double() if add else 0.0)
    tol_x = (outer + 9) * U32 * (dz.double().abs() @ w.double().abs() + (r.double().abs() if add else 0.0)) + half_step(t) * want_x.abs() * (1 + 2.0 ** -8) + tiny(t)
    want_w = dz.double().t() @ x.double() + (old.double() if accumulate else 0.0)
    tol_w = (rows + 9) * U32 * (dz.double().abs().t() @ x.double().abs() + (old.double().abs() if accumulate else 0.0))
    if dw_type != torch.float32:
        tol_w = tol_w + half_step(dw_type) * want_w.abs() * (1 + 2.0 ** -8) + tiny(dw_type)
    at = lambda v: placed(v, layout)[0] if v is not None else None  # noqa: E731
    gz, gx, gw = at(dz), at(x), at(w)
    dx, dx_buf = placed(torch.zeros_like(x), layout)
    dw, dw_buf = placed(old, layout)
    n = L.z1_linear_grad_workspace(gz, gx, gw)
    ws, ws_buf = workspace(n)
    L.z1_linear_grad(gz, gx, gw, dx=dx, add=at(r), dweight=dw, accumulate=accumulate, workspace=ws)
    torch.cuda.synchronize()
    near(dx, want_x, tol_x, "dx")
    near(dw, want_w, tol_w, "dweight")
    assert untouched(dx, dx_buf) and untouched(dw, dw_buf) and guards(ws_buf, n)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(kind, shape):
    rows, inner, outer = shape
    check_grad(TYPES[kind], rows, inner, outer, accumulate=rows % 2 == 1, add=inner % 2 == 0, seed=sum(shape))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", [(1, 333, 77), (70, 129, 200), (130, 256, 136)])
@pytest.mark.parametrize("layout", ["ld", "odd"])
def test_gradients_of_other_layouts(kind, shape, layout):
    check_grad(TYPES[kind], *shape, layout=layout, add=True, accumulate=True)
    check_grad(TYPES[kind], *shape, layout=layout, dw_type=TYPES[kind])


@pytest.mark.parametrize("kind,shape", [("bf16", (2500, 4200, 130)), ("f16", (130, 2600, 4100)), ("f32", (1700, 2100, 100)),
                                        ("bf16", (4096, 2816, 320)), ("f16", (30000, 96, 33)), ("f32", (20001, 24, 40))])
def test_large_gradients(kind, shape):
    check_grad(TYPES[kind], *shape, add=True, accumulate=True)
    if kind != "f32":
        check_grad(TYPES[kind], *shape, dw_type=TYPES[kind])


def test_one_gradient_alone():
    g = torch.Generator().manual_seed(1)
    dz, x, w = (rand(g, *s, t=torch.bfloat16).cuda() for s in ((70, 40), (70, 56), (40, 56)))
    ws = torch.empty(L.z1_linear_grad_workspace(dz, x, w), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(40, 56, device="cuda")
    L.z1_linear_grad(dz, x, w, dx=dx, dweight=dw, workspace=ws)
    dx2, dw2 = torch.empty_like(x), torch.empty(40, 56, device="cuda")
    L.z1_linear_grad(dz, None, w, dx=dx2, workspace=ws)
    L.z1_linear_grad(dz, x, None, dweight=dw2, workspace=ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    # onto itself: dx may be add
    both = x.clone()
    L.z1_linear_grad(dz, None, w, dx=both, add=both, workspace=ws)
    apart = torch.empty_like(x)
    L.z1_linear_grad(dz, None, w, dx=apart, add=x, workspace=ws)
    assert torch.equal(both, apart)


def test_gradients_against_differences():
    """The whole chain in fp32: the change of sum(y dy) under a step of 2^-6 in one
    direction against the gradient's product with it.  With |f'''| h^2 / 6 of the
    centred difference and sums of at most 40 x 24 terms of order one rounded at
    2^-24 each over 2 h, 2e-3 of the sum of magnitudes covers both."""
    g = torch.Generator().manual_seed(4)
    rows, inner, outer, h = 24, 32, 40, 2.0 ** -6
    x, w, b = rand(g, rows, inner).cuda(), rand(g, outer, inner, by=inner ** -0.5).cuda(), rand(g, outer).cuda()
    m, dy = rand(g, rows, outer).cuda(), rand(g, rows, outer).cuda()
    d = L.Dropout(rng(8, 9), 0.3, 2)
    for name in ("gelu", "gelu_tanh", "silu"):
        def f(x, w, b, m):
            y = torch.empty(rows, outer, device="cuda")
            L.z1_linear(x, w, y, bias=b, act=name, mul=m, dropout=d,
                        workspace=torch.empty(L.z1_linear_workspace(x, w), dtype=torch.uint8, device="cuda"))
            return float((y.double() * dy.double()).sum())
        pre, y = torch.empty(rows, outer, device="cuda"), torch.empty(rows, outer, device="cuda")
        ws = torch.empty(max(L.z1_linear_workspace(x, w), L.z1_linear_dz_workspace(rows, outer), L.z1_linear_grad_workspace(dy, x, w)),
                         dtype=torch.uint8, device="cuda")
        L.z1_linear(x, w, y, bias=b, act=name, mul=m, pre=pre, dropout=d, workspace=ws)
        dz, dm, db = torch.empty_like(dy), torch.empty_like(dy), torch.empty(outer, device="cuda")
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        L.z1_linear_dz(dy, dz, act=name, pre=pre, mul=m, dmul=dm, dbias=db, dropout=d, workspace=ws)
        L.z1_linear_grad(dz, x, w, dx=dx, dweight=dw, workspace=ws)
        for i, (v, grad) in enumerate(((x, dx), (w, dw), (b, db), (m, dm))):
            step = torch.randn(v.shape, generator=g).cuda()
            args = [[x, w, b, m], [x, w, b, m]]
            args[0][i], args[1][i] = v + h * step, v - h * step
            got = float((grad.double() * step.double()).sum())
            diff = (f(*args[0]) - f(*args[1])) / (2 * h)
            size = float((grad.double() * step.double()).abs().sum())
            assert abs(got - diff) <= 2e-3 * size, (name, i, got, diff)


def test_same_bits_every_time_and_on_another_stream():
    g = torch.Generator().manual_seed(6)
    x, w, r = (rand(g, *s, t=torch.bfloat16).cuda() for s in ((100, 4096), (72, 4096), (100, 72)))
    ws = torch.empty(L.z1_linear_workspace(x, w), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0        # few tiles, deep: split
    first = torch.empty_like(r)
    L.z1_linear(x, w, first, residual=r, workspace=ws)
    for _ in range(3):
        y = torch.empty_like(r)
        L.z1_linear(x, w, y, residual=r, workspace=ws)
        assert torch.equal(first, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(r)
    ws2 = torch.empty_like(ws)
    with torch.cuda.stream(s):
        L.z1_linear(x, w, y, residual=r, workspace=ws2)
    y2 = torch.empty_like(r)
    L.z1_linear(x, w, y2, residual=r, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(first, y) and torch.equal(first, y2)


def test_captured_step_draws_new_masks():
    """Forward and backward in one graph; every replay against the eager calls,
    the mask moving on with the seed and offset on the device."""
    g = torch.Generator().manual_seed(7)
    rows, inner, outer = 96, 64, 136
    t = torch.bfloat16
    x, w, b, dy = (rand(g, *s, t=t).cuda() for s in ((rows, inner), (outer, inner), (outer,), (rows, outer)))
    state = rng(11, 0)
    one = torch.tensor([0, 1], dtype=torch.int64, device="cuda")
    need = max(L.z1_linear_workspace(x, w), L.z1_linear_dz_workspace(rows, outer), L.z1_linear_grad_workspace(dy, x, w))

    def buffers():
        f = lambda *s, k=t: torch.zeros(*s, dtype=k, device="cuda")  # noqa: E731
        return dict(y=f(rows, outer), pre=f(rows, outer), dz=f(rows, outer), dx=f(rows, inner), db=f(outer, k=torch.float32),
                    dw=f(outer, inner, k=torch.float32), ws=torch.zeros(need, dtype=torch.uint8, device="cuda"))

    def step(o):
        d = L.Dropout(state, 0.4, 5)
        L.z1_linear(x, w, o["y"], bias=b, act="gelu", pre=o["pre"], dropout=d, workspace=o["ws"])
        L.z1_linear_dz(dy, o["dz"], act="gelu", pre=o["pre"], dbias=o["db"], accumulate=True, dropout=d, workspace=o["ws"])
        L.z1_linear_grad(o["dz"], x, w, dx=o["dx"], dweight=o["dw"], accumulate=True, workspace=o["ws"])
        state.add_(one)

    eager, held = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(buffers())
        state.copy_(rng(11, 0))
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step(held)
    torch.cuda.synchronize()
    last = None
    for i in range(4):
        state.copy_(rng(11, i))
        step(eager)
        torch.cuda.synchronize()
        state.copy_(rng(11, i))
        graph.replay()
        torch.cuda.synchronize()
        for k in ("y", "pre", "dz", "dx", "db", "dw"):
            assert torch.equal(eager[k], held[k]), (i, k)
        assert last is None or not torch.equal(last, held["y"])
        last = held["y"].clone()
        assert state.tolist() == [11, i + 1]


@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_activations_far_from_zero(name, t):
    """Where a square of z is infinite in fp32 all of them are z or 0, and their
    slopes 1 or 0, exactly."""
    t = TYPES[t]
    z = torch.tensor([[s * v for s in (1, -1) for v in (100.0, 1e10, 2e19, 1e25, 3e38)]]).to(t).repeat(5, 1)
    dz, dm = (torch.empty_like(z, device="cuda") for _ in range(2))
    one = torch.ones_like(z, device="cuda")
    L.z1_linear_dz(one, dz, act=name, pre=z.cuda(), dmul=dm)
    torch.cuda.synchronize()
    assert torch.equal(dz.cpu(), (z > 0).to(t)) and torch.equal(dm.cpu(), z.clamp(min=0))


def test_gelu_to_its_ends():
    """Value and slope in fp32 relative to themselves.  Of Phi(-|z|), in U32: the fit 1, t 4
    (argument and reciprocal) times at most 2.2, the polynomial 5, the exponential 3, three
    products: at most 21, with its complement's no more; the value adds one, and the slope's
    two terms may cancel."""
    z = torch.cat([torch.linspace(-12.9, 12.9, 258001), torch.tensor([0.0, -0.0, 1e-30, -1e-30])]).float()[None]
    dz, dm = (torch.empty_like(z, device="cuda") for _ in range(2))
    L.z1_linear_dz(torch.ones_like(z, device="cuda"), dz, act="gelu", pre=z.cuda(), dmul=dm)
    zd = z.double()
    phi, bell = 0.5 * torch.erfc(-zd / 2 ** 0.5), torch.exp(-zd * zd / 2) / (2 * torch.pi) ** 0.5
    near(dm, zd * phi, 22 * U32 * (zd * phi).abs() + 2.0 ** -126, "value")
    near(dz, phi + zd * bell, 22 * U32 * (phi + (zd * bell).abs()) + 2.0 ** -126, "slope")
