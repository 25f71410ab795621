"""z1_qk_norm_rope and its gradient against their definitions in 64 bits.

Tolerances.  The norm's mean sums dim squares: (dim + 4) 2^-24 relative, half of it
in the root; weight, norm and element are three more roundings.  An angle reduced
in binary64 to a part of a turn is rounded once to fp32 (2^-25 of a turn, times
2 pi) and its sine and cosine are a few units off: 2^-21 in all; a rotated element
then is off by that and two roundings of |a| + |b|.  Altogether (dim + 24) 2^-24 +
2^-20 of |a| + |b|, and half a step of the type.  The gradient's mean over a head
is one more sum of dim terms; a weight's gradient sums tokens * heads terms."""
import math

import pytest
import torch

from layer_refs import TYPES, U32, half_step, near, tiny
from mixed_precision_zero_amd import layers as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def turned(x, angle, n_freq, interleaved, back=False):
    """The rotation (64 bits) and, for every element, |a| + |b| of its pair."""
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None] * (-1 if back else 1)
    first = slice(0, 2 * n_freq, 2) if interleaved else slice(0, n_freq)
    second = slice(1, 2 * n_freq, 2) if interleaved else slice(n_freq, 2 * n_freq)
    y, size = x.clone(), x.abs().clone()
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    size[..., first] = size[..., second] = a.abs() + b.abs()
    return y, size


def reference(x, w, dout, angle, n_freq, inter, eps):
    """(out, its size, dx, its size, dw, its size) of one kind of heads."""
    d = x.shape[-1]
    x, g0 = x.double(), dout.double()
    inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) if w is not None else torch.ones_like(x[..., :1])
    xh = x * inv
    out, size = turned(xh * w.double() if w is not None else x, angle, n_freq, inter)
    g, gsize = turned(g0, angle, n_freq, inter, back=True)
    if w is None:
        return out, size, g, gsize, None, None
    dw, dwsize = (g * xh).sum((0, 1)), (gsize * xh.abs()).sum((0, 1))
    gw, gwsize = g * w.double(), gsize * w.double().abs()
    dx = inv * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    dxsize = inv * (gwsize + xh.abs() * (gwsize * xh.abs()).mean(-1, keepdim=True))
    assert d == x.shape[-1]
    return out, size, dx, dxsize, dw, dwsize


def heads_in(kind, n, h, c, d, g, layout):
    """q and k on the GPU: of one projection, padded, or head by head, and the
    buffer they lie in (NaN elsewhere)."""
    t = TYPES[kind]
    if layout == "fused":
        buf = torch.full((n, (h + 2 * c) * d), float("nan"), dtype=t, device="cuda")
        q, k = (x.unflatten(1, (-1, d)) for x in buf.split([h * d, c * d, c * d], 1)[:2])
    elif layout == "odd":
        buf = torch.full((n * (h + c + 1) * (d + 3) + 7,), float("nan"), dtype=t, device="cuda")
        both = buf[1:1 + n * (h + c + 1) * (d + 3)].view(n, h + c + 1, d + 3)[..., :d]
        q, k = both[:, :h], both[:, h:h + c]
    else:       # heads outside, tokens inside
        buf = torch.full((h + c, n, d), float("nan"), dtype=t, device="cuda")
        q, k = buf[:h].transpose(0, 1), buf[h:].transpose(0, 1)
    for x in (q, k):
        x.copy_(torch.randn(x.shape, generator=g).to(t))
    return q, k, buf


def check(kind, n, h, c, d, n_freq, inter=False, norm=True, layout="fused", itype=torch.int64, eps=1e-6, seed=0):
    t = TYPES[kind]
    g = torch.Generator().manual_seed(seed + n + d)
    q, k, _ = heads_in(kind, n, h, c, d, g, layout)
    dqo, dko, _ = heads_in(kind, n, h, c, d, g, layout)
    pos = torch.randint(-5, 200000, (n,), generator=g)
    freq = torch.exp(-torch.arange(n_freq, dtype=torch.float64) * (9.0 / max(n_freq, 1)))
    angle = pos.double()[:, None] * freq
    ws = [1 + 0.2 * torch.randn(d, generator=g) if norm else None for _ in range(2)]
    ws = [w.to(t) if w is not None else None for w in ws]
    gw = [w.cuda() if w is not None else None for w in ws]
    qo, ko, buf = heads_in(kind, n, h, c, d, g, layout)
    same = dict(q_weight=gw[0], k_weight=gw[1], eps=eps, interleaved=inter)
    gp, gf = pos.to(itype).cuda(), freq.cuda()
    holes = torch.isnan(buf).clone()
    L.z1_qk_norm_rope(q, k, qo, ko, gp, gf, **same)
    dq, dk, dbuf = heads_in(kind, n, h, c, d, g, layout)
    dw = [torch.full((d,), 0.25, device="cuda") for _ in range(2)] if norm else [None, None]
    work = torch.empty(L.z1_qk_norm_rope_grad_workspace(n, h, c, d), dtype=torch.uint8, device="cuda")
    L.z1_qk_norm_rope_grad(q, k, dqo, dko, dq, dk, gp, gf, dq_weight=dw[0], dk_weight=dw[1], accumulate=True, workspace=work, **same)
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(buf), holes) and torch.equal(torch.isnan(dbuf), holes)
    rel = (d + 24) * U32 + 2.0 ** -20
    for x, w, do, out, dx, dwg, name in ((q, ws[0], dqo, qo, dq, dw[0], "q"), (k, ws[1], dko, ko, dk, dw[1], "k")):
        o, so, wx, sx, ww, sw = reference(x.cpu(), w, do.cpu(), angle, n_freq, inter, eps)
        near(out, o, rel * so + half_step(t) * o.abs() * (1 + 2.0 ** -8) + tiny(t), name + "_out")
        near(dx, wx, 2 * rel * sx + half_step(t) * wx.abs() * (1 + 2.0 ** -8) + tiny(t), "d" + name)
        if norm:
            near(dwg, ww + 0.25, (rel + (n * x.shape[1] + 8) * U32) * (sw + 0.25), f"d{name}_weight")
    # over the inputs: the bits of the same layout written elsewhere (another
    # layout's sums may be of another order)
    a, b = q.clone(), k.clone()
    ea, eb = torch.empty_like(a), torch.empty_like(b)
    L.z1_qk_norm_rope(a, b, ea, eb, gp, gf, **same)
    a0, b0 = a.clone(), b.clone()
    L.z1_qk_norm_rope(a, b, a, b, gp, gf, **same)
    assert torch.equal(a, ea) and torch.equal(b, eb)
    c0, d0 = dqo.clone(), dko.clone()
    ec, ed = torch.empty_like(c0), torch.empty_like(d0)
    sums = [[w.clone() if w is not None else None for w in dw] for _ in range(2)]
    L.z1_qk_norm_rope_grad(a0, b0, c0, d0, ec, ed, gp, gf, dq_weight=sums[0][0], dk_weight=sums[0][1], workspace=work, **same)
    L.z1_qk_norm_rope_grad(a0, b0, c0, d0, c0, d0, gp, gf, dq_weight=sums[1][0], dk_weight=sums[1][1], workspace=work, **same)
    assert torch.equal(c0, ec) and torch.equal(d0, ed)
    if norm:
        for x, y, z, heads in zip(*sums, dw, (h, c)):
            assert torch.equal(x, y)
            # written instead of added to: the same sum but for its order
            near(x, z.double().cpu() - 0.25, (n * heads + 16) * U32 * float(y.abs().max() + 0.25) * 8, "written")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("n,h,c,d,n_freq", [(1, 1, 1, 64, 32), (1, 32, 8, 128, 64), (5, 9, 3, 64, 16), (77, 4, 1, 128, 64),
                                            (300, 3, 3, 80, 40), (33, 2, 2, 96, 24), (9, 7, 2, 256, 128), (4, 2, 1, 512, 256),
                                            (12, 5, 5, 32, 0), (3, 65, 2, 16, 8)])
@pytest.mark.parametrize("inter", [False, True])
def test_heads(kind, n, h, c, d, n_freq, inter):
    check(kind, n, h, c, d, n_freq, inter=inter)
    check(kind, n, h, c, d, n_freq, inter=inter, norm=False)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("d,n_freq", [(1, 0), (2, 1), (3, 1), (10, 5), (33, 7), (65, 32), (100, 50), (127, 63), (511, 255), (512, 250), (510, 255)])
@pytest.mark.parametrize("inter", [False, True])
def test_odd_heads(kind, d, n_freq, inter):
    check(kind, 7, 3, 2, d, n_freq, inter=inter, layout="odd", itype=torch.int32)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("layout", ["odd", "outside"])
def test_layouts(kind, layout):
    check(kind, 50, 6, 2, 64, 32, layout=layout)
    check(kind, 50, 6, 2, 64, 20, layout=layout, inter=True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_many_tokens(kind):
    check(kind, 5000, 3, 2, 32, 16)


def test_far_positions():
    """Angles of positions near 2^40 in fp32: binary64 has 2^-52 of 2^40 rad, 2^-12
    of one, so frequencies that are powers of two are used, whose angles are exact;
    the reduction by a rounded 1 / (2 pi) then is off by 2^-53 of the turns."""
    n = 16
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 31 + 7, -(2 ** 33) - 3] + [2 ** 24 + i for i in range(10)])
    freq = torch.tensor([1.0, 2.0 ** -3, 2.0 ** -10, 2.0 ** -20], dtype=torch.float64)
    x = torch.randn(n, 1, 8)
    out = torch.empty(n, 1, 8, device="cuda")
    L.z1_qk_norm_rope(x.cuda(), None, out, None, pos.cuda(), freq.cuda())
    want, size = turned(x.double(), pos.double()[:, None] * freq, 4, False)
    turns = (pos.double().abs()[:, None] * freq).max() / (2 * math.pi)
    near(out, want, (2.0 ** -20 + 4 * math.pi * float(turns) * 2.0 ** -52) * size, "far")


def test_norm_and_rotation_keep_the_length():
    """Without weights other than one, every head has mean square 1 (eps 0)."""
    x = torch.randn(40, 5, 128, device="cuda")
    one, freq = torch.ones(128, device="cuda"), torch.rand(64, dtype=torch.float64, device="cuda")
    out = torch.empty_like(x)
    L.z1_qk_norm_rope(x, None, out, None, torch.arange(40, device="cuda"), freq, q_weight=one, eps=0.0)
    near(out.double().square().mean(2), torch.ones(40, 5, dtype=torch.float64), 2.0 ** -18, "mean square")


def test_heads_that_are_zero_or_not_finite():
    """A zero head stays zero with eps > 0; NaN and infinities stay in their head."""
    x = torch.randn(6, 4, 64, device="cuda")
    x[1, 1], x[2, 2, 5], x[3, 3, 7] = 0.0, float("nan"), float("inf")
    w, freq, pos = torch.ones(64, device="cuda"), torch.rand(32, dtype=torch.float64, device="cuda"), torch.arange(6, device="cuda")
    out, clean = torch.empty_like(x), torch.empty_like(x)
    L.z1_qk_norm_rope(x, None, out, None, pos, freq, q_weight=w)
    assert bool((out[1, 1] == 0).all())
    bad = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    bad[2, 2] = bad[3, 3] = True
    assert bool(torch.isfinite(out[~bad]).all()) and not bool(torch.isfinite(out[bad]).all(1).any())
    L.z1_qk_norm_rope(torch.where(bad[..., None], torch.zeros_like(x), x), None, clean, None, pos, freq, q_weight=w)
    assert torch.equal(out[~bad], clean[~bad])
    # a zero head has the gradient g w / sqrt(eps)
    g, dx, dw = torch.randn_like(x), torch.empty_like(x), torch.empty(64, device="cuda")
    zero = torch.zeros_like(x)
    ws = torch.empty(L.z1_qk_norm_rope_grad_workspace(6, 4, 0, 64), dtype=torch.uint8, device="cuda")
    L.z1_qk_norm_rope_grad(zero, None, g, None, dx, None, pos, freq, q_weight=w, dq_weight=dw, eps=1e-4, workspace=ws)
    back, size = turned(g.double().cpu(), pos.cpu().double()[:, None] * freq.cpu(), 32, False, back=True)
    near(dx, 100 * back, 100 * 2.0 ** -19 * size, "zero head")
    assert bool((dw == 0).all())


def test_one_kind_alone_no_tokens_no_heads():
    t = torch.bfloat16
    q, k = torch.randn(9, 4, 64, device="cuda", dtype=t), torch.randn(9, 2, 64, device="cuda", dtype=t)
    pos, freq = torch.arange(9, device="cuda"), torch.rand(32, dtype=torch.float64, device="cuda")
    w = torch.rand(64, device="cuda").to(t)
    qo, ko, alone = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
    L.z1_qk_norm_rope(q, k, qo, ko, pos, freq, q_weight=w)          # keys without a norm
    L.z1_qk_norm_rope(None, k, None, alone, pos, freq)
    assert torch.equal(ko, alone)
    L.z1_qk_norm_rope(q[:, :0], k, qo[:, :0], alone.zero_(), pos, freq)
    assert torch.equal(ko, alone)
    empty = torch.empty(0, 4, 64, device="cuda", dtype=t)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    L.z1_qk_norm_rope(empty, None, empty, None, none, freq)
    dw = torch.full((64,), 2.0, device="cuda")
    ws = torch.empty(L.z1_qk_norm_rope_grad_workspace(0, 4, 0, 64), dtype=torch.uint8, device="cuda")
    for acc, left in ((True, 2.0), (False, 0.0)):
        L.z1_qk_norm_rope_grad(empty, None, empty, None, empty, None, none, freq, q_weight=w, dq_weight=dw, accumulate=acc, workspace=ws)
        assert bool((dw == left).all())


def test_gradient_against_differences():
    """Centred differences in fp32 with a step of 2^-6, as for the linear layer:
    2e-3 of the sum of magnitudes."""
    g = torch.Generator().manual_seed(2)
    n, h, c, d, f = 6, 3, 2, 40, 12
    q, k = torch.randn(n, h, d, generator=g).cuda(), torch.randn(n, c, d, generator=g).cuda()
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g).cuda() for _ in range(2))
    dqo, dko = torch.randn(n, h, d, generator=g).cuda(), torch.randn(n, c, d, generator=g).cuda()
    pos, freq = torch.randint(0, 1000, (n,), generator=g).cuda(), torch.rand(f, dtype=torch.float64, generator=g).cuda()

    def loss(q, k, wq, wk):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        L.z1_qk_norm_rope(q, k, qo, ko, pos, freq, q_weight=wq, k_weight=wk, interleaved=True)
        return float((qo.double() * dqo.double()).sum() + (ko.double() * dko.double()).sum())

    dq, dk, dwq, dwk = (torch.empty_like(x) for x in (q, k, wq, wk))
    ws = torch.empty(L.z1_qk_norm_rope_grad_workspace(n, h, c, d), dtype=torch.uint8, device="cuda")
    L.z1_qk_norm_rope_grad(q, k, dqo, dko, dq, dk, pos, freq, q_weight=wq, k_weight=wk, dq_weight=dwq, dk_weight=dwk,
                           interleaved=True, workspace=ws)
    step = 2.0 ** -6
    for i, grad in enumerate((dq, dk, dwq, dwk)):
        args = [[q, k, wq, wk], [q, k, wq, wk]]
        v = torch.randn(grad.shape, generator=g).cuda()
        args[0][i], args[1][i] = args[0][i] + step * v, args[1][i] - step * v
        diff = (loss(*args[0]) - loss(*args[1])) / (2 * step)
        got, size = float((grad.double() * v.double()).sum()), float((grad.double() * v.double()).abs().sum())
        assert abs(got - diff) <= 2e-3 * size, (i, got, diff)


def test_same_bits_every_time_streams_and_a_graph():
    g = torch.Generator().manual_seed(9)
    n, h, c, d = 700, 6, 2, 64
    q, k, _ = heads_in("bf16", n, h, c, d, g, "fused")
    dqo, dko, _ = heads_in("bf16", n, h, c, d, g, "fused")
    pos, freq = torch.arange(n, device="cuda"), torch.rand(32, dtype=torch.float64, device="cuda")
    w = torch.rand(d, device="cuda").bfloat16()
    need = L.z1_qk_norm_rope_grad_workspace(n, h, c, d)

    def run(stream=None):
        o = [torch.empty_like(x) for x in (q, k, q, k)] + [torch.empty(d, device="cuda") for _ in range(2)]
        o.append(torch.empty(need, dtype=torch.uint8, device="cuda"))
        call(o, stream)
        return o

    def call(o, stream=None):
        L.z1_qk_norm_rope(q, k, o[0], o[1], pos, freq, q_weight=w, k_weight=w, stream=stream)
        L.z1_qk_norm_rope_grad(q, k, dqo, dko, o[2], o[3], pos, freq, q_weight=w, k_weight=w, dq_weight=o[4], dk_weight=o[5],
                               workspace=o[6], stream=stream)

    first = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    others = [run(), run(s)]
    torch.cuda.synchronize()
    held = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        call(held)
    for i in range(3):
        for t in held[:6]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        others.append([t.clone() for t in held])
    for o in others:
        assert all(torch.equal(a, b) for a, b in zip(o[:6], first[:6]))
