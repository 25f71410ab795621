"""The loss operators against their definitions in binary64.

Log-probabilities are sums of fp32 values no larger than the row's spread R =
max - min plus log V: exponentials are taken from an argument rounded at R
log2(e) 2^-24 and added in runs of at most 512 in a lane and 10 joins, so lse
is off by at most (R + 530 + 3) 2^-24 in the worst case, and logp by two more
roundings at its own size: LOGP below bounds all of it for the ranges used here.
The gradient d (1 - p) is then off by 2 LOGP d p, and by one rounding to its
type (half of eps, or half of the smallest subnormal)."""
import math

import pytest
import torch

from mixed_precision_zero_amd import ops as O

pytestmark = pytest.mark.gpu
DT = [torch.float32, torch.bfloat16, torch.float16]
LOGP = 700 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rows(n, V, dtype, seed=0, pad=0, shift=0, itype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(n, V + pad, generator=g, device="cuda") * 3).to(dtype)
    if shift:
        flat = torch.empty(x.numel() + 16, device="cuda", dtype=dtype)[shift:shift + x.numel()]
        x = flat.view(x.shape).copy_(x)
    x = x[:, :V]
    y = torch.randint(0, V, (n,), generator=g, device="cuda")
    if n > 3:
        y[torch.rand(n, generator=g, device="cuda") < 0.2] = -100
    return x, y.to(itype), g


def exact(x, y):
    z = x.double()
    lse = z.logsumexp(1)
    logp = z.gather(1, y.long().clamp(0, x.shape[1] - 1)[:, None])[:, 0] - lse
    here = y >= 0
    return torch.where(here, logp, 0.0), torch.where(here, lse, 0.0), here


def exact_grad(x, y, lse, d):
    here = y >= 0
    d = torch.where(here, d.double(), 0.0)
    g = -d[:, None] * torch.exp(x.double() - lse.double()[:, None])
    g.scatter_add_(1, y.long().clamp(min=0)[:, None], d[:, None])
    return torch.where(here[:, None], g, 0.0), d


def check_grad(got, want, d, p_bound=2 * LOGP):
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny * torch.finfo(got.dtype).eps
    bound = p_bound * d.abs()[:, None] + half * want.abs() + tiny + 2.0 ** -126
    bad = (got.double() - want).abs() > bound
    assert not bad.any(), float(((got.double() - want).abs() - bound).max())


SIZES = [(1, 1), (3, 2), (5, 7), (4, 8), (5, 9), (9, 64), (7, 1000), (3, 2047), (6, 2049), (2, 8200), (5, 32001),
         (3, 49152), (2, 70000), (2, 100001), (1100, 1100), (1500, 9)]


@pytest.mark.parametrize("dtype", DT, ids=str)
@pytest.mark.parametrize("n,V", SIZES)
def test_logprob_and_its_gradient(n, V, dtype):
    for pad, shift in ((0, 0), (3, 0), (8, 1)):
        x, y, g = rows(n, V, dtype, V, pad, shift)
        logp, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
        O.z1_token_logprob(x, y, logp, lse)
        wp, wl, here = exact(x, y)
        assert ((logp.double() - wp).abs() <= LOGP).all() and ((lse.double() - wl).abs() <= LOGP).all()
        d = torch.randn(n, generator=g, device="cuda")
        out = torch.full((n, V + 5), 9.0, device="cuda", dtype=dtype)
        O.z1_logprob_grad(x, y, lse, d, out[:, :V])
        want, dd = exact_grad(x, y, wl, d)
        check_grad(out[:, :V], want, dd)
        assert (out[:, V:] == 9).all()
        ref = out[:, :V].clone()
        O.z1_logprob_grad(x, y, lse, d, x)      # in place
        assert torch.equal(x, ref)


def policy_exact(x, y, old, adv, ref, w, lo, hi, kl, scale):
    logp, lse, here = exact(x, y)
    here = here & (w != 0)
    rho = torch.exp(logp - old.double())
    A = adv.double()
    near = rho.clamp(1 - lo, 1 + hi)
    low = torch.minimum(rho * A, near * A)
    gap = ref.double() - logp
    token = torch.where(here, -low + kl * (torch.expm1(gap) - gap), 0.0)
    moves = (rho == near) | (rho * A < near * A)
    d = torch.where(moves, -rho * A, 0.0) - kl * torch.expm1(gap)
    d = torch.where(here, d * w.double() * scale, 0.0)
    return logp, lse, token, (torch.where(here, w.double(), 0.0) * token).sum() * scale, d, here, rho


@pytest.mark.parametrize("dtype", DT, ids=str)
@pytest.mark.parametrize("n,V", SIZES)
def test_policy(n, V, dtype):
    lo, hi, kl, scale = 0.2, 0.3, 0.05, 1.0 / n
    for pad, shift, weighted, grad in ((0, 0, False, True), (3, 1, True, True), (0, 0, True, False)):
        x, y, g = rows(n, V, dtype, V + 1, pad, shift, torch.int32 if weighted else torch.int64)
        now = exact(x, y)[0].float()
        old, ref = (now + 0.3 * torch.randn(n, generator=g, device="cuda") for _ in range(2))
        adv = torch.randn(n, generator=g, device="cuda")
        w = torch.rand(n, generator=g, device="cuda").round(decimals=1) if weighted else torch.ones(n, device="cuda")
        loss, token, logp = torch.empty(1, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        out = torch.empty(n, V, device="cuda", dtype=dtype) if grad else None
        O.z1_policy_loss(x, y, old, adv, loss=loss, token_loss=token, logp=logp, dlogits=out, ref_logp=ref,
                         weights=w if weighted else None, clip_low=lo, clip_high=hi, kl_coef=kl, scale=scale)
        wp, wl, wt, wloss, d, here, rho = policy_exact(x, y, old, adv, ref, w, lo, hi, kl, scale)
        # a ratio within LOGP of a clamp's end may fall on either side of it
        sure = ((rho - (1 - lo)).abs() > 4 * LOGP) & ((rho - (1 + hi)).abs() > 4 * LOGP)
        size = 4 * LOGP * (rho * adv.abs() + kl * (torch.exp(ref - wp) + 2) + 1)
        assert ((logp.double() - torch.where(here, wp, 0.0)).abs() <= LOGP).all()
        assert ((token.double() - wt).abs() <= size).all()
        assert abs(float(loss) - float(wloss)) <= float((size * w).sum()) * scale + 2.0 ** -24 * abs(float(wloss))
        if grad:
            want, _ = exact_grad(x, torch.where(here, y, torch.full_like(y, -1)), wl, d)
            slope = (size * w * scale)[:, None] + 2 * LOGP * d.abs()[:, None]
            half, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).tiny * torch.finfo(dtype).eps
            bad = ((out.double() - want).abs() > slope + half * want.abs() + tiny + 2.0 ** -126) & sure[:, None]
            assert not bad.any()
            assert (out[~here] == 0).all()
            again = torch.empty_like(loss), torch.empty_like(token)
            O.z1_policy_loss(x, y, old, adv, loss=again[0], token_loss=again[1], dlogits=x, ref_logp=ref,
                             weights=w if weighted else None, clip_low=lo, clip_high=hi, kl_coef=kl, scale=scale)
            assert torch.equal(x, out) and torch.equal(again[0], loss) and torch.equal(again[1], token)


def test_policy_without_kl_and_clamp_ends():
    """No reference, infinite-looking clamps: the loss is -rho A."""
    x, y, g = rows(40, 500, torch.float32)
    old = exact(x, y)[0].float() + 0.5
    adv = torch.randn(40, generator=g, device="cuda")
    loss, token = torch.empty(1, device="cuda"), torch.empty(40, device="cuda")
    O.z1_policy_loss(x, y, old, adv, loss=loss, token_loss=token, clip_low=1.0, clip_high=1e6, scale=1.0)
    logp, _, here = exact(x, y)
    want = torch.where(here, -torch.exp(logp - old.double()) * adv.double(), 0.0)
    assert ((token.double() - want).abs() <= 4 * LOGP * (1 + want.abs())).all()


def test_policy_gradient_against_differences():
    """Central differences of the loss over single logits; the loss is an fp32
    number near 1 (2^-24), the step 2^-5 adds a third-order term below
    step^2 / 6 * 2."""
    x, y, g = rows(6, 20, torch.float32, 11)
    y.clamp_(min=0)
    old = exact(x, y)[0].float() + 0.05
    ref = old + 0.1
    adv = torch.tensor([1.0, -1.0, 0.5, 2.0, -0.3, 0.0], device="cuda")
    loss, token, out = torch.empty(1, device="cuda"), torch.empty(6, device="cuda"), torch.empty_like(x)
    args = dict(ref_logp=ref, clip_low=0.5, clip_high=0.5, kl_coef=0.2, scale=1.0, token_loss=token)
    O.z1_policy_loss(x, y, old, adv, loss=loss, dlogits=out, **args)
    h = 2.0 ** -5
    for r in range(6):
        for v in (int(y[r]), (int(y[r]) + 3) % 20):
            f = []
            for s in (h, -h):
                z = x.clone()
                z[r, v] += s
                O.z1_policy_loss(z, y, old, adv, loss=loss, **args)
                f.append(float(loss))
            assert abs((f[0] - f[1]) / (2 * h) - float(out[r, v])) <= 2 * h * h / 6 + 8 * 2.0 ** -24 / h


@pytest.mark.parametrize("dtype", DT, ids=str)
@pytest.mark.parametrize("V", [37, 5000, 20000])
def test_masked_and_infinite_entries(dtype, V):
    x, y, g = rows(8, V, dtype)
    y[:] = torch.tensor([0, 1, -1, 3, V, 5, -100, 7], device="cuda")
    x[2] = float("nan")              # masked rows are not read
    x[6] = float("-inf")
    x[0, V // 2:] = float("-inf")    # masked vocabulary
    x[1] = float("-inf")             # one entry left
    x[1, 1] = 0.5
    x[3] = torch.finfo(dtype).min    # the type's lowest value everywhere
    x[5] = float("-inf")             # nothing left
    x[7, 7] = float("-inf")          # the target itself masked
    n = 8
    one = torch.ones(n, device="cuda")
    logp, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    O.z1_token_logprob(x, y, logp, lse)
    want = exact(x, y)[0]
    assert abs(float(logp[0] - want[0])) <= LOGP and float(logp[1]) == 0.0 and float(lse[1]) == 0.5
    assert float(logp[2]) == 0.0 and float(logp[6]) == 0.0 and float(lse[2]) == 0.0
    assert abs(float(logp[3]) + math.log(V)) <= LOGP
    assert math.isnan(float(logp[4])) and math.isnan(float(logp[5])) and float(logp[7]) == -math.inf
    out = torch.empty(n, V, device="cuda", dtype=dtype)
    loss, token = torch.empty(1, device="cuda"), torch.empty(n, device="cuda")
    for w in (None, torch.tensor([1., 1., 1., 1., 0., 0., 1., 1.], device="cuda")):
        O.z1_policy_loss(x, y, one * 0, one, loss=loss, token_loss=token, dlogits=out, weights=w)
        assert (out[2] == 0).all() and (out[6] == 0).all() and float(token[2]) == 0.0
        assert (out[0, V // 2:] == 0).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[7]).all()
        if w is None:
            assert torch.isnan(out[4]).all() and torch.isnan(token[4]) and torch.isnan(loss[0])
        else:
            assert (out[4:6] == 0).all() and torch.isfinite(loss[0])
    O.z1_logprob_grad(x, y, lse, one, out)
    assert (out[2] == 0).all() and (out[6] == 0).all() and torch.isnan(out[4]).all()
    assert abs(float(out[1, 1])) <= 2 * LOGP and (out[1, 2:] == 0).all()


def preference_exact(logp, ref, y, cu, beta, e, scale):
    diff = torch.where(y >= 0, logp.double() - torch.where(y >= 0, ref, torch.zeros_like(ref)).double(), 0.0)
    d = torch.zeros_like(diff)
    loss, pair, margin = 0.0, [], []
    for p in range((len(cu) - 1) // 2):
        a, b, c = cu[2 * p], cu[2 * p + 1], cu[2 * p + 2]
        z = beta * (diff[a:b].sum() - diff[b:c].sum())
        f = torch.nn.functional.softplus
        l = (1 - e) * f(-z, threshold=1e9) + e * f(z, threshold=1e9)
        s = scale * beta * (e * torch.sigmoid(z) - (1 - e) * torch.sigmoid(-z))
        d[a:b], d[b:c] = s, -s
        pair.append(float(l))
        margin.append(float(z))
    return sum(pair) * scale, pair, margin, torch.where(y >= 0, d, 0.0)


@pytest.mark.parametrize("itype", [torch.int64, torch.int32])
@pytest.mark.parametrize("cu,e", [([0, 1, 2], 0.0), ([0, 5, 9, 30, 300], 0.1), ([3, 3, 7, 7, 7, 40, 900], 0.0),
                                  ([0, 600, 1000], 0.5), ([2], 0.0)])
def test_preference(cu, e, itype):
    n = cu[-1] + 11
    g = torch.Generator(device="cuda").manual_seed(n)
    logp, ref = (-3 + torch.randn(n, generator=g, device="cuda") for _ in range(2))
    y = torch.randint(-3, 50, (n,), generator=g, device="cuda")
    ref[y < 0] = float("nan")
    P = (len(cu) - 1) // 2
    out = [torch.full((k,), float("nan"), device="cuda") for k in (1, P, P, n)]
    O.z1_preference_loss(logp, ref, y.to(itype), torch.tensor(cu, device="cuda", dtype=itype), beta=0.3, scale=0.7,
                         label_smoothing=e, loss=out[0], pair_loss=out[1], margins=out[2], dlogp=out[3])
    loss, pair, margin, d = preference_exact(logp, ref, y, cu, 0.3, e, 0.7)
    half = 2.0 ** -24 * 2      # binary64 sums, one rounding to fp32
    assert abs(float(out[0]) - loss) <= half * (abs(loss) + P)
    for a, b in ((out[1], pair), (out[2], margin)):
        b = torch.tensor(b, device="cuda", dtype=torch.float64)
        assert ((a.double() - b).abs() <= half * b.abs() + 1e-12).all()
    assert ((out[3].double() - d).abs() <= half * d.abs() + 1e-14).all()


def test_preference_far_margins_and_differences():
    cu = torch.tensor([0, 1, 2, 3, 4, 5, 6], device="cuda")
    y = torch.zeros(6, dtype=torch.long, device="cuda")
    logp = torch.tensor([400.0, -400.0, -400.0, 400.0, 0.1, 0.2], device="cuda")
    zero = torch.zeros(6, device="cuda")
    loss, pair, d = torch.empty(1, device="cuda"), torch.empty(3, device="cuda"), torch.empty(6, device="cuda")
    args = dict(beta=1.0, loss=loss, pair_loss=pair, dlogp=d)
    O.z1_preference_loss(logp, zero, y, cu, **args)
    assert float(pair[0]) == 0.0 and float(pair[1]) == 800.0 and torch.isfinite(d).all()
    assert d[:4].tolist() == [0.0, 0.0, -1.0, 1.0]
    slope, h = d.clone(), 2.0 ** -6
    for i in (4, 5):
        f = []
        for s in (h, -h):
            z = logp.clone()
            z[i] += s
            O.z1_preference_loss(z, zero, y, cu, **args)
            f.append(float(pair[2]))
        assert abs((f[0] - f[1]) / (2 * h) - float(slope[i])) <= h * h / 6 + 2.0 ** -23 / h


def test_no_rows():
    x = torch.zeros(0, 10, device="cuda")
    y = torch.zeros(0, dtype=torch.long, device="cuda")
    v = torch.zeros(0, device="cuda")
    loss = torch.full((1,), 5.0, device="cuda")
    O.z1_policy_loss(x, y, v, v, loss=loss, token_loss=v, dlogits=x)
    assert float(loss) == 0.0
    O.z1_token_logprob(x, y, v, v)
    O.z1_logprob_grad(x, y, v, v, x)


def test_offsets_past_32_bits():
    """Rows beyond the 2^31st element of the logits, in place."""
    n, V = 45000, 49152
    x = torch.zeros(n, V, device="cuda", dtype=torch.bfloat16)
    y = torch.full((n,), -1, dtype=torch.long, device="cuda")
    y[n - 1], y[0] = 3, 4
    x[n - 1, 3] = 5.0
    logp = torch.empty(n, device="cuda")
    O.z1_token_logprob(x, y, logp)
    want = 5.0 - math.log(math.exp(5.0) + V - 1)
    assert abs(float(logp[n - 1]) - want) <= LOGP and abs(float(logp[0]) + math.log(V)) <= LOGP
    loss, token = torch.empty(1, device="cuda"), torch.empty(n, device="cuda")
    O.z1_policy_loss(x, y, logp, torch.ones(n, device="cuda"), loss=loss, token_loss=token, dlogits=x)
    assert abs(float(x[n - 1, 3]) + (1 - math.exp(want))) <= 2.0 ** -8 and float(token[n - 1]) == -1.0
    assert float(x[n - 2].abs().max()) == 0.0


def test_other_stream_and_graph():
    x, y, g = rows(64, 3000, torch.bfloat16)
    logp, lse = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    old = exact(x, y)[0].float() + 0.1
    adv = torch.randn(64, generator=g, device="cuda")
    loss, token, out = torch.empty(1, device="cuda"), torch.empty(64, device="cuda"), torch.empty_like(x)
    cu = torch.tensor([0, 20, 40, 50, 64], device="cuda")
    pair, d, ploss, pd = (torch.empty(2, device="cuda"), torch.empty(64, device="cuda"), torch.empty(1, device="cuda"),
                          torch.empty_like(x))

    def call(stream=None):
        O.z1_policy_loss(x, y, old, adv, loss=loss, token_loss=token, dlogits=out, ref_logp=old, kl_coef=0.1, stream=stream)
        O.z1_token_logprob(x, y, logp, lse, stream=stream)
        O.z1_preference_loss(logp, old, y, cu, beta=0.2, loss=ploss, pair_loss=pair, dlogp=d, stream=stream)
        O.z1_logprob_grad(x, y, lse, d, pd, stream=stream)

    call()
    torch.cuda.synchronize()
    held = (loss, token, out, logp, lse, ploss, pair, d, pd)
    ref = [t.clone() for t in held]

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for a, b in zip(held, ref))

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in held:
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(4):
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        assert same(), k
        call()
        assert same(), k


@pytest.mark.parametrize("itype", [torch.int64, torch.int32])
@pytest.mark.parametrize("weight", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("n", [8, 1500])
def test_weights_of_rows_that_do_not_count(n, weight, itype):
    """Negative targets with an infinite or NaN weight (mask / mask.sum() of an
    answer that is masked throughout): the loss is that of the other rows."""
    x, y, g = rows(n, 50, torch.float32, 5)
    y[::3] = -1
    old = exact(x, y)[0].float() + 0.1
    adv = torch.randn(n, generator=g, device="cuda")
    w = torch.rand(n, generator=g, device="cuda")
    got = []
    for bad in (0.0, weight):
        w[::3] = bad
        loss, token = torch.empty(1, device="cuda"), torch.empty(n, device="cuda")
        out = torch.empty_like(x)
        O.z1_policy_loss(x, y.to(itype), old, adv, loss=loss, token_loss=token, dlogits=out, weights=w, scale=0.5)
        got.append((loss, token, out))
    assert torch.isfinite(got[0][0]).all()
    assert all(torch.equal(a, b) for a, b in zip(*got))


def shifted(n, V, dtype, shift):
    """Logits around `shift` with the spread that `rows` has, or (None) the
    type's lowest value throughout."""
    x, y, g = rows(n, V, torch.float32, V + 7)
    y.clamp_(min=0)
    x = torch.full_like(x, torch.finfo(dtype).min) if shift is None else x + shift
    return x.to(dtype), y, g


SHIFTS = [1e3, -1e3, 1e4, -1e4, 1e6, None]


@pytest.mark.parametrize("dtype,shift", [(d, s) for d in DT for s in SHIFTS if not (d == torch.float16 and s == 1e6)], ids=str)
@pytest.mark.parametrize("n,V", [(6, 100), (5, 2049), (3, 32001), (2, 100001)])
def test_policy_gradient_far_from_zero(n, V, dtype, shift):
    """A constant added to a row changes no probability: the bounds are those
    of rows around zero, whose spread alone counts."""
    x, y, g = shifted(n, V, dtype, shift)
    z = x.double() - x.double().amax(1, keepdim=True)
    wp, wl, _ = exact(z, y)
    old = wp.float()
    adv = torch.randn(n, generator=g, device="cuda")
    loss, token, logp, out = (torch.empty(1, device="cuda"), torch.empty(n, device="cuda"),
                              torch.empty(n, device="cuda"), torch.empty_like(x))
    O.z1_policy_loss(x, y, old, adv, loss=loss, token_loss=token, logp=logp, dlogits=out)
    assert ((logp.double() - wp).abs() <= LOGP).all()
    d = -torch.exp(logp.double() - old.double()) * adv.double()    # the ratio is 1 to a few roundings
    want, d = exact_grad(z, y, wl, d)
    check_grad(out, want, d, 3 * LOGP)
    O.z1_policy_loss(x, y, old, adv, loss=loss, token_loss=token, dlogits=x)
    assert torch.equal(x, out)


@pytest.mark.parametrize("dtype,shift", [(d, s) for d in DT for s in SHIFTS if not (d == torch.float16 and s == 1e6)], ids=str)
@pytest.mark.parametrize("n,V", [(6, 100), (5, 2049), (3, 32001), (2, 100001)])
def test_logprob_gradient_far_from_zero(n, V, dtype, shift):
    """As for the policy gradient, through the fp32 lse, which alone is rounded
    at its own size."""
    x, y, g = shifted(n, V, dtype, shift)
    z = x.double() - x.double().amax(1, keepdim=True)
    wp, wl, _ = exact(z, y)
    logp, lse, out = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(x)
    O.z1_token_logprob(x, y, logp, lse)
    assert ((logp.double() - wp).abs() <= LOGP).all()
    true = x.double().amax(1) + wl
    assert ((lse.double() - true).abs() <= LOGP + true.abs() * 2.0 ** -24).all()
    d = torch.randn(n, generator=g, device="cuda")
    O.z1_logprob_grad(x, y, lse, d, out)
    want, dd = exact_grad(z, y, wl, d)
    check_grad(out, want, dd)
    O.z1_logprob_grad(x, y, lse, d, x)
    assert torch.equal(x, out)


@pytest.mark.parametrize("n,V", [(6, 100), (2, 100001)])
def test_logprob_gradient_takes_another_lse_as_it_is(n, V):
    """An lse that is not the row's own: exp(x - lse) with it, also far from
    zero, where x - lse is exact here (integers below 2^24)."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randint(990, 1000, (n, V), generator=g, device="cuda").float()
    y = torch.randint(0, V, (n,), generator=g, device="cuda")
    lse, d = torch.full((n,), 1005.0, device="cuda"), torch.randn(n, generator=g, device="cuda")
    out = torch.empty_like(x)
    O.z1_logprob_grad(x, y, lse, d, out)
    want, dd = exact_grad(x, y, lse, d)
    check_grad(out, want, dd)
    # infinite and NaN ones
    for odd, p in ((math.inf, 0.0), (math.nan, math.nan)):
        lse.fill_(odd)
        O.z1_logprob_grad(x, y, lse, torch.ones_like(d), out)
        assert torch.equal(out[0, y[0]].isnan(), torch.tensor(math.isnan(p), device="cuda"))
        assert float(out.nan_to_num(7.0).min()) == (0.0 if p == 0.0 else 7.0)


@pytest.mark.parametrize("V", [5, 5000, 100001])
def test_ids_past_the_vocabulary_have_no_lse(V):
    """NaN in all of their outputs; the rows beside them keep theirs."""
    x, y, g = rows(4, V, torch.float32, V)
    y[:] = torch.tensor([V, 0, -1, V + 9], device="cuda")
    logp, lse = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    O.z1_token_logprob(x, y, logp, lse)
    for out in (logp, lse):
        assert out.isnan().tolist() == [True, False, False, True] and float(out[2]) == 0.0
    assert abs(float(lse[1]) - float(exact(x, y.clamp(max=V - 1))[1][1])) <= LOGP


@pytest.mark.parametrize("e,z,want", [(1.0, -math.inf, 0.0), (1.0, math.inf, math.inf), (0.0, math.inf, 0.0),
                                      (0.0, -math.inf, math.inf), (0.5, math.inf, math.inf)])
def test_preference_of_infinite_margins(e, z, want):
    """A target whose logit is masked has log-probability -inf: the side of the
    loss that smoothing gives no weight does not count."""
    logp = torch.tensor([z, 0.0] if z < 0 else [0.0, -z], device="cuda")
    zero, y = torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.long, device="cuda")
    loss, pair, d = torch.empty(1, device="cuda"), torch.empty(1, device="cuda"), torch.empty(2, device="cuda")
    O.z1_preference_loss(logp, zero, y, torch.tensor([0, 1, 2], device="cuda"), beta=0.5, label_smoothing=e, loss=loss,
                         pair_loss=pair, dlogp=d)
    assert float(pair) == want and float(loss) == want
    slope = 0.5 * (e - 1.0 if z < 0 else e)
    assert d.tolist() == [slope, -slope]


def test_no_kl_coefficient_no_kl_term():
    """kl_coef 0: whatever the reference holds, exp(ref - logp) past fp32's
    range and NaN among it, the result is that without a reference."""
    x, y, g = rows(30, 200, torch.float32, 3)
    old, adv = exact(x, y)[0].float(), torch.randn(30, generator=g, device="cuda")
    ref = old + 100.0
    ref[::4] = float("nan")
    got = []
    for r in (None, ref):
        loss, token, out = torch.empty(1, device="cuda"), torch.empty(30, device="cuda"), torch.empty_like(x)
        O.z1_policy_loss(x, y, old, adv, loss=loss, token_loss=token, dlogits=out, ref_logp=r, kl_coef=0.0)
        got.append((loss, token, out))
    assert torch.isfinite(got[0][0]).all() and torch.isfinite(got[0][2]).all()
    assert all(torch.equal(a, b) for a, b in zip(*got))
