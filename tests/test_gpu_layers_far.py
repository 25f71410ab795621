"""The layers on matrices whose rows lie past 2^32 elements: the same bits as on
dense copies of them."""
import pytest
import torch

from mixed_precision_zero_amd import layers as L

pytestmark = pytest.mark.gpu
ROWS, LD = 4104, 1 << 20   # the last rows start at element 4103 * 2^20 > 2^32


@pytest.fixture(scope="module")
def columns():
    """Gives out matrices of n columns of one 8.6 GB buffer, so many elements apart."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    buf, used = torch.empty(ROWS, LD, dtype=torch.bfloat16, device="cuda"), [0]

    def take(like):
        at, n = used[0], like.shape[1]
        used[0] = at + (n + 7) // 8 * 8
        m = buf[:, at:at + n]
        m.copy_(like)
        return m
    return take


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def work(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("inner,outer", [(64, 72), (43, 51)])
def test_linear(columns, inner, outer):
    x, w, b = rand(0, ROWS, inner), rand(1, outer, inner), rand(2, outer)
    mul, res, dy = rand(3, ROWS, outer), rand(4, ROWS, outer), rand(5, ROWS, outer)
    d = L.Dropout(torch.tensor([3, 4], device="cuda"), 0.25)

    def run(place):
        f = lambda t: place(torch.full_like(t, float("nan")))  # noqa: E731
        X, M, R, D, Y, P, Z, DM, DX = place(x), place(mul), place(res), place(dy), f(res), f(res), f(res), f(res), f(x)
        L.z1_linear(X, w, Y, bias=b, act="silu", mul=M, residual=R, pre=P, dropout=d, workspace=work(L.z1_linear_workspace(X, w)))
        db, dw = torch.zeros(outer, device="cuda"), torch.zeros(outer, inner, device="cuda")
        L.z1_linear_dz(D, Z, act="silu", pre=P, mul=M, dmul=DM, dbias=db, dropout=d, workspace=work(L.z1_linear_dz_workspace(ROWS, outer)))
        L.z1_linear_grad(Z, X, w, dx=DX, add=X, dweight=dw, accumulate=True, workspace=work(L.z1_linear_grad_workspace(Z, X, w)))
        return [Y, P, Z, DM, DX, db, dw]

    for i, (far, dense) in enumerate(zip(run(columns), run(lambda t: t.clone()))):
        assert torch.equal(far, dense), i
        assert torch.isfinite(dense).all(), i


def test_dropout(columns):
    x, r = rand(6, ROWS, 77), rand(7, ROWS, 77)
    d, y, dense = L.Dropout(torch.tensor([3, 4], device="cuda"), 0.25), columns(torch.zeros_like(x)), torch.empty_like(x)
    L.z1_dropout(columns(x), y, d, residual=columns(r))
    L.z1_dropout(x, dense, d, residual=r)
    assert torch.equal(y, dense)


@pytest.mark.parametrize("dim", [32, 20])
def test_heads(columns, dim):
    q, k, dq, dk = (rand(8 + i, ROWS, h * dim) for i, h in enumerate((4, 2, 4, 2)))
    w, pos = rand(12, dim), torch.arange(ROWS, device="cuda")
    freq = 100.0 ** -torch.arange(dim // 2, dtype=torch.float64, device="cuda").div(dim // 2)

    def run(place):
        p = lambda t: place(t).unflatten(1, (-1, dim))  # noqa: E731
        Q, K, A, B, OQ, OK, DQ, DK = (p(t) for t in (q, k, dq, dk, torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(q),
                                                     torch.zeros_like(k)))
        wq, wk = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
        L.z1_qk_norm_rope(Q, K, OQ, OK, pos, freq, q_weight=w, k_weight=w)
        L.z1_qk_norm_rope_grad(Q, K, A, B, DQ, DK, pos, freq, q_weight=w, k_weight=w, dq_weight=wq, dk_weight=wk,
                               workspace=work(L.z1_qk_norm_rope_grad_workspace(ROWS, 4, 2, dim)))
        return [OQ, OK, DQ, DK, wq, wk]

    for i, (far, dense) in enumerate(zip(run(columns), run(lambda t: t.clone()))):
        assert torch.equal(far, dense), i
        assert float(dense.abs().max()) > 0, i
