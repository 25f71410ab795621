"""z1_dropout against its definition: the mask bit for bit, the values to half a
step (the product with the scale and the sum with the residual are rounded in
fp32 before: two steps of 2^-24)."""
import pytest
import torch

from layer_refs import TYPES, U32, drop, half_step, keep_mask, near, placed, tiny, untouched
from mixed_precision_zero_amd import layers as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rng(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (2, 9), (37, 333), (64, 64), (1, 40000), (5000, 3), (300, 1000)])
@pytest.mark.parametrize("layout", ["plain", "ld", "odd"])
def test_values(kind, rows, cols, layout):
    t = TYPES[kind]
    g = torch.Generator().manual_seed(rows + cols)
    x, r = torch.randn(rows, cols, generator=g).to(t), torch.randn(rows, cols, generator=g).to(t)
    for p, seed, offset, more, res in ((0.1, 1, 0, 0, True), (0.5, -3, -1, 2 ** 63 + 5, False), (0.3, 2 ** 62 + 12345, 2 ** 33 - 1, 1, True)):
        want = drop(x.double(), seed, offset + more, p)
        tol = 2 * U32 * want.abs()
        if res:
            want = want + r.double()
            tol = tol + U32 * want.abs()
        y, buf = placed(torch.zeros_like(x), layout)
        L.z1_dropout(placed(x, layout)[0], y, L.Dropout(rng(seed, offset), p, more), residual=placed(r, layout)[0] if res else None)
        torch.cuda.synchronize()
        near(y, want, tol + half_step(t) * want.abs() * (1 + 2.0 ** -8) + tiny(t), (p, res))
        assert untouched(y, buf)


def test_ends_of_the_probability():
    x = torch.randn(33, 70, device="cuda")
    x[3, 3], x[4, 4] = float("nan"), float("inf")
    y = torch.empty_like(x)
    L.z1_dropout(x, y, L.Dropout(rng(1, 2), 1.0))
    assert bool((y == 0).all())
    r = torch.randn_like(x)
    L.z1_dropout(x, y, L.Dropout(rng(1, 2), 1.0), residual=r)
    assert torch.equal(y, r)
    L.z1_dropout(x, y, L.Dropout(rng(1, 2), 0.0))
    assert torch.equal(y.nan_to_num(), x.nan_to_num())
    L.z1_dropout(x, y, L.Dropout(rng(1, 2), 2.0 ** -18))     # rounds to no dropout at all
    assert torch.equal(y.nan_to_num(), x.nan_to_num())


def test_in_place_and_empty():
    x, r = torch.randn(50, 90, device="cuda"), torch.randn(50, 90, device="cuda")
    d = L.Dropout(rng(4, 4), 0.2)
    y = torch.empty_like(x)
    L.z1_dropout(x, y, d, residual=r)
    a, b = x.clone(), r.clone()
    L.z1_dropout(a, a, d, residual=r)
    L.z1_dropout(x, b, d, residual=b)
    assert torch.equal(a, y) and torch.equal(b, y)
    L.z1_dropout(torch.empty(0, 8, device="cuda"), torch.empty(0, 8, device="cuda"), d)


def test_share_of_kept_elements():
    """2^22 draws: the count is binomial; six standard deviations."""
    x = torch.ones(2048, 2048, device="cuda")
    y = torch.empty_like(x)
    for i, p in enumerate((0.1, 0.5, 0.9)):
        q = 1 - round(p * 65536) / 65536
        L.z1_dropout(x, y, L.Dropout(rng(77, i), p))
        kept = int((y != 0).sum())
        assert abs(kept - q * 2 ** 22) <= 6 * (q * (1 - q) * 2 ** 22) ** 0.5
        assert float(y.max()) == torch.tensor(1 / q, dtype=torch.float64).float()


def test_masks_differ_by_seed_offset_and_row():
    x = torch.ones(64, 256, device="cuda")
    masks = []
    for seed, offset, more in ((1, 0, 0), (2, 0, 0), (1, 1, 0), (1, 2 ** 32, 0), (1 + 2 ** 32, 0, 0)):
        y = torch.empty_like(x)
        L.z1_dropout(x, y, L.Dropout(rng(seed, offset), 0.5, more))
        masks.append(y != 0)
    for i in range(len(masks)):
        assert not torch.equal(masks[i][0], masks[i][1])
        for j in range(i):
            agree = float((masks[i] == masks[j]).float().mean())
            assert abs(agree - 0.5) < 6 * 0.5 / 128      # 2^14 draws
    y = torch.empty_like(x)
    L.z1_dropout(x, y, L.Dropout(rng(1, 0), 0.5, 1))     # offset 0 + 1 is offset 1
    assert torch.equal(y != 0, masks[2])
    assert torch.equal(masks[0].cpu(), keep_mask(64, 256, 1, 0, 0.5))


def test_replayed_graph_draws_from_the_device():
    x = torch.randn(40, 77, device="cuda", dtype=torch.float32)
    state = rng(5, 0)
    y, e = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.z1_dropout(x, y, L.Dropout(state, 0.5))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            L.z1_dropout(x, y, L.Dropout(state, 0.5))
    for i in range(4):
        state.copy_(rng(5, i))
        L.z1_dropout(x, e, L.Dropout(state, 0.5))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, e)


def test_rows_past_32_bits_of_elements():
    """More than 2^32 elements: the last rows, where offsets no longer fit 32 bits."""
    rows, cols = 2 ** 20 + 3, 4104
    x = torch.ones(1, 1, dtype=torch.float16, device="cuda").expand(rows, cols).contiguous()
    d = L.Dropout(rng(9, 9), 0.5)
    L.z1_dropout(x, x, d)
    torch.cuda.synchronize()
    import numpy as np
    from layer_refs import philox
    for row in (0, rows // 2, rows - 1):
        c = np.arange(cols // 8, dtype=np.uint64)
        w = philox((c, np.full_like(c, row), np.full_like(c, 9), np.zeros_like(c)), (9, 0))
        u = np.stack([(w[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xffff) for j in range(8)], 1).reshape(-1)
        assert torch.equal(x[row].cpu() != 0, torch.from_numpy(u >= 32768))
