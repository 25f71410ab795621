"""z1_linear and z1_linear_grad at 2^30 rows, the most there can be: 2^24 tiles of 64,
which no launch holds, so the tiles are of 128.  The rows repeat a block of 4093, whose
own products are checked in 64 bits: (depth + 9) 2^-24 of the sum of magnitudes and half
a step, as in test_gpu_linear.py."""
import pytest
import torch

from layer_refs import U32, half_step, near, tiny
from mixed_precision_zero_amd import layers as L

pytestmark = pytest.mark.gpu
ROWS, BLOCK = 2 ** 30, 4093
T = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def repeated(block):
    m = torch.empty(ROWS, block.shape[1], dtype=T, device="cuda")
    whole = ROWS // BLOCK
    m[:whole * BLOCK].view(whole, BLOCK, -1).copy_(block)
    m[whole * BLOCK:].copy_(block[:ROWS - whole * BLOCK])
    return m


def repeats(m, block):
    whole = ROWS // BLOCK
    return all(bool((part == block).all()) for part in m[:whole * BLOCK].view(whole, BLOCK, -1).split(1 << 16)) \
        and torch.equal(m[whole * BLOCK:], block[:ROWS - whole * BLOCK])


def test_product_and_gradient_of_the_most_rows():
    g = torch.Generator().manual_seed(1)
    x, w, dz = (torch.randn(*s, generator=g).to(T) for s in ((BLOCK, 8), (1, 8), (BLOCK, 1)))
    gw = w.cuda()
    y = torch.full((ROWS, 1), float("nan"), dtype=T, device="cuda")
    far = repeated(x.cuda())
    assert L.z1_linear_workspace(far, gw) == 0
    L.z1_linear(far, gw, y)
    z, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    near(y[:BLOCK], z, 17 * U32 * size + half_step(T) * z.abs() * (1 + 2.0 ** -8) + tiny(T), "y")
    assert repeats(y, y[:BLOCK].clone())
    far_dz = repeated(dz.cuda())
    ws = torch.empty(L.z1_linear_grad_workspace(far_dz, None, gw), dtype=torch.uint8, device="cuda")
    L.z1_linear_grad(far_dz, None, gw, dx=far, workspace=ws)
    z, size = dz.double() @ w.double(), dz.double().abs() @ w.double().abs()
    near(far[:BLOCK], z, 10 * U32 * size + half_step(T) * z.abs() * (1 + 2.0 ** -8) + tiny(T), "dx")
    assert repeats(far, far[:BLOCK].clone())
