"""Angles of positions up to 2^52.  The frequencies are powers of two, so that the angle in
binary64 is exact, and the turn it is part of has to be as well: as for near positions
(test_gpu_qk.py), 2^-25 of a turn in fp32 and its sine and cosine are 2^-21 in all, two
roundings of |a| + |b| more; 2^-20 of it covers them."""
import math

import pytest
import torch

from layer_refs import near
from mixed_precision_zero_amd import layers as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("inter", [False, True])
def test_angles_far_from_zero(inter):
    pos = [s * (2 ** e + 12345 * e + 7) for e in range(20, 53, 2) for s in (1, -1)]
    freq = [1.0, 0.5, 2.0 ** -3, 2.0 ** -7, 2.0 ** -12, 2.0 ** -20]
    n, d = len(pos), 2 * len(freq)
    g = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(n, 1, d, generator=g) for _ in range(2))
    out, dx = (torch.empty(n, 1, d, device="cuda") for _ in range(2))
    at, fr = torch.tensor(pos, device="cuda"), torch.tensor(freq, dtype=torch.float64, device="cuda")
    L.z1_qk_norm_rope(x.cuda(), None, out, None, at, fr, interleaved=inter)
    L.z1_qk_norm_rope_grad(None, None, dy.cuda(), None, dx, None, at, fr, interleaved=inter)
    cos, sin = (torch.tensor([[f(p * w) for w in freq] for p in pos], dtype=torch.float64) for f in (math.cos, math.sin))
    first, second = (slice(0, d, 2), slice(1, d, 2)) if inter else (slice(0, d // 2), slice(d // 2, d))
    for got, v, s in ((out, x, sin), (dx, dy, -sin)):
        a, b = v[:, 0, first].double(), v[:, 0, second].double()
        size = 2.0 ** -20 * (a.abs() + b.abs())
        near(got[:, 0, first], a * cos - b * s, size, "first")
        near(got[:, 0, second], b * cos + a * s, size, "second")
