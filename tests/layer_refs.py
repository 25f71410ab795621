"""The layers' definitions in 64 bits on the CPU, and where tests put matrices."""
import math

import numpy as np
import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U32 = 2.0 ** -24


def half_step(t):
    """The largest relative rounding of type t."""
    return torch.finfo(t).eps / 2


def tiny(t):
    """The largest absolute rounding near zero: half the smallest subnormal."""
    return {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}[t]


def philox(counter, key):
    """Philox4x32-10 (Salmon et al. 2011) of Python integers or uint64 arrays."""
    c, k = [np.asarray(x, dtype=np.uint64) for x in counter], [int(x) for x in key]
    low, shift = np.uint64(0xffffffff), np.uint64(32)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> shift) ^ c[1] ^ np.uint64(k[0]), q & low, (p >> shift) ^ c[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]
    return c


def keep_mask(rows, cols, seed, offset, p):
    """Which elements of a [rows, cols] matrix a dropout keeps."""
    blocks = -(-cols // 8)
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    r, b = np.meshgrid(np.arange(rows, dtype=np.uint64), np.arange(blocks, dtype=np.uint64), indexing="ij")
    words = philox((b, r, np.full_like(b, offset & 0xffffffff), np.full_like(b, offset >> 32)), (seed & 0xffffffff, seed >> 32))
    u = np.stack([(words[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xffff) for j in range(8)], 2)
    return torch.from_numpy(u.reshape(rows, blocks * 8)[:, :cols].astype(np.int64) >= int(round(p * 65536)))


def drop(x, seed, offset, p):
    """x (64 bits) after dropout."""
    if not p:
        return x
    n = int(round(p * 65536))
    scale = 65536.0 / (65536 - n) if n < 65536 else 0.0
    return torch.where(keep_mask(x.shape[0], x.shape[1], seed, offset, p), x * scale, torch.zeros_like(x))


def act(z, name):
    """(act(z), act'(z)) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "relu2":
        return z.clamp(min=0) ** 2, 2 * z.clamp(min=0)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        phi = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * a * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * (1 - s) * 2 * a * (1 + 3 * 0.044715 * z ** 2)


def placed(x, layout="plain", fill=float("nan")):
    """x on the GPU inside a larger buffer of `fill`: (matrix, buffer).  layouts:
    plain; ld: rows further apart, 16-byte aligned; odd: rows an odd distance
    apart, the base at an odd element."""
    rows, cols = x.shape
    ld, off = {"plain": (cols, 0), "ld": (-(-cols // 8) * 8 + 16, 8), "odd": ((cols + 3) | 1, 1)}[layout]
    buf = torch.full((off + rows * ld + 16,), fill, dtype=x.dtype, device="cuda")
    m = buf[off:off + rows * ld].view(rows, ld)[:, :cols]
    m.copy_(x)
    return m, buf


def untouched(m, buf, fill_is_nan=True):
    """Whether everything of the buffer outside the matrix still is NaN."""
    seen = torch.zeros_like(buf, dtype=torch.bool)
    off = (m.data_ptr() - buf.data_ptr()) // buf.element_size()
    seen[off:].as_strided(m.shape, m.stride()).fill_(True)
    return bool(torch.isnan(buf[~seen]).all())


def near(got, want, tol, what=""):
    """|got - want| <= tol elementwise (64 bits, NaN equal to NaN)."""
    got, want, tol = got.detach().double().cpu(), want.double(), torch.as_tensor(tol, dtype=torch.float64).expand_as(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), what
    off = (got - want).abs()
    bad = ~nan & ~(off <= tol) & ~(got == want)
    assert not bad.any(), (what, int(bad.sum()), float((off / tol.clamp(min=1e-300))[bad].max()), bad.nonzero()[0].tolist())
