"""Thin ctypes binding of libz1's operators (include/z1_ops.h): Muon, embedding
lookup and gradient, and the policy and preference losses.

As in ``binding``: argument marshalling and checks only, every operator runs in
the HIP library, there is no fallback.  Calls run on the current GPU, on
``stream`` or torch's current stream, and return without waiting.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import numpy as np
import torch

from .binding import LIB_PATH, _check, _dptr, _held, _p64, _stream as _any_stream, lib

EXPORTS = ("z1_ops_abi_version", "z1_muon_create", "z1_muon_create_wide", "z1_muon_destroy",
           "z1_muon_step", "z1_muon_orthogonalize", "z1_embed_lookup", "z1_embed_grad_workspace",
           "z1_embed_grad", "z1_token_logprob", "z1_logprob_grad", "z1_policy_loss",
           "z1_preference_loss")

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ITYPES = {torch.int64: 0, torch.int32: 1}
MUON_COEFFS = (3.4445, -4.7750, 2.0315)

_P, _I32, _I64, _F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
_PP, _PI64, _PF64 = ctypes.POINTER(_P), ctypes.POINTER(_I64), ctypes.POINTER(_F64)


class MuonBind(ctypes.Structure):
    _fields_ = [("n", _I32), ("grad_dtype", _I32), ("rows", _PI64), ("cols", _PI64),
                ("grad", _PP), ("momentum", _PP), ("master", _PP), ("weights", _PP),
                ("ortho", _PP), ("lr_scale", _PF64), ("wd_scale", _PF64),
                ("a", _F64), ("b", _F64), ("c", _F64), ("eps", _F64),
                ("ns_steps", _I32), ("reserved", _I32)]


class MuonHP(ctypes.Structure):
    _fields_ = [("lr", _F64), ("momentum", _F64), ("weight_decay", _F64), ("clip", _F64),
                ("nesterov", _I32), ("reserved", _I32)]


class EmbedArgs(ctypes.Structure):
    _fields_ = [("n_ids", _I64), ("vocab", _I64), ("dim", _I64), ("ids", _P),
                ("id_type", _I32), ("dtype", _I32), ("scale", _F64)]


class Logits(ctypes.Structure):
    _fields_ = [("n_rows", _I64), ("vocab", _I64), ("logits", _P), ("ld", _I64),
                ("targets", _P), ("target_type", _I32), ("dtype", _I32)]


class PolicyArgs(ctypes.Structure):
    _fields_ = [("old_logp", _P), ("ref_logp", _P), ("advantages", _P), ("weights", _P),
                ("clip_low", _F64), ("clip_high", _F64), ("kl_coef", _F64), ("scale", _F64),
                ("loss", _P), ("token_loss", _P), ("logp", _P), ("dlogits", _P),
                ("ld_dlogits", _I64)]


class PreferenceArgs(ctypes.Structure):
    _fields_ = [("n_rows", _I64), ("n_pairs", _I64), ("logp", _P), ("ref_logp", _P),
                ("targets", _P), ("cu_seqlens", _P), ("target_type", _I32), ("cu_type", _I32),
                ("beta", _F64), ("label_smoothing", _F64), ("scale", _F64),
                ("loss", _P), ("pair_loss", _P), ("margins", _P), ("dlogp", _P)]


def _declare():
    ref = ctypes.POINTER
    sig = {
        "z1_ops_abi_version": ([], _I32),
        "z1_muon_create": ([ref(_P), ref(MuonBind), _P], ctypes.c_int),
        "z1_muon_create_wide": ([ref(_P), ref(MuonBind), _P], ctypes.c_int),
        "z1_muon_destroy": ([_P], ctypes.c_int),
        "z1_muon_step": ([_P, ref(MuonHP), _P, _P], ctypes.c_int),
        "z1_muon_orthogonalize": ([_P, _P], ctypes.c_int),
        "z1_embed_lookup": ([ref(EmbedArgs), _P, _I64, _P, _I64, _P], ctypes.c_int),
        "z1_embed_grad_workspace": ([_I64, _I64, _I64, _PI64], ctypes.c_int),
        "z1_embed_grad": ([ref(EmbedArgs), _P, _I64, _P, _I32, _P, _I64, _P], ctypes.c_int),
        "z1_token_logprob": ([ref(Logits), _P, _P, _P], ctypes.c_int),
        "z1_logprob_grad": ([ref(Logits), _P, _P, _P, _I64, _P], ctypes.c_int),
        "z1_policy_loss": ([ref(Logits), ref(PolicyArgs), _P], ctypes.c_int),
        "z1_preference_loss": ([ref(PreferenceArgs), _P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        if not hasattr(lib, name):
            raise ImportError(f"{LIB_PATH} has no {name}; run __graft_entry__.build()")
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res


_declare()


def z1_ops_abi_version() -> int:
    return int(lib.z1_ops_abi_version())


def _dtype_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name}: dtype {t.dtype}, expected float32, bfloat16 or float16")
    return DTYPES[t.dtype]


def _itype_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype not in ITYPES:
        raise TypeError(f"{name}: dtype {t.dtype}, expected int64 or int32")
    return ITYPES[t.dtype]


def _rows_of(t, name: str, dtype=None, shape=None) -> int:
    """Distance in elements of two rows of a 2-D tensor with contiguous rows
    that do not overlap."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected 2")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    n, d = t.shape
    if t.is_contiguous():
        return d
    step = t.stride()
    if d > 1 and step[1] != 1:
        raise ValueError(f"{name}: rows not contiguous")
    ld = step[0] if n > 1 else d
    if ld < d:
        raise ValueError(f"{name}: rows overlap (stride {ld} of {d} elements)")
    return ld


def _on_gpu(items) -> None:
    """Every tensor on the current GPU.  (A tensor on a GPU means that torch
    has initialised it, so the current one is asked for without torch's own
    check of that: a small operator takes less time than its checks.)"""
    here = -1
    for t, name in items:
        if t is None or isinstance(t, int):
            continue
        at = t.get_device()
        if at < 0:
            raise ValueError(f"{name}: on {t.device}, expected the current GPU")
        if here < 0:
            here = torch._C._cuda_getDevice()
        if at != here:
            raise ValueError(f"{name}: on {t.device}, expected cuda:{here}")


def _checked(items, rows=()) -> None:
    """Reject tensors the library would read or write out of bounds or
    misread, as binding._check_tensors does (items: tensor, name, dtype or
    None, elements or bytes), with fewer calls into torch.  rows: further
    (tensor, name) whose device alone is still to be looked at."""
    for t, name, dtype, need in items:
        if t is None or isinstance(t, int):
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch tensor or a device address, "
                            f"got {type(t).__name__}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: not contiguous")
        have = t.numel() if dtype is not None else t.numel() * t.element_size()
        if have < need:
            unit = "elements" if dtype is not None else "bytes"
            raise ValueError(f"{name}: {have} {unit}, the call touches {need}")
    _on_gpu([i[:2] for i in items] + list(rows))


def _stream(stream):
    """hipStream_t of a torch stream (default: torch's current stream)."""
    if stream is None and torch.cuda.is_initialized():
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) or None
    return _any_stream(stream)


# --------------------------------------------------------------------------
# Muon
# --------------------------------------------------------------------------

class Muon:
    """Owner of a z1_muon handle (destroyed with z1_muon_destroy)."""

    def __init__(self, handle: int, n: int, keep):
        self.handle = handle
        self.n = n
        self._keep = keep   # the bound memory: the handle writes into it until it is destroyed

    def close(self):
        if self.handle:
            _check(lib.z1_muon_destroy(self.handle), "z1_muon_destroy")
            self.handle = 0
            self._keep = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def z1_muon_create(shapes: Sequence, grads: Sequence, *, momentum: Optional[Sequence] = None,
                   master: Optional[Sequence] = None, weights: Optional[Sequence] = None,
                   ortho: Optional[Sequence] = None, lr_scale: Optional[Sequence[float]] = None,
                   wd_scale: Optional[Sequence[float]] = None, ns_steps: int = 5,
                   coeffs=MUON_COEFFS, eps: float = 1e-7, wide: bool = False,
                   stream=None) -> Muon:
    """Bind a list of matrices: shapes[i] = (rows, cols), grads[i] fp32 or
    bf16 (one type for all), momentum / master fp32 and weights bf16 (all
    three for z1_muon_step, or none), ortho bf16 (for z1_muon_orthogonalize).
    Every tensor is row-major and contiguous with rows * cols elements.
    wide: products of 22-bit instead of 11-bit operands (z1_muon_create_wide),
    as exact as fp32 ones, at two to three times the time."""
    rows = np.ascontiguousarray([int(s[0]) for s in shapes], dtype=np.int64)
    cols = np.ascontiguousarray([int(s[1]) for s in shapes], dtype=np.int64)
    n = rows.size
    lists = dict(grads=grads, momentum=momentum, master=master, weights=weights, ortho=ortho)
    for name, x in lists.items():
        if x is not None and len(x) != n:
            raise ValueError(f"{name} must list one tensor per matrix")
    for name, x in (("lr_scale", lr_scale), ("wd_scale", wd_scale)):
        if x is not None and len(x) != n:
            raise ValueError(f"{name} needs one entry per matrix")
    gtype = torch.float32
    if n and isinstance(grads[0], torch.Tensor):
        gtype = grads[0].dtype
    if gtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"grads: dtype {gtype}, expected float32 or bfloat16")
    want = dict(grads=gtype, momentum=torch.float32, master=torch.float32,
                weights=torch.bfloat16, ortho=torch.bfloat16)
    _checked([(x[i], f"{name}[{i}]", want[name], int(rows[i] * cols[i]))
                    for name, x in lists.items() if x is not None for i in range(n)])

    def table(x):
        if x is None:
            return None
        return (ctypes.c_void_p * max(n, 1))(*[_dptr(t) for t in x])

    arr = {name: table(x) for name, x in lists.items()}
    scales = [None if x is None else np.ascontiguousarray(x, dtype=np.float64)
              for x in (lr_scale, wd_scale)]
    pp = lambda x: None if x is None else ctypes.cast(x, _PP)  # noqa: E731
    pd = lambda x: None if x is None else x.ctypes.data_as(_PF64)  # noqa: E731
    b = MuonBind(n=n, grad_dtype=DTYPES[gtype], rows=_p64(rows), cols=_p64(cols),
                 grad=pp(arr["grads"]), momentum=pp(arr["momentum"]), master=pp(arr["master"]),
                 weights=pp(arr["weights"]), ortho=pp(arr["ortho"]), lr_scale=pd(scales[0]),
                 wd_scale=pd(scales[1]), a=float(coeffs[0]), b=float(coeffs[1]),
                 c=float(coeffs[2]), eps=float(eps), ns_steps=int(ns_steps), reserved=0)
    h = ctypes.c_void_p()
    name = "z1_muon_create_wide" if wide else "z1_muon_create"
    _check(getattr(lib, name)(ctypes.byref(h), ctypes.byref(b), _stream(stream)), name)
    return Muon(h.value, n, _held(tuple(lists.values())))


def z1_muon_step(muon: Muon, *, lr: float, momentum: float = 0.95, weight_decay: float = 0.0,
                 nesterov: bool = True, clip: float = 0.0, d_S=None, stream=None) -> None:
    """One update of every bound matrix.  d_S: device float64, the squared
    global gradient norm, needed when clip > 0."""
    if d_S is not None:
        _checked([(d_S, "d_S", torch.float64, 1)])
    hp = MuonHP(lr, momentum, weight_decay, clip, int(bool(nesterov)), 0)
    _check(lib.z1_muon_step(muon.handle, ctypes.byref(hp), _dptr(d_S), _stream(stream)),
           "z1_muon_step")


def z1_muon_orthogonalize(muon: Muon, stream=None) -> None:
    """ortho[i] = the orthogonalised grads[i]."""
    _check(lib.z1_muon_orthogonalize(muon.handle, _stream(stream)), "z1_muon_orthogonalize")


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------

def _embed_args(ids, vocab: int, dim: int, dtype: int, scale: float) -> EmbedArgs:
    it = _itype_of(ids, "ids")
    if ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids: expected one contiguous dimension")
    return EmbedArgs(ids.numel(), vocab, dim, ids.data_ptr(), it, dtype, float(scale))


def z1_embed_lookup(weight, ids, out, *, scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * weight[ids[t]]; weight [V, d] and out [T, d] of one
    type with contiguous rows, ids [T] int64 or int32.  A negative id gives a
    zero row, an id of V or more a NaN row."""
    dt = _dtype_of(weight, "weight")
    ld_w = _rows_of(weight, "weight")
    args = _embed_args(ids, weight.shape[0], weight.shape[1], dt, scale)
    ld_o = _rows_of(out, "out", weight.dtype, (ids.numel(), weight.shape[1]))
    _on_gpu([(weight, "weight"), (ids, "ids"), (out, "out")])
    _check(lib.z1_embed_lookup(ctypes.byref(args), weight.data_ptr(), ld_w, out.data_ptr(), ld_o,
                               _stream(stream)), "z1_embed_lookup")


def z1_embed_grad_workspace(n_ids: int, vocab: int, dim: int) -> int:
    """Bytes of device workspace z1_embed_grad needs."""
    b = ctypes.c_int64()
    _check(lib.z1_embed_grad_workspace(int(n_ids), int(vocab), int(dim), ctypes.byref(b)),
           "z1_embed_grad_workspace")
    return b.value


def z1_embed_grad(ids, dout, dweight, *, scale: float = 1.0, accumulate: bool = False, workspace,
                  stream=None) -> None:
    """dweight[v] (+)= scale * the sum of dout's rows with ids[t] == v, in
    fp32.  dweight [V, d] fp32 contiguous (for example a view of the step's
    acc arena); accumulate False writes all of it.  Ids outside [0, V) are
    skipped."""
    dt = _dtype_of(dout, "dout")
    if not isinstance(dweight, torch.Tensor) or dweight.dim() != 2:
        raise ValueError("dweight: expected a 2-D torch tensor")
    vocab, dim = dweight.shape
    args = _embed_args(ids, vocab, dim, dt, scale)
    ld = _rows_of(dout, "dout", None, (ids.numel(), dim))
    need = z1_embed_grad_workspace(ids.numel(), vocab, dim)
    _checked([(dweight, "dweight", torch.float32, vocab * dim), (workspace, "workspace", None, need)],
             ((ids, "ids"), (dout, "dout")))
    nbytes = workspace.numel() * workspace.element_size() if isinstance(workspace, torch.Tensor) else need
    _check(lib.z1_embed_grad(ctypes.byref(args), dout.data_ptr(), ld, dweight.data_ptr(),
                             int(bool(accumulate)), _dptr(workspace), nbytes, _stream(stream)),
           "z1_embed_grad")


# --------------------------------------------------------------------------
# losses
# --------------------------------------------------------------------------

def _logits_args(logits, targets) -> Logits:
    dt = _dtype_of(logits, "logits")
    ld = _rows_of(logits, "logits")
    it = _itype_of(targets, "targets")
    if targets.shape != logits.shape[:1] or not targets.is_contiguous():
        raise ValueError(f"targets: expected {logits.shape[0]} contiguous entries")
    return Logits(logits.shape[0], logits.shape[1], logits.data_ptr(), ld, targets.data_ptr(), it, dt)


def z1_token_logprob(logits, targets, logp, lse=None, *, stream=None) -> None:
    """logp[r] = log softmax(logits[r])[targets[r]] and lse[r], fp32; 0 where
    the target is negative, NaN where it is the vocabulary's size or more."""
    x = _logits_args(logits, targets)
    _checked([(logp, "logp", torch.float32, x.n_rows), (lse, "lse", torch.float32, x.n_rows)],
             ((logits, "logits"), (targets, "targets")))
    _check(lib.z1_token_logprob(ctypes.byref(x), _dptr(logp), _dptr(lse), _stream(stream)),
           "z1_token_logprob")


def z1_logprob_grad(logits, targets, lse, dlogp, dlogits, *, stream=None) -> None:
    """dlogits[r, v] = dlogp[r] (1[v == targets[r]] - softmax(logits[r])[v]),
    in the logits' type; dlogits may be logits."""
    x = _logits_args(logits, targets)
    ld = _rows_of(dlogits, "dlogits", logits.dtype, logits.shape)
    _checked([(lse, "lse", torch.float32, x.n_rows), (dlogp, "dlogp", torch.float32, x.n_rows)],
             ((logits, "logits"), (targets, "targets"), (dlogits, "dlogits")))
    _check(lib.z1_logprob_grad(ctypes.byref(x), _dptr(lse), _dptr(dlogp), dlogits.data_ptr(), ld,
                               _stream(stream)), "z1_logprob_grad")


def z1_policy_loss(logits, targets, old_logp, advantages, *, loss, token_loss, logp=None,
                   dlogits=None, ref_logp=None, weights=None, clip_low: float = 0.2,
                   clip_high: float = 0.2, kl_coef: float = 0.0, scale: float = 1.0,
                   stream=None) -> None:
    """Clipped policy loss with a KL term to ref_logp (None, or kl_coef 0: no such term):
    loss[0] = scale * sum of weights * token_loss, and dlogits (None: no
    gradient) its gradient in the logits.  Rows with a negative target or a
    zero weight count for nothing.  dlogits may be logits."""
    x = _logits_args(logits, targets)
    n = x.n_rows
    ld = 0
    if dlogits is not None:
        ld = _rows_of(dlogits, "dlogits", logits.dtype, logits.shape)
    f32 = torch.float32
    _checked([(t, name, f32, n) for t, name in (
        (old_logp, "old_logp"), (advantages, "advantages"), (ref_logp, "ref_logp"),
        (weights, "weights"), (token_loss, "token_loss"), (logp, "logp"))] + [(loss, "loss", f32, 1)],
        ((logits, "logits"), (targets, "targets"), (dlogits, "dlogits")))
    a = PolicyArgs(_dptr(old_logp), _dptr(ref_logp), _dptr(advantages), _dptr(weights),
                   float(clip_low), float(clip_high), float(kl_coef), float(scale), _dptr(loss),
                   _dptr(token_loss), _dptr(logp), _dptr(dlogits), ld)
    _check(lib.z1_policy_loss(ctypes.byref(x), ctypes.byref(a), _stream(stream)), "z1_policy_loss")


def z1_preference_loss(logp, ref_logp, targets, cu_seqlens, *, beta: float, scale: float = 1.0,
                       label_smoothing: float = 0.0, loss, pair_loss, margins=None, dlogp=None,
                       stream=None) -> None:
    """Preference loss of pairs of answers: sequence 2p (chosen) and 2p + 1
    (rejected) hold rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1.  loss[0] =
    scale * sum of pair_loss, dlogp its gradient in logp."""
    it = _itype_of(targets, "targets")
    ct = _itype_of(cu_seqlens, "cu_seqlens")
    n = targets.numel()
    if cu_seqlens.numel() % 2 != 1:
        raise ValueError(f"cu_seqlens: {cu_seqlens.numel()} entries, expected 2 pairs + 1")
    pairs = (cu_seqlens.numel() - 1) // 2
    f32 = torch.float32
    _checked([(targets, "targets", targets.dtype, n),
                    (cu_seqlens, "cu_seqlens", cu_seqlens.dtype, 2 * pairs + 1),
                    (logp, "logp", f32, n), (ref_logp, "ref_logp", f32, n), (dlogp, "dlogp", f32, n),
                    (pair_loss, "pair_loss", f32, pairs), (margins, "margins", f32, pairs),
                    (loss, "loss", f32, 1)])
    a = PreferenceArgs(n, pairs, _dptr(logp), _dptr(ref_logp), _dptr(targets), _dptr(cu_seqlens),
                       it, ct, float(beta), float(label_smoothing), float(scale), _dptr(loss),
                       _dptr(pair_loss), _dptr(margins), _dptr(dlogp))
    _check(lib.z1_preference_loss(ctypes.byref(a), _stream(stream)), "z1_preference_loss")
