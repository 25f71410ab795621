"""Thin ctypes binding of libz1's layers (include/z1_layers.h): linear with its
epilogue and gradients, dropout, and norm and rotation of queries and keys.

As in ``ops``: argument marshalling and checks only, every layer runs in the HIP
library, there is no fallback.  Calls run on the current GPU, on ``stream`` or
torch's current stream, and return without waiting.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from .binding import LIB_PATH, _check, lib
from .ops import DTYPES, _checked, _dtype_of, _itype_of, _on_gpu, _rows_of, _stream

EXPORTS = ("z1_layers_abi_version", "z1_dropout", "z1_linear_workspace", "z1_linear", "z1_linear_dz_workspace",
           "z1_linear_dz", "z1_linear_grad_workspace", "z1_linear_grad", "z1_qk_norm_rope",
           "z1_qk_norm_rope_grad_workspace", "z1_qk_norm_rope_grad")

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "relu2": 5}

_P, _I32, _I64, _U64, _F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_double
_PI64 = ctypes.POINTER(_I64)


class Drop(ctypes.Structure):
    _fields_ = [("rng", _P), ("offset", _U64), ("p", _F64)]


class DropoutArgs(ctypes.Structure):
    _fields_ = [("rows", _I64), ("cols", _I64), ("x", _P), ("residual", _P), ("y", _P), ("ld_x", _I64),
                ("ld_residual", _I64), ("ld_y", _I64), ("drop", Drop), ("dtype", _I32), ("reserved", _I32)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("rows", _I64), ("in_", _I64), ("out", _I64), ("x", _P), ("weight", _P), ("bias", _P), ("mul", _P),
                ("residual", _P), ("pre", _P), ("y", _P), ("ld_x", _I64), ("ld_weight", _I64), ("ld_mul", _I64),
                ("ld_residual", _I64), ("ld_pre", _I64), ("ld_y", _I64), ("drop", Drop), ("dtype", _I32), ("act", _I32)]


class LinearDzArgs(ctypes.Structure):
    _fields_ = [("rows", _I64), ("out", _I64), ("dy", _P), ("pre", _P), ("mul", _P), ("dz", _P), ("dmul", _P),
                ("dbias", _P), ("ld_dy", _I64), ("ld_pre", _I64), ("ld_mul", _I64), ("ld_dz", _I64), ("ld_dmul", _I64),
                ("drop", Drop), ("dtype", _I32), ("act", _I32), ("accumulate", _I32), ("reserved", _I32)]


class LinearGradArgs(ctypes.Structure):
    _fields_ = [("rows", _I64), ("in_", _I64), ("out", _I64), ("dz", _P), ("x", _P), ("weight", _P), ("add", _P),
                ("dx", _P), ("dweight", _P), ("ld_dz", _I64), ("ld_x", _I64), ("ld_weight", _I64), ("ld_add", _I64),
                ("ld_dx", _I64), ("ld_dweight", _I64), ("dtype", _I32), ("dweight_dtype", _I32), ("accumulate", _I32),
                ("reserved", _I32)]


class Heads(ctypes.Structure):
    _fields_ = [("heads", _I64), ("x", _P), ("out", _P), ("dout", _P), ("weight", _P), ("dweight", _P),
                ("x_token", _I64), ("x_head", _I64), ("out_token", _I64), ("out_head", _I64), ("dout_token", _I64),
                ("dout_head", _I64)]


class QkArgs(ctypes.Structure):
    _fields_ = [("tokens", _I64), ("dim", _I32), ("n_freq", _I32), ("q", Heads), ("k", Heads), ("positions", _P),
                ("inv_freq", _P), ("eps", _F64), ("position_type", _I32), ("dtype", _I32), ("interleaved", _I32),
                ("accumulate", _I32)]


def _declare():
    ref = ctypes.POINTER
    sig = {
        "z1_layers_abi_version": ([], _I32),
        "z1_dropout": ([ref(DropoutArgs), _P], ctypes.c_int),
        "z1_linear_workspace": ([ref(LinearArgs), _PI64], ctypes.c_int),
        "z1_linear": ([ref(LinearArgs), _P, _I64, _P], ctypes.c_int),
        "z1_linear_dz_workspace": ([_I64, _I64, _PI64], ctypes.c_int),
        "z1_linear_dz": ([ref(LinearDzArgs), _P, _I64, _P], ctypes.c_int),
        "z1_linear_grad_workspace": ([ref(LinearGradArgs), _PI64], ctypes.c_int),
        "z1_linear_grad": ([ref(LinearGradArgs), _P, _I64, _P], ctypes.c_int),
        "z1_qk_norm_rope": ([ref(QkArgs), _P], ctypes.c_int),
        "z1_qk_norm_rope_grad_workspace": ([_I64, _I64, _I64, _I32, _PI64], ctypes.c_int),
        "z1_qk_norm_rope_grad": ([ref(QkArgs), _P, _I64, _P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        if not hasattr(lib, name):
            raise ImportError(f"{LIB_PATH} has no {name}; run __graft_entry__.build()")
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res


_declare()


def z1_layers_abi_version() -> int:
    return int(lib.z1_layers_abi_version())


class Dropout(NamedTuple):
    """What a dropout draws its mask from.  rng: device int64 or uint64 [2], seed
    and offset of the step; offset tells the dropouts of one step apart.  The
    gradient takes the same values as the forward pass."""
    rng: torch.Tensor
    p: float
    offset: int = 0


class _Call:
    """The checks of one call.  What is right in every respect (type, shape, dense
    rows, the first tensor's device) takes few calls into torch, as a small layer
    takes less time than its checks; anything else goes through the full ones,
    which raise what is wrong with it.  Devices come last, as one reads types and
    shapes first."""

    __slots__ = ("here", "odd")

    def __init__(self, lead):
        self.here = lead.get_device()
        self.odd = [] if self.here >= 0 else [(lead, "the first tensor")]

    def matrix(self, t, name: str, dtype, shape):
        """(address, distance of rows) of a matrix, or (None, 0)."""
        if t is None:
            return None, 0
        if getattr(t, "dtype", None) is dtype and t.shape == shape and t.is_contiguous():
            ld = shape[1]
        else:
            ld = _rows_of(t, name, dtype, shape)
        if t.get_device() != self.here:
            self.odd.append((t, name))
        return t.data_ptr(), ld

    def vector(self, t, name: str, dtype, need: int):
        """Address of a contiguous tensor of at least `need` elements, or None."""
        if t is None:
            return None
        if (getattr(t, "dtype", None) is not dtype or not t.is_contiguous() or t.numel() < need
                or t.get_device() != self.here):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
            _checked([(t, name, dtype, need)])
            self.odd.append((t, name))
        return t.data_ptr()

    def workspace(self, t):
        """(address, bytes) of a workspace, or (None, 0)."""
        if t is None:
            return None, 0
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"workspace: expected a torch tensor, got {type(t).__name__}")
        n = t.numel() * t.element_size()
        if n == 0:
            return None, 0
        if not t.is_contiguous() or t.get_device() != self.here:
            _checked([(t, "workspace", None, 0)])
            self.odd.append((t, "workspace"))
        return t.data_ptr(), n

    def dropout(self, d: Optional[Dropout]) -> Drop:
        if d is None:
            return _NO_DROP
        if not isinstance(d.rng, torch.Tensor) or d.rng.dtype not in (torch.int64, torch.uint64):
            raise TypeError("dropout.rng: expected a torch tensor of int64 or uint64")
        return Drop(self.vector(d.rng, "dropout.rng", d.rng.dtype, 2), d.offset & 0xffffffffffffffff, d.p)

    def done(self):
        """Every tensor on the current GPU."""
        if self.odd or torch._C._cuda_getDevice() != self.here:
            _on_gpu(self.odd)
            raise ValueError(f"the tensors are on cuda:{self.here}, which is not the current GPU")


_NO_DROP = Drop(None, 0, 0.0)


def _act_of(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act: {act!r}, expected one of {', '.join(ACTS)}")
    return ACTS[act]


# --------------------------------------------------------------------------
# dropout
# --------------------------------------------------------------------------

def z1_dropout(x, y, dropout: Dropout, *, residual=None, stream=None) -> None:
    """y = residual + drop(x) (residual None: drop(x)) of 2-D tensors of one
    type; y may be x or residual.  The gradient is the same call on dy."""
    dt = _dtype_of(x, "x")
    ld_x = _rows_of(x, "x")
    call, shape, kind = _Call(x), x.shape, x.dtype
    py, ld_y = call.matrix(y, "y", kind, shape)
    pr, ld_r = call.matrix(residual, "residual", kind, shape)
    drop = call.dropout(dropout)
    call.done()
    a = DropoutArgs(shape[0], shape[1], x.data_ptr(), pr, py, ld_x, ld_r, ld_y, drop, dt, 0)
    _check(lib.z1_dropout(ctypes.byref(a), _stream(stream)), "z1_dropout")


# --------------------------------------------------------------------------
# linear
# --------------------------------------------------------------------------

def _operands(x, weight):
    """(the call, dtype, rows, in, out, distances of x's and weight's rows)"""
    dt = _dtype_of(x, "x")
    ld_x = _rows_of(x, "x")
    call = _Call(x)
    ld_w = _rows_of(weight, "weight", x.dtype)
    (n, k), (m, k_w) = x.shape, weight.shape
    if k_w != k:
        raise ValueError(f"weight: {k_w} columns, x has {k}")
    if weight.get_device() != call.here:
        call.odd.append((weight, "weight"))
    return call, dt, n, k, m, ld_x, ld_w


def z1_linear_workspace(x, weight) -> int:
    """Bytes of device workspace z1_linear needs for these operands."""
    _, dt, n, k, m, ld_x, ld_w = _operands(x, weight)
    a = LinearArgs(rows=n, in_=k, out=m, x=x.data_ptr(), weight=weight.data_ptr(), ld_x=ld_x, ld_weight=ld_w, dtype=dt)
    b = _I64()
    _check(lib.z1_linear_workspace(ctypes.byref(a), ctypes.byref(b)), "z1_linear_workspace")
    return b.value


def z1_linear(x, weight, y, *, bias=None, act: str = "none", mul=None, residual=None, pre=None,
              dropout: Optional[Dropout] = None, workspace=None, stream=None) -> None:
    """y = residual + drop(act(x weight^T + bias) * mul) and pre = x weight^T +
    bias, for x [rows, in], weight [out, in], bias [out] and the others [rows,
    out], all of one type; None leaves a term out.  y may be residual or mul."""
    call, dt, n, k, m, ld_x, ld_w = _operands(x, weight)
    kind, shape = x.dtype, (n, m)
    py, ld_y = call.matrix(y, "y", kind, shape)
    pm, ld_m = call.matrix(mul, "mul", kind, shape)
    pr, ld_r = call.matrix(residual, "residual", kind, shape)
    pp, ld_p = call.matrix(pre, "pre", kind, shape)
    pb = call.vector(bias, "bias", kind, m)
    act = _act_of(act)
    drop = call.dropout(dropout)
    work, size = call.workspace(workspace)
    call.done()
    a = LinearArgs(n, k, m, x.data_ptr(), weight.data_ptr(), pb, pm, pr, pp, py, ld_x, ld_w, ld_m, ld_r, ld_p, ld_y, drop,
                   dt, act)
    _check(lib.z1_linear(ctypes.byref(a), work, size, _stream(stream)), "z1_linear")


def z1_linear_dz_workspace(rows: int, out: int) -> int:
    """Bytes of device workspace z1_linear_dz needs for dbias."""
    b = _I64()
    _check(lib.z1_linear_dz_workspace(int(rows), int(out), ctypes.byref(b)), "z1_linear_dz_workspace")
    return b.value


def z1_linear_dz(dy, dz=None, *, act: str = "none", pre=None, mul=None, dmul=None, dbias=None, accumulate: bool = False,
                 dropout: Optional[Dropout] = None, workspace=None, stream=None) -> None:
    """The gradient through z1_linear's epilogue: dz = drop(dy) * mul * act'(pre),
    dmul = drop(dy) * act(pre), and dbias [out] fp32 (+)= the column sums of dz.
    dz, dmul and dbias may be None; dz may be dy, pre or mul, dmul may be mul or
    pre."""
    dt = _dtype_of(dy, "dy")
    ld_dy = _rows_of(dy, "dy")
    call, kind, shape = _Call(dy), dy.dtype, dy.shape
    pp, ld_p = call.matrix(pre, "pre", kind, shape)
    pm, ld_m = call.matrix(mul, "mul", kind, shape)
    pz, ld_z = call.matrix(dz, "dz", kind, shape)
    pd, ld_d = call.matrix(dmul, "dmul", kind, shape)
    pb = call.vector(dbias, "dbias", torch.float32, shape[1])
    act = _act_of(act)
    drop = call.dropout(dropout)
    work, size = call.workspace(workspace)
    call.done()
    a = LinearDzArgs(shape[0], shape[1], dy.data_ptr(), pp, pm, pz, pd, pb, ld_dy, ld_p, ld_m, ld_z, ld_d, drop, dt, act,
                     1 if accumulate else 0, 0)
    _check(lib.z1_linear_dz(ctypes.byref(a), work, size, _stream(stream)), "z1_linear_dz")


def _grad_operands(dz, x, weight):
    """(the call, the arguments without the outputs, the shape of dx, that of dweight)"""
    dt = _dtype_of(dz, "dz")
    ld_dz = _rows_of(dz, "dz")
    call, kind = _Call(dz), dz.dtype
    n, m = dz.shape
    known = x if x is not None else weight
    if known is None:
        raise ValueError("x and weight: both None")
    _dtype_of(known, "x" if x is not None else "weight")
    k = known.shape[-1]
    px, ld_x = call.matrix(x, "x", kind, (n, k))
    pw, ld_w = call.matrix(weight, "weight", kind, (m, k))
    return call, LinearGradArgs(n, k, m, dz.data_ptr(), px, pw, None, None, None, ld_dz, ld_x, ld_w, 0, 0, 0, dt, 0, 0, 0), (n, k), (m, k)


def z1_linear_grad_workspace(dz, x, weight) -> int:
    """Bytes of device workspace z1_linear_grad needs for these operands, for
    either gradient or both."""
    a = _grad_operands(dz, x, weight)[1]
    # the outputs are not looked at, but for being there
    a.dx, a.dweight = a.weight, a.x
    b = _I64()
    _check(lib.z1_linear_grad_workspace(ctypes.byref(a), ctypes.byref(b)), "z1_linear_grad_workspace")
    return b.value


def z1_linear_grad(dz, x, weight, *, dx=None, add=None, dweight=None, accumulate: bool = False, workspace=None,
                   stream=None) -> None:
    """dx = dz weight (+ add) and dweight (+)= dz^T x, for dz [rows, out], x
    [rows, in] (None without dweight) and weight [out, in] (None without dx).
    dweight: fp32, written or with accumulate added to (for example a view of the
    step's acc arena), or of dz's type and written.  dx may be add."""
    call, a, like_x, like_w = _grad_operands(dz, x, weight)
    kind = dz.dtype
    if dx is None and dweight is None:
        raise ValueError("dx and dweight: both None")
    a.dx, a.ld_dx = call.matrix(dx, "dx", kind, like_x)
    a.add, a.ld_add = call.matrix(add, "add", kind, like_x)
    if dweight is not None:
        to = getattr(dweight, "dtype", None)
        if to is not torch.float32 and to is not kind:
            raise TypeError(f"dweight: dtype {to}, expected float32 or {kind}")
        a.dweight, a.ld_dweight = call.matrix(dweight, "dweight", to, like_w)
        a.dweight_dtype = DTYPES[to]
    a.accumulate = 1 if accumulate else 0
    work, size = call.workspace(workspace)
    call.done()
    _check(lib.z1_linear_grad(ctypes.byref(a), work, size, _stream(stream)), "z1_linear_grad")


# --------------------------------------------------------------------------
# queries and keys
# --------------------------------------------------------------------------

def _heads_of(call, t, name: str, dtype, shape):
    """(address, token stride, head stride) of [tokens, heads, dim] whose heads
    are contiguous and do not overlap; the addresses of no elements are null."""
    if getattr(t, "dtype", None) is not dtype:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != call.here:
        call.odd.append((t, name))
    n, h, d = shape
    st, sh, sd = t.stride()
    if sd == 1 and n > 1 and sh >= d and st >= h * sh:
        return t.data_ptr(), st, sh   # the usual order
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: heads not contiguous")
    if h <= 1:
        sh = d
    if n <= 1:
        st = max(h * sh, d)
    # either the heads of a token lie within its stride, or tokens within a head's
    if n * h > 0 and (sh < d or st < d or (st < (h - 1) * sh + d and sh < (n - 1) * st + d)):
        raise ValueError(f"{name}: tokens or heads overlap (strides {st}, {sh} of {d} elements)")
    return t.data_ptr() or None, st, sh


_NO_HEADS = Heads()


def _kind_of_heads(call, name, x, weight, out, dout, dweight, dtype, n, d, grad):
    """The z1_heads of queries or keys."""
    shaped = x if x is not None else out
    if shaped is None:
        return _NO_HEADS
    if not isinstance(shaped, torch.Tensor) or shaped.dim() != 3:
        raise ValueError(f"{name}: expected a 3-D torch tensor (tokens, heads, dim)")
    shape = (n, shaped.shape[1], d)
    px = sx = hx = pd = sd = hd = None
    if x is not None:
        px, sx, hx = _heads_of(call, x, name, dtype, shape)
    po, so, ho = _heads_of(call, out, "d" + name if grad else name + "_out", dtype, shape)
    if grad:
        pd, sd, hd = _heads_of(call, dout, f"d{name}_out", dtype, shape)
    return Heads(shape[1], px, po, pd, call.vector(weight, name + "_weight", dtype, d),
                 call.vector(dweight, f"d{name}_weight", torch.float32, d), sx or 0, hx or 0, so, ho, sd or 0, hd or 0)


def _qk_args(q, k, positions, inv_freq, weights, eps, interleaved, outs, douts=(None, None), dweights=(None, None),
             accumulate=False, grad=False):
    lead = next((t for t in (q, k) + outs + douts if t is not None), None)
    dt = _dtype_of(lead, "q")
    if lead.dim() != 3:
        raise ValueError(f"q: {lead.dim()} dimensions, expected 3 (tokens, heads, dim)")
    call, kind = _Call(lead), lead.dtype
    n, _, d = lead.shape
    it = _itype_of(positions, "positions")
    if positions.shape != (n,):
        raise ValueError(f"positions: shape {tuple(positions.shape)}, expected ({n},)")
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq: expected a 1-D torch tensor")
    n_freq = inv_freq.numel()
    a = QkArgs(n, d, n_freq,
               _kind_of_heads(call, "q", q, weights[0], outs[0], douts[0], dweights[0], kind, n, d, grad),
               _kind_of_heads(call, "k", k, weights[1], outs[1], douts[1], dweights[1], kind, n, d, grad),
               call.vector(positions, "positions", positions.dtype, n), call.vector(inv_freq, "inv_freq", torch.float64, n_freq),
               eps, it, dt, 1 if interleaved else 0, 1 if accumulate else 0)
    return call, a


def z1_qk_norm_rope(q, k, q_out, k_out, positions, inv_freq, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                    interleaved: bool = False, stream=None) -> None:
    """The root-mean-square norm of every head of q and k [tokens, heads, dim]
    times q_weight / k_weight [dim] (None: no norm), and the rotation of its first
    2 * len(inv_freq) elements by the angles positions[t] * inv_freq (fp64), into
    q_out and k_out (which may be q and k).  Pairs are halves of the rotated part,
    or neighbours with interleaved.  k and k_out may be None."""
    call, a = _qk_args(q, k, positions, inv_freq, (q_weight, k_weight), eps, interleaved, (q_out, k_out))
    call.done()
    _check(lib.z1_qk_norm_rope(ctypes.byref(a), _stream(stream)), "z1_qk_norm_rope")


def z1_qk_norm_rope_grad_workspace(tokens: int, q_heads: int, k_heads: int, dim: int) -> int:
    """Bytes of device workspace z1_qk_norm_rope_grad needs for the weights' gradients."""
    b = _I64()
    _check(lib.z1_qk_norm_rope_grad_workspace(int(tokens), int(q_heads), int(k_heads), int(dim), ctypes.byref(b)),
           "z1_qk_norm_rope_grad_workspace")
    return b.value


def z1_qk_norm_rope_grad(q, k, dq_out, dk_out, dq, dk, positions, inv_freq, *, q_weight=None, k_weight=None,
                         dq_weight=None, dk_weight=None, eps: float = 1e-6, interleaved: bool = False,
                         accumulate: bool = False, workspace=None, stream=None) -> None:
    """dq and dk from the gradients dq_out and dk_out of z1_qk_norm_rope's
    outputs, and dq_weight / dk_weight [dim] fp32 (+)= those of the weights (None:
    not wanted; two buffers, also for a weight that both share).  q, k are the
    forward's inputs (None where there is no norm); dq may be dq_out, dk dk_out."""
    call, a = _qk_args(q, k, positions, inv_freq, (q_weight, k_weight), eps, interleaved, (dq, dk), (dq_out, dk_out),
                       (dq_weight, dk_weight), accumulate, True)
    work, size = call.workspace(workspace)
    call.done()
    _check(lib.z1_qk_norm_rope_grad(ctypes.byref(a), work, size, _stream(stream)), "z1_qk_norm_rope_grad")
