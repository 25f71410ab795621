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

from .binding import LIB_PATH, _check, _dptr, lib
from .ops import DTYPES, _checked, _dtype_of, _itype_of, _rows_of, _stream

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


def _drop_of(d: Optional[Dropout], items: list) -> Drop:
    if d is None:
        return Drop(None, 0, 0.0)
    if not isinstance(d.rng, torch.Tensor) or d.rng.dtype not in (torch.int64, torch.uint64):
        raise TypeError("dropout.rng: expected a torch tensor of int64 or uint64")
    items.append((d.rng, "dropout.rng", d.rng.dtype, 2))
    return Drop(d.rng.data_ptr(), int(d.offset) & 0xffffffffffffffff, float(d.p))


def _bytes_of(workspace) -> int:
    if workspace is None:
        return 0
    if not isinstance(workspace, torch.Tensor):
        raise TypeError(f"workspace: expected a torch tensor, got {type(workspace).__name__}")
    return workspace.numel() * workspace.element_size()


def _matrix(t, name: str, rows: list, dtype=None, shape=None):
    """(address, distance of rows) of a matrix or (None, 0)."""
    if t is None:
        return None, 0
    ld = _rows_of(t, name, dtype, shape)
    rows.append((t, name))
    return t.data_ptr(), ld


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
    items, rows = [], []
    px, ld_x = _matrix(x, "x", rows)
    py, ld_y = _matrix(y, "y", rows, x.dtype, x.shape)
    pr, ld_r = _matrix(residual, "residual", rows, x.dtype, x.shape)
    drop = _drop_of(dropout, items)
    _checked(items, rows)
    a = DropoutArgs(x.shape[0], x.shape[1], px, pr, py, ld_x, ld_r, ld_y, drop, dt, 0)
    _check(lib.z1_dropout(ctypes.byref(a), _stream(stream)), "z1_dropout")


# --------------------------------------------------------------------------
# linear
# --------------------------------------------------------------------------

def _linear_args(x, weight, rows: list) -> LinearArgs:
    dt = _dtype_of(x, "x")
    px, ld_x = _matrix(x, "x", rows)
    pw, ld_w = _matrix(weight, "weight", rows, x.dtype)
    if weight.shape[1] != x.shape[1]:
        raise ValueError(f"weight: {weight.shape[1]} columns, x has {x.shape[1]}")
    return LinearArgs(rows=x.shape[0], in_=x.shape[1], out=weight.shape[0], x=px, weight=pw, ld_x=ld_x, ld_weight=ld_w,
                      dtype=dt)


def z1_linear_workspace(x, weight) -> int:
    """Bytes of device workspace z1_linear needs for these operands."""
    b = _I64()
    _check(lib.z1_linear_workspace(ctypes.byref(_linear_args(x, weight, [])), ctypes.byref(b)), "z1_linear_workspace")
    return b.value


def z1_linear(x, weight, y, *, bias=None, act: str = "none", mul=None, residual=None, pre=None,
              dropout: Optional[Dropout] = None, workspace=None, stream=None) -> None:
    """y = residual + drop(act(x weight^T + bias) * mul) and pre = x weight^T +
    bias, for x [rows, in], weight [out, in], bias [out] and the others [rows,
    out], all of one type; None leaves a term out.  y may be residual or mul."""
    items, rows = [], []
    a = _linear_args(x, weight, rows)
    shape = (a.rows, a.out)
    a.y, a.ld_y = _matrix(y, "y", rows, x.dtype, shape)
    a.mul, a.ld_mul = _matrix(mul, "mul", rows, x.dtype, shape)
    a.residual, a.ld_residual = _matrix(residual, "residual", rows, x.dtype, shape)
    a.pre, a.ld_pre = _matrix(pre, "pre", rows, x.dtype, shape)
    a.act = _act_of(act)
    if bias is not None:
        items.append((bias, "bias", x.dtype, a.out))
        a.bias = _dptr(bias)
    if dropout is not None:
        a.drop = _drop_of(dropout, items)
    n = _bytes_of(workspace)
    if n:
        items.append((workspace, "workspace", None, 0))
    _checked(items, rows)
    _check(lib.z1_linear(ctypes.byref(a), _dptr(workspace) if n else None, n, _stream(stream)), "z1_linear")


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
    items, rows = [], []
    a = LinearDzArgs(dtype=dt, act=_act_of(act), accumulate=int(bool(accumulate)))
    a.dy, a.ld_dy = _matrix(dy, "dy", rows)
    a.rows, a.out = dy.shape
    for name, t in (("pre", pre), ("mul", mul), ("dz", dz), ("dmul", dmul)):
        p, ld = _matrix(t, name, rows, dy.dtype, dy.shape)
        setattr(a, name, p)
        setattr(a, "ld_" + name, ld)
    if dbias is not None:
        items.append((dbias, "dbias", torch.float32, a.out))
        a.dbias = _dptr(dbias)
    if dropout is not None:
        a.drop = _drop_of(dropout, items)
    n = _bytes_of(workspace)
    if n:
        items.append((workspace, "workspace", None, 0))
    _checked(items, rows)
    _check(lib.z1_linear_dz(ctypes.byref(a), _dptr(workspace) if n else None, n, _stream(stream)), "z1_linear_dz")


def _linear_grad_args(dz, x, weight, dx, dweight, rows: list) -> LinearGradArgs:
    a = LinearGradArgs(dtype=_dtype_of(dz, "dz"))
    a.dz, a.ld_dz = _matrix(dz, "dz", rows)
    n, out = dz.shape
    known = x if x is not None else weight
    if known is None:
        raise ValueError("x and weight: both None")
    _dtype_of(known, "x" if x is not None else "weight")
    cols = known.shape[-1]
    a.x, a.ld_x = _matrix(x, "x", rows, dz.dtype, (n, cols))
    a.weight, a.ld_weight = _matrix(weight, "weight", rows, dz.dtype, (out, cols))
    a.rows, a.in_, a.out = n, cols, out
    a.dx, a.ld_dx = _matrix(dx, "dx", rows, dz.dtype, (n, cols))
    if dweight is not None:
        a.dweight, a.ld_dweight = _matrix(dweight, "dweight", rows, None, (out, cols))
        if dweight.dtype != torch.float32 and dweight.dtype != dz.dtype:
            raise TypeError(f"dweight: dtype {dweight.dtype}, expected float32 or {dz.dtype}")
        a.dweight_dtype = DTYPES[dweight.dtype]
    return a


def z1_linear_grad_workspace(dz, x, weight) -> int:
    """Bytes of device workspace z1_linear_grad needs for these operands, for
    either gradient or both."""
    a = _linear_grad_args(dz, x, weight, None, None, [])
    # the outputs are not looked at, but for being there
    a.dx = a.weight
    a.dweight = a.x
    b = _I64()
    _check(lib.z1_linear_grad_workspace(ctypes.byref(a), ctypes.byref(b)), "z1_linear_grad_workspace")
    return b.value


def z1_linear_grad(dz, x, weight, *, dx=None, add=None, dweight=None, accumulate: bool = False, workspace=None,
                   stream=None) -> None:
    """dx = dz weight (+ add) and dweight (+)= dz^T x, for dz [rows, out], x
    [rows, in] (None without dweight) and weight [out, in] (None without dx).
    dweight: fp32, written or with accumulate added to (for example a view of the
    step's acc arena), or of dz's type and written.  dx may be add."""
    rows = []
    a = _linear_grad_args(dz, x, weight, dx, dweight, rows)
    if dx is None and dweight is None:
        raise ValueError("dx and dweight: both None")
    a.add, a.ld_add = _matrix(add, "add", rows, dz.dtype, (a.rows, a.in_))
    a.accumulate = int(bool(accumulate))
    n = _bytes_of(workspace)
    _checked([(workspace, "workspace", None, 0)] if n else [], rows)
    _check(lib.z1_linear_grad(ctypes.byref(a), _dptr(workspace) if n else None, n, _stream(stream)), "z1_linear_grad")


# --------------------------------------------------------------------------
# queries and keys
# --------------------------------------------------------------------------

def _heads_of(t, name: str, dtype, shape, rows: list):
    """(address, token stride, head stride) of [tokens, heads, dim] whose heads
    are contiguous and do not overlap; the addresses of no elements are null."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    n, h, d = shape
    rows.append((t, name))
    st, sh, sd = t.stride()
    if d > 1 and sd != 1:
        raise ValueError(f"{name}: heads not contiguous")
    sh = sh if h > 1 else d
    st = st if n > 1 else max(h * sh, d)
    # either the heads of a token lie within its stride, or tokens within a head's
    if n * h > 0 and (sh < d or st < d or (st < (h - 1) * sh + d and sh < (n - 1) * st + d)):
        raise ValueError(f"{name}: tokens or heads overlap (strides {st}, {sh} of {d} elements)")
    return t.data_ptr() or None, st, sh


def _qk_args(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, items, rows, outs, douts):
    lead = q if q is not None else k
    if lead is None:
        lead = next((t for t in outs + (douts or ()) if t is not None), None)
    dt = _dtype_of(lead, "q")
    if lead.dim() != 3:
        raise ValueError(f"q: {lead.dim()} dimensions, expected 3 (tokens, heads, dim)")
    n, _, d = lead.shape
    a = QkArgs(tokens=n, dim=d, eps=float(eps), dtype=dt, interleaved=int(bool(interleaved)))
    a.position_type = _itype_of(positions, "positions")
    if positions.shape != (n,):
        raise ValueError(f"positions: shape {tuple(positions.shape)}, expected ({n},)")
    items.append((positions, "positions", positions.dtype, n))
    a.positions = positions.data_ptr()
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq: expected a 1-D torch tensor")
    a.n_freq = inv_freq.numel()
    items.append((inv_freq, "inv_freq", torch.float64, a.n_freq))
    a.inv_freq = inv_freq.data_ptr()
    for i, (name, x, weight, heads) in enumerate((("q", q, q_weight, a.q), ("k", k, k_weight, a.k))):
        shaped = x if x is not None else outs[i]
        if shaped is None:
            continue
        if not isinstance(shaped, torch.Tensor) or shaped.dim() != 3:
            raise ValueError(f"{name}: expected a 3-D torch tensor (tokens, heads, dim)")
        shape = (n, shaped.shape[1], d)
        heads.heads = shape[1]
        if x is not None:
            heads.x, heads.x_token, heads.x_head = _heads_of(x, name, lead.dtype, shape, rows)
        out = "d" + name if douts else name + "_out"
        heads.out, heads.out_token, heads.out_head = _heads_of(outs[i], out, lead.dtype, shape, rows)
        if douts:
            heads.dout, heads.dout_token, heads.dout_head = _heads_of(douts[i], f"d{name}_out", lead.dtype, shape, rows)
        if weight is not None:
            items.append((weight, name + "_weight", lead.dtype, d))
            heads.weight = _dptr(weight)
    return a


def z1_qk_norm_rope(q, k, q_out, k_out, positions, inv_freq, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                    interleaved: bool = False, stream=None) -> None:
    """The root-mean-square norm of every head of q and k [tokens, heads, dim]
    times q_weight / k_weight [dim] (None: no norm), and the rotation of its first
    2 * len(inv_freq) elements by the angles positions[t] * inv_freq (fp64), into
    q_out and k_out (which may be q and k).  Pairs are halves of the rotated part,
    or neighbours with interleaved.  k and k_out may be None."""
    items, rows = [], []
    a = _qk_args(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, items, rows, (q_out, k_out), None)
    _checked(items, rows)
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
    not wanted).  q, k are the forward's inputs (None where there is no norm);
    dq may be dq_out, dk dk_out."""
    items, rows = [], []
    a = _qk_args(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, items, rows, (dq, dk),
                 (dq_out, dk_out))
    for name, t, heads in (("dq_weight", dq_weight, a.q), ("dk_weight", dk_weight, a.k)):
        if t is not None:
            items.append((t, name, torch.float32, a.dim))
            heads.dweight = _dptr(t)
    a.accumulate = int(bool(accumulate))
    n = _bytes_of(workspace)
    if n:
        items.append((workspace, "workspace", None, 0))
    _checked(items, rows)
    _check(lib.z1_qk_norm_rope_grad(ctypes.byref(a), _dptr(workspace) if n else None, n, _stream(stream)),
           "z1_qk_norm_rope_grad")
