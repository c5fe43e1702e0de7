"""Binding of the operators around a block's products (``include/w4_block.h``):
the norms before and after a block with its gate and residual sum, the tokens
sorted by expert and brought back, and the gradients of these.

Argument marshalling only, as in the package's other functions.  Tensors of
one call must live on one device; the call runs there, on ``stream`` or the
device's current stream.  Outputs and workspaces belong to the caller.
"""
from __future__ import annotations

import ctypes

import torch

from . import lib
from . import step as _step
from .step import _addresses, _bf16, _call, _device_of, _f32, _INT_MAX, _int32, _near, _optional_addresses, _ptr, _refuse, \
    _too_large

__all__ = ["w4_block_norm", "w4_block_norm_grad", "w4_block_norm_grad_workspace_bytes", "w4_moe_sort",
           "w4_moe_sort_workspace_bytes", "w4_moe_combine", "w4_moe_combine_grad", "NORM_MAX_DIM", "MOE_MAX_TOP",
           "MOE_SORT_MAX_EXPERTS"]

NORM_MAX_DIM = 16384
MOE_MAX_TOP = 64
MOE_SORT_MAX_EXPERTS = 1024

_vp = ctypes.c_void_p
_i32 = ctypes.c_int
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_fl = ctypes.c_float


class _NormArgs(ctypes.Structure):
    """struct w4_norm_args (include/w4_block.h)."""
    _fields_ = [("h", _vp), ("y", _vp), ("h_out", _vp), ("z", _vp), ("y_weight", _vp), ("z_weight", _vp),
                ("gate", _vp), ("h_stride", _i64), ("y_stride", _i64), ("h_out_stride", _i64), ("z_stride", _i64),
                ("gate_stride", _i64), ("T", _i32), ("D", _i32), ("h_f32", _i32), ("residual_scale", _fl),
                ("branch_scale", _fl), ("eps", _fl), ("weight_add", _fl)]


class _NormGradArgs(ctypes.Structure):
    """struct w4_norm_grad_args (include/w4_block.h)."""
    _fields_ = [("dh_out", _vp), ("dz", _vp), ("dh", _vp), ("dy", _vp), ("dh_out_stride", _i64), ("dz_stride", _i64),
                ("dh_stride", _i64), ("dy_stride", _i64), ("d_gate_stride", _i64), ("d_y_weight", _vp),
                ("d_z_weight", _vp), ("d_gate", _vp)]


class _SortArgs(ctypes.Structure):
    """struct w4_moe_sort_args (include/w4_block.h)."""
    _fields_ = [("experts", _vp), ("row_start", _vp), ("row_of", _vp), ("source", _vp), ("x", _vp), ("rows", _vp),
                ("x_stride", _i64), ("rows_stride", _i64), ("T", _i32), ("top", _i32), ("num_experts", _i32),
                ("capacity", _i32), ("R", _i32), ("D", _i32)]


class _CombineArgs(ctypes.Structure):
    """struct w4_moe_combine_args (include/w4_block.h)."""
    _fields_ = [("y", _vp), ("row_of", _vp), ("weights", _vp), ("add", _vp), ("out", _vp), ("y_stride", _i64),
                ("add_stride", _i64), ("out_stride", _i64), ("T", _i32), ("top", _i32), ("R", _i32), ("N", _i32)]


class _CombineGradArgs(ctypes.Structure):
    """struct w4_moe_combine_grad_args (include/w4_block.h)."""
    _fields_ = [("dout", _vp), ("y", _vp), ("row_of", _vp), ("weights", _vp), ("dy", _vp), ("dweights", _vp),
                ("dout_stride", _i64), ("y_stride", _i64), ("dy_stride", _i64), ("T", _i32), ("top", _i32),
                ("R", _i32), ("N", _i32)]


# name -> (restype, argtypes), mirroring include/w4_block.h
SIGNATURES = {
    "w4_block_norm": (_i32, [ctypes.POINTER(_NormArgs), _vp]),
    "w4_block_norm_grad_workspace_bytes": (_sz, [_i32, _i32]),
    "w4_block_norm_grad": (_i32, [ctypes.POINTER(_NormArgs), ctypes.POINTER(_NormGradArgs), _vp, _sz, _vp]),
    "w4_moe_sort_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "w4_moe_sort": (_i32, [ctypes.POINTER(_SortArgs), _vp, _sz, _vp]),
    "w4_moe_combine": (_i32, [ctypes.POINTER(_CombineArgs), _vp]),
    "w4_moe_combine_grad": (_i32, [ctypes.POINTER(_CombineGradArgs), _vp]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args


def _rows(device, n, wide, *spec):
    """Address and row stride, one behind the other, of each of some tensors [n, wide], given as (tensor, name,
    dtype), whose rows lie at any stride; (None, 0) for None."""
    out = []
    for t, name, dtype in zip(spec[0::3], spec[1::3], spec[2::3]):
        if t is None:
            out += (None, 0)
            continue
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a tensor [rows, values]")
        if t.shape != (n, wide):
            raise ValueError(f"{name} must be {[n, wide]}; got {list(t.shape)}")
        if t.dtype is not dtype or t.get_device() != device:
            _refuse(t, name, dtype, device)
        step, unit = t.stride()
        if n > 0 and wide > 1 and unit != 1:
            raise ValueError(f"{name}: the values of a row must lie together")
        # one row or none: whatever stride it has is not used
        out += (t.data_ptr(), step if n > 1 else max(wide, 8))
    return tuple(out)


_rows_in_python = _rows
if _step._marshal is not None and _step._fits(_step._marshal):  # the same check compiled
    _step._marshal.begin_rows(_rows)
    _rows = _step._marshal.rows


def _space(workspace, device):
    if workspace is None:
        return None, 0
    return _ptr(workspace, "workspace", workspace.dtype, device), workspace.numel() * workspace.element_size()


def _matrix(t, name):
    """Sizes of a tensor of two dimensions, each within 32 bits."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a tensor of 2 dimensions")
    n, wide = t.shape
    if n > _INT_MAX or wide > _INT_MAX:
        _too_large(name, max(n, wide))
    return n, wide


def _stream_of(h):
    """(rows, values, dtype, device) of the residual stream."""
    T, D = _matrix(h, "h")
    kind = h.dtype
    if kind is not _bf16 and kind is not _f32:
        raise TypeError(f"h: dtype {kind}, not torch.bfloat16 or torch.float32")
    return T, D, kind, _device_of(h, "h", kind)


def _given(i, T, D, y_weight, z_weight, gate):
    """Addresses of the weights and the gate, the gate's row stride (0: one for all tokens)."""
    if not isinstance(gate, torch.Tensor) or gate.dim() == 1:
        return (*_optional_addresses(i, y_weight, "y_weight", _bf16, D, z_weight, "z_weight", _bf16, D, gate, "gate", _bf16, D), 0)
    gp, gs = _rows(i, T, D, gate, "gate", _bf16)
    if gs == 0:
        raise ValueError("gate: one for all tokens is [D]")
    return (*_optional_addresses(i, y_weight, "y_weight", _bf16, D, z_weight, "z_weight", _bf16, D), gp, gs)


def w4_block_norm(h, y=None, h_out=None, z=None, y_weight=None, z_weight=None, gate=None, residual_scale: float = 1.0,
                  branch_scale: float = 1.0, eps: float = 1e-6, weight_add: float = 0.0, stream=None) -> None:
    """``h_out = residual_scale * h + branch_scale * gate * norm(y) * y_weight`` and ``z = norm(h_out) * z_weight``,
    where norm(x) = x / sqrt(mean(x^2) + eps) and ``weight_add`` is added to each weight.

    ``h``, ``h_out`` [T, D] bfloat16 or float32 (``h_out`` may be ``h``), ``y``, ``z`` bfloat16 [T, D] (``z`` may be
    ``y``), weights bfloat16 [D] (None: no norm), ``gate`` bfloat16 [D] or [T, D].  Without ``y`` only ``z`` of ``h``."""
    T, D, kind, i = _stream_of(h)
    hp, hs, yp, ys, op, os, zp, zs = _rows(i, T, D, h, "h", kind, y, "y", _bf16, h_out, "h_out", kind, z, "z", _bf16)
    wy, wz, gp, gs = _given(i, T, D, y_weight, z_weight, gate)
    a = _NormArgs(hp, yp, op, zp, wy, wz, gp, hs, ys, os, zs, gs, T, D, kind is _f32, residual_scale, branch_scale, eps,
                  weight_add)
    _call("w4_block_norm", lib.w4_block_norm, (ctypes.byref(a),), stream, i)


def w4_block_norm_grad_workspace_bytes(T: int, D: int) -> int:
    return lib.w4_block_norm_grad_workspace_bytes(_near(T), _near(D))


def w4_block_norm_grad(h, y=None, dh_out=None, dz=None, dh=None, dy=None, y_weight=None, z_weight=None, gate=None,
                       d_y_weight=None, d_z_weight=None, d_gate=None, residual_scale: float = 1.0,
                       branch_scale: float = 1.0, eps: float = 1e-6, weight_add: float = 0.0, workspace=None,
                       stream=None) -> None:
    """Gradients of ``w4_block_norm``'s inputs (as they were before it) from ``dh_out`` and ``dz`` (either may be None).

    ``dh`` (may be ``dh_out``) has ``h``'s type, ``dy`` (may be ``dz``) is bfloat16, ``d_y_weight``, ``d_z_weight`` and a
    shared gate's ``d_gate`` are float32 [D], a gate of [T, D] has a bfloat16 ``d_gate`` of that shape; each may be None.
    ``workspace``: ``w4_block_norm_grad_workspace_bytes(T, D)``, for the sums over tokens."""
    T, D, kind, i = _stream_of(h)
    hp, hs, yp, ys, hop, hos, zp, zs, dhp, dhs, dyp, dys = _rows(
        i, T, D, h, "h", kind, y, "y", _bf16, dh_out, "dh_out", kind, dz, "dz", _bf16, dh, "dh", kind, dy, "dy", _bf16)
    wy, wz, gp, gs = _given(i, T, D, y_weight, z_weight, gate)
    sy, sz = _optional_addresses(i, d_y_weight, "d_y_weight", _f32, D, d_z_weight, "d_z_weight", _f32, D)
    if gs:
        dgp, dgs = _rows(i, T, D, d_gate, "d_gate", _bf16)
    else:
        (dgp,), dgs = _optional_addresses(i, d_gate, "d_gate", _f32, D), 0
    a = _NormArgs(hp, yp, None, None, wy, wz, gp, hs, ys, 0, 0, gs, T, D, kind is _f32, residual_scale, branch_scale, eps,
                  weight_add)
    g = _NormGradArgs(hop, zp, dhp, dyp, hos, zs, dhs, dys, dgs, sy, sz, dgp)
    pw, nbytes = _space(workspace, i)
    _call("w4_block_norm_grad", lib.w4_block_norm_grad, (ctypes.byref(a), ctypes.byref(g), pw, nbytes), stream, i)


def w4_moe_sort_workspace_bytes(T: int, top: int, num_experts: int) -> int:
    return lib.w4_moe_sort_workspace_bytes(_near(T), _near(top), _near(num_experts))


def w4_moe_sort(experts, num_experts: int, row_start, row_of, source=None, x=None, rows=None, capacity: int = 0,
                workspace=None, stream=None) -> None:
    """Where the choices ``experts`` (int32 [T, top]) go when sorted by expert, and the tokens there.

    Outputs, int32: ``row_start`` [num_experts + 1] (``w4_moe_gemm``'s, with expert ids 0, 1, ...), ``row_of`` [T, top]
    (-1: none), ``source`` [T * top] (the choice of each row, -1 behind the last; may be None).  With ``x`` bfloat16
    [T, D], ``rows`` [R, D] gets ``x[t]`` at each of token t's rows.  An expert takes its first ``capacity`` choices
    (0: all)."""
    T, top = _matrix(experts, "experts")
    i, v = _device_of(experts, "experts", _int32), _int32
    if not -1 <= num_experts <= _INT_MAX:
        _too_large("w4_moe_sort", num_experts)
    if not isinstance(row_of, torch.Tensor) or row_of.shape != experts.shape:
        raise ValueError(f"row_of must be {[T, top]}")
    ep, sp, rp = _addresses(i, experts, "experts", v, None, row_start, "row_start", v, max(num_experts, 0) + 1,
                            row_of, "row_of", v, None)
    so, = _optional_addresses(i, source, "source", v, T * top)
    R = D = xs = rs = 0
    xp = op = None
    if x is not None or rows is not None:
        if x is None or rows is None:
            raise ValueError("x and rows go together")
        (R, D), _ = _matrix(rows, "rows"), _matrix(x, "x")
        xp, xs = _rows(i, T, D, x, "x", _bf16)
        op, rs = _rows(i, R, D, rows, "rows", _bf16)
    a = _SortArgs(ep, sp, rp, so, xp, op, xs, rs, T, top, num_experts, _near(capacity), R, D)
    pw, nbytes = _space(workspace, i)
    _call("w4_moe_sort", lib.w4_moe_sort, (ctypes.byref(a), pw, nbytes), stream, i)


def _choices(row_of, weights, T, R, device):
    """(choices a token, row_of's address, weights' address)."""
    given = row_of if row_of is not None else weights
    if given is None:
        if R % T if T else R:
            raise ValueError(f"without row_of and weights, {R} rows must be as many for each of {T} tokens")
        top = R // T if T else 1
    else:
        if not isinstance(given, torch.Tensor) or given.dim() != 2 or given.shape[0] != T:
            raise ValueError(f"row_of and weights must be [{T}, top]")
        top = given.shape[1]
        for name, t in (("row_of", row_of), ("weights", weights)):
            if t is not None and t is not given and t.shape != (T, top):
                raise ValueError(f"{name} must be {[T, top]}; got {list(t.shape)}")
    return (top, *_optional_addresses(device, row_of, "row_of", _int32, None, weights, "weights", _f32, None))


def w4_moe_combine(y, out, row_of=None, weights=None, add=None, stream=None) -> torch.Tensor:
    """``out[t] = add[t] + sum_j weights[t, j] * y[row_of[t, j]]`` for bfloat16 ``y`` [R, N] and ``out`` [T, N].

    ``row_of`` int32 [T, top] (``w4_moe_sort``'s; None: row t * top + j), ``weights`` float32 [T, top] (None: 1),
    ``add`` bfloat16 [T, N] (None: 0; may be ``out``).  A row outside ``y`` counts for nothing."""
    (R, N), (T, _) = _matrix(y, "y"), _matrix(out, "out")
    i = _device_of(out, "out", _bf16)
    top, rp, wp = _choices(row_of, weights, T, R, i)
    yp, ys = _rows(i, R, N, y, "y", _bf16)
    ap, as_, op, os = _rows(i, T, N, add, "add", _bf16, out, "out", _bf16)
    a = _CombineArgs(yp, rp, wp, ap, op, ys, as_, os, T, top, R, N)
    _call("w4_moe_combine", lib.w4_moe_combine, (ctypes.byref(a),), stream, i)
    return out


def w4_moe_combine_grad(dout, y=None, row_of=None, weights=None, dy=None, dweights=None, stream=None) -> None:
    """Gradients of ``w4_moe_combine``'s rows and weights: ``dy[row_of[t, j]] = weights[t, j] * dout[t]`` (``dy`` may
    be ``y``; rows that no choice has are left) and ``dweights[t, j] = dout[t] . y[row_of[t, j]]`` (0 without a row)."""
    T, N = _matrix(dout, "dout")
    given = y if y is not None else dy
    if given is None:
        raise ValueError("y or dy must be given")
    R, _ = _matrix(given, "y" if y is not None else "dy")
    i = _device_of(dout, "dout", _bf16)
    top, rp, wp = _choices(row_of, weights, T, R, i)
    gp, gs = _rows(i, T, N, dout, "dout", _bf16)
    yp, ys, dp, ds = _rows(i, R, N, y, "y", _bf16, dy, "dy", _bf16)
    dw = None
    if dweights is not None:
        if not isinstance(dweights, torch.Tensor) or dweights.shape != (T, top):
            raise ValueError(f"dweights must be a tensor {[T, top]}")
        dw, = _addresses(i, dweights, "dweights", _f32, None)
    a = _CombineGradArgs(gp, yp, rp, wp, dp, dw, gs, ys, ds, T, top, R, N)
    _call("w4_moe_combine_grad", lib.w4_moe_combine_grad, (ctypes.byref(a),), stream, i)
