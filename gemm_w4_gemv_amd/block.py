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


def _rows(t, name, dtype, device, shape):
    """A tensor [rows, values] whose rows lie at any stride: (address, stride); None: (None, 0)."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a tensor [rows, values]")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}; got {list(t.shape)}")
    if t.dtype is not dtype or t.get_device() != device:
        _refuse(t, name, dtype, device)
    step, unit = t.stride()
    if shape[0] > 0 and shape[1] > 1 and unit != 1:
        raise ValueError(f"{name}: the values of a row must lie together")
    # one row or none: whatever stride it has is not used
    return t.data_ptr(), step if shape[0] > 1 else max(shape[1], 8)


def _space(workspace, device):
    if workspace is None:
        return None, 0
    return _ptr(workspace, "workspace", workspace.dtype, device), workspace.numel() * workspace.element_size()


def _sized(t, name, dims):
    """Sizes of a tensor, each within 32 bits."""
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{name} must be a tensor of {dims} dimensions")
    if t.numel() and max(t.shape) > _INT_MAX:
        _too_large(name, max(t.shape))
    return t.shape


def _norm_args(h, y, y_weight, z_weight, gate, residual_scale, branch_scale, eps, weight_add):
    """(struct without outputs, device, shape, h's dtype) of a norm's inputs."""
    shape = T, D = _sized(h, "h", 2)
    kind = h.dtype
    if kind is not _bf16 and kind is not _f32:
        raise TypeError(f"h: dtype {kind}, not torch.bfloat16 or torch.float32")
    i = _device_of(h, "h", kind)
    hp, hs = _rows(h, "h", kind, i, shape)
    yp, ys = _rows(y, "y", _bf16, i, shape)
    if gate is None or gate.dim() == 1:
        gs = 0
        wy, wz, gp = _optional_addresses(i, y_weight, "y_weight", _bf16, D, z_weight, "z_weight", _bf16, D,
                                         gate, "gate", _bf16, D)
    else:
        gp, gs = _rows(gate, "gate", _bf16, i, shape)
        if gs == 0:
            raise ValueError("gate: one for all tokens is [D]")
        wy, wz = _optional_addresses(i, y_weight, "y_weight", _bf16, D, z_weight, "z_weight", _bf16, D)
    a = _NormArgs(h=hp, y=yp, y_weight=wy, z_weight=wz, gate=gp, h_stride=hs, y_stride=ys, gate_stride=gs, T=T, D=D,
                  h_f32=kind is _f32, residual_scale=residual_scale, branch_scale=branch_scale, eps=eps,
                  weight_add=weight_add)
    return a, i, shape, kind


def w4_block_norm(h, y=None, h_out=None, z=None, y_weight=None, z_weight=None, gate=None, residual_scale: float = 1.0,
                  branch_scale: float = 1.0, eps: float = 1e-6, weight_add: float = 0.0, stream=None) -> None:
    """``h_out = residual_scale * h + branch_scale * gate * norm(y) * y_weight`` and ``z = norm(h_out) * z_weight``,
    where norm(x) = x / sqrt(mean(x^2) + eps) and ``weight_add`` is added to each weight.

    ``h``, ``h_out`` [T, D] bfloat16 or float32 (``h_out`` may be ``h``), ``y``, ``z`` bfloat16 [T, D] (``z`` may be
    ``y``), weights bfloat16 [D] (None: no norm), ``gate`` bfloat16 [D] or [T, D].  Without ``y`` only ``z`` of ``h``."""
    a, i, shape, kind = _norm_args(h, y, y_weight, z_weight, gate, residual_scale, branch_scale, eps, weight_add)
    a.h_out, a.h_out_stride = _rows(h_out, "h_out", kind, i, shape)
    a.z, a.z_stride = _rows(z, "z", _bf16, i, shape)
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
    a, i, shape, kind = _norm_args(h, y, y_weight, z_weight, gate, residual_scale, branch_scale, eps, weight_add)
    g = _NormGradArgs()
    g.dh_out, g.dh_out_stride = _rows(dh_out, "dh_out", kind, i, shape)
    g.dz, g.dz_stride = _rows(dz, "dz", _bf16, i, shape)
    g.dh, g.dh_stride = _rows(dh, "dh", kind, i, shape)
    g.dy, g.dy_stride = _rows(dy, "dy", _bf16, i, shape)
    g.d_y_weight, g.d_z_weight = _optional_addresses(i, d_y_weight, "d_y_weight", _f32, shape[1],
                                                     d_z_weight, "d_z_weight", _f32, shape[1])
    if gate is not None and gate.dim() == 2:
        g.d_gate, g.d_gate_stride = _rows(d_gate, "d_gate", _bf16, i, shape)
    else:
        g.d_gate, = _optional_addresses(i, d_gate, "d_gate", _f32, shape[1])
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
    T, top = _sized(experts, "experts", 2)
    i = _device_of(experts, "experts", _int32)
    if not -1 <= num_experts <= _INT_MAX:
        _too_large("w4_moe_sort", num_experts)
    v = _int32
    ep, rs = _addresses(i, experts, "experts", v, None, row_start, "row_start", v, max(num_experts, 0) + 1)
    if not isinstance(row_of, torch.Tensor) or row_of.shape != experts.shape:
        raise ValueError(f"row_of must be {[T, top]}")
    ro, so = _optional_addresses(i, row_of, "row_of", v, None, source, "source", v, T * top)
    a = _SortArgs(experts=ep, row_start=rs, row_of=ro, source=so, T=T, top=top, num_experts=num_experts,
                  capacity=_near(capacity))
    if x is not None or rows is not None:
        if x is None or rows is None:
            raise ValueError("x and rows go together")
        D = _sized(x, "x", 2)[1]
        R = _sized(rows, "rows", 2)[0]
        a.x, a.x_stride = _rows(x, "x", _bf16, i, (T, D))
        a.rows, a.rows_stride = _rows(rows, "rows", _bf16, i, (R, D))
        a.R, a.D = R, D
    pw, nbytes = _space(workspace, i)
    _call("w4_moe_sort", lib.w4_moe_sort, (ctypes.byref(a), pw, nbytes), stream, i)


def _choices(row_of, weights, T, R, device):
    """(choices a token, row_of's address, weights' address)."""
    given = row_of if row_of is not None else weights
    if given is None:
        if T == 0 or R % T:
            raise ValueError(f"without row_of and weights, {R} rows must be as many for each of {T} tokens")
        top = R // T
    else:
        if not isinstance(given, torch.Tensor) or given.dim() != 2 or given.shape[0] != T:
            raise ValueError(f"row_of and weights must be [{T}, top]")
        top = given.shape[1]
    for name, t in (("row_of", row_of), ("weights", weights)):
        if t is not None and t.shape != (T, top):
            raise ValueError(f"{name} must be {[T, top]}; got {list(t.shape)}")
    return (top, *_optional_addresses(device, row_of, "row_of", _int32, None, weights, "weights", _f32, None))


def w4_moe_combine(y, out, row_of=None, weights=None, add=None, stream=None) -> torch.Tensor:
    """``out[t] = add[t] + sum_j weights[t, j] * y[row_of[t, j]]`` for bfloat16 ``y`` [R, N] and ``out`` [T, N].

    ``row_of`` int32 [T, top] (``w4_moe_sort``'s; None: row t * top + j), ``weights`` float32 [T, top] (None: 1),
    ``add`` bfloat16 [T, N] (None: 0; may be ``out``).  A row outside ``y`` counts for nothing."""
    R, N = _sized(y, "y", 2)
    T = _sized(out, "out", 2)[0]
    i = _device_of(out, "out", _bf16)
    a = _CombineArgs(T=T, R=R, N=N)
    a.top, a.row_of, a.weights = _choices(row_of, weights, T, R, i)
    a.y, a.y_stride = _rows(y, "y", _bf16, i, (R, N))
    a.add, a.add_stride = _rows(add, "add", _bf16, i, (T, N))
    a.out, a.out_stride = _rows(out, "out", _bf16, i, (T, N))
    _call("w4_moe_combine", lib.w4_moe_combine, (ctypes.byref(a),), stream, i)
    return out


def w4_moe_combine_grad(dout, y=None, row_of=None, weights=None, dy=None, dweights=None, stream=None) -> None:
    """Gradients of ``w4_moe_combine``'s rows and weights: ``dy[row_of[t, j]] = weights[t, j] * dout[t]`` (``dy`` may
    be ``y``; rows that no choice has are left) and ``dweights[t, j] = dout[t] . y[row_of[t, j]]`` (0 without a row)."""
    T, N = _sized(dout, "dout", 2)
    given = y if y is not None else dy
    if given is None:
        raise ValueError("y or dy must be given")
    R = _sized(given, "y" if y is not None else "dy", 2)[0]
    i = _device_of(dout, "dout", _bf16)
    a = _CombineGradArgs(T=T, R=R, N=N)
    a.top, a.row_of, a.weights = _choices(row_of, weights, T, R, i)
    a.dout, a.dout_stride = _rows(dout, "dout", _bf16, i, (T, N))
    a.y, a.y_stride = _rows(y, "y", _bf16, i, (R, N))
    a.dy, a.dy_stride = _rows(dy, "dy", _bf16, i, (R, N))
    if dweights is not None:
        if dweights.shape != (T, a.top):
            raise ValueError(f"dweights must be {[T, a.top]}; got {list(dweights.shape)}")
        a.dweights, = _addresses(i, dweights, "dweights", _f32, None)
    _call("w4_moe_combine_grad", lib.w4_moe_combine_grad, (ctypes.byref(a),), stream, i)
