"""Binding of the decode step's operators (``include/w4_step.h``): the 4-bit
key/value cache, what fills it, the attention that reads it, the sampler.

Argument marshalling only, as in the package's other functions.  Tensors of
one call must live on one device; the call runs there, on ``stream`` or the
device's current stream.  Outputs and workspaces belong to the caller.
"""
from __future__ import annotations

import ctypes
import math
import sys

import torch

from . import _check, lib

__all__ = ["Kv4Cache", "w4_kv4_plan", "w4_qk_norm_rope", "w4_kv4_read", "w4_kv4_attn", "w4_kv4_attn_workspace_bytes",
           "w4_sample", "w4_sample_workspace_bytes", "KV4_GROUP", "KV4_PLAN_MAX_BATCH", "SAMPLE_MAX_VOCAB"]

KV4_GROUP = 128
KV4_PLAN_MAX_BATCH = 4096
SAMPLE_MAX_VOCAB = 1048576
_INT_MAX = 2 ** 31 - 1

_vp = ctypes.c_void_p
_i32 = ctypes.c_int
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t


class _CacheStruct(ctypes.Structure):
    """struct w4_kv4_cache (include/w4_step.h)."""
    _fields_ = [("k_codes", _vp), ("k_meta", _vp), ("v_codes", _vp), ("v_meta", _vp), ("num_blocks", _i32),
                ("block_size", _i32), ("kv_heads", _i32), ("head_dim", _i32)]


class _QkArgs(ctypes.Structure):
    """struct w4_qk_args (include/w4_step.h)."""
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("q_weight", _vp), ("k_weight", _vp), ("cos_sin", _vp), ("positions", _vp), ("slots", _vp),
                ("q_out", _vp), ("k_out", _vp), ("q_out_stride", _i64), ("k_out_stride", _i64), ("T", _i32),
                ("q_heads", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("rot_dim", _i32), ("max_pos", _i32),
                ("interleaved", _i32), ("eps", ctypes.c_float), ("weight_add", ctypes.c_float)]


class _AttnArgs(ctypes.Structure):
    """struct w4_attn_args (include/w4_step.h)."""
    _fields_ = [("q", _vp), ("out", _vp), ("q_stride", _i64), ("out_stride", _i64), ("block_table", _vp),
                ("kv_lens", _vp), ("q_start", _vp), ("T", _i32), ("B", _i32), ("q_heads", _i32), ("max_blocks", _i32),
                ("max_q", _i32), ("max_kv", _i32), ("window", _i32), ("sinks", _i32), ("scale", ctypes.c_float)]


_cache_p = ctypes.POINTER(_CacheStruct)
# name -> (restype, argtypes), mirroring include/w4_step.h
SIGNATURES = {
    "w4_kv4_plan": (_i32, [_vp] * 5 + [_i32] * 5 + [_vp] * 6),
    "w4_qk_norm_rope": (_i32, [ctypes.POINTER(_QkArgs), _cache_p, _vp]),
    "w4_kv4_read": (_i32, [_cache_p, _vp, _i32, _vp, _vp, _vp]),
    "w4_kv4_attn_workspace_bytes": (_sz, [ctypes.POINTER(_AttnArgs), _cache_p]),
    "w4_kv4_attn": (_i32, [ctypes.POINTER(_AttnArgs), _cache_p, _vp, _sz, _vp]),
    "w4_sample_workspace_bytes": (_sz, [_i32, _i32]),
    "w4_sample": (_i32, [_vp, _i64] + [_vp] * 6 + [_i32, _i32, _vp, _sz, _vp]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args


_bf16, _f16, _f32, _f64, _int32 = torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.int32

# The current stream's handle and the current device, without the Python
# objects around them: a small call costs about as much as its launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(t, name, dtype, device):
    """Raises what is wrong with a tensor that failed the quick test of ``_ptr``."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, not {dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} lies on {t.device}, other tensors of this call on cuda:{device}")


# ctypes cuts a number to 32 bits without a word.
def _too_large(where, size):
    raise ValueError(f"{where}: a size of {size} does not fit 32 bits")


def _near(value):
    """A bound of which any value past the largest means the same; one below 0 is refused by the library."""
    return value if -1 <= value <= _INT_MAX else max(min(value, _INT_MAX), -1)


def _device_of(t, name, dtype):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() < 0:
        _refuse(t, name, dtype, None)
    return t.get_device()


def _ptr(t, name, dtype, device):
    """Address of a contiguous tensor of ``dtype`` on GPU ``device``."""
    try:
        if t.dtype is dtype and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, device)


def _vector(t, name, dtype, device, n):
    """Address of a contiguous vector of n values."""
    try:
        if t.dtype is dtype and t.get_device() == device and t.shape == (n,) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, torch.Tensor) and tuple(t.shape) != (n,):
        raise ValueError(f"{name} must be [{n}]; got {list(t.shape)}")
    _refuse(t, name, dtype, device)


def _heads(t, name, device, rows=None, heads=None, dim=None):
    """[rows, heads, dim] BF16 whose heads lie together: (address, row stride)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a tensor [tokens, heads, head_dim]")
    n, h, d = t.shape
    if (rows is not None and n != rows) or (heads is not None and h != heads) or (dim is not None and d != dim):
        raise ValueError(f"{name} must be {[rows, heads, dim]}; got {[n, h, d]}")
    step, inner, unit = t.stride()
    if (d > 1 and unit != 1) or (h > 1 and inner != d):
        raise ValueError(f"{name}: the heads of a row must lie together")
    if n <= 1:  # one row or none: whatever stride it has is not used
        step = max(h * d, 8)
    if t.dtype is not _bf16 or t.get_device() != device:
        _refuse(t, name, _bf16, device)
    return t.data_ptr(), step


def _addresses(device, *spec):
    """Addresses of tensors, each given as (tensor, name, dtype, length; None: any contiguous tensor)."""
    return tuple(_ptr(t, name, dtype, device) if n is None else _vector(t, name, dtype, device, n)
                 for t, name, dtype, n in zip(spec[0::4], spec[1::4], spec[2::4], spec[3::4]))


def _optional_addresses(device, *spec):
    """The same; None where a tensor is None."""
    return tuple(None if t is None else _addresses(device, t, name, dtype, n)[0]
                 for t, name, dtype, n in zip(spec[0::4], spec[1::4], spec[2::4], spec[3::4]))


# The same checks compiled (csrc/marshal.cpp), for host time alone: where a
# tensor fails one, they call these, which say what is wrong.  They know how this
# torch lays out a tensor, so a module built for another one is not taken.
_in_python = (_addresses, _optional_addresses, _heads)


def _fits(module) -> bool:
    here = (f"{torch.version.__version__} {torch.version.git_version}", sys.hexversion >> 16)
    return getattr(module, "built_for", None) == here


try:
    from . import _marshal
except ImportError:  # not built, or for another torch
    _marshal = None
if _marshal is not None and _fits(_marshal):
    _marshal.begin(*_in_python)
    _addresses, _optional_addresses, _heads = _marshal.addresses, _marshal.optional_addresses, _marshal.heads


def _call(where, fn, args, stream, device):
    """fn(*args, stream) on GPU ``device``."""
    if device != _current_device():
        with torch.cuda.device(device):
            return _call(where, fn, args, stream, device)
    if stream is None:
        stream = _raw_stream(device)
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device.index != device:
            raise ValueError(f"{where}: stream of {stream.device}, tensors on cuda:{device}")
        stream = stream.cuda_stream
    status = fn(*args, int(stream))
    if status:
        _check(status, where)


def _cache_ref(cache, device):
    if not isinstance(cache, Kv4Cache):
        raise TypeError("cache must be a Kv4Cache")
    if cache.device_index != device:
        raise ValueError(f"the cache lies on cuda:{cache.device_index}, other tensors of this call on cuda:{device}")
    return cache.ref


class Kv4Cache:
    """The paged 4-bit key/value cache: four tensors in the layout of ``w4_kv4_cache``.

    ``Kv4Cache.empty(...)`` allocates one; the constructor takes tensors that
    exist.  Unwritten slots hold no meaning and are never read by attention."""

    def __init__(self, k_codes, k_meta, v_codes, v_meta):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be int32 [num_blocks, kv_heads, block_size, head_dim / 8]")
        nb, h, bs, words = k_codes.shape
        d = 8 * words
        groups = max(1, d // KV4_GROUP)
        for name, t, shape in (("v_codes", v_codes, (nb, h, bs // 4, words, 4)),
                               ("k_meta", k_meta, (nb, h, groups, bs, 2)), ("v_meta", v_meta, (nb, h, groups, bs, 2))):
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {shape}; got {tuple(t.shape)}")
        i = _device_of(k_codes, "k_codes", _int32)
        self.k_codes, self.k_meta, self.v_codes, self.v_meta = k_codes, k_meta, v_codes, v_meta
        self.num_blocks, self.kv_heads, self.block_size, self.head_dim = nb, h, bs, d
        self.device_index = i
        self.struct = _CacheStruct(_ptr(k_codes, "k_codes", _int32, i), _ptr(k_meta, "k_meta", _f16, i),
                                   _ptr(v_codes, "v_codes", _int32, i), _ptr(v_meta, "v_meta", _f16, i), nb, bs, h, d)
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, num_blocks: int, block_size: int, kv_heads: int, head_dim: int, device="cuda") -> "Kv4Cache":
        groups = max(1, head_dim // KV4_GROUP)
        codes = dict(dtype=torch.int32, device=device)
        meta = dict(dtype=torch.float16, device=device)
        return cls(torch.empty(num_blocks, kv_heads, block_size, head_dim // 8, **codes),
                   torch.empty(num_blocks, kv_heads, groups, block_size, 2, **meta),
                   torch.empty(num_blocks, kv_heads, block_size // 4, head_dim // 8, 4, **codes),
                   torch.empty(num_blocks, kv_heads, groups, block_size, 2, **meta))


def w4_kv4_plan(cached, new_tokens, block_table, free_blocks, free_count, block_size: int, q_start, kv_lens,
                positions, slots, counts, stream=None) -> None:
    """Block tables, slot map, positions and row ranges of a step from the requests' lengths.

    ``cached``, ``new_tokens`` int32 [B]; ``block_table`` int32 [B, max_blocks] (new
    pages' entries are written); ``free_blocks`` int32 [n], ``free_count`` int32 [1].
    Outputs: ``q_start`` [B + 1], ``kv_lens`` [B], ``positions`` and ``slots`` [rows] (-1
    behind the last request), ``counts`` [2] (pages left, pages short)."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    B, width = block_table.shape
    rows, pages = positions.numel(), free_blocks.numel()
    if max(B, width, rows, pages, abs(block_size)) > _INT_MAX:
        _too_large("w4_kv4_plan", max(B, width, rows, pages, abs(block_size)))
    i, v = _device_of(block_table, "block_table", _int32), _int32
    p = _addresses(i, cached, "cached", v, B, new_tokens, "new_tokens", v, B, block_table, "block_table", v, None,
                   free_blocks, "free_blocks", v, pages, free_count, "free_count", v, 1, q_start, "q_start", v, B + 1,
                   kv_lens, "kv_lens", v, B, positions, "positions", v, rows, slots, "slots", v, rows,
                   counts, "counts", v, 2)
    _call("w4_kv4_plan", lib.w4_kv4_plan, (*p[:5], B, width, pages, block_size, rows, *p[5:]), stream, i)


def w4_qk_norm_rope(q, k, positions=None, cos_sin=None, q_out=None, k_out=None, q_weight=None, k_weight=None,
                    eps: float = 1e-6, weight_add: float = 0.0, interleaved: bool = False, v=None, cache=None,
                    slots=None, stream=None) -> None:
    """RMS norm of each query and key head, rotation by position, and with ``cache`` the keys and
    ``v`` quantised into their ``slots``.

    ``q`` [T, q_heads, head_dim] (None: keys only), ``k``, ``v`` [T, kv_heads, head_dim], BF16, rows at
    any stride; ``cos_sin`` float [max_pos, rot_dim] (cosines, then sines; None: no rotation).
    ``q_out`` and ``k_out`` may be ``q`` and ``k`` themselves; ``k_out`` may be None with a cache."""
    i = _device_of(k, "k", _bf16)
    kp, ks = _heads(k, "k", i)
    T, kv_heads, dim = k.shape
    qp = qs = vp = vs = qop = qos = kop = kos = 0
    q_heads = reach = rot = 0
    sp = ref = None
    if q is not None:
        qp, qs = _heads(q, "q", i, T, None, dim)
        q_heads = q.shape[1]
        if q_out is None:
            raise ValueError("q_out must be given with q")
        qop, qos = _heads(q_out, "q_out", i, T, q_heads, dim)
    if k_out is not None:
        kop, kos = _heads(k_out, "k_out", i, T, kv_heads, dim)
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_pos, rot_dim]")
        reach, rot = cos_sin.shape
    qw, kw, cs, pos = _optional_addresses(i, q_weight, "q_weight", _bf16, dim, k_weight, "k_weight", _bf16, dim,
                                          cos_sin, "cos_sin", _f32, None, positions, "positions", _int32, T)
    if cache is not None:
        if v is None or slots is None:
            raise ValueError("v and slots must be given with a cache")
        vp, vs = _heads(v, "v", i, T, kv_heads, dim)
        sp, = _addresses(i, slots, "slots", _int32, T)
        ref = _cache_ref(cache, i)
    a = _QkArgs(qp, kp, vp, qs, ks, vs, qw, kw, cs, pos, sp, qop, kop, qos, kos, T, q_heads, kv_heads, dim, rot, reach,
                1 if interleaved else 0, eps, weight_add)
    _call("w4_qk_norm_rope", lib.w4_qk_norm_rope, (ctypes.byref(a), ref), stream, i)


def w4_kv4_read(cache, slots, k_out=None, v_out=None, stream=None) -> None:
    """The keys and values that ``slots`` of the cache stand for, in BF16 [n, kv_heads, head_dim]."""
    if not isinstance(cache, Kv4Cache):
        raise TypeError("cache must be a Kv4Cache")
    i, n = cache.device_index, slots.numel()
    shape = (n, cache.kv_heads, cache.head_dim)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None and t.shape != shape:
            raise ValueError(f"{name} must be {shape}; got {tuple(t.shape)}")
    sp, kp, vp = _optional_addresses(i, slots, "slots", _int32, n, k_out, "k_out", _bf16, None, v_out, "v_out", _bf16, None)
    _call("w4_kv4_read", lib.w4_kv4_read, (cache.ref, sp, n, kp, vp), stream, i)


def w4_kv4_attn_workspace_bytes(cache, T: int, B: int, q_heads: int, max_q: int, max_kv: int, window: int = 0,
                                sinks: int = 0) -> int:
    a = _AttnArgs(T=_near(T), B=_near(B), q_heads=_near(q_heads), max_q=_near(max_q), max_kv=_near(max_kv),
                  window=_near(window), sinks=_near(sinks))
    return lib.w4_kv4_attn_workspace_bytes(ctypes.byref(a), cache.ref)


def w4_kv4_attn(q, cache, block_table, kv_lens, out, q_start=None, max_q: int = 1, max_kv: int | None = None,
                scale: float | None = None, window: int = 0, sinks: int = 0, workspace=None,
                stream=None) -> torch.Tensor:
    """Causal attention of ``q`` [T, q_heads, head_dim] over the cached tokens of each request.

    Request b owns rows ``q_start[b]`` .. ``q_start[b + 1] - 1`` (None: row b), at most ``max_q`` of them,
    the last at position ``kv_lens[b] - 1``.  With ``window`` > 0 a row sees the last ``window`` tokens up
    to its own and the first ``sinks``.  ``max_kv`` (default: the block table's reach) and ``max_q`` size
    the split and the workspace (``w4_kv4_attn_workspace_bytes``).  ``scale``: 1 / sqrt(head_dim)."""
    if not isinstance(cache, Kv4Cache):
        raise TypeError("cache must be a Kv4Cache")
    i, d = cache.device_index, cache.head_dim
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    B, width = block_table.shape
    if B > _INT_MAX or width > _INT_MAX:
        _too_large("w4_kv4_attn", max(B, width))
    qp, qs = _heads(q, "q", i, None, None, d)
    T, q_heads, _ = q.shape
    op, os = _heads(out, "out", i, T, q_heads, d)
    if max_kv is None:
        max_kv = width * cache.block_size
    tp, lp = _addresses(i, block_table, "block_table", _int32, None, kv_lens, "kv_lens", _int32, B)
    sp, = _optional_addresses(i, q_start, "q_start", _int32, B + 1)
    a = _AttnArgs(qp, op, qs, os, tp, lp, sp, T, B, q_heads, width, _near(max_q), _near(max_kv), _near(window),
                  _near(sinks), 1.0 / math.sqrt(d) if scale is None else scale)
    pw, nbytes = None, 0
    if workspace is not None:
        pw, nbytes = _ptr(workspace, "workspace", workspace.dtype, i), workspace.numel() * workspace.element_size()
    _call("w4_kv4_attn", lib.w4_kv4_attn, (ctypes.byref(a), cache.ref, pw, nbytes), stream, i)
    return out


def w4_sample_workspace_bytes(rows: int, vocab: int) -> int:
    return lib.w4_sample_workspace_bytes(_near(rows), _near(vocab))


def w4_sample(logits, uniform, tokens, temperature=None, top_k=None, top_p=None, min_p=None, workspace=None,
              stream=None) -> torch.Tensor:
    """One token of each row of BF16 ``logits`` [rows, vocab] from ``uniform`` (float64 [rows], in [0, 1)).

    ``temperature``, ``top_p``, ``min_p`` float32 [rows], ``top_k`` int32 [rows], each None for "off"
    (temperature 1).  ``tokens`` int32 [rows]; ``workspace`` as ``w4_sample_workspace_bytes``."""
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = logits.shape
    if rows > _INT_MAX or vocab > _INT_MAX:
        _too_large("w4_sample", max(rows, vocab))
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("logits: the values of a row must lie together")
    stride = logits.stride(0) if rows > 1 else vocab
    i = _device_of(logits, "logits", _bf16)
    pw, nbytes = None, 0
    if workspace is not None:
        pw, nbytes = _ptr(workspace, "workspace", workspace.dtype, i), workspace.numel() * workspace.element_size()
    up, out = _addresses(i, uniform, "uniform", _f64, rows, tokens, "tokens", _int32, rows)
    settings = _optional_addresses(i, temperature, "temperature", _f32, rows, top_k, "top_k", _int32, rows,
                                   top_p, "top_p", _f32, rows, min_p, "min_p", _f32, rows)
    args = (logits.data_ptr(), stride, up, *settings, out, rows, vocab, pw, nbytes)
    _call("w4_sample", lib.w4_sample, args, stream, i)
    return tokens
