"""Binding of the decode step's operators (``include/w4_step.h``): the 4-bit
key/value cache, what fills it, the attention that reads it, the sampler.

Argument marshalling only, as in the package's other functions.  Tensors of
one call must live on one device; the call runs there, on ``stream`` or the
device's current stream.  Outputs and workspaces belong to the caller.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _check, lib

__all__ = ["Kv4Cache", "w4_kv4_plan", "w4_qk_norm_rope", "w4_kv4_read", "w4_kv4_attn", "w4_kv4_attn_workspace_bytes",
           "w4_sample", "w4_sample_workspace_bytes", "KV4_GROUP", "KV4_PLAN_MAX_BATCH", "SAMPLE_MAX_VOCAB"]

KV4_GROUP = 128
KV4_PLAN_MAX_BATCH = 4096
SAMPLE_MAX_VOCAB = 1048576
_INT_MAX = 2 ** 31 - 1  # ctypes would cut a larger length to 32 bits without a word

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


class _Call:
    """Checks one call's tensors: on one GPU, of the given dtype and layout."""

    def __init__(self, where: str):
        self.where, self.device = where, None

    def ptr(self, t, name, dtype, contiguous=True):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, not {dtype}")
        d = t.device
        if d.type != "cuda":
            raise ValueError(f"{name} must be a device tensor (got {d})")
        if d != self.device:
            if self.device is not None:
                raise ValueError(f"{name} lies on {d}, other tensors of this call on {self.device}")
            self.device = d
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def maybe(self, t, name, dtype):
        return None if t is None else self.ptr(t, name, dtype)

    def heads(self, t, name, rows=None, heads=None, dim=None):
        """[rows, heads, dim] BF16 whose heads lie together: (pointer, row stride)."""
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a tensor [tokens, heads, head_dim]")
        got = t.shape
        if (rows is not None and got[0] != rows) or (heads is not None and got[1] != heads) or \
                (dim is not None and got[2] != dim):
            raise ValueError(f"{name} must be {[rows, heads, dim]}; got {list(got)}")
        step, inner, unit = t.stride()
        if (got[2] > 1 and unit != 1) or (got[1] > 1 and inner != got[2]):
            raise ValueError(f"{name}: the heads of a row must lie together")
        if got[0] <= 1:  # one row or none: whatever stride it has is not used
            step = max(got[1] * got[2], 8)
        return self.ptr(t, name, torch.bfloat16, contiguous=False), step

    def run(self, fn, args, stream):
        """fn(*args, stream) on the tensors' device."""
        index = self.device.index
        if index == torch.cuda.current_device():
            self._run(fn, args, stream)
        else:
            with torch.cuda.device(index):
                self._run(fn, args, stream)

    def _run(self, fn, args, stream):
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        elif isinstance(stream, torch.cuda.Stream):
            if stream.device != self.device:
                raise ValueError(f"{self.where}: stream of {stream.device}, tensors on {self.device}")
            stream = stream.cuda_stream
        _check(fn(*args, int(stream)), self.where)


def _length(t, name, n):
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must be [{n}]; got {list(t.shape)}")


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
        call = _Call("Kv4Cache")
        self.k_codes, self.k_meta, self.v_codes, self.v_meta = k_codes, k_meta, v_codes, v_meta
        self.num_blocks, self.kv_heads, self.block_size, self.head_dim = nb, h, bs, d
        self.struct = _CacheStruct(call.ptr(k_codes, "k_codes", torch.int32), call.ptr(k_meta, "k_meta", torch.float16),
                                   call.ptr(v_codes, "v_codes", torch.int32), call.ptr(v_meta, "v_meta", torch.float16),
                                   nb, bs, h, d)
        self.ref = ctypes.byref(self.struct)
        self.device = call.device

    @classmethod
    def empty(cls, num_blocks: int, block_size: int, kv_heads: int, head_dim: int, device="cuda") -> "Kv4Cache":
        groups = max(1, head_dim // KV4_GROUP)
        codes = dict(dtype=torch.int32, device=device)
        meta = dict(dtype=torch.float16, device=device)
        return cls(torch.empty(num_blocks, kv_heads, block_size, head_dim // 8, **codes),
                   torch.empty(num_blocks, kv_heads, groups, block_size, 2, **meta),
                   torch.empty(num_blocks, kv_heads, block_size // 4, head_dim // 8, 4, **codes),
                   torch.empty(num_blocks, kv_heads, groups, block_size, 2, **meta))


def _with_cache(call, cache):
    if not isinstance(cache, Kv4Cache):
        raise TypeError("cache must be a Kv4Cache")
    if call.device is not None and call.device != cache.device:
        raise ValueError(f"the cache lies on {cache.device}, other tensors of this call on {call.device}")
    call.device = cache.device
    return cache.ref


def w4_kv4_plan(cached, new_tokens, block_table, free_blocks, free_count, block_size: int, q_start, kv_lens,
                positions, slots, counts, stream=None) -> None:
    """Block tables, slot map, positions and row ranges of a step from the requests' lengths.

    ``cached``, ``new_tokens`` int32 [B]; ``block_table`` int32 [B, max_blocks] (new
    pages' entries are written); ``free_blocks`` int32 [n], ``free_count`` int32 [1].
    Outputs: ``q_start`` [B + 1], ``kv_lens`` [B], ``positions`` and ``slots`` [rows] (-1
    behind the last request), ``counts`` [2] (pages left, pages short)."""
    call, i32 = _Call("w4_kv4_plan"), torch.int32
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    B, width = block_table.shape
    rows = positions.numel()
    for name, t, n in (("cached", cached, B), ("new_tokens", new_tokens, B), ("q_start", q_start, B + 1),
                       ("kv_lens", kv_lens, B), ("slots", slots, rows), ("positions", positions, rows),
                       ("free_count", free_count, 1), ("counts", counts, 2), ("free_blocks", free_blocks, free_blocks.numel())):
        _length(t, name, n)
    args = (call.ptr(cached, "cached", i32), call.ptr(new_tokens, "new_tokens", i32),
            call.ptr(block_table, "block_table", i32), call.ptr(free_blocks, "free_blocks", i32),
            call.ptr(free_count, "free_count", i32), B, width, free_blocks.shape[0], int(block_size), rows,
            call.ptr(q_start, "q_start", i32), call.ptr(kv_lens, "kv_lens", i32),
            call.ptr(positions, "positions", i32), call.ptr(slots, "slots", i32), call.ptr(counts, "counts", i32))
    call.run(lib.w4_kv4_plan, args, stream)


def w4_qk_norm_rope(q, k, positions=None, cos_sin=None, q_out=None, k_out=None, q_weight=None, k_weight=None,
                    eps: float = 1e-6, weight_add: float = 0.0, interleaved: bool = False, v=None, cache=None,
                    slots=None, stream=None) -> None:
    """RMS norm of each query and key head, rotation by position, and with ``cache`` the keys and
    ``v`` quantised into their ``slots``.

    ``q`` [T, q_heads, head_dim] (None: keys only), ``k``, ``v`` [T, kv_heads, head_dim], BF16, rows at
    any stride; ``cos_sin`` float [max_pos, rot_dim] (cosines, then sines; None: no rotation).
    ``q_out`` and ``k_out`` may be ``q`` and ``k`` themselves; ``k_out`` may be None with a cache."""
    call = _Call("w4_qk_norm_rope")
    a = _QkArgs()
    a.k, a.k_stride = call.heads(k, "k")
    T, a.kv_heads, a.head_dim = k.shape
    a.T = T
    if q is not None:
        a.q, a.q_stride = call.heads(q, "q", T, None, a.head_dim)
        a.q_heads = q.shape[1]
        if q_out is None:
            raise ValueError("q_out must be given with q")
        a.q_out, a.q_out_stride = call.heads(q_out, "q_out", T, a.q_heads, a.head_dim)
    if k_out is not None:
        a.k_out, a.k_out_stride = call.heads(k_out, "k_out", T, a.kv_heads, a.head_dim)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _length(w, name, a.head_dim)
            setattr(a, name, call.ptr(w, name, torch.bfloat16))
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_pos, rot_dim]")
        a.max_pos, a.rot_dim = cos_sin.shape
        a.cos_sin = call.ptr(cos_sin, "cos_sin", torch.float32)
    if positions is not None:
        _length(positions, "positions", T)
        a.positions = call.ptr(positions, "positions", torch.int32)
    a.eps, a.weight_add, a.interleaved = eps, weight_add, bool(interleaved)
    ref = None
    if cache is not None:
        if v is None or slots is None:
            raise ValueError("v and slots must be given with a cache")
        a.v, a.v_stride = call.heads(v, "v", T, a.kv_heads, a.head_dim)
        _length(slots, "slots", T)
        a.slots = call.ptr(slots, "slots", torch.int32)
        ref = _with_cache(call, cache)
    call.run(lib.w4_qk_norm_rope, (ctypes.byref(a), ref), stream)


def w4_kv4_read(cache, slots, k_out=None, v_out=None, stream=None) -> None:
    """The keys and values that ``slots`` of the cache stand for, in BF16 [n, kv_heads, head_dim]."""
    call = _Call("w4_kv4_read")
    ref = _with_cache(call, cache)
    _length(slots, "slots", slots.numel())
    n = slots.shape[0]
    outs = []
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None and tuple(t.shape) != (n, cache.kv_heads, cache.head_dim):
            raise ValueError(f"{name} must be {(n, cache.kv_heads, cache.head_dim)}; got {tuple(t.shape)}")
        outs.append(call.maybe(t, name, torch.bfloat16))
    call.run(lib.w4_kv4_read, (ref, call.ptr(slots, "slots", torch.int32), n, *outs), stream)


def w4_kv4_attn_workspace_bytes(cache, T: int, B: int, q_heads: int, max_q: int, max_kv: int, window: int = 0,
                                sinks: int = 0) -> int:
    a = _AttnArgs(T=T, B=B, q_heads=q_heads, max_q=max_q, max_kv=min(max_kv, _INT_MAX), window=min(window, _INT_MAX),
                  sinks=min(sinks, _INT_MAX))
    return lib.w4_kv4_attn_workspace_bytes(ctypes.byref(a), cache.ref)


def w4_kv4_attn(q, cache, block_table, kv_lens, out, q_start=None, max_q: int = 1, max_kv: int | None = None,
                scale: float | None = None, window: int = 0, sinks: int = 0, workspace=None,
                stream=None) -> torch.Tensor:
    """Causal attention of ``q`` [T, q_heads, head_dim] over the cached tokens of each request.

    Request b owns rows ``q_start[b]`` .. ``q_start[b + 1] - 1`` (None: row b), at most ``max_q`` of them,
    the last at position ``kv_lens[b] - 1``.  With ``window`` > 0 a row sees the last ``window`` tokens up
    to its own and the first ``sinks``.  ``max_kv`` (default: the block table's reach) and ``max_q`` size
    the split and the workspace (``w4_kv4_attn_workspace_bytes``).  ``scale``: 1 / sqrt(head_dim)."""
    call = _Call("w4_kv4_attn")
    ref = _with_cache(call, cache)
    a = _AttnArgs()
    d = cache.head_dim
    a.q, a.q_stride = call.heads(q, "q", None, None, d)
    a.T, a.q_heads, _ = q.shape
    a.out, a.out_stride = call.heads(out, "out", a.T, a.q_heads, d)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    a.B, a.max_blocks = block_table.shape
    a.block_table = call.ptr(block_table, "block_table", torch.int32)
    _length(kv_lens, "kv_lens", a.B)
    a.kv_lens = call.ptr(kv_lens, "kv_lens", torch.int32)
    if q_start is not None:
        _length(q_start, "q_start", a.B + 1)
        a.q_start = call.ptr(q_start, "q_start", torch.int32)
    a.max_q, a.window, a.sinks = max_q, min(window, _INT_MAX), min(sinks, _INT_MAX)
    a.max_kv = min(a.max_blocks * cache.block_size if max_kv is None else max_kv, _INT_MAX)
    a.scale = 1.0 / math.sqrt(d) if scale is None else scale
    pw, nbytes = None, 0
    if workspace is not None:
        pw, nbytes = call.ptr(workspace, "workspace", workspace.dtype), workspace.numel() * workspace.element_size()
    call.run(lib.w4_kv4_attn, (ctypes.byref(a), ref, pw, nbytes), stream)
    return out


def w4_sample_workspace_bytes(rows: int, vocab: int) -> int:
    return lib.w4_sample_workspace_bytes(rows, vocab)


def w4_sample(logits, uniform, tokens, temperature=None, top_k=None, top_p=None, min_p=None, workspace=None,
              stream=None) -> torch.Tensor:
    """One token of each row of BF16 ``logits`` [rows, vocab] from ``uniform`` (float64 [rows], in [0, 1)).

    ``temperature``, ``top_p``, ``min_p`` float32 [rows], ``top_k`` int32 [rows], each None for "off"
    (temperature 1).  ``tokens`` int32 [rows]; ``workspace`` as ``w4_sample_workspace_bytes``."""
    call = _Call("w4_sample")
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = logits.shape
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("logits: the values of a row must lie together")
    stride = logits.stride(0) if rows > 1 else vocab
    f32 = torch.float32
    for name, t in (("uniform", uniform), ("tokens", tokens), ("temperature", temperature), ("top_k", top_k),
                    ("top_p", top_p), ("min_p", min_p)):
        if t is not None:
            _length(t, name, rows)
    args = [call.ptr(logits, "logits", torch.bfloat16, contiguous=False), stride,
            call.ptr(uniform, "uniform", torch.float64), call.maybe(temperature, "temperature", f32),
            call.maybe(top_k, "top_k", torch.int32), call.maybe(top_p, "top_p", f32), call.maybe(min_p, "min_p", f32),
            call.ptr(tokens, "tokens", torch.int32), rows, vocab, None, 0]
    if workspace is not None:
        args[-2:] = (call.ptr(workspace, "workspace", workspace.dtype), workspace.numel() * workspace.element_size())
    call.run(lib.w4_sample, args, stream)
    return tokens
