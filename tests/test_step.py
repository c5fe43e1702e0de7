"""CPU tests of the decode step's operators: the header against the library and
the binding, every refusal (checked before any HIP call), and hand-built pins
of the FP64 oracle they are compared with."""
from __future__ import annotations

import ctypes
import pathlib
import re

import numpy as np
import pytest
import torch

import oracle
from oracle import step as ref

w4 = pytest.importorskip("gemm_w4_gemv_amd")
from gemm_w4_gemv_amd import step  # noqa: E402

lib = w4.lib
HEADER = pathlib.Path(__file__).resolve().parents[1] / "include" / "w4_step.h"
OK, NULL, SHAPE, UNSUP, ALIGN, WS, ALIAS, ARG = 0, 1, 2, 3, 4, 5, 6, 7
P = 1 << 40  # addresses that are never read: 64 GiB apart
at = lambda i: P + (i << 36)  # noqa: E731


# --------------------------------------------------------------- the header
def test_header_binding_and_exports_agree():
    text = HEADER.read_text()
    names = set(re.findall(r"W4_API\s+[\w\s\*]+?\b(w4_\w+)\s*\(", text))
    assert names == set(step.SIGNATURES)
    assert all(hasattr(lib, n) and hasattr(w4, n) for n in names)
    for name, value in (("W4_KV4_GROUP", step.KV4_GROUP), ("W4_KV4_PLAN_MAX_BATCH", step.KV4_PLAN_MAX_BATCH),
                        ("W4_SAMPLE_MAX_VOCAB", step.SAMPLE_MAX_VOCAB)):
        assert re.search(rf"#define {name} {value}\b", text)


# ---------------------------------------------------------------- refusals
def plan(**k):
    names = ("cached", "new", "table", "free", "count")
    outs = ("q_start", "kv_lens", "positions", "slots", "counts")
    ins = [k.get(n, at(i)) for i, n in enumerate(names)]
    sizes = [k.get("B", 4), k.get("width", 8), k.get("cap", 16), k.get("block", 16), k.get("rows", 9)]
    return lib.w4_kv4_plan(*ins, *sizes, *[k.get(n, at(8 + i)) for i, n in enumerate(outs)], None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(cached=None), NULL), (dict(new=None), NULL), (dict(table=None), NULL), (dict(free=None), NULL),
    (dict(count=None), NULL), (dict(q_start=None), NULL), (dict(kv_lens=None), NULL), (dict(positions=None), NULL),
    (dict(slots=None), NULL), (dict(counts=None), NULL), (dict(B=-1), SHAPE), (dict(width=-1), SHAPE),
    (dict(cap=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(B=4097), SHAPE), (dict(B=4096, width=1 << 20), SHAPE),
    (dict(block=0), ARG), (dict(block=24), ARG), (dict(block=8192), ARG), (dict(table=at(2) + 2), ALIGN),
    (dict(slots=at(8) + 4), ALIAS), (dict(kv_lens=at(0)), ALIAS), (dict(table=at(3) + 8), ALIAS), (dict(counts=at(4)), ALIAS),
])
def test_plan_refusals(kwargs, status):
    assert plan(**kwargs) == status
    assert "w4_kv4_plan" in w4.w4_last_error()


def cache_struct(**k):
    return step._CacheStruct(k.get("kc", at(20)), k.get("km", at(21)), k.get("vc", at(22)), k.get("vm", at(23)),
                             k.get("blocks", 10), k.get("block", 64), k.get("hkv", 2), k.get("dim", 128))


CACHE_BAD = [(dict(kc=None), NULL), (dict(vm=None), NULL), (dict(dim=96), UNSUP), (dict(dim=0), UNSUP), (dict(dim=512), UNSUP),
             (dict(block=8), UNSUP), (dict(block=48), UNSUP), (dict(block=512), UNSUP), (dict(blocks=0), SHAPE),
             (dict(hkv=0), SHAPE), (dict(blocks=1 << 26), SHAPE), (dict(km=at(21) + 8), ALIGN), (dict(vc=at(22) + 4), ALIGN)]


def qk(cache=True, **k):
    c = cache_struct(**k)
    hq, hkv, dim = k.get("hq", 4), k.get("call_hkv", k.get("hkv", 2)), k.get("call_dim", k.get("dim", 128))
    a = step._QkArgs(q=k.get("q", at(0)), k=k.get("k", at(1)), v=k.get("v", at(2)), q_stride=k.get("qs", hq * dim),
                     k_stride=k.get("ks", hkv * dim), v_stride=k.get("vs", hkv * dim), q_weight=k.get("qw", at(3)),
                     k_weight=k.get("kw", at(4)), cos_sin=k.get("cs", at(5)), positions=k.get("pos", at(6)),
                     slots=k.get("slots", at(7)), q_out=k.get("qo", at(8)), k_out=k.get("ko", at(9)),
                     q_out_stride=k.get("qos", hq * dim), k_out_stride=k.get("kos", hkv * dim), T=k.get("T", 5),
                     q_heads=hq, kv_heads=hkv, head_dim=dim, rot_dim=k.get("rot", dim), max_pos=k.get("reach", 100),
                     interleaved=0, eps=k.get("eps", 1e-6), weight_add=k.get("add", 0.0))
    return lib.w4_qk_norm_rope(ctypes.byref(a), ctypes.byref(c) if cache else None, None)


@pytest.mark.parametrize("kwargs,status", CACHE_BAD + [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(qo=None), NULL),
    (dict(cs=None), NULL), (dict(pos=None), NULL), (dict(cache=False, ko=None), NULL), (dict(T=-1), SHAPE),
    (dict(hq=-1), SHAPE), (dict(call_hkv=0), SHAPE), (dict(call_hkv=4), SHAPE), (dict(call_dim=64, rot=64), SHAPE),
    (dict(reach=0), SHAPE), (dict(rot=8), ARG), (dict(rot=144), ARG), (dict(rot=-16), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(add=float("nan")), ARG), (dict(qs=511), ARG),
    (dict(qs=516), ARG), (dict(ks=128), ARG), (dict(vs=0), ARG), (dict(kos=12), ARG), (dict(q=at(0) + 8), ALIGN),
    (dict(qw=at(3) + 2), ALIGN), (dict(cs=at(5) + 4), ALIGN), (dict(pos=at(6) + 2), ALIGN), (dict(qo=at(8) + 2), ALIGN),
    (dict(qo=at(0) + 16), ALIAS), (dict(qo=at(1)), ALIAS), (dict(ko=at(2)), ALIAS), (dict(ko=at(8)), ALIAS),
    (dict(qo=at(20)), ALIAS), (dict(k=at(22) + 64), ALIAS), (dict(qo=at(3)), ALIAS), (dict(vc=at(20)), ALIAS),
    (dict(qo=at(0), qos=1024), ALIAS), (dict(slots=at(20)), ALIAS), (dict(T=2 ** 31 - 1, hq=60000, rot=0), SHAPE),
])
def test_qk_norm_rope_refusals(kwargs, status):
    assert qk(**kwargs) == status
    assert "w4_qk_norm_rope" in w4.w4_last_error()


def test_qk_norm_rope_accepts_side_by_side_rows():
    """q, k and v in one buffer, outputs over their inputs: no overlap (T = 0 launches nothing either way)."""
    b, s = at(0), 8 * 128
    side = dict(q=b, k=b + 4 * 128 * 2, v=b + 6 * 128 * 2, qs=s, ks=s, vs=s)
    assert qk(T=0, **side, qo=b, qos=s, ko=b + 4 * 128 * 2, kos=s) == OK
    assert qk(T=3, **side, qo=b + 4 * 128 * 2, qos=s) == ALIAS  # over k and v
    assert qk(T=3, **side, qo=b, qos=s, ko=b + 6 * 128 * 2, kos=s) == ALIAS  # k_out over v
    assert qk(T=3, **side, qo=b + 2 * 128 * 2, qos=s) == ALIAS  # half over its own input


def read(**k):
    c = cache_struct(**k)
    return lib.w4_kv4_read(ctypes.byref(c), k.get("slots", at(7)), k.get("n", 5), k.get("ko", at(8)), k.get("vo", at(9)), None)


@pytest.mark.parametrize("kwargs,status", CACHE_BAD + [
    (dict(slots=None), NULL), (dict(ko=None, vo=None), NULL), (dict(n=-1), SHAPE), (dict(n=2 ** 31 - 1), SHAPE),
    (dict(ko=at(8) + 8), ALIGN), (dict(slots=at(7) + 1), ALIGN), (dict(ko=at(9) + 16), ALIAS), (dict(vo=at(23)), ALIAS),
    (dict(ko=at(7)), ALIAS),
])
def test_read_refusals(kwargs, status):
    assert read(**kwargs) == status
    assert "w4_kv4_read" in w4.w4_last_error()


def attn(**k):
    c = cache_struct(**k)
    hq, dim = k.get("hq", 4), k.get("dim", 128)
    a = step._AttnArgs(q=k.get("q", at(0)), out=k.get("out", at(1)), q_stride=k.get("qs", hq * dim),
                       out_stride=k.get("os", hq * dim), block_table=k.get("table", at(2)), kv_lens=k.get("lens", at(3)),
                       q_start=k.get("q_start", at(4)), T=k.get("T", 6), B=k.get("B", 3), q_heads=hq,
                       max_blocks=k.get("width", 8), max_q=k.get("max_q", 2), max_kv=k.get("max_kv", 100),
                       window=k.get("window", 0), sinks=k.get("sinks", 0), scale=k.get("scale", 0.1))
    return lib.w4_kv4_attn(ctypes.byref(a), ctypes.byref(c), k.get("ws", at(5)), k.get("wsb", 1 << 30), None)


@pytest.mark.parametrize("kwargs,status", CACHE_BAD + [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(T=-1), SHAPE),
    (dict(B=-1), SHAPE), (dict(hq=0), SHAPE), (dict(hq=5), SHAPE), (dict(width=-1), SHAPE), (dict(max_q=-1), SHAPE),
    (dict(max_kv=-1), SHAPE), (dict(q_start=None), SHAPE), (dict(max_q=2 ** 30), SHAPE), (dict(B=2 ** 30), SHAPE),
    (dict(window=-1), ARG), (dict(sinks=-1), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(qs=100), ARG), (dict(os=516), ARG),
    (dict(q=at(0) + 2), ALIGN), (dict(out=at(1) + 8), ALIGN), (dict(lens=at(3) + 2), ALIGN),
    (dict(max_kv=100000, ws=None), WS), (dict(max_kv=100000, wsb=16), WS), (dict(max_kv=100000, ws=at(5) + 4), ALIGN),
    (dict(out=at(0)), ALIAS), (dict(out=at(20) + 1024), ALIAS), (dict(out=at(4)), ALIAS), (dict(max_kv=100000, ws=at(1)), ALIAS),
    (dict(max_kv=100000, ws=at(23)), ALIAS),
])
def test_attn_refusals(kwargs, status):
    assert attn(**kwargs) == status
    assert "w4_kv4_attn" in w4.w4_last_error()


@pytest.mark.parametrize("kwargs", [dict(T=0), dict(B=0), dict(max_q=0), dict(T=0, B=0, q_start=None)])
def test_attn_empty_problem_launches_nothing(kwargs):
    assert attn(**kwargs) == OK


def sample(**k):
    return lib.w4_sample(k.get("logits", at(0)), k.get("stride", 40000), k.get("u", at(1)), k.get("t", at(2)), k.get("k", at(3)),
                         k.get("p", at(4)), k.get("m", at(5)), k.get("tokens", at(6)), k.get("rows", 3), k.get("vocab", 40000),
                         k.get("ws", at(7)), k.get("wsb", 1 << 30), None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(logits=None), NULL), (dict(u=None), NULL), (dict(tokens=None), NULL), (dict(rows=-1), SHAPE),
    (dict(rows=65536), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=(1 << 20) + 1, stride=1 << 21), SHAPE),
    (dict(stride=999), ARG), (dict(logits=at(0) + 1), ALIGN), (dict(u=at(1) + 4), ALIGN), (dict(tokens=at(6) + 2), ALIGN),
    (dict(ws=None), WS), (dict(wsb=0), WS), (dict(ws=at(7) + 8), ALIGN), (dict(tokens=at(0) + 400), ALIAS),
    (dict(tokens=at(3)), ALIAS), (dict(ws=at(0)), ALIAS), (dict(ws=at(6)), ALIAS),
])
def test_sample_refusals(kwargs, status):
    assert sample(**kwargs) == status
    assert "w4_sample" in w4.w4_last_error()


def test_sample_empty_problem_launches_nothing():
    assert sample(rows=0) == OK
    assert w4.w4_sample_workspace_bytes(0, 100) == w4.w4_sample_workspace_bytes(3, 0) == 0


def test_binding_refuses_host_tensors_and_wrong_layouts():
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w4.w4_qk_norm_rope(None, x, k_out=x)  # host memory
    with pytest.raises(TypeError):
        w4.w4_qk_norm_rope(None, x.float(), k_out=x)
    with pytest.raises(ValueError):
        w4.w4_qk_norm_rope(None, x.transpose(1, 2), k_out=x)
    with pytest.raises(ValueError):
        w4.w4_sample(torch.zeros(5, dtype=torch.bfloat16), None, None)
    with pytest.raises(ValueError):
        w4.Kv4Cache(torch.zeros(2, 2, 16, 16, dtype=torch.int32), *[torch.zeros(1)] * 3)
    with pytest.raises(TypeError):
        w4.w4_kv4_attn(x, None, x, x, x)


# -------------------------------------------------------- pins of the oracle
def bits(*v):
    return ref.round_to_bf16(np.array(v, dtype=np.float64))


def test_pin_quantise_by_hand():
    """0 .. 15 thrice over: scale 1, minimum 0, codes the values; a constant group: scale 0, codes 0."""
    x = np.tile(np.arange(16.0), 4)
    q, meta = ref.quantise(ref.round_to_bf16(x))
    assert np.array_equal(q, x) and meta.tolist() == [[1.0, 0.0]]
    q, meta = ref.quantise(ref.round_to_bf16(np.full(64, -2.5)))
    assert not q.any() and meta.tolist() == [[0.0, -2.5]]
    assert np.array_equal(ref.dequantise(q, meta), np.full(64, -2.5))
    # two groups, the second shifted and twice as wide
    x = np.concatenate((np.tile(np.arange(16.0), 8), 10 + 2 * np.tile(np.arange(16.0), 8)))
    q, meta = ref.quantise(ref.round_to_bf16(x))
    assert meta.tolist() == [[1.0, 0.0], [2.0, 10.0]] and np.array_equal(ref.dequantise(q, meta), x)


def test_pin_quantise_error_is_half_a_step():
    x = oracle.bf16_to_f64(ref.round_to_bf16(np.random.default_rng(1).normal(0, 3, (50, 256))))
    q, meta = ref.quantise(ref.round_to_bf16(x))
    err = np.abs(ref.dequantise(q, meta) - x).reshape(50, 2, 128).max(axis=-1)
    # half a step, the scale's own rounding over 15 steps, and the minimum's
    s, m = meta[..., 0].astype(np.float64), np.abs(meta[..., 1].astype(np.float64))
    assert np.all(err <= s * (0.5 + 15 * 2.0 ** -11) + m * 2.0 ** -11 + 2.0 ** -20)


def test_pin_packing_and_the_cache_layout():
    assert ref.pack(np.arange(16, dtype=np.uint8)).view(np.uint32).tolist() == [0x76543210, 0xFEDCBA98]
    assert np.array_equal(ref.unpack(ref.pack(np.arange(16, dtype=np.uint8))), np.arange(16))
    c = ref.Cache(2, 16, 1, 64)
    k = np.zeros((1, 64))
    k[0, 9] = 15.0
    c.put(16 + 6, ref.round_to_bf16(k), ref.round_to_bf16(k))
    assert c.k_codes[1, 0, 6].view(np.uint32).tolist() == [0, 0xF0, 0, 0, 0, 0, 0, 0]
    assert c.v_codes[1, 0, 1, 1, 2] == 0xF0 and np.count_nonzero(c.v_codes) == 1  # token 6: row 1, place 2
    assert c.k_meta[1, 0, 0, 6].tolist() == [1.0, 0.0]


def test_pin_rotation_by_hand():
    cs = np.array([[1.0] * 8 + [0.0] * 8, [0.0] * 8 + [1.0] * 8])  # position 1: a quarter turn
    x = ref.round_to_bf16(np.arange(64.0)).reshape(1, 1, 64)
    far = ref.norm_rope(x, None, cs, [1], 16, False, 0, 0)[0, 0]
    assert far[:16].tolist() == [-8.0, -9, -10, -11, -12, -13, -14, -15, 0, 1, 2, 3, 4, 5, 6, 7]
    near = ref.norm_rope(x, None, cs, [1], 16, True, 0, 0)[0, 0]
    assert near[:16].tolist() == [-1.0, 0, -3, 2, -5, 4, -7, 6, -9, 8, -11, 10, -13, 12, -15, 14]
    assert far[16:].tolist() == near[16:].tolist() == list(range(16, 64))
    assert np.array_equal(ref.norm_rope(x, None, cs, [0], 16, True, 0, 0)[0, 0], np.arange(64.0))


def test_pin_norm_by_hand():
    x = ref.round_to_bf16(np.tile([3.0, -4.0], 32)).reshape(1, 1, 64)  # mean square 12.5
    w = ref.round_to_bf16(np.full(64, 0.5))
    y = ref.norm_rope(x, w, None, None, 0, False, 3.5, 1.0)[0, 0]  # sqrt(12.5 + 3.5) = 4
    assert np.array_equal(y, np.tile([3.0, -4.0], 32) / 4 * 1.5)


def test_pin_visible():
    assert ref.visible(4, 8, 0, 0).tolist() == [1, 1, 1, 1, 1, 0, 0, 0]
    assert ref.visible(4, 8, 2, 0).tolist() == [0, 0, 0, 1, 1, 0, 0, 0]
    assert ref.visible(4, 8, 2, 1).tolist() == [1, 0, 0, 1, 1, 0, 0, 0]
    assert ref.visible(1, 8, 2, 9).tolist() == [1, 1, 0, 0, 0, 0, 0, 0]
    assert not ref.visible(-1, 8, 0, 3).any()


def test_pin_attention_by_hand():
    """Equal scores give the mean of the visible values; one large score gives that value; no token gives 0."""
    c = ref.Cache(2, 16, 1, 64)
    for t in range(20):
        k = np.zeros((1, 64))
        k[0, 0] = 15.0 if t == 7 else 0.0
        c.put(t, ref.round_to_bf16(k), ref.round_to_bf16(np.full((1, 64), float(t))))
    q = np.zeros((3, 1, 64))
    q[1, 0, 0] = 100.0
    out, noise = ref.attention(ref.round_to_bf16(q), c, [[0, 1], [0, 1], [0, 1]], [20, 20, 0], [0, 1, 2, 3], 1.0)
    assert np.allclose(out[0], 9.5) and np.allclose(out[1], 7.0) and np.all(out[2] == 0) and np.all(noise >= 0)
    out, _ = ref.attention(ref.round_to_bf16(q[:1]), c, [[0, 1]], [20], [0, 1], 1.0, window=2, sinks=1)
    assert np.allclose(out[0], (0 + 18 + 19) / 3)
    out, _ = ref.attention(ref.round_to_bf16(q), c, [[1, 0]], [3], [0, 3], 1.0)  # pages swapped: tokens 16 ..
    assert np.allclose(out[0], 16) and np.allclose(out[2], 17)


def test_pin_plan_by_hand():
    got = ref.plan([3, 4, 0], [2, 0, 1], [[5, -1], [6, -1], [-1, -1]], [7, 8, 9], 2, 4, 5)
    assert got[0] == [0, 2, 2, 3] and got[1] == [5, 4, 1]
    assert got[2] == [3, 4, 0, -1, -1] and got[3] == [23, 32, 28, -1, -1]
    assert got[4].tolist() == [[5, 8], [6, -1], [7, -1]] and got[5] == [0, 0]
    got = ref.plan([0], [9], [[-1, -1]], [3], 1, 4, 9)  # one page short, one token past the table
    assert got[3] == [12, 13, 14, 15, -1, -1, -1, -1, -1] and got[5] == [0, 1]


def test_pin_sample_by_hand():
    x = bits(0.0, 2.0, 1.0, 2.0)
    assert ref.sample(x, 0.0) == 1 and ref.sample(x, 0.999) == 0
    w = np.exp([0.0, 0.0, -1.0, -2.0])
    assert ref.sample(x, (w[0] + 1e-6) / w.sum()) == 3 and ref.sample(x, (2 + 1e-6) / w.sum()) == 2
    assert ref.sample(x, 0.99, top_k=2) == 3 and ref.sample(x, 0.99, min_p=0.3) == 2
    assert ref.sample(x, 0.99, temperature=0.0) == 1
    assert ref.sample(x, 0.99, top_p=0.3) == 1  # 1 of 2.5: the first weighs 0.4
    assert ref.sample(x, 0.99, top_p=0.5) == 3 and ref.sample(x, 0.99, top_p=0.9) == 2
    assert ref.sample(bits(-np.inf, np.nan), 0.5) == -1
    assert ref.sample(bits(0.0, -0.0, 0.0), 0.5) == 1
