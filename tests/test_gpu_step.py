"""GPU parity of the decode step's operators against the FP64 oracle.

Tolerances, from the arithmetic (a rounding to BF16 is off by at most 2^-8
relative, one to FP32 by 2^-24):
  * keys, codes, scales, tables, tokens, read-back values: equal, bit for bit;
  * queries: one rounding to BF16 of a value formed in FP32 from at most 256
    squares and a handful of products, so 2^-8 |y| + 2^-20 of the pair's size;
  * attention: ``noise`` of ``oracle.step.attention``.  A score is a sum of
    exact products in FP32: at most 40 additions of partial sums no larger
    than (136 s + |m|) sum |x|, each off by 2^-24, and the exponential's
    argument and result by a few 2^-24 more; that moves a weight by
    delta = that, relative, and the output by 2 sum w delta |v - o| at most
    (the norm moves too).  Each weight times its value's scale is rounded to
    BF16 (2^-8 of w |s (q - 8)|, added up without help from signs), sums over
    the tokens are FP32 (at most 64 roundings of partial sums, 2^-18), the
    result is rounded once (2^-8 |o|).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import seeded_inputs as si
from oracle import step as ref

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemm_w4_gemv_amd")
from gemm_w4_gemv_amd import host  # noqa: E402

DEV = "cuda"
bf16, i32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device=DEV)


def to_device(c: ref.Cache):
    return w4.Kv4Cache(*(torch.from_numpy(np.ascontiguousarray(t)).to(DEV)
                         for t in (c.k_codes, c.k_meta, c.v_codes, c.v_meta)))


def random_cache(seed, blocks, block, heads, dim):
    """Random codes and (s, m) pairs: values of about unit size."""
    c, g = ref.Cache(blocks, block, heads, dim), si.rng(seed, 40)
    for name in ("k", "v"):
        codes, meta = getattr(c, name + "_codes"), getattr(c, name + "_meta")
        codes[...] = si.random_words(g, codes.shape, np.int32)
        meta[..., 0] = g.uniform(0.05, 0.4, meta.shape[:-1])
        meta[..., 1] = -7.5 * meta[..., 0].astype(np.float64) + g.normal(0, 0.3, meta.shape[:-1])
    return c


def same_bits(a, b):
    return np.array_equal(np.asarray(a).view(np.uint16), np.asarray(b).view(np.uint16))


# -------------------------------------------------------------------- plan
def run_plan(cached, new, table, free, count, block, rows):
    B = len(cached)
    t = ints(table)
    out = dict(q_start=torch.full((B + 1,), 77, dtype=i32, device=DEV), kv_lens=torch.full((B,), 77, dtype=i32, device=DEV),
               positions=torch.full((rows,), 77, dtype=i32, device=DEV), slots=torch.full((rows,), 77, dtype=i32, device=DEV),
               counts=torch.full((2,), 77, dtype=i32, device=DEV))
    w4.w4_kv4_plan(ints(cached), ints(new), t, ints(free), ints([count]), block, **out)
    torch.cuda.synchronize()
    return {**{k: v.cpu().numpy() for k, v in out.items()}, "table": t.cpu().numpy()}


def check_plan(got, want):
    for name, w in zip(("q_start", "kv_lens", "positions", "slots", "table", "counts"), want):
        assert np.array_equal(got[name], np.asarray(w)), name


@pytest.mark.parametrize("B,block,new_max,kv_max,spare", [
    (1, 16, 1, 1, 0), (1, 64, 700, 2000, 0), (5, 16, 40, 100, 2), (257, 32, 1, 900, 0), (600, 16, 7, 300, -40),
    (4096, 128, 2, 1000, 0), (3, 1, 5, 9, 0),
])
def test_plan(B, block, new_max, kv_max, spare):
    """Requests at rest, at a page's edge and new; a stack that runs short (spare < 0); padding rows."""
    g = si.rng(41, B, block, new_max)
    new = g.integers(0, new_max + 1, B)
    cached = g.integers(0, kv_max + 1, B)
    cached[::3] = cached[::3] // block * block
    width = -(-(int(cached.max()) + new_max) // block) + 1
    held = -(-cached // block)
    pages = g.permutation(int(held.sum()) + B * (new_max // block + 2))
    table = np.full((B, width), -7)
    at = 0
    for b in range(B):
        table[b, :held[b]] = pages[at:at + held[b]]
        at += held[b]
    need = int((-(-(cached + new) // block) - held).sum())
    free = pages[at:at + max(need + spare, 0) + 3]
    count = min(max(need + spare, 0), len(free))
    rows = int(new.sum()) + 5
    check_plan(run_plan(cached, new, table, free, count, block, rows),
               ref.plan(cached, new, table, free, count, block, rows))


@pytest.mark.parametrize("cached,new,width,count,rows", [
    ([0], [0], 3, 4, 6), ([10, -3], [3, -2], 2, 4, 9), ([30, 0], [10, 4], 2, 4, 20),  # past max_blocks
    ([0, 0], [5, 5], 4, 0, 10), ([0, 0], [5, 5], 4, 99, 4), ([16], [1], 0, 4, 3),
])
def test_plan_edges(cached, new, width, count, rows):
    """Nothing to do, negative lengths, more tokens than the table or the rows hold, an empty stack, no table."""
    table = np.arange(len(cached) * width).reshape(len(cached), width) + 100
    free = [9, 8, 7, 6]
    got = run_plan(cached, new, table, free, count, 16, rows)
    check_plan(got, ref.plan(cached, new, table, free, count, 16, rows))


def test_plan_no_requests():
    got = run_plan([], [], np.zeros((0, 4)), [1, 2], 2, 16, 3)
    check_plan(got, ref.plan([], [], np.zeros((0, 4)), [1, 2], 2, 16, 3))


# ------------------------------------------------------------------- store
def qk_case(seed, T, hq, hkv, dim, block):
    qkv = si.bf16_normal(seed, (42, T, hq), (T, hq + 2 * hkv, dim))
    return qkv, host.bf16_tensor(qkv)


def rope_table(rot, reach=500):
    turn = np.arange(reach)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.concatenate((np.cos(turn), np.sin(turn)), axis=1).astype(np.float32)


def check_queries(got, want, what):
    """FP32 arithmetic and one rounding to BF16."""
    size = np.abs(want).max(axis=-1, keepdims=True)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size), what


@pytest.mark.parametrize("T,hq,hkv,dim,rot,inter,norm,block,add", [
    (1, 16, 8, 256, 256, False, True, 64, 0.0), (3, 4, 2, 128, 128, False, True, 16, 1.0),
    (37, 3, 1, 64, 64, True, True, 32, 0.0), (5, 8, 8, 128, 64, True, False, 128, 0.0),
    (129, 6, 3, 64, 16, False, True, 16, 0.0), (9, 5, 5, 256, 0, False, True, 256, 0.0),
    (2, 1, 1, 256, 32, True, False, 64, 0.0), (700, 2, 1, 128, 48, False, True, 64, 1.0),
])
def test_norm_rope_store(T, hq, hkv, dim, rot, inter, norm, block, add):
    """Side-by-side q, k, v; queries within their rounding, keys, codes and pairs bit for bit; slots
    that are not written stay; read-back equals the values that the codes stand for."""
    qkv, dev = qk_case(1, T, hq, hkv, dim, block)
    g = si.rng(43, T, dim, rot)
    qw = si.bf16_normal(2, (1, dim), (dim,)) if norm else None
    kw = si.bf16_normal(2, (2, dim), (dim,)) if norm else None
    cs = rope_table(rot) if rot else None
    pos = g.integers(0, 500, T)
    blocks = -(-T // block) + 2
    slots = g.permutation(blocks * block)[:T]
    if T > 4:
        slots[1], slots[2] = -1, blocks * block  # not stored
    host_cache = random_cache(3, blocks, block, hkv, dim)
    cache = to_device(host_cache)
    q_out = torch.full((T, hq, dim), 7.0, dtype=bf16, device=DEV)
    k_out = torch.full((T, hkv, dim), 7.0, dtype=bf16, device=DEV)
    w4.w4_qk_norm_rope(dev[:, :hq], dev[:, hq:hq + hkv], ints(pos) if rot else None,
                       torch.from_numpy(cs).to(DEV) if rot else None, q_out=q_out, k_out=k_out,
                       q_weight=None if qw is None else host.bf16_tensor(qw),
                       k_weight=None if kw is None else host.bf16_tensor(kw), eps=1e-6, weight_add=add,
                       interleaved=inter, v=dev[:, hq + hkv:], cache=cache, slots=ints(slots))
    torch.cuda.synchronize()
    args = (cs, pos, rot, inter, 1e-6, add)
    check_queries(host.bf16_values(q_out), ref.norm_rope(qkv[:, :hq], qw, *args), "q")
    k_bits = ref.round_to_bf16(ref.norm_rope(qkv[:, hq:hq + hkv], kw, *args))
    assert same_bits(host.bits_of(k_out), k_bits)
    for t in range(T):
        host_cache.put(slots[t], k_bits[t], qkv[t, hq + hkv:])
    for name in ("k_codes", "v_codes", "k_meta", "v_meta"):
        got = getattr(cache, name).cpu().numpy()
        want = getattr(host_cache, name)
        assert np.array_equal(got.view(np.int16), want.view(np.int16)), name
    kr, vr = torch.full_like(k_out, 7.0), torch.full_like(k_out, 7.0)
    w4.w4_kv4_read(cache, ints(slots), kr, vr)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < blocks * block)
    for got, want in zip((kr, vr), host_cache.values(slots[live])):
        assert same_bits(host.bits_of(got)[live], ref.round_to_bf16(want))
        assert np.all(host.bf16_values(got)[~live] == 7.0)  # rows without a slot are left


def test_norm_rope_in_place_and_padding():
    """Outputs that are their inputs, inside one fused buffer; rows of negative position are left as they were."""
    T, hq, hkv, dim = 11, 4, 2, 128
    qkv, dev = qk_case(5, T, hq, hkv, dim, 16)
    pos = np.arange(T)
    pos[[3, 10]] = -1
    cs = rope_table(128)
    before = host.bits_of(dev)
    cache = w4.Kv4Cache.empty(3, 16, hkv, dim)
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(5)
    w4.w4_qk_norm_rope(dev[:, :hq], dev[:, hq:hq + hkv], ints(pos), torch.from_numpy(cs).to(DEV), q_out=dev[:, :hq],
                       k_out=dev[:, hq:hq + hkv], v=dev[:, hq + hkv:], cache=cache, slots=ints(np.arange(T)))
    torch.cuda.synchronize()
    live = pos >= 0
    want = ref.norm_rope(qkv[:, :hq + hkv], None, cs, pos, 128, False, 1e-6, 0.0)
    check_queries(host.bf16_values(dev)[live][:, :hq], want[live][:, :hq], "q")
    assert same_bits(host.bits_of(dev)[live][:, hq:hq + hkv], ref.round_to_bf16(want[live][:, hq:]))
    assert same_bits(host.bits_of(dev)[~live], before[~live])
    assert same_bits(host.bits_of(dev)[:, hq + hkv:], before[:, hq + hkv:])
    assert np.all(cache.k_codes.cpu().numpy()[0, :, 3] == 5) and np.all(cache.k_codes.cpu().numpy()[0, :, 11:] == 5)


def test_norm_rope_position_past_the_table_is_nan():
    qkv, dev = qk_case(6, 2, 2, 1, 64, 16)
    q_out, k_out = torch.zeros(2, 2, 64, dtype=bf16, device=DEV), torch.zeros(2, 1, 64, dtype=bf16, device=DEV)
    w4.w4_qk_norm_rope(dev[:, :2], dev[:, 2:3], ints([4, 500]), torch.from_numpy(rope_table(64)).to(DEV), q_out=q_out,
                       k_out=k_out)
    torch.cuda.synchronize()
    assert torch.isfinite(q_out[0]).all() and torch.isnan(q_out[1]).all() and torch.isnan(k_out[1]).all()


def test_keys_alone():
    qkv, dev = qk_case(7, 5, 2, 2, 128, 16)
    k_out = torch.zeros(5, 2, 128, dtype=bf16, device=DEV)
    w4.w4_qk_norm_rope(None, dev[:, 2:4], ints(np.arange(5)), torch.from_numpy(rope_table(128)).to(DEV), k_out=k_out)
    torch.cuda.synchronize()
    want = ref.norm_rope(qkv[:, 2:4], None, rope_table(128), np.arange(5), 128, False, 1e-6, 0.0)
    assert same_bits(host.bits_of(k_out), ref.round_to_bf16(want))


def test_store_of_odd_values():
    """Constant groups, zeros, tiny and huge values, infinities and NaN in some heads: as the format says."""
    T, h, d = 8, 2, 128
    x = si.rng(8, 1).normal(0, 1, (T, h, d))
    x[0] = 0.0
    x[1] = -3.25
    x[2] *= 1e-6
    x[3] *= 1e30
    x[4, 0, 5] = np.inf
    x[5, 1, 127] = np.nan
    x[6] = 1000 + x[6]
    x[7] *= 1e-41
    bits = ref.round_to_bf16(x)
    v_bits = bits[:, ::-1].copy()
    k, v = host.bf16_tensor(bits), host.bf16_tensor(v_bits)
    want = ref.Cache(1, 16, h, d)
    cache = to_device(want)
    w4.w4_qk_norm_rope(None, k, v=v, cache=cache, slots=ints(np.arange(T)))
    torch.cuda.synchronize()
    for t in range(T):
        want.put(t, bits[t], v_bits[t])
    assert np.array_equal(cache.k_codes.cpu().numpy(), want.k_codes)
    assert np.array_equal(cache.v_codes.cpu().numpy(), want.v_codes)
    for name in ("k_meta", "v_meta"):
        assert np.array_equal(getattr(cache, name).cpu().numpy(), getattr(want, name), equal_nan=True)


# ------------------------------------------------------------------ attend
def attn_case(seed, lens, news, hq, hkv, dim, block, spare=2):
    g = si.rng(seed, 44, hq, dim, block)
    need = [-(-max(n, 0) // block) for n in lens]
    blocks = sum(need) + spare
    cache = random_cache(seed, blocks, block, hkv, dim)
    pages = g.permutation(blocks)
    table = np.full((len(lens), max(need + [0]) + 1), 123456789)  # entries past a request's pages are never used
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = pages[at:at + n]
        at += n
    q_start = np.concatenate(([0], np.cumsum(news)))
    T = int(q_start[-1])
    return cache, table, q_start, si.bf16_normal(seed, (45, T, hq, dim), (T, hq, dim))


def run_attn(cache, q_bits, table, lens, q_start, stride_pad=0, tail=0, **kw):
    T, hq, d = q_bits.shape
    space = torch.zeros(T + tail, hq * d + stride_pad, dtype=bf16, device=DEV)
    q = space[:, :hq * d].unflatten(1, (hq, d))
    q[:T] = host.bf16_tensor(q_bits)
    out = torch.full((T + tail, hq, d), 7.0, dtype=bf16, device=DEV)
    max_q = max(int(np.max(np.diff(q_start))), 1) if q_start is not None else 1
    kw.setdefault("max_kv", max(max(lens), 0))
    size = w4.w4_kv4_attn_workspace_bytes(cache, T + tail, len(lens), hq, max_q, kw["max_kv"],
                                          kw.get("window", 0), kw.get("sinks", 0))
    work = torch.full((size // 4,), float("nan"), dtype=torch.float32, device=DEV) if size else None
    w4.w4_kv4_attn(q, cache, ints(table), ints(lens), out, q_start=None if q_start is None else ints(q_start),
                   max_q=max_q, workspace=work, **kw)
    torch.cuda.synchronize()
    return host.bf16_values(out)


def check_attn(got, want, noise, what=""):
    err = np.abs(got - want)
    bad = ~(err <= noise)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outputs, worst {np.nanmax(err / noise):.3g} x the bound"


ATTN = [  # lens, news, hq, hkv, dim, block, window, sinks
    ([1], [1], 16, 8, 256, 64, 0, 0), ([33], [1], 2, 1, 64, 16, 0, 0), ([1000], [1], 16, 8, 256, 64, 1024, 0),
    ([0, 5, 31, 32, 33, 700], [1] * 6, 8, 2, 128, 16, 0, 0),
    ([700, 129, 64], [1] * 3, 64, 8, 64, 16, 100, 4), ([2500], [1], 3, 1, 128, 128, 0, 0),
    ([300, 2100], [1, 1], 20, 1, 128, 64, 64, 200),               # more than 16 heads to a key head
    ([40], [40], 4, 2, 128, 32, 0, 0), ([300], [77], 6, 2, 64, 16, 0, 0),
    ([260, 17, 9, 0], [100, 17, 1, 0], 4, 4, 256, 64, 0, 0),
    ([5, 40], [9, 40], 4, 2, 128, 16, 0, 0),                      # more rows than tokens: rows that see nothing
    ([513, 200], [130, 3], 3, 1, 256, 16, 50, 33), ([150], [150], 5, 5, 64, 256, 1, 1),
    ([20000], [1], 8, 1, 64, 32, 0, 0),
]


@pytest.mark.parametrize("lens,news,hq,hkv,dim,block,window,sinks", ATTN)
def test_attn(lens, news, hq, hkv, dim, block, window, sinks):
    cache, table, q_start, q = attn_case(9, lens, news, hq, hkv, dim, block)
    scale = 1.0 / np.sqrt(dim)
    got = run_attn(to_device(cache), q, table, lens, q_start, window=window, sinks=sinks)
    check_attn(got, *ref.attention(q, cache, table, lens, q_start, float(np.float32(scale)), window, sinks))


def test_attn_is_the_same_for_any_max_kv_and_stride():
    """The split goes by max_kv alone; strided queries; rows behind the last request are left."""
    lens, news = [1500, 64, 900], [1, 2, 1]
    cache, table, q_start, q = attn_case(10, lens, news, 8, 2, 128, 64)
    want, noise = ref.attention(q, cache, table, lens, q_start, 0.5)
    dev = to_device(cache)
    for max_kv in (0, 1, 1500, 100000):
        got = run_attn(dev, q, table, lens, q_start, stride_pad=24, tail=3, max_kv=max_kv, scale=0.5)
        check_attn(got[:4], want, noise, f"max_kv {max_kv}")
        assert np.all(got[4:] == 7.0)


def test_attn_without_q_start_is_one_row_a_request():
    lens = [90, 0, 1, 450]
    cache, table, q_start, q = attn_case(11, lens, [1] * 4, 4, 1, 64, 32)
    dev = to_device(cache)
    a = run_attn(dev, q, table, lens, q_start)
    b = run_attn(dev, q, table, lens, None)
    assert np.array_equal(a, b)
    assert np.all(a[1] == 0)


def test_attn_hidden_garbage_does_not_reach_a_row():
    """NaN and infinite pairs in slots past the end, in tokens before a window and after a row's own."""
    lens, news, window, sinks = [100, 61], [5, 1], 20, 3
    cache, table, q_start, q = attn_case(12, lens, news, 4, 2, 128, 32)
    want, noise = ref.attention(q, cache, table, lens, q_start, 0.1, window, sinks)
    for b, (kv, n) in enumerate(zip(lens, news)):
        seen = np.zeros(len(table[b]) * 32, dtype=bool)
        for i in range(n):
            seen[:kv] |= ref.visible(kv - n + i, kv, window, sinks)
        for j in range(-(-kv // 32) * 32):
            if not seen[j]:
                for meta in (cache.k_meta, cache.v_meta):
                    meta[table[b, j // 32], :, :, j % 32] = [np.nan, np.inf] if j % 2 else [np.inf, -np.inf]
    for page in set(range(cache.blocks)) - set(table[:, :4].ravel()):
        cache.k_meta[page] = cache.v_meta[page] = np.nan
    got = run_attn(to_device(cache), q, table, lens, q_start, window=window, sinks=sinks, scale=0.1)
    check_attn(got, want, noise)
    # the chunk's last token hides from the rows before it
    last = 99
    cache.v_meta[table[0, last // 32], :, :, last % 32] = np.nan
    got = run_attn(to_device(cache), q, table, lens, q_start, window=window, sinks=sinks, scale=0.1)
    assert np.isnan(got[4]).all()
    check_attn(np.delete(got, 4, 0), np.delete(want, 4, 0), np.delete(noise, 4, 0))


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_attn_row_that_sees_a_bad_page_is_nan(bad):
    lens, news = [100, 100], [40, 1]
    cache, table, q_start, q = attn_case(13, lens, news, 2, 1, 128, 32)
    table[0, 2] = bad  # tokens 64 .. 95: rows 4 (position 64) to the last
    want, noise = ref.attention(q, cache, np.where(table == bad, 0, table), lens, q_start, 0.1)
    got = run_attn(to_device(cache), q, table, lens, q_start, scale=0.1)
    assert np.isnan(got[4:40]).all()
    keep = [0, 1, 2, 3, 40]
    check_attn(got[keep], want[keep], noise[keep])


def test_attn_tokens_past_the_table_are_nan():
    cache, table, q_start, q = attn_case(14, [96], [1], 2, 1, 64, 32)
    got = run_attn(to_device(cache), q, table[:, :2], [96], q_start)
    assert np.isnan(got).all()


def test_attn_large_scores():
    """Scores of hundreds: the running maximum moves often and most weights vanish."""
    lens = [900]
    cache, table, q_start, q = attn_case(15, lens, [3], 4, 2, 128, 64)
    got = run_attn(to_device(cache), q, table, lens, q_start, scale=12.0)
    check_attn(got, *ref.attention(q, cache, table, lens, q_start, 12.0))


def test_attn_cache_past_32_bit_offsets():
    """Pages whose bytes lie past 2^32 in the codes and past 2^31 in the pairs."""
    hkv, dim, block = 8, 256, 256
    blocks = (5 << 30) // (hkv * block * dim // 2)
    cache = w4.Kv4Cache.empty(blocks, block, hkv, dim)
    T = 300
    k = host.bf16_tensor(si.bf16_normal(16, (1,), (T, hkv, dim)))
    v = host.bf16_tensor(si.bf16_normal(16, (2,), (T, hkv, dim)))
    pages = np.array([blocks - 1, blocks - 3])
    place = np.arange(T)
    slots = pages[place // block] * block + place % block
    assert slots.max() * hkv * dim // 2 > 2 ** 32
    w4.w4_qk_norm_rope(None, k, v=v, cache=cache, slots=ints(slots))
    small = ref.Cache(2, block, hkv, dim)
    for t in range(T):
        small.put(t, host.bits_of(k[t]), host.bits_of(v[t]))
    kr, vr = torch.empty_like(k), torch.empty_like(v)
    w4.w4_kv4_read(cache, ints(slots), kr, vr)
    q = si.bf16_normal(16, (3,), (1, 16, dim))
    got = run_attn(cache, q, pages[None], [T], np.array([0, 1]))
    for a, b in zip((kr, vr), small.values(place)):
        assert same_bits(host.bits_of(a), ref.round_to_bf16(b))
    check_attn(got, *ref.attention(q, small, np.array([[0, 1]]), [T], [0, 1], 1 / 16))


# ------------------------------------------------------------------ sample
def run_sample(bits, u, stride_pad=0, shift=0, **kw):
    rows, vocab = bits.shape
    space = torch.zeros(rows * (vocab + stride_pad) + shift + 8, dtype=bf16, device=DEV)
    logits = torch.as_strided(space, (rows, vocab), (vocab + stride_pad, 1), shift)
    logits.copy_(host.bf16_tensor(bits))
    tokens = torch.full((rows,), -77, dtype=i32, device=DEV)
    size = w4.w4_sample_workspace_bytes(rows, vocab)
    work = torch.full((size // 4,), -1, dtype=i32, device=DEV) if size else None
    dev = {k: torch.tensor(np.asarray(v), dtype=i32 if k == "top_k" else torch.float32, device=DEV) for k, v in kw.items()}
    w4.w4_sample(logits, torch.tensor(u, dtype=torch.float64, device=DEV), tokens, workspace=work, **dev)
    torch.cuda.synchronize()
    return tokens.cpu().numpy()


SETTINGS = [dict(), dict(temperature=0.7), dict(temperature=0.0), dict(top_k=1), dict(top_k=7), dict(top_p=0.9),
            dict(top_p=0.0), dict(min_p=0.05), dict(min_p=1.0), dict(temperature=1.5, top_k=50, top_p=0.8, min_p=0.01),
            dict(top_k=10 ** 6, top_p=0.5), dict(temperature=1e-4), dict(temperature=30.0, top_p=0.999)]
DEFAULT = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)


@pytest.mark.parametrize("vocab,pad,shift", [(1, 0, 0), (2, 5, 1), (100, 0, 3), (1000, 1, 0), (32768, 0, 0),
                                             (32769, 7, 5), (262144, 0, 0), (70001, 0, 1)])
def test_sample(vocab, pad, shift):
    """Every setting in one call, a row each, at rows of any alignment; the token is the oracle's."""
    g = si.rng(17, vocab)
    rows = len(SETTINGS) * 2
    bits = ref.round_to_bf16(g.normal(0, 3, (rows, vocab)))
    u = g.random(rows)
    u[0] = 0.0
    each = [{**DEFAULT, **SETTINGS[r % len(SETTINGS)]} for r in range(rows)]
    got = run_sample(bits, u, pad, shift, **{k: [e[k] for e in each] for k in DEFAULT})
    want = [ref.sample(bits[r], u[r], **each[r]) for r in range(rows)]
    assert got.tolist() == want


def test_sample_without_settings():
    g = si.rng(18, 1)
    bits, u = ref.round_to_bf16(g.normal(0, 2, (3, 5000))), g.random(3)
    assert run_sample(bits, u).tolist() == [ref.sample(b, x) for b, x in zip(bits, u)]


def test_sample_ties_and_odd_logits():
    """Equal logits go by index; -0 and +0 are equal; NaN, infinities, rows of nothing."""
    inf, nan = np.inf, np.nan
    rows = [([1.0] * 8, 0.5, {}), ([1.0] * 8, 0.999, dict(top_p=0.5)), ([1.0] * 8, 0.99, dict(top_k=3)),
            ([0.0, -0.0, 0.0, -0.0] * 2, 0.3, {}), ([-inf] * 8, 0.3, {}), ([nan] * 8, 0.3, {}),
            ([nan, 1.0, -inf, 2.0, nan, 0.5, -inf, 1.5], 0.7, {}), ([5.0, inf, 3.0, inf, inf, 1.0, 0.0, -1.0], 0.5, {}),
            ([-inf, -inf, -3.0, -inf, -inf, -inf, -inf, -inf], 0.99, dict(top_p=0.3)),
            ([2.0, 1.0, 2.0, 1.0, 2.0, 1.0, 2.0, 1.0], 0.6, dict(temperature=0.0)),
            ([3e38, -3e38, 3e38, 0, 0, 0, 0, 0], 0.75, {}), ([1e-40, 0, 0, 0, 0, 0, 0, 0], 0.9, dict(temperature=1e-38)),
            ([0.0, -200.0, -200.0, -200.0, -900.0, -900.0, -900.0, -900.0], 1.0, {})]
    bits = ref.round_to_bf16(np.array([r[0] for r in rows], dtype=np.float64))
    u = np.array([r[1] for r in rows])
    each = [{**DEFAULT, **r[2]} for r in rows]
    got = run_sample(bits, u, **{k: [e[k] for e in each] for k in DEFAULT})
    assert got.tolist() == [ref.sample(bits[r], u[r], **each[r]) for r in range(len(rows))]


def test_sample_follows_the_weights():
    """4096 rows of one distribution: every token's share within five standard deviations."""
    p = np.array([0.5, 0.25, 0.125, 0.125])
    bits = np.tile(ref.round_to_bf16(np.log2(p) * 1.0), (4096, 1))  # weights 2^x at temperature 1 / ln 2
    heat = np.full(4096, 1.0 / np.log(2.0))
    got = run_sample(bits, si.rng(19, 1).random(4096), temperature=heat)
    share = np.bincount(got, minlength=4) / 4096
    assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / 4096))


# ------------------------------------------------- together, graphs, streams
class Step:
    """Plan, store, attend and sample of one decode step over static buffers."""

    def __init__(self, seed, lens, block=16, hq=8, hkv=2, dim=128, vocab=3000):
        g = si.rng(seed, 50)
        self.hq, self.hkv, self.dim, self.block, B = hq, hkv, dim, block, len(lens)
        width = -(-max(lens) // block) + 2
        held = [-(-n // block) for n in lens]
        blocks = sum(held) + 2 * B
        self.host = random_cache(seed, blocks, block, hkv, dim)
        self.cache = to_device(self.host)
        pages = g.permutation(blocks)
        table = np.full((B, width), -1)
        at = 0
        for b in range(B):
            table[b, :held[b]] = pages[at:at + held[b]]
            at += held[b]
        self.table, self.free, self.count = ints(table), ints(pages[at:]), ints([blocks - at])
        self.cached, self.new = ints(lens), ints([1] * B)
        self.q_start, self.kv = torch.zeros(B + 1, dtype=i32, device=DEV), torch.zeros(B, dtype=i32, device=DEV)
        self.pos, self.slots = (torch.zeros(B + 2, dtype=i32, device=DEV) for _ in range(2))
        self.counts = torch.zeros(2, dtype=i32, device=DEV)
        self.qkv_bits = si.bf16_normal(seed, (51,), (B + 2, hq + 2 * hkv, dim))
        self.qkv = host.bf16_tensor(self.qkv_bits)
        self.cs = rope_table(dim, 3000)
        self.cs_dev = torch.from_numpy(self.cs).to(DEV)
        self.q = torch.zeros(B + 2, hq, dim, dtype=bf16, device=DEV)
        self.out = torch.zeros(B + 2, hq, dim, dtype=bf16, device=DEV)
        self.logits = host.bf16_tensor(ref.round_to_bf16(g.normal(0, 3, (B, vocab))))
        self.u = torch.tensor(g.random(B), dtype=torch.float64, device=DEV)
        self.tokens = torch.zeros(B, dtype=i32, device=DEV)
        self.reach = width * block
        n = w4.w4_kv4_attn_workspace_bytes(self.cache, B + 2, B, hq, 1, self.reach)
        self.work = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        self.swork = torch.empty(w4.w4_sample_workspace_bytes(B, vocab), dtype=torch.uint8, device=DEV)

    def run(self, stream=None):
        s = dict(stream=stream)
        w4.w4_kv4_plan(self.cached, self.new, self.table, self.free, self.count, self.block, self.q_start, self.kv,
                       self.pos, self.slots, self.counts, **s)
        q, k, v = self.qkv[:, :self.hq], self.qkv[:, self.hq:self.hq + self.hkv], self.qkv[:, self.hq + self.hkv:]
        w4.w4_qk_norm_rope(q, k, self.pos, self.cs_dev, q_out=self.q, v=v, cache=self.cache, slots=self.slots, **s)
        w4.w4_kv4_attn(self.q, self.cache, self.table, self.kv, self.out, q_start=self.q_start, max_q=1,
                       max_kv=self.reach, workspace=self.work, **s)
        w4.w4_sample(self.logits, self.u, self.tokens, workspace=self.swork, **s)

    def outputs(self):
        torch.cuda.synchronize()
        return [host.bits_of(self.out), self.tokens.cpu().numpy(), self.slots.cpu().numpy(), self.table.cpu().numpy(),
                self.cache.k_codes.cpu().numpy(), self.cache.v_codes.cpu().numpy()]


def test_step_together():
    """Tables, store, attention and sampling in a row, each fed by the one before, against the oracle; padding rows last."""
    lens = [0, 5, 16, 700, 33]
    s = Step(20, lens)
    table0 = s.table.cpu().numpy()
    s.run()
    out, tokens, slots, table, _, _ = s.outputs()
    want = ref.plan(lens, [1] * 5, table0, s.free.cpu().numpy(), int(s.count), 16, 7)
    assert slots.tolist() == list(want[3]) and np.array_equal(table, want[4])
    B, hq, hkv = 5, s.hq, s.hkv
    k_bits = ref.round_to_bf16(ref.norm_rope(s.qkv_bits[:B, hq:hq + hkv], None, s.cs, want[2][:B], s.dim, False, 1e-6, 0))
    for b in range(B):
        s.host.put(slots[b], k_bits[b], s.qkv_bits[b, hq + hkv:])
    q = host.bits_of(s.q)[:B]
    check_queries(host.bf16_values(s.q)[:B], ref.norm_rope(s.qkv_bits[:B, :hq], None, s.cs, want[2][:B], s.dim, False, 1e-6, 0), "q")
    o, noise = ref.attention(q, s.host, table, want[1], want[0], float(np.float32(128 ** -0.5)))
    check_attn(oracle.bf16_to_f64(out[:B]), o, noise)
    assert np.all(out[B:] == 0)
    assert tokens.tolist() == [ref.sample(host.bits_of(s.logits)[b], float(s.u[b])) for b in range(B)]


def test_step_graph_replays():
    """The step captured in a graph and replayed four times with other eager work between, its inputs
    changed in place for each replay: every replay equals an eager run of a copy."""
    lens = [3, 40, 900]
    a, b = Step(21, lens), Step(21, lens)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    w4.w4_graph_begin(stream)
    try:
        a.run(stream=stream)
    finally:
        graph = w4.w4_graph_end(stream)
    for rep in range(4):
        bits = si.bf16_normal(22, (rep,), a.qkv_bits.shape)
        for s in (a, b):
            s.qkv.copy_(host.bf16_tensor(bits))
            s.u.fill_(0.1 + 0.2 * rep)
            s.cached.add_(1)
        torch.cuda.synchronize()
        graph.replay(stream)
        stream.synchronize()
        b.run()
        b.run()  # other eager work on the same cache changes nothing
        for x, y in zip(a.outputs(), b.outputs()):
            assert np.array_equal(x, y), rep
    graph.destroy()


def test_two_graphs_in_turn():
    """Two captured steps of different sizes, each with its own buffers, replayed in turn on one stream."""
    steps = [Step(23, [5, 300]), Step(24, [1200])]
    eager = [Step(23, [5, 300]), Step(24, [1200])]
    stream = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for s in steps:
        w4.w4_graph_begin(stream)
        try:
            s.run(stream=stream)
        finally:
            graphs.append(w4.w4_graph_end(stream))
    for _ in range(3):
        for g in graphs:
            g.replay(stream)
    stream.synchronize()
    for s, e in zip(steps, eager):
        e.run()
        for x, y in zip(s.outputs(), e.outputs()):
            assert np.array_equal(x, y)
    for g in graphs:
        g.destroy()


def test_two_streams_at_once():
    """Steps on two streams, with their own buffers, at once: the same bits as one after the other."""
    steps = [Step(25, [700, 20]), Step(26, [90, 1500, 4])]
    eager = [Step(25, [700, 20]), Step(26, [90, 1500, 4])]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(steps, streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    for s, e in zip(steps, eager):
        e.run()
        for x, y in zip(s.outputs(), e.outputs()):
            assert np.array_equal(x, y)
