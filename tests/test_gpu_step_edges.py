"""GPU: values and sizes at which the decode step's operators could go wrong, against the FP64 oracle.

Tolerances are those of ``test_gpu_step.py``: keys, codes and pairs equal bit for bit, queries within one rounding
to BF16 and FP32 arithmetic, attention within ``noise`` of ``oracle.step.attention``.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import seeded_inputs as si
from gemm_w4_gemv_amd.decode import DecodeStep
from oracle import step as ref
from test_gpu_step import DEV, attn_case, bf16, check_attn, check_queries, host, ints, rope_table, same_bits, to_device, w4
from test_gpu_decode_attention import build, feed
from test_gpu_step_paths import MANY, TWO_PARTS, attn, many

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


# ------------------------------------------------------------- stored keys
def check_cache(cache, want):
    for name in ("k_codes", "v_codes", "k_meta", "v_meta"):
        got, w = getattr(cache, name).cpu().numpy(), getattr(want, name)
        assert np.array_equal(got.view(np.int16), w.view(np.int16)), name


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_keys_go_to_bf16_through_fp32(dim, inter):
    """Rotations that end 2^-30 beside the middle between two BF16 values: FP32 drops that, and the tie goes to
    the even one.  Rounded at once from FP64 half of them would go the other way."""
    half, T, h = dim // 2, 8, 3
    cs = np.zeros((T, dim), dtype=np.float32)
    for t in range(T):
        cs[t, :half] = 1 + (2 * t + 1) * 2.0 ** -8  # the middles above 1
        cs[t, half:] = 2.0 ** -30 * (-1) ** np.arange(half)
    bits = ref.round_to_bf16(np.ones((T, h, dim)))
    y = ref.norm_rope(bits, None, cs, np.arange(T), dim, inter, 1e-6, 0.0)
    k_bits = ref.round_to_bf16(y)
    # what a single rounding gives: ties broken by the part that FP32 cannot hold
    low = (y.astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)
    once = np.where(y - low > 2.0 ** -8, low + 2.0 ** -7, low)
    assert bool(np.any(once != oracle.bf16_to_f64(k_bits)))
    k, v = host.bf16_tensor(bits), host.bf16_tensor(si.bf16_normal(80, (1, dim), (T, h, dim)))
    want = ref.Cache(1, 16, h, dim)
    cache = w4.Kv4Cache(*(torch.from_numpy(a.copy()).to(DEV) for a in (want.k_codes, want.k_meta, want.v_codes, want.v_meta)))
    k_out = torch.zeros_like(k)
    w4.w4_qk_norm_rope(None, k, ints(np.arange(T)), torch.from_numpy(cs).to(DEV), k_out=k_out, v=v, cache=cache,
                       slots=ints(np.arange(T)), interleaved=inter)
    torch.cuda.synchronize()
    assert same_bits(host.bits_of(k_out), k_bits)
    for t in range(T):
        want.put(t, k_bits[t], host.bits_of(v[t]))
    check_cache(cache, want)


def test_prompt_store_bit_for_bit():
    """A prompt's 4099 tokens, 8 heads of 256, pages in any order: every key, code and pair is the oracle's."""
    T, h, dim, block = 4099, 8, 256, 64
    x, w = si.bf16_normal(81, (1,), (2, T, h, dim)), si.bf16_normal(81, (2,), (dim,))
    cs, pos = rope_table(dim, 5000), np.arange(T) + 17
    y = oracle.bf16_to_f64(x[0])
    y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + float(np.float32(1e-6))) * oracle.bf16_to_f64(w)
    c, s = (cs[pos, at:at + dim // 2].astype(np.float64)[:, None] for at in (0, dim // 2))
    a, b = y[..., :dim // 2], y[..., dim // 2:]
    k_bits = ref.round_to_bf16(np.concatenate((a * c - b * s, b * c + a * s), axis=-1))
    pages = si.rng(81, 3).permutation(-(-T // block) + 3)
    place = np.arange(T)
    slots = pages[place // block] * block + place % block
    want = ref.Cache(len(pages), block, h, dim)
    p, o = pages[place // block], place % block
    q, want.k_meta[p, :, :, o] = ref.quantise(k_bits)
    want.k_codes[p, :, o] = ref.pack(q)
    q, want.v_meta[p, :, :, o] = ref.quantise(x[1])
    want.v_codes[p, :, o // 4, :, o % 4] = ref.pack(q)
    cache = w4.Kv4Cache(*(torch.from_numpy(np.zeros_like(t)).to(DEV) for t in (want.k_codes, want.k_meta, want.v_codes, want.v_meta)))
    k, v = host.bf16_tensor(x[0]), host.bf16_tensor(x[1])
    k_out = torch.zeros_like(k)
    w4.w4_qk_norm_rope(None, k, ints(pos), torch.from_numpy(cs).to(DEV), k_out=k_out, k_weight=host.bf16_tensor(w), v=v,
                       cache=cache, slots=ints(slots))
    torch.cuda.synchronize()
    assert same_bits(host.bits_of(k_out), k_bits)
    check_cache(cache, want)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scales_go_to_fp16_through_fp32(dim):
    """Groups whose span over 15 is, in FP32, the middle between two FP16 values: the tie goes to the even one.
    The product of the span and fp32(1/15) lies above it, so rounded at once it would go up."""
    pairs = []
    for n in range(2049, 2345, 4):  # of twelve bits, the even neighbour below
        for high in np.arange(128, 256) * 128.0:
            low = high - 15 * n
            if low <= 0 and oracle.bf16_to_f64(ref.round_to_bf16(low)) == low:
                pairs.append((low, high))
    assert len(pairs) >= 8
    T, groups, size = len(pairs), max(1, dim // 128), min(dim, 128)
    x = np.zeros((T, 1, groups, size))
    g = si.rng(82, dim)
    for t, (low, high) in enumerate(pairs):
        x[t] = g.uniform(low, high, (1, groups, size))
        x[t, ..., 3], x[t, ..., size - 2] = low, high
    bits = ref.round_to_bf16(x.reshape(T, 1, dim))
    q, meta = ref.quantise(bits)
    span = np.array([h - lo for lo, h in pairs])
    once = (span * float(np.float32(1 / 15))).astype(np.float16)
    assert np.all(once != meta[:, 0, 0, 0])
    want = ref.Cache(-(-T // 16), 16, 1, dim)
    cache = w4.Kv4Cache(*(torch.from_numpy(a.copy()).to(DEV) for a in (want.k_codes, want.k_meta, want.v_codes, want.v_meta)))
    k = host.bf16_tensor(bits)
    w4.w4_qk_norm_rope(None, k, v=k, cache=cache, slots=ints(np.arange(T)))
    torch.cuda.synchronize()
    for t in range(T):
        want.put(t, bits[t], bits[t])
    check_cache(cache, want)


# ----------------------------------------------------------------- queries
FAR = [(1e20, 1e-6), (3e36, 1e-6), (1e-12, 0.0), (1e-25, 0.0), (1e-38, 0.0), (1e-30, 1e-6), (0.0, 1e-6), (1e3, 1e30), (1.0, 1e-6)]


@pytest.mark.parametrize("inter,rot,weight", [(False, 1, 1.0), (True, 0.5, 1.0), (False, 0, 1e30), (True, 1, 1e-30), (False, 1, 1e38)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_queries_of_any_size(dim, inter, rot, weight):
    """Queries whose squares leave FP32's range, above and below, beside ordinary ones of the same row; norm
    weights at its ends.  A row's ordinary queries keep their bits whatever stands beside them."""
    T, h, rot = 5, 7, int(rot * dim)
    w = ref.round_to_bf16(oracle.bf16_to_f64(si.bf16_normal(83, (1, dim), (dim,))) * weight)
    w[:4] = ref.round_to_bf16([0.5, 1.0, -2.0, 0.0])
    base = oracle.bf16_to_f64(si.bf16_normal(83, (2, dim), (T, h, dim)))
    cs, pos = rope_table(rot) if rot else None, np.arange(T) * 90
    plain = None
    for size, eps in [(1.0, 1e-6)] + FAR:
        x = base.copy()
        x[1, 2:4] *= size
        x[2] *= size
        x[4, ::2] *= -size
        bits = ref.round_to_bf16(x)
        with np.errstate(all="ignore"):
            want = ref.norm_rope(bits, w, cs, pos, rot, inter, eps, 0.0)
        q, k_out = torch.zeros(T, h, dim, dtype=bf16, device=DEV), torch.zeros(T, 1, dim, dtype=bf16, device=DEV)
        w4.w4_qk_norm_rope(host.bf16_tensor(bits), host.bf16_tensor(bits[:, :1]), ints(pos) if rot else None,
                           torch.from_numpy(cs).to(DEV) if rot else None, q_out=q, k_out=k_out, q_weight=host.bf16_tensor(w),
                           k_weight=host.bf16_tensor(w), eps=eps, interleaved=inter)
        torch.cuda.synchronize()
        keys = oracle.bf16_to_f64(ref.round_to_bf16(want[:, :1]))  # as numbers: a zero weight's zeros have either sign
        assert np.array_equal(host.bf16_values(k_out), keys, equal_nan=True)
        got = host.bf16_values(q)
        # results past BF16's range, and what is 0 / 0, are what the definition makes of them
        top = np.abs(want) >= 3.38e38
        tiny = np.abs(want) < 1e-37  # BF16's last bits there are steps of 2^-133
        assert np.array_equal(np.isnan(got), np.isnan(want)), (size, eps)
        assert np.all(np.abs(got[top]) >= 3.376e38)  # the nearest BF16 to 3.38e38
        sound = ~(top | tiny | np.isnan(want))
        check_queries(np.where(sound, got, 0.0), np.where(sound, want, 0.0), (size, eps))
        assert np.all(np.abs(got - want)[tiny] <= 2.0 ** -8 * np.abs(want)[tiny] + 2.0 ** -133)
        if size == 1.0 and eps == 1e-6:
            plain = host.bits_of(q) if plain is None else plain
            assert same_bits(host.bits_of(q), plain)
        elif eps == 1e-6:
            keep = np.ones((T, h), dtype=bool)
            keep[1, 2:4] = keep[2] = keep[4, ::2] = False
            assert same_bits(host.bits_of(q)[keep], plain[keep])


# -------------------------------------------------- queries of any size, again
@pytest.mark.parametrize("T,h,dim,inter", [(9, 21, 256, False), (8200, 21, 256, True), (8200, 9, 128, False), (3, 40, 64, True)])
def test_far_queries_in_place(T, h, dim, inter):
    """Outputs over their inputs, with few and with many tokens (runs of heads in waves of their own, and in turn in one):
    the same bits as with outputs apart; infinities and NaN as the definition has them."""
    x = oracle.bf16_to_f64(si.bf16_normal(86, (1, T, h), (T, h + 1, dim))).copy()
    x[1, ::3] *= 1e25
    x[T - 1, 1::2] *= 1e-30
    x[2, h - 1] *= 1e38 / 8
    x[0, 2, 5], x[0, 4, 7], x[0, 4, 8] = np.inf, np.nan, -np.inf
    bits = ref.round_to_bf16(x)
    w = si.bf16_normal(86, (2, dim), (dim,))
    cs, pos = rope_table(dim, 500), np.arange(T) % 500
    args = (ints(pos), torch.from_numpy(cs).to(DEV))
    kw = dict(q_weight=host.bf16_tensor(w), k_weight=host.bf16_tensor(w), interleaved=inter)
    both = host.bf16_tensor(bits)
    apart, k_out = torch.zeros(T, h, dim, dtype=bf16, device=DEV), torch.zeros(T, 1, dim, dtype=bf16, device=DEV)
    w4.w4_qk_norm_rope(both[:, :h], both[:, h:], *args, q_out=apart, k_out=k_out, **kw)
    w4.w4_qk_norm_rope(both[:, :h], both[:, h:], *args, q_out=both[:, :h], k_out=both[:, h:], **kw)
    torch.cuda.synchronize()
    assert same_bits(host.bits_of(both[:, :h]), host.bits_of(apart)) and same_bits(host.bits_of(both[:, h:]), host.bits_of(k_out))
    at = [0, 1, 2, T - 1]
    with np.errstate(all="ignore"):
        want = ref.norm_rope(bits[at], w, cs, pos[at], dim, inter, 1e-6, 0.0)[:, :h]
    got = host.bf16_values(apart[at])
    assert np.array_equal(np.isnan(got), np.isnan(want))
    sound = ~np.isnan(want)
    check_queries(np.where(sound, got, 0.0), np.where(sound, want, 0.0), "q")


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 3), (2 ** 31 - 20, 0), (2 ** 31 - 64, 2 ** 31 - 1)])
@pytest.mark.parametrize("dim,B,rows,block", [(256, 56, 64, 64), (128, 56, 128, 16), (64, 128, 128, 32), (256, 3, 40, 16), (64, 2, 5, 16)])
def test_window_of_everything_with_more_rows_than_tokens(dim, B, rows, block, window, sinks):
    """Rows before the first token beside a window near 2^31: what the others see is not passed over."""
    heads, tokens = 8, max(rows - 10, rows // 2)
    lens, news = [tokens] * B, [rows] * B
    cache, table, q_start, q = attn_case(84, lens, news, heads, heads, dim, block)
    got = attn(to_device(cache), q, table, lens, q_start, rows, window=window, sinks=sinks, scale=0.1)
    hidden = rows - tokens
    for b in sorted({0, B // 2, B - 1}):
        at = slice(b * rows, (b + 1) * rows)
        assert np.all(got[at][:hidden] == 0)
        check_attn(got[at], *ref.attention(q[at], cache, table[b:b + 1], [tokens], [0, rows], 0.1), f"request {b}")


@pytest.mark.parametrize("lens,news,hq,hkv,dim,block,window,sinks", MANY)
def test_prompts_are_as_exact_as_few_rows(lens, news, hq, hkv, dim, block, window, sinks):
    """Weights keep 16 bits in calls for long prompts too: a request's rounding does not go by the company it is in."""
    cache, table, q_start, q = attn_case(61, lens, news, hq, hkv, dim, block)
    got = attn(to_device(cache), q, table, lens, q_start, many(hq, hkv), window=window, sinks=sinks)
    check_attn(got, *ref.attention(q, cache, table, lens, q_start, float(np.float32(dim ** -0.5)), window, sinks, TWO_PARTS))


# ----------------------------------------------------------- empty problems
def test_a_step_without_rows():
    """What w4_kv4_plan gives when every request rests, through the binding: no rows, nothing written, no error."""
    cache = w4.Kv4Cache.empty(2, 16, 2, 128)
    empty = lambda *shape: torch.zeros(*shape, dtype=bf16, device=DEV)  # noqa: E731
    none = ints([])
    q, k, out = empty(0, 4, 128), empty(0, 2, 128), empty(0, 4, 128)
    table, lens = ints([[0, 1]]), ints([20])
    q_start, kv_lens, counts = ints([7, 7]), ints([7]), ints([7, 7])
    w4.w4_kv4_plan(lens, ints([0]), table, none, ints([0]), 16, q_start, kv_lens, none, none, counts)
    w4.w4_qk_norm_rope(q, k, none, torch.from_numpy(rope_table(128)).to(DEV), q_out=q, v=k, cache=cache, slots=none)
    w4.w4_qk_norm_rope(q, k, q_out=q, k_out=k)
    w4.w4_kv4_read(cache, none, k, k.clone())
    assert w4.w4_kv4_attn(q, cache, table, lens, out, q_start=q_start) is out
    w4.w4_kv4_attn(q, cache, table[:0], lens[:0], out)
    tokens = ints([])
    assert w4.w4_sample(empty(0, 50000), torch.zeros(0, dtype=torch.float64, device=DEV), tokens) is tokens
    torch.cuda.synchronize()
    assert q_start.tolist() == [0, 0] and kv_lens.tolist() == [20] and counts.tolist() == [0, 0]


# ------------------------------------------------------------- launch sizes
def test_the_largest_call():
    """As many tokens as a launch counts work-items for: the first and the last are done like any others."""
    T, dim = 2 ** 26 - 4, 64
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("less than 24 GiB of memory is free")
    x = si.bf16_normal(85, (1,), (8, 1, dim))
    w = si.bf16_normal(85, (2,), (dim,))
    k = torch.zeros(T, 1, dim, dtype=bf16, device=DEV)
    k[:4], k[-4:] = host.bf16_tensor(x[:4]), host.bf16_tensor(x[4:])
    out = torch.full_like(k, 7.0)
    w4.w4_qk_norm_rope(None, k, k_out=out, k_weight=host.bf16_tensor(w))
    torch.cuda.synchronize()
    want = ref.round_to_bf16(ref.norm_rope(x, w, None, None, 0, False, 1e-6, 0.0))
    assert same_bits(host.bits_of(out[:4]), want[:4]) and same_bits(host.bits_of(out[-4:]), want[4:])
    assert int(torch.count_nonzero(out[4:-4])) == 0


# --------------------------------------------------------------- decode step
@pytest.mark.parametrize("order", [("v", "k", "q"), ("k", "v", "q"), ("q", "v", "k")])
def test_decode_step_in_any_order_of_q_k_and_v(order):
    """The attention of a layer runs when its three outputs are there, whichever comes last: same bits, also captured."""
    a, b = build(32)[0], build(32)[0]
    first = {"q": order[0], "k": order[1], "v": order[2]}
    by = {(lin["layer"], lin["name"]): lin for lin in b.linears}
    b.linears = [by[lin["layer"], first.get(lin["name"], lin["name"])] for lin in b.linears]
    c = DecodeStep(b.linears, attention=b.attention, sampler=b.sampler)
    assert len({lin["x"].data_ptr() for lin in b.linears[:3]}) == 1
    for t in range(6):
        for s in (a, b):
            feed(s, t)  # into the input that layer 0's three share
        a.run_eager()
        c.replay() if t % 2 else c.run_eager()
        torch.cuda.synchronize()
        for lin in a.linears:
            other = by[lin["layer"], lin["name"]]
            assert torch.equal(lin["y"].view(torch.int16), other["y"].view(torch.int16)), (t, lin["layer"], lin["name"])
        assert torch.equal(a.attention.out.view(torch.int16), b.attention.out.view(torch.int16))
        assert int(a.sampler.tokens) == int(b.sampler.tokens)
    c.destroy()


