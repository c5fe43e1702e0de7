"""Each way a call of the decode step's operators can be cut, at the cases where one can go wrong.

Attention has a kernel for up to 8 rows of a key/value head, one for up to a
few thousand and one for long prompts (chosen by the sizes of the call, of
which ``max_q`` may be larger than any request), each with tokens of one page
or two in a tile.  Tolerances are those of ``test_gpu_step.py``; where a
weight is kept in two BF16 parts its rounding is off by 2^-16 of it (2^-8 of
what the first left, which is 2^-8), not 2^-8.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle  # noqa: F401
import seeded_inputs as si
from oracle import step as ref
from test_gpu_step import (DEV, attn_case, check_attn, host, i32, ints, random_cache, run_sample, to_device, w4)

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16
TWO_PARTS = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def attn(cache, q_bits, table, lens, q_start, max_q, **kw):
    T, hq, d = q_bits.shape
    out = torch.full((T, hq, d), 7.0, dtype=bf16, device=DEV)
    kw.setdefault("max_kv", max(max(lens), 0))
    size = w4.w4_kv4_attn_workspace_bytes(cache, T, len(lens), hq, max_q, kw["max_kv"], kw.get("window", 0),
                                          kw.get("sinks", 0))
    work = torch.full((size // 4,), float("nan"), dtype=torch.float32, device=DEV) if size else None
    w4.w4_kv4_attn(host.bf16_tensor(q_bits), cache, ints(table), ints(lens), out, q_start=ints(q_start), max_q=max_q,
                   workspace=work, **kw)
    torch.cuda.synchronize()
    return host.bf16_values(out)


# Rows of a key/value head that put a call on the kernel for long prompts:
# 1024 workgroups of 64 or 128 rows, most of which find no rows.
def many(hq, hkv):
    return 1024 * 128 * hkv // hq


FEW = [  # lens, news, hq, hkv, dim, block, window, sinks: 2 and 4 sets of columns, and none
    ([1], [1], 1, 1, 64, 16, 0, 0), ([2], [1], 4, 1, 128, 64, 0, 0), ([17, 40], [1, 1], 5, 1, 128, 16, 0, 0),
    ([1, 2, 31, 0, 65, 130], [1] * 6, 8, 1, 64, 32, 0, 0), ([600, 7], [2, 1], 8, 2, 256, 16, 0, 0),
    ([600, 7], [2, 1], 8, 2, 256, 64, 0, 0), ([129, 300], [1, 1], 6, 2, 256, 32, 40, 5),
    ([1100, 64], [1, 4], 2, 1, 64, 16, 200, 70), ([2100], [1], 7, 1, 128, 16, 1000, 1), ([4000, 1, 900], [1] * 3, 16, 8, 256, 64, 0, 0),
    ([3, 50], [3, 4], 9, 3, 64, 64, 3, 0), ([40, 3], [20, 3], 8, 2, 256, 16, 0, 0), ([999], [33], 4, 4, 128, 32, 100, 100),
]


@pytest.mark.parametrize("lens,news,hq,hkv,dim,block,window,sinks", FEW)
def test_few_rows(lens, news, hq, hkv, dim, block, window, sinks):
    cache, table, q_start, q = attn_case(60, lens, news, hq, hkv, dim, block)
    got = attn(to_device(cache), q, table, lens, q_start, max(news), window=window, sinks=sinks)
    check_attn(got, *ref.attention(q, cache, table, lens, q_start, float(np.float32(dim ** -0.5)), window, sinks, TWO_PARTS))


MANY = [
    ([1], [1], 8, 8, 256, 64, 0, 0), ([150], [150], 4, 2, 128, 16, 0, 0), ([300, 70, 0, 9], [100, 70, 0, 1], 4, 2, 128, 64, 0, 0),
    ([513, 200], [130, 3], 3, 1, 256, 16, 50, 33), ([260, 17], [100, 17], 8, 8, 256, 64, 0, 0),
    ([400], [260], 2, 2, 64, 32, 100, 4), ([90], [90], 8, 1, 64, 16, 0, 0), ([5, 40], [9, 40], 4, 2, 256, 128, 0, 0),
    ([33, 300], [33, 20], 16, 2, 128, 32, 1, 1),
]


@pytest.mark.parametrize("lens,news,hq,hkv,dim,block,window,sinks", MANY)
def test_many_rows(lens, news, hq, hkv, dim, block, window, sinks):
    cache, table, q_start, q = attn_case(61, lens, news, hq, hkv, dim, block)
    got = attn(to_device(cache), q, table, lens, q_start, many(hq, hkv), window=window, sinks=sinks)
    check_attn(got, *ref.attention(q, cache, table, lens, q_start, float(np.float32(dim ** -0.5)), window, sinks))


@pytest.mark.parametrize("lens,news,hq,hkv,block,window,sinks", [
    ([1], [1], 8, 8, 64, 0, 0), ([150], [150], 4, 2, 16, 0, 0), ([300, 70, 0, 9], [100, 70, 0, 1], 4, 2, 64, 0, 0),
    ([513, 200], [130, 3], 3, 1, 16, 50, 33), ([5, 40], [9, 40], 4, 2, 128, 0, 0), ([33, 300], [33, 20], 16, 2, 32, 1, 1),
])
def test_rows_by_32(lens, news, hq, hkv, block, window, sinks):
    """Heads of 128 with room for 768 workgroups of 32 rows, and for fewer than 448 of 128."""
    cache, table, q_start, q = attn_case(77, lens, news, hq, hkv, 128, block)
    max_q = 32 * (800 // (len(lens) * hkv) + 1) * hkv // hq
    assert max_q >= max(news)
    got = attn(to_device(cache), q, table, lens, q_start, max_q, window=window, sinks=sinks)
    check_attn(got, *ref.attention(q, cache, table, lens, q_start, float(np.float32(128 ** -0.5)), window, sinks, TWO_PARTS))


@pytest.mark.parametrize("rows,heads", [(57 * 64, 8), (60 * 64 - 5, 8), (64 * 64, 8)])
def test_many_rows_that_fill_the_chip_once(rows, heads):
    """Up to 512 workgroups the row tiles go in pairs, an odd one too: every row is answered once."""
    g, dim = 8, 256
    n = -(-rows // g)
    cache, table, q_start, q = attn_case(62, [n], [n], heads * g, heads, dim, 64)
    got = attn(to_device(cache), q, table, [n], q_start, n)
    # a sample of rows, each row tile's first and last among them
    at = sorted({0, n - 1} | {min(64 // g * i + j, n - 1) for i in range(-(-rows // 64)) for j in (0, 64 // g - 1)})
    for t in at:
        # the row alone, as the last of a shorter context
        want, noise = ref.attention(q[t:t + 1, ::g], cache, table, [t + 1], [0, 1], float(np.float32(dim ** -0.5)))
        check_attn(got[t:t + 1, ::g], want, noise, f"row {t}")
    assert not np.any(got == 7.0)


KINDS = [("few", 4, 2, 64, 16), ("few", 4, 2, 128, 64), ("few", 4, 2, 256, 16), ("few", 16, 1, 128, 32),
         ("many", 4, 2, 64, 32), ("many", 4, 2, 128, 16), ("many", 4, 2, 256, 64)]


def rows_of(kind, hq, hkv, news):
    return max(news) if kind == "few" else many(hq, hkv)


@pytest.mark.parametrize("kind,hq,hkv,dim,block", KINDS)
def test_hidden_garbage(kind, hq, hkv, dim, block):
    """NaN and infinite pairs in what a row does not see, in pages of others and behind each end."""
    lens, news, window, sinks = [100, 61], [3, 1], 20, 3
    cache, table, q_start, q = attn_case(63, lens, news, hq, hkv, dim, block)
    want, noise = ref.attention(q, cache, table, lens, q_start, 0.1, window, sinks)
    for b, (kv, n) in enumerate(zip(lens, news)):
        seen = np.zeros(len(table[b]) * block, dtype=bool)
        for i in range(n):
            seen[:kv] |= ref.visible(kv - n + i, kv, window, sinks)
        for j in range(-(-kv // block) * block):
            if not seen[j]:
                for meta in (cache.k_meta, cache.v_meta):
                    meta[table[b, j // block], :, :, j % block] = [np.nan, np.inf] if j % 2 else [np.inf, -np.inf]
    used = {int(p) for b, kv in enumerate(lens) for p in table[b, :-(-kv // block)]}
    for page in set(range(cache.blocks)) - used:
        cache.k_meta[page] = cache.v_meta[page] = np.nan
    last = lens[0] - 1  # hides from the rows before it
    cache.v_meta[table[0, last // block], :, :, last % block] = np.nan
    got = attn(to_device(cache), q, table, lens, q_start, rows_of(kind, hq, hkv, news), window=window, sinks=sinks, scale=0.1)
    assert np.isnan(got[2]).all()
    keep = [0, 1, 3]
    check_attn(got[keep], want[keep], noise[keep])


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("kind,hq,hkv,dim,block", KINDS)
def test_bad_page(kind, hq, hkv, dim, block, bad):
    lens, news = [2 * block + 1, 50], [2, 1]
    cache, table, q_start, q = attn_case(64, lens, news, hq, hkv, dim, block)
    want, noise = ref.attention(q, cache, table, lens, q_start, 0.1)
    table[0, 2] = bad  # the page of the first request's last token
    got = attn(to_device(cache), q, table, lens, q_start, rows_of(kind, hq, hkv, news), scale=0.1)
    assert np.isnan(got[1]).all()
    check_attn(got[[0, 2]], want[[0, 2]], noise[[0, 2]])


@pytest.mark.parametrize("kind,hq,hkv,dim,block", KINDS)
def test_no_table(kind, hq, hkv, dim, block):
    """A table without columns: rows that see tokens are NaN, rows that see none 0."""
    cache, _, q_start, q = attn_case(65, [20, 0], [1, 1], hq, hkv, dim, block)
    got = attn(to_device(cache), q, np.zeros((2, 0)), [20, 0], q_start, rows_of(kind, hq, hkv, [1]))
    assert np.isnan(got[0]).all() and np.all(got[1] == 0)


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (40, 0), (1000, 0), (3, 30), (3, 10 ** 9), (2 ** 30, 5)])
@pytest.mark.parametrize("kind,hq,hkv,dim,block", KINDS)
def test_tokens_past_the_table(kind, hq, hkv, dim, block, window, sinks):
    """Rows before, at and past the table's end, and lengths far past it: NaN exactly where a row sees a token there."""
    reach = 2 * block
    lens, news = [reach + 2, reach + 70, 2 ** 31 - 1, reach], [4, 2, 1, 1]
    cache, table, q_start, q = attn_case(71, [reach] * 4, news, hq, hkv, dim, block)
    got = attn(to_device(cache), q, table[:, :2], lens, q_start, rows_of(kind, hq, hkv, news), window=window, sinks=sinks,
               scale=0.1, max_kv=reach + 70)
    for b, (kv, n) in enumerate(zip(lens, news)):
        for i in range(n):
            row, pos = int(q_start[b]) + i, kv - n + i
            near = max(pos - window + 1, 0) if window else 0  # the window's first token
            past = pos >= reach and (near <= pos) and (max(near, reach) <= pos or sinks > reach)
            if past:
                assert np.isnan(got[row]).all(), (b, i)
            else:
                want, noise = ref.attention(q[row:row + 1], cache, table[b:b + 1], [pos + 1], [0, 1], 0.1, window, sinks)
                check_attn(got[row:row + 1], want, noise, f"request {b} row {i}")


@pytest.mark.parametrize("kind,hq,hkv,dim,block", KINDS)
def test_tiny_scale(kind, hq, hkv, dim, block):
    """A scale at the end of FP32: every visible token weighs the same."""
    cache, table, q_start, q = attn_case(72, [70], [2], hq, hkv, dim, block)
    got = attn(to_device(cache), q, table, [70], q_start, rows_of(kind, hq, hkv, [2]), scale=1.2e-38)
    check_attn(got, *ref.attention(q, cache, table, [70], q_start, 0.0))


def test_many_requests_of_long_prompts_are_one_call():
    """256 requests with room for 2048 rows of 64 heads each, of which few are used."""
    lens, news = [3] * 256, [1, 2] * 128
    cache, table, q_start, q = attn_case(73, lens, news, 64, 8, 64, 16)
    got = attn(to_device(cache), q, table, lens, q_start, 2048, scale=0.1)
    want, noise = ref.attention(q[:6], cache, table[:4], lens[:4], q_start[:5], 0.1)
    check_attn(got[:6], want, noise)
    assert np.isfinite(got).all() and not np.any(got == 7.0)


@pytest.mark.parametrize("hq,dim,block", [(16, 64, 16), (64, 64, 64), (8, 128, 32), (40, 128, 16), (16, 256, 16), (32, 256, 64)])
@pytest.mark.parametrize("B,max_kv", [(70, 50), (70, 10 ** 6), (3, 50), (3, 1100), (3, 10 ** 6), (25, 3000)])
def test_any_cut(hq, dim, block, B, max_kv):
    """Four waves and eight, split and whole, with and without tokens for every part."""
    g = si.rng(76, B, dim)
    lens = [int(v) for v in g.integers(0, 90, B)]
    lens[0], lens[-1] = 0, 300
    cache, table, q_start, q = attn_case(76, lens, [1] * B, hq, 8, dim, block)
    got = attn(to_device(cache), q, table, lens, q_start, 1, max_kv=max_kv, scale=0.1)
    check_attn(got, *ref.attention(q, cache, table, lens, q_start, 0.1, 0, 0, TWO_PARTS))


@pytest.mark.parametrize("hq,dim,block", [(16, 64, 16), (16, 64, 64), (16, 128, 16), (16, 256, 16), (16, 256, 64)])
@pytest.mark.parametrize("lens,news,max_kv,window", [
    ([300, 9, 70], [20, 9, 1], 600, 0), ([300, 9, 70], [20, 9, 1], 200, 0), ([300, 9, 70], [20, 9, 1], 10 ** 6, 0),
    ([90] * 9, [10] * 9, 1500, 0), ([90, 40] * 4, [9, 1] * 4, 700, 50),
])
def test_any_cut_of_some_rows(hq, dim, block, lens, news, max_kv, window):
    """16 rows a wave: four waves and eight, split and whole."""
    cache, table, q_start, q = attn_case(78, lens, news, hq, 8, dim, block)
    got = attn(to_device(cache), q, table, lens, q_start, max(news), max_kv=max_kv, scale=0.1, window=window)
    check_attn(got, *ref.attention(q, cache, table, lens, q_start, 0.1, window, 0, TWO_PARTS))


@pytest.mark.parametrize("kind,hq,hkv,dim,block", KINDS)
def test_shared_pages_and_strided_rows(kind, hq, hkv, dim, block):
    """Requests that share their first pages; q and out as strided rows of one buffer, side by side."""
    lens, news = [3 * block, 2 * block + 5, 3 * block], [1, 2, 1]
    cache, table, q_start, q = attn_case(74, lens, news, hq, hkv, dim, block)
    table[1, :2] = table[0, :2]
    table[2] = table[0]
    T, wide = q.shape[0], hq * dim
    space = torch.full((T, 2 * wide + 16), 7.0, dtype=bf16, device=DEV)
    rows, out = (space[:, at:at + wide].unflatten(1, (hq, dim)) for at in (0, wide + 8))
    rows.copy_(host.bf16_tensor(q))
    with pytest.raises(w4.W4Error):  # the rows' spans overlap: refused, for out must not overlap an input
        w4.w4_kv4_attn(rows, to_device(cache), ints(table), ints(lens), out, q_start=ints(q_start), max_q=2, max_kv=1)
    out = torch.full((T, wide + 24), 7.0, dtype=bf16, device=DEV)[:, 8:8 + wide].unflatten(1, (hq, dim))
    max_q = rows_of(kind, hq, hkv, news)
    w4.w4_kv4_attn(rows, to_device(cache), ints(table), ints(lens), out, q_start=ints(q_start), max_q=max_q, max_kv=1, scale=0.1)
    torch.cuda.synchronize()
    check_attn(host.bf16_values(out.contiguous()), *ref.attention(q, cache, table, lens, q_start, 0.1))
    around = out._base if out._base is not None else out
    assert torch.all(around.view(T, -1)[:, :8] == 7.0) and torch.all(around.view(T, -1)[:, 8 + wide:] == 7.0)


@pytest.mark.parametrize("hq,dim,block", [(128, 64, 16), (100, 256, 64), (17, 128, 32)])
def test_many_heads_to_a_key_head(hq, dim, block):
    lens = [70, 1, 400]
    cache, table, q_start, q = attn_case(75, lens, [1] * 3, hq, 1, dim, block)
    got = attn(to_device(cache), q, table, lens, q_start, 1)
    check_attn(got, *ref.attention(q, cache, table, lens, q_start, float(np.float32(dim ** -0.5)), 0, 0, TWO_PARTS))


@pytest.mark.parametrize("max_q", [1, 2, 30])
def test_rows_past_max_q_are_left(max_q):
    lens, news = [80, 9], [40, 1]
    cache, table, q_start, q = attn_case(66, lens, news, 4, 2, 128, 32)
    want, noise = ref.attention(q, cache, table, lens, q_start, 0.1)
    got = attn(to_device(cache), q, table, lens, q_start, max_q, scale=0.1)
    keep = [*range(max_q), 40]
    check_attn(got[keep], want[keep], noise[keep])
    assert np.all(got[max_q:40] == 7.0)


def test_two_graphs_share_one_workspace():
    """Split attention of two captured graphs over one workspace, replayed in turn on one stream."""
    cases = []
    size = 0
    for seed, lens in ((67, [3000]), (68, [2000, 2500])):
        cache, table, q_start, q = attn_case(seed, lens, [1] * len(lens), 4, 1, 128, 64)
        dev = to_device(cache)
        size = max(size, w4.w4_kv4_attn_workspace_bytes(dev, len(lens), len(lens), 4, 1, max(lens)))
        cases.append((dev, q, table, lens, ref.attention(q, cache, table, lens, q_start, 0.1)))
    assert size > 0
    work = torch.zeros(size // 4, dtype=torch.float32, device=DEV)
    stream, graphs = torch.cuda.Stream(), []
    for dev, q, table, lens, _ in cases:
        out = torch.zeros(q.shape, dtype=bf16, device=DEV)
        args = (host.bf16_tensor(q), dev, ints(table), ints(lens), out)
        torch.cuda.synchronize()
        w4.w4_graph_begin(stream)
        try:
            w4.w4_kv4_attn(*args, max_kv=max(lens), scale=0.1, workspace=work, stream=stream)
        finally:
            graphs.append((w4.w4_graph_end(stream), out, args))
    for _ in range(3):
        for graph, out, _ in graphs:
            out.fill_(9.0)
        torch.cuda.synchronize()
        for graph, *_ in graphs:
            w4.w4_graph_replay(graph, stream)
        torch.cuda.synchronize()
        for (_, out, _), case in zip(graphs, cases):
            check_attn(host.bf16_values(out), *case[4])
    for graph, *_ in graphs:
        graph.destroy()


# ------------------------------------------------------------------ sample
def check_sample(bits, u, **kw):
    rows = bits.shape[0]
    full = {**dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **kw}
    want = [ref.sample(bits[r], u[r], *(np.broadcast_to(full[k], rows)[r] for k in ("temperature", "top_k", "top_p", "min_p")))
            for r in range(rows)]
    got = run_sample(bits, u, **{k: np.broadcast_to(v, rows).copy() for k, v in kw.items()})
    assert got.tolist() == want


def test_sample_many_equal_values():
    """Rows with more equal logits than 16 bits count, alone, among others and shared out over chunks."""
    vocab = 200001
    bits = np.zeros((5, vocab), dtype=np.uint16)
    bits[1, ::2] = 0x3F80  # 100001 ones
    bits[2, 150000:] = 0xBF80
    bits[3, :70000] = 0xFF80
    bits[4, 1:] = 0x8000  # -0 and 0 are one value
    u = [0.0, 0.37, 0.999999, 0.5, 1.0 - 2.0 ** -41]
    check_sample(bits, u)
    check_sample(bits, u, top_p=0.6, top_k=120000)


@pytest.mark.parametrize("vocab", [3, 5000, 100000])
def test_sample_hidden_logits(vocab):
    """-inf logits (a grammar's mask) with top_k past what is left, all but one hidden, u out of range."""
    g = si.rng(69, vocab)
    bits = si.bf16_normal(69, (vocab,), (4, vocab)).copy()
    bits[0, g.permutation(vocab)[: vocab // 2]] = 0xFF80
    bits[1] = 0xFF80
    bits[1, vocab // 2] = 0xC000
    bits[2, 1:] = 0xFF80
    u = [0.3, 0.9, -0.5, 0.999]
    check_sample(bits, u, top_k=[vocab - 1, 5, 2, vocab])
    check_sample(bits, u, min_p=[0.001, 0.5, 1.0, 0.0], temperature=[0.5, 2.0, 0.0, 1.0])
