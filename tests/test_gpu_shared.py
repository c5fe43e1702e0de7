"""GPU parity of the attention behind a shared prefix against the FP64 oracle of
the attention itself (each request with all of its tokens), with its bounds: two
parts of a weight, 2^-16 of it; the parts' join is a few more FP32 roundings,
within the 64 that the bound has for the sums."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import seeded_inputs as si
from oracle import step as ref
from test_gpu_step import check_attn, ints, random_cache, run_attn, to_device

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemm_w4_gemv_amd")
from gemm_w4_gemv_amd import host  # noqa: E402

DEV = "cuda"
bf16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def case(seed, prefix, lens, news, hq, hkv, dim, block, spare=2):
    """Requests of lens tokens in all, the first ``prefix`` of each (or all it has) in the same pages."""
    g = si.rng(seed, 94, hq, dim, block, prefix)
    shared = -(-prefix // block)
    need = [max(-(-max(n, 0) // block) - shared, 0) for n in lens]
    blocks = shared + sum(need) + spare
    cache = random_cache(seed, blocks, block, hkv, dim)
    pages = g.permutation(blocks)
    table = np.full((len(lens), shared + max(need + [0]) + 1), 123456789)
    table[:, :shared] = pages[:shared]
    at = shared
    for b, n in enumerate(need):
        table[b, shared:shared + n] = pages[at:at + n]
        at += n
    q_start = np.concatenate(([0], np.cumsum(news)))
    T = int(q_start[-1])
    return cache, pages[:shared], table, q_start, si.bf16_normal(seed, (95, T, hq, dim), (T, hq, dim))


def run(cache, q_bits, table, lens, q_start, prefix_table, prefix, pad=0, tail=0, stream=None, **kw):
    T, hq, d = q_bits.shape
    space = torch.zeros(T + tail, hq * d + pad, dtype=bf16, device=DEV)
    q = space[:, :hq * d].unflatten(1, (hq, d))
    q[:T] = host.bf16_tensor(q_bits)
    out = torch.full((T + tail, hq * d + 2 * pad), 7.0, dtype=bf16, device=DEV)[:, :hq * d].unflatten(1, (hq, d))
    max_q = max(int(np.max(np.diff(q_start))), 1) if q_start is not None else 1
    kw.setdefault("max_kv", max(max(lens), 0))
    size = w4.w4_kv4_attn_shared_workspace_bytes(cache, T + tail, len(lens), hq, max_q, kw["max_kv"], prefix,
                                                 kw.get("window", 0), kw.get("sinks", 0))
    work = torch.full((size // 4,), float("nan"), dtype=torch.float32, device=DEV) if size else None
    torch.cuda.synchronize()
    w4.w4_kv4_attn_shared(q, cache, ints(table), ints(lens), out, ints(prefix_table), prefix,
                          q_start=None if q_start is None else ints(q_start), max_q=max_q, workspace=work, stream=stream,
                          **kw)
    torch.cuda.synchronize()
    return host.bf16_values(out)


def expect(cache, q, table, lens, q_start, dim, window=0, sinks=0):
    table = np.where(table == 123456789, 0, table)
    return ref.attention(q, cache, table, lens, q_start, float(np.float32(1 / np.sqrt(dim))), window, sinks, 2.0 ** -16)


def apart(prefix, lens, news, hq, hkv, dim, block, window=0, sinks=0):
    """Whether a call does the shared tokens apart: its workspace then differs from the attention's."""
    c = w4.step._CacheStruct(16, 16, 16, 16, 1 << 15, block, hkv, dim)
    fake = type("Cache", (), {"ref": w4.step.ctypes.byref(c)})()
    args = (sum(news), len(lens), hq, max(news), max(lens))
    return (w4.w4_kv4_attn_shared_workspace_bytes(fake, *args, prefix, window, sinks) !=
            w4.w4_kv4_attn_workspace_bytes(fake, *args, window, sinks))


TOGETHER = [  # prefix, lens, news, hq, hkv, dim, block, window, sinks
    (560, [561, 600, 575] * 16, [1] * 48, 8, 8, 64, 16, 0, 0),               # half a tile of the prefix is each one's own
    (1024, [1025] * 50, [1] * 50, 16, 8, 64, 32, 0, 0), (3904, [3950, 3905, 4100] * 17, [1] * 51, 64, 8, 64, 64, 0, 0),
    (896, [900, 1000] * 20, [1] * 40, 8, 4, 128, 64, 0, 0), (848, [850, 900, 1400] * 14, [1] * 42, 8, 4, 128, 16, 0, 0),
    (1024, [1030, 2000, 1024, 1500] * 6, [1] * 24, 16, 8, 256, 64, 0, 0), (720, [721, 800] * 12, [1] * 24, 16, 8, 256, 16, 0, 0),
    (4096, [4200] * 9, [1] * 9, 8, 8, 256, 256, 0, 0), (2112, [2150, 2113] * 16, [1] * 32, 128, 8, 128, 128, 0, 0),  # 16 rows a request
    (1888, [1900] * 18, [1] * 18, 160, 8, 128, 64, 0, 0),                    # 20
    (4160, [4200, 4170, 4300] * 4, [5, 1, 3] * 4, 16, 8, 128, 32, 0, 0), (2080, [2200] * 18, [8, 1, 7, 2, 8, 3] * 3, 24, 8, 256, 16, 0, 0),
    (1024, [10, 1200, 0, 1024, 1025, 31] * 7, [1, 1, 0, 1, 1, 1] * 7, 8, 4, 128, 32, 0, 0),  # requests inside the prefix, empty ones
    (1760, [5, 1900, 1800] * 8, [9, 4, 1] * 8, 8, 8, 128, 32, 0, 0),         # rows that see nothing
    (1024, [1100, 1030, 1500] * 12, [1] * 36, 8, 4, 128, 64, 300, 0), (1024, [1100, 1030, 1500] * 12, [1] * 36, 8, 4, 128, 16, 100, 4),
    (1024, [1100, 1030, 1500] * 8, [1] * 24, 16, 8, 256, 64, 1050, 33), (2048, [2050, 2300] * 16, [1, 2] * 16, 8, 8, 64, 64, 2100, 700),
    (1024, [1040, 5000] * 10, [1] * 20, 8, 8, 128, 64, 0, 0),                # own tokens in splits of their own
]


@pytest.mark.parametrize("prefix,lens,news,hq,hkv,dim,block,window,sinks", TOGETHER)
def test_attn_shared(prefix, lens, news, hq, hkv, dim, block, window, sinks):
    assert apart(prefix, lens, news, hq, hkv, dim, block, window, sinks)
    cache, shared, table, q_start, q = case(1, prefix, lens, news, hq, hkv, dim, block)
    got = run(to_device(cache), q, table, lens, q_start, shared, prefix, window=window, sinks=sinks)
    check_attn(got, *expect(cache, q, table, lens, q_start, dim, window, sinks))


@pytest.mark.parametrize("prefix,lens,news,hq,hkv,dim,block,window,sinks", [
    (32, [33, 40], [1, 1], 2, 1, 64, 16, 0, 0), (48, [60, 49, 300], [1] * 3, 4, 2, 64, 16, 0, 0),
    (1024, [1030, 1100, 1024, 1500], [1] * 4, 16, 8, 256, 64, 0, 0), (256, [400] * 4, [33, 1, 70, 2], 4, 2, 256, 64, 0, 0),
    (160, [10, 200, 0, 160, 161], [1, 1, 0, 1, 1], 8, 2, 128, 32, 0, 0), (512, [700, 520, 900], [1] * 3, 8, 2, 128, 64, 300, 4),
])
def test_attn_shared_of_few_requests(prefix, lens, news, hq, hkv, dim, block, window, sinks):
    """Where it does not pay, the tokens are read through each request's table as ever."""
    assert not apart(prefix, lens, news, hq, hkv, dim, block, window, sinks)
    cache, shared, table, q_start, q = case(1, prefix, lens, news, hq, hkv, dim, block)
    dev = to_device(cache)
    got = run(dev, q, table, lens, q_start, shared, prefix, window=window, sinks=sinks)
    check_attn(got, *expect(cache, q, table, lens, q_start, dim, window, sinks))
    table = np.where(table == 123456789, 0, table)
    assert np.array_equal(got, run_attn(dev, q, table, lens, q_start, window=window, sinks=sinks))


@pytest.mark.parametrize("prefix", [0, 1, 31])
def test_attn_shared_without_a_whole_tile_is_the_attention(prefix):
    lens, news = [50, 70], [1, 1]
    cache, shared, table, q_start, q = case(2, prefix, lens, news, 4, 2, 128, 16)
    dev = to_device(cache)
    got = run(dev, q, table, lens, q_start, shared, prefix)
    assert np.array_equal(got, run_attn(dev, q, table, lens, q_start, max_kv=70))


@pytest.mark.parametrize("rows", [2, 40])
def test_attn_shared_without_q_start_strided_and_with_rows_behind(rows):
    lens = [930 + 3 * i for i in range(rows)]
    assert apart(900, lens, [1] * rows, 8, 4, 128, 64) == (rows == 40)
    cache, shared, table, q_start, q = case(3, 900, lens, [1] * rows, 8, 4, 128, 64)
    dev = to_device(cache)
    want = run(dev, q, table, lens, q_start, shared, 900)
    check_attn(want, *expect(cache, q, table, lens, q_start, 128))
    assert np.array_equal(run(dev, q, table, lens, None, shared, 900, pad=24), want)
    got = run(dev, q, table, lens, q_start, shared, 900, pad=8, tail=3)
    assert np.all(got[rows:] == 7.0)
    check_attn(got[:rows], *expect(cache, q, table, lens, q_start, 128))


def test_attn_shared_is_right_for_any_max_kv():
    lens = [700, 650, 1200] * 20
    assert apart(640, lens, [1] * 60, 8, 8, 64, 64)
    cache, shared, table, q_start, q = case(4, 640, lens, [1] * 60, 8, 8, 64, 64)
    dev = to_device(cache)
    want = expect(cache, q, table, lens, q_start, 64)
    for max_kv in (0, 1, 640, 641, 100000, 2 ** 31 - 1):
        check_attn(run(dev, q, table, lens, q_start, shared, 640, max_kv=max_kv), *want, f"max_kv {max_kv}")


@pytest.mark.parametrize("rows", [3, 50])
def test_attn_shared_bad_pages_and_odd_values(rows):
    """A page out of range makes NaN of the rows that see it and of no other; what no row sees may hold anything."""
    prefix, last = 704, 43  # pages of 16, 22 tiles
    lens = [708 + 4 * i for i in range(rows)]
    lens[0] = 678  # inside the prefix: sees tokens 0 .. 677
    make = lambda: case(5, prefix, lens, [1] * rows, 8, 4, 128, 16)  # noqa: E731
    assert apart(prefix, lens, [1] * rows, 8, 4, 128, 16) == (rows == 50)
    cache, shared, table, q_start, q = make()
    want = expect(cache, q, table, lens, q_start, 128)
    cache.k_meta[shared[last], :, :, 15] = np.nan  # token 703: seen by all but the first
    cache.v_meta[shared[last - 1], :, :, 6:] = np.inf  # tokens 678 on
    got = run(to_device(cache), q, table, lens, q_start, shared, prefix)
    check_attn(got[:1], want[0][:1], want[1][:1])
    assert np.all(np.isnan(got[1:]))
    cache, shared, table, q_start, q = make()
    for bad in (-1, 10 ** 6):
        broken = shared.copy()
        broken[last] = bad
        both = table.copy()
        both[:, last] = bad  # the rows of the table hold the prefix's pages too
        got = run(to_device(cache), q, both, lens, q_start, broken, prefix)
        check_attn(got[:1], want[0][:1], want[1][:1])
        assert np.all(np.isnan(got[1:]))
    own = table.copy()
    own[1, last + 1] = -1  # a request's own first page
    got = run(to_device(cache), q, own, lens, q_start, shared, prefix)
    assert np.all(np.isnan(got[1]))
    rest = [i for i in range(rows) if i != 1]
    check_attn(got[rest], want[0][rest], want[1][rest])


def test_attn_shared_table_that_ends_with_the_prefix():
    """No page of a request's own in the table: a row past the prefix is NaN, one inside it is not."""
    lens = [1024, 1025, 40] * 10
    assert apart(1024, lens, [1] * 30, 8, 8, 128, 32)
    cache, shared, table, q_start, q = case(6, 1024, lens, [1] * 30, 8, 8, 128, 32)
    want = expect(cache, q, table, lens, q_start, 128)
    inside = [i for i in range(30) if i % 3 != 1]
    for width in (32, 0):
        got = run(to_device(cache), q, table[:, :width], lens, q_start, shared, 1024)
        check_attn(got[inside], want[0][inside], want[1][inside])
        assert np.all(np.isnan(got[1::3]))


def test_attn_shared_graph_replays_with_growing_requests():
    """Two captured calls over one workspace, replayed in turn; each request grows between, its table in place."""
    lens, B, hq, dim, prefix = [721, 730, 750, 800, 722] * 10, 50, 8, 128, 704
    assert apart(prefix, lens, [1] * B, hq, 4, dim, 32)
    cache, shared, table, q_start, q = case(7, prefix, [n + 40 for n in lens], [1] * B, hq, 4, dim, 32)
    dev = to_device(cache)
    stream = torch.cuda.Stream()
    size = w4.w4_kv4_attn_shared_workspace_bytes(dev, B, B, hq, 1, 900, prefix)
    work = torch.full((size // 4,), float("nan"), dtype=torch.float32, device=DEV)
    dev_q = [host.bf16_tensor(q), host.bf16_tensor(q[::-1].copy())]
    dev_lens, dev_table, dev_shared = ints(lens), ints(table), ints(shared)
    outs, graphs = [torch.zeros(B, hq, dim, dtype=bf16, device=DEV) for _ in range(2)], []
    torch.cuda.synchronize()
    for x, out in zip(dev_q, outs):
        w4.w4_graph_begin(stream)
        try:
            w4.w4_kv4_attn_shared(x, dev, dev_table, dev_lens, out, dev_shared, prefix, max_kv=900, workspace=work, stream=stream)
        finally:
            graphs.append(w4.w4_graph_end(stream))
    for k in range(4):
        now = [n + 9 * k for n in lens]
        dev_lens.copy_(ints(now))
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay(stream)
        torch.cuda.synchronize()
        for bits, out in zip((q, q[::-1]), outs):
            check_attn(host.bf16_values(out), *expect(cache, bits, table, now, q_start, dim), f"replay {k}")
    for graph in graphs:
        graph.destroy()


def test_attn_shared_repeats_its_bits_on_another_stream():
    lens = [1100 + i for i in range(30)]
    assert apart(1024, lens, [1] * 30, 8, 8, 64, 64)
    cache, shared, table, q_start, q = case(8, 1024, lens, [1] * 30, 8, 8, 64, 64)
    dev = to_device(cache)
    want = run(dev, q, table, lens, q_start, shared, 1024)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert np.array_equal(run(dev, q, table, lens, q_start, shared, 1024, stream=side), want)


@pytest.mark.parametrize("prefix", [2 ** 31 - 1, 2 ** 31 - 255])
def test_attn_shared_prefix_within_a_page_of_2_31(prefix):
    """A prefix far longer than any request, its last page's end past 2^31 - 1: what the requests hold of it is read."""
    lens, B, hq, hkv, dim, block = [700, 1, 900, 256, 0, 257], 48, 8, 8, 64, 256
    lens = lens * (B // len(lens))
    assert apart(prefix, lens, [1] * B, hq, hkv, dim, block)
    cache, q = random_cache(9, 6, block, hkv, dim), si.bf16_normal(9, (96,), (B, hq, dim))
    pages = si.rng(9, 97).permutation(6)
    far = ints(np.resize(pages, -(-prefix // block)))
    table, out = ints(np.tile(pages[:4], (B, 1))), torch.full((B, hq, dim), 7.0, dtype=bf16, device=DEV)
    dev = to_device(cache)
    size = w4.w4_kv4_attn_shared_workspace_bytes(dev, B, B, hq, 1, 900, prefix)
    work = torch.full((size // 4,), float("nan"), dtype=torch.float32, device=DEV)
    w4.w4_kv4_attn_shared(q=host.bf16_tensor(q), cache=dev, block_table=table, kv_lens=ints(lens), out=out, prefix_table=far,
                          prefix=prefix, max_kv=900, workspace=work)
    torch.cuda.synchronize()
    check_attn(host.bf16_values(out), *expect(cache, q, np.tile(pages[:4], (B, 1)), lens, range(B + 1), dim))


def test_attn_shared_window_with_rows_that_see_nothing():
    """A window over a part of the prefix, requests with more rows than tokens and empty ones among the rest."""
    prefix, lens, news = 2048, [5, 2100, 0, 2049] * 8, [9, 1, 0, 2] * 8
    assert apart(prefix, lens, news, 8, 8, 128, 64, 1500)
    cache, shared, table, q_start, q = case(10, prefix, lens, news, 8, 8, 128, 64)
    dev = to_device(cache)
    for window, sinks in ((1500, 0), (1500, 40), (1900, 0)):
        got = run(dev, q, table, lens, q_start, shared, prefix, window=window, sinks=sinks, tail=3)
        assert np.all(got[-3:] == 7.0)
        check_attn(got[:-3], *expect(cache, q, table, lens, q_start, 128, window, sinks), f"window {window}, {sinks} first tokens")


def test_attn_shared_window_is_not_passed_by_for_a_row_that_is_not_there():
    """40 rows, of which the last block of 16 is half empty, and rows of no request take a window's tiles, not all of the
    prefix's: 512 tiles of 32768, where 48 rows take as many.  (Three times is far from both: 64 times the tiles.)"""
    prefix, block, hq, hkv, dim, window = 1 << 20, 256, 16, 8, 128, 1 << 14
    dev = to_device(random_cache(11, 6, block, hkv, dim))
    far = ints(np.resize(np.arange(6), prefix // block))
    times = {}
    for rows, tail in ((24, 0), (20, 0), (22, 2)):
        lens = [prefix + 1 + i for i in range(rows)]
        assert apart(prefix, lens, [1] * rows, hq, hkv, dim, block, window)
        T = rows + tail
        q, q_start = host.bf16_tensor(si.bf16_normal(11, (98, rows), (T, hq, dim))), ints(range(rows + 1))
        table, out = torch.cat((far, ints([0]))).repeat(rows, 1), torch.zeros(T, hq, dim, dtype=bf16, device=DEV)
        size = w4.w4_kv4_attn_shared_workspace_bytes(dev, T, rows, hq, 1, max(lens), prefix, window)
        work = torch.empty(size, dtype=torch.uint8, device=DEV)
        args = (q, dev, table, ints(lens), out, far, prefix)
        kw = dict(q_start=q_start, max_kv=max(lens), window=window, workspace=work)
        took = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                w4.w4_kv4_attn_shared(*args, **kw)
            b.record()
            torch.cuda.synchronize()
            took.append(a.elapsed_time(b))
        times[T, tail] = min(took)
    assert max(times.values()) < 3 * times[24, 0], times


@pytest.mark.parametrize("prefix,lens,news,hq,hkv,dim,block,window,sinks", [
    (2048, [2100, 2060, 2300] * 14, [1] * 42, 8, 4, 128, 64, 2000, 0), (1504, [1600, 1510] * 25, [1] * 50, 8, 4, 128, 16, 1400, 6),
    (2560, [2600, 2561, 2570] * 8, [1, 3, 2] * 8, 16, 8, 256, 64, 2500, 0), (3200, [3300, 3201, 3350] * 11, [1] * 33, 8, 8, 64, 32, 3000, 700),
    (4096, [4150, 30, 4100] * 8, [1, 2, 1] * 8, 8, 8, 128, 128, 2048, 0),
])
def test_attn_shared_window_over_a_part_of_a_long_prefix(prefix, lens, news, hq, hkv, dim, block, window, sinks):
    assert apart(prefix, lens, news, hq, hkv, dim, block, window, sinks)
    cache, shared, table, q_start, q = case(12, prefix, lens, news, hq, hkv, dim, block)
    got = run(to_device(cache), q, table, lens, q_start, shared, prefix, window=window, sinks=sinks)
    check_attn(got, *expect(cache, q, table, lens, q_start, dim, window, sinks))


def test_attn_shared_cache_and_rows_past_32_bit_offsets():
    """Shared and own pages whose bytes lie past 2^32, queries and outputs 2^31 values apart."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("less than 120 GiB of memory is free")
    hq, hkv, dim, block, prefix = 8, 8, 128, 256, 4096
    shared = prefix // block
    lens = [prefix + 1 + 7 * i for i in range(12)]
    assert apart(prefix, lens, [1] * 12, hq, hkv, dim, block)
    small = random_cache(13, shared + 12, block, hkv, dim)
    blocks = (5 << 30) // (hkv * block * dim // 2)
    far = w4.Kv4Cache.empty(blocks, block, hkv, dim)
    pages = blocks - 1 - si.rng(13, 99).permutation(shared + 12)
    for name in ("k_codes", "k_meta", "v_codes", "v_meta"):
        getattr(far, name)[torch.from_numpy(pages).to(DEV)] = torch.from_numpy(getattr(small, name)).to(DEV)
    q = si.bf16_normal(13, (100,), (12, hq, dim))
    step = (1 << 31) + 8
    space = [torch.empty(11 * step + hq * dim, dtype=bf16, device=DEV) for _ in range(2)]
    far_q, out = (torch.as_strided(s, (12, hq, dim), (step, dim, 1)) for s in space)
    far_q.copy_(host.bf16_tensor(q))
    own = np.concatenate((np.tile(np.arange(shared), (12, 1)), np.arange(shared, shared + 12)[:, None]), axis=1)
    size = w4.w4_kv4_attn_shared_workspace_bytes(far, 12, 12, hq, 1, max(lens), prefix)
    work = torch.full((size // 4,), float("nan"), dtype=torch.float32, device=DEV)
    w4.w4_kv4_attn_shared(far_q, far, ints(pages[own]), ints(lens), out, ints(pages[:shared]), prefix, max_kv=max(lens),
                          workspace=work)
    torch.cuda.synchronize()
    check_attn(host.bf16_values(out.contiguous()), *expect(small, q, own, lens, range(13), dim))
