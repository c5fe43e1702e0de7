"""The operators around the products run as they are used: a decode step's norms between its linears, and one layer of
a batch behind a shared prompt with experts.  Every stage against the FP64 oracle, fed with the bits that the stage
before produced."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import seeded_inputs as si
from oracle import block as blk
from oracle import step as ref
from parity import check_outputs
from test_gpu_block import ROUND, close, f64, norm_bounds, tensor
from test_gpu_step import check_attn, check_queries, ints, random_cache, rope_table, to_device

w4 = pytest.importorskip("gemm_w4_gemv_amd")
from gemm_w4_gemv_amd import host  # noqa: E402
from gemm_w4_gemv_amd.decode import DecodeAttention, DecodeNorms, DecodeStep, TokenSampler, link_decoder_inputs  # noqa: E402

HQ, HKV, DIM, HIDDEN, VOCAB, LAYERS = 4, 2, 128, 512, 700, 2
SHAPES = [("q", HIDDEN, HQ * DIM), ("k", HIDDEN, HKV * DIM), ("v", HIDDEN, HKV * DIM), ("o", HQ * DIM, HIDDEN),
          ("gate", HIDDEN, 256), ("up", HIDDEN, 256), ("down", 256, HIDDEN)]
bf16 = torch.bfloat16


def names(*order):
    return [{"name": n, "layer": layer, "x": None, "y": None} for n, layer in order]


def test_norms_refuse_an_order_that_could_not_work():
    w = [torch.zeros(8, dtype=bf16)] * 2
    norms = DecodeNorms(w[:1], w[:1], w[0])
    good = [("q", 0), ("k", 0), ("v", 0), ("o", 0), ("gate", 0), ("up", 0), ("down", 0), ("logits", 1)]
    step = DecodeStep.__new__(DecodeStep)
    step.norms = norms

    def check(order):
        step.linears = names(*order)
        step._check_blocks()

    check(good)
    for bad in (good[:3] + good[4:], good[:6] + good[7:], [good[3]] + good[:3] + good[4:], good[:4] + [good[6]] + good[4:6] + good[7:],
                [("logits", 1)] + good[:-1], [("q", 1)] + good[1:], good[:4] + good[3:], [("w", 0)] + good):
        with pytest.raises(ValueError):
            check(bad)
    with pytest.raises(ValueError):
        DecodeNorms(w, w[:1], w[0])
    with pytest.raises(ValueError):
        DecodeNorms(w, w, w[0], attn_out=w[:1])
    with pytest.raises(ValueError):
        DecodeStep([], mode="chain", norms=norms)


def test_linears_read_the_stream():
    norms = type("N", (), {"z": torch.zeros(1, HIDDEN)})()
    lins = [{"name": n, "layer": layer, "x": None, "y": (n, layer)} for layer in range(LAYERS) for n, _, _ in SHAPES]
    lins.append({"name": "logits", "layer": LAYERS, "x": None, "y": "end"})
    link_decoder_inputs(lins, None, norms)
    for lin in lins:
        if lin["name"] in ("q", "k", "v", "gate", "up", "logits"):
            assert lin["x"].data_ptr() == norms.z.data_ptr()
    assert [lin["x"] for lin in lins if lin["name"] == "down"] == [("gate", 0), ("gate", 1)]


def build(wide, after):
    lins = []
    for layer in range(LAYERS + 1):
        for i, (name, K, N) in enumerate(SHAPES if layer < LAYERS else [("logits", HIDDEN, VOCAB)]):
            bits = si.int4_linear(80, (layer, i), K, N)
            lins.append(dict(host.int4_tensors(bits), bits=bits, name=name, layer=layer, x=None,
                             y=torch.zeros(N, dtype=bf16, device="cuda")))
    w = lambda k: [tensor(100 * k + i, (HIDDEN,), 0.2, mean=0.1) for i in range(LAYERS)]  # noqa: E731
    norms = DecodeNorms(w(1), w(2), tensor(7, (HIDDEN,), 0.2), attn_out=w(3) if after else None, mlp_out=w(4) if after else None,
                        wide=wide, weight_add=1.0, branch_scale=0.5)
    attention = DecodeAttention(LAYERS, HQ, HKV, DIM, 64, torch.from_numpy(rope_table(DIM)).cuda(), block_size=16)
    sampler = TokenSampler(1, VOCAB)
    link_decoder_inputs(lins, attention, norms)
    return DecodeStep(lins, attention=attention, sampler=sampler, norms=norms)


def check_norm(h, y, y_weight, z_weight, b, got_h, got_z, kind):
    x, z, ex, ez = norm_bounds(dict(h=h, y=y, y_weight=y_weight, z_weight=z_weight, gate=None), 1.0, b, 1e-6, 1.0)
    if got_h is not None:
        close(got_h, x, ex + ROUND[kind] * np.abs(x), "h")
    close(got_z, z, ez, "z")


@pytest.mark.gpu
@pytest.mark.parametrize("wide,after", [(False, True), (True, False)])
def test_decode_with_norms(wide, after):
    """Each norm of a token's step against the oracle, the linears reading what it wrote; then the captured step
    against eager ones."""
    assert torch.cuda.is_available()
    step, twin = build(wide, after), build(wide, after)
    kind = torch.float32 if wide else bf16
    seen = []
    norms = step.norms
    begin, run = norms.begin, norms.run

    def watched_begin(stream):
        begin(stream)
        stream.synchronize()
        check_norm(norms.h, None, None, norms.first, 1.0, None, norms.z, kind)

    def watched_run(layer, name, y, stream):
        stream.synchronize()
        before = norms.h.clone()
        torch.cuda.synchronize()
        run(layer, name, y, stream)
        stream.synchronize()
        check_norm(before, y.view(1, -1), *norms.after[layer, name], 0.5, norms.h, norms.z, kind)
        seen.append((layer, name))

    norms.begin, norms.run = watched_begin, watched_run
    for t in range(3):
        x = tensor(200 + t, (1, HIDDEN), 1.0, kind)
        for s in (step, twin):
            s.norms.h.copy_(x)
            s.sampler.uniform.fill_(0.3)
        torch.cuda.synchronize()
        step.run_eager()
        step.stream.synchronize()
        twin.replay()
        twin.stream.synchronize()
        assert torch.equal(step.norms.h, twin.norms.h) and int(step.sampler.tokens) == int(twin.sampler.tokens)
        for a, b in zip(step.linears, twin.linears):
            assert torch.equal(a["y"], b["y"]), (t, a["name"])
        logits = step.linears[-1]
        z, W = f64(norms.z), oracle.dequant_int4(*(logits["bits"][n] for n in ("qw", "s", "z")))
        check_outputs(host.bf16_values(logits["y"])[None], oracle.linear(z, W), np.linalg.norm(z, axis=1), np.abs(W).max(axis=1), "logits")
    assert seen == [(layer, name) for layer in range(LAYERS) for name in ("o", "down")] * 3
    for s in (step, twin):
        s.destroy()


@pytest.mark.gpu
def test_layer_of_a_batch_with_experts():
    """Forty requests behind one prompt take a token each through a layer: rotation and store, attention, o, norms,
    a router's choice, the experts' products and the way back, norms."""
    assert torch.cuda.is_available()
    g = si.rng(81, 1)
    B, hq, hkv, dim, block, prefix, hidden, inner, E, top = 40, 8, 4, 128, 32, 896, 512, 256, 16, 3
    lens = [int(x) for x in g.integers(prefix + 1, prefix + 90, B)]  # with the new token
    shared = prefix // block
    need = [-(-n // block) - shared for n in lens]
    pages = g.permutation(shared + sum(need) + 2)
    table = np.full((B, shared + max(need)), -1)
    table[:, :shared] = pages[:shared]
    at = shared
    for b in range(B):
        table[b, shared:shared + need[b]] = pages[at:at + need[b]]
        at += need[b]
    host_cache = random_cache(82, len(pages), block, hkv, dim)
    cache = to_device(host_cache)
    slots = np.array([table[b, (n - 1) // block] * block + (n - 1) % block for b, n in enumerate(lens)])
    positions = np.array(lens) - 1

    # rotation and store, attention
    qkv_bits = si.bf16_normal(82, (2,), (B, hq + 2 * hkv, dim))
    qkv, cs = host.bf16_tensor(qkv_bits), rope_table(dim, 2000)
    q, att = (torch.zeros(B, hq, dim, dtype=bf16, device="cuda") for _ in range(2))
    w4.w4_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], ints(positions), torch.from_numpy(cs).cuda(), q_out=q,
                       v=qkv[:, hq + hkv:], cache=cache, slots=ints(slots))
    size = w4.w4_kv4_attn_shared_workspace_bytes(cache, B, B, hq, 1, max(lens), prefix)
    assert size != w4.w4_kv4_attn_workspace_bytes(cache, B, B, hq, 1, max(lens))
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    w4.w4_kv4_attn_shared(q, cache, ints(table), ints(lens), att, ints(pages[:shared]), prefix, max_kv=max(lens), workspace=work)
    torch.cuda.synchronize()
    turned = ref.norm_rope(qkv_bits[:, :hq + hkv], None, cs, positions, dim, False, 1e-6, 0.0)
    check_queries(host.bf16_values(q), turned[:, :hq], "q")
    for b in range(B):
        host_cache.put(slots[b], ref.round_to_bf16(turned[b, hq:]), qkv_bits[b, hq + hkv:])
    check_attn(host.bf16_values(att), *ref.attention(host.bits_of(q), host_cache, np.maximum(table, 0), lens, range(B + 1),
                                                     float(np.float32(dim ** -0.5)), weights=2.0 ** -16))

    # o, the norms around it
    lin = si.int4_linear(83, (3,), hq * dim, hidden)
    t = host.int4_tensors(lin)
    y = torch.zeros(B, hidden, dtype=bf16, device="cuda")
    n = w4.w4_gemm_workspace_bytes(B, hq * dim, hidden)
    w4.w4_gemm(att.view(B, -1), t["qw"], t["s"], t["z"], y, workspace=torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    xf, W = f64(att.view(B, -1)), oracle.dequant_int4(lin["qw"], lin["s"], lin["z"])
    check_outputs(host.bf16_values(y), oracle.linear(xf, W), np.linalg.norm(xf, axis=1), np.abs(W).max(axis=1), "o")
    h = tensor(84, (B, hidden), 3.0, torch.float32)
    before, z = h.clone(), torch.zeros(B, hidden, dtype=bf16, device="cuda")
    weights = [tensor(85 + i, (hidden,), 0.2) for i in range(4)]
    w4.w4_block_norm(h, y, h_out=h, z=z, y_weight=weights[0], z_weight=weights[1], weight_add=1.0)
    torch.cuda.synchronize()
    check_norm(before, y, weights[0], weights[1], 1.0, h, z, torch.float32)

    # router, experts, back
    score = z.float() @ tensor(90, (hidden, E), 0.05, torch.float32)
    weight, ids = torch.topk(torch.softmax(score, dim=1), top, dim=1)
    ids = ids.int()
    start, row_of = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, top, dtype=torch.int32, device="cuda")
    rows = torch.zeros(B * top, hidden, dtype=bf16, device="cuda")
    w4.w4_moe_sort(ids, E, start, row_of, x=z, rows=rows)
    up, down = (si.fp4_pool(86, (i,), E, K, N) for i, (K, N) in enumerate(((hidden, 2 * inner), (inner, hidden))))
    du, dd = host.fp4_tensors(up), host.fp4_tensors(down)
    mid = torch.zeros(B * top, 2 * inner, dtype=bf16, device="cuda")
    every = torch.arange(E, dtype=torch.int32, device="cuda")
    w4.w4_moe_gemm(rows, start, every, du["qw"], du["s"], mid, B)
    act = (torch.nn.functional.silu(mid[:, :inner].float()) * mid[:, inner:].float()).to(bf16)
    made = torch.zeros(B * top, hidden, dtype=bf16, device="cuda")
    w4.w4_moe_gemm(act, start, every, dd["qw"], dd["s"], made, B)
    back = torch.zeros(B, hidden, dtype=bf16, device="cuda")
    w4.w4_moe_combine(made, back, row_of=row_of, weights=weight)
    torch.cuda.synchronize()
    want = blk.moe_sort(ids.cpu().numpy(), E)
    assert start.tolist() == want[0] and np.array_equal(row_of.cpu().numpy(), want[1])
    assert torch.equal(rows, z[torch.tensor(want[2], device="cuda") // top])
    for x, made_by, pool in ((rows, mid, up), (act, made, down)):
        got, expected = f64(made_by), oracle.moe_gemm_fp4(host.bits_of(x), want[0], np.arange(E), pool["qw"], pool["s"])
        assert np.linalg.norm(got - expected) <= 4e-3 * np.linalg.norm(expected)
    out, size = blk.combine(f64(made), want[1], f64(weight))
    close(back, out, (top + 1) * 2.0 ** -24 * size + ROUND[bf16] * np.abs(out), "back")
    before = h.clone()
    w4.w4_block_norm(h, back, h_out=h, z=z, y_weight=weights[2], z_weight=weights[3], weight_add=1.0)
    torch.cuda.synchronize()
    check_norm(before, back, weights[2], weights[3], 1.0, h, z, torch.float32)
