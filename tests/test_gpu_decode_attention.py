"""The decode step with its attention and sampler: each token's stages against the FP64 oracle,
fed with the bits that the stage before produced; then the captured step against the eager one."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import seeded_inputs as si
from oracle import step as ref
from parity import check_outputs
from test_gpu_step import check_attn, check_queries, rope_table

w4 = pytest.importorskip("gemm_w4_gemv_amd")
from gemm_w4_gemv_amd import host  # noqa: E402
from gemm_w4_gemv_amd.decode import DecodeAttention, DecodeStep, TokenSampler, link_decoder_inputs  # noqa: E402

HQ, HKV, DIM, HIDDEN, VOCAB, LAYERS = 4, 2, 128, 256, 1000, 2
SHAPES = [("q", HIDDEN, HQ * DIM), ("k", HIDDEN, HKV * DIM), ("v", HIDDEN, HKV * DIM), ("o", HQ * DIM, HIDDEN),
          ("gate", HIDDEN, 512), ("up", HIDDEN, 512), ("down", 512, HIDDEN)]


def test_o_and_logits_read_what_they_should():
    out = [torch.zeros(1, HQ, DIM) for _ in range(LAYERS)]
    attention = type("A", (), {"out": out})()
    lins = [{"name": n, "layer": layer, "x": None, "y": (n, layer)} for layer in range(LAYERS) for n, _, _ in SHAPES]
    lins.append({"name": "logits", "layer": LAYERS, "x": None, "y": "end"})
    link_decoder_inputs(lins, attention)
    by = {(lin["name"], lin["layer"]): lin for lin in lins}
    for layer in range(LAYERS):
        assert by[("o", layer)]["x"].data_ptr() == out[layer].data_ptr()
    assert by[("q", 1)]["x"] == by[("v", 1)]["x"] == ("down", 0) and by[("logits", LAYERS)]["x"] == ("down", LAYERS - 1)


def test_chain_refuses_attention():
    with pytest.raises(ValueError):
        DecodeStep([], mode="chain", attention=object())
    with pytest.raises(ValueError):
        DecodeStep([], mode="chain", sampler=object())


def build(max_kv, window=0):
    lins = []
    for layer in range(LAYERS + 1):
        for i, (name, K, N) in enumerate(SHAPES if layer < LAYERS else [("logits", HIDDEN, VOCAB)]):
            bits = si.int4_linear(70, (layer, i), K, N)
            t = host.int4_tensors(bits)
            lins.append(dict(t, bits=bits, name=name, layer=layer, x=torch.zeros(K, dtype=torch.bfloat16, device="cuda"),
                             y=torch.zeros(N, dtype=torch.bfloat16, device="cuda")))
    lins[1]["x"] = lins[2]["x"] = lins[0]["x"]
    cs = rope_table(DIM)
    weights = [si.bf16_normal(70, (9, layer), (2, DIM)) for layer in range(LAYERS)]
    attention = DecodeAttention(LAYERS, HQ, HKV, DIM, max_kv, torch.from_numpy(cs).cuda(),
                                [host.bf16_tensor(w[0]) for w in weights], [host.bf16_tensor(w[1]) for w in weights],
                                block_size=16, window=window)
    sampler = TokenSampler(1, VOCAB, temperature=torch.full((1,), 0.8, device="cuda"),
                           top_k=torch.full((1,), 40, dtype=torch.int32, device="cuda"))
    link_decoder_inputs(lins, attention)
    return DecodeStep(lins, attention=attention, sampler=sampler), cs, weights


def feed(step, t):
    x = si.bf16_normal(71, (t,), (HIDDEN,))
    step.linears[0]["x"].copy_(host.bf16_tensor(x))
    step.sampler.uniform.fill_((0.37 * t + 0.1) % 1.0)
    torch.cuda.synchronize()
    return (0.37 * t + 0.1) % 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 7])
def test_decode_tokens(window):
    assert torch.cuda.is_available()
    step, cs, weights = build(48, window)
    a = step.attention
    caches = [ref.Cache(3, 16, HKV, DIM) for _ in range(LAYERS)]
    scale = float(np.float32(DIM ** -0.5))
    for t in range(20):
        u = feed(step, t)
        step.run_eager()
        step.stream.synchronize()
        assert int(a.cached) == t + 1 and int(a.slot) == t and int(a.free_count) == 3 - (t // 16 + 1)
        made = {}
        for lin in step.linears:
            x = host.bits_of(lin["x"])
            W = oracle.dequant_int4(lin["bits"]["qw"], lin["bits"]["s"], lin["bits"]["z"])
            xf = oracle.bf16_to_f64(x)[None]
            check_outputs(host.bf16_values(lin["y"])[None], oracle.linear(xf, W), np.linalg.norm(xf, axis=1),
                          np.abs(W).max(axis=1), f"{t} {lin['layer']} {lin['name']}")
            made[lin["name"]] = host.bits_of(lin["y"])
            if lin["name"] != "v":
                continue
            layer, w = lin["layer"], weights[lin["layer"]]
            rope = (cs, np.array([t]), DIM, False, 1e-6, 0.0)
            check_queries(host.bf16_values(a.q[layer]), ref.norm_rope(made["q"].reshape(1, HQ, DIM), w[0], *rope), "q")
            k = ref.round_to_bf16(ref.norm_rope(made["k"].reshape(1, HKV, DIM), w[1], *rope))
            caches[layer].put(t, k[0], made["v"].reshape(HKV, DIM))
            want = ref.attention(host.bits_of(a.q[layer]), caches[layer], np.arange(3)[None], [t + 1], [0, 1], scale, window)
            check_attn(host.bf16_values(a.out[layer]), *want, f"token {t} layer {layer}")
        assert int(step.sampler.tokens) == ref.sample(made["logits"], u, float(np.float32(0.8)), 40)
    step.destroy()


@pytest.mark.gpu
def test_decode_graph():
    """One captured step replayed token after token, its cache and lengths moving on inside the graph,
    equals eager steps; past max_kv the answers are NaN and the token -1, and nothing else is touched."""
    assert torch.cuda.is_available()
    (a, *_), (b, *_) = build(32), build(32)
    for t in range(34):
        for s in (a, b):
            feed(s, t)
        a.replay()
        b.run_eager()
        torch.cuda.synchronize()
        for x, y in zip(a.linears, b.linears):
            assert torch.equal(x["y"].view(torch.int16), y["y"].view(torch.int16)), (t, x["name"])
        assert int(a.sampler.tokens) == int(b.sampler.tokens) and (int(a.sampler.tokens) == -1) == (t >= 32)
        assert torch.equal(a.attention.table, b.attention.table)
    for s in (a, b):
        s.destroy()
