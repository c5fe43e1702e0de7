"""The decode step's GEMV chain captured once into a HIP graph.

Two ways to run the step are offered:

* ``launches``: one ``w4_gemv`` launch per linear (336 graph nodes);
* ``chain``: one ``w4_chain_run`` launch (a single graph node) of the
  persistent chain kernel, with the decoder's linears as stages: per layer
  {q, k, v} -> {o} -> {gate, up} -> {down}.  A linear whose input is another
  linear's output (see ``link_decoder_inputs``) waits for exactly that
  output.

"Lab 5: Gemma4 端到端推理优化", section "CUDA Graph": after the fused GEMV the
remaining cost was launch and Python overhead, so the whole decode step is
captured once into a static graph and replayed once per token; the graph
needs static buffers.  Here the step is the chain of INT4 linears of every
layer in launch order (q, k, v, o, gate, up, down), each an ``w4_gemv``
recorded on one stream; every linear keeps its own static input and output
buffers, so one replay recomputes every output.

With a ``DecodeAttention`` the step is a whole token's: between a layer's q, k,
v and its o it stores the token in the layer's 4-bit cache and attends over
it, and with a ``TokenSampler`` it ends in the next token.
"""
from __future__ import annotations

import torch

from . import w4_gemv, w4_graph_begin, w4_graph_end, W4Graph, w4_chain_create, w4_chain_run, \
    w4_chain_workspace_bytes, Kv4Cache, w4_kv4_plan, w4_qk_norm_rope, w4_kv4_attn, w4_kv4_attn_workspace_bytes, \
    w4_sample, w4_sample_workspace_bytes

# Stage of each decoder linear within its layer.  Along the decoder's data
# flow q -> o -> gate -> down -> (next layer's) q each of these waits for the
# one before; k, v and up are read by no linear of this path, so each pair
# gets a stage of its own right after the linear that shares its input
# (k, v after q; up after gate): their weights stream while the chain
# kernel awaits the next reader's input (o's, down's), instead of delaying it.
LAYER_STAGES = 6
LAYER_STAGE = {"q": 0, "k": 1, "v": 1, "o": 2, "gate": 3, "up": 4, "down": 5}
# The grouped schedule: linears that share an input in one stage.
LAYER_STAGES_GROUPED = 4
LAYER_STAGE_GROUPED = {"q": 0, "k": 0, "v": 0, "o": 1, "gate": 2, "up": 2, "down": 3}


# the output each decoder linear reads: "h" is the layer's input (the first
# layer's own input; for later layers the previous layer's down output)
DECODER_INPUT = {"q": "h", "k": "h", "v": "h", "o": "q", "gate": "o", "up": "o", "down": "gate", "logits": "h"}


def decoder_stages(names, layers_of, grouped: bool = False):
    """Stage number of every linear, from its name and layer index."""
    per, table = (LAYER_STAGES_GROUPED, LAYER_STAGE_GROUPED) if grouped else (LAYER_STAGES, LAYER_STAGE)
    return [per * layer + table[name] for name, layer in zip(names, layers_of)]


def link_decoder_inputs(linears, attention: "DecodeAttention | None" = None) -> None:
    """Make every linear read the output it reads in a decoder layer.

    ``linears`` are dicts with ``name``, ``layer``, ``x`` and ``y``, in layer
    order.  The first layer's q, k and v keep their own ``x`` (they must share
    one buffer); every other input becomes the producing linear's ``y``: o
    reads q's output, or with ``attention`` its layer's output there (the
    gate/up product is outside this path); gate and up read o's, down reads
    gate's, and a layer's q, k and v read the previous layer's down output,
    as a linear named "logits" does (its layer is one past the last).
    """
    out = {}
    for lin in linears:
        layer, name = lin["layer"], lin["name"]
        src = DECODER_INPUT[name]
        if attention is not None and name == "o":
            lin["x"] = attention.out[layer].view(-1)
        elif src == "h":
            if layer > 0:
                lin["x"] = out[(layer - 1, "down")]
        else:
            lin["x"] = out[(layer, src)]
        out[(layer, name)] = lin["y"]


def decode_linears(device: str = "cuda"):
    """The decode step's 336 INT4 linears as device tensors, from the seeded
    synthetic workload (48 layers x q, k, v, o, gate, up, down; hidden 3840;
    group 128), each reading its own seeded N(0,1) input and writing its own
    zeroed output.  Each dict holds ``qw``, ``s``, ``z``, ``x``, ``y``,
    ``name``, ``layer``, ``index`` (position in its layer), ``K``, ``N`` and
    ``stage`` (six stages per layer).  The seeded inputs are synthetic data,
    not part of the method: the generator module is imported here only."""
    import seeded_inputs as si
    from . import host

    lins = []
    for layer, idx, name, K, N in si.decode_step_specs():
        lin_np, x_bits = si.decode_linear(layer, idx)
        t = host.int4_tensors(lin_np, device)
        t["x"] = host.bf16_tensor(x_bits, device)
        t["y"] = torch.zeros(N, dtype=torch.bfloat16, device=device)
        t["name"], t["layer"], t["index"], t["K"], t["N"] = name, layer, idx, K, N
        t["stage"] = decoder_stages([name], [layer])[0]
        lins.append(t)
    torch.cuda.synchronize()
    return lins


def linked_copy(lins):
    """The same linears (same weights and output buffers), each reading the
    output it reads in a decoder (``link_decoder_inputs``); layer 0's q, k
    and v share q's input.  This is the decode step as it is timed."""
    out = [dict(t) for t in lins]
    for t in out[1:3]:
        t["x"] = out[0]["x"]
    link_decoder_inputs(out)
    return out


class DecodeAttention:
    """One request's attention in a decode step: a 4-bit cache a layer, one block table for all.

    ``cos_sin`` float32 [max_pos, rot_dim] (None: no rotation); ``q_weight`` and ``k_weight``
    are each None or a list of a layer's bfloat16 [head_dim].  Every layer's ``out`` is
    bfloat16 [1, q_heads, head_dim], what its o linear reads.  ``cached`` (int32 [1]) counts the
    tokens held; a step adds one.  A prompt is stored by the same calls with more rows: its
    tokens' slots are what ``w4_kv4_plan`` gives on ``table``, ``free`` and ``free_count``.
    A token past the last page (``max_kv`` in whole pages) has no slot, and its outputs are NaN.
    All layers have the same heads, window and rotation; weights are taken as they are and a
    rotation's pairs are (i, i + rot_dim / 2)."""

    def __init__(self, layers: int, q_heads: int, kv_heads: int, head_dim: int, max_kv: int, cos_sin=None,
                 q_weight=None, k_weight=None, block_size: int = 64, window: int = 0, sinks: int = 0,
                 scale: float | None = None, eps: float = 1e-6, device: str = "cuda"):
        pages = -(-max_kv // block_size)
        self.shape = (q_heads, kv_heads, head_dim)
        self.block_size, self.max_kv = block_size, max_kv
        self.seen = dict(window=window, sinks=sinks, scale=scale)
        self.cos_sin, self.eps = cos_sin, eps
        self.weights = [(None if q_weight is None else q_weight[i], None if k_weight is None else k_weight[i])
                        for i in range(layers)]
        self.caches = [Kv4Cache.empty(pages, block_size, kv_heads, head_dim, device) for _ in range(layers)]
        ints = dict(dtype=torch.int32, device=device)
        self.table = torch.full((1, pages), -1, **ints)
        self.free = torch.arange(pages - 1, -1, -1, **ints)
        self.free_count = torch.full((1,), pages, **ints)
        self.cached, self.new = torch.zeros(1, **ints), torch.ones(1, **ints)
        self.q_start, self.kv_lens, self.counts = torch.zeros(2, **ints), torch.zeros(1, **ints), torch.zeros(2, **ints)
        self.position, self.slot = torch.zeros(1, **ints), torch.zeros(1, **ints)
        self.q = torch.zeros(layers, 1, q_heads, head_dim, dtype=torch.bfloat16, device=device)
        self.out = torch.zeros_like(self.q)
        n = max(w4_kv4_attn_workspace_bytes(c, 1, 1, q_heads, 1, max_kv, window, sinks) for c in self.caches)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=device) if n else None

    def begin(self, stream: torch.cuda.Stream) -> None:
        """The new token's position and slot, before the first layer."""
        w4_kv4_plan(self.cached, self.new, self.table, self.free, self.free_count, self.block_size, self.q_start,
                    self.kv_lens, self.position, self.slot, self.counts, stream=stream)

    def run(self, layer: int, q, k, v, stream: torch.cuda.Stream) -> None:
        """Stores the token of ``layer`` (its q, k and v linears' outputs) and attends into ``out[layer]``."""
        hq, hkv, d = self.shape
        q_weight, k_weight = self.weights[layer]
        cache = self.caches[layer]
        w4_qk_norm_rope(q.view(1, hq, d), k.view(1, hkv, d), None if self.cos_sin is None else self.position,
                        self.cos_sin, q_out=self.q[layer], q_weight=q_weight, k_weight=k_weight, eps=self.eps,
                        v=v.view(1, hkv, d), cache=cache, slots=self.slot, stream=stream)
        w4_kv4_attn(self.q[layer], cache, self.table, self.kv_lens, self.out[layer], max_kv=self.max_kv,
                    workspace=self.workspace, stream=stream, **self.seen)

    def end(self, stream: torch.cuda.Stream) -> None:
        """The token counts as held, its page as taken: what the next step begins from."""
        with torch.cuda.stream(stream):
            torch.add(self.kv_lens, 0, out=self.cached)
            torch.add(self.counts[:1], 0, out=self.free_count)


class TokenSampler:
    """Draws a token from each row of logits [rows, vocab]: settings are tensors (or None) that
    the caller changes in place, ``uniform`` (float64 [rows], in [0, 1)) anew for every token."""

    def __init__(self, rows: int, vocab: int, temperature=None, top_k=None, top_p=None, min_p=None, device: str = "cuda"):
        self.settings = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
        self.shape = (rows, vocab)
        self.uniform = torch.zeros(rows, dtype=torch.float64, device=device)
        self.tokens = torch.zeros(rows, dtype=torch.int32, device=device)
        n = w4_sample_workspace_bytes(rows, vocab)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=device) if n else None

    def run(self, logits, stream: torch.cuda.Stream) -> None:
        w4_sample(logits.view(self.shape), self.uniform, self.tokens, workspace=self.workspace, stream=stream,
                  **self.settings)


class DecodeStep:
    """A captured chain of ``w4_gemv`` calls.

    ``linears`` is a sequence of dicts with device tensors ``qw`` (int32
    [N, K/8]), ``s``, ``z`` (float16 [N, K/128]), ``x`` (bfloat16 [K]) and
    ``y`` (bfloat16 [N]).  The tensors must stay alive while the graph does.

    With ``attention`` (and then ``name`` and ``layer`` in the dicts, see
    ``link_decoder_inputs``) every layer's q, k and v, in any order, go through its
    cache before its o; with ``sampler`` the step ends in a token from the output of
    the linear named "logits".  Both are launches of their own, not stages of the chain.
    """

    def __init__(self, linears, stream: torch.cuda.Stream | None = None, mode: str = "launches",
                 attention: DecodeAttention | None = None, sampler: TokenSampler | None = None):
        if mode not in ("launches", "chain"):
            raise ValueError("mode must be 'launches' or 'chain'")
        if mode == "chain" and (attention is not None or sampler is not None):
            raise ValueError("the chain runs linears alone: attention and sampler go with mode 'launches'")
        self.attention, self.sampler = attention, sampler
        self.linears = list(linears)
        if attention is not None:
            self._check_layers()
        if sampler is not None and [lin["name"] for lin in self.linears].count("logits") != 1:
            raise ValueError("a sampler needs one linear named 'logits'")
        self.stream = stream if stream is not None else torch.cuda.Stream()
        if attention is not None or sampler is not None:  # their buffers are filled on the current stream
            self.stream.wait_stream(torch.cuda.current_stream(self.stream.device))
        self.mode = mode
        self.graph: W4Graph | None = None
        self.chain = None
        if mode == "chain":
            nbytes = w4_chain_workspace_bytes(self.linears)
            self.workspace = torch.zeros(nbytes + 256, dtype=torch.uint8, device="cuda")
            off = (-self.workspace.data_ptr()) % 256
            self.chain = w4_chain_create(self.linears, self.workspace[off:off + nbytes])

    def _check_layers(self) -> None:
        """Each layer is one of the attention's and has q, k and v once, and its o after them."""
        seen = {}
        for lin in self.linears:
            name, layer = lin["name"], lin["layer"]
            if name not in ("q", "k", "v", "o"):
                continue
            if not 0 <= layer < len(self.attention.caches):
                raise ValueError(f"layer {layer}: the attention has {len(self.attention.caches)} layers")
            names = seen.setdefault(layer, [])
            if name in names:
                raise ValueError(f"layer {layer} has two linears named '{name}'")
            if "o" in names:
                raise ValueError(f"layer {layer}: o comes before {name}, which its attention reads")
            names.append(name)
        for layer, names in seen.items():
            for name in ("q", "k", "v"):
                if name not in names:
                    raise ValueError(f"layer {layer} has no linear named '{name}'")

    def run_eager(self) -> None:
        """Run the step directly on the step's stream (no graph)."""
        if self.mode == "chain":
            w4_chain_run(self.chain, stream=self.stream)
            return
        if self.attention is not None:
            self.attention.begin(self.stream)
        made = {}  # of each layer: its q, k and v
        for lin in self.linears:
            w4_gemv(lin["x"], lin["qw"], lin["s"], lin["z"], lin["y"], stream=self.stream)
            if self.attention is None and self.sampler is None:
                continue
            name, layer = lin["name"], lin["layer"]
            if self.attention is not None and name in ("q", "k", "v"):
                got = made.setdefault(layer, {})
                got[name] = lin["y"]
                if len(got) == 3:
                    self.attention.run(layer, got["q"], got["k"], got["v"], self.stream)
            if self.sampler is not None and name == "logits":
                self.sampler.run(lin["y"], self.stream)
        if self.attention is not None:
            self.attention.end(self.stream)

    def capture(self) -> W4Graph:
        """Record the chain into a graph (nothing runs during capture)."""
        if self.graph is not None:
            self.graph.destroy()
        torch.cuda.synchronize()
        w4_graph_begin(self.stream)
        try:
            self.run_eager()
        finally:
            # ending the capture also ends it after a failed launch
            graph = w4_graph_end(self.stream)
        self.graph = graph
        return graph

    def replay(self) -> None:
        if self.graph is None:
            self.capture()
        self.graph.replay(self.stream)

    def destroy(self) -> None:
        if self.graph is not None:
            self.graph.destroy()
            self.graph = None
        if self.chain is not None:
            self.chain.destroy()
            self.chain = None
