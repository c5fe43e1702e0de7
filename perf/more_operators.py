"""Operators of a batched layer around its 4-bit products, as cases to measure.

Four operators that a serving (or tuning) program calls next to the library's
linears, experts and 4-bit key/value cache:

  share   attention of a batch whose requests begin with the same tokens: the
          shared pages are worked on once for all requests, each one's own
          tokens after them as ever; over the paged 4-bit cache
  norm    the norm of a block's output, its gate and residual sum, and the norm
          that the next block reads, in one pass; and the gradient of these
  sort    tokens sorted by expert: row ranges, every choice's row, and the
          rows of activations that the experts' products read
  back    the experts' rows back to their tokens with weights applied, and the
          gradient of sorting and going back

The cache is as in ``perf/operators.py``: codes of 4 bits, eight to an int32
word, an FP16 scale s and minimum m for each token and group of
min(head_dim, 128) values, x = q * s + m.

``own`` false computes each operator from elementary torch operations; true
calls the library.
"""
import math
import random

import torch

own = False

GROUP = 128
NEG = float("-inf")
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # Four requests behind one system prompt, a token each: the smallest
        # batch that shares anything, all latency.
        {"name": "share-few", "op": "share", "batch": 4, "new": 1, "prefix": 1024, "own": 100, "hq": 16, "hkv": 8,
         "dim": 256, "block": 64, "window": 0, "sinks": 0, "mix": 1},
        # A decode batch behind a long prompt, each with a history of its own.
        {"name": "share-batch", "op": "share", "batch": 32, "new": 1, "prefix": 8192, "own": 1024, "hq": 16,
         "hkv": 8, "dim": 256, "block": 64, "window": 0, "sinks": 0, "mix": 2},
        # Questions about one long document: the most work.
        {"name": "share-long", "op": "share", "batch": 64, "new": 1, "prefix": 16384, "own": 2000, "hq": 32,
         "hkv": 8, "dim": 128, "block": 128, "window": 0, "sinks": 0, "mix": 3},
        # Drafted tokens checked, up to five a request; small pages, an odd
        # number of them shared, eight query heads to a key head.
        {"name": "share-drafts", "op": "share", "batch": 24, "new": 5, "prefix": 4112, "own": 300, "hq": 64,
         "hkv": 8, "dim": 64, "block": 16, "window": 0, "sinks": 0, "mix": 4},
        # One token between two blocks of the decoder (hidden size 3840).
        {"name": "norm-one", "op": "norm", "tokens": 1, "dim": 3840, "wide": False, "gate": "none", "post": True,
         "grad": False, "mix": 5},
        # A prompt of odd length, with a gate for each channel.
        {"name": "norm-prompt", "op": "norm", "tokens": 4099, "dim": 3840, "wide": False, "gate": "channel",
         "post": True, "grad": False, "mix": 6},
        # Its gradient over a training batch, the residual stream in FP32.
        {"name": "norm-grad", "op": "norm", "tokens": 8192, "dim": 4096, "wide": True, "gate": "channel",
         "post": True, "grad": True, "mix": 7},
        # A decode batch routed to 6 of 64 experts (hidden size 4096).
        {"name": "sort-batch", "op": "sort", "tokens": 64, "top": 6, "experts": 64, "dim": 4096, "capacity": 0,
         "padding": 0.0, "mix": 8},
        # A prompt's tokens, with room for a bounded number at each expert and
        # some padding that no expert gets.
        {"name": "sort-prompt", "op": "sort", "tokens": 8191, "top": 6, "experts": 64, "dim": 4096, "capacity": 1024,
         "padding": 0.02, "mix": 9},
        # The way back of the same batch, onto the output of a shared expert.
        {"name": "back-batch", "op": "back", "tokens": 64, "top": 6, "experts": 64, "dim": 4096, "capacity": 0,
         "padding": 0.0, "add": True, "grad": False, "mix": 10},
        {"name": "back-prompt", "op": "back", "tokens": 8191, "top": 6, "experts": 64, "dim": 4096, "capacity": 1024,
         "padding": 0.02, "add": True, "grad": False, "mix": 11},
        # The gradients that tuning a router needs: of the experts' rows, the
        # weights and the tokens.
        {"name": "back-grad", "op": "back", "tokens": 4096, "top": 6, "experts": 64, "dim": 4096, "capacity": 0,
         "padding": 0.0, "add": False, "grad": True, "mix": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("share", "share", "share", "norm", "norm", "sort", "back", "back"))
    mix = rng.randrange(1 << 20)
    if op == "share":
        dim = rng.choice((64, 128, 256))
        hkv = rng.choice((1, 2, 4, 8))
        hq = hkv * rng.choice((1, 2, 3, 4, 8))
        block = rng.choice((16, 32, 64, 128))
        batch = _log(rng, 2, 64)
        new = rng.choice((1, 1, 1, 1, 3, 8))
        most = (1 << 32) // (batch * new * hq * dim)  # no more work than share-long
        mine = max(new, _log(rng, 1, min(2000, most // 2)))
        prefix = max(block, _log(rng, 32, min(16384, most - mine)) // block * block)
        return {"op": op, "batch": batch, "new": new, "prefix": prefix, "own": mine, "hq": hq, "hkv": hkv, "dim": dim,
                "block": block, "window": rng.choice((0, 0, 0, 500, 1024)), "sinks": rng.choice((0, 0, 4)), "mix": mix}
    if op == "norm":
        dim = 8 * _log(rng, 16, 2048)
        return {"op": op, "tokens": _log(rng, 1, 8192 * 4096 // max(dim, 4096)), "dim": dim,
                "wide": rng.random() < 0.4, "gate": rng.choice(("none", "channel", "token")),
                "post": rng.random() < 0.8, "grad": rng.random() < 0.4, "mix": mix}
    experts = _log(rng, 4, 256)
    case = {"op": op, "tokens": _log(rng, 1, 8191), "top": min(experts, rng.choice((1, 2, 4, 6, 8))),
            "experts": experts, "dim": 8 * _log(rng, 16, 512), "capacity": 0, "padding": rng.choice((0.0, 0.0, 0.1)),
            "mix": mix}
    if case["tokens"] * case["top"] * case["dim"] > 8191 * 6 * 4096:
        case["tokens"] = 8191 * 6 * 4096 // (case["top"] * case["dim"])
    if rng.random() < 0.3:  # a little more than an even share
        case["capacity"] = 1 + case["tokens"] * case["top"] * 5 // (4 * experts)
    if op == "back":
        case["grad"] = rng.random() < 0.4
        case["add"] = not case["grad"] and rng.random() < 0.5
        if case["grad"]:
            case["tokens"] = -(-case["tokens"] // 2)
    return case


def _lengths(case):
    """(new tokens, cached and new tokens) of every request: the case's alone."""
    rng = random.Random(case["mix"])
    new = [rng.randint(1, case["new"]) for _ in range(case["batch"])]
    return new, [case["prefix"] + max(n, rng.randint(1, case["own"])) for n in new]


def _routed(case):
    """int32 [tokens, top] on the host: each token's experts, some popular, -1 for padding; the case's alone."""
    g = torch.Generator().manual_seed(case["mix"])
    t, e = case["tokens"], case["experts"]
    popular = 1.5 * torch.rand(e, generator=g)
    ids = torch.topk(popular + torch.randn((t, e), generator=g), case["top"], dim=1).indices.int()
    ids[torch.rand(t, generator=g) < case["padding"]] = -1
    return ids


def _kept(case):
    """How many choices get a row."""
    ids = _routed(case).flatten()
    counts = torch.bincount(ids[ids >= 0].long(), minlength=case["experts"])
    return int((counts.clamp(max=case["capacity"]) if case["capacity"] else counts).sum())


def work(case):
    op = case["op"]
    if op == "share":
        d, w, s = case["dim"], case["window"], case["sinks"]
        new, kv = _lengths(case)
        pairs = own = 0
        first = case["prefix"]  # the first shared token that some row sees (but for the first tokens)
        for n, t in zip(new, kv):
            for p in range(t - n, t):
                low = max(0, p - w + 1) if w else 0
                pairs += p + 1 - low + min(s, low)
            low = max(0, t - n - w + 1) if w else 0
            own += t - max(low, case["prefix"])
            first = min(first, low)
        keys = own + case["prefix"] - first + min(s, first)
        packed = 2 * (d // 2 + 4 * max(1, d // GROUP))
        return {"bytes": keys * case["hkv"] * packed + 4 * sum(new) * case["hq"] * d, "flops": 4 * pairs * case["hq"] * d}
    t, d = case["tokens"], case["dim"]
    if op == "norm":
        h = 4 if case["wide"] else 2
        gate = {"none": 0, "channel": 2 * d, "token": 2 * t * d}[case["gate"]]
        if case["grad"]:  # h, y and both gradients in; two gradients, and the gate's, out
            return {"bytes": t * d * (3 * h + 6) + 2 * gate + 12 * d, "flops": 30 * t * d}
        return {"bytes": t * d * (2 * h + 4) + gate + 4 * d, "flops": 12 * t * d}
    rows, ids = _kept(case), 4 * t * case["top"]
    if op == "sort":  # ids in, row numbers and sources out; tokens in, rows out
        return {"bytes": 3 * ids + 2 * d * (t + rows), "flops": 0}
    if case["grad"]:  # the output's gradient and the rows in, the rows' gradient out; that of the sorted rows in, the tokens' out
        return {"bytes": 3 * ids + 2 * d * (2 * t + 3 * rows), "flops": 4 * rows * d}
    return {"bytes": 2 * ids + 2 * d * (rows + t * (2 if case["add"] else 1)), "flops": 2 * rows * d}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _words(g, shape):
    """Packed codes whose values lie about the middle of 0..15, as quantised values do."""
    a, b, c = (torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device="cuda", dtype=torch.int32)
               for _ in range(3))
    # two draws of 0..7 and one of 0..1 in each nibble; no carry leaves it
    return (a & 0x77777777) + (b & 0x77777777) + (c & 0x11111111)


def _scales(g, shape):
    """FP16 (scale, minimum) of groups whose values have about unit variance and a mean near 0."""
    s = 0.25 + 0.2 * torch.rand(shape, generator=g, device="cuda")
    m = -7.5 * s + 0.3 * torch.randn(shape, generator=g, device="cuda")
    return torch.stack((s, m), dim=-1).half()


def _normal(g, shape, dtype=torch.bfloat16, size=1.0):
    return (size * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_share(case, s, g):
    new, kv = _lengths(case)
    block, h, d, b = case["block"], case["hkv"], case["dim"], case["batch"]
    groups = max(1, d // GROUP)
    shared = case["prefix"] // block
    need = [-(-t // block) - shared for t in kv]
    pages = shared + sum(need) + 3
    s["cache"] = {"k_codes": _words(g, (pages, h, block, d // 8)),
                  "v_codes": _words(g, (pages, h, block // 4, d // 8, 4)),
                  "k_meta": _scales(g, (pages, h, groups, block)), "v_meta": _scales(g, (pages, h, groups, block))}
    order = torch.randperm(pages, generator=g, device="cuda").int()
    s["prefix_table"] = order[:shared].contiguous()
    table, at = torch.full((b, shared + max(need) + 1), -1, dtype=torch.int32, device="cuda"), shared
    table[:, :shared] = s["prefix_table"]
    for i, n in enumerate(need):
        table[i, shared:shared + n] = order[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["table"], s["kv_lens"], s["q_start"] = table, _int(kv), _int(starts)
    s["max_q"], s["max_kv"] = max(new), max(kv)
    s["q"] = _normal(g, (sum(new), case["hq"], d))
    s["out"] = torch.zeros_like(s["q"])


def _prepare_norm(case, s, g):
    t, d = case["tokens"], case["dim"]
    kind = torch.float32 if case["wide"] else torch.bfloat16
    # a residual stream has grown over the layers, in some channels more than in others
    grown = torch.exp(0.7 * torch.randn(d, generator=g, device="cuda"))
    s["h"] = (3 * grown * torch.randn((t, d), generator=g, device="cuda")).to(kind)
    s["y"] = _normal(g, (t, d))
    s["y_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16() if case["post"] else None
    s["z_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16()
    s["gate"] = None if case["gate"] == "none" else _normal(g, (d,) if case["gate"] == "channel" else (t, d), size=0.5)
    rng = random.Random(case["mix"])
    s["scales"] = {"residual_scale": rng.choice((1.0, 1.0, 0.9)), "branch_scale": rng.choice((1.0, 1.0, 0.22))}
    if not case["grad"]:
        s["h_out"], s["z"] = torch.zeros_like(s["h"]), torch.zeros_like(s["y"])
        return
    s["dh_out"], s["dz"] = _normal(g, (t, d), kind, 0.1), _normal(g, (t, d))
    s["dh"], s["dy"] = torch.zeros_like(s["h"]), torch.zeros_like(s["y"])
    s["d_z_weight"] = torch.zeros(d, device="cuda")
    s["d_y_weight"] = torch.zeros(d, device="cuda") if case["post"] else None
    s["d_gate"] = {"none": None, "channel": torch.zeros(d, device="cuda"),
                   "token": torch.zeros_like(s["y"])}[case["gate"]]


def _rows_of(ids, experts, capacity):
    """(first row of every expert, row of every choice) by a stable sort; -1 where a choice gets none."""
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    begin = torch.cumsum(counts, 0) - counts
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order), device=order.device)
    sound = key < experts
    inside = key.clamp(max=experts - 1)
    place = place - begin[inside]  # among its expert's choices
    if capacity:
        counts = counts.clamp(max=capacity)
        sound = sound & (place < capacity)
    start = torch.cat((counts.new_zeros(1), torch.cumsum(counts, 0)))
    return start.int(), torch.where(sound, start[inside] + place, -1).int().view(ids.shape)


def _prepare_routed(case, s, g):
    t, k, d = case["tokens"], case["top"], case["dim"]
    s["experts"] = _routed(case).cuda()
    if case["op"] == "sort":
        s["x"] = _normal(g, (t, d))
        s["rows"] = torch.zeros((t * k, d), dtype=torch.bfloat16, device="cuda")
        s["row_start"] = torch.zeros(case["experts"] + 1, dtype=torch.int32, device="cuda")
        s["row_of"] = torch.zeros((t, k), dtype=torch.int32, device="cuda")
        s["source"] = torch.zeros(t * k, dtype=torch.int32, device="cuda")
        return
    s["row_of"] = _rows_of(s["experts"], case["experts"], case["capacity"])[1]
    s["weights"] = torch.softmax(torch.randn((t, k), generator=g, device="cuda"), dim=1)
    s["y"] = _normal(g, (t * k, d))
    if not case["grad"]:
        s["add"] = _normal(g, (t, d)) if case["add"] else None
        s["out"] = torch.zeros((t, d), dtype=torch.bfloat16, device="cuda")
        return
    s["dout"], s["drows"] = _normal(g, (t, d)), _normal(g, (t * k, d))
    s["dy"], s["dx"] = torch.zeros_like(s["y"]), torch.zeros_like(s["dout"])
    s["dweights"] = torch.zeros_like(s["weights"])


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": dict(case)}
    {"share": _prepare_share, "norm": _prepare_norm}.get(case["op"], _prepare_routed)(case, s, g)
    return s


# ------------------------------------------------------------- plain forms
def _unpack(words):
    """int32 [..., n] -> codes [..., 8 n], int32."""
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device=words.device)
    return ((words[..., None] >> shifts) & 15).flatten(-2)


def _values(words, meta):
    """Packed words [..., dim / 8] and their (s, m) [..., groups, 2] -> values in 32 bits."""
    groups = meta.shape[-2]
    q = _unpack(words).float().unflatten(-1, (groups, -1))
    return (q * meta[..., 0:1].float() + meta[..., 1:2].float()).flatten(-2)


def _pages_of(c, pages):
    """Keys and values [..., heads, tokens, dim] of pages [..., n]."""
    k = _values(c["k_codes"][pages], c["k_meta"][pages].transpose(-3, -2))
    v = _values(c["v_codes"][pages].transpose(-2, -1).flatten(-3, -2), c["v_meta"][pages].transpose(-3, -2))
    return tuple(x.transpose(-4, -3).flatten(-3, -2).contiguous() for x in (k, v))


def _plain_share(s):
    case, c, table = s["case"], s["cache"], s["table"]
    hkv, d, g = case["hkv"], case["dim"], case["hq"] // case["hkv"]
    q, start, lens, nq, b, far = s["q"], s["q_start"], s["kv_lens"], s["max_q"], case["batch"], case["prefix"]
    first = far // case["block"]
    k0, v0 = _pages_of(c, s["prefix_table"].long())  # [heads, prefix, dim], once for all
    k1, v1 = _pages_of(c, table[:, first:-(-s["max_kv"] // case["block"])].clamp(min=0).long())
    i = torch.arange(nq, device=q.device)
    rows = (start[:-1, None] + i).clamp(max=q.shape[0] - 1).long()
    qp = q[rows].float().unflatten(2, (hkv, g)).permute(2, 0, 3, 1, 4)  # [heads, batch, g, nq, dim]
    z0 = torch.matmul(qp.flatten(1, 3), k0.transpose(1, 2).contiguous()).unflatten(1, (b, g, nq))
    z1 = torch.matmul(qp.flatten(2, 3), k1.transpose(0, 1).transpose(2, 3).contiguous()).unflatten(2, (g, nq))
    z = torch.cat((z0, z1), dim=-1) / math.sqrt(d)
    place = ((lens - (start[1:] - start[:-1]))[:, None] + i)[:, None, :, None]  # each query's position
    t = torch.arange(z.shape[-1], device=q.device)
    see = t <= place
    if case["window"]:
        see = see & ((t > place - case["window"]) | (t < case["sinks"]))
    z = z.masked_fill(~see, NEG)
    top = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - torch.where(top == NEG, 0.0, top))
    total = p.sum(dim=-1, keepdim=True)
    p0, p1 = p[..., :far].contiguous(), p[..., far:].contiguous()
    o = torch.matmul(p0.flatten(1, 3), v0).unflatten(1, (b, g, nq))
    o = o + torch.matmul(p1.flatten(2, 3), v1.transpose(0, 1).contiguous()).unflatten(2, (g, nq))
    o = (o / torch.where(total > 0, total, 1.0)).permute(1, 3, 0, 2, 4).flatten(2, 3)  # [batch, nq, query heads, dim]
    row = torch.arange(q.shape[0], device=q.device)
    seq = (torch.searchsorted(start, row.int(), right=True) - 1).clamp(max=b - 1)
    return o[seq, row - start[seq]].bfloat16()


def _scaled(x):
    """1 / root mean square of each row."""
    return torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)


def _branch(s):
    """(norm of y before its weight, the block's gated output, h after it), in 32 bits."""
    y = s["y"].float()
    n1 = y * _scaled(y) if s["y_weight"] is not None else None
    u = y if n1 is None else n1 * s["y_weight"].float()
    gated = u if s["gate"] is None else u * s["gate"].float()
    return n1, u, s["scales"]["residual_scale"] * s["h"].float() + s["scales"]["branch_scale"] * gated


def _plain_norm(s):
    case = s["case"]
    n1, u, h = _branch(s)
    r2 = _scaled(h)
    if not case["grad"]:
        return h.to(s["h"].dtype), (h * r2 * s["z_weight"].float()).bfloat16()
    dz, n2 = s["dz"].float(), h * r2
    d2 = dz * s["z_weight"].float()
    dh = s["dh_out"].float() + r2 * (d2 - n2 * (d2 * n2).mean(dim=-1, keepdim=True))
    branch = s["scales"]["branch_scale"] * dh
    out = [(s["scales"]["residual_scale"] * dh).to(s["h"].dtype)]
    du = branch if s["gate"] is None else branch * s["gate"].float()
    if n1 is None:
        out.append(du.bfloat16())
    else:
        d1 = du * s["y_weight"].float()
        out.append((_scaled(s["y"].float()) * (d1 - n1 * (d1 * n1).mean(dim=-1, keepdim=True))).bfloat16())
        out.append((du * n1).sum(dim=0, dtype=torch.float64).float())
    out.append((dz * n2).sum(dim=0, dtype=torch.float64).float())
    if case["gate"] == "channel":
        out.append((branch * u).sum(dim=0, dtype=torch.float64).float())
    elif case["gate"] == "token":
        out.append((branch * u).bfloat16())
    return out


def _plain_sort(s):
    case = s["case"]
    start, row_of = _rows_of(s["experts"], case["experts"], case["capacity"])
    flat = row_of.flatten().long()
    choice = torch.arange(len(flat), dtype=torch.int32, device=flat.device)
    source = torch.full((len(flat) + 1,), -1, dtype=torch.int32, device=flat.device)
    source[torch.where(flat >= 0, flat, len(flat))] = choice
    source[-1] = -1
    source = source[:-1]
    live = (source >= 0)[:, None]
    s["rows"].copy_(torch.where(live, s["x"][(source.clamp(min=0) // case["top"]).long()], s["rows"]))
    return start, row_of, source, s["rows"]


def _plain_back(s):
    case = s["case"]
    live = s["row_of"] >= 0
    at = s["row_of"].clamp(min=0).long()
    if not case["grad"]:
        out = torch.zeros(s["out"].shape, device="cuda") if s["add"] is None else s["add"].float()
        for j in range(case["top"]):
            part = s["weights"][:, j:j + 1] * s["y"][at[:, j]].float()
            out = out + torch.where(live[:, j:j + 1], part, 0.0)
        return out.bfloat16()
    dout = s["dout"].float()
    dx = torch.zeros_like(dout)
    dw = torch.zeros_like(s["weights"])
    for j in range(case["top"]):
        here = live[:, j:j + 1]
        dw[:, j] = torch.where(live[:, j], (dout * s["y"][at[:, j]].float()).sum(dim=1), 0.0)
        dx = dx + torch.where(here, s["drows"][at[:, j]].float(), 0.0)
        s["dy"][at[live[:, j], j]] = (s["weights"][:, j:j + 1] * dout)[live[:, j]].bfloat16()
    return s["dy"], dw, dx.bfloat16()


# -------------------------------------------------------- the library's own
def _handle(s):
    """The cache object and workspace that a program keeps."""
    import gemm_w4_gemv_amd as w4
    if "work" not in s:
        case, size = s["case"], 0
        if case["op"] == "share":
            c = s["cache"]
            s["handle"] = w4.Kv4Cache(c["k_codes"], c["k_meta"], c["v_codes"], c["v_meta"])
            size = w4.w4_kv4_attn_shared_workspace_bytes(s["handle"], s["q"].shape[0], case["batch"], case["hq"],
                                                         s["max_q"], s["max_kv"], case["prefix"],
                                                         window=case["window"], sinks=case["sinks"])
        elif case["op"] == "norm" and case["grad"]:
            size = w4.w4_block_norm_grad_workspace_bytes(case["tokens"], case["dim"])
        elif case["op"] == "sort":
            size = w4.w4_moe_sort_workspace_bytes(case["tokens"], case["top"], case["experts"])
        s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    return w4, s.get("handle"), s["work"]


def _own(s):
    w4, cache, space = _handle(s)
    case, op = s["case"], s["case"]["op"]
    if op == "share":
        return w4.w4_kv4_attn_shared(s["q"], cache, s["table"], s["kv_lens"], s["out"], s["prefix_table"],
                                     case["prefix"], q_start=s["q_start"], max_q=s["max_q"], max_kv=s["max_kv"],
                                     window=case["window"], sinks=case["sinks"], workspace=space)
    if op == "norm" and not case["grad"]:
        w4.w4_block_norm(s["h"], s["y"], h_out=s["h_out"], z=s["z"], y_weight=s["y_weight"], z_weight=s["z_weight"],
                         gate=s["gate"], eps=EPS, **s["scales"])
        return s["h_out"], s["z"]
    if op == "norm":
        w4.w4_block_norm_grad(s["h"], s["y"], dh_out=s["dh_out"], dz=s["dz"], dh=s["dh"], dy=s["dy"],
                              y_weight=s["y_weight"], z_weight=s["z_weight"], gate=s["gate"],
                              d_y_weight=s["d_y_weight"], d_z_weight=s["d_z_weight"], d_gate=s["d_gate"], eps=EPS,
                              workspace=space, **s["scales"])
        return [x for x in (s["dh"], s["dy"], s["d_y_weight"], s["d_z_weight"], s["d_gate"]) if x is not None]
    if op == "sort":
        w4.w4_moe_sort(s["experts"], case["experts"], s["row_start"], s["row_of"], source=s["source"], x=s["x"],
                       rows=s["rows"], capacity=case["capacity"], workspace=space)
        return s["row_start"], s["row_of"], s["source"], s["rows"]
    if not case["grad"]:
        return w4.w4_moe_combine(s["y"], s["out"], row_of=s["row_of"], weights=s["weights"], add=s["add"])
    w4.w4_moe_combine_grad(s["dout"], s["y"], row_of=s["row_of"], weights=s["weights"], dy=s["dy"],
                           dweights=s["dweights"])
    w4.w4_moe_combine(s["drows"], s["dx"], row_of=s["row_of"])
    return s["dy"], s["dweights"], s["dx"]


def run(state):
    if own:
        return _own(state)
    return {"share": _plain_share, "norm": _plain_norm, "sort": _plain_sort, "back": _plain_back}[
        state["case"]["op"]](state)


# ------------------------------------------------------------ in 64 bits
def _nibbles(words):
    w = words.long() & 0xFFFFFFFF
    return torch.stack([(w >> (4 * j)) & 15 for j in range(8)], dim=-1).flatten(-2).double()


def _exact_share(case, s):
    c, d, block = s["cache"], case["dim"], case["block"]
    g, size = case["hq"] // case["hkv"], min(case["dim"], GROUP)

    def tokens(table, first, last, h):
        place = torch.arange(first, last, device="cuda")
        page, off = table.long()[place // block], place % block
        both = []
        for words, meta in ((c["k_codes"][page, h, off], c["k_meta"]),
                            (c["v_codes"][page, h, off // 4, :, off % 4], c["v_meta"])):
            m = meta[page, h, :, off].double().repeat_interleave(size, dim=1)
            both.append(_nibbles(words) * m[..., 0] + m[..., 1])
        return both

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    new, kv = _lengths(case)
    for h in range(case["hkv"]):
        shared = tokens(s["table"][0], 0, case["prefix"], h)
        at = 0
        for i, (n, t) in enumerate(zip(new, kv)):
            k, v = (torch.cat(x) for x in zip(shared, tokens(s["table"][i], case["prefix"], t, h)))
            q = s["q"][at:at + n, h * g:h * g + g].double()
            z = torch.matmul(q, k.T) / d ** 0.5  # [new, g, tokens]
            back = torch.arange(t - n, t, device="cuda")[:, None] - torch.arange(t, device="cuda")
            dark = back < 0
            if case["window"]:
                dark = dark | ((back >= case["window"]) & (torch.arange(t, device="cuda") >= case["sinks"]))
            z = z.masked_fill(dark[:, None], NEG)
            out[at:at + n, h * g:h * g + g] = torch.matmul(torch.softmax(z, dim=-1), v)
            at += n
    return out


def _exact_norm(case, s):
    """The forward from its definition; the gradient from its derivatives by torch's own rules."""
    leaves = {n: s[n].double().requires_grad_(case["grad"]) for n in ("h", "y", "y_weight", "z_weight", "gate")
              if s[n] is not None}

    def normed(x, weight):
        return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * weight

    u = normed(leaves["y"], leaves["y_weight"]) if case["post"] else leaves["y"]
    if "gate" in leaves:
        u = leaves["gate"] * u
    h = s["scales"]["residual_scale"] * leaves["h"] + s["scales"]["branch_scale"] * u
    z = normed(h, leaves["z_weight"])
    if not case["grad"]:
        return h, z
    names = [n for n in ("h", "y", "y_weight", "z_weight", "gate") if n in leaves]
    return list(torch.autograd.grad((h, z), [leaves[n] for n in names], (s["dh_out"].double(), s["dz"].double())))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "share":
        return _exact_share(case, s)
    if op == "norm":
        return _exact_norm(case, s)
    t, k, d = case["tokens"], case["top"], case["dim"]
    if op == "sort":  # whole numbers, and the tokens expert by expert
        flat, rows, at = s["experts"].flatten(), s["rows"].double(), 0
        for e in range(case["experts"]):
            here = (flat == e).nonzero()[:, 0][:case["capacity"] or None]
            rows[at:at + len(here)] = s["x"][here // k].double()
            at += len(here)
        return None, None, None, rows
    # a matrix [tokens, choices] would be the definition; choice by choice it is the same sums
    token = torch.arange(t, device="cuda")[:, None].expand(t, k)[s["row_of"] >= 0]
    row = s["row_of"][s["row_of"] >= 0].long()
    w = s["weights"][s["row_of"] >= 0].double()[:, None]
    if not case["grad"]:
        out = s["add"].double() if case["add"] else torch.zeros((t, d), dtype=torch.float64, device="cuda")
        return out.index_add_(0, token, w * s["y"][row].double())
    dout = s["dout"].double()[token]
    dy = torch.zeros((t * k, d), dtype=torch.float64, device="cuda")
    dy[row] = w * dout
    dw = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    dw[s["row_of"] >= 0] = (dout * s["y"][row].double()).sum(dim=1)
    dx = torch.zeros((t, d), dtype=torch.float64, device="cuda")
    return dy, dw, dx.index_add_(0, token, s["drows"][row].double())
