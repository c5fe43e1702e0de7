"""The decode step's operators between its INT4 linears, as cases to measure.

Four operators of a serving step over a paged cache that holds keys and
values in 4 bits:

  plan    block tables, slot maps and positions from the requests' lengths
  store   per-head norm of queries and keys, position rotation, and the keys
          and values written into the 4-bit cache (read back from it here,
          as the values that the codes stand for)
  attend  attention over the 4-bit cache: one query a sequence or many,
          causal, with an optional sliding window and first tokens that stay
          visible
  sample  a token from each row of logits: temperature, top-k, top-p, min-p
          and a given uniform number

The cache.  A page holds ``block`` tokens of every key/value head.  Codes are
4 bits, eight to an int32 word (bits 4j..4j+3 of word p: d = 8p + j), with an
FP16 scale s and an FP16 minimum m for each token and group of
min(head_dim, 128) values: x = q * s + m.
  k_codes int32 [pages, heads, block, dim / 8]
  v_codes int32 [pages, heads, block / 4, dim / 8, 4]   (the last axis: token % 4)
  k_meta, v_meta float16 [pages, heads, groups, block, 2]   (s, m)

``own`` false computes each operator from elementary torch operations; true
calls the library.
"""
import math
import random

import torch

own = False

GROUP = 128
NEG = float("-inf")


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One request's next token on a sliding-window layer (window 1024, 16
        # query and 8 key/value heads of 256): the smallest call, all latency.
        {"name": "attend-one", "op": "attend", "batch": 1, "new": 1, "kv": 1000, "ragged": False, "hq": 16, "hkv": 8,
         "dim": 256, "block": 64, "window": 1024, "sinks": 0, "mix": 1},
        # A decode batch on a global layer: requests of very different lengths.
        {"name": "attend-batch", "op": "attend", "batch": 32, "new": 1, "kv": 8192, "ragged": True, "hq": 16, "hkv": 8,
         "dim": 256, "block": 64, "window": 0, "sinks": 0, "mix": 2},
        # One request with a very long context: few rows, so the keys are split.
        {"name": "attend-long", "op": "attend", "batch": 1, "new": 1, "kv": 131071, "ragged": False, "hq": 32,
         "hkv": 8, "dim": 128, "block": 128, "window": 0, "sinks": 0, "mix": 3},
        # A decode batch of long requests on window layers whose first tokens
        # stay visible; small pages, eight query heads to a key head.
        {"name": "attend-window", "op": "attend", "batch": 64, "new": 1, "kv": 8000, "ragged": True, "hq": 64,
         "hkv": 8, "dim": 64, "block": 16, "window": 1024, "sinks": 4, "mix": 4},
        # A prompt's chunk of 2048 tokens after 2048 that are cached already.
        {"name": "attend-chunk", "op": "attend", "batch": 1, "new": 2048, "kv": 4096, "ragged": False, "hq": 16,
         "hkv": 8, "dim": 256, "block": 64, "window": 0, "sinks": 0, "mix": 5},
        # The step of a decode batch of 16 on the decoder's own head layout.
        {"name": "store-batch", "op": "store", "tokens": 16, "hq": 16, "hkv": 8, "dim": 256, "rot": 256,
         "pairs": False, "block": 64, "norm": True, "cached": True, "mix": 6},
        # A prompt of odd length.
        {"name": "store-prompt", "op": "store", "tokens": 4099, "hq": 16, "hkv": 8, "dim": 256, "rot": 256,
         "pairs": False, "block": 64, "norm": True, "cached": True, "mix": 7},
        # Norm and rotation alone (keys returned, no cache): heads of 128, a
        # rotation of half the head in neighbouring pairs.
        {"name": "norm-rope", "op": "store", "tokens": 8192, "hq": 32, "hkv": 8, "dim": 128, "rot": 64,
         "pairs": True, "block": 64, "norm": True, "cached": False, "mix": 8},
        # The tables of a decode batch: one new token a request.
        {"name": "plan-decode", "op": "plan", "batch": 256, "new": 1, "kv": 8192, "block": 16, "mix": 9},
        # The tables of a step that mixes prompts and decoding requests.
        {"name": "plan-prompts", "op": "plan", "batch": 1000, "new": 300, "kv": 16384, "block": 64, "mix": 10},
        # One row of the decoder's logits (vocabulary 262144).
        {"name": "sample-one", "op": "sample", "rows": 1, "vocab": 262144, "mix": 11},
        # A batch's rows, each with settings of its own.
        {"name": "sample-batch", "op": "sample", "rows": 64, "vocab": 262144, "mix": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "store", "store", "plan", "sample"))
    mix = rng.randrange(1 << 20)
    if op == "attend":
        dim = rng.choice((64, 128, 256))
        hkv = rng.choice((1, 2, 4, 8))
        hq = hkv * rng.choice((1, 2, 3, 4, 8))
        case = {"op": op, "batch": 1, "new": 1, "kv": 1, "ragged": rng.random() < 0.7, "hq": hq, "hkv": hkv,
                "dim": dim, "block": rng.choice((16, 32, 64, 128)), "window": rng.choice((0, 0, 128, 1000, 1024)),
                "sinks": rng.choice((0, 0, 1, 4, 33)), "mix": mix}
        if rng.random() < 0.6:  # decoding
            case["batch"] = _log(rng, 1, 64)
            case["kv"] = _log(rng, 1, min(131072, 262144 * 8 // (case["batch"] * hkv)))
        else:  # prompts and their chunks
            case["batch"] = _log(rng, 1, 8)
            case["new"] = _log(rng, 2, 2048 // case["batch"])
            case["kv"] = case["new"] + rng.choice((0, _log(rng, 1, 2048)))
        return case
    if op == "store":
        dim = rng.choice((64, 128, 256))
        hkv = rng.choice((1, 2, 4, 8))
        cached = rng.random() < 0.7
        return {"op": op, "tokens": _log(rng, 1, 4100), "hq": hkv * rng.choice((1, 2, 4)), "hkv": hkv, "dim": dim,
                "rot": rng.choice((dim, dim, dim // 2, 16)), "pairs": rng.random() < 0.4,
                "block": rng.choice((16, 32, 64, 128)), "norm": rng.random() < 0.8, "cached": cached, "mix": mix}
    if op == "plan":
        return {"op": op, "batch": _log(rng, 1, 1000), "new": rng.choice((1, 1, 2, 17, 300)),
                "kv": _log(rng, 16, 16384), "block": rng.choice((16, 32, 64, 128)), "mix": mix}
    return {"op": op, "rows": _log(rng, 1, 64), "vocab": _log(rng, 100, 262144), "mix": mix}


def _lengths(case):
    """(new tokens, cached and new tokens) of every request: the case's alone."""
    rng = random.Random(case["mix"])
    new, kv = [], []
    for _ in range(case["batch"]):
        n, t = case["new"], case["kv"]
        if case["op"] == "plan":
            n = rng.choice((0, 1, 1, 1)) if n == 1 else rng.choice((1, 1, rng.randint(1, n)))
            t = n + (0 if rng.random() < 0.1 else rng.randint(0, max(0, t - n)))
        elif case["ragged"]:
            n = rng.randint(1, n)
            t = max(n, rng.randint(1, t))
        new.append(n)
        kv.append(t)
    return new, kv


def _visible(case):
    """(query-key pairs that a row sees, keys that some row of their request sees), over all requests."""
    pairs = keys = 0
    w, s = case["window"], case["sinks"]
    for n, t in zip(*_lengths(case)):
        first = t - n
        if not w:
            pairs += n * first + n * (n + 1) // 2
            keys += t
            continue
        for p in range(first, t):
            low = max(0, p - w + 1)
            pairs += p + 1 - low + min(s, low)
        low = max(0, first - w + 1)
        keys += t - low + min(s, low)
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "attend":
        pairs, keys = _visible(case)
        groups = max(1, case["dim"] // GROUP)
        rows = sum(_lengths(case)[0])
        token = 2 * (case["dim"] // 2 + 4 * groups)
        return {"bytes": keys * case["hkv"] * token + 2 * 2 * rows * case["hq"] * case["dim"],
                "flops": 4 * pairs * case["hq"] * case["dim"]}
    if op == "store":
        t, d, hq, hkv = case["tokens"], case["dim"], case["hq"], case["hkv"]
        table = 4 * case["rot"] * t
        packed = 2 * (d // 2 + 4 * max(1, d // GROUP))
        if case["cached"]:  # q, k, v in; q and the cache's rows out; these rows in again and k, v out
            size = 2 * t * d * (2 * hq + 4 * hkv) + 2 * t * hkv * packed
        else:
            size = 2 * t * d * (2 * hq + 2 * hkv)
        return {"bytes": size + table, "flops": 8 * t * d * (hq + hkv)}
    if op == "plan":
        new, kv = _lengths(case)
        pages = sum(-(-t // case["block"]) for t in kv)
        return {"bytes": 4 * (4 * case["batch"] + 2 * pages + 2 * sum(new)), "flops": 0}
    return {"bytes": 2 * case["rows"] * case["vocab"], "flops": 4 * case["rows"] * case["vocab"]}


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


def _cache(case, g, pages):
    h, b, d = case["hkv"], case["block"], case["dim"]
    groups = max(1, d // GROUP)
    return {"k_codes": _words(g, (pages, h, b, d // 8)), "v_codes": _words(g, (pages, h, b // 4, d // 8, 4)),
            "k_meta": _scales(g, (pages, h, groups, b)), "v_meta": _scales(g, (pages, h, groups, b))}


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op == "attend":
        new, kv = _lengths(case)
        need = [-(-t // case["block"]) for t in kv]
        pages, wide = sum(need) + 3, max(need) + 1
        s["cache"] = _cache(case, g, pages)
        order = torch.randperm(pages, generator=g, device="cuda").int()
        table, at = torch.full((case["batch"], wide), -1, dtype=torch.int32, device="cuda"), 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        s["table"], s["kv_lens"], s["q_start"] = table, _int(kv), _int(_starts(new))
        s["max_q"], s["max_kv"] = max(new), max(kv)
        s["q"] = torch.randn((sum(new), case["hq"], case["dim"]), generator=g, device="cuda").bfloat16()
        s["out"] = torch.zeros_like(s["q"])
    elif op == "store":
        t, hq, hkv, d = (case[n] for n in ("tokens", "hq", "hkv", "dim"))
        # the three linears' outputs side by side, as a fused product leaves them
        qkv = torch.randn((t, hq + 2 * hkv, d), generator=g, device="cuda").bfloat16()
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16()
                                        for _ in range(2)) if case["norm"] else (None, None)
        reach = 8192
        turn = torch.arange(reach, dtype=torch.float64, device="cuda")[:, None] * torch.pow(
            torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
            -torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        s["cos_sin"] = torch.cat((turn.cos(), turn.sin()), dim=1).float().contiguous()
        s["positions"] = torch.randint(0, reach, (t,), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.zeros((t, hq, d), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros((t, hkv, d), dtype=torch.bfloat16, device="cuda")
        if case["cached"]:
            pages = -(-t // case["block"]) + 2
            s["cache"] = _cache(case, g, pages)
            s["slots"] = torch.randperm(pages * case["block"], generator=g, device="cuda")[:t].int()
            s["v_out"] = torch.zeros_like(s["k_out"])
    elif op == "plan":
        new, kv = _lengths(case)
        b, block = case["batch"], case["block"]
        wide = max(-(-t // block) for t in kv) + 1
        pages = sum(-(-t // block) for t in kv) + 5
        order = torch.randperm(pages, generator=g, device="cuda").int()
        table, at = torch.full((b, wide), -1, dtype=torch.int32), 0
        order_host = order.cpu()
        for i, (n, t) in enumerate(zip(new, kv)):
            held = -(-(t - n) // block)
            table[i, :held] = order_host[at:at + held]
            at += held
        s["table"] = table.cuda()
        s["free"] = order[at:].contiguous()
        s["free_count"] = _int([pages - at])
        s["cached"], s["new"] = _int([t - n for n, t in zip(new, kv)]), _int(new)
        rows = sum(new) + 7  # a few rows of padding behind the last request
        s["q_start"], s["kv_lens"] = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (b + 1, b))
        s["positions"], s["slots"] = (torch.zeros(rows, dtype=torch.int32, device="cuda") for _ in range(2))
        s["counts"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    else:
        r, v = case["rows"], case["vocab"]
        s["logits"] = (3 * torch.randn((r, v), generator=g, device="cuda")).bfloat16()
        rng = random.Random(case["mix"])
        kinds = [(rng.choice((0.0, 0.6, 0.7, 1.0, 1.0, 1.3)), rng.choice((0, 0, 1, 20, 50, 1000)),
                  rng.choice((1.0, 0.9, 0.95, 0.5)), rng.choice((0.0, 0.0, 0.05, 0.001))) for _ in range(r)]
        if r == 1:
            kinds = [(0.7, 64, 0.95, 0.0)]
        for name, column, dtype in (("temperature", 0, torch.float32), ("top_k", 1, torch.int32),
                                    ("top_p", 2, torch.float32), ("min_p", 3, torch.float32)):
            s[name] = torch.tensor([k[column] for k in kinds], dtype=dtype, device="cuda")
        s["uniform"] = torch.rand(r, generator=g, device="cuda", dtype=torch.float64)
        s["tokens"] = torch.zeros(r, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _unpack(words):
    """int32 [..., n] -> codes [..., 8 n], int32."""
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device=words.device)
    return ((words[..., None] >> shifts) & 15).flatten(-2)


def _pack(codes):
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device=codes.device)
    return (codes.unflatten(-1, (-1, 8)) << shifts).sum(dim=-1, dtype=torch.int32)


def _values(words, meta):
    """Packed words [..., dim / 8] and their (s, m) [..., groups, 2] -> values in 32 bits."""
    groups = meta.shape[-2]
    q = _unpack(words).float().unflatten(-1, (groups, -1))
    return (q * meta[..., 0:1].float() + meta[..., 1:2].float()).flatten(-2)


def _plain_attend(s):
    case, c = s["case"], s["cache"]
    hkv, d, block, g = case["hkv"], case["dim"], case["block"], case["hq"] // case["hkv"]
    q, start, lens = s["q"], s["q_start"], s["kv_lens"]
    b, nq, reach = lens.numel(), s["max_q"], s["max_kv"]
    used = -(-reach // block)
    pages = s["table"][:, :used].clamp(min=0).long()
    # [batch, heads, tokens, dim]
    k = _values(c["k_codes"][pages], c["k_meta"][pages].transpose(3, 4)).transpose(1, 2).flatten(2, 3)
    v = _values(c["v_codes"][pages].transpose(4, 5).flatten(3, 4), c["v_meta"][pages].transpose(3, 4)).transpose(
        1, 2).flatten(2, 3)
    i = torch.arange(nq, device=q.device)
    rows = (start[:-1, None] + i).clamp(max=q.shape[0] - 1).long()
    qp = q[rows].float().unflatten(2, (hkv, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [batch, heads, g nq, dim]
    scores = torch.matmul(qp, k.transpose(2, 3).contiguous()) / math.sqrt(d)
    place = (lens - (start[1:] - start[:-1]))[:, None] + i  # each query's position
    t = torch.arange(k.shape[2], device=q.device)
    see = t <= place[..., None]
    if case["window"]:
        see = see & ((t > place[..., None] - case["window"]) | (t < case["sinks"]))
    see = see[:, None].repeat(1, g, 1, 1).flatten(1, 2)[:, None]
    scores = scores.masked_fill(~see, NEG)
    top = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == NEG, 0.0, top))
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v.contiguous()) / torch.where(total > 0, total, 1.0)
    o = o.unflatten(2, (g, nq)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [batch, nq, query heads, dim]
    row = torch.arange(q.shape[0], device=q.device)
    seq = (torch.searchsorted(start, row.int(), right=True) - 1).clamp(max=b - 1)
    return o[seq, row - start[seq]].bfloat16()


def _turned(x, weight, s):
    """Norm over each head and rotation, in 64 bits (a cached key's code lies next to a border now and then)."""
    case = s["case"]
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(dim=-1, keepdim=True) + 1e-6) * weight.double()
    rot = case["rot"]
    half = rot // 2
    table = s["cos_sin"][s["positions"].long()].double()[:, None]
    cos, sin = table[..., :half], table[..., half:]
    head, tail = y[..., :rot], y[..., rot:]
    if case["pairs"]:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((head, tail), dim=-1).float().bfloat16()


def _quantised(x):
    """bfloat16 [..., dim] -> packed words and (s, m)."""
    groups = max(1, x.shape[-1] // GROUP)
    y = x.float().unflatten(-1, (groups, -1))
    low, high = y.amin(dim=-1), y.amax(dim=-1)
    s = ((high - low) * (1.0 / 15.0)).half()
    m = low.half()
    inverse = torch.where(s > 0, 1.0 / s.double(), 0.0).float()
    codes = torch.round((y - m.float()[..., None]) * inverse[..., None]).clamp(0, 15).int()
    return _pack(codes.flatten(-2)), torch.stack((s, m), dim=-1)


def _plain_store(s):
    q = _turned(s["q"], s["q_weight"], s)
    k = _turned(s["k"], s["k_weight"], s)
    if not s["case"]["cached"]:
        return q, k
    c, block = s["cache"], s["case"]["block"]
    page, at = s["slots"].long() // block, s["slots"].long() % block
    c["k_codes"][page, :, at], k_meta = _quantised(k)
    c["k_meta"][page, :, :, at] = k_meta
    c["v_codes"][page, :, at // 4, :, at % 4], v_meta = _quantised(s["v"])
    c["v_meta"][page, :, :, at] = v_meta
    kr = _values(c["k_codes"][page, :, at], c["k_meta"][page, :, :, at])
    vr = _values(c["v_codes"][page, :, at // 4, :, at % 4], c["v_meta"][page, :, :, at])
    return q, kr.bfloat16(), vr.bfloat16()


def _plain_plan(s):
    block, table, cached, new = s["case"]["block"], s["table"], s["cached"], s["new"]
    b, wide = table.shape
    total = cached + new
    held = torch.div(cached + block - 1, block, rounding_mode="floor").clamp(max=wide)
    pages = torch.div(total + block - 1, block, rounding_mode="floor").clamp(max=wide)
    need = pages - held
    ends = torch.cumsum(need, 0, dtype=torch.int32)
    column = torch.arange(wide, dtype=torch.int32, device=table.device)
    take = s["free_count"] - 1 - ((ends - need)[:, None] + column - held[:, None])
    fresh = (column >= held[:, None]) & (column < pages[:, None])
    given = torch.where(take >= 0, s["free"][take.clamp(0, max(0, s["free"].numel() - 1)).long()], -1)
    table.copy_(torch.where(fresh, given, table))
    start = torch.cat((torch.zeros_like(ends[:1]), torch.cumsum(new, 0, dtype=torch.int32)))
    row = torch.arange(s["slots"].numel(), dtype=torch.int32, device=table.device)
    seq = (torch.searchsorted(start, row, right=True) - 1).clamp(max=b - 1)
    live = row < start[-1]
    place = cached[seq] + row - start[seq]
    page = table[seq, torch.div(place, block, rounding_mode="floor").clamp(max=wide - 1).long()]
    slot = torch.where(live & (page >= 0), page * block + place % block, -1)
    counts = torch.stack((s["free_count"][0] - ends[-1], ends[-1] - s["free_count"][0])).clamp(min=0)
    return start, total, torch.where(live, place, -1), slot, table, counts


def _plain_sample(s):
    x = s["logits"].double()
    heat = s["temperature"].double()[:, None]
    values, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((values - values[:, :1]) / torch.where(heat > 0, heat, 1.0))
    rank = torch.arange(x.shape[1], device=x.device)
    k = torch.where(s["top_k"] > 0, s["top_k"], x.shape[1])[:, None]
    keep = rank < torch.where(heat > 0, k, 1)
    ends = torch.cumsum(w, dim=1)
    before = torch.cat((torch.zeros_like(ends[:, :1]), ends[:, :-1]), dim=1)
    p = s["top_p"].double()[:, None]
    keep = keep & ((p >= 1) | (before < p * (w * keep).sum(dim=1, keepdim=True)) | (rank == 0))
    keep = keep & ((w >= s["min_p"].double()[:, None]) | (rank == 0))
    target = s["uniform"][:, None] * (w * keep).sum(dim=1, keepdim=True)
    at = torch.minimum((ends <= target).sum(dim=1), keep.sum(dim=1) - 1)
    return order.gather(1, at[:, None])[:, 0].int()


# -------------------------------------------------------- the library's own
def _handle(s):
    """The cache object and workspace that a program keeps."""
    import gemm_w4_gemv_amd as w4
    if "handle" not in s and "cache" in s:
        c = s["cache"]
        s["handle"] = w4.Kv4Cache(c["k_codes"], c["k_meta"], c["v_codes"], c["v_meta"])
    if "work" not in s:
        case, size = s["case"], 0
        if case["op"] == "attend":
            size = w4.w4_kv4_attn_workspace_bytes(s["handle"], s["q"].shape[0], case["batch"], case["hq"], s["max_q"],
                                                  s["max_kv"], window=case["window"], sinks=case["sinks"])
        elif case["op"] == "sample":
            size = w4.w4_sample_workspace_bytes(case["rows"], case["vocab"])
        s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    return w4, s.get("handle"), s["work"]


def _own(s):
    w4, cache, space = _handle(s)
    case, op = s["case"], s["case"]["op"]
    if op == "attend":
        return w4.w4_kv4_attn(s["q"], cache, s["table"], s["kv_lens"], s["out"], q_start=s["q_start"],
                              max_q=s["max_q"], max_kv=s["max_kv"], window=case["window"], sinks=case["sinks"],
                              workspace=space)
    if op == "store":
        more = {"v": s["v"], "cache": cache, "slots": s["slots"]} if case["cached"] else {"k_out": s["k_out"]}
        w4.w4_qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], q_out=s["q_out"], q_weight=s["q_weight"],
                           k_weight=s["k_weight"], eps=1e-6, interleaved=case["pairs"], **more)
        if not case["cached"]:
            return s["q_out"], s["k_out"]
        w4.w4_kv4_read(cache, s["slots"], s["k_out"], s["v_out"])
        return s["q_out"], s["k_out"], s["v_out"]
    if op == "plan":
        w4.w4_kv4_plan(s["cached"], s["new"], s["table"], s["free"], s["free_count"], case["block"], s["q_start"],
                       s["kv_lens"], s["positions"], s["slots"], s["counts"])
        return s["q_start"], s["kv_lens"], s["positions"], s["slots"], s["table"], s["counts"]
    return w4.w4_sample(s["logits"], s["uniform"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"],
                        top_p=s["top_p"], min_p=s["min_p"], workspace=space)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "attend":
        return _plain_attend(state)
    if op == "store":
        return _plain_store(state)
    if op == "plan":
        return _plain_plan(state)
    return _plain_sample(state)


# ------------------------------------------------------------ in 64 bits
def _nibbles(words):
    w = words.long() & 0xFFFFFFFF
    return torch.stack([(w >> (4 * j)) & 15 for j in range(8)], dim=-1).flatten(-2).double()


def _exact_attend(case, s):
    c, d, block = s["cache"], case["dim"], case["block"]
    g = case["hq"] // case["hkv"]
    size = min(d, GROUP)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    new, kv = _lengths(case)
    at = 0
    for i, (n, t) in enumerate(zip(new, kv)):
        place = torch.arange(t, device="cuda")
        page, off = s["table"][i].long()[place // block], place % block
        see = torch.arange(t - n, t, device="cuda")[:, None] - place  # how far back each key lies
        dark = see < 0
        if case["window"]:
            dark = dark | ((see >= case["window"]) & (place >= case["sinks"]))
        for h in range(case["hkv"]):
            both = []
            for words, meta in ((c["k_codes"][page, h, off], c["k_meta"]),
                                (c["v_codes"][page, h, off // 4, :, off % 4], c["v_meta"])):
                m = meta[page, h, :, off].double().repeat_interleave(size, dim=1)
                both.append(_nibbles(words) * m[..., 0] + m[..., 1])
            for j in range(h * g, h * g + g):
                z = s["q"][at:at + n, j].double() @ both[0].T / d ** 0.5
                z[dark] = NEG
                out[at:at + n, j] = torch.softmax(z, dim=1) @ both[1]
        at += n
    return out


def _exact_heads(case, s, x, weight):
    y = x.double()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.double()
    n = case["rot"] // 2
    row = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(row[:, :n], row[:, n:])[:, None]
    first = torch.arange(n, device="cuda") * (2 if case["pairs"] else 1)
    second = first + (1 if case["pairs"] else n)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_cached(x):
    """What the cache stands for: the nearest of 16 steps up from each group's minimum."""
    size = min(x.shape[-1], GROUP)
    y = x.bfloat16().double().unflatten(-1, (-1, size))
    low = y.min(-1, keepdim=True).values
    step = ((y.max(-1, keepdim=True).values - low) / 15).half().double()
    low = low.half().double()
    q = torch.where(step > 0, ((y - low) / step).round(), 0.0).clamp(0, 15)
    return (q * step + low).flatten(-2)


def exact(case, seed):
    if case["op"] in ("plan", "sample"):
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    q, k = _exact_heads(case, s, s["q"], s["q_weight"]), _exact_heads(case, s, s["k"], s["k_weight"])
    return (q, _exact_cached(k), _exact_cached(s["v"])) if case["cached"] else (q, k)
