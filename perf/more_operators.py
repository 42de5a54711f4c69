"""Rotary positions on the way into the quantised cache, and attention through a window: cases, plain forms, exact results.

Three operators are measured here:

  append  binding.kv_append_rotary: new keys turned by their positions and quantised into the paged cache with their values,
          the queries of the same rows turned beside them
  rotary  binding.rotary: rows turned by positions of one or several axes (time, height, width), or turned back, which is
          also the turning's gradient
  window  binding.window_attention: the rows of every request's block (1 row = plain decoding) over the last tokens before
          each of them and over a few first ones that stay visible, of a prefix that the batch shares and of its own

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits (angles in 64).
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}
_AMAX_FLOOR = 2.0 ** -100     # the least row maximum a scale is made from
_BASE = 10000.0               # frequencies of pair i: _BASE ** (-i / pairs)


# ---------------------------------------------------------------------------------------------------------- cases ---
def listed():
    return [
        # one new token for each request of a small decoding batch: latency
        dict(name="append decode", op="append", B=32, rows_lo=1, rows_hi=1, ctx_lo=100, ctx_hi=2000, prefix=0, Hq=32, Hkv=8,
             D=128, page=64, dtype="bf16", format="e4m3", pairs=64, pairing="halves", axes=1, order="blocks"),
        # the scheduled block rows (1 to 6 of each request) of a large batch behind a shared prompt; a quarter of the head
        # turned, in adjacent pairs
        dict(name="append blocks", op="append", B=256, rows_lo=1, rows_hi=6, ctx_lo=0, ctx_hi=500, prefix=700, Hq=16, Hkv=4,
             D=64, page=16, dtype="fp16", format="int8", pairs=8, pairing="adjacent", axes=1, order="blocks"),
        # prompts of many requests entering the cache at once
        dict(name="append prompts", op="append", B=13, rows_lo=500, rows_hi=8000, ctx_lo=0, ctx_hi=77, prefix=0, Hq=32,
             Hkv=8, D=128, page=64, dtype="bf16", format="e4m3", pairs=64, pairing="halves", axes=1, order="blocks"),
        # prompts with images in them: positions of three axes
        dict(name="append images", op="append", B=7, rows_lo=300, rows_hi=2500, ctx_lo=0, ctx_hi=40, prefix=0, Hq=28, Hkv=4,
             D=128, page=32, dtype="bf16", format="e4m3", pairs=64, pairing="halves", axes=3, order="blocks"),
        # the patches of one small image
        dict(name="rotary image", op="rotary", rows=529, heads=16, D=64, dtype="fp16", layout="rows", inverse=False,
             pairs=32, pairing="halves", axes=2, order="blocks"),
        # a video's patches, heads first, heads of 80
        dict(name="rotary video", op="rotary", rows=60001, heads=16, D=80, dtype="bf16", layout="heads", inverse=False,
             pairs=40, pairing="halves", axes=3, order="cycled"),
        # gradients of turned rows, in 32 bits
        dict(name="rotary gradient", op="rotary", rows=9000, heads=32, D=128, dtype="fp32", layout="rows", inverse=True,
             pairs=64, pairing="adjacent", axes=1, order="blocks"),
        # a single request, a single token: the smallest step of plain decoding
        dict(name="window one token", op="window", B=1, rows_lo=1, rows_hi=1, ctx_lo=8999, ctx_hi=8999, prefix=0, window=1024,
             sinks=4, Hq=32, Hkv=8, D=128, page=64, dtype="bf16", format="e4m3", mask="causal"),
        # plain decoding of a batch whose contexts have mostly passed the window
        dict(name="window decode", op="window", B=64, rows_lo=1, rows_hi=1, ctx_lo=500, ctx_hi=20000, prefix=0, window=4096,
             sinks=4, Hq=64, Hkv=8, D=128, page=64, dtype="bf16", format="e4m3", mask="causal"),
        # the scheduled blocks of a batch of 256 behind a short system prompt that holds the first tokens
        dict(name="window blocks", op="window", B=256, rows_lo=1, rows_hi=6, ctx_lo=100, ctx_hi=6000, prefix=700, window=1024,
             sinks=16, Hq=32, Hkv=8, D=128, page=64, dtype="bf16", format="e4m3", mask="causal"),
        # drafted trees of up to 40 nodes, small heads, small pages, no first tokens
        dict(name="window trees", op="window", B=48, rows_lo=9, rows_hi=40, ctx_lo=50, ctx_hi=1500, prefix=333, window=500,
             sinks=0, Hq=24, Hkv=8, D=64, page=16, dtype="fp16", format="int8", mask="tree"),
        # prompts of a few requests, read in one pass
        dict(name="window prompts", op="window", B=4, rows_lo=1500, rows_hi=4096, ctx_lo=0, ctx_hi=2000, prefix=0, window=1024,
             sinks=4, Hq=32, Hkv=8, D=128, page=64, dtype="bf16", format="e4m3", mask="causal"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm when the range is wide."""
    if hi <= 10 * max(lo, 1):
        return rng.randint(lo, hi)
    return int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))


def _draw_rotary(rng, D):
    pairing = rng.choice(["halves", "halves", "adjacent"])
    return dict(pairs=8 * rng.randint(1, D // 16) if rng.random() < 0.3 else D // 2, pairing=pairing,
                axes=rng.choice([1, 1, 2, 3]), order=rng.choice(["blocks", "cycled"]))


def draw(rng):
    op = rng.choice(["append", "rotary", "window", "window"])
    fmt = rng.choice(["e4m3", "e4m3", "int8"])
    Hkv, D, page = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 128, 96]), rng.choice([16, 32, 64, 128, 48])
    if op == "rotary":
        D, heads = rng.choice([64, 80, 96, 128, 128, 256]), rng.choice([1, 3, 8, 16, 32])
        return dict(op=op, rows=_spread(rng, 1, min(60000, (1 << 27) // (heads * D))), heads=heads, D=D,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), layout=rng.choice(["rows", "heads"]),
                    inverse=rng.choice([False, False, True]), **_draw_rotary(rng, D))
    group = rng.choice([1, 2, 4, 5, 8])
    if op == "append":
        B = _spread(rng, 1, 256)
        hi = _spread(rng, 1, max(1, min(8000, (1 << 25) // (B * Hkv * (group + 2) * D))))
        return dict(op=op, B=B, rows_lo=max(1, hi // rng.choice([1, 2, 10])), rows_hi=hi, ctx_lo=0, ctx_hi=_spread(rng, 1, 500),
                    prefix=rng.choice([0, rng.randint(1, 2000), 1000003]), Hq=Hkv * group, Hkv=Hkv, D=D, page=page,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), format=fmt, **_draw_rotary(rng, D))
    B, hi = _spread(rng, 1, 256), rng.choice([1, 1, 1, 2, 5, 6, 9, 17, 33, _spread(rng, 64, 4000)])
    ctx_hi = _spread(rng, 16, 60000)
    case = dict(op=op, B=B, rows_lo=max(1, hi - rng.choice([0, 2, 16])), rows_hi=hi, ctx_lo=ctx_hi // rng.choice([1, 2, 8, 64]),
                ctx_hi=ctx_hi, prefix=rng.choice([0, 0, _spread(rng, 16, 3000)]), window=_spread(rng, 64, 32000),
                sinks=rng.choice([0, 1, 4, 4, 16, 133]), Hq=Hkv * group, Hkv=Hkv, D=D, page=page,
                dtype=rng.choice(["bf16", "fp16"]), format=fmt,
                mask=rng.choice(["causal", "causal", "full", "tree" if hi <= 64 else "causal"]))
    while True:     # no more tokens or products than the largest listed cases, and scores that the plain form can hold
        w = work(case)
        tokens = min(case["window"] + case["rows_hi"], case["ctx_hi"] + case["prefix"] + case["rows_hi"]) + case["sinks"]
        if w["flops"] <= 2e11 and w["bytes"] <= 6e8 and case["B"] * case["rows_hi"] * case["Hq"] * tokens <= 3e9 \
                and case["B"] * tokens * Hkv * D <= 6e8 and case["B"] * (ctx_hi + hi) * Hkv * D <= 3e9:
            return case
        case["B"] = max(1, case["B"] * 3 // 4)
        case["ctx_hi"] = ctx_hi = max(1, case["ctx_hi"] * 3 // 4)
        case["ctx_lo"] = min(case["ctx_lo"], ctx_hi)
        if case["B"] == 1 and case["rows_hi"] > 64:
            case["rows_hi"] = max(64, case["rows_hi"] * 3 // 4)
            case["rows_lo"] = min(case["rows_lo"], case["rows_hi"])


def _lengths(case):
    """Rows and earlier tokens of every request: fixed by the case alone, so that ``work`` is exact."""
    rng = random.Random("%(B)d %(rows_lo)d %(rows_hi)d %(ctx_lo)d %(ctx_hi)d" % case)
    rows = [rng.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["B"])]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    return rows, ctx


def _tree_words(case):
    """The drafted trees: node i of a request hangs under an earlier node (node 0 is the committed token); a node's word
    has the bits of its ancestors and its own."""
    rng = random.Random("tree %(B)d %(rows_lo)d %(rows_hi)d" % case)
    words = []
    for n in _lengths(case)[0]:
        seen = [1]
        for i in range(1, n):
            seen.append(1 << i | seen[rng.randrange(max(0, i - 4), i)])
        words.append(seen)
    return words


def work(case):
    D = case["D"]
    size = _DTYPES[case["dtype"]].itemsize
    if case["op"] == "rotary":
        elements = case["rows"] * case["heads"] * D
        return {"bytes": 2 * elements * size + 4 * case["axes"] * case["rows"], "flops": 3 * elements}
    rows, ctx = _lengths(case)
    R, Hq, Hkv, P = sum(rows), case["Hq"], case["Hkv"], case["prefix"]
    if case["op"] == "append":
        return {"bytes": R * (Hkv * (2 * D * size + 2 * D + 8) + 2 * Hq * D * size), "flops": R * D * (5 * Hkv + 3 * Hq)}
    W, S, words = case["window"], case["sinks"], _tree_words(case) if case["mask"] == "tree" else None
    tokens, pairs, first = 0, 0, P
    for b, (n, c) in enumerate(zip(rows, ctx)):
        C = P + c
        low = max(0, C - W + 1)                                   # the first row's first token of the window
        first = min(first, low)
        tokens += min(max(0, S - P), c + n) + max(0, C + n - max(low, S, P))
        if words:
            for w in words[b]:
                depth = bin(w).count("1")
                pairs += min(S, C) + max(0, C - max(S, C - max(0, W - depth), 0)) + depth
        elif case["mask"] == "full":
            pairs += sum(min(S, C + n) + max(0, C + n - max(S, C + i - W + 1, 0)) for i in range(n))
        else:
            pairs += sum(min(S, C + i + 1) + max(0, C + i + 1 - max(S, C + i - W + 1, 0)) for i in range(n))
    tokens += min(S, P) + max(0, P - max(first, S))               # the prefix's, once for all
    return {"bytes": tokens * Hkv * (2 * D + 8) + R * Hq * (2 * D * size + 4), "flops": 4 * D * Hq * pairs}


# --------------------------------------------------------------------------------------------------------- inputs ---
def _quantise(x, fmt):
    """Codes and scales of the rows of x, in 32 bits: the format's definition."""
    dt, top = _FORMATS[fmt]
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True).clamp_min(_AMAX_FLOOR)
    q = torch.full_like(amax, top)      # a tensor: dividing by or into a plain number may go through its reciprocal
    y = (x * (q / amax)).clamp(-top, top)
    codes = y.to(dt) if fmt == "e4m3" else torch.round(y).to(dt)
    return codes, (amax / q).squeeze(-1)


def _tables(case, gen, device):
    """Shuffled pages: [B, max_pages] of each request and [prefix pages] of the shared prefix."""
    rows, ctx = _lengths(case)
    page = case["page"]
    need = [-(-(c + n) // page) for c, n in zip(ctx, rows)]
    shared = -(-case["prefix"] // page) if case["op"] == "window" else 0
    n_pages = sum(need) + shared + 3
    order = torch.randperm(n_pages, generator=gen, device=device).to(torch.int32)
    slot = torch.arange(max(need), device=device)[None, :]
    first = torch.tensor([0] + need, device=device).cumsum(0)[:-1, None]
    held = slot < torch.tensor(need, device=device)[:, None]
    table = torch.where(held, order[torch.where(held, first + slot, 0)], 0).to(torch.int32)
    return n_pages, table.contiguous(), order[sum(need):sum(need) + shared].contiguous()


def _axis_of_pair(case):
    """Which axis turns each pair: sections one after the other (the first, time's, half as wide), or in turns."""
    pairs, axes = case["pairs"], case["axes"]
    if case["order"] == "cycled" or axes == 1:
        return [i % axes for i in range(pairs)]
    ends = [(2 * a + 1) * pairs // (2 * axes - 1) for a in range(axes)]
    return [sum(i >= e for e in ends) for i in range(pairs)]


def _positions(case, starts, counts, gen, device):
    """Positions [axes, rows] of rows that follow each other: the first axis by row (or frame), the others by a grid."""
    n = sum(counts)
    row = torch.arange(n, device=device) - torch.repeat_interleave(
        torch.tensor([0] + list(counts), device=device).cumsum(0)[:-1], torch.tensor(counts, device=device), output_size=n)
    start = torch.repeat_interleave(torch.tensor(starts, device=device), torch.tensor(counts, device=device), output_size=n)
    if case["axes"] == 1:
        return (start + row)[None].to(torch.int32)
    width = int(torch.randint(20, 60, (1,), generator=gen, device=device))
    height = int(torch.randint(20, 60, (1,), generator=gen, device=device))
    grid = [row // (height * width), row // width % height, row % width]
    return torch.stack([start + g for g in grid[-case["axes"]:]]).to(torch.int32).contiguous()


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    st = dict(case=case)
    if case["op"] != "window":
        st["inv_freq"] = _BASE ** (-torch.arange(case["pairs"], dtype=torch.float64) / case["pairs"])
        st["freq"], st["axis"] = st["inv_freq"].to(dev), torch.tensor(_axis_of_pair(case), device=dev)
    if case["op"] == "rotary":
        shape = (case["rows"], case["heads"]) if case["layout"] == "rows" else (case["heads"], case["rows"])
        x = torch.randn((*shape, case["D"]), generator=gen, device=dev).to(dt)
        st["x"] = x if case["layout"] == "rows" else x.transpose(0, 1)
        st["positions"] = _positions(case, [seed % 100], [case["rows"]], gen, dev)
        return st
    rows, ctx = _lengths(case)
    R, Hq, Hkv, D, page, fmt = sum(rows), case["Hq"], case["Hkv"], case["D"], case["page"], case["format"]
    n_pages, st["table"], st["prefix_pages"] = _tables(case, gen, dev)
    st["row0"] = torch.tensor([0] + rows, device=dev, dtype=torch.int64).cumsum(0)
    st["ctx"] = torch.tensor(ctx, device=dev, dtype=torch.int32)
    st["rows_host"], st["ctx_host"] = rows, ctx
    shape = (n_pages, Hkv, page, D)

    def channels():     # keys and values have a few channels much larger than the others
        return torch.exp(0.5 * torch.randn((Hkv, 1, D), generator=gen, device=dev))

    if case["op"] == "append":
        st["codes"] = [torch.zeros(shape, dtype=torch.uint8, device=dev).view(_FORMATS[fmt][0]) for _ in range(2)]
        st["scales"] = [torch.zeros(shape[:3], device=dev) for _ in range(2)]
        qkv = torch.randn((R, Hq + 2 * Hkv, D), generator=gen, device=dev).to(dt)      # one fused projection's rows
        qkv[:, Hq:Hq + Hkv] *= channels()[:, 0].to(dt)
        qkv[:, Hq + Hkv:] *= channels()[:, 0].to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        # of one axis the call knows the positions itself: behind the prefix and the cached tokens
        st["positions"] = _positions(case, [case["prefix"] + c for c in ctx], rows, gen, dev) if case["axes"] > 1 else None
        return st
    st["codes"], st["scales"] = [], []
    for _ in range(2):
        codes = torch.empty(shape, dtype=torch.uint8, device=dev).view(_FORMATS[fmt][0])
        scales = torch.empty(shape[:3], device=dev)
        ch = channels()
        step = max(1, (1 << 28) // (Hkv * page * D))
        for i in range(0, n_pages, step):
            x = torch.randn((min(step, n_pages - i), Hkv, page, D), generator=gen, device=dev) * ch
            c, scales[i:i + step] = _quantise(x, fmt)
            codes.view(torch.uint8)[i:i + step] = c.view(torch.uint8)
        st["codes"].append(codes)
        st["scales"].append(scales)
    st["q"] = (1.2 * torch.randn((R, Hq, D), generator=gen, device=dev)).to(dt)
    st["kv_len"] = torch.tensor([c + n for c, n in zip(ctx, rows)], device=dev, dtype=torch.int32)
    st["scale"] = D ** -0.5
    st["words"] = None
    if case["mask"] == "tree":
        words = [w - (1 << 64) if w >> 63 else w for seen in _tree_words(case) for w in seen]
        st["words"] = torch.tensor(words, device=dev, dtype=torch.int64)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:     # what a program keeps between calls: the cache's handle and the frequencies'
        from speculative_decoding_draft_head_gb300 import binding
        if "codes" in st:
            st["cache"] = binding.KVCache(st["codes"][0], st["codes"][1], st["scales"][0], st["scales"][1])
        if "freq" in st:
            st["rotary"] = binding.Rotary(st["inv_freq"], axis=_axis_of_pair(case) if case["axes"] > 1 else None,
                                          adjacent=case["pairing"] == "adjacent")
    return st


# ------------------------------------------------------------------------------------------------------------ run ---
def _stored(st):
    """The cache's codes as the numbers that they are, and the scales."""
    codes = [c.to(torch.float16) if c.dtype == torch.int8 else c for c in st["codes"]]
    return codes + st["scales"]


def run(st):
    case = st["case"]
    if own:
        from speculative_decoding_draft_head_gb300 import binding
        if case["op"] == "rotary":
            return binding.rotary(st["x"], st["rotary"], st["positions"], inverse=case["inverse"])
        if case["op"] == "append":
            q = binding.kv_append_rotary(st["k"], st["v"], st["cache"], st["table"], st["ctx"], st["row0"], st["rotary"],
                                         q=st["q"], positions=st["positions"], offset=0 if case["axes"] > 1 else case["prefix"])
            return _stored(st) + [q]
        got = binding.window_attention(st["q"], st["cache"], st["table"], st["kv_len"], st["row0"], window=case["window"],
                                       sinks=case["sinks"], prefix_pages=st["prefix_pages"], prefix_len=case["prefix"],
                                       mask="full" if case["mask"] == "full" else "causal", row_mask=st["words"],
                                       scale=st["scale"])
        return [got["out"], got["lse"]]
    if case["op"] == "rotary":
        return _turn(st, st["x"], st["positions"], case["inverse"]).to(st["x"].dtype)
    return _plain_append(st) if case["op"] == "append" else _plain_window(st)


def _turn(st, x, positions, inverse=False):
    """Rows x [n, heads, D] with their pairs turned by the angles of their positions [axes, n], in 32 bits."""
    n, case = st["case"]["pairs"], st["case"]
    angle = positions.double()[st["axis"]].T * st["freq"]         # [n, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sin = -sin
    x = x.float()
    y = x.clone()
    a, b = (slice(0, n), slice(n, 2 * n)) if case["pairing"] == "halves" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_append(st):
    case, page = st["case"], st["case"]["page"]
    row = torch.arange(st["k"].shape[0], device=st["k"].device)
    b = torch.searchsorted(st["row0"], row, right=True) - 1
    pos = st["ctx"].long()[b] + row - st["row0"][b]
    pg, off = st["table"].long()[b, pos // page], pos % page
    at = st["positions"] if st["positions"] is not None else (pos + case["prefix"])[None]
    for x, codes, scales in zip((_turn(st, st["k"], at), st["v"]), st["codes"], st["scales"]):
        c, s = _quantise(x, case["format"])
        codes.view(torch.uint8)[pg, :, off] = c.view(torch.uint8)
        scales[pg, :, off] = s
    return _stored(st) + [_turn(st, st["q"], at).to(st["q"].dtype)]


def _plain_window(st):
    case = st["case"]
    Hq, Hkv, D, page, P, W, S = (case[k] for k in ("Hq", "Hkv", "D", "page", "prefix", "window", "sinks"))
    dev, R = st["q"].device, st["q"].shape[0]
    n = st["row0"].diff()
    most = max(st["rows_host"])
    C = P + st["ctx"].long()                                      # tokens before each block
    end = C + n
    # the tokens that a request's rows can see: the first ones, then the window's from its first row on
    first = torch.arange(S, device=dev).expand(len(n), S)
    low = (C - W + 1).clamp_min(S)
    span = max(max(0, P + c + m - max(S, P + c - W + 1)) for m, c in zip(st["rows_host"], st["ctx_host"]))
    pos = torch.cat([first, low[:, None] + torch.arange(span, device=dev)], 1)
    there = pos < end[:, None]
    safe = torch.where(there, pos, 0)
    slot = (torch.where(safe < P, safe, safe - P)) // page
    pages = st["table"].long().gather(1, slot.clamp_max(st["table"].shape[1] - 1))
    if P:
        pages = torch.where(safe < P, st["prefix_pages"].long()[slot.clamp_max(len(st["prefix_pages"]) - 1)], pages)
    off = torch.where(safe < P, safe, safe - P) % page
    k, v = [codes.view(torch.uint8)[pages, :, off].view(codes.dtype).float() * scales[pages, :, off][..., None]
            for codes, scales in zip(st["codes"], st["scales"])]  # [B, T, Hkv, D]
    i = torch.arange(most, device=dev)
    row = (st["row0"][:-1, None] + i).clamp_max(R - 1)            # [B, most]
    q = st["q"].float()[row] * st["scale"]
    s = torch.einsum("bihgd,bthd->bhgit", q.view(len(n), most, Hkv, Hq // Hkv, D), k)
    t = pos[:, None, :] - C[:, None, None]                        # block token (or, below 0, one before)
    near = i[None, :, None] - t < W
    see = near & (t <= i[None, :, None]) if case["mask"] == "causal" else near
    if case["mask"] == "tree":
        word = st["words"][row]
        bits = word[..., None] >> torch.arange(64, device=dev) & 1
        see = torch.where(t >= 0, bits.gather(2, t.clamp(0, 63).expand(-1, most, -1)) == 1, -t <= W - bits.sum(2, keepdim=True))
    sink = pos[:, None, :] < S
    if case["mask"] == "causal":
        see = see | sink & (t <= i[None, :, None])
    else:
        see = see | sink & (t < 0) if case["mask"] == "tree" else see | sink
    see = (see & there[:, None])[:, None, None]
    s.masked_fill_(~see, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s.sub_(m))
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgit,bthd->bihgd", p, v) / total.squeeze(-1).permute(0, 3, 1, 2)[..., None]
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)
    held = i < n[:, None]                                         # padded rows leave
    return [out.reshape(len(n), most, Hq, D)[held].to(st["q"].dtype), lse.reshape(len(n), most, Hq)[held].contiguous()]


# ---------------------------------------------------------------------------------------------------------- exact ---
def _turned64(case, x, positions):
    """The same turning as products of complex numbers, in 64 bits: positions are a list with one tensor [n] per axis."""
    p = case["pairs"]
    axis = _axis_of_pair(case)
    x = x.double()
    turned = x.clone()
    for i in range(p):
        a, b = (i, i + p) if case["pairing"] == "halves" else (2 * i, 2 * i + 1)
        theta = positions[axis[i]].double() * _BASE ** (-i / p) * (-1 if case.get("inverse") else 1)
        z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(theta), theta)[:, None]
        turned[..., a], turned[..., b] = z.real, z.imag
    return turned


def exact(case, seed):
    """The operators' definitions in 64 bits.  Codes of e4m3 are given as the numbers before they are rounded to codes;
    int8 codes are whole numbers that the rounding of the 32-bit product decides, so they have no such value."""
    st = _inputs(case, seed)
    if case["op"] == "rotary":
        return _turned64(case, st["x"], list(st["positions"]))
    rows, ctx = _lengths(case)
    page, P, D = case["page"], case["prefix"], case["D"]
    if case["op"] == "append":
        own_pos = torch.cat([torch.arange(c, c + n, device="cuda") for n, c in zip(rows, ctx)])
        at = [own_pos + P] if st["positions"] is None else list(st["positions"])
        top = _FORMATS[case["format"]][1]
        stored = []
        for x in (_turned64(case, st["k"], at), st["v"].double()):
            amax = x.abs().amax(-1).clamp_min(_AMAX_FLOOR)
            c = torch.zeros(st["codes"][0].shape, dtype=torch.float64, device="cuda")
            s = torch.zeros(st["codes"][0].shape[:3], dtype=torch.float64, device="cuda")
            r = 0
            for b, n in enumerate(rows):
                pos = own_pos[r:r + n]
                pg, off = st["table"][b].long()[pos // page], pos % page
                c[pg, :, off] = x[r:r + n] * (top / amax[r:r + n])[..., None]
                s[pg, :, off] = amax[r:r + n] / top
                r += n
            stored.append((c if case["format"] == "e4m3" else None, s))
        return [stored[0][0], stored[1][0], stored[0][1], stored[1][1], _turned64(case, st["q"], at)]
    W, S, (R, Hq, _) = case["window"], case["sinks"], st["q"].shape
    if work(case)["flops"] > 1e12:
        return None
    group = Hq // case["Hkv"]
    out = torch.zeros((R, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((R, Hq), dtype=torch.float64, device="cuda")
    words = _tree_words(case) if case["mask"] == "tree" else None
    r = 0
    for b, (n, c) in enumerate(zip(rows, ctx)):
        C = P + c
        token = torch.arange(C + n, device="cuda")
        i = torch.arange(n, device="cuda")[:, None]
        if words is None:
            sees = (token > C + i - W) | (token < S)
            if case["mask"] == "causal":
                sees &= token <= C + i
        else:
            inside = torch.tensor([[w >> t & 1 for t in range(n)] for w in words[b]], device="cuda") == 1
            before = (token[:C] >= C - W + inside.sum(1, keepdim=True)) | (token[:C] < S)
            sees = torch.cat([before, inside], 1)
        use = sees.any(0).nonzero()[:, 0]
        sees, mine = sees[:, use], use >= P
        at = torch.where(mine, use - P, use)
        pages = torch.where(mine, st["table"][b].long()[(at // page).clamp_max(st["table"].shape[1] - 1)], 0)
        if P:
            shared = st["prefix_pages"].long()
            pages = torch.where(mine, pages, shared[(at // page).clamp_max(len(shared) - 1)])
        for h in range(case["Hkv"]):
            k, v = [codes.view(torch.uint8)[pages, h, at % page].view(codes.dtype).double()
                    * scales[pages, h, at % page].double()[:, None] for codes, scales in zip(st["codes"], st["scales"])]
            heads = slice(h * group, (h + 1) * group)
            s = torch.einsum("igd,td->igt", st["q"][r:r + n, heads].double(), k) * st["scale"]
            s = s + torch.where(sees, 0.0, float("-inf")).double()[:, None]
            lse[r:r + n, heads] = torch.logsumexp(s, -1)
            out[r:r + n, heads] = torch.einsum("igt,td->igd", torch.softmax(s, -1), v)
        r += n
    return [out, lse]
