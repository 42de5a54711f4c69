"""The quantised cache and the block attention that reads it: cases, plain forms and exact results.

Three operators of a decoding round's target side are measured here:

  append     binding.kv_append: new keys and values, quantised into a paged cache as they are written
  read       binding.kv_read: ranges of cached tokens, read back as rows
  attention  binding.block_attention: the rows of every request's block (1 row = plain decoding) over a prefix that the
             whole batch shares and over the request's own cached tokens

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}
_AMAX_FLOOR = 2.0 ** -100     # the least row maximum a scale is made from


# ---------------------------------------------------------------------------------------------------------- cases ---
def listed():
    return [
        # one new token for each request of a small decoding batch: latency
        dict(name="append decode", op="append", B=32, rows_lo=1, rows_hi=1, ctx_lo=100, ctx_hi=2000,
             Hkv=8, D=128, page=64, dtype="bf16", format="e4m3"),
        # the scheduled block rows (1 to 6 of each request) of a large batch, small heads and pages
        dict(name="append blocks", op="append", B=256, rows_lo=1, rows_hi=6, ctx_lo=0, ctx_hi=500,
             Hkv=4, D=64, page=16, dtype="fp16", format="int8"),
        # prompts of many requests entering the cache at once
        dict(name="append prompts", op="append", B=29, rows_lo=500, rows_hi=8000, ctx_lo=0, ctx_hi=77,
             Hkv=8, D=128, page=64, dtype="bf16", format="e4m3"),
        # a few hundred tokens taken out again for a request that moves
        dict(name="read small", op="read", B=3, rows_lo=100, rows_hi=400, ctx_lo=0, ctx_hi=300,
             Hkv=8, D=128, page=32, dtype="bf16", format="int8"),
        # whole contexts of a batch read back
        dict(name="read contexts", op="read", B=24, rows_lo=1000, rows_hi=9000, ctx_lo=0, ctx_hi=9,
             Hkv=8, D=128, page=64, dtype="bf16", format="e4m3"),
        # a single request, a single token: the smallest step of plain decoding
        dict(name="attention one token", op="attention", B=1, rows_lo=1, rows_hi=1, ctx_lo=777, ctx_hi=777, prefix=0,
             Hq=32, Hkv=8, D=128, page=64, dtype="bf16", format="e4m3", mask="causal"),
        # plain decoding of a batch over contexts of thousands of tokens, nothing shared
        dict(name="attention decode", op="attention", B=64, rows_lo=1, rows_hi=1, ctx_lo=500, ctx_hi=9000, prefix=0,
             Hq=64, Hkv=8, D=128, page=64, dtype="bf16", format="e4m3", mask="causal"),
        # the scheduled blocks of a batch of 256 (up to 5 drafted tokens) over own contexts, with a short system prompt
        dict(name="attention blocks", op="attention", B=256, rows_lo=1, rows_hi=6, ctx_lo=100, ctx_hi=3000, prefix=700,
             Hq=32, Hkv=8, D=128, page=64, dtype="bf16", format="e4m3", mask="causal"),
        # the same blocks over a long shared prompt: the prefix's products dominate
        dict(name="attention shared prompt", op="attention", B=256, rows_lo=4, rows_hi=6, ctx_lo=20, ctx_hi=600,
             prefix=8192, Hq=64, Hkv=8, D=128, page=64, dtype="bf16", format="e4m3", mask="causal"),
        # few requests with long blocks (16 drafted tokens) asking about one very long document
        dict(name="attention long document", op="attention", B=9, rows_lo=17, rows_hi=17, ctx_lo=30, ctx_hi=200,
             prefix=131007, Hq=32, Hkv=4, D=128, page=128, dtype="fp16", format="int8", mask="causal"),
        # drafted trees of up to 40 nodes, small heads, small pages
        dict(name="attention trees", op="attention", B=48, rows_lo=9, rows_hi=40, ctx_lo=50, ctx_hi=1500, prefix=333,
             Hq=24, Hkv=8, D=64, page=16, dtype="fp16", format="e4m3", mask="tree"),
        # a parallel drafter's blocks, in which every position sees every other one
        dict(name="attention drafter", op="attention", B=64, rows_lo=8, rows_hi=16, ctx_lo=0, ctx_hi=4000, prefix=0,
             Hq=16, Hkv=2, D=128, page=64, dtype="bf16", format="int8", mask="full"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm when the range is wide."""
    if hi <= 10 * max(lo, 1):
        n = rng.randint(lo, hi)
    else:
        n = int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))
    return n - 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention"])
    fmt = rng.choice(["e4m3", "e4m3", "int8"])
    dtype = rng.choice(["bf16", "fp16"])
    Hkv, D, page = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 128, 96]), rng.choice([16, 32, 64, 128, 48])
    if op != "attention":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        B = _spread(rng, 1, 256)
        hi = _spread(rng, 1, max(1, min(8000, 120000 // B)))
        lo = max(1, hi // rng.choice([1, 2, 10]))
        return dict(op=op, B=B, rows_lo=lo, rows_hi=hi, ctx_lo=0, ctx_hi=_spread(rng, 1, 500), Hkv=Hkv, D=D, page=page,
                    dtype=dtype, format=fmt)
    mask = rng.choice(["causal", "causal", "full", "tree"])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    B = _spread(rng, 1, 256)
    hi = rng.choice([1, 1, 2, 5, 6, 9, 17, 33])
    lo = max(1, hi - rng.choice([0, 2, 16]))
    ctx_hi = _spread(rng, 16, 9000)
    ctx_lo = ctx_hi // rng.choice([1, 2, 8, 64])
    prefix = rng.choice([0, _spread(rng, 16, 1000), _spread(rng, 1000, 100000)])
    case = dict(op=op, B=B, rows_lo=lo, rows_hi=hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, prefix=prefix, Hq=Hq, Hkv=Hkv, D=D,
                page=page, dtype=dtype, format=fmt, mask=mask)
    while True:     # no more tokens or products than the largest listed cases
        w = work(case)
        if w["flops"] > 3e11 and case["prefix"] > 16:
            case["prefix"] = case["prefix"] // 2 + 1
        elif w["flops"] > 3e11 or w["bytes"] > 6e8:
            case["ctx_hi"] = max(1, case["ctx_hi"] // 2)
            case["ctx_lo"] = min(case["ctx_lo"], case["ctx_hi"])
            case["B"] = max(1, case["B"] * 3 // 4)
        else:
            return case


def _lengths(case):
    """Rows and earlier tokens of every request: fixed by the case alone, so that ``work`` is exact."""
    rng = random.Random("%(B)d %(rows_lo)d %(rows_hi)d %(ctx_lo)d %(ctx_hi)d" % case)
    rows = [rng.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["B"])]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    return rows, ctx


def _tree_parents(case):
    """The drafted trees: node i of a request hangs under an earlier node (node 0 is the committed token)."""
    rng = random.Random("tree %(B)d %(rows_lo)d %(rows_hi)d" % case)
    return [[-1] + [rng.randrange(max(0, i - 4), i) for i in range(1, n)] for n in _lengths(case)[0]]


def _visible_block_tokens(case):
    """Pairs (row, block token) that see each other, over the whole batch."""
    rows = _lengths(case)[0]
    if case["mask"] == "causal":
        return sum(n * (n + 1) // 2 for n in rows)
    if case["mask"] == "full":
        return sum(n * n for n in rows)
    total = 0
    for parents in _tree_parents(case):
        depth = []
        for p in parents:
            depth.append(1 if p < 0 else depth[p] + 1)
        total += sum(depth)
    return total


def work(case):
    rows, ctx = _lengths(case)
    R, Hkv, D = sum(rows), case["Hkv"], case["D"]
    size = _DTYPES[case["dtype"]].itemsize
    if case["op"] in ("append", "read"):
        return {"bytes": R * Hkv * (2 * D * size + 2 * D + 8), "flops": 2 * R * Hkv * D}
    Hq = case["Hq"]
    tokens = case["prefix"] + sum(ctx) + R
    pairs = R * case["prefix"] + sum(n * c for n, c in zip(rows, ctx)) + _visible_block_tokens(case)
    return {"bytes": tokens * Hkv * (2 * D + 8) + R * Hq * (2 * D * size + 4), "flops": 4 * D * Hq * pairs}


# --------------------------------------------------------------------------------------------------------- inputs ---
def _quantise(x, fmt):
    """Codes and scales of the rows of x, in 32 bits: the format's definition."""
    dt, top = _FORMATS[fmt]
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    good = torch.isfinite(amax)
    amax = torch.where(good, amax, torch.ones_like(amax)).clamp_min(_AMAX_FLOOR)
    q = torch.full_like(amax, top)      # a tensor: dividing by or into a plain number may go through its reciprocal
    y = torch.where(good, x * (q / amax), torch.zeros_like(x)).clamp(-top, top)
    codes = y.to(dt) if fmt == "e4m3" else torch.round(y).to(dt)
    scale = torch.where(good, amax / q, torch.full_like(amax, float("nan")))
    return codes, scale.squeeze(-1)


def _tables(case, gen, device):
    """Shuffled pages: [B, max_pages] of each request and [prefix pages] of the shared prefix."""
    rows, ctx = _lengths(case)
    page = case["page"]
    need = [-(-(c + n) // page) for c, n in zip(ctx, rows)]
    shared = -(-case.get("prefix", 0) // page)
    n_pages = sum(need) + shared + 3
    order = torch.randperm(n_pages, generator=gen, device=device).to(torch.int32)
    width = max(need)
    slot = torch.arange(width, device=device)[None, :]
    first = torch.tensor([0] + need, device=device).cumsum(0)[:-1, None]
    held = slot < torch.tensor(need, device=device)[:, None]
    table = torch.where(held, order[torch.where(held, first + slot, 0)], 0).to(torch.int32)
    return n_pages, table.contiguous(), order[sum(need):sum(need) + shared].contiguous()


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rows, ctx = _lengths(case)
    B, R, Hkv, D, page, fmt = case["B"], sum(rows), case["Hkv"], case["D"], case["page"], case["format"]
    dt = _DTYPES[case["dtype"]]
    n_pages, table, shared = _tables(case, gen, dev)
    st = dict(case=case, table=table, prefix_pages=shared,
              row0=torch.tensor([0] + rows, device=dev, dtype=torch.int64).cumsum(0),
              ctx=torch.tensor(ctx, device=dev, dtype=torch.int32))
    shape = (n_pages, Hkv, page, D)

    def channels():     # keys and values have a few channels much larger than the others
        return torch.exp(0.5 * torch.randn((Hkv, 1, D), generator=gen, device=dev))

    if case["op"] == "append":
        st["codes"] = [torch.zeros(shape, dtype=torch.uint8, device=dev).view(_FORMATS[fmt][0]) for _ in range(2)]
        st["scales"] = [torch.zeros(shape[:3], device=dev) for _ in range(2)]
        st["k"], st["v"] = [(torch.randn((R, Hkv, D), generator=gen, device=dev) * channels()[:, 0]).to(dt)
                            for _ in range(2)]
        return st
    st["codes"], st["scales"] = [], []
    for _ in range(2):
        codes = torch.empty(shape, dtype=torch.uint8, device=dev).view(_FORMATS[fmt][0])
        scales = torch.empty(shape[:3], device=dev)
        ch = channels()
        step = max(1, (1 << 27) // (Hkv * page * D))
        for i in range(0, n_pages, step):
            n = min(step, n_pages - i)
            x = torch.randn((n, Hkv, page, D), generator=gen, device=dev) * ch
            c, scales[i:i + n] = _quantise(x, fmt)
            codes.view(torch.uint8)[i:i + n] = c.view(torch.uint8)
        st["codes"].append(codes)
        st["scales"].append(scales)
    if case["op"] == "read":
        return st
    st["q"] = (1.2 * torch.randn((R, case["Hq"], D), generator=gen, device=dev)).to(dt)
    st["kv_len"] = torch.tensor([c + n for c, n in zip(ctx, rows)], device=dev, dtype=torch.int32)
    st["scale"] = D ** -0.5
    st["words"] = None
    if case["mask"] == "tree":
        words = []
        for parents in _tree_parents(case):
            seen = []
            for i, p in enumerate(parents):
                seen.append((1 << i) | (seen[p] if p >= 0 else 0))
            words += seen
        st["words"] = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], device=dev, dtype=torch.int64)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["rows_host"], st["ctx_host"] = _lengths(case)
    if own:     # what a program keeps between calls: the cache's handle
        from speculative_decoding_draft_head_gb300 import binding
        st["cache"] = binding.KVCache(st["codes"][0], st["codes"][1], st["scales"][0], st["scales"][1])
    return st


# ------------------------------------------------------------------------------------------------------------ run ---
def run(st):
    case = st["case"]
    if own:
        from speculative_decoding_draft_head_gb300 import binding
        if case["op"] == "append":
            binding.kv_append(st["k"], st["v"], st["cache"], st["table"], st["ctx"], st["row0"])
            return st["codes"] + st["scales"]
        if case["op"] == "read":
            got = binding.kv_read(st["cache"], st["table"], st["ctx"], st["row0"], sum(st["rows_host"]),
                                  dtype=_DTYPES[case["dtype"]])
            return [got["k"], got["v"]]
        got = binding.block_attention(st["q"], st["cache"], st["table"], st["kv_len"], st["row0"],
                                      prefix_pages=st["prefix_pages"], prefix_len=case["prefix"],
                                      mask="causal" if case["mask"] == "causal" else "full", row_mask=st["words"],
                                      scale=st["scale"])
        return [got["out"], got["lse"]]
    return {"append": _plain_append, "read": _plain_read, "attention": _plain_attention}[case["op"]](st)


def _places(st, n_rows):
    """Page and offset of every packed row's token."""
    page = st["case"]["page"]
    row = torch.arange(n_rows, device=st["row0"].device)
    b = torch.searchsorted(st["row0"], row, right=True) - 1
    pos = st["ctx"].long()[b] + row - st["row0"][b]
    return st["table"].long()[b, pos // page], pos % page


def _plain_append(st):
    pg, off = _places(st, st["k"].shape[0])
    for x, codes, scales in zip((st["k"], st["v"]), st["codes"], st["scales"]):
        c, s = _quantise(x, st["case"]["format"])
        codes.view(torch.uint8)[pg, :, off] = c.view(torch.uint8)
        scales[pg, :, off] = s
    return st["codes"] + st["scales"]


def _plain_read(st):
    pg, off = _places(st, sum(st["rows_host"]))
    out = []
    for codes, scales in zip(st["codes"], st["scales"]):
        c = codes.view(torch.uint8)[pg, :, off].view(codes.dtype).float()
        out.append((c * scales[pg, :, off][..., None]).to(_DTYPES[st["case"]["dtype"]]))
    return out


def _gather(st, pages, n):
    """Keys and values [Hkv, n, D] in 32 bits of the first n tokens of the given pages."""
    got = []
    for codes, scales in zip(st["codes"], st["scales"]):
        c = codes.view(torch.uint8)[pages].view(codes.dtype).float() * scales[pages][..., None]
        got.append(c.transpose(0, 1).flatten(1, 2)[:, :n])
    return got


def _gather_head(st, pages, n, h):
    """The same for one head: [n, D] each."""
    got = []
    for codes, scales in zip(st["codes"], st["scales"]):
        c = codes.view(torch.uint8)[pages, h].view(codes.dtype).float() * scales[pages, h][..., None]
        got.append(c.flatten(0, 1)[:n])
    return got


def _part(s, v):
    """Maximum, sum and weighted values of one part's scores."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return m, p.sum(-1, keepdim=True), p @ v


def _plain_attention(st):
    case = st["case"]
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    group, R, dev = Hq // Hkv, st["q"].shape[0], st["q"].device
    q = st["q"].float().view(R, Hkv, group, D).transpose(0, 1).reshape(Hkv, R * group, D) * st["scale"]
    m0 = torch.full((Hkv, R * group, 1), float("-inf"), device=dev)
    l0 = torch.zeros_like(m0)
    o0 = torch.zeros_like(q)
    if case["prefix"]:
        step = max(1, (1 << 29) // max(1, case["prefix"]))     # rows whose scores fill 2 GB
        for h in range(Hkv):                                    # the prefix once for all requests
            k, v = _gather_head(st, st["prefix_pages"].long(), case["prefix"], h)
            for i in range(0, R * group, step):
                m0[h, i:i + step], l0[h, i:i + step], o0[h, i:i + step] = _part(q[h, i:i + step] @ k.T, v)
    out = torch.empty_like(q)
    lse = torch.empty_like(m0)
    r = 0
    for b, (n, ctx) in enumerate(zip(st["rows_host"], st["ctx_host"])):
        T = ctx + n
        k, v = _gather(st, st["table"][b, : -(-T // page)].long(), T)
        rows = slice(r * group, (r + n) * group)
        s = q[:, rows] @ k.transpose(1, 2)
        i = torch.arange(n, device=dev)
        if case["mask"] == "tree":
            see = (st["words"][r:r + n, None] >> i[None, :]) & 1 == 1
        else:
            see = i[None, :] <= i[:, None] if case["mask"] == "causal" else torch.ones((n, n), dtype=torch.bool, device=dev)
        see = see.repeat_interleave(group, 0)
        s[:, :, ctx:] = s[:, :, ctx:].masked_fill(~see, float("-inf"))
        m1, l1, o1 = _part(s, v)
        m = torch.maximum(m0[:, rows], m1)
        base = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        a0, a1 = torch.exp(m0[:, rows] - base), torch.exp(m1 - base)
        total = a0 * l0[:, rows] + a1 * l1
        out[:, rows] = (a0 * o0[:, rows] + a1 * o1) / torch.where(total > 0, total, torch.ones_like(total))
        lse[:, rows] = m + torch.log(total)
        r += n
    out = out.view(Hkv, R, group, D).transpose(0, 1).reshape(R, Hq, D).to(st["q"].dtype)
    return [out, lse.view(Hkv, R, group).transpose(0, 1).reshape(R, Hq).contiguous()]


# ---------------------------------------------------------------------------------------------------------- exact ---
def exact(case, seed):
    """The operators' definitions in 64 bits.  Codes of 8 bits: e4m3 gives the value before it is rounded to a code;
    int8 codes are whole numbers that the rounding of the 32-bit product decides, so they have no such value."""
    st = _inputs(case, seed)
    rows, ctx = _lengths(case)
    page = case["page"]
    top = _FORMATS[case["format"]][1]
    if case["op"] == "append":
        out = []
        for x, codes in zip((st["k"], st["v"]), st["codes"]):
            x = x.double()
            amax = x.abs().amax(-1).clamp_min(_AMAX_FLOOR)
            c = torch.zeros(codes.shape, dtype=torch.float64, device=x.device)
            s = torch.zeros(codes.shape[:3], dtype=torch.float64, device=x.device)
            r = 0
            for b, (n, c0) in enumerate(zip(rows, ctx)):
                pos = torch.arange(c0, c0 + n, device=x.device)
                pg, off = st["table"][b].long()[pos // page], pos % page
                c[pg, :, off] = x[r:r + n] * (top / amax[r:r + n])[..., None]
                s[pg, :, off] = amax[r:r + n] / top
                r += n
            out.append((c if case["format"] == "e4m3" else None, s))
        return [out[0][0], out[1][0], out[0][1], out[1][1]]

    def tokens(which, pages, n, h):
        c = st["codes"][which].view(torch.uint8)[pages, h].view(st["codes"][which].dtype).double()
        return (c * st["scales"][which][pages, h].double()[..., None]).reshape(-1, case["D"])[:n]

    if case["op"] == "read":
        R = sum(rows)
        out = [torch.empty((R, case["Hkv"], case["D"]), dtype=torch.float64, device="cuda") for _ in range(2)]
        for which in range(2):
            r = 0
            for b, (n, c0) in enumerate(zip(rows, ctx)):
                pages = st["table"][b, : -(-(c0 + n) // page)].long()
                for h in range(case["Hkv"]):
                    out[which][r:r + n, h] = tokens(which, pages, c0 + n, h)[c0:]
                r += n
        return out
    R, Hq, D = st["q"].shape
    group = Hq // case["Hkv"]
    out = torch.zeros((R, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((R, Hq), dtype=torch.float64, device="cuda")
    for h in range(case["Hkv"]):
        kp, vp = [tokens(w, st["prefix_pages"].long(), case["prefix"], h) for w in range(2)]
        heads = slice(h * group, (h + 1) * group)
        r = 0
        for b, (n, c0) in enumerate(zip(rows, ctx)):
            pages = st["table"][b, : -(-(c0 + n) // page)].long()
            k = torch.cat([kp, tokens(0, pages, c0 + n, h)])
            v = torch.cat([vp, tokens(1, pages, c0 + n, h)])
            s = torch.einsum("igd,td->igt", st["q"][r:r + n, heads].double(), k) * st["scale"]
            sees = torch.ones((n, n), dtype=torch.bool, device="cuda")
            if case["mask"] == "causal":
                sees = sees.tril()
            elif case["mask"] == "tree":
                for t in range(n):
                    sees[:, t] = (st["words"][r:r + n] >> t) % 2 == 1
            s[:, :, case["prefix"] + c0:] += torch.where(sees, 0.0, float("-inf"))[:, None, :].double()
            lse[r:r + n, heads] = torch.logsumexp(s, -1)
            out[r:r + n, heads] = torch.einsum("igt,td->igd", torch.softmax(s, -1), v)
            r += n
    return [out, lse]
