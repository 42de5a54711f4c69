"""dspark_window_attention against its formula in 64 bits: every element of out
and lse has to be inside the bound that plain_window.attention gives it."""
import math

import pytest
import torch

import plain_cache
import plain_window
from speculative_decoding_draft_head_gb300 import binding

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16, F16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16, torch.float16


def _check(got, want, allow_nan=False):
    out, lse, tol_out, tol_lse = want
    g, l = got["out"].double().cpu(), got["lse"].double().cpu()
    assert torch.equal(g.isnan(), out.isnan()) and torch.equal(l.isnan(), lse.isnan())
    assert allow_nan or not bool(out.isnan().any())
    err = torch.where(out.isnan(), torch.zeros_like(out), (g - out).abs())
    i = int((err / tol_out).nan_to_num(0).argmax())
    assert not bool((err > tol_out).any()), "out: %d of %d outside, worst %g against %g" % (
        int((err > tol_out).sum()), err.numel(), err.view(-1)[i], tol_out.view(-1)[i])
    empty = lse == -math.inf
    assert torch.equal(l == -math.inf, empty)
    err = torch.where(empty | lse.isnan(), torch.zeros_like(lse), (l - lse).abs())
    assert bool((err <= tol_lse).all()), "lse: worst %g" % float(err.max())


def _run(rows, ctx, prefix, Hq, Hkv, D, page, window, sinks, fmt=E4M3, dtype=BF16, mask="causal", words=None, scale=None,
         q_size=1.0, seed=0, pool_kw=None, evict=True, check=True, **kw):
    gen = torch.Generator().manual_seed(seed)
    lens = [c + n for c, n in zip(ctx, rows)]
    pool = plain_cache.Pool(gen, lens, prefix, Hkv, D, page, fmt, **(pool_kw or {}))
    q = (torch.randn((sum(rows), Hq, D), generator=gen) * q_size).to(dtype)
    row0 = torch.tensor([0] + list(rows)).cumsum(0)
    table, shared = pool.table.clone(), pool.prefix_pages.clone()
    if evict:       # pages that nobody sees are no pages any more
        reach = torch.zeros(prefix, dtype=torch.bool)
        for b, n in enumerate(rows):
            C = prefix + ctx[b]
            see = plain_window.sees(n, C, window, sinks, mask, None if words is None else words[row0[b]:row0[b + 1]])
            any_see = see.any(0) if n else torch.zeros(C, dtype=torch.bool)
            any_see[C:] = True      # the block's own tokens have just been written
            reach |= any_see[:prefix]
            for slot in range(table.shape[1]):
                if not any_see[prefix + slot * page:prefix + (slot + 1) * page].any():
                    table[b, slot] = -5
        for slot in range(len(shared)):
            if not reach[slot * page:(slot + 1) * page].any():
                shared[slot] = 1 << 30
    cache = pool.cache(binding)
    got = binding.window_attention(
        q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), row0.cuda(), window=window, sinks=sinks,
        prefix_pages=shared.cuda() if prefix else None, prefix_len=prefix, mask=mask,
        row_mask=None if words is None else words.cuda(), scale=scale, **kw)
    torch.cuda.synchronize()
    assert binding.read_device_flags(cache.flags) == 0
    if check:
        _check(got, plain_window.attention(q, pool, row0, lens, window, sinks, mask, words, scale))
    return got, q, pool, row0, lens


# rows, ctx, prefix, Hq, Hkv, D, page, window, sinks
SHAPES = {
    "one token, nothing before": ([1], [0], 0, 1, 1, 16, 16, 1, 0),
    "one token sees itself": ([1], [700], 0, 8, 2, 128, 64, 1, 0),
    "one token": ([1], [777], 0, 8, 2, 128, 64, 200, 4),
    "window of the whole context": ([1, 3], [777, 20], 60, 8, 2, 128, 64, 10 ** 6, 4),
    "lengths around the window": ([1] * 9, [126, 127, 128, 0, 254, 255, 256, 129, 500], 0, 8, 2, 64, 32, 128, 3),
    "sinks past the window": ([2, 1], [100, 40], 0, 4, 2, 64, 16, 20, 90),
    "sinks past everything": ([2, 4], [100, 0], 30, 4, 2, 64, 16, 3, 10 ** 9),
    "verify blocks": ([6, 1, 4, 2], [100, 30, 513, 0], 0, 8, 2, 128, 64, 77, 16),
    "requests without rows": ([0, 3, 0, 0, 2, 0], [9, 200, 0, 50, 129, 4], 100, 4, 2, 64, 16, 50, 5),
    "prefix of one token": ([2, 3], [4, 0], 1, 8, 8, 128, 16, 3, 1),
    "window into the prefix": ([5, 6, 1], [40, 3, 300], 515, 8, 1, 128, 128, 129, 33),
    "sinks past the prefix": ([5, 2], [400, 31], 21, 8, 2, 128, 32, 65, 50),
    "odd head and page sizes": ([4, 3], [61, 7], 95, 6, 3, 80, 48, 31, 2),
    "head of 48, group of 5": ([3, 1], [130, 500], 33, 10, 2, 48, 16, 100, 1),
    "head of 96": ([7, 2], [140, 20], 250, 4, 4, 96, 64, 64, 4),
    "block longer than the window": ([40, 33], [90, 10], 70, 16, 1, 64, 32, 9, 4),
    "blocks of many row blocks": ([40, 3, 1], [300, 128, 0], 260, 24, 2, 128, 64, 150, 4),
    "many query heads on one": ([2, 1], [60, 600], 0, 128, 1, 128, 64, 256, 4),
    "long context": ([3, 1], [9000, 20], 0, 4, 1, 128, 64, 4096, 4),
    "long context, window as long": ([1], [20011], 0, 4, 1, 64, 64, 19999, 4),
    "long prefix": ([2, 5], [3, 70], 20011, 4, 1, 64, 64, 900, 133),
    "prompt": ([700], [10], 5, 4, 2, 128, 16, 200, 4),
    "prompts": ([700, 1, 90, 260], [10, 500, 300, 0], 205, 8, 2, 128, 64, 150, 30),
    "prompts longer than the window": ([1300, 900], [700, 2000], 0, 6, 2, 64, 48, 129, 1),
    "prompt of wide heads, no first tokens": ([300, 280], [1000, 140], 90, 64, 1, 96, 16, 333, 0),
    "many short requests": ([1, 2, 3] * 60, [5, 40, 130] * 60, 20, 4, 2, 64, 16, 33, 4),
}


@pytest.mark.parametrize("fmt,dtype", [(E4M3, BF16), (INT8, F16), (E4M3, F16), (INT8, BF16)])
@pytest.mark.parametrize("name", SHAPES)
def test_shapes(name, fmt, dtype):
    _run(*SHAPES[name], fmt=fmt, dtype=dtype)


@pytest.mark.parametrize("name", ["verify blocks", "window into the prefix", "block longer than the window",
                                  "blocks of many row blocks", "sinks past everything", "prompt", "prompts"])
def test_full_block(name):
    _run(*SHAPES[name], mask="full")


@pytest.mark.parametrize("ctx,prefix,window,sinks", [(0, 0, 64, 0), (5, 0, 64, 9), (0, 40, 70, 4), (200, 130, 100, 150),
                                                     (300, 0, 64, 0), (90, 20, 1000, 0)])
@pytest.mark.parametrize("n", [1, 9, 40, 64])
def test_tree_masks_and_rows_that_see_nothing(n, ctx, prefix, window, sinks):
    """Random words, one of them empty and one full: with nothing before the block the empty one's row has no token."""
    gen = torch.Generator().manual_seed(n)
    words = torch.randint(-2 ** 63, 2 ** 63 - 1, (2 * n,), generator=gen)
    words[0], words[2 * n - 1] = 0, -1
    got, *_ = _run([n, n], [ctx, ctx], prefix, 4, 2, 64, 16, window, sinks, mask="full", words=words)
    if ctx == 0 and prefix == 0:
        assert bool((got["out"][0] == 0).all()) and bool((got["lse"][0] == -math.inf).all())


@pytest.mark.parametrize("ctx,prefix,window,sinks", [(0, 0, 64, 0), (5, 20, 64, 9), (700, 130, 100, 150), (300, 0, 64, 0),
                                                     (90, 300, 200, 40)])
def test_trees_of_many_query_heads(ctx, prefix, window, sinks):
    gen = torch.Generator().manual_seed(ctx)
    n = 50
    words = torch.randint(-2 ** 63, 2 ** 63 - 1, (2 * n + 9,), generator=gen)
    words[0], words[2 * n - 1] = 0, -1
    _run([n, 9, n], [ctx, 3, ctx + 77], prefix, 20, 2, 64, 16, window, sinks, mask="full", words=words)


@pytest.mark.parametrize("mask,tree", [("causal", False), ("full", False), ("full", True)])
def test_a_window_of_everything_is_the_block_attention(mask, tree):
    gen = torch.Generator().manual_seed(9)
    rows, ctx = [6, 1, 9], [300, 50, 7]
    words = torch.randint(2 ** 62, (16,), generator=gen) if tree else None
    got, q, pool, row0, lens = _run(rows, ctx, 130, 8, 2, 128, 32, 10 ** 9, 0, mask=mask, words=words, check=False)
    _check(got, plain_cache.attention(q, pool, row0, lens, mask, words))


@pytest.mark.parametrize("q_size,kw", [
    (30.0, {}),                                            # sharp: one token takes nearly all
    (1e-3, {}),                                            # flat
    (1e30, dict(k_scale=1e-30)),                           # far from fp16's range, in both directions
    (1e-30, dict(k_scale=1e30)),
    (1.0, dict(v_scale=1e-30)),
    (1.0, dict(v_scale=1e25)),
    (1.0, dict(token_scale=lambda gen, s: 2.0 ** torch.randint(-14, 3, s, generator=gen).float())),
    (4.0, dict(token_scale=lambda gen, s: 2.0 ** torch.randint(-3, 3, s, generator=gen).float())),
], ids=["sharp", "flat", "large q", "small q", "small v", "large v", "uneven tokens", "uneven and sharp"])
@pytest.mark.parametrize("rows", [[6, 1], [1, 1], [70, 3]])
def test_ranges(q_size, kw, rows):
    _run(rows, [700, 300], 400, 8, 2, 128, 64, 500, 6, q_size=q_size, pool_kw=kw)


def test_zero_queries_weigh_every_token_alike():
    got, *_ = _run([2], [100], 0, 4, 2, 64, 16, 30, 4, q_size=0.0)
    # 30 of the window and the 4 first ones
    assert ((got["lse"].cpu() - math.log(34)).abs() < 1e-5).all()


def _place(pool, pages, t):
    return int(pages[t // pool.page]), t % pool.page


def test_tokens_stored_as_no_number_reach_only_rows_that_see_them():
    gen = torch.Generator().manual_seed(4)
    rows, ctx, window, sinks = [5, 3], [200, 90], 40, 4
    lens = [c + n for c, n in zip(ctx, rows)]
    pool = plain_cache.Pool(gen, lens, 0, 2, 64, 16, E4M3)
    q = torch.randn((8, 4, 64), generator=gen).to(BF16)
    # row i of request 0 sees tokens 161 + i .. 200 + i: token 162 is for rows 0 and 1, 150 for none; of request 1 a sink
    for b, t, scales in ((0, 162, pool.k_scale), (0, 150, pool.v_scale), (1, 2, pool.v_scale)):
        pg, off = _place(pool, pool.table[b], t)
        scales[pg, 1, off] = math.nan
    row0 = torch.tensor([0, 5, 8])
    got = binding.window_attention(q.cuda(), pool.cache(binding), pool.table.cuda(), torch.tensor(lens).int().cuda(),
                                   row0.cuda(), window=window, sinks=sinks)
    want = plain_window.attention(q, pool, row0, lens, window, sinks)
    assert want[0][:2, 2:].isnan().all() and not want[0][2:5].isnan().any() and want[0][5:, 2:].isnan().all()
    assert not want[0][:, :2].isnan().any()
    _check(got, want, allow_nan=True)


def test_queries_that_are_no_numbers():
    gen = torch.Generator().manual_seed(6)
    pool = plain_cache.Pool(gen, [90], 0, 2, 64, 16, INT8)
    q = torch.randn((6, 4, 64), generator=gen).to(F16)
    args = (pool.cache(binding), pool.table.cuda(), torch.tensor([90]).int().cuda(), torch.tensor([0, 6]).cuda())
    clean = binding.window_attention(q.cuda(), *args, window=20)
    q[2, 1, 5], q[4, 3, 0] = math.nan, math.inf
    got = binding.window_attention(q.cuda(), *args, window=20)
    bad = torch.zeros((6, 4), dtype=torch.bool)
    bad[2, 1] = bad[4, 3] = True
    assert got["out"].cpu()[bad].isnan().all() and torch.equal(got["out"].cpu()[~bad], clean["out"].cpu()[~bad])


def test_bad_lengths_and_pages():
    gen = torch.Generator().manual_seed(7)
    lens = [60, 50, 40, 33]
    pool = plain_cache.Pool(gen, lens, 20, 2, 64, 16, E4M3)
    rows = [2, 3, 1, 2]
    row0 = torch.tensor([0] + rows).cumsum(0)
    q = torch.randn((8, 4, 64), generator=gen).to(BF16)
    kv_len = torch.tensor(lens).int()
    kv_len[1] = 2                                     # shorter than its block
    kv_len[2] = pool.table.shape[1] * 16 + 1          # beyond its pages
    table = pool.table.clone()
    table[0, 2] = pool.k.shape[0]                     # own tokens 32 .. 47
    cache = pool.cache(binding)
    # request 0's rows are own tokens 58 and 59: a window of 11 ends at 48
    got = binding.window_attention(q.cuda(), cache, table.cuda(), kv_len.cuda(), row0.cuda(), window=11, sinks=22,
                                   prefix_pages=pool.prefix_pages.cuda(), prefix_len=20)
    torch.cuda.synchronize()
    assert binding.read_device_flags(cache.flags) == binding.FLAG_BAD_LENGTH
    want = plain_window.attention(q, pool, row0, lens, 11, 22)
    for part in (slice(0, 2), slice(6, 8)):
        _check({k: t[part] for k, t in got.items()}, [t[part] for t in want])
    assert got["out"][2:6].isnan().all() and got["lse"][2:6].isnan().all()
    # a window that reaches the bad page from its first row only
    got = binding.window_attention(q.cuda(), cache, table.cuda(), kv_len.cuda(), row0.cuda(), window=12, sinks=22,
                                   prefix_pages=pool.prefix_pages.cuda(), prefix_len=20)
    assert binding.read_device_flags(cache.flags) == binding.FLAG_BAD_LENGTH | binding.FLAG_BAD_PAGE
    assert got["out"][0].isnan().all() and not got["out"][1].isnan().any()


def test_rows_of_no_request_and_strided_queries():
    gen = torch.Generator().manual_seed(1)
    pool = plain_cache.Pool(gen, [20, 30], 40, 2, 64, 16, E4M3)
    wide = torch.full((9, 7, 64), math.nan, dtype=BF16)
    wide[:5, 2:6] = torch.randn((5, 4, 64), generator=gen).to(BF16)
    out = dict(out=torch.full((9, 4, 64), 7.0, dtype=BF16, device="cuda"), lse=torch.full((9, 4), 7.0, device="cuda"))
    row0 = torch.tensor([0, 2, 5])
    binding.window_attention(wide.cuda()[:, 2:6], pool.cache(binding), pool.table.cuda(), torch.tensor([20, 30]).int().cuda(),
                             row0.cuda(), window=25, sinks=3, prefix_pages=pool.prefix_pages.cuda(), prefix_len=40, out=out)
    assert bool((out["out"][5:] == 7).all()) and bool((out["lse"][5:] == 7).all())
    _check({k: t[:5] for k, t in out.items()}, plain_window.attention(wide[:5, 2:6], pool, row0, [20, 30], 25, 3))


@pytest.mark.parametrize("rows", [[3, 1, 6], [130, 70, 90]])
def test_the_same_call_gives_the_same_bits_on_a_stream_and_replayed(rows):
    shape = (rows, [700, 20, 90], 50, 8, 2, 128, 64, 300, 4)
    got, q, pool, row0, lens = _run(*shape)
    cache, args = pool.cache(binding), (pool.table.cuda(), torch.tensor(lens).int().cuda(), row0.cuda())
    kw = dict(window=300, sinks=4, prefix_pages=pool.prefix_pages.cuda(), prefix_len=50)
    qd = q.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = binding.window_attention(qd, cache, *args, stream=side, **kw)
    side.synchronize()
    assert torch.equal(other["out"], got["out"]) and torch.equal(other["lse"], got["lse"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = binding.window_attention(qd, cache, *args, **kw)
    kept["out"].zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept["out"], got["out"]) and torch.equal(kept["lse"], got["lse"])


def test_pages_beyond_32_bits_of_codes():
    """A cache of 2.1e9 codes and more: the last page's rows lie behind 2^31 bytes."""
    gen = torch.Generator().manual_seed(2)
    pool = plain_cache.Pool(gen, [40], 0, 2, 128, 64, INT8, spare=0)
    n_pages = (1 << 31) // (2 * 64 * 128) + 5
    cache = binding.KVCache.empty(n_pages, 2, 64, 128, dtype=INT8)
    last = n_pages - 1
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(cache, name)[last] = getattr(pool, name)[int(pool.table[0, 0])].cuda()
    q = torch.randn((2, 4, 128), generator=gen).to(BF16)
    got = binding.window_attention(q.cuda(), cache, torch.tensor([[last]], dtype=torch.int32).cuda(),
                                   torch.tensor([40]).int().cuda(), torch.tensor([0, 2]).cuda(), window=30, sinks=1)
    _check(got, plain_window.attention(q, pool, torch.tensor([0, 2]), [40], 30, 1))


@pytest.mark.parametrize("B", [70, 1100])
def test_a_long_block_among_many_short_ones(B):
    """Requests without rows, of one row and one of 90: every row is some block's, whatever the average."""
    rows = [(b % 3) for b in range(B)]
    rows[B // 2] = 90
    _run(rows, [(37 * b) % 200 for b in range(B)], 20, 4, 2, 64, 16, 33, 4)


def test_as_many_rows_as_requests_but_not_one_each():
    _run([0, 5, 0, 0, 0, 2, 0], [9, 200, 3, 50, 0, 129, 4], 30, 8, 2, 64, 16, 50, 5)


def test_row_starts_that_are_no_good():
    """Flagged; the requests between good ones keep their results."""
    gen = torch.Generator().manual_seed(8)
    lens = [30, 40, 50]
    pool = plain_cache.Pool(gen, lens, 0, 2, 64, 16, E4M3)
    q = torch.randn((9, 4, 64), generator=gen).to(BF16)
    row0 = torch.tensor([0, 4, 2, 6])       # request 1 ends before it begins
    cache = pool.cache(binding)
    out = dict(out=torch.full((9, 4, 64), 7.0, dtype=BF16, device="cuda"))
    binding.window_attention(q.cuda(), cache, pool.table.cuda(), torch.tensor(lens).int().cuda(), row0.cuda(), window=20, out=out)
    torch.cuda.synchronize()
    assert binding.read_device_flags(cache.flags) == binding.FLAG_BAD_LENGTH
    assert bool((out["out"][6:] == 7).all())
    for bad in (torch.tensor([-3, 2, 4, 6]), torch.tensor([0, 2, 4, 1 << 40])):
        cache.flags.zero_()
        binding.window_attention(q.cuda(), cache, pool.table.cuda(), torch.tensor(lens).int().cuda(), bad.cuda(), window=20, out=out)
        torch.cuda.synchronize()
        assert binding.read_device_flags(cache.flags) == binding.FLAG_BAD_LENGTH


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("rows,ctx,prefix,Hq,Hkv,D,page,window,sinks", [
    ([1], [9000], 0, 4, 1, 96, 48, 8000, 40),
    ([1, 1], [5000, 3], 700, 8, 2, 80, 16, 5200, 4),
    ([2], [4000], 0, 8, 1, 128, 64, 3900, 1),          # 16 rows of a kv head
    ([3], [4000], 900, 8, 1, 128, 64, 4500, 1000),     # 24
    ([5, 0], [4000, 7], 0, 20, 2, 64, 32, 3000, 4),    # 50: several row blocks
])
def test_few_rows_over_long_windows(rows, ctx, prefix, Hq, Hkv, D, page, window, sinks, fmt):
    """An item's tokens are split over a cluster's blocks."""
    _run(rows, ctx, prefix, Hq, Hkv, D, page, window, sinks, fmt=fmt)


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("name", ["one token", "lengths around the window", "verify blocks", "window into the prefix",
                                  "head of 96", "blocks of many row blocks"])
def test_fp16_results_have_little_but_their_own_rounding(name, fmt):
    """Of few rows the softmax terms count in two fp16 parts: 2^-22 in the place of 2^-11."""
    got, q, pool, row0, lens = _run(*SHAPES[name], fmt=fmt, dtype=F16, check=False)
    window, sinks = SHAPES[name][-2:]
    _check(got, plain_window.attention(q, pool, row0, lens, window, sinks, terms=2.0 ** -22))
