"""dspark_block_attention against its formula in 64 bits.

The bounds are derived in plain_cache.attention from the roundings that the
definition allows; every element of out and lse has to be inside its own."""
import math

import pytest
import torch

import plain_cache
from speculative_decoding_draft_head_gb300 import binding

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16, F16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16, torch.float16


def _row0(rows):
    return torch.tensor([0] + list(rows)).cumsum(0)


def _check(got, want, what="", allow_nan=False):
    out, lse, tol_out, tol_lse = want
    g, l = got["out"].double().cpu(), got["lse"].double().cpu()
    if allow_nan:
        assert torch.equal(g.isnan(), out.isnan()) and torch.equal(l.isnan(), lse.isnan())
    err = torch.where(out.isnan(), torch.zeros_like(out), (g - out).abs())
    over = err > tol_out
    i = int((err / tol_out).argmax())
    assert not bool(over.any()) and not bool(g[~out.isnan()].isnan().any()), \
        "%s out: %d of %d outside, worst %g against %g" % (what, int(over.sum()), over.numel(), err.view(-1)[i],
                                                           tol_out.view(-1)[i])
    empty = lse == -math.inf
    assert torch.equal(l == -math.inf, empty)
    err = torch.where(empty | lse.isnan(), torch.zeros_like(lse), (l - lse).abs())
    assert bool((err <= tol_lse).all()), "%s lse: worst %g" % (what, float(err.max()))


def _run(rows, ctx, prefix, Hq, Hkv, D, page, fmt=E4M3, dtype=BF16, mask="causal", words=None, scale=None, q_size=1.0,
         seed=0, pool_kw=None, check=True):
    gen = torch.Generator().manual_seed(seed)
    lens = [c + n for c, n in zip(ctx, rows)]
    pool = plain_cache.Pool(gen, lens, prefix, Hkv, D, page, fmt, **(pool_kw or {}))
    q = (torch.randn((sum(rows), Hq, D), generator=gen) * q_size).to(dtype)
    row0 = _row0(rows)
    cache = pool.cache(binding)
    got = binding.block_attention(
        q.cuda(), cache, pool.table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), row0.cuda(),
        prefix_pages=pool.prefix_pages.cuda() if prefix else None, prefix_len=prefix, mask=mask,
        row_mask=None if words is None else words.cuda(), scale=scale)
    torch.cuda.synchronize()
    assert binding.read_device_flags(cache.flags) == 0
    if check:
        _check(got, plain_cache.attention(q, pool, row0, lens, mask, words, scale))
    return got, q, pool, row0, lens


# rows, ctx, prefix, Hq, Hkv, D, page
SHAPES = {
    "one token, nothing before": ([1], [0], 0, 1, 1, 16, 16),
    "one token": ([1], [777], 0, 8, 2, 128, 64),
    "lengths around a tile": ([1] * 7, [126, 127, 128, 0, 254, 255, 256], 0, 8, 2, 64, 32),
    "verify blocks": ([6, 1, 4, 2], [100, 30, 513, 0], 0, 8, 2, 128, 64),
    "requests without rows": ([0, 3, 0, 0, 2, 0], [9, 200, 0, 50, 129, 4], 100, 4, 2, 64, 16),
    "prefix of one token": ([2, 3], [4, 0], 1, 8, 8, 128, 16),
    "prefix and blocks": ([5, 6, 1], [40, 3, 300], 515, 8, 1, 128, 128),
    "odd head and page sizes": ([4, 3], [61, 7], 95, 6, 3, 80, 48),
    "head of 48, group of 5": ([3, 1], [130, 500], 33, 10, 2, 48, 16),
    "head of 96": ([7, 2], [140, 20], 250, 4, 4, 96, 64),
    "more rows than a tile": ([17, 33], [90, 10], 70, 16, 1, 64, 32),
    "more rows than two tiles": ([40, 3], [300, 128], 260, 24, 2, 128, 64),
    "many query heads on one": ([2, 1], [60, 600], 0, 128, 1, 128, 64),
    "long own context": ([3, 1], [9000, 20], 0, 4, 1, 128, 64),
    "long prefix": ([2, 5], [3, 70], 20011, 4, 1, 64, 64),
    "block longer than a tile": ([150], [10], 5, 2, 1, 64, 16),
    "many short requests": ([1, 2, 3] * 60, [5, 40, 130] * 60, 20, 4, 2, 64, 16),
}


@pytest.mark.parametrize("fmt,dtype", [(E4M3, BF16), (INT8, F16), (E4M3, F16), (INT8, BF16)])
@pytest.mark.parametrize("name", SHAPES)
def test_shapes(name, fmt, dtype):
    _run(*SHAPES[name], fmt=fmt, dtype=dtype)


@pytest.mark.parametrize("rows,prefix,Hq,Hkv,D", [
    ([7] * 60, 300, 30, 6, 64),              # groups of 5: rows of one request on both sides of a row tile's end
    ([7] * 60, 0, 30, 6, 64),                # rows that one worker finishes and rows that several share
    ([1, 0, 6, 33] * 13, 140, 21, 3, 128),
    ([1] * 331, 0, 30, 30, 48),              # a row a head: nothing to take together
])
def test_batches_with_several_rows_a_joining_warp(rows, prefix, Hq, Hkv, D):
    _run(rows, [(37 * b) % 300 for b in range(len(rows))], prefix, Hq, Hkv, D, 16)


@pytest.mark.parametrize("name", ["verify blocks", "prefix and blocks", "more rows than two tiles",
                                  "block longer than a tile"])
def test_full_block(name):
    _run(*SHAPES[name], mask="full")


@pytest.mark.parametrize("ctx,prefix", [(0, 0), (5, 0), (0, 40), (200, 130)])
@pytest.mark.parametrize("n", [1, 9, 40, 64])
def test_tree_masks_and_rows_that_see_nothing(n, ctx, prefix):
    """Random words, one of them empty and one full: with neither context nor
    prefix the empty one's row has no token at all."""
    gen = torch.Generator().manual_seed(n)
    words = torch.randint(-2 ** 63, 2 ** 63 - 1, (2 * n,), generator=gen)
    words[0], words[2 * n - 1] = 0, -1
    got, *_ = _run([n, n], [ctx, ctx], prefix, 4, 2, 64, 16, mask="full", words=words)
    if ctx == 0 and prefix == 0:
        assert bool((got["out"][0] == 0).all()) and bool((got["lse"][0] == -math.inf).all())


def test_rows_of_no_request_are_left_alone():
    gen = torch.Generator().manual_seed(1)
    pool = plain_cache.Pool(gen, [20, 30], 40, 2, 64, 16, E4M3)
    q = torch.full((9, 4, 64), math.nan, dtype=BF16)
    q[:5] = torch.randn((5, 4, 64), generator=gen).to(BF16)
    out = dict(out=torch.full((9, 4, 64), 7.0, dtype=BF16, device="cuda"), lse=torch.full((9, 4), 7.0, device="cuda"))
    row0 = _row0([2, 3])
    binding.block_attention(q.cuda(), pool.cache(binding), pool.table.cuda(),
                            torch.tensor([20, 30], dtype=torch.int32).cuda(), row0.cuda(),
                            prefix_pages=pool.prefix_pages.cuda(), prefix_len=40, out=out)
    assert bool((out["out"][5:] == 7).all()) and bool((out["lse"][5:] == 7).all())
    _check({k: t[:5] for k, t in out.items()}, plain_cache.attention(q[:5], pool, row0, [20, 30]))


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
def test_ranges(q_size, kw):
    _run([6, 1], [700, 300], 400, 8, 2, 128, 64, q_size=q_size, pool_kw=kw)


def test_a_growing_maximum_and_a_strong_first_token():
    """Scores that rise along the context (the running maximum moves in every
    tile) and a first token with a large score and tiny values."""
    gen = torch.Generator().manual_seed(2)
    n, D = 3000, 64
    for rising in (True, False):
        pool = plain_cache.Pool(gen, [n + 2], 0, 1, D, 64, E4M3)
        q = torch.ones((2, 2, D)).to(BF16)
        level = torch.arange(n + 2) * 0.02 if rising else torch.zeros(n + 2)
        x = level[:, None, None].expand(-1, 1, D).clone() + 0.01 * torch.randn((n + 2, 1, D), generator=gen)
        if not rising:
            x[0] = 2.0
        v = torch.randn((n + 2, 1, D), generator=gen)
        v[0] *= 2.0 ** -8
        pos = torch.arange(n + 2)
        pg, off = pool.table[0].long()[pos // 64], pos % 64
        for codes, scales, t in ((pool.k, pool.k_scale, x), (pool.v, pool.v_scale, v)):
            c, s = plain_cache.quantise(t, E4M3)
            codes.view(torch.uint8)[pg, :, off] = c.view(torch.uint8)
            scales[pg, :, off] = s
        got = binding.block_attention(q.cuda(), pool.cache(binding), pool.table.cuda(),
                                      torch.tensor([n + 2], dtype=torch.int32).cuda(), _row0([2]).cuda())
        _check(got, plain_cache.attention(q, pool, _row0([2]), [n + 2]), "rising" if rising else "first token")


def test_nan_tokens_reach_only_the_rows_that_see_them():
    """Appended NaN rows (code 0, scale NaN): one in the block, seen by the later
    rows only, and one in request 1's context, seen by all its rows."""
    gen = torch.Generator().manual_seed(4)
    rows, ctx, page = [4, 3], [70, 20], 32
    lens = [c + n for c, n in zip(ctx, rows)]
    pool = plain_cache.Pool(gen, lens, 50, 2, 64, page, E4M3)
    for b, t in ((0, ctx[0] + 2), (1, 5)):
        pg, off = int(pool.table[b, t // page]), t % page
        for codes, scales in ((pool.k, pool.k_scale), (pool.v, pool.v_scale)):
            codes.view(torch.uint8)[pg, :, off] = 0
            scales[pg, :, off] = math.nan
    q = torch.randn((7, 4, 64), generator=gen).to(BF16)
    q[3, 1, 7] = math.inf           # and a row of q of its own
    row0 = _row0(rows)
    got = binding.block_attention(q.cuda(), pool.cache(binding), pool.table.cuda(),
                                  torch.tensor(lens, dtype=torch.int32).cuda(), row0.cuda(),
                                  prefix_pages=pool.prefix_pages.cuda(), prefix_len=50)
    out = got["out"].cpu()
    assert not bool(out[:2].isnan().any())
    assert bool(out[2:].isnan().all())
    clean = plain_cache.attention(q[:2], pool, _row0([2]), [ctx[0] + 2])
    _check({k: t[:2] for k, t in got.items()}, clean)


def test_an_infinite_query_spoils_its_own_row_only():
    gen = torch.Generator().manual_seed(6)
    pool = plain_cache.Pool(gen, [40], 30, 1, 64, 16, INT8)
    q = torch.randn((3, 2, 64), generator=gen).to(F16)
    q[1, 0, 3], q[2, 1, 5] = math.inf, math.nan
    got = binding.block_attention(q.cuda(), pool.cache(binding), pool.table.cuda(),
                                  torch.tensor([40], dtype=torch.int32).cuda(), _row0([3]).cuda(),
                                  prefix_pages=pool.prefix_pages.cuda(), prefix_len=30)
    bad = torch.zeros((3, 2), dtype=torch.bool)
    bad[1, 0] = bad[2, 1] = True
    nan = got["out"].cpu().isnan()
    assert torch.equal(nan.all(2), bad) and torch.equal(nan.any(2), bad)
    assert torch.equal(got["lse"].cpu().isnan(), bad)


def test_bad_requests_and_pages_are_flagged():
    gen = torch.Generator().manual_seed(7)
    rows, lens = [2, 2, 2, 2, 2], [30, 40, 35, 50, 20]
    pool = plain_cache.Pool(gen, lens, 20, 1, 64, 16, E4M3)
    table = pool.table.clone()
    table[2, 1] = -1                                 # a page of request 2
    given = torch.tensor(lens, dtype=torch.int32)
    given[1] = 1                                     # shorter than its block
    given[3] = table.shape[1] * 16 + 1               # longer than its pages
    q = torch.randn((10, 2, 64), generator=gen).to(BF16)
    cache = pool.cache(binding)
    got = binding.block_attention(q.cuda(), cache, table.cuda(), given.cuda(), _row0(rows).cuda(),
                                  prefix_pages=pool.prefix_pages.cuda(), prefix_len=20)
    assert binding.read_device_flags(cache.flags) == binding.FLAG_BAD_PAGE | binding.FLAG_BAD_LENGTH
    nan = got["out"].cpu().isnan()
    assert bool(nan[2:8].all()) and not bool(nan[:2].any()) and not bool(nan[8:].any())
    want = plain_cache.attention(q, pool, _row0(rows), lens)
    _check({k: t[:2] for k, t in got.items()}, [t[:2] for t in want])
    _check({k: t[8:] for k, t in got.items()}, [t[8:] for t in want])
    # a bad page of the prefix reaches everyone
    pages = pool.prefix_pages.clone()
    pages[0] = cache.n_pages
    got = binding.block_attention(q.cuda(), cache, pool.table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                  _row0(rows).cuda(), prefix_pages=pages.cuda(), prefix_len=20)
    assert bool(got["out"].isnan().all())


def test_bad_row_starts_are_flagged_and_stay_in_bounds():
    gen = torch.Generator().manual_seed(8)
    pool = plain_cache.Pool(gen, [20, 20, 20], 0, 1, 64, 16, E4M3)
    q = torch.randn((6, 2, 64), generator=gen).to(BF16)
    lens = torch.tensor([20, 20, 20], dtype=torch.int32).cuda()
    for starts in ([0, 2, 4, 50], [0, 4, 2, 6], [-5, 2, 4, 6], [9, 9, 9, 9], [0, 2 ** 40, 4, 6]):
        cache = pool.cache(binding)
        binding.block_attention(q.cuda(), cache, pool.table.cuda(), lens, torch.tensor(starts).cuda())
        assert binding.read_device_flags(cache.flags) & binding.FLAG_BAD_LENGTH, starts


def test_a_row_mask_longer_than_its_word_is_flagged():
    gen = torch.Generator().manual_seed(9)
    pool = plain_cache.Pool(gen, [70, 30], 0, 1, 64, 16, E4M3)
    q = torch.randn((68, 2, 64), generator=gen).to(BF16)
    cache = pool.cache(binding)
    got = binding.block_attention(q.cuda(), cache, pool.table.cuda(), torch.tensor([70, 30], dtype=torch.int32).cuda(),
                                  _row0([65, 3]).cuda(), row_mask=torch.full((68,), -1).cuda())
    assert binding.read_device_flags(cache.flags) == binding.FLAG_BAD_LENGTH
    assert bool(got["out"][:65].isnan().all()) and not bool(got["out"][65:].isnan().any())


def test_a_query_slice_of_a_fused_projection_and_no_lse():
    gen = torch.Generator().manual_seed(10)
    pool = plain_cache.Pool(gen, [45, 300], 100, 2, 64, 32, INT8)
    fused = torch.randn((7, 12, 64), generator=gen).to(F16).cuda()
    row0 = _row0([3, 4])
    args = (pool.cache(binding), pool.table.cuda(), torch.tensor([45, 300], dtype=torch.int32).cuda(), row0.cuda())
    kw = dict(prefix_pages=pool.prefix_pages.cuda(), prefix_len=100)
    a = binding.block_attention(fused[:, 2:10], *args, **kw)
    b = binding.block_attention(fused[:, 2:10].contiguous(), *args, **kw)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    out = dict(out=torch.empty_like(a["out"]))
    binding.block_attention(fused[:, 2:10], *args, out=out, **kw)
    assert torch.equal(out["out"], a["out"])
    _check(a, plain_cache.attention(fused[:, 2:10].cpu(), pool, row0, [45, 300]))


def test_repeats_are_bit_equal_and_a_batch_does_not_change_a_request():
    got, q, pool, row0, lens = _run([5, 2, 6], [3000, 10, 130], 1500, 8, 2, 128, 64, check=False)
    args = (pool.cache(binding), pool.table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), row0.cuda())
    for _ in range(3):
        again = binding.block_attention(q.cuda(), *args, prefix_pages=pool.prefix_pages.cuda(), prefix_len=1500)
        assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])


def test_calls_on_two_streams_at_once_keep_apart():
    """Calls without a workspace of their own on two streams, whose parts would meet in a shared one; and a captured
    call, replayed after a larger call has wanted a larger workspace."""
    shapes = [([6] * 50, [700] * 50, 1500, 8, 2, 64, 16), ([5] * 64, [300] * 64, 2100, 8, 2, 64, 16)]
    calls = []
    for i, (rows, ctx, prefix, Hq, Hkv, D, page) in enumerate(shapes):
        want, q, pool, row0, lens = _run(rows, ctx, prefix, Hq, Hkv, D, page, seed=i, check=False)
        kw = dict(q=q.cuda(), cache=pool.cache(binding), block_table=pool.table.cuda(),
                  kv_len=torch.tensor(lens, dtype=torch.int32).cuda(), row0=row0.cuda(),
                  prefix_pages=pool.prefix_pages.cuda(), prefix_len=prefix)
        calls.append((kw, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(8):
        for i, (kw, _) in enumerate(calls):
            with torch.cuda.stream(streams[i]):
                got[i].append(binding.block_attention(**kw))
    torch.cuda.synchronize()
    for i, (_, want) in enumerate(calls):
        for g in got[i]:
            assert torch.equal(g["out"], want["out"]) and torch.equal(g["lse"], want["lse"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        out = binding.block_attention(**calls[0][0])
    _run([2] * 90, [40] * 90, 64, 32, 4, 64, 16, check=False)
    filler = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["out"], calls[0][1]["out"]) and all(int(f[0]) == 255 for f in filler)


def test_a_captured_graph_follows_lengths_and_pages_on_its_own_stream():
    gen = torch.Generator().manual_seed(11)
    rows = [4, 1, 6]
    full = [500, 260, 90]
    pool = plain_cache.Pool(gen, full, 150, 2, 128, 64, E4M3)
    q = torch.randn((11, 8, 128), generator=gen).to(BF16)
    cache, qd, table = pool.cache(binding), q.cuda(), pool.table.cuda()
    lens_d, row0_d = torch.tensor([rows[0], 1, 6], dtype=torch.int32).cuda(), _row0(rows).cuda()
    pp = pool.prefix_pages.cuda()
    n = binding.attention_workspace_bytes(3, 11, 8, 2, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = dict(out=torch.empty((11, 8, 128), dtype=BF16, device="cuda"), lse=torch.empty((11, 8), device="cuda"))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        binding.block_attention(qd, cache, table, lens_d, row0_d, prefix_pages=pp, prefix_len=150, out=out, workspace=ws)
    for lens, rr in ((full, rows), ([130, 7, 90], rows), ([300, 260, 12], [1, 1, 4])):
        lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        row0_d.copy_(_row0(rr))
        g.replay()
        torch.cuda.synchronize()
        pool.lens = lens
        _check({k: t[:sum(rr)] for k, t in out.items()},
               plain_cache.attention(q[:sum(rr)], pool, _row0(rr), lens), str(lens))


def test_pages_beyond_32_bit_offsets():
    n_pages, Hkv, page, D = 70000, 8, 64, 128      # 4.6 GB each of keys and values
    gen = torch.Generator().manual_seed(12)
    codes = [torch.empty((n_pages, Hkv, page, D), dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.empty((n_pages, Hkv, page), device="cuda") for _ in range(2)]
    cache = binding.KVCache(*codes, *scales)
    small = plain_cache.Pool(gen, [100], 70, Hkv, D, page, INT8, spare=0)
    where = torch.tensor([n_pages - 1, 5, n_pages - 2, n_pages - 7], dtype=torch.int32)
    for big, few in zip(codes + scales, (small.k, small.v, small.k_scale, small.v_scale)):
        big[where.long().cuda()] = few.cuda()
    q = torch.randn((2, 8, D), generator=gen).to(BF16)
    got = binding.block_attention(q.cuda(), cache, where[small.table.long()].cuda(),
                                  torch.tensor([100], dtype=torch.int32).cuda(), _row0([2]).cuda(),
                                  prefix_pages=where[small.prefix_pages.long()].cuda(), prefix_len=70)
    _check(got, plain_cache.attention(q, small, _row0([2]), [100]))


def test_append_attend_and_read_back_together():
    """A round's use: the block's keys and values go in, its rows attend."""
    gen = torch.Generator().manual_seed(13)
    rows, ctx, page, Hkv, D = [3, 6, 1], [61, 5, 130], 64, 2, 128
    lens = [c + n for c, n in zip(ctx, rows)]
    pool = plain_cache.Pool(gen, lens, 90, Hkv, D, page, E4M3)
    row0 = _row0(rows)
    cache = pool.cache(binding)
    k, v = [torch.randn((10, Hkv, D), generator=gen).to(BF16) for _ in range(2)]
    table = pool.table.cuda()
    binding.kv_append(k.cuda(), v.cuda(), cache, table, torch.tensor(ctx, dtype=torch.int32).cuda(), row0.cuda())
    q = torch.randn((10, 8, D), generator=gen).to(BF16)
    got = binding.block_attention(q.cuda(), cache, table, torch.tensor(lens, dtype=torch.int32).cuda(), row0.cuda(),
                                  prefix_pages=pool.prefix_pages.cuda(), prefix_len=90)
    pool.k, pool.v, pool.k_scale, pool.v_scale = [t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    _check(got, plain_cache.attention(q, pool, row0, lens))
