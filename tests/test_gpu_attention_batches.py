"""dspark_block_attention over large batches, over pages that hold more than a
tile of tokens, and a request by itself against the same one in a batch.  The
bounds are those of plain_cache.attention for one rounding of the inner terms."""
import math

import pytest
import torch

import plain_cache
from speculative_decoding_draft_head_gb300 import binding

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16, F16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16, torch.float16


def _row0(rows):
    return torch.tensor([0] + list(rows)).cumsum(0)


def _attend(q, cache, pool, lens, row0, table=None, **kw):
    got = binding.block_attention(
        q.cuda(), cache, (pool.table if table is None else table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
        row0.cuda(), prefix_pages=pool.prefix_pages.cuda() if pool.prefix else None, prefix_len=pool.prefix, **kw)
    torch.cuda.synchronize()
    return {k: t.double().cpu() for k, t in got.items()}


def _inside(got, want):
    out, lse, tol_out, tol_lse = want
    assert not bool(got["out"].isnan().any())
    assert bool(((got["out"] - out).abs() <= tol_out).all()), float(((got["out"] - out).abs() / tol_out).max())
    assert bool(((got["lse"] - lse).abs() <= tol_lse).all())


def _many(B, seed):
    """B requests of 0 to 4 rows over 0 to 150 earlier tokens."""
    gen = torch.Generator().manual_seed(seed)
    rows = torch.randint(0, 5, (B,), generator=gen).tolist()
    ctx = torch.randint(0, 151, (B,), generator=gen).tolist()
    return gen, rows, [c + n for c, n in zip(ctx, rows)]


@pytest.mark.parametrize("B,prefix", [(641, 0), (700, 40), (1280, 0), (1301, 130)])
def test_more_requests_than_a_block_has_threads(B, prefix):
    gen, rows, lens = _many(B, B)
    pool = plain_cache.Pool(gen, lens, prefix, 1, 64, 16, E4M3)
    q = torch.randn((sum(rows), 2, 64), generator=gen).to(BF16)
    cache = pool.cache(binding)
    got = _attend(q, cache, pool, lens, _row0(rows))
    assert binding.read_device_flags(cache.flags) == 0
    _inside(got, plain_cache.attention(q, pool, _row0(rows), lens, terms=2.0 ** -11))


def test_a_pair_tile_and_a_bad_length_among_the_last_of_many_requests():
    gen, rows, lens = _many(1000, 5)
    rows[800], lens[800] = 40, 300          # 160 rows of a kv head: the only item of its class
    rows[900], lens[900] = 3, 20
    pool = plain_cache.Pool(gen, lens, 0, 1, 64, 16, E4M3)
    q = torch.randn((sum(rows), 4, 64), generator=gen).to(BF16)
    cache = pool.cache(binding)
    given = list(lens)
    given[900] = 2                           # shorter than its block
    row0 = _row0(rows)
    got = _attend(q, cache, pool, given, row0)
    assert binding.read_device_flags(cache.flags) == binding.FLAG_BAD_LENGTH
    bad = slice(int(row0[900]), int(row0[901]))
    assert bool(got["out"][bad].isnan().all()) and bool(got["lse"][bad].isnan().all())
    want = plain_cache.attention(q, pool, row0, lens, terms=2.0 ** -11)
    good = torch.ones(len(q), dtype=torch.bool)
    good[bad] = False
    _inside({k: t[good] for k, t in got.items()}, [t[good] for t in want])


@pytest.mark.parametrize("fmt,dtype", [(E4M3, BF16), (INT8, F16)])
@pytest.mark.parametrize("page", [144, 160, 256, 512, 1040])
def test_pages_of_more_than_a_tile(page, fmt, dtype):
    gen = torch.Generator().manual_seed(page)
    rows, ctx, prefix = [5, 1, 33], [page - 3, 3 * page + 17, 129], page + 100
    lens = [c + n for c, n in zip(ctx, rows)]
    pool = plain_cache.Pool(gen, lens, prefix, 2, 64, page, fmt)
    q = torch.randn((sum(rows), 8, 64), generator=gen).to(dtype)
    cache = pool.cache(binding)
    got = _attend(q, cache, pool, lens, _row0(rows))
    assert binding.read_device_flags(cache.flags) == 0
    _inside(got, plain_cache.attention(q, pool, _row0(rows), lens, terms=2.0 ** -11))


def test_a_request_alone_and_in_a_batch():
    """Where an item is cut follows from the whole batch, so that bits may differ: each result has to be inside the
    bounds, and the two within both."""
    gen = torch.Generator().manual_seed(21)
    rows, ctx, prefix = [5, 2, 6, 40, 1], [3000, 10, 130, 700, 5000], 1500
    lens = [c + n for c, n in zip(ctx, rows)]
    pool = plain_cache.Pool(gen, lens, prefix, 2, 128, 64, E4M3)
    q = torch.randn((sum(rows), 8, 128), generator=gen).to(BF16)
    cache, row0 = pool.cache(binding), _row0(rows)
    batch = _attend(q, cache, pool, lens, row0)
    want = plain_cache.attention(q, pool, row0, lens, terms=2.0 ** -11)
    _inside(batch, want)
    for b in range(len(rows)):
        at = slice(int(row0[b]), int(row0[b + 1]))
        alone = _attend(q[at], cache, pool, lens[b:b + 1], _row0(rows[b:b + 1]), table=pool.table[b:b + 1].contiguous())
        _inside(alone, [t[at] for t in want])
        for name, tol in (("out", want[2]), ("lse", want[3])):
            assert bool(((alone[name] - batch[name][at]).abs() <= 2 * tol[at]).all())


def test_where_nan_may_stand():
    """Out and lse are NaN exactly where a row sees a NaN token."""
    gen = torch.Generator().manual_seed(22)
    rows, ctx, page = [4, 3], [70, 20], 32
    lens = [c + n for c, n in zip(ctx, rows)]
    pool = plain_cache.Pool(gen, lens, 50, 2, 64, page, E4M3)
    for b, t in ((0, ctx[0] + 2), (1, ctx[1] + 1)):
        pg, off = int(pool.table[b, t // page]), t % page
        pool.v.view(torch.uint8)[pg, 1, off] = 0            # the second kv head's values only
        pool.v_scale[pg, 1, off] = math.nan
    q = torch.randn((7, 4, 64), generator=gen).to(BF16)
    got = _attend(q, pool.cache(binding), pool, lens, _row0(rows))
    bad = torch.zeros((7, 4), dtype=torch.bool)
    bad[2:4, 2:] = bad[5:, 2:] = True
    assert torch.equal(got["out"].isnan(), bad[..., None].expand(7, 4, 64)) and torch.equal(got["lse"].isnan(), bad)
    clean = plain_cache.attention(q, pool, _row0(rows), lens, terms=2.0 ** -11)
    assert bool(((got["out"] - clean[0]).abs() <= clean[2])[~bad].all())
    assert bool(((got["lse"] - clean[1]).abs() <= clean[3])[~bad].all())
