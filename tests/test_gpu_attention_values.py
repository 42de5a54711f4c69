"""Values of very different size in one call of dspark_block_attention.

Each row's output is made of the values that the row sees: what it does not see
may be of any size.  The bounds count one fp16 rounding in the inner terms, that
of the softmax term times the value's scale (the codes themselves are exact in
fp16): plain_cache.attention's derivation with 2^-11 in place of two of them."""
import math

import pytest
import torch

import plain_cache
from speculative_decoding_draft_head_gb300 import binding

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16, F16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16, torch.float16


def _row0(rows):
    return torch.tensor([0] + list(rows)).cumsum(0)


def _put(pool, pages, t, k=None, v=None):
    """Overwrites token t of a list with rows k, v [Hkv, D]."""
    pg, off = int(pages[t // pool.page]), t % pool.page
    for x, codes, scales in ((k, pool.k, pool.k_scale), (v, pool.v, pool.v_scale)):
        if x is not None:
            c, s = plain_cache.quantise(x, pool.dtype)
            codes.view(torch.uint8)[pg, :, off] = c.view(torch.uint8)
            scales[pg, :, off] = s


def _attend(q, pool, lens, row0, prefix, **kw):
    cache = pool.cache(binding)
    got = binding.block_attention(
        q.cuda(), cache, pool.table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), row0.cuda(),
        prefix_pages=pool.prefix_pages.cuda() if prefix else None, prefix_len=prefix, **kw)
    torch.cuda.synchronize()
    assert binding.read_device_flags(cache.flags) == 0
    return {k: t.double().cpu() for k, t in got.items()}


def _inside(got, want):
    out, lse, tol_out, tol_lse = want
    over = ((got["out"] - out).abs() / tol_out).max()
    assert bool(over <= 1), "out: %g of its bound" % over
    empty = lse == -math.inf
    assert torch.equal(got["lse"] == -math.inf, empty)
    assert bool((torch.where(empty, 0.0, got["lse"] - lse).abs() <= tol_lse).all())


@pytest.mark.parametrize("size", [1e5, 1e12, 1e25])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("rows,group", [(4, 2), (40, 4)])
def test_large_values_that_a_row_does_not_see(rows, group, prefix, dtype, size):
    """The block's last token has values `size` times the others': under the causal mask no other row sees it."""
    gen = torch.Generator().manual_seed(1)
    ctx, Hkv, D = 100, 2, 64
    pool = plain_cache.Pool(gen, [ctx + rows], prefix, Hkv, D, 16, E4M3)
    _put(pool, pool.table[0], ctx + rows - 1, v=size * torch.randn((Hkv, D), generator=gen))
    q = torch.randn((rows, group * Hkv, D), generator=gen).to(dtype)
    row0, lens = _row0([rows]), [ctx + rows]
    got = _attend(q, pool, lens, row0, prefix)
    want = plain_cache.attention(q, pool, row0, lens, terms=2.0 ** -11)
    _inside({k: t[:-1] for k, t in got.items()}, [t[:-1] for t in want])
    if dtype is BF16:
        _inside(got, want)


@pytest.mark.parametrize("fmt", [E4M3, INT8])
def test_large_values_outside_a_trees_branches(fmt):
    gen = torch.Generator().manual_seed(2)
    n, ctx, Hkv, D = 24, 37, 1, 128
    pool = plain_cache.Pool(gen, [ctx + n], 0, Hkv, D, 32, fmt)
    for t in range(0, n, 3):        # every third node is large, and seen by itself alone
        _put(pool, pool.table[0], ctx + t, v=2.0 ** 40 * torch.randn((Hkv, D), generator=gen))
    small = sum(1 << t for t in range(n) if t % 3)
    words = torch.tensor([(small & ((2 << i) - 1)) | (1 << i) for i in range(n)])
    q = torch.randn((n, 4, D), generator=gen).to(BF16)
    row0, lens = _row0([n]), [ctx + n]
    _inside(_attend(q, pool, lens, row0, 0, row_mask=words.cuda()),
            plain_cache.attention(q, pool, row0, lens, words=words, terms=2.0 ** -11))


@pytest.mark.parametrize("prefix,first", [(0, "small"), (0, "large"), (256, "small"), (256, "large")])
@pytest.mark.parametrize("top", [2.0 ** 30, 2.0 ** 85])
def test_the_sum_counts_tokens_whose_values_are_far_smaller(top, prefix, first):
    """Half of the tokens have values of zero, the others of size `top`; all weights are alike, so that out and lse
    show whether each token was counted, within one worker's tokens and where parts are joined."""
    gen = torch.Generator().manual_seed(3)
    n, Hkv, D, page = 512 - prefix, 1, 64, 64
    pool = plain_cache.Pool(gen, [n], prefix, Hkv, D, page, E4M3)
    lists = [(pool.prefix_pages, prefix, 0), (pool.table[0], n, prefix)]
    for pages, count, at in lists:
        for t in range(count):
            small = (at + t < 256) == (first == "small")
            _put(pool, pages, t, k=torch.zeros((Hkv, D)),
                 v=torch.zeros((Hkv, D)) if small else top * torch.randn((Hkv, D), generator=gen))
    q = torch.randn((1, 2, D), generator=gen).to(BF16)
    got = _attend(q, pool, [n], _row0([1]), prefix, mask="full")
    _inside(got, plain_cache.attention(q, pool, _row0([1]), [n], mask="full", terms=2.0 ** -11))
    assert bool(((got["lse"] - math.log(512)).abs() < 1e-4).all())


@pytest.mark.parametrize("fmt,dtype", [(E4M3, BF16), (E4M3, F16), (INT8, F16)])
@pytest.mark.parametrize("rows,ctx,prefix,Hq,Hkv,D", [
    ([1], [777], 0, 8, 2, 128),
    ([6, 1, 4], [700, 300, 20], 400, 8, 2, 128),
    ([40, 3], [300, 128], 260, 24, 2, 128),
    ([17, 33], [90, 10], 70, 16, 1, 64),
    ([7, 2], [140, 20], 250, 4, 4, 96),
])
def test_one_rounding_of_the_inner_terms(rows, ctx, prefix, Hq, Hkv, D, fmt, dtype):
    gen = torch.Generator().manual_seed(4)
    lens = [c + n for c, n in zip(ctx, rows)]
    pool = plain_cache.Pool(gen, lens, prefix, Hkv, D, 64, fmt,
                            token_scale=lambda g, s: 2.0 ** torch.randint(-6, 7, s, generator=g).float())
    q = torch.randn((sum(rows), Hq, D), generator=gen).to(dtype)
    _inside(_attend(q, pool, lens, _row0(rows), prefix),
            plain_cache.attention(q, pool, _row0(rows), lens, terms=2.0 ** -11))
