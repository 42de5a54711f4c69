"""Rotary positions, the cache and the attention through a window as a target model uses them together: prompts,
drafted blocks and single tokens appended and attended to step after step, in a cache whose pages are given away
when the window has passed them, and the example's rounds."""
import os
import sys

import pytest
import torch

import plain_cache
import plain_rotary
import plain_window
from speculative_decoding_draft_head_gb300 import binding

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class _Seen:
    """What plain_window needs of a pool: the cache as it is now."""

    def __init__(self, cache, table, prefix_pages, prefix):
        self.k, self.v, self.k_scale, self.v_scale = (t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
        self.page, self.dtype, self.prefix = cache.page_size, cache.k.dtype, prefix
        self.table, self.prefix_pages = table, prefix_pages


def _check(got, want):
    out, lse, tol_out, tol_lse = want
    assert ((got["out"].cpu().double() - out).abs() <= tol_out).all()
    assert ((got["lse"].cpu().double() - lse).abs() <= tol_lse).all()


@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("prefix,window,sinks,page", [(0, 40, 4, 16), (50, 33, 20, 32)])
def test_steps_over_pages_that_are_given_away(prefix, window, sinks, page, fmt):
    gen = torch.Generator().manual_seed(prefix + page)
    B, Hq, Hkv, D = 3, 6, 2, 64
    freq, z = plain_rotary.frequencies(D // 2), binding.Rotary(plain_rotary.frequencies(D // 2))
    slots, shared = 24, -(-prefix // page)
    pages = list(range(60))
    prefix_pages = torch.tensor(pages[:shared], dtype=torch.int32)
    free = pages[shared:]
    table = torch.full((B, slots), -1, dtype=torch.int32)
    cache = binding.KVCache.empty(60, Hkv, page, D, dtype=fmt)

    def rows_of(n, dtype=torch.bfloat16):
        return [torch.randn((n, h, D), generator=gen).to(dtype) for h in (Hq, Hkv, Hkv)]

    if prefix:
        _, k, v = rows_of(prefix)
        binding.kv_append_rotary(k.cuda(), v.cuda(), cache, prefix_pages[None].cuda(), torch.zeros(1).int().cuda(),
                                 torch.tensor([0, prefix]).cuda(), z)
    length = [0] * B
    given_back, again = set(), 0
    # prompts of different lengths, drafted blocks, single tokens
    for rows in ([70, 1, 30], [6, 1, 4], [1, 1, 1], [3, 0, 6], [1, 1, 1], [40, 50, 1], [5, 5, 5], [1, 1, 1]):
        for b in range(B):
            for slot in range(-(-(length[b] + rows[b]) // page)):
                if table[b, slot] < 0 and (slot + 1) * page > length[b]:
                    table[b, slot] = free.pop(0)
                    again += int(table[b, slot]) in given_back
        row0 = torch.tensor([0] + rows).cumsum(0)
        q, k, v = rows_of(sum(rows))
        dev = [t.cuda() for t in (table, torch.tensor(length).int(), row0)]
        turned = binding.kv_append_rotary(k.cuda(), v.cuda(), cache, *dev, z, q=q.cuda(), offset=prefix)
        at = torch.cat([torch.arange(n) + prefix + length[b] for b, n in enumerate(rows)])[None]
        want, tol = plain_rotary.turn(q, at, freq)
        assert ((turned.cpu().double() - want).abs() <= tol * 1.01 + 2.0 ** -8 * want.abs() + 2.0 ** -130).all()
        lens = [length[b] + n for b, n in enumerate(rows)]
        got = binding.window_attention(turned, cache, table.cuda(), torch.tensor(lens).int().cuda(), row0.cuda(), window=window,
                                       sinks=sinks, prefix_pages=prefix_pages.cuda() if prefix else None, prefix_len=prefix)
        assert binding.read_device_flags(cache.flags) == 0
        _check(got, plain_window.attention(turned.cpu(), _Seen(cache, table, prefix_pages, prefix), row0, lens, window, sinks))
        length = lens
        # pages that the next row's window does not reach, and that hold no first token, go back
        for b in range(B):
            low = prefix + length[b] - window + 1
            for slot in range(slots):
                if table[b, slot] >= 0 and prefix + (slot + 1) * page <= low and prefix + slot * page >= sinks:
                    free.insert(0, int(table[b, slot]))
                    given_back.add(int(table[b, slot]))
                    table[b, slot] = -1
    assert again > 0        # some pages have been another's before


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import target_pass
    return target_pass


@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.int8])
def test_rounds_with_positions_and_a_window(example, fmt):
    """The cached keys are those of the tokens given, turned by their places behind the prompt."""
    rounds, G, prompt = 5, 5, 77
    r = example.run(rounds=rounds, B=9, prompt=prompt, G=G, V=1024, page=16, dtype=fmt, rotary=True, window=20, sinks=4)
    assert binding.read_device_flags(r["cache"].flags) == 0
    length, tokens = r["length"].cpu(), r["tokens"].cpu().long()
    row0 = torch.zeros(10, dtype=torch.int64)
    row0[1:] = length.cumsum(0)
    got = binding.kv_read(r["cache"], r["block_table"], torch.zeros_like(r["length"]), row0.cuda(), int(row0[-1]),
                          dtype=torch.float32)
    rows = torch.cat([tokens[b, :length[b]] for b in range(9)])
    want, scale = plain_cache.quantise(r["target"].v.cpu()[rows], fmt)
    assert torch.equal(got["v"].cpu(), want.float() * scale[..., None])
    at = torch.cat([torch.arange(int(n)) + prompt for n in length])[None]
    want, tol = plain_rotary.turn(r["target"].k.cpu()[rows], at, plain_rotary.frequencies(64))
    top = plain_cache.TOP[fmt]
    amax = want.abs().amax(-1, keepdim=True)
    step = amax / top / 2 if fmt == torch.int8 else torch.maximum(2.0 ** -4 * want.abs(), amax / top * 2.0 ** -10)
    assert ((got["k"].cpu().double() - want).abs() <= step * (1 + 2.0 ** -20) + 2 * tol.amax(-1, keepdim=True) + 2.0 ** -20 * want.abs()).all()

