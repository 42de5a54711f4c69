"""dspark_kv_append and dspark_kv_read against the format's definition.

Codes and scales are bit-exact (the definition is a sequence of single fp32
operations), and so is a value read back (one fp32 product, one rounding)."""
import math

import pytest
import torch

import plain_cache
from speculative_decoding_draft_head_gb300 import binding

pytestmark = pytest.mark.gpu
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def _bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def _same_floats(a, b):
    a, b = a.cpu(), b.cpu()
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def _setup(gen, rows, start, page, Hkv, D, fmt):
    B = len(rows)
    need = [-(-(s + n) // page) for s, n in zip(start, rows)]
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=gen).to(torch.int32)
    table = torch.full((B, max(need + [1])), -7, dtype=torch.int32)   # entries past the end are never read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = binding.KVCache.empty(n_pages, Hkv, page, D, dtype=fmt)
    row0 = torch.tensor([0] + rows).cumsum(0)
    return cache, table, row0, torch.tensor(start, dtype=torch.int32)


def _places(table, row0, start, page):
    pg, off = [], []
    for b in range(len(start)):
        pos = torch.arange(int(row0[b + 1] - row0[b])) + int(start[b])
        pg.append(table[b].long()[pos // page])
        off.append(pos % page)
    return torch.cat(pg), torch.cat(off)


CASES = [  # rows, start, page, Hkv, D
    ([1], [0], 16, 1, 16),
    ([1, 1, 1], [0, 15, 16], 16, 2, 64),
    ([0, 5, 0, 3, 1, 0], [7, 0, 3, 30, 31, 5], 32, 3, 80),
    ([6, 2, 4, 1], [100, 64, 63, 1], 48, 8, 128),
    ([700, 1, 260], [5, 0, 1000], 64, 5, 96),
    ([9] * 70, list(range(70)), 16, 4, 48),
    ([3000, 2500], [17, 0], 128, 2, 128),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("rows,start,page,Hkv,D", CASES)
def test_append_then_read_is_exact(rows, start, page, Hkv, D, fmt, dtype):
    gen = torch.Generator().manual_seed(sum(rows) + D)
    cache, table, row0, start = _setup(gen, rows, start, page, Hkv, D, fmt)
    R = sum(rows)
    # rows of very different size, some zero, some below the least maximum
    size = 2.0 ** torch.randint(-20, 8, (R, Hkv, 1), generator=gen).float()
    x = [(torch.randn((R, Hkv, D), generator=gen) * size) for _ in range(2)]
    x[0][:: 5] = 0
    if dtype != torch.float16:
        x[1][:: 7] = 2.0 ** -110
    k, v = [t.to(dtype) for t in x]
    dev = [t.cuda() for t in (table, start, row0)]
    binding.kv_append(k.cuda(), v.cuda(), cache, *dev)
    pg, off = _places(table, row0, start, page)
    for t, codes, scales in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        want, sc = plain_cache.quantise(t, fmt)
        got = codes.view(torch.uint8).cpu()[pg, :, off]
        assert torch.equal(got, want.view(torch.uint8))
        assert torch.equal(scales.cpu()[pg, :, off], sc)
        # nothing else is touched
        rest = codes.view(torch.uint8).cpu()
        rest[pg, :, off] = 0
        assert int(rest.count_nonzero()) == 0
    for out in (torch.bfloat16, torch.float16, torch.float32):
        got = binding.kv_read(cache, *dev, R, dtype=out)
        for name, t in (("k", k), ("v", v)):
            want, sc = plain_cache.quantise(t, fmt)
            assert torch.equal(_bits(got[name]), _bits((want.float() * sc[..., None]).to(out)))
    only = dict(v=torch.empty_like(got["v"]))
    binding.kv_read(cache, *dev, R, dtype=torch.float32, out=only)
    assert torch.equal(only["v"], got["v"])
    assert binding.read_device_flags(cache.flags) == 0


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("Hkv,D", [(3, 64), (1, 16), (9, 32), (5, 80), (11, 128)])
def test_many_rows_and_heads_that_divide_nothing(Hkv, D, fmt):
    """More rows than fit a row a block, heads that end inside a step; rows and
    heads of which no two are alike."""
    rows, starts = [5001, 0, 1, 4999, 3], [3, 0, 15, 16, 31]
    gen = torch.Generator().manual_seed(Hkv * D)
    cache, table, row0, start = _setup(gen, rows, starts, 16, Hkv, D, fmt)
    R = sum(rows)
    k, v = [torch.randn((R, Hkv, D), generator=gen).to(torch.bfloat16) for _ in range(2)]
    k[7, 0, 3], v[5003, Hkv - 1, D - 1] = math.inf, math.nan
    dev = [t.cuda() for t in (table, start, row0)]
    binding.kv_append(k.cuda(), v.cuda(), cache, *dev)
    pg, off = _places(table, row0, start, 16)
    got = binding.kv_read(cache, *dev, R, dtype=torch.float32)
    for name, t, codes, scales in (("k", k, cache.k, cache.k_scale), ("v", v, cache.v, cache.v_scale)):
        want, sc = plain_cache.quantise(t, fmt)
        assert torch.equal(codes.view(torch.uint8).cpu()[pg, :, off], want.view(torch.uint8))
        assert _same_floats(scales.cpu()[pg, :, off], sc)
        assert _same_floats(got[name], want.float() * sc[..., None])
    assert binding.read_device_flags(cache.flags) == binding.FLAG_NONFINITE


@pytest.mark.parametrize("fmt", [E4M3, INT8])
def test_every_code_rounds_and_reads_as_defined(fmt):
    """A dense sweep of values in [-Q, Q] against the plain rounding; the row's
    largest element fixes the scale at 1."""
    top = plain_cache.TOP[fmt]
    x = torch.linspace(-top, top, 127 * 640).view(640, 1, 127)
    x = torch.cat([torch.full((640, 1, 1), top), x], 2)
    cache, table, row0, start = _setup(torch.Generator().manual_seed(0), [640], [0], 64, 1, 128, fmt)
    binding.kv_append(x.cuda(), -x.cuda(), cache, table.cuda(), start.cuda(), row0.cuda())
    got = binding.kv_read(cache, table.cuda(), start.cuda(), row0.cuda(), 640, dtype=torch.float32)
    want, sc = plain_cache.quantise(x, fmt)
    assert torch.equal(got["k"].cpu(), want.float() * sc[..., None])
    assert torch.equal(got["v"].cpu(), -(want.float() * sc[..., None]))


def test_nonfinite_rows_are_contained_and_flagged():
    cache, table, row0, start = _setup(torch.Generator().manual_seed(0), [4], [0], 16, 2, 64, E4M3)
    k = torch.randn(4, 2, 64)
    k[1, 0, 5], k[2, 1, 63] = math.inf, math.nan
    binding.kv_append(k.cuda(), k.cuda(), cache, table.cuda(), start.cuda(), row0.cuda())
    assert binding.read_device_flags(cache.flags) == binding.FLAG_NONFINITE
    got = binding.kv_read(cache, table.cuda(), start.cuda(), row0.cuda(), 4, dtype=torch.float32)["k"].cpu()
    bad = torch.zeros(4, 2, dtype=torch.bool)
    bad[1, 0] = bad[2, 1] = True
    assert torch.equal(got.isnan().all(2), bad) and torch.equal(got.isnan().any(2), bad)
    assert int(cache.k.view(torch.uint8)[int(table[0, 0]), 0, 1].count_nonzero()) == 0


def test_bad_places_are_flagged_and_not_touched():
    cache, table, row0, start = _setup(torch.Generator().manual_seed(0), [2, 2, 2, 2], [0, 0, 0, 14], 16, 1, 32, INT8)
    table = table[:, :1].contiguous()             # request 3 would need a second page for neither row: 14, 15 fit
    table[1, 0] = cache.n_pages                   # one past the end
    start[2] = -1
    start[3] = 15                                 # its second row lies past max_pages
    x = torch.randn(8, 1, 32)
    binding.kv_append(x.cuda(), x.cuda(), cache, table.cuda(), start.cuda(), row0.cuda())
    flags = binding.read_device_flags(cache.flags)
    assert flags == binding.FLAG_BAD_PAGE | binding.FLAG_BAD_LENGTH
    got = binding.kv_read(cache, table.cuda(), start.cuda(), row0.cuda(), 8, dtype=torch.float32)["k"].cpu()
    assert got.isnan().all(2)[:, 0].tolist() == [False, False, True, True, True, True, False, True]
    written = (cache.k_scale.cpu() != 0).sum()
    assert int(written) == 3


def test_rows_of_no_request_are_left_alone():
    cache, table, row0, start = _setup(torch.Generator().manual_seed(0), [2, 3], [0, 4], 16, 2, 64, E4M3)
    x = torch.randn(9, 2, 64)
    x[5:] = math.nan
    binding.kv_append(x.cuda(), x.cuda(), cache, table.cuda(), start.cuda(), row0.cuda())
    out = dict(k=torch.full((9, 2, 64), 7.0, device="cuda"), v=torch.full((9, 2, 64), 7.0, device="cuda"))
    binding.kv_read(cache, table.cuda(), start.cuda(), row0.cuda(), 9, dtype=torch.float32, out=out)
    assert bool((out["k"][5:] == 7).all()) and bool((out["k"][:5] != 7).any())
    assert binding.read_device_flags(cache.flags) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slices_of_a_fused_projection(dtype):
    gen = torch.Generator().manual_seed(3)
    cache, table, row0, start = _setup(gen, [40, 7], [3, 0], 32, 2, 64, E4M3)
    fused = torch.randn((47, 8, 64), generator=gen).to(dtype).cuda()
    k, v = fused[:, 4:6], fused[:, 6:8]
    binding.kv_append(k, v, cache, table.cuda(), start.cuda(), row0.cuda())
    got = binding.kv_read(cache, table.cuda(), start.cuda(), row0.cuda(), 47, dtype=torch.float32)
    for name, t in (("k", k), ("v", v)):
        want, sc = plain_cache.quantise(t.cpu(), E4M3)
        assert torch.equal(got[name].cpu(), want.float() * sc[..., None])
    with pytest.raises(ValueError, match="contiguous"):
        binding.kv_append(fused[:, ::4], v, cache, table.cuda(), start.cuda(), row0.cuda())


def test_places_beyond_32_bit_offsets():
    """A cache whose codes pass 2^32 bytes: the last pages are the ones used."""
    n_pages, Hkv, page, D = 70000, 8, 64, 128       # 4.6 GB each of keys and values
    codes = [torch.empty((n_pages, Hkv, page, D), dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.empty((n_pages, Hkv, page), device="cuda") for _ in range(2)]
    cache = binding.KVCache(*codes, *scales)
    table = torch.tensor([[n_pages - 1, 3]], dtype=torch.int32).cuda()
    row0, start = torch.tensor([0, 80]).cuda(), torch.tensor([20], dtype=torch.int32).cuda()
    k, v = [torch.randn(80, Hkv, D).half() for _ in range(2)]
    binding.kv_append(k.cuda(), v.cuda(), cache, table, start, row0)
    got = binding.kv_read(cache, table, start, row0, 80, dtype=torch.float32)
    for name, t in (("k", k), ("v", v)):
        want, sc = plain_cache.quantise(t, INT8)
        assert torch.equal(got[name].cpu(), want.float() * sc[..., None])
    assert _same_floats(scales[0][n_pages - 1, :, 20:], plain_cache.quantise(k, INT8)[1][:44].T)


def test_on_another_stream_and_in_a_graph():
    gen = torch.Generator().manual_seed(5)
    cache, table, row0, start = _setup(gen, [33, 12], [2, 9], 16, 2, 64, INT8)
    k, v = [torch.randn((45, 2, 64), generator=gen).cuda() for _ in range(2)]
    dev = [t.cuda() for t in (table, start, row0)]
    out = dict(k=torch.zeros(45, 2, 64, device="cuda"), v=torch.zeros(45, 2, 64, device="cuda"))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            binding.kv_append(k, v, cache, *dev)
            binding.kv_read(cache, *dev, 45, dtype=torch.float32, out=out)
        for _ in range(2):
            k.copy_(torch.randn((45, 2, 64), generator=gen))
            g.replay()
    s.synchronize()
    want, sc = plain_cache.quantise(k.cpu(), INT8)
    assert torch.equal(out["k"].cpu(), want.float() * sc[..., None])
