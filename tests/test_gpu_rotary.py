"""dspark_rotary_rows and dspark_kv_append_rotary against the turning's formula in
64 bits (see plain_rotary for the bounds)."""
import math

import pytest
import torch

import plain_cache
import plain_rotary
from speculative_decoding_draft_head_gb300 import binding

pytestmark = pytest.mark.gpu
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
FAR = 2 ** 31 - 1


def _rounded(y, tol, dtype):
    info = torch.finfo(dtype)
    return tol * (1 + 2.0 ** -8) + info.eps / 2 * y.abs() + info.smallest_normal * info.eps / 2


def _positions(gen, axes, n):
    p = torch.randint(0, 5000, (axes, n), generator=gen)
    p[0, :: 3] = torch.randint(-FAR, FAR, p[0, :: 3].shape, generator=gen)
    p.view(-1)[-1] = FAR
    p.view(-1)[0] = -FAR - 1
    return p.int()


CASES = [  # rows, heads, D, pairs, adjacent, axes
    (1, 1, 8, 4, False, 1),
    (1, 3, 64, 32, True, 1),
    (7, 1, 128, 64, False, 1),
    (33, 5, 80, 40, False, 3),
    (129, 2, 72, 36, True, 2),
    (65, 4, 96, 20, False, 3),
    (40, 3, 256, 128, False, 1),
    (500, 9, 128, 16, True, 2),
    (20011, 1, 64, 32, False, 1),
    (40003, 2, 32, 12, True, 3),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["rows", "heads", "slice"])
@pytest.mark.parametrize("n,heads,D,pairs,adjacent,axes", CASES)
def test_rows(n, heads, D, pairs, adjacent, axes, layout, dtype):
    gen = torch.Generator().manual_seed(n + heads)
    freq = plain_rotary.frequencies(pairs)
    axis = None if axes == 1 else torch.randint(axes, (pairs,), generator=gen)
    if axis is not None:
        axis[-1] = axes - 1
    pos = _positions(gen, axes, n)
    if layout == "rows":
        x = torch.randn((n, heads, D), generator=gen).to(dtype).cuda()
    elif layout == "heads":
        x = torch.randn((heads, n, D), generator=gen).to(dtype).cuda().transpose(0, 1)
    else:
        x = torch.randn((n, heads + 3, D), generator=gen).to(dtype).cuda()[:, 2:2 + heads]
    z = binding.Rotary(freq, axis=None if axis is None else axis.tolist(), adjacent=adjacent)
    before = x.clone()
    for inverse in (False, True):
        got = binding.rotary(x, z, pos.cuda(), inverse=inverse)
        want, tol = plain_rotary.turn(x.cpu(), pos, freq, axis, adjacent, inverse)
        assert got.shape == x.shape and got.dtype == dtype
        assert ((got.cpu().double() - want).abs() <= _rounded(want, tol, dtype)).all()
        assert torch.equal(got[..., 2 * pairs:], x[..., 2 * pairs:])
    assert torch.equal(x, before)
    assert binding.rotary(x, z, pos.cuda(), inverse=True, out=x) is x and torch.equal(x, got)   # in place
    if layout == "slice":       # what lies between the rows stays
        whole = torch.zeros((n, heads + 3, D), dtype=dtype, device="cuda")
        binding.rotary(before, z, pos.cuda(), inverse=True, out=whole[:, 2:2 + heads])
        assert torch.equal(whole[:, 2:2 + heads], got) and not whole[:, :2].any() and not whole[:, 2 + heads:].any()


def test_nothing_to_turn():
    z = binding.Rotary(plain_rotary.frequencies(32))
    x = torch.zeros((0, 4, 64), device="cuda")
    assert binding.rotary(x, z, torch.zeros(0, dtype=torch.int32, device="cuda")).shape == x.shape


def test_position_zero_changes_no_bit():
    x = torch.randn((50, 3, 128), device="cuda").bfloat16()
    z = binding.Rotary(plain_rotary.frequencies(64))
    assert torch.equal(binding.rotary(x, z, torch.zeros(50, dtype=torch.int32, device="cuda")), x)


def test_frequencies_past_a_turn_and_below_zero():
    gen = torch.Generator().manual_seed(0)
    freq = torch.tensor([0.0, -0.5, 7.0, -1e4], dtype=torch.float64)
    pos, x = _positions(gen, 1, 30), torch.randn((30, 1, 8), generator=gen)
    got = binding.rotary(x.cuda(), binding.Rotary(freq), pos.cuda())
    want, tol = plain_rotary.turn(x, pos, freq)
    assert ((got.cpu().double() - want).abs() <= _rounded(want, tol, torch.float32)).all()


@pytest.mark.parametrize("adjacent", [False, True])
def test_inverse_is_the_gradient(adjacent):
    """Of L = sum(g * turned(x)): by the formula's own derivative, and by differences of L in 64 bits (L is linear in
    x, so a difference has the turning's own bound only)."""
    gen = torch.Generator().manual_seed(5)
    freq, axis = plain_rotary.frequencies(40), [i % 3 for i in range(40)]
    pos = torch.randint(0, 3000, (3, 21), generator=gen).int()
    x = torch.randn((21, 4, 96), generator=gen)
    g = torch.randn((21, 4, 96), generator=gen)
    z = binding.Rotary(freq, axis=axis, adjacent=adjacent)
    grad = binding.rotary(g.cuda(), z, pos.cuda(), inverse=True).cpu().double()
    leaf = x.double().requires_grad_()
    n = 40
    t = plain_rotary.angles(pos, freq, axis)[:, None]
    a, b = (leaf[..., 0:2 * n:2], leaf[..., 1:2 * n:2]) if adjacent else (leaf[..., :n], leaf[..., n:2 * n])
    ya, yb = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
    y = torch.cat([torch.stack([ya, yb], -1).flatten(2) if adjacent else torch.cat([ya, yb], -1), leaf[..., 2 * n:]], -1)
    (y * g.double()).sum().backward()
    _, tol = plain_rotary.turn(g, pos, freq, axis, adjacent, True)
    assert ((grad - leaf.grad).abs() <= _rounded(leaf.grad, tol, torch.float32)).all()
    for r, h, d in ((0, 0, 0), (20, 3, 95), (7, 1, 41), (9, 2, 79)):
        step = torch.zeros_like(x)
        step[r, h, d] = 0.5
        up, down = (binding.rotary((x + k * step).cuda(), z, pos.cuda()).cpu().double() for k in (1, -1))
        diff = ((up - down) * g.double())[r, h].sum()
        # two turned rows' bounds times |g| over the three elements that x[r, h, d] reaches at most
        reach = ((x[r, h].abs().max() + 0.5) * 2 * plain_rotary.ANGLE * 2 + 2 * 2.0 ** -24 * 8) * g[r, h].abs().max() * 3
        assert (diff - grad[r, h, d]).abs() <= reach + tol[r, h, d] + 2.0 ** -23 * grad[r, h, d].abs()


# --------------------------------------------------------------------------------------------------- the append
def _setup(gen, rows, start, page, Hkv, D, fmt):
    need = [-(-(s + n) // page) for s, n in zip(start, rows)]
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=gen).to(torch.int32)
    table = torch.full((len(rows), max(need + [1])), -7, dtype=torch.int32)   # entries past the end are never read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = binding.KVCache.empty(n_pages, Hkv, page, D, dtype=fmt)
    return cache, table, torch.tensor([0] + rows).cumsum(0), torch.tensor(start, dtype=torch.int32)


def _places(table, row0, start, page):
    pg, off, pos = [], [], []
    for b in range(len(start)):
        p = torch.arange(int(row0[b + 1] - row0[b])) + int(start[b])
        pg.append(table[b].long()[p // page])
        off.append(p % page)
        pos.append(p)
    return torch.cat(pg), torch.cat(off), torch.cat(pos)


def _check_keys(codes, scales, pg, off, want, tol, fmt):
    """Codes and scales of turned keys: the scale is the row's largest element (off by `tol`) over Q, a code half a step."""
    top = plain_cache.TOP[fmt]
    sc = scales.cpu()[pg, :, off].double()
    assert ((sc * top - want.abs().amax(-1)).abs() <= tol.amax(-1) + 2.0 ** -22 * want.abs().amax(-1) + 2.0 ** -100).all()
    got = codes.cpu().view(torch.uint8)[pg, :, off].view(fmt).double() * sc[..., None]
    step = sc[..., None] * 0.5 if fmt == INT8 else torch.maximum(2.0 ** -4 * want.abs(), sc[..., None] * 2.0 ** -10)
    assert ((got - want).abs() <= step * (1 + 2.0 ** -20) + 2 * tol + 2.0 ** -21 * want.abs()).all()


APPENDS = [  # rows, start, page, Hq, Hkv, D, pairs, adjacent, axes
    ([1], [0], 16, 1, 1, 16, 8, False, 1),
    ([1, 1, 1], [0, 15, 16], 16, 6, 2, 64, 32, True, 1),
    ([0, 5, 0, 3, 1, 0], [7, 0, 3, 30, 31, 5], 32, 3, 3, 80, 40, False, 3),
    ([6, 2, 4, 1], [100, 64, 63, 1], 48, 32, 8, 128, 64, False, 1),
    ([300, 1, 260], [5, 0, 1000], 64, 5, 5, 96, 12, True, 2),
    ([9] * 70, list(range(70)), 16, 0, 4, 48, 24, False, 1),
    ([1500, 1400], [17, 0], 128, 2, 1, 128, 64, False, 3),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("rows,start,page,Hq,Hkv,D,pairs,adjacent,axes", APPENDS)
def test_append(rows, start, page, Hq, Hkv, D, pairs, adjacent, axes, fmt, dtype):
    gen = torch.Generator().manual_seed(sum(rows) + D)
    cache, table, row0, start = _setup(gen, rows, start, page, Hkv, D, fmt)
    R = sum(rows)
    freq = plain_rotary.frequencies(pairs)
    axis = None if axes == 1 else torch.randint(axes, (pairs,), generator=gen)
    if axis is not None:
        axis[-1] = axes - 1
    qkv = torch.randn((R, Hq + 2 * Hkv, D), generator=gen)
    qkv = (qkv * 2.0 ** torch.randint(-9, 8, (R, Hq + 2 * Hkv, 1), generator=gen).float()).to(dtype).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    z = binding.Rotary(freq, axis=None if axis is None else axis.tolist(), adjacent=adjacent)
    dev = [t.cuda() for t in (table, start, row0)]
    pg, off, pos = _places(table, row0, start, page)
    offset = 1000003
    if axes > 1:
        at, kw = _positions(gen, axes, R), {}
        kw = dict(positions=at.cuda())
    else:
        at, kw = (pos + offset)[None], dict(offset=offset)
    got = binding.kv_append_rotary(k, v, cache, *dev, z, q=q if Hq else None, **kw)
    want, tol = plain_rotary.turn(k.cpu(), at, freq, axis, adjacent)
    _check_keys(cache.k, cache.k_scale, pg, off, want, tol, fmt)
    # the values as the plain append stores them, and nothing else written
    other = binding.KVCache.empty(cache.n_pages, Hkv, page, D, dtype=fmt)
    binding.kv_append(k, v, other, *dev)
    assert torch.equal(other.v.view(torch.uint8), cache.v.view(torch.uint8)) and torch.equal(other.v_scale, cache.v_scale)
    assert torch.equal(other.k_scale == 0, cache.k_scale == 0)
    if Hq:
        want, tol = plain_rotary.turn(q.cpu(), at, freq, axis, adjacent)
        assert ((got.cpu().double() - want).abs() <= _rounded(want, tol, dtype)).all()
        inplace = binding.kv_append_rotary(k, v, other, *dev, z, q=q, out=q, **kw)
        assert inplace is q and torch.equal(q, got)
        assert torch.equal(other.k.view(torch.uint8), cache.k.view(torch.uint8)) and torch.equal(other.k_scale, cache.k_scale)
    else:
        assert got is None
    assert binding.read_device_flags(cache.flags) == 0


def test_positions_of_zero_store_what_the_plain_append_stores():
    gen = torch.Generator().manual_seed(2)
    cache, table, row0, start = _setup(gen, [50, 3], [0, 9], 32, 4, 64, E4M3)
    k, v = (torch.randn((53, 4, 64), generator=gen).bfloat16().cuda() for _ in range(2))
    dev = [t.cuda() for t in (table, start, row0)]
    z = binding.Rotary(plain_rotary.frequencies(32))
    binding.kv_append_rotary(k, v, cache, *dev, z, positions=torch.zeros(53, dtype=torch.int32, device="cuda"))
    other = binding.KVCache.empty(cache.n_pages, 4, 32, 64)
    binding.kv_append(k, v, other, *dev)
    for a, b in ((cache.k, other.k), (cache.v, other.v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(cache.k_scale, other.k_scale)


def test_rows_of_no_request_bad_pages_and_numbers():
    gen = torch.Generator().manual_seed(3)
    cache, table, row0, start = _setup(gen, [2, 3, 2], [0, 14, 0], 16, 2, 64, INT8)
    table[1, 1] = cache.n_pages               # positions 16 of request 1: no page
    start[2] = -1
    n = 7 + 4                                 # four rows behind the last request
    q, k, v = (torch.randn((n, 2, 64), generator=gen).half() for _ in range(3))
    k[1, 1, 5] = math.inf
    v[0, 0, 3] = math.nan
    out = torch.full_like(q, 7.0).cuda()
    z = binding.Rotary(plain_rotary.frequencies(32))
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    binding.kv_append_rotary(k.cuda(), v.cuda(), cache, table.cuda(), start.cuda(), row0.cuda(), z, q=q.cuda(), out=out)
    assert (out[7:] == 7).all() and not (out[:7] == 7).all(-1).any()
    assert binding.read_device_flags(cache.flags) == (binding.FLAG_BAD_PAGE | binding.FLAG_BAD_LENGTH | binding.FLAG_NONFINITE)
    page = int(table[0, 0])
    assert cache.k_scale[page, 1, 1].isnan() and not cache.k[page, 1, 1].any()
    assert cache.v_scale[page, 0, 0].isnan() and not cache.v[page, 0, 0].any()
    assert not cache.k_scale[page, 0].isnan().any()
    # only requests 0 and the first two rows of 1 are written
    changed = [(a != b).flatten(3).any(-1) if a.dim() == 4 else (a != b) for a, b in zip((cache.k, cache.v), before)]
    held = torch.zeros(changed[0].shape, dtype=torch.bool)
    held[page, :, :2] = True
    held[int(table[1, 0]), :, 14:] = True
    for c in changed:
        assert not (c.cpu() & ~held).any()


def test_a_side_stream_and_a_captured_graph():
    gen = torch.Generator().manual_seed(4)
    cache, table, row0, start = _setup(gen, [5] * 9, [3] * 9, 16, 2, 128, E4M3)
    q, k, v = (torch.randn((45, h, 128), generator=gen).bfloat16().cuda() for h in (4, 2, 2))
    z = binding.Rotary(plain_rotary.frequencies(64))
    dev = [t.cuda() for t in (table, start, row0)]
    want = binding.kv_append_rotary(k, v, cache, *dev, z, q=q)
    pos = torch.arange(45, dtype=torch.int32, device="cuda")
    want_rows = binding.rotary(q, z, pos)
    kept = cache.k.view(torch.uint8).clone()
    side = torch.cuda.Stream()
    cache.k.view(torch.uint8).zero_()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.kv_append_rotary(k, v, cache, *dev, z, q=q, stream=side)
    rows = binding.rotary(q, z, pos, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(rows, want_rows) and torch.equal(cache.k.view(torch.uint8), kept)
    cache.k.view(torch.uint8).zero_()
    graph, out, rows = torch.cuda.CUDAGraph(), torch.zeros_like(q), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        binding.kv_append_rotary(k, v, cache, *dev, z, q=q, out=out)
        binding.rotary(q, z, pos, out=rows)
    q.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want * 2) and torch.equal(rows, want_rows * 2) and torch.equal(cache.k.view(torch.uint8), kept)
