"""dspark_window_attention of blocks with many rows, whose kernels meet in a
workspace, against its formula in 64 bits (the bounds are plain_window's)."""
import math

import pytest
import torch

import plain_cache
import plain_window
from speculative_decoding_draft_head_gb300 import binding
from test_gpu_window_attention import BF16, E4M3, F16, INT8, _check, _run

pytestmark = pytest.mark.gpu


def _run_blocks(rows, ctx, prefix, Hq, Hkv, D, page, window, sinks, **kw):
    """_run with a workspace of the test's own, which the kernels for many rows write to."""
    n = binding.window_workspace_bytes(len(rows), sum(rows), Hq, Hkv, D)
    assert n > 0
    buf = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    buf = buf[(-buf.data_ptr()) % 256:][:n]
    got = _run(rows, ctx, prefix, Hq, Hkv, D, page, window, sinks, workspace=buf, **kw)
    assert bool(buf.any()), "these sizes go another way: the case says nothing"
    return got


# rows, ctx, prefix, Hq, Hkv, D, page, window, sinks
SHAPES = {
    "long and short": ([700, 1, 90, 260], [10, 500, 300, 0], 205, 64, 2, 128, 64, 150, 30),
    "longer than the window": ([1300, 900], [700, 2000], 0, 16, 2, 64, 48, 129, 1),
    "wide heads, no first tokens": ([300, 280], [1000, 140], 90, 96, 1, 96, 16, 333, 0),
    "a window of everything": ([500, 130], [300, 900], 140, 48, 4, 128, 32, 10 ** 9, 0),
    "first tokens past the window": ([600, 300], [100, 5], 77, 64, 4, 64, 16, 20, 700),
    "first tokens past everything": ([400, 500], [100, 5], 30, 64, 4, 64, 16, 7, 10 ** 9),
    "first tokens of the prefix and behind it": ([500, 600], [900, 0], 33, 40, 2, 80, 48, 250, 60),
    "a window into a long prefix": ([200, 300, 100], [30, 0, 400], 3000, 48, 2, 128, 64, 1111, 133),
    "a prefix that no window reaches": ([200, 300, 100], [1500, 1400, 2000], 500, 48, 2, 128, 128, 1111, 20),
    "neither": ([300, 400], [1500, 1600], 500, 40, 2, 128, 128, 900, 0),
    "requests without rows": ([0, 700, 0, 300, 0], [5, 300, 0, 0, 800], 64, 48, 2, 64, 16, 400, 16),
    "windows at a tile's ends": ([513, 511], [1280, 1151], 0, 40, 4, 64, 64, 128, 128),
    "row tiles of odd groups": ([333, 222], [1001, 77], 19, 75, 3, 48, 16, 499, 17),
    "a window of one": ([1100, 1300], [40, 0], 0, 40, 2, 64, 16, 1, 3),
}


@pytest.mark.parametrize("fmt,dtype", [(E4M3, BF16), (INT8, F16)])
@pytest.mark.parametrize("name", SHAPES)
def test_shapes(name, fmt, dtype):
    _run_blocks(*SHAPES[name], fmt=fmt, dtype=dtype)


@pytest.mark.parametrize("name", ["long and short", "longer than the window", "a window into a long prefix",
                                  "first tokens past everything", "windows at a tile's ends"])
def test_full_block(name):
    _run_blocks(*SHAPES[name], mask="full")


@pytest.mark.parametrize("ctx,prefix,window,sinks", [(0, 0, 64, 0), (5, 20, 64, 9), (700, 130, 100, 150), (300, 0, 64, 0),
                                                     (90, 300, 200, 40), (200, 900, 500, 0)])
def test_trees(ctx, prefix, window, sinks):
    gen = torch.Generator().manual_seed(ctx)
    rows = [50, 9, 64, 33] * 20
    words = torch.randint(-2 ** 63, 2 ** 63 - 1, (sum(rows),), generator=gen)
    words[0], words[50] = 0, -1
    words[::7] &= 3
    got, *_ = _run_blocks(rows, [ctx + 13 * (b % 5) for b in range(len(rows))], prefix, 40, 2, 64, 16, window, sinks, mask="full",
                          words=words)
    if ctx == 0 and prefix == 0:
        assert bool((got["out"][0] == 0).all()) and bool((got["lse"][0] == -math.inf).all())


@pytest.mark.parametrize("q_size,kw", [
    (30.0, {}),
    (1e30, dict(k_scale=1e-30)),
    (1.0, dict(v_scale=1e-30)),
    (4.0, dict(token_scale=lambda gen, s: 2.0 ** torch.randint(-3, 3, s, generator=gen).float())),
], ids=["sharp", "large q", "small v", "uneven and sharp"])
def test_ranges(q_size, kw):
    _run_blocks([300, 200], [700, 300], 400, 80, 4, 128, 64, 500, 6, q_size=q_size, pool_kw=kw)


def _setting(rows, ctx, prefix, Hq, Hkv, D, page, seed=3):
    gen = torch.Generator().manual_seed(seed)
    lens = [c + n for c, n in zip(ctx, rows)]
    pool = plain_cache.Pool(gen, lens, prefix, Hkv, D, page, E4M3)
    q = torch.randn((sum(rows), Hq, D), generator=gen).to(BF16)
    return pool, q, torch.tensor([0] + rows).cumsum(0), lens


def test_tokens_stored_as_no_number():
    pool, q, row0, lens = _setting([600, 500], [200, 90], 0, 48, 2, 64, 16)
    window, sinks = 400, 40
    # tokens of both windows' reach, a first one, and one that no row sees
    for b, t, scales in ((0, 300, pool.k_scale), (0, 700, pool.v_scale), (1, 39, pool.v_scale)):
        scales[int(pool.table[b, t // 16]), 1, t % 16] = math.nan
    got = binding.window_attention(q.cuda(), pool.cache(binding), pool.table.cuda(), torch.tensor(lens).int().cuda(),
                                   row0.cuda(), window=window, sinks=sinks)
    want = plain_window.attention(q, pool, row0, lens, window, sinks)
    assert want[0][:600, 24:].isnan().any() and not want[0][:600, 24:].isnan().all() and want[0][600:, 24:].isnan().all()
    assert not want[0][:, :24].isnan().any()
    _check(got, want, allow_nan=True)


def test_bad_lengths_and_pages():
    pool, q, row0, lens = _setting([400, 300, 200, 350], [60, 50, 40, 33], 20, 64, 2, 64, 16)
    kv_len = torch.tensor(lens).int()
    kv_len[1] = 299                                   # shorter than its block
    kv_len[2] = pool.table.shape[1] * 16 + 1          # beyond its pages
    table = pool.table.clone()
    table[0, 4] = pool.k.shape[0]                     # own tokens 64 .. 79: rows 4 .. and later see them
    cache = pool.cache(binding)
    got = binding.window_attention(q.cuda(), cache, table.cuda(), kv_len.cuda(), row0.cuda(), window=100, sinks=22,
                                   prefix_pages=pool.prefix_pages.cuda(), prefix_len=20)
    torch.cuda.synchronize()
    assert binding.read_device_flags(cache.flags) == binding.FLAG_BAD_LENGTH | binding.FLAG_BAD_PAGE
    assert got["out"][400:900].isnan().all() and got["lse"][400:900].isnan().all()
    want = plain_window.attention(q, pool, row0, lens, 100, 22)
    # own token t is seen by rows t - 60 .. t + 39 of request 0: 64 .. 79 by rows 4 .. 118
    for part in (slice(0, 4), slice(119, 400), slice(900, 1250)):
        _check({k: t[part] for k, t in got.items()}, [t[part] for t in want])
    assert got["out"][4:119].isnan().all()


@pytest.mark.parametrize("prefix", [0, 50])
def test_bad_requests_without_and_with_a_prefix_are_nan(prefix):
    pool, q, row0, lens = _setting([400, 300, 200], [60, 50, 40], prefix, 64, 2, 64, 16)
    kv_len = torch.tensor(lens).int()
    kv_len[1] = -7
    cache = pool.cache(binding)
    got = binding.window_attention(q.cuda(), cache, pool.table.cuda(), kv_len.cuda(), row0.cuda(), window=300,
                                   prefix_pages=pool.prefix_pages.cuda() if prefix else None, prefix_len=prefix)
    torch.cuda.synchronize()
    assert binding.read_device_flags(cache.flags) == binding.FLAG_BAD_LENGTH
    assert got["out"][400:700].isnan().all() and got["lse"][400:700].isnan().all()
    want = plain_window.attention(q, pool, row0, lens, 300, 0)
    for part in (slice(0, 400), slice(700, 900)):
        _check({k: t[part] for k, t in got.items()}, [t[part] for t in want])


def test_rows_of_no_request_and_strided_queries():
    pool, q, row0, lens = _setting([400, 500], [20, 30], 40, 64, 2, 64, 16)
    wide = torch.full((909, 70, 64), math.nan, dtype=BF16)
    wide[:900, 3:67] = q
    out = dict(out=torch.full((909, 64, 64), 7.0, dtype=BF16, device="cuda"), lse=torch.full((909, 64), 7.0, device="cuda"))
    binding.window_attention(wide.cuda()[:, 3:67], pool.cache(binding), pool.table.cuda(), torch.tensor(lens).int().cuda(),
                             row0.cuda(), window=300, sinks=3, prefix_pages=pool.prefix_pages.cuda(), prefix_len=40, out=out)
    assert bool((out["out"][900:] == 7).all()) and bool((out["lse"][900:] == 7).all())
    _check({k: t[:900] for k, t in out.items()}, plain_window.attention(q, pool, row0, lens, 300, 3))


def test_streams_graphs_and_two_calls_at_once():
    """Each stream has a workspace of its own, a captured graph one of the graph's; the bits are the same everywhere."""
    pool, q, row0, lens = _setting([500, 300, 200], [700, 20, 90], 50, 48, 2, 128, 64)
    cache, args = pool.cache(binding), (pool.table.cuda(), torch.tensor(lens).int().cuda(), row0.cuda())
    kw = dict(window=600, sinks=4, prefix_pages=pool.prefix_pages.cuda(), prefix_len=50)
    qs = [q.cuda(), (q * 2).cuda()]
    want = [binding.window_attention(x, cache, *args, **kw) for x in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, kept = [], []
    for x in qs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            kept.append(binding.window_attention(x, cache, *args, **kw))
    for _ in range(3):
        outs = []
        for x, s, graph in zip(qs, streams, graphs):
            outs.append(binding.window_attention(x, cache, *args, stream=s, **kw))
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for a, b, k in zip(outs, want, kept):
            for name in ("out", "lse"):
                assert torch.equal(a[name], b[name]) and torch.equal(k[name], b[name])
