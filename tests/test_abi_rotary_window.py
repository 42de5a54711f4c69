"""The rotary and window entry points reject bad host-side arguments before any
launch, and the binding passes on what it is given (no compute calls here)."""
import ctypes
import types

import pytest
import torch

from speculative_decoding_draft_head_gb300 import binding

P = 1 << 20


def _cache(**over):
    f = dict(k=P, v=P, k_scale=P, v_scale=P, flags=P, n_pages=8, n_kv_heads=2, page_size=32, head_dim=64, format=0)
    f.update(over)
    return binding._CacheStruct(*[f[n] for n, _ in binding._CacheStruct._fields_])


def _rotary(**over):
    f = dict(step=P, axis=None, n_pairs=32, n_axes=1, adjacent=0)
    f.update(over)
    return binding._RotaryStruct(*[f[n] for n, _ in binding._RotaryStruct._fields_])


def _err():
    return binding.load().dspark_last_error().decode()


FAR = P << 8


def _rows(z=None, x=P, rs=256, hs=64, n=4, heads=4, d=64, dt=0, pos=P, inverse=0, out=FAR, ors=256, ohs=64):
    return binding.load().dspark_rotary_rows(_rotary() if z is None else z, x, rs, hs, n, heads, d, dt, pos, inverse, out, ors,
                                             ohs, None)


def _append(cache=None, z=None, q=P, qs=256, hq=4, k=2 * P, v=3 * P, ks=128, vs=128, dt=0, row0=P, n=4, start=P, table=P,
            max_pages=4, B=2, pos=None, offset=0, qo=FAR, qos=256):
    return binding.load().dspark_kv_append_rotary(_cache() if cache is None else cache, _rotary() if z is None else z, q, qs, hq,
                                                  k, v, ks, vs, dt, row0, n, start, table, max_pages, B, pos, offset, qo, qos,
                                                  None)


def _attend(cache=None, q=P, qs=256, dt=0, Hq=4, row0=P, n=4, B=2, table=P, max_pages=4, lens=P, pp=None, npp=0, plen=0,
            window=64, sinks=0, mask=0, words=None, scale=0.125, out=FAR, lse=None, ws=None, wsb=0):
    return binding.load().dspark_window_attention(_cache() if cache is None else cache, q, qs, dt, Hq, row0, n, B, table,
                                                  max_pages, lens, pp, npp, plen, window, sinks, mask, words, scale, out, lse,
                                                  ws, wsb, None)


@pytest.mark.parametrize("call", [_append, _attend])
@pytest.mark.parametrize("over,status,needle", [
    (dict(k=None), 1, "pointer of the cache"),
    (dict(v=P + 8), 1, "aligned"),
    (dict(page_size=24), 1, "page_size"),
    (dict(head_dim=40), 1, "head_dim"),
    (dict(head_dim=144), 2, "head_dim"),
    (dict(format=2), 1, "format"),
])
def test_a_bad_cache(call, over, status, needle):
    assert call(cache=_cache(**over)) == status and needle in _err()


@pytest.mark.parametrize("call", [_append, _attend])
@pytest.mark.parametrize("over,needle", [
    (dict(B=0), "B must be"),
    (dict(n=-1), "n_rows"),
    (dict(max_pages=0), "max_pages"),
    (dict(max_pages=1 << 27), "2^31"),
    (dict(row0=None), "NULL"),
    (dict(table=None), "NULL"),
    (dict(dt=7), "unknown dtype"),
])
def test_bad_rows(call, over, needle):
    assert call(**over) == 1 and needle in _err()


@pytest.mark.parametrize("call", [_rows, _append, _attend])
def test_no_rows_is_no_work(call):
    assert call(n=0) == 0


@pytest.mark.parametrize("call", [_rows, _append])
@pytest.mark.parametrize("over,needle", [
    (dict(step=None), "steps"),
    (dict(step=P + 8), "aligned"),
    (dict(axis=P + 2), "aligned"),
    (dict(n_pairs=0), "n_pairs"),
    (dict(n_pairs=6), "n_pairs"),
    (dict(n_pairs=36), "n_pairs"),
    (dict(n_axes=0), "n_axes"),
    (dict(n_axes=2), "n_axes"),
    (dict(adjacent=2), "adjacent"),
])
def test_a_bad_rotary(call, over, needle):
    assert call(z=_rotary(**over)) == 1 and needle in _err()


def test_a_missing_rotary():
    assert binding.load().dspark_rotary_rows(None, P, 256, 64, 4, 4, 64, 0, P, 0, FAR, 256, 64, None) == 1
    assert "rotary is NULL" in _err()


@pytest.mark.parametrize("over,status,needle", [
    (dict(d=60), 1, "multiple of 8"),
    (dict(d=264), 2, "at most 256"),
    (dict(n=-1), 1, "n_rows"),
    (dict(heads=0), 1, "n_heads"),
    (dict(heads=1 << 17, rs=1 << 24, ors=1 << 24), 2, "n_heads"),
    (dict(dt=3), 1, "dtype"),
    (dict(inverse=2), 1, "inverse"),
    (dict(x=None), 1, "NULL"),
    (dict(out=None), 1, "NULL"),
    (dict(pos=None), 1, "NULL"),
    (dict(x=P + 8), 1, "aligned"),
    (dict(out=FAR + 4), 1, "aligned"),
    (dict(pos=P + 2), 1, "aligned"),
    (dict(hs=0), 1, "strides"),               # a broadcast head
    (dict(rs=0), 1, "strides"),
    (dict(rs=255), 1, "strides"),
    (dict(rs=252, hs=60), 1, "strides"),
    (dict(ohs=68), 1, "strides"),
    (dict(rs=100, hs=200), 1, "strides"),     # rows inside heads, but not all of them
    (dict(out=P + 16), 1, "overlap"),
    (dict(out=P + 3 * 512), 1, "overlap"),
    (dict(out=P, ors=512), 1, "overlap"),     # the same place with other strides
])
def test_rows_rejects(over, status, needle):
    assert _rows(**over) == status and needle in _err(), _err()


@pytest.mark.parametrize("over,status,needle", [
    (dict(k=None), 1, "NULL"),
    (dict(v=3 * P + 2), 1, "aligned"),
    (dict(ks=127), 1, "strides"),
    (dict(vs=132), 1, "strides"),
    (dict(start=None), 1, "NULL"),
    (dict(pos=P, offset=3), 1, "offset"),
    (dict(pos=P + 2), 1, "aligned"),
    (dict(hq=0), 1, "n_q_heads"),
    (dict(hq=(1 << 16) + 1), 2, "heads"),
    (dict(qo=None), 1, "q_out is NULL"),
    (dict(q=P + 8), 1, "aligned"),
    (dict(qs=255), 1, "strides"),
    (dict(qos=252), 1, "strides"),
    (dict(qo=P + 512), 1, "overlap"),
    (dict(qo=P, qos=512), 1, "overlap"),
    (dict(qo=2 * P), 1, "overlap"),
    (dict(qo=3 * P - 1024), 1, "overlap"),
])
def test_append_rejects(over, status, needle):
    assert _append(**over) == status and needle in _err(), _err()


@pytest.mark.parametrize("call", [_rows, _append])
@pytest.mark.parametrize("n", [(1 << 30) + 1, (1 << 31) - 1])
def test_more_rows_than_the_kernels_count(call, n):
    """Rounded up to what a block takes, numbers of rows near 2^31 would wrap."""
    assert call(n=n) == 2 and "n_rows must be at most 2^30" in _err(), _err()


@pytest.mark.parametrize("over,status,needle", [
    (dict(dt=1), 2, "bf16 or fp16"),
    (dict(Hq=3), 1, "multiple of n_kv_heads"),
    (dict(n=1 << 29, Hq=4), 2, "2^30"),
    (dict(plen=-1), 1, "prefix_len"),
    (dict(pp=P, npp=1, plen=33), 1, "does not fit"),
    (dict(npp=2, plen=33), 1, "prefix_pages is NULL"),
    (dict(mask=2), 1, "mask"),
    (dict(scale=0.0), 1, "scale"),
    (dict(q=None), 1, "NULL"),
    (dict(out=None), 1, "NULL"),
    (dict(q=P + 8), 1, "aligned"),
    (dict(qs=255), 1, "q_stride"),
    (dict(out=P + 16), 1, "overlap"),
    (dict(window=0), 1, "window"),
    (dict(window=-5), 1, "window"),
    (dict(sinks=-1), 1, "sinks"),
    (dict(words=P, window=63), 1, "64"),
    (dict(pp=P, npp=1 << 26, plen=(1 << 31) - 1 - 128, max_pages=4), 1, "2^31 - 256"),
    (dict(n=200), 1, "workspace is NULL"),    # 100 rows of 2 query heads a kv head
    (dict(n=200, ws=P + 16, wsb=1 << 30), 1, "256-byte"),
    (dict(n=200, ws=P, wsb=16), 1, "too small"),
])
def test_window_rejects(over, status, needle):
    assert _attend(**over) == status and needle in _err(), _err()


def test_workspace_sizes():
    f = binding.window_workspace_bytes
    assert f(64, 64, 32, 8, 128) == 0 and f(64, 384, 32, 8, 128) == 0      # decoding, drafted blocks: none
    assert f(2, 256, 32, 8, 128) >= binding.attention_workspace_bytes(2, 256, 32, 8, 128)
    for bad in ((0, 8, 8, 2, 64), (4, -1, 8, 2, 64), (4, 8, 7, 2, 64), (4, 8, 8, 2, 40)):
        assert f(*bad) == 0


def test_the_struct_matches_the_header():
    assert ctypes.sizeof(binding._RotaryStruct) == 2 * 8 + 3 * 4 + 4


# ------------------------------------------------------------------------------------------------ the binding
def test_a_handle_checks_its_frequencies():
    assert binding.Rotary([1.0, 0.5, 0.25, 0.125], device="cpu").n_pairs == 4
    for bad in ([], [1.0] * 3, [1.0] * 6):
        with pytest.raises(ValueError, match="multiple of 4"):
            binding.Rotary(bad, device="cpu")
    with pytest.raises(ValueError, match="finite"):
        binding.Rotary([1.0, float("nan"), 1.0, 1.0], device="cpu")
    for axis in ([0, 1], [0, 1, 2, -1], [0, 1, 2, 16]):
        with pytest.raises(ValueError, match="axis"):
            binding.Rotary([1.0] * 4, axis=axis, device="cpu")
    assert binding.Rotary([1.0] * 4, axis=[0, 2, 0, 1], device="cpu").n_axes == 3


def test_steps_are_turns_in_64_bits():
    import math
    z = binding.Rotary([0.0, 2 * math.pi, 1.0, -1.0], device="cpu")
    steps = [int(t) % 2 ** 64 for t in z.step]
    # 2 pi in 64 bits is off by 2.4e-16, 7e2 steps of 2^-64 turns
    assert steps[0] == 0 and min(steps[1], 2 ** 64 - steps[1]) < 1000
    assert abs(steps[2] - 2 ** 64 / (2 * math.pi)) < 2 ** 12 and steps[2] + steps[3] == 2 ** 64


class _Library:
    """Takes the calls' arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def setting(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(binding, "_lib", lib)
    monkeypatch.setattr(binding, "_default_ws", binding.WorkspaceCache())
    monkeypatch.setattr(binding, "window_workspace_bytes", lambda B, n, *sizes: 1024 if n > 4 else 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 5, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    cache = object.__new__(binding.KVCache)
    cache._index, cache.device, cache._ref = -1, torch.device("cpu"), None
    cache.n_pages, cache.n_kv_heads, cache.page_size, cache.head_dim = 4, 2, 16, 64
    return lib, cache, binding.Rotary([1.0] * 32, device="cpu")


TABLE, LENS = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)


def test_windows_wider_than_any_cache_are_all_of_it(setting):
    lib, cache, _ = setting
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    binding.window_attention(q, cache, TABLE, LENS, torch.tensor([0, 3]), window=10 ** 15, sinks=2 ** 40)
    name, args = lib.calls[-1]
    assert name == "dspark_window_attention" and args[14:16] == (0x7fffffff, 0x7fffffff) and args[-3:-1] == (None, 0)
    binding.window_attention(q, cache, TABLE, LENS, torch.tensor([0, 3]), window=-10 ** 15)
    assert lib.calls[-1][1][14] < 1


def test_a_workspace_only_where_one_is_needed(setting):
    lib, cache, _ = setting
    q = torch.zeros((9, 4, 64), dtype=torch.bfloat16)
    for _ in range(2):
        binding.window_attention(q, cache, TABLE, LENS, torch.tensor([0, 9]), window=8)
    a, b = (c[1][-3:-1] for c in lib.calls[-2:])
    assert a == b and a[0] and a[0] % 256 == 0 and a[1] >= 1024


def test_numbers_past_32_bits(setting):
    _, cache, z = setting
    rows = torch.empty((2 ** 32 + 3, 2, 64), dtype=torch.float16, device="meta")
    with pytest.raises(ValueError, match="2.31"):
        binding.window_attention(rows, cache, TABLE, LENS, torch.tensor([0, 3]), window=5)
    with pytest.raises(ValueError, match="2.31"):
        binding.kv_append_rotary(rows, rows, cache, TABLE, LENS, torch.tensor([0, 3]), z)
    k = torch.zeros((3, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="offset"):
        binding.kv_append_rotary(k, k, cache, TABLE, LENS, torch.tensor([0, 3]), z, offset=2 ** 63)
    with pytest.raises(ValueError, match="2.31"):
        binding.window_attention(k, cache, TABLE, LENS, torch.tensor([0, 3]), window=5, prefix_len=2 ** 32 + 3)


def test_queries_positions_and_outputs_have_to_fit(setting):
    lib, cache, z = setting
    row0 = torch.tensor([0, 3])
    k, q = torch.zeros((3, 2, 64), dtype=torch.float16), torch.zeros((3, 4, 64), dtype=torch.float16)
    call = lambda **kw: binding.kv_append_rotary(k, k, cache, TABLE, LENS, row0, z, **kw)  # noqa: E731
    assert call() is None and call(q=q).shape == q.shape and call(q=q, out=q) is q
    with pytest.raises(ValueError, match="q is required"):
        call(out=q)
    with pytest.raises(TypeError, match="type and the rows"):
        call(q=q.float())
    with pytest.raises(TypeError, match="type and the rows"):
        call(q=q[:2])
    with pytest.raises(ValueError, match="shape and type"):
        call(q=q, out=q.float())
    for bad in (torch.zeros(2, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)):
        with pytest.raises(ValueError):
            call(positions=bad)
    with pytest.raises((TypeError, ValueError)):
        call(positions=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="shape and type"):
        binding.rotary(q, z, torch.zeros(3, dtype=torch.int32), out=q[:2])
    with pytest.raises(ValueError, match="contiguous"):
        binding.rotary(torch.zeros((3, 64, 4)).transpose(1, 2), z, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="bf16, fp16 and fp32|bf16, fp16 or fp32"):
        binding.rotary(q.double(), z, torch.zeros(3, dtype=torch.int32))


def test_another_device_or_stream_is_refused(setting, monkeypatch):
    lib, cache, z = setting
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    row0, pos = torch.tensor([0, 3]), torch.zeros(3, dtype=torch.int32)
    calls = [lambda **kw: binding.window_attention(k, cache, TABLE, LENS, row0, window=4, **kw),
             lambda **kw: binding.kv_append_rotary(k, k, cache, TABLE, LENS, row0, z, **kw),
             lambda **kw: binding.rotary(k, z, pos, **kw)]
    for call in calls:
        with pytest.raises(ValueError, match="stream is of cuda:3"):
            call(stream=types.SimpleNamespace(device_index=3, cuda_stream=5))
    other = binding.Rotary([1.0] * 32, device="cpu")
    other._index = 1
    with pytest.raises(ValueError, match="rotary must be on"):
        binding.kv_append_rotary(k, k, cache, TABLE, LENS, row0, other)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    for call in calls:
        with pytest.raises(ValueError, match="not the current device"):
            call()
    assert not lib.calls
