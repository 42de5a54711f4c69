"""The cache and attention entry points reject bad host-side arguments before
any launch (no compute calls here)."""
import ctypes

import pytest
import torch

from speculative_decoding_draft_head_gb300 import binding

P = 1 << 12


def _struct(**over):
    f = dict(k=P, v=P, k_scale=P, v_scale=P, flags=P, n_pages=8, n_kv_heads=2, page_size=32, head_dim=64, format=0)
    f.update(over)
    return binding._CacheStruct(*[f[n] for n, _ in binding._CacheStruct._fields_])


def _err():
    return binding.load().dspark_last_error().decode()


BAD_CACHES = [
    (dict(k=None), 1, "pointer of the cache"),
    (dict(flags=None), 1, "pointer of the cache"),
    (dict(v=P + 8), 1, "aligned"),
    (dict(k_scale=P + 4), 1, "aligned"),
    (dict(n_pages=0), 1, "n_pages"),
    (dict(n_kv_heads=0), 1, "n_kv_heads"),
    (dict(page_size=24), 1, "page_size"),
    (dict(page_size=0), 1, "page_size"),
    (dict(head_dim=40), 1, "head_dim"),
    (dict(head_dim=144), 2, "head_dim"),
    (dict(format=2), 1, "format"),
]


def _append(cache=None, k=P, v=P, ks=128, vs=128, dt=0, row0=P, n=4, start=P, table=P, max_pages=4, B=2):
    c = _struct() if cache is None else cache
    return binding.load().dspark_kv_append(c, k, v, ks, vs, dt, row0, n, start, table, max_pages, B, None)


def _read(cache=None, row0=P, n=4, start=P, table=P, max_pages=4, B=2, dt=0, ko=P, vo=P):
    c = _struct() if cache is None else cache
    return binding.load().dspark_kv_read(c, row0, n, start, table, max_pages, B, dt, ko, vo, None)


def _attend(cache=None, q=P, qs=256, dt=0, Hq=4, row0=P, n=4, B=2, table=P, max_pages=4, lens=P, pp=None, npp=0, plen=0,
            mask=0, words=None, scale=0.125, out=P, lse=None, ws=P, wsb=1 << 30):
    c = _struct() if cache is None else cache
    return binding.load().dspark_block_attention(c, q, qs, dt, Hq, row0, n, B, table, max_pages, lens, pp, npp, plen,
                                                 mask, words, scale, out, lse, ws, wsb, None)


@pytest.mark.parametrize("call", [_append, _read, _attend])
@pytest.mark.parametrize("over,status,needle", BAD_CACHES)
def test_every_call_rejects_a_bad_cache(call, over, status, needle):
    assert call(cache=_struct(**over)) == status and needle in _err()


@pytest.mark.parametrize("call", [_append, _read, _attend])
@pytest.mark.parametrize("over,needle", [
    (dict(B=0), "B must be"),
    (dict(n=-1), "n_rows"),
    (dict(max_pages=0), "max_pages"),
    (dict(max_pages=1 << 27), "2^31"),
    (dict(row0=None), "NULL"),
    (dict(table=None), "NULL"),
    (dict(dt=7), "unknown dtype"),
])
def test_every_call_rejects_bad_rows(call, over, needle):
    assert call(**over) == 1 and needle in _err()


@pytest.mark.parametrize("call", [_append, _read, _attend])
def test_no_rows_is_no_work(call):
    assert call(n=0) == 0


def test_a_missing_cache_is_rejected():
    assert binding.load().dspark_kv_append(None, P, P, 128, 128, 0, P, 4, P, P, 4, 2, None) == 1
    assert "cache is NULL" in _err()


@pytest.mark.parametrize("over,needle", [
    (dict(k=None), "NULL"),
    (dict(v=P + 2), "aligned"),
    (dict(ks=127), "strides"),
    (dict(vs=132), "strides"),          # 264 bytes
    (dict(start=None), "NULL"),
])
def test_append_rejects(over, needle):
    assert _append(**over) == 1 and needle in _err()


@pytest.mark.parametrize("over,needle", [
    (dict(ko=None, vo=None), "both NULL"),
    (dict(vo=P + 8), "aligned"),
])
def test_read_rejects(over, needle):
    assert _read(**over) == 1 and needle in _err()


@pytest.mark.parametrize("over,status,needle", [
    (dict(dt=1), 2, "bf16 or fp16"),
    (dict(Hq=3), 1, "multiple of n_kv_heads"),
    (dict(Hq=0), 1, "multiple of n_kv_heads"),
    (dict(n=1 << 29, Hq=4), 2, "2^30"),
    (dict(plen=-1), 1, "prefix_len"),
    (dict(pp=P, npp=1, plen=33), 1, "does not fit"),
    (dict(npp=2, plen=33), 1, "prefix_pages is NULL"),
    (dict(mask=2), 1, "mask"),
    (dict(scale=0.0), 1, "scale"),
    (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"),
    (dict(q=None), 1, "NULL"),
    (dict(lens=None), 1, "NULL"),
    (dict(out=None), 1, "NULL"),
    (dict(q=P + 8), 1, "aligned"),
    (dict(qs=255), 1, "q_stride"),
    (dict(ws=None), 1, "workspace is NULL"),
    (dict(ws=P + 16), 1, "256-byte"),
    (dict(wsb=16), 1, "too small"),
])
def test_attention_rejects(over, status, needle):
    assert _attend(**over) == status and needle in _err(), _err()


def test_attention_workspace_sizes():
    f = binding.attention_workspace_bytes
    assert f(4, 8, 8, 2, 64) >= 256
    assert f(4, 16, 8, 2, 64) >= f(4, 8, 8, 2, 64)
    for bad in ((0, 8, 8, 2, 64), (4, -1, 8, 2, 64), (4, 8, 7, 2, 64), (4, 8, 8, 0, 64), (4, 8, 8, 2, 40),
                (4, 8, 8, 2, 256)):
        assert f(*bad) == 0


def test_binding_checks_tensors_before_the_call():
    codes = torch.zeros((2, 1, 16, 16), dtype=torch.uint8)
    with pytest.raises(TypeError):
        binding.KVCache(codes, codes, torch.zeros(2, 1, 16), torch.zeros(2, 1, 16))
    with pytest.raises(ValueError, match="CUDA"):
        c8 = codes.view(torch.int8)
        binding.KVCache(c8, c8, torch.zeros(2, 1, 16), torch.zeros(2, 1, 16))
    with pytest.raises(KeyError):
        binding._MASKS["tree"]


def test_the_struct_matches_the_header():
    assert ctypes.sizeof(binding._CacheStruct) == 5 * 8 + 5 * 4 + 4
