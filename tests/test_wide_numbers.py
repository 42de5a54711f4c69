"""Numbers that pass 32 bits are refused, not cut to their low half (no GPU is
used here: the library and the current device are stand-ins)."""
import pytest
import torch

from speculative_decoding_draft_head_gb300 import binding


class _Never:
    """A library of which no entry point may be called."""

    def __getattr__(self, name):
        raise AssertionError(name + " was called")


@pytest.fixture
def cache(monkeypatch):
    monkeypatch.setattr(binding, "_lib", _Never())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 5, raising=False)
    cache = object.__new__(binding.KVCache)
    cache._index, cache.device, cache._ref = -1, torch.device("cpu"), None
    cache.n_pages, cache.n_kv_heads, cache.page_size, cache.head_dim = 4, 1, 16, 16
    return cache


TABLE, LENS, ROW0 = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.tensor([0, 3])
WIDE = 2 ** 32 + 3


@pytest.mark.parametrize("n", [WIDE, 2 ** 31, WIDE - 2 ** 34])
def test_prefix_lengths(cache, n):
    with pytest.raises(ValueError, match="2.31"):
        binding.block_attention(torch.zeros((3, 1, 16), dtype=torch.float16), cache, TABLE, LENS, ROW0,
                                prefix_pages=torch.zeros(1, dtype=torch.int32), prefix_len=n)


def test_rows(cache):
    rows = torch.empty((WIDE, 1, 16), dtype=torch.float16, device="meta")
    with pytest.raises(ValueError, match="2.31"):
        binding.block_attention(rows, cache, TABLE, LENS, ROW0)
    with pytest.raises(ValueError, match="2.31"):
        binding.kv_append(rows, rows, cache, TABLE, LENS, ROW0)
    with pytest.raises(ValueError, match="2.31"):
        binding.kv_read(cache, TABLE, LENS, ROW0, WIDE)


def test_pages(cache):
    table = torch.empty((1, WIDE), dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="2.31"):
        binding.kv_read(cache, table, LENS, ROW0, 3)
