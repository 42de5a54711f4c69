"""The library launches on the current device: calls whose tensors or stream are
on another one are refused before anything is launched (no GPU is used here: the
library and the current device are stand-ins)."""
import types

import pytest
import torch

from speculative_decoding_draft_head_gb300 import binding


class _Never:
    """A library of which no entry point may be called."""

    def __getattr__(self, name):
        raise AssertionError(name + " was called")


@pytest.fixture
def elsewhere(monkeypatch):
    """A cache on device 1 while device 0 is current."""
    monkeypatch.setattr(binding, "_lib", _Never())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    cache = object.__new__(binding.KVCache)
    cache._index, cache.device, cache._ref = 1, torch.device("cuda", 1), None
    cache.n_pages, cache.n_kv_heads, cache.page_size, cache.head_dim = 4, 2, 16, 64
    return cache


def _calls(cache, **kw):
    rows, table = torch.zeros((3, 2, 64)), torch.zeros((1, 2), dtype=torch.int32)
    lens, row0 = torch.ones(1, dtype=torch.int32), torch.tensor([0, 3])
    return [lambda: binding.kv_append(rows, rows, cache, table, lens, row0, **kw),
            lambda: binding.kv_read(cache, table, lens, row0, 3, **kw),
            lambda: binding.block_attention(rows.bfloat16(), cache, table, lens, row0, **kw)]


def test_a_cache_on_another_device_is_refused(elsewhere):
    for call in _calls(elsewhere):
        with pytest.raises(ValueError, match="cuda:1, which is not the current device"):
            call()


def test_a_stream_of_another_device_is_refused(elsewhere, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in _calls(elsewhere, stream=types.SimpleNamespace(device_index=0, cuda_stream=5)):
        with pytest.raises(ValueError, match="stream is of cuda:0"):
            call()


def test_the_rounds_calls_use_the_same_check(elsewhere):
    with pytest.raises(ValueError, match="not the current device"):
        binding._stream(None, torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream is of cuda:3"):
        binding._stream(types.SimpleNamespace(device_index=3, cuda_stream=5), torch.device("cuda", 0))
    stream = types.SimpleNamespace(device_index=0, cuda_stream=5)
    assert binding._stream(stream, torch.device("cuda", 0)).value == 5
