"""dspark_kv_append and dspark_kv_read on both sides of the rule that gives a
block one row or several, for few and many heads: bit-exact either way."""
import pytest
import torch

import plain_cache
from speculative_decoding_draft_head_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("H,D", [(1, 64), (1, 128), (32, 64), (32, 128), (17, 48)])
@pytest.mark.parametrize("n", [100, 700, 2100, 11000])
def test_rows_of_few_and_many_heads(n, H, D, fmt, dtype):
    gen = torch.Generator(device="cuda").manual_seed(n + H)
    page = 32
    rows = [n // 3, 0, n - n // 3]
    start = torch.tensor([5, 9, 40], dtype=torch.int32)
    need = [-(-(int(s) + r) // page) for s, r in zip(start, rows)]
    order = torch.randperm(sum(need), generator=gen, device="cuda").int().cpu()
    table = torch.zeros((3, max(need)), dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    cache = binding.KVCache.empty(sum(need), H, page, D, dtype=fmt)
    row0 = torch.tensor([0] + rows).cumsum(0)
    k, v = [torch.randn((n, H, D), generator=gen, device="cuda").to(dtype) for _ in range(2)]
    dev = [t.cuda() for t in (table, start, row0)]
    binding.kv_append(k, v, cache, *dev)
    got = binding.kv_read(cache, *dev, n, dtype=dtype)
    for name, t in (("k", k), ("v", v)):
        codes, scale = plain_cache.quantise(t, fmt)
        assert torch.equal(got[name], (codes.float() * scale[..., None]).to(dtype))
    assert binding.read_device_flags(cache.flags) == 0
