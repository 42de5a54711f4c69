"""The example that runs a whole round: draft, schedule, cache, attention and
verification together."""
import os
import sys

import pytest
import torch

import plain_cache

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import target_pass
    return target_pass


@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.int8])
def test_rounds_leave_the_given_tokens_in_the_cache(example, fmt):
    """After some rounds every request's cached keys and values are those of the
    tokens it was given, whatever was rejected on the way."""
    from speculative_decoding_draft_head_gb300 import binding
    rounds, G = 5, 5
    r = example.run(rounds=rounds, B=9, prompt=77, G=G, V=1024, page=16, dtype=fmt)
    assert binding.read_device_flags(r["cache"].flags) == 0
    length, tokens = r["length"].cpu(), r["tokens"].cpu().long()
    assert (length >= rounds).all() and (length <= rounds * (G + 1)).all()
    row0 = torch.zeros(10, dtype=torch.int64)
    row0[1:] = length.cumsum(0)
    n = int(row0[-1])
    got = binding.kv_read(r["cache"], r["block_table"], torch.zeros_like(r["length"]), row0.cuda(), n,
                          dtype=torch.float32)
    rows = torch.cat([tokens[b, :length[b]] for b in range(9)])
    assert (rows >= 0).all() and (tokens[torch.arange(9), length.long()] >= 0).all()
    for name in ("k", "v"):
        want, scale = plain_cache.quantise(getattr(r["target"], name).cpu()[rows], fmt)
        assert torch.equal(got[name].cpu(), want.float() * scale[..., None])


def test_a_run_repeats(example):
    a = example.run(rounds=3, B=5, prompt=33, V=1024)
    b = example.run(rounds=3, B=5, prompt=33, V=1024)
    assert torch.equal(a["tokens"], b["tokens"])
