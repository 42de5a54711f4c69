"""Calls whose `stream` is not the current one: the tensors that a call makes
belong to the stream that writes them, so that the allocator neither gives out
memory that another stream's queued work still reads nor takes it back early."""
import pytest
import torch

import plain_cache
from speculative_decoding_draft_head_gb300 import binding
from speculative_decoding_draft_head_gb300.synth import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu


def _streams_of(tensors):
    """The stream in whose order each tensor's memory was given out."""
    at = {}
    for seg in torch.cuda.memory_snapshot():
        for name, t in tensors.items():
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                at[name] = seg["stream"]
    assert set(at) == set(tensors)
    return at


@pytest.fixture
def side():
    s = torch.cuda.Stream()
    yield s
    torch.cuda.synchronize()


def _cache_inputs():
    gen = torch.Generator().manual_seed(3)
    pool = plain_cache.Pool(gen, [40, 25], 30, 2, 64, 16, torch.float8_e4m3fn)
    row0 = torch.tensor([0, 3, 7])
    q = torch.randn((7, 4, 64), generator=gen).bfloat16()
    args = (pool.cache(binding), pool.table.cuda(), torch.tensor([40, 25], dtype=torch.int32).cuda(), row0.cuda())
    kw = dict(prefix_pages=pool.prefix_pages.cuda(), prefix_len=30)
    torch.cuda.synchronize()
    return pool, row0, q, args, kw


def test_attention_and_cache_rows_belong_to_their_call(side):
    pool, row0, q, args, kw = _cache_inputs()
    qd, start = q.cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    want = binding.block_attention(qd, *args, **kw)
    rows = binding.kv_read(args[0], args[1], start, args[3], 7)
    torch.cuda.synchronize()
    got = binding.block_attention(qd, *args, stream=side, **kw)
    read = binding.kv_read(args[0], args[1], start, args[3], 7, stream=side)
    side.synchronize()
    made = {**got, **read}
    assert _streams_of(made) == {name: side.cuda_stream for name in made}
    for name, t in {**want, **rows}.items():
        assert torch.equal(made[name], t)


def test_the_rounds_results_belong_to_their_calls(side):
    w = WORKLOADS["dspark5"].scaled(B=4, V=2056)
    inp = make_inputs(w, 0, device=torch.device("cuda"))
    torch.cuda.synchronize()

    def a_round(stream):
        d = binding.draft_sample(inp["base"], inp["e_in"], inp["w_out"], inp["anchor"], inp["temperature"],
                                 inp["request_id"], 0, stream=stream)
        s = binding.schedule_prefix(inp["conf_logits"], inp["pos_temp"], inp["sps"], w.L_min, w.G, stream=stream)
        v = binding.verify(inp["target"], inp["base"], inp["e_in"], inp["w_out"], inp["anchor"], d, s["verify_len"],
                           inp["temperature"], inp["request_id"], 0, stream=stream)
        p = binding.pack_target(inp["target"], s["verify_len"], stream=stream)
        torch.cuda.synchronize()
        n = int(p["n_rows"])
        return {k + str(i): t for i, part in enumerate((d, s, v, p)) for k, t in part.items()}, n

    want, n = a_round(None)
    got, _ = a_round(side)
    assert _streams_of(got) == {name: side.cuda_stream for name in got}
    for name in ("tokens0", "verify_len1", "accept_len2", "out_tokens2"):
        assert torch.equal(got[name], want[name])
    assert torch.equal(got["target3"][:n], want["target3"][:n])


def test_lagged_confidences_are_kept_in_the_calls_stream(side):
    G = 5
    sched = binding.LaggedScheduler(torch.ones(G, device="cuda"), torch.ones(64, device="cuda"), 1, G, lag=1)
    conf = torch.randn((3, G), device="cuda")
    torch.cuda.synchronize()
    sched.step(conf, stream=side)
    torch.cuda.synchronize()
    assert _streams_of(dict(kept=sched._ring[0])) == dict(kept=side.cuda_stream)
