"""Decoding rounds with a target model's attention in them.

    python examples/target_pass.py [--rounds 8] [--batch 64] [--prompt 1000] [--rotary] [--window 256 --sinks 4]

A target of one attention layer (a token's query, key and value are rows of
three tables; with --rotary turned by the token's position) answers a batch of
requests that share a prompt.  The prompt enters the quantised cache once, on pages that every
request's attention reads.  Each round then

  1. drafts a block per request and schedules how much of it to verify,
  2. packs the anchor and the scheduled tokens of every request into rows,
  3. writes their keys and values behind the request's own cached tokens,
  4. lets every row attend to the prompt, the own tokens and its block (with
     --window to the last tokens of these and the first --sinks ones),
  5. verifies the drafted tokens with the logits of these rows.

The tokens that the verification rejects leave nothing to undo: the next round
starts at the accepted length and writes over them.  Nothing in a round waits
for the device: sizes that depend on the schedule stay on it, and the packed
arrays have room for the longest blocks.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from speculative_decoding_draft_head_gb300 import binding  # noqa: E402


class Target:
    """One attention layer over the cache, then logits."""

    def __init__(self, V, Hq, Hkv, D, gen, device):
        def table(n, *shape):
            return torch.randn((n, *shape), generator=gen, device=device).bfloat16()
        self.q, self.k, self.v = table(V, Hq, D), table(V, Hkv, D), table(V, Hkv, D)
        self.unembed = table(V, Hq * D)

    def logits(self, attended):
        return attended.flatten(1) @ self.unembed.t() / 16


def run(rounds=8, B=64, prompt=1000, G=5, V=4096, r=64, Hq=16, Hkv=4, D=128, page=64, dtype=torch.float8_e4m3fn, seed=0,
        rotary=False, window=None, sinks=0):
    """Runs ``rounds`` rounds; returns dict(target, cache, prompt, pages, block_table, tokens, length): ``tokens``
    [B, rounds * (G + 1) + 1] what each request was given, -1 padded, the first ``length`` of them cached."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    target = Target(V, Hq, Hkv, D, gen, dev)
    base = torch.randn((B, G, V), generator=gen, device=dev).bfloat16()
    e_in, w_out = ((torch.randn((V, r), generator=gen, device=dev) / r ** 0.5).bfloat16() for _ in range(2))
    temperature = torch.ones(B, device=dev)
    conf_logits = torch.randn((B, G), generator=gen, device=dev) + 1
    pos_temp = torch.ones(G, device=dev)
    # steps per second against the tokens of a step
    sps = 1 / (1 + torch.arange(B * (G + 1) + 1, device=dev, dtype=torch.float32) / (2 * B))

    # pages: the prompt's first, then every request's own
    prompt_pages = -(-prompt // page)
    own = -(-(rounds * (G + 1) + 1) // page)
    order = torch.randperm(prompt_pages + B * own, generator=gen, device=dev).int()
    pages, block_table = order[:prompt_pages].contiguous(), order[prompt_pages:].view(B, own).contiguous()
    cache = binding.KVCache.empty(order.numel(), Hkv, page, D, dtype=dtype, device=dev)
    given = torch.randint(V, (prompt,), generator=gen, device=dev)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    # (D / 2 pairs, the usual frequencies)
    turn = binding.Rotary(10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))) if rotary else None
    prompt_row0 = torch.tensor([0, prompt], device=dev)
    if rotary:
        binding.kv_append_rotary(target.k[given], target.v[given], cache, pages[None], zero, prompt_row0, turn)
    else:
        binding.kv_append(target.k[given], target.v[given], cache, pages[None], zero, prompt_row0)

    n = B * (G + 1)
    j = torch.arange(G + 1, device=dev)
    row0 = torch.zeros(B + 1, dtype=torch.int64, device=dev)
    anchor = torch.randint(V, (B,), generator=gen, device=dev).int()
    length = torch.zeros(B, dtype=torch.int32, device=dev)
    tokens = torch.full((B, rounds * (G + 1) + 2), -1, dtype=torch.int32, device=dev)
    tokens[:, 0] = anchor
    for t in range(rounds):
        draft = binding.draft_sample(base, e_in, w_out, anchor, temperature, seed=seed + t)
        verify_len = binding.schedule_prefix(conf_logits, pos_temp, sps, 1, G)["verify_len"]

        torch.cumsum(verify_len + 1, 0, out=row0[1:])
        block = torch.cat([anchor[:, None], draft["tokens"]], 1).long()
        to = torch.where(j <= verify_len[:, None], row0[:-1, None] + j, n)  # row n takes what is not verified
        rows = torch.zeros(n + 1, dtype=torch.int64, device=dev).scatter_(0, to.flatten(), block.flatten())[:n]

        q = target.q[rows]
        if rotary:
            binding.kv_append_rotary(target.k[rows], target.v[rows], cache, block_table, length, row0, turn, q=q, out=q,
                                     offset=prompt)
        else:
            binding.kv_append(target.k[rows], target.v[rows], cache, block_table, length, row0)
        seen = (q, cache, block_table, length + verify_len + 1, row0)
        if window:
            att = binding.window_attention(*seen, window=window, sinks=sinks, prefix_pages=pages, prefix_len=prompt)
        else:
            att = binding.block_attention(*seen, prefix_pages=pages, prefix_len=prompt)
        out = binding.verify(target.logits(att["out"]), base, e_in, w_out, anchor, draft, verify_len, temperature,
                             seed=seed + t, target_row0=row0[:-1])

        # the anchor and what was accepted are cached now; the last token given is the next anchor
        new = out["out_tokens"]
        at = torch.where(j < out["num_out"][:, None], length[:, None] + 1 + j, tokens.shape[1] - 1)
        tokens.scatter_(1, at, new)
        tokens[:, -1] = -1
        length = length + out["num_out"]
        anchor = new.gather(1, out["num_out"][:, None].long() - 1)[:, 0].contiguous()
    return dict(target=target, cache=cache, prompt=given, pages=pages, block_table=block_table,
                tokens=tokens[:, :-1], length=length)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=8)
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--rotary", action="store_true")
    ap.add_argument("--window", type=int)
    ap.add_argument("--sinks", type=int, default=0)
    a = ap.parse_args()
    r = run(a.rounds, a.batch, a.prompt, rotary=a.rotary, window=a.window, sinks=a.sinks)
    flags = binding.read_device_flags(r["cache"].flags)
    total = int(r["length"].sum())
    print("%d requests, %d rounds, %d tokens given (%.2f a request and round), cache flags %d"
          % (a.batch, a.rounds, total, total / a.batch / a.rounds, flags))


if __name__ == "__main__":
    main()
