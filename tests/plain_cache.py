"""Plain 64-bit forms of the quantised cache and of the attention over it, on
the CPU, with the error bounds the GPU results are held to.

A rounding to a type is off by at most finfo(type).eps / 2 relative.  The
attention's bound counts the roundings of its definition: the output's own, the
fp16 roundings of each softmax term and of each value with its scale, and fp32
sums and exponentials in between (see ``attention``)."""
import math

import torch

TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
AMAX_FLOOR = 2.0 ** -100


def quantise(x, dtype):
    """Codes (as the cache type) and fp32 scales of rows x [..., D]: fp32
    operations in the order of the definition, so results are bit-exact."""
    x = x.float()
    amax = x.abs().amax(-1)
    good = torch.isfinite(amax)
    a = torch.where(good, amax, torch.ones_like(amax)).clamp_min(AMAX_FLOOR)
    top = torch.full_like(a, TOP[dtype])  # a tensor: dividing by or into a plain number may go through its reciprocal
    y = torch.where(good[..., None], x * (top / a)[..., None], torch.zeros_like(x)).clamp(-TOP[dtype], TOP[dtype])
    codes = y.to(dtype) if dtype == torch.float8_e4m3fn else torch.round(y).to(dtype)
    return codes, torch.where(good, a / top, torch.full_like(a, math.nan))


class Pool:
    """A CPU cache of shuffled pages, filled with quantised random tokens."""

    def __init__(self, gen, lens, prefix, Hkv, D, page, dtype, k_scale=1.0, v_scale=1.0, token_scale=None,
                 spare=2, filler=0x7F):
        need = [-(-n // page) for n in lens]
        shared = -(-prefix // page)
        self.page, self.prefix, self.lens, self.dtype = page, prefix, list(lens), dtype
        n_pages = sum(need) + shared + spare
        order = torch.randperm(n_pages, generator=gen).to(torch.int32)
        self.table = torch.zeros((len(lens), max(need + [1])), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.prefix_pages = order[at:at + shared].clone()
        shape = (n_pages, Hkv, page, D)
        # places that hold no token of anyone: garbage that must never be used
        self.k = torch.full(shape, filler, dtype=torch.uint8).view(dtype)
        self.v = torch.full(shape, filler, dtype=torch.uint8).view(dtype)
        self.k_scale = torch.full(shape[:3], math.nan)
        self.v_scale = torch.full(shape[:3], math.nan)
        for pages, n in [(self.prefix_pages, prefix)] + [(self.table[b], n) for b, n in enumerate(lens)]:
            if n == 0:
                continue
            pos = torch.arange(n)
            pg, off = pages.long()[pos // page], pos % page
            for codes, scales, s in ((self.k, self.k_scale, k_scale), (self.v, self.v_scale, v_scale)):
                x = torch.randn((n, Hkv, D), generator=gen) * s
                if token_scale is not None:
                    x = x * token_scale(gen, (n, Hkv, 1))
                c, sc = quantise(x, dtype)
                codes.view(torch.uint8)[pg, :, off] = c.view(torch.uint8)
                scales[pg, :, off] = sc

    def tokens(self, pages, n):
        """Keys and values [n, Hkv, D] in 64 bits."""
        pos = torch.arange(n)
        pg, off = pages.long()[pos // self.page], pos % self.page
        return [codes.view(torch.uint8)[pg, :, off].view(self.dtype).double() * scales[pg, :, off].double()[..., None]
                for codes, scales in ((self.k, self.k_scale), (self.v, self.v_scale))]

    def cache(self, binding, device="cuda"):
        return binding.KVCache(self.k.to(device), self.v.to(device), self.k_scale.to(device), self.v_scale.to(device))


def block_sees(mask, words, n):
    """[n, n] truth values: row i sees block token t."""
    t = torch.arange(n)
    if words is not None:
        return torch.stack([(words >> int(j)) % 2 == 1 for j in t], 1) if n else torch.ones((0, 0), dtype=torch.bool)
    return t[None, :] <= t[:, None] if mask == "causal" else torch.ones((n, n), dtype=torch.bool)


def attention(q, pool, row0, lens, mask="causal", words=None, scale=None, terms=2.0 ** -10):
    """out, lse and their bounds, in 64 bits.

    With p_j the softmax, A = max_j scale sum_d |q_d k_jd| and n seen tokens:
      scores: fp32 sums of D products and a few fp32 factors, each rounding (or
        truncation inside a tensor-core sum) at most 2^-23 of A: ds = 2 (D + 8) 2^-24 A
      terms: relative ds + 2^-20 (fp32 exponential) + 2^-11 (fp16 rounding of the
        term) + 2^-11 (fp16 rounding of the value with its scale); terms that fp16
        holds as subnormals are off by 2^-25 against a largest one of at least 2^6
        where the values are largest: 2^-30 n max|v| in all
      q of fp16 or bf16 is exact in fp16 after a power-of-two scaling, but for
        elements 2^-14 below the row's largest: 2^-24 max|q| sum_d |k_jd|
      sums: fp32 over n terms in many partial sums: 2^-18
      (`terms` bounds the fp16 roundings: 2^-10 for the two above, 2^-11 for one)
      output: eps / 2 relative, and half the least subnormal."""
    R, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    Hkv = pool.k.shape[1]
    group = Hq // Hkv
    out = torch.zeros((R, Hq, D), dtype=torch.float64)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64)
    tol_out, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    half = torch.finfo(q.dtype).eps / 2
    kp, vp = pool.tokens(pool.prefix_pages, pool.prefix)
    for b in range(len(row0) - 1):
        r, n = int(row0[b]), int(row0[b + 1] - row0[b])
        if n == 0:
            continue
        ko, vo = pool.tokens(pool.table[b], lens[b])
        k, v = torch.cat([kp, ko]), torch.cat([vp, vo])
        sees = torch.ones((n, k.shape[0]), dtype=torch.bool)
        sees[:, k.shape[0] - n:] = block_sees(mask, None if words is None else words[r:r + n], n)
        for g in range(Hq):
            x = q[r:r + n, g].double()
            kh, vh = k[:, g // group], v[:, g // group]
            s = (x @ kh.T) * scale
            s = torch.where(sees, s, torch.full_like(s, -math.inf))
            some = sees.any(1)
            mag = ((x.abs() @ kh.abs().T + 2.0 ** -8 * x.abs().amax(1, keepdim=True) * kh.abs().sum(1)[None]) * scale)
            A = torch.where(sees, mag, torch.zeros_like(mag)).nan_to_num(0).amax(1)
            ds = 2 * (D + 8) * 2.0 ** -24 * A
            p = torch.where(some[:, None], torch.softmax(s, -1), torch.zeros_like(s))
            # a token no row sees may hold anything
            use = sees.any(0)
            vz = torch.where(use[:, None], vh, torch.zeros_like(vh))
            pz = torch.where(sees, p, torch.zeros_like(p))
            o = torch.stack([(pz[i, sees[i]] @ vz[sees[i]]) if some[i] else torch.zeros(D).double() for i in range(n)])
            spread = pz.nan_to_num(0) @ vz.nan_to_num(0).abs()
            vmax = torch.stack([vz[sees[i]].nan_to_num(0).abs().amax() if some[i] else torch.zeros(()).double()
                                for i in range(n)])
            out[r:r + n, g] = o
            lse[r:r + n, g] = torch.logsumexp(s, -1)
            tol_out[r:r + n, g] = (half * o.abs().nan_to_num(0) * (1 + 2.0 ** -8)
                                   + (2 * ds + terms + 2.0 ** -18)[:, None] * spread
                                   + (sees.sum(1) * 2.0 ** -30 * vmax)[:, None]
                                   + torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps / 2)
            tol_lse[r:r + n, g] = ds + 2.0 ** -18 + 2.0 ** -22 * lse[r:r + n, g].abs().nan_to_num(0, posinf=0)
    return out, lse, tol_out, tol_lse
