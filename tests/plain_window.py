"""Plain 64-bit form of the attention through a window, on the CPU, with the
bounds of plain_cache.attention (one fp16 rounding of each softmax term with its
value's scale)."""
import math

import torch


def sees(n, ctx, window, sinks, mask="causal", words=None):
    """[n, ctx + n] truth values: row i of a block behind ctx tokens sees token t."""
    t, i = torch.arange(ctx + n), torch.arange(n)[:, None]
    if words is None:
        see = (t > ctx + i - window) | (t < sinks)
        return see & (t <= ctx + i) if mask == "causal" else see
    inside = torch.stack([(words >> j) % 2 == 1 for j in range(n)], 1)
    before = (t[:ctx] >= ctx - (window - inside.sum(1, keepdim=True)).clamp_min(0)) | (t[:ctx] < sinks)
    return torch.cat([before, inside], 1)


def attention(q, pool, row0, lens, window, sinks, mask="causal", words=None, scale=None, terms=2.0 ** -11):
    """out, lse and their bounds, in 64 bits (see plain_cache.attention for how the bounds are made)."""
    R, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    group = Hq // pool.k.shape[1]
    out = torch.zeros((R, Hq, D), dtype=torch.float64)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64)
    tol_out, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    info = torch.finfo(q.dtype)
    P = pool.prefix
    for b in range(len(row0) - 1):
        r, n = int(row0[b]), int(row0[b + 1] - row0[b])
        if n == 0:
            continue
        see = sees(n, P + lens[b] - n, window, sinks, mask, None if words is None else words[r:r + n])
        use = see.any(0).nonzero()[:, 0]
        see = see[:, use]
        k, v = [torch.empty((len(use), pool.k.shape[1], D), dtype=torch.float64) for _ in range(2)]
        for mine, pages, at in ((use < P, pool.prefix_pages, use), (use >= P, pool.table[b], use - P)):
            if mine.any():
                pg, off = pages.long()[at[mine] // pool.page], at[mine] % pool.page
                for to, codes, scales in ((k, pool.k, pool.k_scale), (v, pool.v, pool.v_scale)):
                    to[mine] = (codes.view(torch.uint8)[pg, :, off].view(pool.dtype).double()
                                * scales[pg, :, off].double()[..., None])
        seen = see.sum(1)
        for g in range(Hq):
            x, kh, vh = q[r:r + n, g].double(), k[:, g // group], v[:, g // group]
            s = torch.where(see, (x @ kh.T) * scale, torch.tensor(-math.inf, dtype=torch.float64))
            mag = (x.abs() @ kh.abs().T + 2.0 ** -8 * x.abs().amax(1, keepdim=True) * kh.abs().sum(1)[None]) * scale
            A = torch.where(see, mag, torch.zeros_like(mag)).nan_to_num(0)
            A = A.amax(1) if A.shape[1] else torch.zeros(n, dtype=torch.float64)
            ds = 2 * (D + 8) * 2.0 ** -24 * A
            p = torch.where(see & (seen > 0)[:, None], torch.softmax(s, -1), torch.zeros_like(s))
            clean = torch.isfinite(s) | ~see
            vz = vh.nan_to_num(0)
            o = p.nan_to_num(0) @ vz
            # a row that sees a NaN (in a score or a value) is NaN
            bad = (~clean).any(1) | ((see & vh.isnan().any(1)[None]).any(1))
            o[bad] = math.nan
            spread = p.nan_to_num(0) @ vz.abs()
            top = vz.abs().amax(1) if len(use) else torch.zeros(0, dtype=torch.float64)
            vmax = (see * top).amax(1) if len(use) else torch.zeros(n, dtype=torch.float64)
            out[r:r + n, g] = o
            lse[r:r + n, g] = torch.where(bad, torch.full((n,), math.nan, dtype=torch.float64),
                                          torch.logsumexp(s.nan_to_num(0, neginf=-math.inf), -1))
            tol_out[r:r + n, g] = (info.eps / 2 * o.abs().nan_to_num(0) * (1 + 2.0 ** -8)
                                   + (2 * ds + terms + 2.0 ** -18)[:, None] * spread + (seen * 2.0 ** -30 * vmax)[:, None]
                                   + info.smallest_normal * info.eps / 2)
            tol_lse[r:r + n, g] = ds + 2.0 ** -18 + 2.0 ** -22 * lse[r:r + n, g].abs().nan_to_num(0, posinf=0)
    return out, lse, tol_out, tol_lse
