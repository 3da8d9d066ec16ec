"""Plain 64-bit restatement of the shared-prefix cache's operations on CPU
tensors, with the error bounds its results are compared under."""
import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def attend(q, k, v, lens, prefix_k, prefix_v, prefix_lens, prefix_of, scale=None):
    """(out, lse, own weights [S, Hkv, cap], bounds of the three) in fp64.

    Bounds, u the half step of fp32 (2^-24): a logit is a dot product of d
    terms accumulated in 32 bits (at most two half steps a term, for tensor
    cores that truncate), so it is off by at most e = 2 (d + 2) u max sum |q k|
    scale; a weight exp(x - lse) by a factor of 2 e + 2 (n + 16) u, n being
    the keys summed and 16 half steps the exponentials'.  Outputs of a bf16
    cache also round each weight and the result to 8 bits."""
    S, H, T, d = q.shape
    Hk = k.shape[1]
    rep = H // Hk
    u = U[torch.float32]
    half = U[q.dtype] if q.dtype == torch.bfloat16 else u
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(S, H, T, d, dtype=torch.float64)
    lse = torch.full((S, H, T), -math.inf, dtype=torch.float64)
    wgt = torch.zeros(S, Hk, k.shape[2], dtype=torch.float64)
    b_out, b_lse, b_wgt = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(wgt)
    q, k, v = q.double(), k.double(), v.double()
    G = 0 if prefix_k is None else prefix_k.shape[0]
    for s in range(S):
        g = int(prefix_of[s]) if G else -1
        has = 0 <= g < G
        p = min(max(int(prefix_lens[g]), 0), prefix_k.shape[2]) if has else 0
        for h in range(H):
            hk = h // rep
            n = min(max(int(lens[s, hk]), 0), k.shape[2])
            for t in range(T):
                lim = max(0, n - T + t + 1)
                kk, vv = k[s, hk, :lim], v[s, hk, :lim]
                if p:
                    kk = torch.cat([prefix_k[g, hk, :p].double(), kk])
                    vv = torch.cat([prefix_v[g, hk, :p].double(), vv])
                if kk.shape[0] == 0:
                    continue
                x = kk @ q[s, h, t] * sc
                e = 2 * (d + 2) * u * float((kk.abs() @ q[s, h, t].abs()).max()) * abs(sc)
                ls = torch.logsumexp(x, 0)
                w = (x - ls).exp()
                rel = 2 * e + 2 * (kk.shape[0] + 16) * u
                out[s, h, t] = w @ vv
                mag = w @ vv.abs()
                b_out[s, h, t] = (rel + (half if half > u else 0.0)) * mag + half * out[s, h, t].abs() * 1.01
                lse[s, h, t] = ls
                b_lse[s, h, t] = rel + 2 * u * abs(float(ls))
                wgt[s, hk, :lim] += w[p:]
                b_wgt[s, hk, :lim] += w[p:] * (rel + 2 * rep * T * u)
    return out, lse, wgt, b_out, b_lse, b_wgt


def assert_within(got, want, bound, what, floor=1e-30):
    got = got.double().cpu()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), what
    bad = (got - want).abs().nan_to_num(0.0) > bound + floor
    bad &= torch.isfinite(want)
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs().nan_to_num(0.0).max()))
    assert torch.equal(got[~torch.isfinite(want)], want[~torch.isfinite(want)]), what


def evict(k, v, pos, weight, lens, budgets, recent, slack):
    """The eviction on numpy arrays (k, v as row payloads), in place."""
    S, Hk, cap = pos.shape
    for s in range(S):
        for h in range(Hk):
            n, B = min(max(int(lens[s, h]), 0), cap), max(0, int(budgets[s, h]))
            if n < B + slack:
                continue
            p, w = pos[s, h, :n].astype(np.int64), weight[s, h, :n].astype(np.float64)
            newest = p.max()
            # (recent, weight with NaN above every number, position, slot)
            key = [(1, 0.0, 0.0, int(p[i]), i) if newest - p[i] < recent else
                   (0, float(np.isnan(w[i])), 0.0 if np.isnan(w[i]) else float(w[i]), int(p[i]), i) for i in range(n)]
            gone = np.zeros(n, bool)
            gone[sorted(range(n), key=lambda i: key[i])[: n - B]] = True
            holes, movers = np.nonzero(gone[:B])[0], B + np.nonzero(~gone[B:])[0]
            assert len(holes) == len(movers)
            for a in (k, v, pos, weight):
                a[s, h, holes] = a[s, h, movers]
            lens[s, h] = B
