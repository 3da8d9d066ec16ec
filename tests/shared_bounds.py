"""Bounds for attention whose softmax weights are not rounded to the rows' type:
the restatement in 64 bits a (sequence, KV head) at a time, and inputs on which
a weight's rounding shows at any number of keys, a value row left out up to 2000.

A bf16 cache's kernels multiply the values by a weight's first 8 bits and by
what they leave, so an output is off by its own rounding, 2^-8 of it, by 2^-15
of sum w |v| (two roundings to 8 bits, at most a step each), and by 32-bit
arithmetic.  u = 2^-24 is half a step of fp32:
  logits    their scaling, the scale's rounding and the reference's, of
            magnitude |x|: 8 u max |x|; the dot product of d terms, at most two
            half steps each: 2 (d + 2) u max sum |q k| scale, or nothing where
            every partial sum is exact;
  weights   2^-21 for the exponential;
  sums      each of n / 16 steps of 16 products, and 64 more to join
            the pieces, off by four half steps of the running sum (tensor
            cores truncate): 4 u (n / 16 + 64).
The sum of the weights (the divisor) has the same errors: twice the total."""
import math

import torch

U = 2.0 ** -24
BF16_HALF = 2.0 ** -8
KEPT = 2.0 ** -15


def attend(q, k, v, lens, prefix_k=None, prefix_v=None, prefix_lens=None, prefix_of=None, scale=None,
           exact_logits=False):
    """(out, lse, own weights, bounds of the three) in fp64, of bf16 CPU tensors."""
    S, H, T, d = q.shape
    Hk, cap = k.shape[1:3]
    rep = H // Hk
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(S, H, T, d, dtype=torch.float64)
    lse = torch.full((S, H, T), -math.inf, dtype=torch.float64)
    wgt = torch.zeros(S, Hk, cap, dtype=torch.float64)
    b_out, b_lse, b_wgt = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(wgt)
    G = 0 if prefix_k is None else prefix_k.shape[0]
    for s in range(S):
        g = int(prefix_of[s]) if G else -1
        p = int(prefix_lens[g]) if 0 <= g < G else 0
        for hk in range(Hk):
            n = int(lens[s, hk])
            kk, vv = k[s, hk, :n].double(), v[s, hk, :n].double()
            if p:
                kk = torch.cat([prefix_k[g, hk, :p].double(), kk])
                vv = torch.cat([prefix_v[g, hk, :p].double(), vv])
            if p + n == 0:
                continue
            hs = slice(hk * rep, hk * rep + rep)
            qq = q[s, hs].double()
            hidden = torch.arange(p + n)[None] > (p + n - T + torch.arange(T))[:, None]
            hidden &= torch.arange(p + n)[None] >= p
            x = (qq @ kk.T * sc).masked_fill(hidden, -math.inf)
            ls = torch.logsumexp(x, -1)
            w = (x - ls[..., None]).exp().nan_to_num(0.0)
            e = 8 * U * x.masked_fill(hidden, 0.0).abs().amax(-1)
            if not exact_logits:
                e = e + 2 * (d + 2) * U * (qq.abs() @ kk.abs().T * abs(sc)).masked_fill(hidden, 0.0).amax(-1)
            rel = 2 * (e + 2.0 ** -21 + 4 * U * ((~hidden).sum(-1) / 16 + 64))
            out[s, hs], lse[s, hs] = w @ vv, ls
            b_out[s, hs] = (rel + KEPT)[..., None] * (w @ vv.abs()) + 1.01 * BF16_HALF * out[s, hs].abs()
            b_lse[s, hs] = rel + 2 * U * ls.abs()
            wgt[s, hk, :n] = w[..., p:].sum((0, 1))
            b_wgt[s, hk, :n] = (w[..., p:] * (rel + 2 * rep * T * U)[..., None]).sum((0, 1))
    return out, lse, wgt, b_out, b_lse, b_wgt


#: Factors of the query rows' logits, row t of a head having STEPS[t % 3].
STEPS = (1.0, 0.5, 2.0)


def comb(S, H, Hk, T, d, n, G=0, P=0, seed=0):
    """bf16 q, k, v, prefix_k, prefix_v whose logits are exact in 32 bits (scale 1):
    0 at every eighth key, so that every piece of 8 keys has the reference, and
    elsewhere one of some levels whose weights bf16 rounds by much; V's columns
    hold, for one factor of the rows, the signs of these roundings, which so add
    up."""
    g = torch.Generator().manual_seed(seed)
    signs = torch.randint(0, 2, (d,), generator=g) * 2.0 - 1
    signs[:2] = 1
    q = signs * torch.tensor([STEPS[t % 3] for t in range(T)])[:, None]
    levels = -torch.arange(1, 129).double() / 64  # exact in bf16, as their halves and doubles are
    err = (levels.exp().bfloat16().double() - levels.exp()).abs() / levels.exp()
    levels = levels[err > 2.0 ** -9.7]

    def keys(*lead):
        x = levels[torch.randint(0, len(levels), lead, generator=g)]
        x[..., ::8] = 0
        kk = torch.randint(-1, 2, (*lead, d), generator=g).double()
        kk[..., 1] = x
        kk[..., 0] = -(kk[..., 2:] * signs[2:]).sum(-1)  # an integer below 2^8
        vv = torch.empty(*lead, d, dtype=torch.float64)
        for c in range(d):
            p = (x * STEPS[c % 3]).exp()
            up = torch.sign(p.bfloat16().double() - p)
            vv[..., c] = torch.where(up == 0, torch.randint(0, 2, lead, generator=g) * 2.0 - 1, up) * (-1) ** (c // 3)
        assert torch.equal(kk.bfloat16().double(), kk)
        return kk.bfloat16(), vv.bfloat16()

    k, v = keys(S, Hk, n)
    pk, pv = keys(G, Hk, P) if G else (None, None)
    return q.expand(S, H, T, d).contiguous().bfloat16(), k, v, pk, pv
