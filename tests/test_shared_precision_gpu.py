"""Attention of bf16 caches within bounds that grant no rounding of the softmax
weights (tests/shared_bounds.py), by every kernel and shape of block."""
import pytest
import torch

import kv_cache_compression_hkv_b200 as hkv

import shared_bounds as B
import shared_oracle as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_compression_hkv_b200 import build
    build.build()
    assert torch.cuda.is_available(), "these tests need a CUDA device"


def check(q, k, v, pk, pv, lens, plens, of, accumulate=True, **kw):
    S, H, T, d = q.shape
    Hk, cap = k.shape[1:3]
    G = 0 if pk is None else pk.shape[0]
    up = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    c = hkv.SharedPrefixCache(hkv.SharedConfig(S, H, Hk, d, cap, G, pk.shape[2] if G else 0), DEV, k=up(k), v=up(v),
                              prefix_k=up(pk), prefix_v=up(pv))
    c.lens.copy_(lens)
    if G:
        c.prefix_lens.copy_(torch.tensor(plens))
        c.prefix_of.copy_(torch.tensor(of))
    out, lse = c.attend(up(q), accumulate=accumulate, scale=kw.get("scale"))
    assert c.check() == (0, 0)
    o, e, w, bo, be, bw = B.attend(q, k, v, lens, pk, pv, plens, of, **kw)
    O.assert_within(out, o, bo, "out")
    O.assert_within(lse, e, be, "lse")
    if accumulate:
        O.assert_within(c.weight, w, bw, "weight")
    else:
        assert not c.weight.any()


# (S, H, Hk, T, own slots, prefix slots): what the shape reaches
SHAPES = [(2, 4, 4, 1, 500, 200),       # one row streamed, several pieces
          (300, 4, 4, 1, 40, 20),       # one warp a head, final
          (3, 8, 1, 1, 1300, 100),      # 8 rows
          (3, 12, 1, 1, 1300, 100),     # 9 to 16: a second product
          (80, 32, 2, 1, 90, 33),       # the same, final
          (40, 2, 2, 1, 60, 4100),      # long prefixes read once, own keys beside
          (40, 32, 2, 1, 60, 4100),
          (2, 4, 2, 10, 900, 300),      # row tiles in pieces
          (3, 2, 1, 400, 800, 300),     # two row tiles a block in pieces
          (40, 4, 4, 49, 210, 90),      # final, weights by the block
          (20, 4, 2, 200, 330, 65),     # several blocks a head
          (2, 4, 1, 70, 140, 100),      # keys of one piece
          (2, 8, 1, 100, 140, 100)]     # the same, two row tiles a block


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,H,Hk,T,n,P", SHAPES)
def test_weights_keep_what_bf16_leaves(S, H, Hk, T, n, P, d):
    q, k, v, pk, pv = B.comb(S, H, Hk, T, d, n, 2, P, seed=n + d)
    of = [s % 3 - (s % 3 == 2) * 3 for s in range(S)]  # every third without
    check(q, k, v, pk, pv, torch.full((S, Hk), n), [P, P - P // 3], of, scale=1.0, exact_logits=True)
