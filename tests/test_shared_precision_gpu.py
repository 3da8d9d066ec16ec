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


def random_call(S, H, Hk, T, d, cap, P, seed):
    """Normal rows, queries that look for some own key, lengths from 0 to the
    capacity, two prefixes of unequal lengths and sequences without."""
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(S, Hk, cap, d, generator=g).bfloat16() for _ in range(2))
    pk, pv = (torch.randn(2, Hk, P, d, generator=g).bfloat16() for _ in range(2))
    lens = torch.randint(T, cap + 1, (S, Hk), generator=g)
    lens.view(-1)[:4] = torch.tensor([cap, T, max(0, T - 5), 0])[:lens.numel()]
    at = torch.randint(0, cap, (S, H, T), generator=g) % lens.clamp(min=1).repeat_interleave(H // Hk, 1)[..., None]
    near = k.repeat_interleave(H // Hk, 1).gather(2, at[..., None].expand(-1, -1, -1, d))
    q = (torch.randn(S, H, T, d, generator=g) + 0.4 * near.float()).bfloat16()
    free = torch.arange(cap) >= lens[..., None]
    k[free], v[free] = float("nan"), float("inf")
    return q, k, v, pk, pv, lens, [P, max(1, P // 2 - 3)], [(s + 1) % 3 - ((s + 1) % 3 == 2) * 3 for s in range(S)]


# (S, H, Hk, T, capacity, prefix): rows a head H / Hk T in blocks of 256 above 512, of 128 up to it
LARGE = [(2, 8, 1, 100, 150, 100),    # 800 rows, keys of one piece: final in two row tiles
         (3, 14, 2, 75, 130, 70),     # 525: the last block holds 13 rows of its first tile
         (40, 4, 2, 300, 390, 100),   # 600: the last block's second tile is empty; 240 blocks
         (50, 1, 1, 513, 640, 33),    # 513: one row in the last block
         (25, 14, 2, 100, 900, 130),  # 700: its second tile holds 60 rows; more key tiles than places in the ring
         (38, 2, 1, 400, 470, 65),    # 800 again, 152 blocks
         (40, 1, 1, 400, 470, 65),    # 400: four blocks a head, their sums joined
         (40, 1, 1, 512, 513, 1),     # 512 exactly
         (40, 4, 4, 49, 1300, 200),   # 49 rows over more than twenty key tiles
         (3, 4, 2, 700, 1500, 300),   # two row tiles in pieces, a pass of sums behind
         (1, 2, 1, 1000, 1003, 64)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,H,Hk,T,cap,P", LARGE)
def test_many_rows_of_many_blocks(S, H, Hk, T, cap, P, d):
    args = random_call(S, H, Hk, T, d, cap, P, seed=T + d)
    check(*args)
    check(*args, accumulate=False, scale=-0.07)
