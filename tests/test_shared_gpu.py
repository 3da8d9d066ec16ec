"""The shared-prefix cache on the GPU against its 64-bit restatement
(tests/shared_oracle.py), at the sizes and masks where it can go wrong."""
import ctypes as C

import numpy as np
import pytest
import torch

import kv_cache_compression_hkv_b200 as hkv

import shared_oracle as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_compression_hkv_b200 import build
    build.build()
    assert torch.cuda.is_available(), "these tests need a CUDA device"


def rows(g, dtype, S, H, n, d, slot_major=False):
    x = torch.randn((S, n, H, d) if slot_major else (S, H, n, d), generator=g).to(DT[dtype]).to(DEV)
    return x.transpose(1, 2) if slot_major else x


def make(dtype="bf16", S=3, H=4, Hk=2, d=64, T=1, cap=40, lens=None, G=2, P=21, plens=None, of=None, seed=0,
         slot_major=False, sharp=0.4):
    """A cache whose free slots hold NaN, and queries that look for some keys."""
    g = torch.Generator().manual_seed(seed)
    cfg = hkv.SharedConfig(S, H, Hk, d, cap, G, P if G else 0, hkv.DTYPE_F32 if dtype == "f32" else hkv.DTYPE_BF16)
    c = hkv.SharedPrefixCache(cfg, DEV, k=rows(g, dtype, S, Hk, cap, d, slot_major),
                              v=rows(g, dtype, S, Hk, cap, d, slot_major),
                              prefix_k=rows(g, dtype, G, Hk, P, d, slot_major) if G else None,
                              prefix_v=rows(g, dtype, G, Hk, P, d, slot_major) if G else None)
    if lens is None:
        lens = torch.randint(T, cap + 1, (S, Hk), generator=g)
    c.lens.copy_(torch.as_tensor(lens).expand(S, Hk))
    c.weight.copy_(torch.rand(S, Hk, cap, generator=g))
    c.pos.copy_(torch.arange(cap).expand(S, Hk, cap))
    free = (torch.arange(cap, device=DEV) >= c.lens.clamp(0, cap)[..., None])[..., None]
    c.k.masked_fill_(free, float("nan"))
    c.v.masked_fill_(free, float("nan"))
    if G:
        c.prefix_lens.copy_(torch.as_tensor([P, max(1, P // 2), 0][:G] if plens is None else plens))
        c.prefix_of.copy_(torch.arange(S) % G if of is None else torch.as_tensor(of))
        gone = (torch.arange(P, device=DEV) >= c.prefix_lens.clamp(0, P)[:, None])[:, None, :, None]
        c.prefix_k.masked_fill_(gone, float("nan"))
        c.prefix_v.masked_fill_(gone, float("inf"))
    q = torch.randn(S, H, T, d, generator=g)
    at = torch.randint(0, cap, (S, H, T), generator=g) % c.lens.cpu().clamp(1, cap).repeat_interleave(H // Hk, 1)[..., None]
    near = c.k.float().cpu().repeat_interleave(H // Hk, 1).gather(2, at[..., None].expand(-1, -1, -1, d))
    q = (q + sharp * near.nan_to_num(0.0)).to(DT[dtype]).to(DEV)
    return c, q


def check(c, q, **kw):
    before = c.weight.clone()
    held = [x.clone() for x in (c.k, c.v, c.pos, c.lens)]
    out, lse = c.attend(q, **kw)
    assert c.check() == (0, 0)
    cpu = [None if x is None else x.cpu() for x in (q, c.k, c.v, c.lens, c.prefix_k, c.prefix_v, c.prefix_lens,
                                                    c.prefix_of)]
    o, e, w, bo, be, bw = O.attend(*cpu, scale=kw.get("scale"))
    O.assert_within(out, o, bo, "out")
    O.assert_within(lse, e, be, "lse")
    if kw.get("accumulate", True):
        O.assert_within(c.weight, before.double().cpu() + w, bw + 2.0 ** -23 * (before.double().cpu() + w), "weight")
    else:
        assert torch.equal(c.weight, before)
    for x, y in zip(held, (c.k, c.v, c.pos, c.lens)):
        assert torch.equal(x.view(torch.uint8) if x.is_contiguous() else x.contiguous().view(torch.uint8),
                           y.contiguous().view(torch.uint8))
    return out, lse


HEADS = [(4, 4), (4, 2), (4, 1), (7, 1), (8, 1), (16, 1), (17, 1), (40, 1), (20, 20)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", HEADS)
def test_one_token(dtype, d, H, Hk):
    lens = torch.tensor([0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 150, 149, 17, 5] * 5)[:4 * Hk].view(4, Hk)
    c, q = make(dtype, S=4, H=H, Hk=Hk, d=d, cap=150, P=70, lens=lens, seed=H * 10 + Hk)
    check(c, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,Hk,d", [(2, 4, 2, 64), (3, 7, 1, 128), (16, 2, 2, 64), (17, 2, 2, 128), (5, 8, 2, 64),
                                      (49, 4, 4, 128), (64, 4, 1, 64), (127, 2, 1, 128), (130, 3, 1, 64),
                                      (129, 2, 2, 128)])
def test_many_tokens(dtype, T, H, Hk, d):
    c, q = make(dtype, S=3, H=H, Hk=Hk, d=d, T=T, cap=T + 90, P=37, seed=T)
    check(c, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,Hk,d,P", [(1, 4, 4, 128, 2100), (1, 8, 2, 128, 4100), (4, 4, 2, 64, 4100),
                                        (2, 14, 2, 128, 3001)])
def test_long_prefixes_read_once(dtype, T, H, Hk, d, P):
    """Prefixes too long to be read again by every sequence: their rows of all
    sequences together, sequences in any order, some without a prefix."""
    S = 17
    of = [1, 0, 2, 1, 1, -1, 0, 2, 1, 0, 1, 5, 1, 0, 0, 1, 2]
    lens = torch.arange(S * Hk).view(S, Hk) * 7 % 60
    c, q = make(dtype, S=S, H=H, Hk=Hk, d=d, T=T, cap=61, G=3, P=P, plens=[P, P - 77, 0], of=of, lens=lens, seed=T)
    check(c, q)
    check(c, q, accumulate=False)


@pytest.mark.parametrize("T,H,Hk,d,P", [(1, 2, 2, 128, 4100), (1, 8, 2, 128, 4100), (4, 4, 2, 64, 8300),
                                        (2, 14, 2, 128, 4099), (16, 2, 2, 128, 4100)])
def test_more_sequences_over_long_prefixes(T, H, Hk, d, P):
    """The same with more sequences: beyond 128 MiB of prefix rows a pass, which
    bf16 caches read again up to."""
    S = 37
    assert S * Hk * P * d * 4 > 128 << 20
    of = [(i * i + i // 7) % 4 - 1 for i in range(S)]
    lens = torch.arange(S * Hk).view(S, Hk) * 7 % 60
    c, q = make("bf16", S=S, H=H, Hk=Hk, d=d, T=T, cap=61, G=3, P=P, plens=[P, P - 77, 0], of=of, lens=lens, seed=T)
    check(c, q)
    check(c, q, accumulate=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk,T", [(1, 1, 1), (2, 1, 1), (3, 1, 1), (4, 1, 1), (5, 1, 1), (8, 1, 1), (9, 1, 1), (3, 1, 3),
                                    (2, 1, 4), (10, 10, 2)])
@pytest.mark.parametrize("S", [2, 90])
def test_few_rows(dtype, d, H, Hk, T, S):
    """Every row count of the streaming kernels, with several blocks a head, one,
    and several heads a block."""
    c, q = make(dtype, S=S, H=H, Hk=Hk, d=d, T=T, cap=T + 300 if S == 2 else T + 30, G=3, P=70 if S == 2 else 9,
                plens=[70, 33, 0] if S == 2 else [9, 4, 0], seed=H + T, slot_major=T == 3)
    check(c, q)


@pytest.mark.parametrize("dtype,S,H,Hk,T", [("bf16", 10, 16, 16, 20), ("bf16", 37, 4, 2, 130), ("bf16", 1, 2, 1, 300),
                                            ("f32", 10, 16, 16, 20), ("f32", 1, 3, 1, 150)])
def test_many_rows_one_pass(dtype, S, H, Hk, T):
    """Enough row tiles for whole key lists, and more rows of a head than one
    block holds: outputs final, weights by the blocks or in a pass of their own."""
    c, q = make(dtype, S=S, H=H, Hk=Hk, d=64, T=T, cap=T + 33, G=2, P=30, seed=S)
    check(c, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_rows_that_see_nothing(dtype, T):
    """No prefix (an index outside the prefixes, a length of zero) and fewer
    own tokens than queries: zeros and -inf, no weight."""
    c, q = make(dtype, S=5, H=4, Hk=2, T=T, cap=64, G=3, P=16, plens=[16, 0, -4], of=[0, 1, 2, -1, 7],
                lens=[[0, 1], [0, 2], [3, 0], [0, 64], [1, 0]])
    out, lse = check(c, q)
    assert (out[3, :2] == 0).all() and torch.isneginf(lse[3, :2]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 33])
def test_lengths_out_of_range_are_clamped(dtype, T):
    c, q = make(dtype, S=3, H=2, Hk=1, T=T, cap=48, G=1, P=16, lens=48)
    c.lens.copy_(torch.tensor([[48], [1000000], [48]]))
    c.prefix_lens.fill_(1 << 30)
    c.prefix_k.normal_()
    c.prefix_v.normal_()
    check(c, q)
    c.lens.fill_(-7)
    c.prefix_lens.fill_(-1)
    out, lse = c.attend(q)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 20])
def test_no_prefixes_scale_no_accumulation(dtype, T):
    c, q = make(dtype, G=0, T=T, cap=100, d=128)
    check(c, q, scale=0.3)
    check(c, q, accumulate=False)
    check(c, q, scale=-0.05)


@pytest.mark.parametrize("T", [1, 3, 50])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides(dtype, T):
    """Slot-major caches, queries and outputs as slices of wider tensors."""
    c, q = make(dtype, S=3, H=6, Hk=3, T=T, cap=70, slot_major=True, d=64)
    wide = torch.zeros(3, T, 6, 3 * 64, dtype=q.dtype, device=DEV)
    wide[..., 64:128] = q.transpose(1, 2)
    out = torch.full_like(wide, 7.0)
    view = out[..., 64:128].transpose(1, 2)
    check(c, wide[..., 64:128].transpose(1, 2), out=view)
    assert (out[..., :64] == 7).all() and (out[..., 128:] == 7).all()


@pytest.mark.parametrize("T", [1, 2, 24])
def test_offsets_past_32_bits(T):
    """Slots 2^26 elements apart: the last ones lie beyond 2^31 elements."""
    d, n = 64, 40
    base_k = torch.empty(n << 26, dtype=torch.bfloat16, device=DEV)
    k = base_k.as_strided((1, 1, n, d), (n << 26, n << 26, 1 << 26, 1))
    v = base_k[4096:].as_strided((1, 1, n, d), (n << 26, n << 26, 1 << 26, 1))
    g = torch.Generator().manual_seed(3)
    k.copy_(torch.randn(1, 1, n, d, generator=g))
    v.copy_(torch.randn(1, 1, n, d, generator=g))
    c = hkv.SharedPrefixCache(hkv.SharedConfig(1, 2, 1, d, n), DEV, k=k, v=v)
    c.lens.fill_(n - T)
    c.append(torch.randn(1, 1, T, d, generator=g).bfloat16().to(DEV), torch.randn(1, 1, T, d, generator=g).bfloat16().to(DEV))
    q = torch.randn(1, 2, T, d, generator=g).bfloat16().to(DEV)
    check(c, q)
    last = c.k[0, 0, n - 1].clone()
    c.weight.zero_()
    c.weight[0, 0, n - 1] = 5.0
    c.pos.copy_(torch.arange(n).view(1, 1, n))
    c.evict(torch.full((1, 1), 3, dtype=torch.int32, device=DEV))
    assert c.lens.item() == 3 and torch.equal(c.k[0, 0, :3], torch.stack([c.k[0, 0, n - 3], c.k[0, 0, n - 2], last]))


@pytest.mark.parametrize("dtype,sharp", [("bf16", 3.0), ("f32", 3.0), ("bf16", 0.0)])
@pytest.mark.parametrize("T", [1, 40])
def test_sharp_and_flat_rows(dtype, sharp, T):
    c, q = make(dtype, S=2, H=4, Hk=2, T=T, cap=700, G=1, P=600, sharp=sharp, d=128, lens=700)
    check(c, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_places_may_hold_the_lowest_value(dtype):
    """Logits of the type's lowest value and of -inf: no weight, no NaN."""
    c, q = make(dtype, S=1, H=1, Hk=1, cap=20, G=0, lens=20, d=64)
    c.k.normal_()
    c.v.normal_()
    q.fill_(1.0)
    c.k[0, 0, 3] = torch.finfo(c.k.dtype).min          # a logit of -inf
    c.k[0, 0, 5, 0] = -float("inf")
    out, lse = c.attend(q, accumulate=False)
    keep = [i for i in range(20) if i not in (3, 5)]
    x = c.k[0, 0, keep].double() @ q[0, 0, 0].double() / 8
    want = x.softmax(0) @ c.v[0, 0, keep].double()
    assert torch.allclose(out[0, 0, 0].double(), want, rtol=0.02, atol=0.02)
    # a row of -inf logits alone is an empty row
    c.k.fill_(-float("inf"))
    out, lse = c.attend(q, accumulate=False)
    assert (out == 0).all() and torch.isneginf(lse).all()
    # a NaN in a held token reaches its sequence's queries
    c.k.normal_()
    c.k[0, 0, 7] = float("nan")
    out, lse = c.attend(q, accumulate=False)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 20, 40, 130, 600])
def test_infinite_keys_take_no_weight(dtype, T):
    """A key whose logits are all -inf: no weight, and none becomes NaN, whatever
    the row tiles' ends hold (the sums of many rows are formed in whole tiles)."""
    c, q = make(dtype, S=2, H=2, Hk=1, T=T, cap=T + 70, G=1, P=40, lens=T + 70)
    q[..., 0] = q[..., 0].abs() + 0.5
    x, y = c.k.clone(), c.weight.clone()
    c.k[:, :, 5, 0] = -float("inf")
    out, lse = c.attend(q)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert torch.isfinite(c.weight).all() and torch.equal(c.weight[:, :, 5], y[:, :, 5])
    # the same as without it: a logit far below the others
    c.k.copy_(x)
    c.k[:, :, 5] = 0
    c.k[:, :, 5, 0] = -1e6
    w = c.weight.clone()
    c.weight.copy_(y)
    out2, lse2 = c.attend(q)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(w, c.weight)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 20, 130, 600])
@pytest.mark.parametrize("big", [2.0 ** 30, 2.0 ** 100])
def test_logits_far_from_zero(dtype, T, big):
    """Every visible logit near +-big or exactly there: the largest take all the
    weight, shared alike, however large the numbers (2^24 on, fp32 no longer
    holds the logits' fractions).  Powers of two, so that nothing rounds."""
    S, d, n = 1, 64, T + 40
    c, _ = make(dtype, S=S, H=2, Hk=1, T=T, cap=n, G=0, d=d, lens=n)
    g = torch.Generator().manual_seed(T)
    c.v.copy_(torch.randn(c.v.shape, generator=g))
    q = torch.zeros(S, 2, T, d, dtype=DT[dtype], device=DEV)
    q[..., 0] = 1
    for sign in (1.0, -1.0):
        # all alike: the mean of what a query sees
        c.k.zero_()
        c.k[..., 0] = sign * big
        c.weight.zero_()
        out, lse = c.attend(q)
        v = c.v[0, 0].double()
        see = n - T + 1 + torch.arange(T, device=DEV)
        want = v.cumsum(0)[see - 1] / see[:, None]
        bound = 2.0 ** -7 * v.abs().cumsum(0)[see - 1] / see[:, None] + 1e-6
        assert ((out[0].double() - want).abs() <= bound).all()
        assert torch.allclose(lse.double(), torch.full_like(lse, sign * big / 8).double(), rtol=1e-6)
        assert torch.isfinite(c.weight).all() and (c.weight >= 0).all() and (c.weight <= 2 * T).all()
        # the third key twice as large: all of the weight
        c.k[0, 0, 2, 0] = sign * big * (2 if sign > 0 else 0.5)
        c.weight.zero_()
        out, lse = c.attend(q)
        assert ((out[0].double() - v[2]).abs() <= 2.0 ** -8 * v[2].abs()).all()
        assert (c.weight[0, 0, [0, 1, 3]] == 0).all() and 0 <= float(c.weight[0, 0, 2]) <= 2 * T


def test_same_bits_twice():
    for T in (1, 6, 60):
        c, q = make("bf16", S=4, H=8, Hk=2, T=T, cap=500, P=300, d=128)
        w0 = c.weight.clone()
        a, la = c.attend(q)
        wa = c.weight.clone()
        c.weight.copy_(w0)
        b, lb = c.attend(q)
        assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(wa, c.weight)


# -- append --------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,cap", [(1, 5), (3, 40), (200, 300), (1500, 1501)])
def test_append(dtype, T, cap):
    g = torch.Generator().manual_seed(T)
    S, Hk, d = 3, 2, 64
    c, _ = make(dtype, S=S, H=2, Hk=Hk, d=d, cap=cap, G=0, lens=0)
    c.lens.copy_(torch.tensor([[0, 1], [cap - T, cap - T + 1], [cap, 0]]))
    c.next_pos.copy_(torch.tensor([[0, 5], [9, 100], [1 << 30, -3]]))
    src = rows(g, dtype, S, Hk, T, 2 * d, slot_major=True)
    kt, vt = src[..., :d], src[..., d:]
    wt = torch.rand(S, Hk, T, generator=g).to(DEV)
    want = [x.clone() for x in (c.k, c.v, c.pos, c.weight, c.lens, c.next_pos)]
    for s in range(S):
        for h in range(Hk):
            n = int(c.lens[s, h])
            if n + T > cap:
                continue
            want[0][s, h, n:n + T], want[1][s, h, n:n + T], want[3][s, h, n:n + T] = kt[s, h], vt[s, h], wt[s, h]
            want[2][s, h, n:n + T] = torch.arange(T, device=DEV) + c.next_pos[s, h]
            want[4][s, h] += T
            want[5][s, h] += T
    c.append(kt, vt, wt)
    for x, y in zip(want, (c.k, c.v, c.pos, c.weight, c.lens, c.next_pos)):
        assert torch.equal(x.nan_to_num(-5.0), y.nan_to_num(-5.0))
    code, detail = c.check()
    assert code == 3 and detail in (3, 4) + ((1,) if cap == T + 1 else ())
    c.clear_error()
    c.lens.zero_()
    c.append(kt, vt)
    assert (c.weight[..., :T] == 0).all() and c.check() == (0, 0)
    c.append(kt[:, :, :0], vt[:, :, :0])  # nothing


# -- evict ---------------------------------------------------------------------

def evict_both(c, budgets, recent, slack):
    b = torch.as_tensor(budgets, dtype=torch.int32).expand(c.lens.shape).contiguous().to(DEV)
    want = [x.cpu().float().numpy() if x.dtype == torch.bfloat16 else x.cpu().numpy()
            for x in (c.k.contiguous(), c.v.contiguous(), c.pos, c.weight, c.lens)]
    want = [x.copy() for x in want]
    O.evict(*want, b.cpu().numpy(), recent, slack)
    c.evict(b, recent, slack)
    for name, x, y in zip(("k", "v", "pos", "weight", "lens"), want, (c.k, c.v, c.pos, c.weight, c.lens)):
        np.testing.assert_array_equal(y.cpu().float().numpy() if y.dtype == torch.bfloat16 else y.cpu().numpy(), x,
                                      err_msg=name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cap,budget,recent,slack", [(20, 10, 3, 1), (20, 10, 3, 5), (33, 32, 0, 1), (150, 100, 28, 32),
                                                     (600, 413, 56, 64), (64, 0, 5, 1), (64, 5, 40, 1), (1, 0, 0, 1),
                                                     (300, 299, 300, 1), (1025, 512, 0, 1), (5000, 1300, 100, 7)])
def test_evict(dtype, cap, budget, recent, slack):
    g = torch.Generator().manual_seed(cap)
    S, Hk = 3, 3
    c, _ = make(dtype, S=S, H=Hk, Hk=Hk, d=64, cap=cap, G=0, lens=cap, slot_major=cap % 2 == 0)
    c.lens.copy_(torch.randint(0, cap + 1, (S, Hk), generator=g))
    c.lens.view(-1)[:4] = torch.tensor([cap, min(cap, budget + slack), max(0, min(cap, budget + slack - 1)), 0],
                                       dtype=torch.int32)
    c.pos.copy_(torch.argsort(torch.rand(S, Hk, cap, generator=g), -1))
    b = torch.randint(0, budget + 1, (S, Hk), generator=g)
    b[0] = budget
    for _ in range(2):  # the second finds little or nothing due
        evict_both(c, b, recent, slack)


def test_evict_very_long():
    """A head whose weights and positions do not fit shared memory."""
    g = torch.Generator().manual_seed(1)
    cap = 30001
    c, _ = make("bf16", S=1, H=2, Hk=2, d=64, cap=cap, G=0, lens=cap)
    c.pos.copy_(torch.argsort(torch.rand(1, 2, cap, generator=g), -1))
    c.weight[0, 1] = c.weight[0, 1].round(decimals=3)  # ties
    evict_both(c, [[20000, 29000]], 500, 1)


@pytest.mark.parametrize("cap", [48, 700, 3000])
def test_evict_ties_and_odd_values(cap):
    """Equal weights, signed zeros, infinities, NaN, negative weights;
    positions repeated, negative, at the ends of the type."""
    g = torch.Generator().manual_seed(cap)
    S, Hk = 4, 2
    c, _ = make("bf16", S=S, H=Hk, Hk=Hk, d=64, cap=cap, G=0, lens=cap)
    vals = torch.tensor([0.0, -0.0, 1.0, 1.0, float("inf"), -float("inf"), float("nan"), -2.5, 1e-42, -1e-42])
    c.weight.copy_(vals[torch.randint(0, 10, (S, Hk, cap), generator=g)])
    c.weight[1] = 0.5
    c.weight[2] = float("nan")
    ps = torch.tensor([0, 0, -5, 7, 2 ** 31 - 1, -2 ** 31, 100, 2 ** 31 - 2])
    c.pos.copy_(ps[torch.randint(0, 8, (S, Hk, cap), generator=g)])
    c.pos[3] = 4
    for recent in (0, 1, 3, 2 ** 31 - 1):
        c.lens.fill_(cap)
        evict_both(c, [[cap // 3, cap - 1]] * S, recent, 1)


def test_evict_budgets_out_of_range():
    c, _ = make("f32", S=2, H=2, Hk=2, cap=30, G=0, lens=30)
    evict_both(c, [[-5, 2 ** 31 - 1], [31, 30]], 4, 2 ** 31 - 1)   # nothing is due
    c.lens.fill_(1000)                                            # taken as the capacity
    evict_both(c, [[-5, 2 ** 31 - 1], [12, 29]], 4, 1)


# -- as they are used together -------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 4])
def test_generation_run(dtype, T):
    """Prompts shared, a prefill, then steps of append, attend and evict:
    every call against the restatement on the state it found."""
    g = torch.Generator().manual_seed(5)
    S, H, Hk, d, P, budget, steps = 4, 4, 2, 64, 24, 20, 9
    c, _ = make(dtype, S=S, H=H, Hk=Hk, d=d, cap=64, P=P, lens=0)
    c.weight.zero_()
    b = torch.full((S, Hk), budget, dtype=torch.int32, device=DEV)
    b[1, 0] = 12
    for n in [30] + [T] * steps:
        kt, vt = rows(g, dtype, S, Hk, n, d), rows(g, dtype, S, Hk, n, d)
        c.append(kt, vt)
        check(c, rows(g, dtype, S, H, n, d))
        evict_both(c, b, 6, 1)
        assert torch.equal(c.lens, b)
    assert (c.next_pos == 30 + T * steps).all() and (c.pos[0, 0, :budget] >= 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,T,P", [(4, 1, 70), (16, 1, 4200), (4, 20, 70)])
def test_captured_step_replays(dtype, S, T, P):
    """append + attend + evict captured once and replayed equals eager steps;
    two graphs of one cache hold their own scratch."""
    g = torch.Generator().manual_seed(6)
    make_one = lambda: make(dtype, S=S, H=8, Hk=4, d=128, cap=56, P=P, lens=32, seed=9)[0]  # noqa: E731
    c, e = make_one(), make_one()
    q = rows(g, dtype, S, 8, T, 128)
    kt, vt = rows(g, dtype, S, 4, T, 128), rows(g, dtype, S, 4, T, 128)
    b = torch.full((S, 4), 32, dtype=torch.int32, device=DEV)

    def step(x):
        x.append(kt, vt)
        r = x.attend(q)
        x.evict(b, 8)
        return r

    parts = lambda x: (x.k, x.v, x.pos, x.weight, x.lens, x.next_pos)  # noqa: E731
    state = [t.clone() for t in parts(c)]
    with torch.cuda.stream(torch.cuda.Stream()):
        step(c)
    torch.cuda.synchronize()
    for t, x in zip(parts(c), state):
        t.copy_(x)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(c)
    q2 = rows(g, dtype, S, 8, T, 128)
    with torch.cuda.graph(other):
        out2, _ = c.attend(q2, accumulate=False)
    for i in range(5):
        kt.normal_()
        graph.replay()
        other.replay()
        want, wl = step(e)
        want2, _ = e.attend(q2, accumulate=False)
        assert torch.equal(out, want) and torch.equal(lse, wl) and torch.equal(out2, want2), i
    for a, x in zip(parts(c), parts(e)):
        assert torch.equal(a.nan_to_num(-1.0), x.nan_to_num(-1.0))


@pytest.mark.parametrize("S,T,P,cap", [(8, 1, 2000, 3000), (24, 1, 4000, 300), (36, 1, 4000, 300), (3, 40, 500, 900)])
def test_several_streams_at_once(S, T, P, cap):
    """Calls that only read the cache may overlap: each has its own scratch."""
    c, q = make("bf16", S=S, H=8, Hk=2, d=128, T=T, cap=cap, P=P, lens=cap)
    want, wl = c.attend(q, accumulate=False)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [c.attend(q, accumulate=False, stream=streams[i % 3] if i % 2 else streams[i % 3].cuda_stream)
            for i in range(30)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(e, wl) for o, e in outs)


def test_default_stream_by_handle_and_from_another_thread():
    import threading
    c, q = make("bf16", S=4, H=8, Hk=2, d=128, cap=200, P=90, lens=200)
    want, _ = c.attend(q, accumulate=False)
    got = [None] * 8

    def work(i):
        for _ in range(20):
            got[i] = c.attend(q, accumulate=False, stream=0 if i % 2 else None)[0]

    ts = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


def test_python_refusals():
    c, q = make("bf16", S=3, H=4, Hk=2, d=64, cap=20)
    kt = c.k[:, :, :2].contiguous()
    with pytest.raises(ValueError):
        c.attend(q.float())
    with pytest.raises(ValueError):
        c.attend(q.cpu())
    with pytest.raises(ValueError):
        c.attend(q[:, :2])
    with pytest.raises(ValueError):
        c.attend(q.expand(3, 4, 21, 64))
    with pytest.raises(ValueError):
        c.attend(q[:, :, :0])
    with pytest.raises(ValueError):
        c.attend(q, out=q[:1].expand(3, 4, 1, 64))
    with pytest.raises(ValueError, match="not q itself"):
        c.attend(q, out=q)
    with pytest.raises(ValueError):
        c.attend(q, lse=torch.empty(3, 4, 2, device=DEV))
    for s in (0, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            c.attend(q, scale=s)
    off = torch.zeros(3 * 4 * 64 + 8, dtype=torch.bfloat16, device=DEV)[1:769].view(3, 4, 1, 64)
    with pytest.raises(ValueError, match="16-byte"):
        c.attend(off)
    with pytest.raises(ValueError):
        c.append(kt, kt[:, :, :1])
    with pytest.raises(ValueError):
        c.append(kt, kt, torch.zeros(3, 2, 3, device=DEV))
    with pytest.raises(ValueError):
        c.evict(torch.zeros(3, 2, device=DEV))
    ok = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        c.evict(ok, -1)
    with pytest.raises(ValueError):
        c.evict(ok, 0, 0)
    for far in (1 << 31, 1 << 32):
        with pytest.raises(ValueError):
            c.evict(ok, far)
        with pytest.raises(ValueError):
            c.evict(ok, 0, far)
    with pytest.raises(ValueError):
        hkv.SharedPrefixCache(c.cfg, DEV, k=c.k[..., :32])
    with pytest.raises(ValueError):
        hkv.SharedPrefixCache(c.cfg, DEV, pos=c.weight)
    for kw in (dict(head_dim=96), dict(num_heads=5), dict(capacity=0), dict(num_prefixes=1, prefix_capacity=0)):
        with pytest.raises(ValueError):
            hkv.SharedPrefixCache(hkv.SharedConfig(**{**dict(num_seqs=2, num_heads=4, num_kv_heads=2, head_dim=64,
                                                             capacity=32), **kw}), DEV)
    assert isinstance(c._c.k, int) and C.sizeof(c._c) > 0
