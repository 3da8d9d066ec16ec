"""The shared-prefix cache on the GPU at the ends of its ranges: infinities, the
largest sizes, shapes of block that only large calls reach."""
import math

import pytest
import torch

import kv_cache_compression_hkv_b200 as hkv

import shared_oracle as O
from test_shared_gpu import DEV, check, evict_both, make, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_compression_hkv_b200 import build
    build.build()
    assert torch.cuda.is_available(), "these tests need a CUDA device"


# (S, H, Hk, T, own slots, prefix slots): every kernel, final results and pieces
SHAPES = [(2, 4, 4, 1, 500, 100), (300, 4, 4, 1, 40, 20), (3, 12, 1, 1, 900, 100), (80, 32, 2, 1, 50, 33),
          (40, 2, 2, 1, 60, 4100), (2, 4, 2, 10, 900, 100), (3, 2, 1, 400, 700, 100), (20, 8, 8, 49, 90, 30),
          (2, 8, 1, 100, 140, 100)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,H,Hk,T,n,P", SHAPES)
@pytest.mark.parametrize("where", ["own", "prefix"])
def test_infinite_values_give_infinities(dtype, S, H, Hk, T, n, P, where):
    """A value of +-inf that every query sees, with a weight above zero: that
    infinity, in its column alone; both signs in one column: NaN."""
    c, q = make(dtype, S=S, H=H, Hk=Hk, T=T, cap=n, G=1, P=P, plens=[P], of=[0] * S, lens=n, seed=n, sharp=0.0)
    v = c.v if where == "own" else c.prefix_v
    v[:, :, 0, 3] = float("inf")
    v[:, :, 5, 3] = float("inf")
    v[:, :, 7, 4] = -float("inf")
    v[:, :, 1, 5] = -float("inf")
    v[:, :, 2, 5] = float("inf")
    out, lse = c.attend(q)
    assert c.check() == (0, 0)
    assert torch.isposinf(out[..., 3]).all() and torch.isneginf(out[..., 4]).all() and torch.isnan(out[..., 5]).all()
    for x in (out[..., :3], out[..., 6:], lse, c.weight):
        assert torch.isfinite(x).all()


def test_weights_of_heads_past_32_bits_of_slots_times_rows():
    """512 query rows a head over more than 2^22 slots: slot x row is beyond 2^31,
    and every row's weight arrives.  All keys alike, so that each slot receives
    512 / n: to 2^-21 for the exponential, 22 half steps of fp32 for the
    logarithm of the sum and at most 512 for the sums, 4e-5 in all."""
    S, rep, n, d = 37, 512, (1 << 22) + 200, 64
    k = torch.zeros(S, 1, n, d, dtype=torch.bfloat16, device=DEV)
    c = hkv.SharedPrefixCache(hkv.SharedConfig(S, rep, 1, d, n), DEV, k=k, v=k)
    c.lens.fill_(n)
    q = torch.randn(S, rep, 1, d, device=DEV).bfloat16()
    out, lse = c.attend(q)
    assert c.check() == (0, 0)
    assert not out.any() and ((lse - math.log(n)).abs() < 1e-5).all()
    assert ((c.weight * (n / rep) - 1).abs() < 4e-5).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cap", [1025, 1400, 2048])
def test_evict_many_heads_of_many_moves(dtype, cap):
    """More heads than SMs of up to 2048 slots: small blocks that move their own
    rows, up to 512 of them from lists in shared memory, more from the scratch."""
    S, Hk = 19, 8
    g = torch.Generator().manual_seed(cap)
    c, _ = make(dtype, S=S, H=Hk, Hk=Hk, d=64, cap=cap, G=0, lens=cap, seed=cap)
    c.pos.copy_(torch.argsort(torch.rand(S, Hk, cap, generator=g), -1))
    b = torch.randint(cap // 2 - 100, cap // 2 + 100, (S, Hk), generator=g)
    c.lens[3:7] = torch.randint(0, cap + 1, (4, Hk), generator=g).to(DEV)
    # exactly so many moves: light tokens before the budget, and all but as many behind it
    for h, moves in enumerate((0, 1, 511, 512, 513, cap - (cap + 1) // 2)):
        moves = min(moves, cap // 2)
        b[7, h] = (cap + 1) // 2
        w = torch.full((cap,), 2.0)
        w[:moves] = 1.0                                        # holes
        w[(cap + 1) // 2 + moves:] = 1.0                       # gone in place
        c.weight[7, h] = w
    evict_both(c, b, 0, 1)
    assert torch.equal(c.lens[7].cpu(), b[7].int())
    evict_both(c, b // 2, 5, 3)


def test_outputs_in_memory_of_inputs_are_refused():
    """out or lse sharing bytes with q, each other or the cache; slices beside
    q's in one tensor are fine."""
    S, H, Hk, T, d, n = 3, 4, 2, 2, 64, 40
    c, q0 = make("bf16", S=S, H=H, Hk=Hk, T=T, d=d, cap=n, lens=n)
    want, wl = c.attend(q0, accumulate=False)
    wide = torch.zeros(S, T, H, 3 * d, dtype=torch.bfloat16, device=DEV)
    q, out = wide[..., d:2 * d].transpose(1, 2), wide[..., 2 * d:].transpose(1, 2)
    q.copy_(q0)
    got, lse = c.attend(q, out=out, accumulate=False)
    assert got is out and torch.equal(out, want) and torch.equal(lse, wl)
    before = [x.clone() for x in c._buffers]
    k = c.k.view(-1)[:S * H * T * d].view(S, H, T, d)
    bad = [dict(out=wide[..., d + 8:2 * d + 8].transpose(1, 2)), dict(out=k),
           dict(out=c.prefix_v.view(-1)[-S * H * T * d:].view(S, H, T, d)),
           dict(lse=c.weight.view(-1)[:S * H * T].view(S, H, T)),
           dict(out=out, lse=wide.view(torch.float32).view(-1)[-S * H * T:].view(S, H, T)),
           dict(lse=wide.view(torch.float32).view(-1)[d // 2:d // 2 + S * H * T].view(S, H, T))]
    for kw in bad:
        with pytest.raises(ValueError, match="overlaps"):
            c.attend(q, accumulate=False, **kw)
    for x, y in zip(before, c._buffers):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_inputs_that_ask_for_a_gradient_are_refused(dtype):
    c, q = make(dtype, S=2, H=4, Hk=2, T=2, cap=20, lens=10)
    kt = torch.randn(2, 2, 2, 64, device=DEV).to(q.dtype)
    wt = torch.rand(2, 2, 2, device=DEV)
    lens = c.lens.clone()
    with pytest.raises(ValueError, match="q: .*gradient"):
        c.attend(q.clone().requires_grad_())
    with pytest.raises(ValueError, match="k_t: .*gradient"):
        c.append(kt.clone().requires_grad_(), kt)
    with pytest.raises(ValueError, match="v_t: .*gradient"):
        c.append(kt, kt.clone().requires_grad_() * 2)
    with pytest.raises(ValueError, match="weight_t: .*gradient"):
        c.append(kt, kt, wt.clone().requires_grad_())
    with pytest.raises(ValueError, match="out: .*gradient"):
        c.attend(q, out=torch.empty_like(q).requires_grad_())
    with pytest.raises(ValueError, match="prefix_v: .*gradient"):
        hkv.SharedPrefixCache(c.cfg, DEV, prefix_v=c.prefix_v.clone().requires_grad_())
    assert torch.equal(c.lens, lens)
    want, _ = c.attend(q, accumulate=False)
    with torch.no_grad():
        got, _ = c.attend(q.clone().requires_grad_(), accumulate=False)
        c.append(kt.clone().requires_grad_(), kt, wt.clone().requires_grad_())
    assert torch.equal(got, want) and not got.requires_grad


@pytest.mark.parametrize("G", [0, 2])
def test_buffers_cannot_be_replaced(G):
    """The calls go on using the buffers the cache was made over: assigning
    another tensor to the attribute says so.  In place is fine."""
    c, q = make("bf16", S=2, H=4, Hk=2, cap=20, G=G, lens=10)
    for name in ("k", "v", "pos", "weight", "lens", "next_pos", "status") + ("prefix_k", "prefix_v", "prefix_lens",
                                                                             "prefix_of"):
        x = getattr(c, name)
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, torch.zeros(1, device=DEV) if x is None else x.clone())
        assert getattr(c, name) is x
    c.weight *= 2
    c.lens += 1
    c.lens = c.lens
    c.attend(q)


def test_a_config_may_change_behind_the_cache():
    """Sizes are checked against those the cache was made with, whatever becomes
    of the config it was given and of the one it shows."""
    cfg = hkv.SharedConfig(3, 4, 2, 64, 20)
    c = hkv.SharedPrefixCache(cfg, DEV)
    c.lens.fill_(5)
    c.k.normal_()
    c.v.normal_()
    q = torch.randn(3, 4, 2, 64, device=DEV).bfloat16()
    want, _ = c.attend(q, accumulate=False)
    for shown in (cfg, c.cfg):
        shown.num_seqs, shown.num_heads, shown.num_kv_heads, shown.capacity = 1, 2, 1, 4
        assert shown is cfg and c.cfg.num_seqs == 3 or shown is c.cfg
        with pytest.raises(ValueError):
            c.attend(q[:1, :2].contiguous())
        with pytest.raises(ValueError):
            c.append(c.k[:1, :1, :2].clone(), c.v[:1, :1, :2].clone())
        with pytest.raises(ValueError):
            c.evict(torch.zeros(1, 1, dtype=torch.int32, device=DEV))
        assert torch.equal(c.attend(q, accumulate=False)[0], want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 40, 150])
def test_prompts_are_filled_by_a_cache_over_them(dtype, T):
    """The prompts' prefill through a cache whose own buffers they are, the
    shorter one padded, and then sequences that continue them."""
    S, H, Hk, d, P = 4, 4, 2, 64, 160
    g = torch.Generator().manual_seed(T)
    c, q = make(dtype, S=S, H=H, Hk=Hk, d=d, T=2, cap=30, G=2, P=P, plens=[0, 0], lens=20, seed=T)
    prompts = hkv.SharedPrefixCache(hkv.SharedConfig(2, H, Hk, d, P, dtype=c.cfg.dtype), DEV, k=c.prefix_k, v=c.prefix_v)
    kt, vt, qt = rows(g, dtype, 2, Hk, T, d), rows(g, dtype, 2, Hk, T, d), rows(g, dtype, 2, H, T, d)
    prompts.append(kt, vt)
    out, lse = prompts.attend(qt, accumulate=False)
    lens = [T, T // 2]
    c.prefix_lens.copy_(torch.tensor(lens))
    for i, n in enumerate(lens):
        o, e, _, bo, be, _ = O.attend(qt[i:i + 1, :, :n].cpu(), kt[i:i + 1].cpu(), vt[i:i + 1].cpu(),
                                      torch.full((1, Hk), n), None, None, None, None)
        O.assert_within(out[i:i + 1, :, :n], o, bo, "out")
        O.assert_within(lse[i:i + 1, :, :n], e, be, "lse")
    assert torch.equal(c.prefix_k[:, :, :T], kt) and torch.equal(c.prefix_v[:, :, :T], vt)
    check(c, q)


@pytest.mark.parametrize("by_handle", [False, True])
def test_errors_of_calls_on_another_stream(by_handle):
    """check waits for the stream it is given, as the calls go to it: an append
    without room, held up by 50 ms of other work."""
    c, _ = make("bf16", S=2, H=4, Hk=2, cap=20, lens=20)
    kt = torch.randn(2, 2, 1, 64, device=DEV).bfloat16()
    side = torch.cuda.Stream()
    at = side.cuda_stream if by_handle else side
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    c.append(kt, kt, stream=at)
    code, detail = c.check(stream=at)
    assert code == 3 and detail in range(4)
    c.clear_error(stream=at)
    assert c.check(stream=at) == (0, 0)
    assert c.check() == (0, 0) and c.check(stream=0) == (0, 0)
