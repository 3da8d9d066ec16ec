"""Host-side checks of the shared-prefix cache's C calls: every refusal comes
before anything is enqueued, and the scratch sizes are what the sizes say."""
import ctypes as C

import numpy as np
import pytest
import torch

import kv_cache_compression_hkv_b200 as hkv
from kv_cache_compression_hkv_b200 import build
from kv_cache_compression_hkv_b200.shared import _Cache

import shared_oracle as O

ST = C.c_int64 * 3


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def cache(**kw):
    """A well-formed descriptor over addresses that nothing reads."""
    S, H, Hk, cap, d, G, P = 4, 8, 2, 96, 64, 2, 40
    c = _Cache(hkv.DTYPE_BF16, d, S, H, Hk, cap, G, P)
    for i, n in enumerate(("k", "v", "pos", "weight", "len", "next_pos", "prefix_k", "prefix_v", "prefix_len",
                           "prefix_of", "status")):
        setattr(c, n, 0x10000 * (i + 1))
    for n in ("k_stride", "v_stride"):
        setattr(c, n, ST(Hk * cap * d, cap * d, d))
    for n in ("prefix_k_stride", "prefix_v_stride"):
        setattr(c, n, ST(Hk * P * d, P * d, d))
    for n, x in kw.items():
        setattr(c, n, x)
    return c


BAD = [dict(dtype=2), dict(head_dim=96), dict(num_seqs=0), dict(num_heads=7), dict(num_heads=0), dict(num_kv_heads=0),
       dict(num_kv_heads=-2), dict(capacity=0), dict(capacity=1 << 25), dict(num_prefixes=-1), dict(num_prefixes=1025),
       dict(prefix_capacity=0), dict(prefix_capacity=1 << 25), dict(k=None), dict(v=0x10008), dict(len=None),
       dict(len=0x10002), dict(prefix_k=None), dict(prefix_v=0x10001), dict(prefix_len=None), dict(prefix_of=None),
       dict(k_stride=ST(0, 64, 4)), dict(v_stride=ST(12288, 6144, 60)), dict(k_stride=ST(12288, -6144, 64)),
       dict(prefix_k_stride=ST(5120, 2560, 68 + 1)), dict(v_stride=ST(12288, 0, 64)), dict(prefix_v_stride=ST(0, 2560, 64)), dict(pos=0x10002), dict(status=0x10001),
       dict(num_seqs=1 << 30)]


@pytest.mark.parametrize("kw", BAD, ids=[str(sorted(b)[0]) + str(i) for i, b in enumerate(BAD)])
def test_bad_cache_refused_by_every_call(kw):
    L, c, n = hkv.lib(), cache(**kw), C.c_size_t()
    r, st = C.byref(c), ST(512, 64, 64)
    assert L.hkv_shared_attend_bytes(r, 1, 1, C.byref(n)) == 1
    assert L.hkv_shared_evict_bytes(r, C.byref(n)) == 1
    assert L.hkv_shared_append(r, 0x1000, st, 0x2000, st, None, 1, None) == 1
    assert L.hkv_shared_attend(r, 0x1000, st, 0x2000, st, None, 1, 0.0, 1, 0x1000, 1 << 40, None) == 1
    assert L.hkv_shared_evict(r, 0x1000, 0, 1, 0x1000, 1 << 40, None) == 1


def test_bad_arguments_refused():
    L, c, n = hkv.lib(), cache(), C.c_size_t()
    r, st, odd = C.byref(c), ST(512, 64, 64), ST(512, 64, 60)
    assert L.hkv_shared_attend_bytes(None, 1, 1, C.byref(n)) == 1
    for T, acc in ((0, 1), (97, 1), (-1, 0), (1, 2)):
        assert L.hkv_shared_attend_bytes(r, T, acc, C.byref(n)) == 1
    assert L.hkv_shared_attend_bytes(r, 1, 1, None) == 1
    # append
    for a in ((None, st, 0x2000, st, None, 1), (0x1000, None, 0x2000, st, None, 1), (0x1008, st, 0x2000, st, None, 1),
              (0x1000, odd, 0x2000, st, None, 1), (0x1000, st, 0x2000, st, 0x3001, 1),
              (0x1000, st, 0x2000, st, None, 97), (0x1000, st, 0x2000, st, None, -1)):
        assert L.hkv_shared_append(r, *a, None) == 1
    assert L.hkv_shared_append(r, 0x1000, st, 0x2000, st, None, 0, None) == 0  # nothing to do
    # attend
    ok = dict(q=0x1000, qs=st, out=0x2000, os=st, lse=None, T=1, scale=0.0, acc=1, ws=0x10000, n=1 << 40)
    for kw, code in ((dict(q=None), 1), (dict(q=0x1004), 1), (dict(qs=odd), 1), (dict(qs=None), 1), (dict(out=None), 1),
                     (dict(os=odd), 1), (dict(lse=0x1001), 1), (dict(T=0), 1), (dict(T=97), 1),
                     (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=1e-40), 1), (dict(scale=-1e40), 1), (dict(acc=2), 1), (dict(ws=None), 1),
                     (dict(ws=0x10010), 1), (dict(n=16), 3)):
        a = {**ok, **kw}
        assert L.hkv_shared_attend(r, a["q"], a["qs"], a["out"], a["os"], a["lse"], a["T"], a["scale"], a["acc"],
                                   a["ws"], a["n"], None) == code, kw
    bare = cache(weight=None)
    assert L.hkv_shared_attend(C.byref(bare), 0x1000, st, 0x2000, st, None, 1, 0.0, 1, 0x10000, 1 << 40, None) == 1
    # evict
    for a, code in (((None, 0, 1, 0x10000, 1 << 40), 1), ((0x1002, 0, 1, 0x10000, 1 << 40), 1),
                    ((0x1000, -1, 1, 0x10000, 1 << 40), 1), ((0x1000, 0, 0, 0x10000, 1 << 40), 1),
                    ((0x1000, 0, 1, 0x10000, 16), 3), ((0x1000, 0, 1, None, 1 << 40), 1)):
        assert L.hkv_shared_evict(r, *a, None) == code, a
    for miss in ("pos", "weight"):
        assert L.hkv_shared_evict(C.byref(cache(**{miss: None})), 0x1000, 0, 1, 0x10000, 1 << 40, None) == 1


def test_scratch_sizes():
    L, n, m = hkv.lib(), C.c_size_t(), C.c_size_t()
    c = cache()
    assert L.hkv_shared_attend_bytes(C.byref(c), 1, 1, C.byref(n)) == 0
    assert L.hkv_shared_attend_bytes(C.byref(c), 1, 0, C.byref(m)) == 0
    assert 0 <= m.value <= n.value < 64 << 20
    assert L.hkv_shared_evict_bytes(C.byref(c), C.byref(n)) == 0
    assert n.value <= 4 * 2 * 96 * 8 + 4096
    # no prefixes: their pointers are not looked at
    none = cache(num_prefixes=0, prefix_k=None, prefix_v=None, prefix_len=None, prefix_of=None, prefix_capacity=0)
    assert L.hkv_shared_attend_bytes(C.byref(none), 5, 1, C.byref(n)) == 0


def test_config_refusals():
    ok = dict(num_seqs=2, num_heads=4, num_kv_heads=2, head_dim=64, capacity=32)
    with pytest.raises(ValueError, match="CUDA device"):
        hkv.SharedPrefixCache(hkv.SharedConfig(**ok), device="cpu")


# -- the oracle itself ---------------------------------------------------------

def test_oracle_attend_matches_softmax():
    g = torch.Generator().manual_seed(0)
    S, H, Hk, T, d, P, n = 2, 4, 2, 3, 64, 5, 7
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, pk, pv = r(S, H, T, d), r(S, Hk, n, d), r(S, Hk, n, d), r(1, Hk, P, d), r(1, Hk, P, d)
    lens = torch.full((S, Hk), n)
    out, lse, w, *_ = O.attend(q.float(), k.float(), v.float(), lens, pk, pv, [P], [0, 0])
    q, k, v = q.float().double(), k.float().double(), v.float().double()
    kk = torch.cat([pk.expand(S, -1, -1, -1), k], 2).repeat_interleave(2, 1)
    vv = torch.cat([pv.expand(S, -1, -1, -1), v], 2).repeat_interleave(2, 1)
    x = q @ kk.transpose(-1, -2) / 8
    mask = torch.arange(P + n)[None] > (P + n - T + torch.arange(T))[:, None]
    x = x.masked_fill(mask, -torch.inf)
    a = x.softmax(-1)
    assert torch.allclose(out, a @ vv, atol=1e-12) and torch.allclose(lse, x.logsumexp(-1), atol=1e-12)
    assert torch.allclose(w, a[..., P:].sum(2).view(S, Hk, 2, n).sum(2), atol=1e-12)
    # a mistake is not within the bounds: one key too few
    bad, _, _, bound, _, _ = O.attend(q.float(), k.float(), v.float(), lens - 1, pk, pv, [P], [0, 0])
    with pytest.raises(AssertionError):
        O.assert_within(bad, out, bound, "planted")


def test_oracle_evict_worked_example():
    """Five tokens, budget 3, newest position 9, recent 2: positions 9 and 8
    stay; of (w, pos) (.5, 4), (.1, 7), (.5, 2) the lowest go: (.1, 7), then
    the tie at .5 by position: 2.  Slots 0..4: pos 4, 9, 7, 2, 8; hole: slot 2
    (pos 7); slot 3 (pos 2) goes in place; slot 4 (pos 8) moves into slot 2."""
    pos = np.array([[[4, 9, 7, 2, 8, 77]]], np.int32)
    w = np.array([[[.5, 0, .1, .5, 0, 9]]], np.float32)
    k, v = pos[..., None] * 10, pos[..., None] * 100
    lens = np.array([[5]])
    O.evict(k, v, pos, w, lens, np.array([[3]]), 2, 1)
    assert pos[0, 0].tolist() == [4, 9, 8, 2, 8, 77] and lens[0, 0] == 3
    assert k[0, 0, :, 0].tolist() == [40, 90, 80, 20, 80, 770]
    assert w[0, 0, 2] == 0
