"""The restatement and bounds of tests/shared_bounds.py: the same numbers as
the row by row one, and mistakes outside the bounds at any number of keys."""
import pytest
import torch

import shared_bounds as B
import shared_oracle as O


def test_same_as_row_by_row():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    S, H, Hk, T, d, n, P = 3, 4, 2, 3, 64, 9, 5
    q, k, v, pk, pv = r(S, H, T, d), r(S, Hk, n, d), r(S, Hk, n, d), r(2, Hk, P, d), r(2, Hk, P, d)
    lens = torch.tensor([[9, 1], [0, 3], [2, 8]])
    args = q, k, v, lens, pk, pv, [5, 2], [0, -1, 1]
    for x, y in zip(B.attend(*args)[:3], O.attend(*args)[:3]):
        assert torch.equal(torch.isfinite(x), torch.isfinite(y))
        assert (x - y).abs().nan_to_num(0.0).max() < 1e-12


@pytest.mark.parametrize("T,n,P", [(1, 100, 0), (1, 1300, 0), (3, 700, 900), (1, 9000, 300), (3, 1300, 4000)])
def test_mistakes_are_outside(T, n, P):
    """The two products of a weight's bf16 parts lie within the bounds; one of
    them alone outside, and so the value row of any of the largest logits left out
    of up to 2000 (a weight of 1 / n and more; the bounds grant the sums n 2^-25)."""
    q, k, v, pk, pv = B.comb(1, 1, 1, T, 64, n, 1 if P else 0, P, seed=n)
    lens = torch.full((1, 1), n)
    out, *_, bound, _, _ = B.attend(q, k, v, lens, pk, pv, [P], [0], scale=1.0, exact_logits=True)
    kk, vv = (torch.cat([p[0, 0], x[0, 0]]) if P else x[0, 0] for p, x in ((pk, k), (pv, v)))
    vv = vv.double()
    for t in range(T):
        x = kk.double() @ q[0, 0, t].double()
        assert torch.equal(x.float().double(), x) and x.max() == 0
        x[P + n - T + t + 1:] = -torch.inf
        p = x.exp()
        first = p.bfloat16().double()
        second = (p - first).bfloat16().double()
        within = lambda o: bool(((o / p.sum()).bfloat16().double() - out[0, 0, t]).abs().le(bound[0, 0, t]).all())  # noqa: E731
        assert within((first + second) @ vv)
        assert not within(first @ vv)
        for lost in (0, 8, P + n // 16 * 8, P + (n - T) // 8 * 8) if P + n < 2000 else ():
            assert not within((first + second) @ vv - p[lost] * vv[lost]), lost
