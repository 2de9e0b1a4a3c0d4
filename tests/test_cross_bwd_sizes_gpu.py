"""GPU tests of attn_bwd_cross in fp16 where upstream gradients of one call differ
by many powers of two: each sequence's and head's gradients keep the digits that
they have alone, and each query's."""
import pytest
import torch

from tests import cross_bounds
from tests.test_cross_bwd_gpu import dout, run, saved
from tests.test_cross_gpu import make

pytestmark = pytest.mark.gpu
# do is brought to a norm of 1 at least, so dS is rounded at 2^-25 of the norm.
FLOOR = 2.0 ** -25


def mixed(B, Hq, Nq, d, seed, by_row):
    """do whose sizes go down to 2^-12: by sequences, key heads or queries."""
    do = dout(torch.empty(B, Hq, Nq, d), torch.float32, seed)
    at = torch.arange(Nq)[None, None, :, None] if by_row else \
        5 * torch.arange(B)[:, None, None, None] + 2 * (torch.arange(Hq) // 2)[None, :, None, None]
    return (do * 2.0 ** -(at % 13).float()).half()


@pytest.mark.parametrize("by_row", [False, True])
@pytest.mark.parametrize("d,Nq,Nk,lens", [(64, 200, 1000, [1000, 77, 500]), (128, 70, 4000, None),
                                          (96, 130, 600, [600, 599, 128]), (64, 900, 40, [40, 17, 30])])
def test_sizes_that_differ(d, Nq, Nk, lens, by_row):
    B, Hq, Hk = 3, 4, 2
    q, k, v = make(B, Hq, Hk, Nq, Nk, d, torch.float16, seed=Nk, lens=lens, scale=0.5)
    do = mixed(B, Hq, Nq, d, Nq, by_row)
    scale = d ** -0.5
    got = run(q, k, v, *saved(q, k, v, lens, scale), do, lens)
    cross_bounds.within(got, *cross_bounds.gradients(q, k, v, do, lens, scale, FLOOR))


@pytest.mark.parametrize("d", [64, 128])
def test_a_sequence_is_the_same_alone(d):
    B, Hq, Hk, Nq, Nk = 3, 4, 2, 150, 700
    q, k, v = make(B, Hq, Hk, Nq, Nk, d, torch.float16, seed=1, scale=0.5)
    do = mixed(B, Hq, Nq, d, 2, False)
    o, lse = saved(q, k, v, None, d ** -0.5)
    got = run(q, k, v, o, lse, do, None)
    _, tol = cross_bounds.gradients(q, k, v, do, None, d ** -0.5, FLOOR)
    for b in range(B):
        alone = run(*(t[b:b + 1] for t in (q, k, v, o, lse, do)), None)
        for x, y, t in zip(got, alone, tol):
            assert bool(((x[b].double() - y[0].double()).abs().cpu() <= 2 * t[b]).all())


@pytest.mark.parametrize("zero", ["rows", "heads", "sequences"])
def test_gradients_that_are_zero_beside_others(zero):
    q, k, v = make(2, 4, 2, 140, 300, 64, torch.float16, seed=3)
    do = dout(q, torch.float16, 4, 2.0 ** -10)
    if zero == "rows":
        do[:, :, ::2] = 0
    elif zero == "heads":
        do[:, :2] = 0
    else:
        do[0] = 0
    got = run(q, k, v, *saved(q, k, v, None, 0.125), do, None)
    cross_bounds.within(got, *cross_bounds.gradients(q, k, v, do, None, 0.125, FLOOR))


def test_a_gradient_that_is_not_finite_stays_with_its_head():
    q, k, v = make(2, 4, 2, 140, 300, 64, torch.float16, seed=5)
    do = dout(q, torch.float16, 6)
    clean = do.clone()
    do[0, 0, 7, 3] = float("inf")
    do[1, 3, 9, 5] = float("nan")
    o, lse = saved(q, k, v, None, 0.125)
    got, want = run(q, k, v, o, lse, do, None), run(q, k, v, o, lse, clean, None)
    for x, y, heads in zip(got, want, ((0, 3), (0, 1), (0, 1))):
        assert not bool(torch.isfinite(x[0, heads[0]]).all()) and not bool(torch.isfinite(x[1, heads[1]]).all())
    for b, h in ((0, 1), (0, 2), (0, 3), (1, 0), (1, 1), (1, 2)):
        assert torch.equal(got[0][b, h], want[0][b, h])
    for b, h in ((0, 1), (1, 0)):
        assert torch.equal(got[1][b, h], want[1][b, h]) and torch.equal(got[2][b, h], want[2][b, h])
