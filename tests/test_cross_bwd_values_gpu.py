"""GPU tests of attn_bwd_cross in fp16 with large values and small ones: dS beyond
fp16's largest number, and far below its smallest."""
import pytest
import torch

from tests import cross_bounds
from tests.test_cross_bwd_gpu import dout, run, saved
from tests.test_cross_gpu import make
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu
# |dO| |V| of a row is brought to 2^15 at least: half a step of 2^-24 is 2^-40 of it.
FLOOR = 2.0 ** -40


def verify(q, k, v, do, lens=None, scale=0.125):
    got = run(q, k, v, *saved(q, k, v, lens, scale), do, lens, scale=scale)
    assert fattn.device_status() == 0
    cross_bounds.within(got, *cross_bounds.gradients(q, k, v, do, lens, scale, FLOOR, values=True))


@pytest.mark.parametrize("Nq,Nk,size,up", [(8, 2, 2100.0, 1.0), (130, 40, 2100.0, 1.0), (130, 300, 6e4, 4.0),
                                           (8, 2, 3e4, 2.0 ** -14), (300, 129, 3e4, 2.0 ** -20)])
def test_large_values(Nq, Nk, size, up):
    """Halves of the keys with values of one size and opposite signs, under equal
    scores: dS = P dP, some 10^4 to 10^7 with an upstream gradient of ones, and all
    results in fp16's range."""
    g = torch.Generator().manual_seed(Nk)
    sign = torch.where(torch.arange(Nk) % 2 == 0, 1.0, -1.0)[:, None]
    for d in (64, 128):
        q = (torch.randn(1, 2, Nq, d, generator=g) * 2.0 ** -8).half()
        k = (torch.randn(1, 1, Nk, d, generator=g) * 2.0 ** -9).half()
        v = (sign * size).expand(Nk, d)[None, None].contiguous().half()
        do = torch.full((1, 2, Nq, d), up).half()
        # dk adds up 2 Nq queries, dv their P
        verify(q, k, v, do / (1 if Nq < 100 or up < 1 else 64), scale=2.0 ** -3)


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -6, 200.0])
def test_values_of_any_size(size):
    q, k, v = make(2, 4, 2, 150, 500, 64, torch.float16, seed=6, scale=0.5)
    do = dout(q, torch.float16, 7, 2.0 ** 6 if size < 1 else 2.0 ** -6)
    verify(q, k, (v * size).half(), do, [500, 131])


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 6e4])
def test_values_behind_the_last_key_do_not_count(fill):
    lens = [100, 0, 129]
    q, k, v = make(3, 2, 2, 70, 200, 96, torch.float16, seed=8, lens=lens, fill=fill, scale=0.5)
    verify(q, k, v, dout(q, torch.float16, 9, 2.0 ** -12), lens)


def test_a_value_that_is_not_finite_stays_with_its_head():
    q, k, v = make(2, 4, 2, 140, 300, 64, torch.float16, seed=10)
    do = dout(q, torch.float16, 11)
    want = run(q, k, v, *saved(q, k, v, None, 0.125), do, None)
    v[0, 1, 200, 5] = float("inf")
    got = run(q, k, v, *saved(q, k, v, None, 0.125), do, None)
    assert not bool(torch.isfinite(got[0][0, 2]).any())
    assert torch.equal(got[0][1], want[0][1]) and torch.equal(got[0][0, :2], want[0][0, :2])
    assert torch.equal(got[1][0, 0], want[1][0, 0]) and torch.equal(got[1][1], want[1][1])
