"""GPU test of fp16 batches whose tiles are mostly whole and end in a ragged
one: many turns of the ring between the tiles that the V warps write, on two
streams at once, with sums that are exact in every order."""
import pytest
import torch

from tests.paged import make_paged
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("q_lens,Hq,Hk", [([1] * 9, 8, 4), ([1] * 9, 2, 2), ([40] * 9, 2, 1), ([300] * 9, 1, 1)])
def test_ragged_tiles_behind_long_runs_of_whole_ones(q_lens, Hq, Hk, d):
    """Queries of zero: every probability is 1 and o the mean of the values,
    which are 0 or 1 by position, so that sums are whole numbers.  o is off by
    the division (2^-24) and its rounding to fp16 (2^-11 relative)."""
    kv_lens = [n + 128 * t + r for n, t, r in zip(q_lens, (60, 3, 33, 7, 90, 1, 16, 45, 70),
                                                  (1, 127, 0, 5, 64, 77, 31, 100, 9))]
    p = make_paged(q_lens, kv_lens, Hk, d, 32, torch.float16, seed=d)
    p.v_cache.fill_(float("nan"))
    for b, n in enumerate(kv_lens):
        j = torch.arange(n)
        one = ((j[:, None] // 128 + torch.arange(d)) % 5 == 0).half()  # by key tile and column
        p.v_cache[p.table[b, j // 32].long(), :, j % 32] = one[:, None].expand(n, Hk, d)
    q = torch.zeros(p.T, Hq, d, dtype=torch.float16).cuda()
    args = q, p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(), p.max_q
    want = torch.empty(p.T, d, dtype=torch.float64)
    for b, n in enumerate(kv_lens):
        j = torch.arange(n)
        count = ((j[:, None] // 128 + torch.arange(d)) % 5 == 0).double().cumsum(0)
        seen = torch.arange(n - q_lens[b], n)
        want[p.cu[b]:p.cu[b + 1]] = count[seen] / (seen + 1)[:, None]
    want = want[:, None].cuda()
    fattn.device_status()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [fattn.attn_fwd_paged(*args, stream=s) for _ in range(15) for s in streams]
    torch.cuda.synchronize()
    assert fattn.device_status() == 0
    for o, lse in got:
        assert bool(((o.double() - want).abs() <= want * (2.0 ** -11 + 2.0 ** -23)).all())
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])
