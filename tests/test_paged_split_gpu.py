"""GPU tests of long units split over many CTAs, with data that shows a lost
or repeated key tile: queries of zero make every probability 1, so lse is the
logarithm of the number of keys seen, and values that are 1 in the column of
their key tile (modulo d) make o the shares of those tiles."""
import math

import pytest
import torch

from tests.paged import make_paged
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24

CASES = [
    # q_lens, kv_lens, Hq, Hk, d, page, causal
    ([1], [50000], 4, 1, 128, 64, True),           # one unit over every CTA
    ([1], [131072], 8, 8, 64, 128, True),
    ([1], [19001], 1, 1, 96, 16, True),            # fewer key tiles than CTAs
    ([2, 1], [30000, 9000], 8, 2, 64, 16, True),
    ([1] * 20, [2000 + 331 * i for i in range(20)], 8, 4, 96, 32, True),
    ([40], [40000], 4, 4, 128, 32, True),          # single tiles of more than 32 rows
    ([300], [20000], 4, 2, 128, 128, True),        # pairs of tiles
    ([700, 3, 1], [9000, 20000, 777], 2, 1, 64, 256, True),
    ([700, 3, 1], [9000, 20000, 777], 2, 1, 128, 16, False),
    ([1] * 151, [1100 + i for i in range(151)], 2, 2, 64, 16, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk,d,page,causal", CASES)
def test_every_key_tile_counts_once(q_lens, kv_lens, Hq, Hk, d, page, causal, dtype):
    """Bounds.  P = 1, l and O are whole numbers below 2^24: exact.  A partial's
    base-2 lse is log2f(l) (one step of a number below 32: 2^-19, and 2^-20 for
    its sum with m), so its weight in the merge is off by ln 2 times that and
    2^-22 of the exponential; the sums of `merged` weights add 2 U each.  o has
    that twice (its sum and the weights'), its division, and half a step of the
    type; lse has it once and its own logarithm."""
    p = make_paged(q_lens, kv_lens, Hk, d, page, dtype, seed=d, fill=float("nan"), extra_cols=3)
    tiles = -(-max(kv_lens) // 128)
    merged = min(tiles, torch.cuda.get_device_properties(0).multi_processor_count) + 2
    weight = math.log(2) * (2.0 ** -19 + 2.0 ** -20) + 2.0 ** -22 + 2 * merged * U
    lse_tol = weight + math.log(2) * (2.0 ** -19 + 2.0 ** -20) + 16 * U
    o_rel = torch.finfo(dtype).eps / 2 + 2 * weight + 4 * U
    assert lse_tol < 64 / max(kv_lens), "half a key tile is beyond the bound of lse"
    assert o_rel < 1 / 2 / -(-tiles // d) , "half a key tile beyond that of its column"
    p.v_cache.fill_(float("nan"))
    want_o, want_l = [], []
    for b, L in enumerate(kv_lens):
        j = torch.arange(L)
        one = ((j // 128 % d)[:, None] == torch.arange(d)).to(dtype)
        p.v_cache[p.table[b, j // page].long(), :, j % page] = one[:, None].expand(L, Hk, d)
        seen = torch.arange(L - q_lens[b], L) + 1 if causal else torch.full((q_lens[b],), L)
        want_o.append(one.double().cumsum(0)[seen - 1] / seen[:, None])
        want_l.append(seen.double().log())
    want_o, want_l = torch.cat(want_o)[:, None].cuda(), torch.cat(want_l)[:, None].cuda()
    q = torch.zeros(p.T, Hq, d, dtype=dtype, device="cuda")
    args = q, p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(), p.max_q
    fattn.device_status()
    for _ in range(2):
        o, lse = fattn.attn_fwd_paged(*args, causal=causal)
        assert fattn.device_status() == 0
        err = (lse.double() - want_l).abs()
        assert bool((err <= lse_tol).all()), (float(err.max()), lse_tol)
        err = (o.double() - want_o).abs()
        assert bool((err <= o_rel * want_o).all()), float((err / want_o).nan_to_num(0).max())
