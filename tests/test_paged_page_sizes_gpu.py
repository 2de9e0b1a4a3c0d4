"""GPU test of attn_fwd_paged over page sizes: the same keys and values on
pages of 16 to 8192 slots give the same bits, units of every kind in one
batch.  Where a page is longer than a key tile, a tile is a window of it."""
import random

import pytest
import torch

from tests.paged import make_paged
from tests.test_paged_gpu import check, queries, reference, run
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def repaged(p, page, seed):
    """p's sequences on pages of another size, in shuffled order."""
    Hk, d = p.k_cache.shape[1], p.k_cache.shape[3]
    old = p.k_cache.shape[2]
    n = make_paged([b - a for a, b in zip(p.cu, p.cu[1:])], p.kv_len, Hk, d, page, p.k_cache.dtype,
                   seed=seed, fill=float("nan"))
    for b, L in enumerate(p.kv_len):
        j = torch.arange(L)
        for new, was in ((n.k_cache, p.k_cache), (n.v_cache, p.v_cache)):
            new[n.table[b, j // page].long(), :, j % page] = was[p.table[b, j // old].long(), :, j % old]
    return n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,Hq,Hk,seed", [(64, 8, 2, 0), (64, 3, 3, 1), (96, 6, 2, 2), (128, 8, 2, 3), (128, 5, 1, 4)])
def test_page_sizes_give_the_same_bits(d, Hq, Hk, seed, dtype):
    rng = random.Random(seed)
    q_lens, kv_lens = [], []
    for _ in range(14):
        n = rng.choice([1, 1, 1, rng.randint(2, 9), rng.randint(10, 140), rng.randint(100, 300)])
        q_lens.append(n)
        kv_lens.append(n + rng.choice([0, rng.randint(0, 300), rng.randint(1000, 6000)]))
    p = make_paged(q_lens, kv_lens, Hk, d, 16, dtype, seed=seed, fill=float("nan"))
    q = queries(p.T, Hq, d, dtype, seed)
    want = run(p, q)
    check(*want, reference(p, q), dtype, max(kv_lens))
    for page in (32, 64, 128, 256, 512, 2048, 8192):
        got = run(repaged(p, page, page), q)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), page
    assert fattn.device_status() == 0
