"""GPU tests of attn_fwd_paged's numbers given as tensors that change in place
between calls."""
import numpy as np
import pytest
import torch

from tests.paged import make_paged
from tests.test_paged_gpu import check, queries, reference
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def test_max_q_and_scale_are_taken_by_value():
    max_q, scale = torch.tensor(1), torch.tensor(0.125)
    for n, sc in ((1, 0.125), (300, 0.25), (40, 0.0625)):
        p = make_paged([n], [500], 1, 64, 16, seed=n)
        q = queries(300, 4, 64, torch.bfloat16, 1)  # one shape throughout
        max_q.fill_(n)
        scale.fill_(sc)
        o, lse = fattn.attn_fwd_paged(q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(), max_q,
                                      scale=scale)
        assert fattn.device_status() == 0
        check(o[:n], lse[:n], reference(p, q[:n], scale=sc), torch.bfloat16, 500)
        assert fattn.paged_workspace_size(4, 1, 64, max_q) == fattn.paged_workspace_size(4, 1, 64, n)


def test_whole_numbers_of_other_kinds_and_none():
    p = make_paged([3], [50], 1, 64, 16, seed=2)
    q = queries(3, 2, 64, torch.bfloat16, 2)
    args = q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), *p.lists()
    want = fattn.attn_fwd_paged(*args, 3)
    got = fattn.attn_fwd_paged(*args, np.int64(3), scale=np.float32(0.125))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for bad in (3.0, "3", None):
        with pytest.raises(TypeError):
            fattn.attn_fwd_paged(*args, bad)
