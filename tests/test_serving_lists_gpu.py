"""GPU tests of cu_q lists that are none: kv_append and attn_fwd_paged both
report them, and kv_append writes nothing but the new tokens' rows."""
import pytest
import torch

from tests.paged import make_paged
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu

BAD = [[0, 6, 4], [0, 4, 99], [-3, 4, 8], [5, 5, 5], [1, 4, 8], [0, 9, 8], [8, 4, 0], [0, -1, 8],
       [0, 4, -2 ** 31], [2 ** 31 - 1, 0, 8], [9, 9, 9], [-1, -1, -1]]


def bits(t):
    return t.reshape(-1, t.shape[-1]).view(torch.int16)


@pytest.mark.parametrize("cu", BAD, ids=str)
def test_a_list_out_of_order_is_reported(cu):
    p = make_paged([4, 4], [40, 40], 3, 64, 16, seed=5)
    g = torch.Generator().manual_seed(8)
    k, v = [torch.randn(8, 3, 64, generator=g).bfloat16().cuda() for _ in range(2)]
    table, _, kv_len = p.lists()
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    lists = table, torch.tensor(cu, dtype=torch.int32).cuda(), kv_len
    fattn.device_status()
    fattn.kv_append(k, v, kc, vc, *lists)
    word = fattn.device_status()
    assert word & 0xff == 6 and word >> 8 & 0xff == 8, hex(word)
    # Every slot holds what it held, or one of the rows.
    for got, before, rows in ((kc, p.k_cache.cuda(), k), (vc, p.v_cache.cuda(), v)):
        same = (bits(got) == bits(before)).all(-1)
        row = (bits(got)[:, None] == bits(rows)[None]).all(-1).any(-1)
        assert bool((same | row).all())
    fattn.attn_fwd_paged(k, kc, vc, *lists, 8)
    word = fattn.device_status()
    assert word & 0xff == 6 and word >> 8 & 0xff == 1, hex(word)


@pytest.mark.parametrize("at", [1, 127, 128, 129, 400, 699])
def test_one_entry_out_of_order_in_a_long_list(at):
    """More sequences than the block that looks the list over has threads."""
    p = make_paged([1] * 700, [3] * 700, 1, 64, 16, seed=6)
    k = torch.randn(700, 1, 64).bfloat16().cuda()
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    table, cu, kv_len = p.lists()
    fattn.device_status()
    fattn.kv_append(k, k, kc, vc, table, cu, kv_len)
    assert fattn.device_status() == 0
    cu[at] += 2
    fattn.kv_append(k, k, kc, vc, table, cu, kv_len)
    assert fattn.device_status() & 0xff == 6


@pytest.mark.parametrize("cu,T", [([0, 4, 8], 8), ([0, 0, 0], 8), ([0, 8, 8], 8), ([0, 3, 5], 8), ([0, 0, 1], 1)])
def test_lists_in_order_are_not(cu, T):
    p = make_paged([b - a for a, b in zip(cu, cu[1:])], [40, 40], 2, 64, 16, seed=7)
    k = torch.randn(T, 2, 64).bfloat16().cuda()
    fattn.device_status()
    fattn.kv_append(k, k, p.k_cache.cuda(), p.v_cache.cuda(), *p.lists())
    assert fattn.device_status() == 0
    fattn.attn_fwd_paged(k, p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(), 8)
    assert fattn.device_status() == 0
