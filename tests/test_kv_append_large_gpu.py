"""GPU tests of the append at prompt sizes, where an item has more heads than
a warp holds at a time.  Against the fp64 formula, on the GPU."""
import pytest
import torch

from tests import serving_ref as ref
from tests.paged import make_paged
from tests.test_norm_rope_large_gpu import heads_a_item
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("Hk,d,page,rot,inter,dtype", [
    (5, 128, 64, 128, False, torch.bfloat16), (8, 128, 16, 64, True, torch.float16),
    (13, 64, 32, 64, False, torch.float16), (7, 96, 256, 96, False, torch.bfloat16),
    (6, 256, 128, 256, True, torch.bfloat16), (9, 64, 16, 0, False, torch.bfloat16)])
def test_prompts(Hk, d, page, rot, inter, dtype):
    q_lens = [4000, 1, 0, 3999, 4097, 17, 3000, 5000, 4500]
    kv_lens = [n + x for n, x in zip(q_lens, (0, 900, 33, 5, 0, 200, 1000, 1, 0))]
    p = make_paged(q_lens, kv_lens, Hk, d, page, dtype, seed=Hk)
    # the launch counts items of keys and of values
    assert heads_a_item(2 * p.T, Hk, d) > 4
    g = torch.Generator("cuda").manual_seed(d)
    kv = torch.randn(p.T, 2, Hk, d, generator=g, device="cuda").to(dtype)
    rope = ref.rope_rows(max(kv_lens), rot).cuda() if rot else None
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    before = kc.clone(), vc.clone()
    fattn.kv_append(kv[:, 0], kv[:, 1], kc, vc, *p.lists(), rope=rope, interleaved=inter)
    assert fattn.device_status() == 0
    b = torch.repeat_interleave(torch.arange(len(q_lens)), torch.tensor(q_lens))
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(q_lens, kv_lens)])
    at = p.table[b, pos // page].long().cuda(), (pos % page).cuda()
    written = torch.zeros(kc.shape[0], page, dtype=torch.bool, device="cuda")
    written[at] = True
    keep = ~written[:, None, :, None].expand_as(kc)
    for got, was in ((kc, before[0]), (vc, before[1])):
        assert torch.equal(got[keep].view(torch.int16), was[keep].view(torch.int16))
    assert torch.equal(vc[at[0], :, at[1]], kv[:, 1])
    got = kc[at[0], :, at[1]]
    if rot == 0:
        assert torch.equal(got, kv[:, 0])
        return
    ang = rope[pos.cuda()][:, None]
    want, size = ref.turn(kv[:, 0].double(), ang, inter), ref.g_terms(kv[:, 0], ang, inter)
    # a product, a fused product and sum: 2 U of the terms; half a step of the store
    half = torch.finfo(dtype).eps / 2
    tol = half * want.abs() + (1 + half) * 2 * U * size + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    err = (got.double() - want).abs()
    assert bool((err <= tol * (1 + 1e-9)).all()), float((err / tol).max())
    turned_not = got[..., rot:], kv[:, 0][..., rot:]
    assert torch.equal(*turned_not)
