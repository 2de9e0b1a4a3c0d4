"""GPU tests of tokens and heads more than 2^32 elements from their tensor's
base: queries and outputs of the paged attention, rows of the append, and
head-major views (the head's stride above the token's)."""
import pytest
import torch

from tests.paged import make_paged
from tests.test_paged_gpu import check, queries, reference
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def spread(t, stride, base):
    """t [T, H, d] with its tokens `stride` elements apart in base."""
    view = torch.as_strided(base, t.shape, (stride, t.shape[2], 1))
    view.copy_(t)
    return view


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_far_tokens(dtype):
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 36 GB")
    p = make_paged([1, 3], [9000, 70], 2, 128, 16, dtype, seed=3)
    stride = (1 << 31) + 64
    base = torch.zeros(3 * stride + 4096, dtype=dtype, device="cuda")
    far = torch.zeros(3 * stride + 4096, dtype=dtype, device="cuda")
    q = queries(4, 8, 128, dtype, 4)
    out = torch.as_strided(far, (4, 8, 128), (stride, 128, 1))
    lists = p.lists()
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    o, lse = fattn.attn_fwd_paged(spread(q.cuda(), stride, base), kc, vc, *lists, 3, out=out)
    want = fattn.attn_fwd_paged(q.cuda(), kc, vc, *lists, 3)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    check(o, lse, reference(p, q), dtype, 9000)
    k, v = [torch.randn(4, 2, 128, device="cuda").to(dtype) for _ in range(2)]
    pools = [t.clone() for t in (kc, vc)]
    fattn.kv_append(k, v, kc, vc, *lists)
    fattn.kv_append(spread(k, stride, base), spread(v, stride, far), *pools, *lists)
    assert torch.equal(kc, pools[0]) and torch.equal(vc, pools[1])
    assert fattn.device_status() == 0


@pytest.mark.parametrize("d", [64, 96, 128])
def test_head_major_views_give_the_same_bits(d):
    p = make_paged([1, 50, 300], [3000, 50, 700], 2, d, 32, seed=d)
    q = queries(p.T, 8, d, torch.bfloat16, 5).cuda()
    lists = p.lists()
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    want = fattn.attn_fwd_paged(q, kc, vc, *lists, 300)
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(8, p.T, d, dtype=q.dtype, device="cuda").transpose(0, 1)
    got = fattn.attn_fwd_paged(turned, kc, vc, *lists, 300, out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k, v = q[:, :2].contiguous(), q[:, 2:4].contiguous()
    pools = [t.clone() for t in (kc, vc)]
    rope = fattn.rope_table(4096, 64)
    fattn.kv_append(k, v, kc, vc, *lists, rope=rope)
    fattn.kv_append(turned[:, :2], turned[:, 2:4], *pools, *lists, rope=rope)
    assert torch.equal(kc, pools[0]) and torch.equal(vc, pools[1])
    assert fattn.device_status() == 0
