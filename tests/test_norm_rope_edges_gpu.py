"""GPU tests of qk_norm_rope_bwd where a tensor has weights and no rows."""
import pytest
import torch

from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def fill_the_allocator():
    """Blocks that the next small allocations get hold 7."""
    junk = [torch.full((n,), 7.0, device="cuda") for n in (64, 128, 256) for _ in range(64)]
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,N", [(2, 0, 2, 5), (1, 3, 0, 5), (2, 0, 0, 5), (0, 2, 2, 5), (2, 2, 2, 0),
                                       (2, 0, 2, 0)])
def test_weight_gradients_of_no_rows_are_zero(B, Hq, Hk, N, stream):
    d = 64
    g = torch.Generator().manual_seed(1)
    q, k = [torch.randn(B, H, N, d, generator=g).bfloat16().cuda() for H in (Hq, Hk)]
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    fill_the_allocator()
    if stream:
        with torch.cuda.stream(s):
            fill_the_allocator()
    out = fattn.qk_norm_rope_bwd(q, k, q, k, w, w, stream=s)
    torch.cuda.synchronize()
    for dw, H, x in ((out[2], Hq, q), (out[3], Hk, k)):
        if B * H * N == 0:
            assert bool((dw == 0).all()), dw[:4]
        else:  # dy = x, w = 1, no turn: x^2 r summed over the rows
            r = (x.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt()
            want = (x.double().square() * r).sum((0, 1, 2))
            assert bool(((dw.double() - want).abs() <= 64 * 2.0 ** -24 * want).all())
    assert fattn.device_status() == 0
