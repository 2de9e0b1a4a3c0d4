"""GPU tests of attn_fwd_cross' range report for few rows, whose V is not rounded
to fp16."""
import pytest
import torch

from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Nq", [1, 2, 4])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_large_finite_results_are_not_reported(d, Nq):
    """Neighbours of 2.5e38 each are in bf16's range, their sum is not in fp32's."""
    q = torch.randn(2, 3, Nq, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    k = torch.zeros(2, 3, 1, d, dtype=torch.bfloat16, device="cuda")
    for value in (2.5e38, -2.5e38):
        v = torch.full_like(k, value)
        o, _ = fattn.attn_fwd_cross(q, k, v)
        assert torch.equal(o, v.expand_as(o)) and fattn.device_status() == 0


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("column", [0, 1, 62, 63])
def test_results_that_are_not_finite_are_reported(column, value):
    q = torch.randn(1, 1, 1, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    k = torch.zeros(1, 1, 3, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    v[0, 0, 1, column] = value
    o, _ = fattn.attn_fwd_cross(q, k, v)
    assert fattn.device_status() & 0xffff == 5 | 4 << 8
    keep = torch.arange(64) != column
    assert not bool(torch.isfinite(o[..., column]).any()) and bool((o[..., keep] == 1).all())
