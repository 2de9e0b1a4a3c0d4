"""GPU test of the compiled binding with tensors that have no memory."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def test_a_tensor_without_memory_raises():
    """torch's error for its missing address, raised between the checks and the
    library's call; calls behind it go on."""
    q = torch.randn(1, 2, 3, 64, device="cuda").bfloat16()
    cache = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    lists = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0]], [0, 1], [1])]
    with FakeTensorMode(allow_non_fake_inputs=True):
        fake = torch.empty(1, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
        row = torch.empty(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    want = fattn.attn_fwd_cross(q, q, q)
    for call in (lambda: fattn.attn_fwd_cross(fake, q, q), lambda: fattn.kv_append(row, row, cache, cache.clone(), *lists),
                 lambda: fattn.attn_bwd_cross(q, q, q, q, want[1], fake)):
        with pytest.raises(RuntimeError):
            call()
    for x, y in zip(fattn.attn_fwd_cross(q, q, q), want):
        assert torch.equal(x, y)
    assert fattn.device_status() == 0
