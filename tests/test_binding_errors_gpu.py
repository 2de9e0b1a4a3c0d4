"""GPU tests of the compiled binding's errors: those of torch where memory runs
out, and sizes beyond the library's 32 bits."""
import pytest
import torch

from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def test_out_of_memory_is_torchs_own_error():
    """The masks of 65536 tokens with 2^24 words each take 4.4 TB."""
    parents = torch.full((65536,), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        fattn.tree_mask(parents, i32(0, 65536), i32(65536), 2 ** 29)
    mask, _ = fattn.tree_mask(parents[:4], i32(0, 4), i32(4), 4)
    assert mask[:, 0].tolist() == [1, 2, 4, 8] and fattn.device_status() == 0
