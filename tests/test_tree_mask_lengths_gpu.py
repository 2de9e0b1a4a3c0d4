"""GPU tests of fattn_tree_mask with lists out of range: what is written, where
and what is reported."""
import pytest
import torch

from tests import search_ref as ref
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu
REPORT = 6 | 9 << 8


def i32(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("L", [5, 1, 0, -1, -2 ** 31])
def test_fewer_keys_than_new_tokens(L):
    """The new tokens' keys are among the sequence's, so no key is before them:
    positions are depths."""
    parents, other = [-1, 0, 1, 1, 3, -1], [-1, 0, 0]
    mask, pos = fattn.tree_mask(i32(*parents, *other), i32(0, 6, 9), i32(L, 10), 6)
    assert fattn.device_status() & 0xffff == REPORT
    rows = ref.paths(parents) + ref.paths(other)
    assert torch.equal(mask.cpu(), ref.pack(rows, 1))
    assert pos[0].tolist() == [len(r) - 1 + (0 if i < 6 else 7) for i, r in enumerate(rows)]


@pytest.mark.parametrize("L", [6, 7, 2 ** 31 - 1])
def test_lengths_in_range(L):
    parents = [-1, 0, 1, 1, 3, -1]
    mask, pos = fattn.tree_mask(i32(*parents), i32(0, 6), i32(L), 6)
    assert fattn.device_status() == 0
    assert pos[0].tolist() == [L - 6 + len(r) - 1 for r in ref.paths(parents)]


@pytest.mark.parametrize("cu,written", [([1, 3, 6], range(1, 6)), ([0, 7, 6], range(6)), ([0, 4, 9], range(6)),
                                        ([0, -1, 4], range(4)), ([0, 3, 2 ** 31 - 1], range(6)),
                                        ([2, 2, 5], range(2, 5))])
def test_rows_outside_the_sequences_stay(cu, written):
    parents = torch.full((6,), -1, dtype=torch.int32)
    mask = torch.full((6, 1), 77, dtype=torch.int32, device="cuda")
    pos = torch.full((1, 6), -9, dtype=torch.int32, device="cuda")
    fattn.tree_mask(parents.cuda(), i32(*cu), i32(10, 10), 6, mask=mask, positions=pos)
    assert fattn.device_status() & 0xffff == REPORT
    for i in range(6):
        assert (int(mask[i]) != 77) == (i in written) and (int(pos[0, i]) != -9) == (i in written)
