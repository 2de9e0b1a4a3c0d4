"""GPU test of lists with more columns than the library counts."""
import pytest
import torch

from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def test_columns_beyond_32_bits_are_refused():
    """2^32 + 5 columns are not five."""
    wide = torch.empty(1, 2 ** 32 + 5, dtype=torch.int32, device="cuda")
    cache = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    v_cache, q = cache.clone(), cache[0]
    table, cu, n, none = i32(0)[None], i32(0, 1), i32(1), i32(0)
    x = q[:, :1].transpose(0, 1)
    calls = [lambda: fattn.kv_keep(cache, v_cache, table, cu, n, wide, none),
             lambda: fattn.kv_keep(cache, v_cache, wide, cu, n, none[None], none),
             lambda: fattn.kv_append(x, x, cache, v_cache, wide, cu, n),
             lambda: fattn.attn_fwd_tree(x, cache, v_cache, wide, cu, n, n[None], 1),
             lambda: fattn.attn_fwd_tree(x, cache, v_cache, table, cu, n, wide, 1)]
    for call in calls:
        with pytest.raises(ValueError, match="too large"):
            call()
    assert fattn.device_status() == 0
