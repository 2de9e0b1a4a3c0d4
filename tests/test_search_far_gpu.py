"""Trees, kept and forked sequences and cross attention on tensors whose rows lie
beyond 2^31 elements: the same bits as on compact ones."""
import pytest
import torch

from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu
FAR = 2 ** 31 + 64


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def spread(t, step=FAR):
    """t's values with its first dimension `step` elements apart."""
    inner = t[0].numel()
    buf = torch.empty((t.shape[0] - 1) * step + inner, dtype=t.dtype, device="cuda")
    out = buf.as_strided(t.shape, (step,) + t.contiguous().stride()[1:])
    return out.copy_(t)


@pytest.mark.parametrize("Hq,Nq,Nk,d", [(2, 1, 300, 64), (2, 130, 300, 64), (2, 130, 300, 128)])
def test_cross_attention(Hq, Nq, Nk, d):
    g = torch.Generator().manual_seed(1)
    q, do = (torch.randn(2, Hq, Nq, d, generator=g).half().cuda() for _ in range(2))
    k, v = (torch.randn(2, 1, Nk, d, generator=g).half().cuda() for _ in range(2))
    kv_len = torch.tensor([Nk, Nk - 7], dtype=torch.int32, device="cuda")
    o, lse = fattn.attn_fwd_cross(q, k, v, kv_len)
    want = fattn.attn_bwd_cross(q, k, v, o, lse, do, kv_len)
    q, k, v, do = map(spread, (q, k, v, do))
    out = spread(torch.zeros_like(o))
    far, far_lse = fattn.attn_fwd_cross(q, k, v, kv_len, out=out)
    assert torch.equal(far, o) and torch.equal(far_lse, lse)
    dq, dk, dv = (spread(torch.zeros_like(t)) for t in want)
    got = fattn.attn_bwd_cross(q, k, v, far, lse, do, kv_len, dq=dq, dk=dk, dv=dv)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert fattn.device_status() == 0


def test_tree_keep_and_fork():
    g = torch.Generator().manual_seed(2)
    pages, Hk, page, d = 6, 2, 16, 64
    caches = [torch.randn(pages, Hk, page, d, generator=g).half().cuda() for _ in range(2)]
    far = [spread(c, 2 ** 30 - 64) for c in caches]  # page 3 on: beyond 2^31
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[5, 3, -1], [0, 4, -1]], **i32)
    kv_len = torch.tensor([25, 21], **i32)
    cu_q = torch.tensor([0, 7, 12], **i32)
    q = torch.randn(12, 4, d, generator=g).half().cuda()
    mask = torch.randint(-2 ** 31, 2 ** 31, (12, 1), generator=g).int().cuda()
    tall = spread(mask, 2 ** 31 // 8)  # of 12 rows the last four
    kept = torch.tensor([[0, 2, 3, 6], [1, 3, 4, 0]], **i32)
    kept_len = torch.tensor([4, 3], **i32)
    parents = torch.tensor([0, 0], **i32)
    grow = torch.tensor([0, 3, 9], **i32)
    refs = torch.tensor([1, 0, 0, 1, 1, 1], **i32)
    results = []
    for k, v, m in ((*caches, mask), (*far, tall)):
        got = list(fattn.attn_fwd_tree(q, k, v, table, cu_q, kv_len, m, 7))
        got.append(fattn.kv_keep(k, v, table, cu_q, kv_len, kept, kept_len))
        got += fattn.kv_fork(k, v, table, got[-1], refs, parents, grow)
        results.append([t.clone() for t in got] + [k.contiguous(), v.contiguous()])
    assert all(torch.equal(x, y) for x, y in zip(*results))
    assert fattn.device_status() == 0
