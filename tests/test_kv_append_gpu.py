"""GPU tests of kv_append against the fp64 reference: ragged batches, pages of
several sizes, both pool layouts, both element types, rotations, slots that no
token writes, tokens without a place, strided inputs, streams and graphs."""
import pytest
import torch

from tests import serving_ref as ref
from tests.paged import make_paged
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def check_cache(got, want, start, written, dtype, exact):
    """Written slots within half a step of the type (plus three fp32 roundings
    of the turned terms, each below |k| in size), the others untouched bit for
    bit.  exact: copies (values, unturned keys)."""
    got, start = got.cpu(), start.cpu()
    keep = ~written[:, None, :, None].expand_as(got)
    assert torch.equal(got[keep].view(torch.int16), start[keep].view(torch.int16))
    w = written[:, None, :, None].expand_as(got)
    if exact:
        assert torch.equal(got[w].double(), want[w])
        return
    size = want.abs().amax(-1, keepdim=True).expand_as(want)[w] * 2
    floor = 2.0 ** -25 if dtype == torch.float16 else 0.0
    tol = torch.finfo(dtype).eps / 2 * want[w].abs() + 4 * U * size + floor
    assert bool(((got[w].double() - want[w]).abs() <= tol).all())


def new_rows(T, Hk, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, Hk, d, generator=g).to(dtype) for _ in range(2)]


def run(p, k, v, rope, inter, pools=None, **kw):
    kc, vc = pools if pools is not None else (p.k_cache.cuda(), p.v_cache.cuda())
    fattn.kv_append(k.cuda() if not k.is_cuda else k, v.cuda() if not v.is_cuda else v, kc, vc,
                    *p.lists(), rope=None if rope is None else rope.cuda(), interleaved=inter, **kw)
    return kc, vc


CASES = [
    # q_lens, kv_lens, Hk, d, page, rot, interleaved
    ([1], [1], 1, 64, 16, 64, False),
    ([1], [5000], 8, 128, 16, 128, False),
    ([1] * 40, [1 + 37 * i % 300 for i in range(40)], 8, 128, 16, 128, False),
    ([5, 0, 1, 130, 0, 17], [5, 0, 77, 200, 40, 1000], 2, 64, 32, 32, True),
    ([0, 0, 300, 0], [0, 9, 300, 0], 4, 96, 64, 96, False),
    ([33, 64, 31], [33, 129, 4000], 3, 256, 128, 256, False),
    ([70, 3], [100, 3], 1, 256, 256, 64, True),
    ([129] * 3, [129, 500, 257], 5, 96, 16, 0, False),
    ([1] * 1100, [1 + i % 50 for i in range(1100)], 2, 64, 16, 16, False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_lens,kv_lens,Hk,d,page,rot,inter", CASES,
                         ids=["%dx%d_d%d_p%d_r%d" % (len(c[0]), c[2], c[3], c[4], c[5]) for c in CASES])
def test_append(q_lens, kv_lens, Hk, d, page, rot, inter, dtype):
    p = make_paged(q_lens, kv_lens, Hk, d, page, dtype, seed=d + page, fill=float("nan"))
    k, v = new_rows(p.T, Hk, d, dtype, 5)
    rope = ref.rope_rows(max(kv_lens) + 1, rot) if rot else None
    kc, vc = run(p, k, v, rope, inter)
    want_k, want_v, written = ref.append(k, v, p.k_cache, p.v_cache, p.table, p.cu, p.kv_len, rope,
                                         inter)
    check_cache(kc, want_k, p.k_cache, written, dtype, rot == 0)
    check_cache(vc, want_v, p.v_cache, written, dtype, True)
    assert fattn.device_status() == 0


def test_pool_layouts_and_packed_inputs_give_the_same_bits():
    p = make_paged([7, 1, 90], [50, 400, 90], 4, 128, 32, seed=2)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(p.T + 5, 10, 128, generator=g).to(torch.bfloat16).cuda()
    k, v = qkv[:p.T, 2:6], qkv[:p.T, 6:10]
    rope = ref.rope_rows(512, 64)
    want = run(p, k.contiguous(), v.contiguous(), rope, False)
    # [pages, page, Hk, d]
    kc = p.k_cache.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    vc = p.v_cache.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    got = run(p, k, v, rope, False, (kc, vc))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # keys and values of a page side by side: [pages, 2, Hk, page, d]
    both = torch.stack([p.k_cache, p.v_cache], 1).cuda()
    got = run(p, k, v, rope, False, (both[:, 0], both[:, 1]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fattn.device_status() == 0


def test_padding_rows_are_skipped():
    """More rows than cu_q covers (a padded batch, a captured size)."""
    p = make_paged([3, 4], [20, 4], 2, 64, 16, seed=3, fill=1.0)
    k, v = new_rows(p.T + 9, 2, 64, torch.bfloat16, 6)
    k[p.T:] = float("nan")
    kc, vc = run(p, k, v, None, False)
    want_k, want_v, written = ref.append(k, v, p.k_cache, p.v_cache, p.table, p.cu, p.kv_len, None,
                                         False)
    check_cache(kc, want_k, p.k_cache, written, torch.bfloat16, True)
    check_cache(vc, want_v, p.v_cache, written, torch.bfloat16, True)
    assert fattn.device_status() == 0


def test_tokens_without_a_place_are_left_out_and_reported():
    p = make_paged([4, 4, 4, 6], [40, 40, 40, 40], 2, 64, 16, seed=4)
    k, v = new_rows(p.T, 2, 64, torch.bfloat16, 7)
    rope = ref.rope_rows(64, 64)
    fattn.device_status()
    for name in ("page_low", "page_high", "position", "beyond", "rope"):
        q = make_paged([4, 4, 4, 6], [40, 40, 40, 40], 2, 64, 16, seed=4)
        table = rope
        if name == "page_low":
            q.table[1, 2] = -5
        elif name == "page_high":
            q.table[2, 2] = q.k_cache.shape[0]
        elif name == "position":
            q.kv_len[3] = 3          # six new tokens of three keys: three before the start
        elif name == "beyond":
            q.kv_len[0] = 2 ** 31 - 1
        else:
            table = rope[:38].contiguous()
        kc, vc = run(q, k, v, table, False)
        assert fattn.device_status() & 0xff == 6, name
        want_k, want_v, written = ref.append(k, v, q.k_cache, q.v_cache, q.table, q.cu, q.kv_len,
                                             table, False)
        assert 0 < int(written.sum()) < q.T
        check_cache(kc, want_k, q.k_cache, written, torch.bfloat16, False)
        check_cache(vc, want_v, q.v_cache, written, torch.bfloat16, True)
    assert fattn.device_status() == 0


def test_cu_q_out_of_order_or_past_the_rows_writes_nothing_wrong():
    p = make_paged([4, 4], [40, 40], 1, 64, 16, seed=5)
    k, v = new_rows(p.T, 1, 64, torch.bfloat16, 8)
    table, _, kv_len = p.lists()
    fattn.device_status()
    for cu in ([0, 6, 4], [0, 4, 99], [-3, 4, 8], [5, 5, 5]):
        kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
        fattn.kv_append(k.cuda(), v.cuda(), kc, vc, table,
                        torch.tensor(cu, dtype=torch.int32).cuda(), kv_len)
        torch.cuda.synchronize()
        # whatever was written is one of the rows, and no other page changed
        used = set(int(x) for x in p.table.reshape(-1) if x >= 0)
        for page in range(p.k_cache.shape[0]):
            if page not in used:
                assert torch.equal(kc[page].cpu(), p.k_cache[page])
    fattn.device_status()


def test_far_pages():
    """Page offsets past 2^31 elements (a 20 GB pool seen through its stride)."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB")
    stride = (1 << 31) + 4096
    big = torch.zeros(4 * stride, dtype=torch.bfloat16, device="cuda")
    kc = torch.as_strided(big, (4, 1, 16, 64), (stride, 1024, 64, 1))
    vc = torch.as_strided(big[2048:], (4, 1, 16, 64), (stride, 1024, 64, 1))
    p = make_paged([2, 20], [18, 20], 1, 64, 16, seed=6, spare=0)
    k, v = new_rows(p.T, 1, 64, torch.bfloat16, 9)
    run(p, k, v, None, False, (kc, vc))
    want_k, want_v, written = ref.append(k, v, torch.zeros(4, 1, 16, 64), torch.zeros(4, 1, 16, 64),
                                         p.table, p.cu, p.kv_len, None, False)
    assert torch.equal(kc.double().cpu(), want_k) and torch.equal(vc.double().cpu(), want_v)


def test_streams_and_a_replayed_graph_follow_the_lists():
    p = make_paged([1] * 5, [10, 20, 30, 40, 50], 2, 128, 16, seed=7, extra_cols=2)
    p.table[:, :] = torch.randperm(p.table.numel(), generator=torch.Generator().manual_seed(1)).reshape(
        p.table.shape).int()
    pages = p.table.numel()
    k, v = [t.cuda() for t in new_rows(5, 2, 128, torch.bfloat16, 3)]
    rope = fattn.rope_table(128, 128)
    kc = torch.zeros(pages, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    table, cu, kv_len = p.lists()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fattn.kv_append(k, v, kc, vc, table, cu, kv_len, rope=rope, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fattn.kv_append(k, v, kc, vc, table, cu, kv_len, rope=rope)
    lens, rows = list(p.kv_len), [(k.clone(), v.clone())]
    for step in range(4):
        kv_len += 1
        k.copy_(torch.randn_like(k))
        v.copy_(torch.randn_like(v))
        rows.append((k.clone(), v.clone()))
        graph.replay()
    torch.cuda.synchronize()
    want_k = torch.zeros(pages, 2, 16, 128)
    want_v = torch.zeros_like(want_k)
    for step, (a, b) in enumerate(rows):
        want_k, want_v, _ = ref.append(a.cpu(), b.cpu(), want_k, want_v, p.table, p.cu,
                                       [n + step for n in lens], rope.cpu(), False)
    assert torch.equal(vc.double().cpu(), want_v)
    err = (kc.double().cpu() - want_k).abs()
    assert bool((err <= 2.0 ** -8 * want_k.abs() + 16 * U * 8).all())
    assert fattn.device_status() == 0
