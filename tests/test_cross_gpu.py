"""GPU tests of attn_fwd_cross against the fp64 reference: single queries to
long batches against shorter and longer keys, ragged lengths and sequences
without keys, grouped heads, both types, what lies behind a sequence's end,
views of packed projections, splits over many CTAs, streams and graphs."""
import pytest
import torch

from tests import search_ref as ref
from tests.test_paged_gpu import check
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def make(B, Hq, Hk, Nq, Nk, d, dtype, seed=0, lens=None, fill=float("nan"), scale=1.5):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, Hq, Nq, d, generator=g) * scale).to(dtype)
    k, v = (torch.randn(B, Hk, Nk, d, generator=g).to(dtype) for _ in range(2))
    for b, n in enumerate(lens or []):
        k[b, :, n:] = fill
        v[b, :, n:] = fill
    return q, k, v


def run(q, k, v, lens, **kw):
    kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    return fattn.attn_fwd_cross(q.cuda(), k.cuda(), v.cuda(), kv_len=kv_len, **kw)


def verify(got, q, k, v, lens, what="", scale=None):
    scale = fattn.default_scale(q.shape[-1]) if scale is None else scale
    check(*got, ref.cross(q, k, v, lens, scale), q.dtype, k.shape[2], what)


CASES = [
    # B, Hq, Hk, Nq, Nk, d, lens
    (1, 1, 1, 1, 1, 64, None),
    (1, 1, 1, 5, 1, 128, None),                       # one key
    (2, 4, 4, 1, 1500, 64, None),                     # a decoder's single tokens
    (3, 8, 2, 4, 700, 128, [700, 1, 129]),            # beams
    (2, 4, 2, 77, 128, 96, None),
    (3, 12, 4, 333, 501, 64, [501, 128, 77]),
    (2, 2, 2, 1000, 77, 128, [77, 20]),               # longer than the keys
    (1, 2, 1, 300, 4000, 64, None),
    (4, 3, 3, 129, 257, 96, [0, 257, 127, 256]),      # a sequence without keys
    (2, 5, 1, 130, 130, 128, [130, 0]),               # 25 tokens a tile
    (2, 128, 1, 3, 200, 64, [200, 64]),               # a token a tile
    (33, 2, 1, 2, 40, 64, [1 + i for i in range(33)]),
    (500, 1, 1, 3, 20, 64, [i % 21 for i in range(500)]),   # more sequences than threads
    (1, 1, 1, 256, 128, 128, None),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Hq,Hk,Nq,Nk,d,lens", CASES,
                         ids=["B%d_H%d-%d_q%d_k%d_d%d%s" % (*c[:6], "_ragged" if c[6] else "") for c in CASES])
def test_against_reference(B, Hq, Hk, Nq, Nk, d, lens, dtype):
    q, k, v = make(B, Hq, Hk, Nq, Nk, d, dtype, seed=Nk, lens=lens)
    got = run(q, k, v, lens)
    assert fattn.device_status() == 0
    verify(got, q, k, v, lens)


@pytest.mark.parametrize("B,Hq,Hk,Nq,Nk,d", [(1, 1, 1, 1, 60000, 128), (1, 4, 1, 2, 30000, 64),
                                             (2, 2, 1, 300, 9000, 128), (1, 2, 2, 40, 20000, 96)])
def test_long_keys_split_over_the_gpu(B, Hq, Hk, Nq, Nk, d):
    q, k, v = make(B, Hq, Hk, Nq, Nk, d, torch.bfloat16, seed=3, scale=2.5)
    need = fattn.cross_workspace_size(Hq, Hk, Nq, d)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    got, again = run(q, k, v, None, workspace=ws), run(q, k, v, None, workspace=ws)
    assert fattn.device_status() == 0
    verify(got, q, k, v, None)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("G,Nq", [(1, 1), (2, 1), (1, 2), (3, 1), (1, 3), (4, 1), (2, 2), (1, 4), (5, 1)])
def test_few_rows(G, Nq, d, dtype):
    """One to five rows to a key head, keys around the pieces that warps, blocks
    and clusters of them take; few heads and many."""
    for B, Hk, Nk, lens in ((1, 1, 700, None), (2, 3, 65, [65, 64]), (1, 2, 3100, None), (3, 1, 17, [17, 0, 16]),
                            (40, 8, 130, [i * 3 % 131 for i in range(40)]), (1, 1, 1, None)):
        q, k, v = make(B, G * Hk, Hk, Nq, Nk, d, dtype, seed=Nk + G, lens=lens)
        got = run(q, k, v, lens)
        again = run(q, k, v, lens)
        assert fattn.device_status() == 0
        verify(got, q, k, v, lens, "%d keys" % Nk)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("Nq", [1, 40])
def test_scores_that_are_not_finite(Nq):
    """A NaN or +inf score makes its row NaN in both outputs, -inf counts for
    nothing; other rows stay as they are."""
    q, k, v = make(1, 1, 1, Nq, 200, 64, torch.float16, seed=9)
    for bad, where in ((float("nan"), "nan"), (float("inf"), "nan"), (-float("inf"), "gone")):
        k2 = k.clone()
        k2[0, 0, 150] = 0
        k2[0, 0, 150, 0] = bad
        q2 = q.abs()
        o, lse = run(q2, k2, v, None)
        if where == "nan":
            assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())
        else:
            keep = torch.arange(200) != 150
            verify((o, lse), q2, k2[:, :, keep], v[:, :, keep], None)
    assert fattn.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf"), 3e4])
def test_padding_may_hold_anything(fill, dtype):
    lens = [1, 100, 128, 200, 0, 255]
    q, k, v = make(6, 4, 2, 130, 256, 64, dtype, seed=4, lens=lens, fill=fill)
    got = run(q, k, v, lens)
    assert fattn.device_status() == 0
    verify(got, q, k, v, lens, str(fill))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_views_of_packed_projections(dtype):
    """q [B, Nq, Hq, d], keys and values [B, Nk, 2, Hk, d], the output a window
    of a wider buffer whose rest stays as it was."""
    g = torch.Generator().manual_seed(5)
    B, Hq, Hk, Nq, Nk, d = 3, 6, 2, 70, 150, 128
    lens = [150, 33, 128]
    q = torch.randn(B, Nq, Hq, d, generator=g).to(dtype)
    kv = torch.randn(B, Nk, 2, Hk, d, generator=g).to(dtype)
    out = torch.full((B, Nq, Hq + 2, d), 7.0, dtype=dtype, device="cuda")
    kvg = kv.cuda()
    o, lse = fattn.attn_fwd_cross(q.cuda().transpose(1, 2), kvg[:, :, 0].transpose(1, 2),
                                  kvg[:, :, 1].transpose(1, 2),
                                  kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  scale=0.2, out=out[:, :, 1:-1].transpose(1, 2))
    assert fattn.device_status() == 0
    verify((o, lse), q.transpose(1, 2), kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2), lens,
           scale=0.2)
    assert bool((out[:, :, 0] == 7).all()) and bool((out[:, :, -1] == 7).all())


def test_no_keys_at_all():
    q = torch.randn(2, 4, 33, 64).bfloat16().cuda()
    k = torch.zeros(2, 2, 0, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = fattn.attn_fwd_cross(q, k, k)
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all()) and fattn.device_status() == 0


@pytest.mark.parametrize("bad", [-1, 301, 2 ** 31 - 1, -2 ** 31])
def test_lengths_out_of_range_are_brought_into_it(bad):
    q, k, v = make(2, 2, 2, 10, 300, 64, torch.bfloat16, seed=6)
    got = run(q, k, v, [bad, 40])
    assert fattn.device_status() & 0xffff == 6 | 1 << 8
    verify(got, q, k, v, [min(max(bad, 0), 300), 40])


def test_two_streams_and_a_graph():
    """Calls with workspaces of their own on two streams, and a captured call
    that follows its lengths."""
    q, k, v = make(2, 4, 1, 3, 3000, 64, torch.float16, seed=7)
    q2, k2, v2 = make(1, 2, 2, 200, 700, 128, torch.float16, seed=8)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = [t.cuda() for t in (q, k, v)], [t.cuda() for t in (q2, k2, v2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append((fattn.attn_fwd_cross(*a, stream=s1), fattn.attn_fwd_cross(*b, stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        verify(x, q, k, v, None)
        verify(y, q2, k2, v2, None)
    lens = torch.tensor([3000, 5], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(a[0]), torch.empty(2, 4, 3, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fattn.attn_fwd_cross(*a, kv_len=lens, out=out, lse=lse)
    for n in ([3000, 5], [1, 2999], [0, 128]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        verify((out, lse), q, k, v, n)
    assert fattn.device_status() == 0


def test_workspaces_that_do_not_fit():
    q, k, v = (t.cuda() for t in make(2, 4, 2, 9, 40, 64, torch.float16))
    need = fattn.cross_workspace_size(4, 2, 9, 64)
    for ws in (torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2],
               torch.empty(need - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises((ValueError, RuntimeError)):
            fattn.attn_fwd_cross(q, k, v, workspace=ws)
    with pytest.raises(TypeError):
        fattn.attn_fwd_cross(q, k, v, workspace=need)


@pytest.mark.parametrize("B", [5, 31, 32, 33])
@pytest.mark.parametrize("bad", [None, -1, 301, -2 ** 31, 2 ** 31 - 1])
def test_single_tokens_of_sequences_in_any_order_of_length(B, bad):
    lens = [(37 * i * i + 11 * i) % 301 for i in range(B)]
    lens[1] = lens[3] = 150  # equal ones
    given = list(lens)
    if bad is not None:
        given[2], lens[2] = bad, min(max(bad, 0), 300)
    q, k, v = make(B, 6, 6, 1, 300, 64, torch.float16, seed=B, lens=lens)
    got = run(q, k, v, given)
    assert fattn.device_status() & 0xffff == (0 if bad is None else 6 | 1 << 8)
    verify(got, q, k, v, lens)
