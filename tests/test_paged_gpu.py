"""GPU tests of attn_fwd_paged against the fp64 reference: ragged batches of
single tokens, drafts and chunks, grouped heads, page sizes, both element
types, rows without keys, whatever lies in unused slots, layouts, splits over
many CTAs, streams and graphs; and the three serving calls run together."""
import pytest
import torch

from tests import serving_ref as ref
from tests.paged import make_paged
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def check(o, lse, want, dtype, keys, what=""):
    """Bounds, first order.  A score's product adds d terms in fp32: (d + 2) U
    of scale sum |q k|; scaling it to base 2 and subtracting m adds 4 U of
    |x| <= the same sum.  The exponential's instruction is good to 2^-22.  So p
    is off by e = (d + 6) U terms + 2^-22 relative, in the numerator and in l
    alike; P's rounding to fp16 adds half a step, 2^-11, of a normal p and
    2^-25 absolute of a smaller one (l >= 1 in those units); sums of n fp32
    terms, rescalings and the merge add (n + 64) U.  The store rounds by half a
    step of the type."""
    wo, wl, size, terms, vmax = want
    d = wo.shape[-1]
    o, lse = o.double().cpu(), lse.double().cpu()
    rows = ~torch.isnan(wl)
    empty = rows & (wl == -float("inf"))
    assert bool((o[empty] == 0).all()) and bool((lse[empty] == -float("inf")).all()), what
    live = rows & ~empty
    e = (d + 6) * U * terms + 2.0 ** -22 + (keys + 64) * U
    half = torch.finfo(dtype).eps / 2
    tol = half * wo.abs() + (1 + half) * ((2.0 ** -11 + 2 * e)[..., None] * size +
                                          keys * 2.0 ** -25 * vmax[..., None])
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (o - wo).abs()
    assert bool(torch.isfinite(o[live]).all()), what
    bad = (err > tol * (1 + 1e-9))[live]
    assert not bool(bad.any()), "%s: %d of %d beyond the bound, worst ratio %.3g" % (
        what, int(bad.sum()), bad.numel(), float((err / tol)[live].max()))
    lerr = (lse - wl).abs()[live]
    ltol = (e + 2 * U * wl.abs() + 4 * U)[live]
    assert bool((lerr <= ltol).all()), "%s: lse ratio %.3g" % (what, float((lerr / ltol).max()))


def queries(T, Hq, d, dtype, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, Hq, d, generator=g) * scale).to(dtype)


def run(p, q, causal=True, **kw):
    return fattn.attn_fwd_paged(q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(),
                                kw.pop("max_q", max(p.max_q, 1)), causal=causal, **kw)


def reference(p, q, causal=True, scale=None):
    scale = fattn.default_scale(q.shape[-1]) if scale is None else scale
    return ref.paged_attention(q, p.k_cache, p.v_cache, p.table, p.cu, p.kv_len, causal, scale)


CASES = [
    # q_lens, kv_lens, Hq, Hk, d, page, causal
    ([1], [1], 1, 1, 64, 16, True),
    ([1], [7], 4, 1, 128, 16, True),
    ([1, 1, 1], [128, 129, 127], 8, 2, 128, 32, True),
    ([1] * 9, [1, 300, 16, 17, 511, 512, 513, 64, 1000], 8, 8, 64, 16, True),
    ([1, 1], [5000, 3], 32, 8, 128, 16, True),
    ([5, 3, 1, 7], [260, 3, 900, 1300], 12, 4, 96, 64, True),
    ([2, 9], [400, 700], 16, 1, 64, 128, True),       # 16 query heads to one key head
    ([3], [300], 128, 1, 64, 16, True),               # 128: one token a tile
    ([4, 1], [200, 90], 5, 1, 128, 256, True),        # 25 tokens a tile, 3 rows idle
    ([40, 33], [640, 33], 7, 1, 96, 32, True),        # 18 tokens a tile
    ([128], [128], 1, 1, 128, 128, True),
    ([129], [129], 2, 2, 64, 64, True),
    ([256, 1, 130], [256, 77, 700], 2, 1, 128, 16, True),
    ([300, 257], [300, 1024], 4, 4, 64, 32, True),
    ([70, 1, 200, 0, 5], [700, 0, 200, 9, 5], 6, 2, 128, 64, True),
    ([64, 1], [300, 40], 4, 2, 128, 16, False),
    ([1, 17], [1000, 17], 3, 3, 96, 512, False),
    ([513], [513], 8, 1, 64, 16, False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk,d,page,causal", CASES,
                         ids=["B%d_q%d_k%d_H%d-%d_d%d_p%d%s" % (len(c[0]), max(c[0]), max(c[1]), c[2],
                                                                c[3], c[4], c[5], "c" if c[6] else "")
                              for c in CASES])
def test_against_reference(q_lens, kv_lens, Hq, Hk, d, page, causal, dtype):
    p = make_paged(q_lens, kv_lens, Hk, d, page, dtype, seed=sum(kv_lens), fill=float("nan"))
    q = queries(p.T, Hq, d, dtype, 1)
    o, lse = run(p, q, causal)
    assert fattn.device_status() == 0
    check(o, lse, reference(p, q, causal), dtype, max(kv_lens))


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk,d,page", [
    ([1], [50000], 4, 1, 128, 64),                     # one unit over every CTA
    ([2, 1], [30000, 9000], 8, 2, 64, 16),
    ([1] * 20, [2000 + 331 * i for i in range(20)], 8, 4, 96, 32),
    ([300], [20000], 4, 2, 128, 128),                  # pairs of tiles, split
    ([1] * 600, [1 + (i * 37) % 200 for i in range(600)], 2, 1, 64, 16),   # more sequences than threads
])
def test_long_and_many_sequences(q_lens, kv_lens, Hq, Hk, d, page):
    p = make_paged(q_lens, kv_lens, Hk, d, page, torch.bfloat16, seed=7, extra_cols=5)
    q = queries(p.T, Hq, d, torch.bfloat16, 2, 2.5)
    ws = torch.full((fattn.paged_workspace_size(Hq, Hk, d, p.max_q),), 0xff, dtype=torch.uint8,
                    device="cuda")
    o, lse = run(p, q, workspace=ws)
    again = run(p, q, workspace=ws)
    assert fattn.device_status() == 0
    check(o, lse, reference(p, q), torch.bfloat16, max(kv_lens))
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1]), "equal calls give equal bits"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf"), 3e4])
def test_unused_slots_may_hold_anything(fill, dtype):
    """Slots behind the last key and foreign pages; table entries behind the
    last page point nowhere."""
    lens = [1, 100, 128, 200, 255, 1030]
    for unused in (-1, 2 ** 31 - 1, -2 ** 31):
        p = make_paged([1, 2, 128, 30, 1, 5], lens, 2, 64, 16, dtype, seed=9, fill=fill,
                       extra_cols=9, unused=unused)
        q = queries(p.T, 4, 64, dtype, 3)
        o, lse = run(p, q)
        assert fattn.device_status() == 0
        check(o, lse, reference(p, q), dtype, max(lens), "fill %s unused %d" % (fill, unused))


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_around_a_lane_quarter(d, dtype):
    """Tiles of at most 32 rows are shared by the four warps of a warpgroup:
    row counts on both sides of that and of the epilogue's block widths, whole
    and split over CTAs."""
    for G, n in ((1, 32), (1, 33), (1, 31), (32, 1), (33, 1), (16, 2), (11, 3), (10, 3), (8, 4),
                 (8, 1), (9, 1), (5, 2), (11, 1), (5, 3), (4, 4), (17, 1)):
        lens = [n, 130, 700 + n]
        for q_lens, kv_lens in (([n] * 3, lens), ([n], [9000])):
            p = make_paged(q_lens, kv_lens, 1, d, 32, dtype, seed=G + n, fill=float("nan"))
            q = queries(p.T, G, d, dtype, 3)
            for max_q in (n, 150):
                o, lse = run(p, q, max_q=max_q)
                assert fattn.device_status() == 0
                check(o, lse, reference(p, q), dtype, max(kv_lens), "G %d n %d max_q %d" % (G, n, max_q))


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    """Mixed units in any order: empty sequences, rows without keys, single
    tokens, drafts, chunks, long and short caches."""
    import random
    rng = random.Random(seed)
    d, Hk = rng.choice([64, 64, 96, 128]), rng.choice([1, 2, 3])
    G = rng.choice([1, 1, 2, 3, 4, 7, 8, 12, 40])
    dtype = rng.choice([torch.bfloat16, torch.float16])
    q_lens, kv_lens = [], []
    for _ in range(rng.randint(1, 14)):
        n = rng.choice([0, 1, 1, 1, rng.randint(2, 9), rng.randint(10, 140), rng.randint(1, 400)])
        L = rng.choice([n, n + rng.randint(0, 300), n + rng.randint(0, 4000), rng.randint(0, 2 * n + 1), 0])
        q_lens.append(n)
        kv_lens.append(L)
    page, causal = rng.choice([16, 32, 64, 128, 256]), rng.random() < 0.8
    p = make_paged(q_lens, kv_lens, Hk, d, page, dtype, seed=seed, fill=float("nan"))
    if p.T == 0:
        pytest.skip("no tokens")
    q = queries(p.T, Hk * G, d, dtype, seed, 1.5)
    o, lse = run(p, q, causal, max_q=p.max_q + rng.randint(0, 50))
    assert fattn.device_status() == 0
    check(o, lse, reference(p, q, causal), dtype, max(kv_lens + [1]),
          "q %s k %s G %d Hk %d d %d page %d" % (q_lens, kv_lens, G, Hk, d, page))


def test_rows_that_see_no_key():
    """More new tokens than keys: the first ones see nothing (o = 0, lse =
    -inf), in units that start, end and lie wholly there; and no keys at all."""
    q_lens, kv_lens = [10, 300, 700, 5, 129, 1], [3, 40, 690, 0, 128, 0]
    for dtype in (torch.bfloat16, torch.float16):
        for Hq, Hk, causal in ((2, 1, True), (2, 2, True), (3, 1, False)):
            p = make_paged(q_lens, kv_lens, Hk, 64, 16, dtype, seed=10, fill=float("nan"))
            q = queries(p.T, Hq, 64, dtype, 4)
            o, lse = run(p, q, causal)
            assert fattn.device_status() == 0
            want = reference(p, q, causal)
            assert bool((want[1] == -float("inf")).any())
            check(o, lse, want, dtype, max(kv_lens))


def test_no_sequence_no_keys_and_pool_of_one_page():
    p = make_paged([0, 0], [0, 5], 2, 128, 16, seed=1)
    q = queries(4, 4, 128, torch.bfloat16, 5).cuda()
    o = torch.full_like(q, 7.0)
    lse = torch.full((4, 4), 7.0, device="cuda")
    fattn.attn_fwd_paged(q, p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(), 1, out=o, lse=lse)
    torch.cuda.synchronize()
    assert bool((o == 7).all()) and bool((lse == 7).all())
    p = make_paged([3], [3], 1, 64, 16, seed=2, spare=0)
    q = queries(3, 1, 64, torch.bfloat16, 6)
    check(*run(p, q), reference(p, q), torch.bfloat16, 3)
    assert fattn.device_status() == 0


def test_rows_behind_the_last_sequence_stay():
    p = make_paged([3, 40], [50, 600], 2, 128, 32, seed=11)
    q = queries(p.T + 30, 6, 128, torch.bfloat16, 7).cuda()
    o = torch.full_like(q, 7.0)
    lse = torch.full((p.T + 30, 6), 7.0, device="cuda")
    q[p.T:] = float("nan")
    fattn.attn_fwd_paged(q, p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(), 40, out=o, lse=lse)
    assert bool((o[p.T:] == 7).all()) and bool((lse[p.T:] == 7).all())
    check(o[:p.T], lse[:p.T], reference(p, q[:p.T].cpu()), torch.bfloat16, 600)
    assert fattn.device_status() == 0


def test_layouts_give_the_same_bits():
    p = make_paged([1, 50, 7], [900, 50, 300], 2, 128, 16, seed=12)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(p.T, 12, 128, generator=g).to(torch.bfloat16).cuda()
    q = qkv[:, 2:8]
    want = run(p, q.contiguous())
    kc = p.k_cache.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    both = torch.stack([p.k_cache, p.v_cache], 1).cuda()
    buf = torch.full((6, p.T, 128 + 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :, :128].transpose(0, 1)
    for k, v, o in ((kc, p.v_cache.cuda(), None), (both[:, 0], both[:, 1], out)):
        table = torch.cat([p.table, p.table], 1).cuda()[:, :p.table.shape[1]]  # a strided table
        lists = (table,) + p.lists()[1:]
        got = fattn.attn_fwd_paged(q, k, v, *lists, 50, out=o)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((buf[:, :, 128:] == 3).all())
    check(*want, reference(p, q.cpu()), torch.bfloat16, 900)
    assert fattn.device_status() == 0


def test_a_page_shared_by_sequences():
    """A common prefix: the same pages in several rows of the table, and one
    page twice in one row."""
    p = make_paged([1, 4, 1], [64, 64, 64], 2, 64, 16, seed=13)
    p.table[1, :3] = p.table[0, :3]
    p.table[2, 1] = p.table[2, 0]
    q = queries(p.T, 4, 64, torch.bfloat16, 8)
    check(*run(p, q), reference(p, q), torch.bfloat16, 64)
    assert fattn.device_status() == 0


def test_scale_wide_logits_and_large_values():
    """Scores spread over hundreds (rescaling on most tiles), a given scale,
    values near fp16's largest."""
    for Hq in (1, 4):
        p = make_paged([1, 200], [3000, 1500], 1, 128, 32, seed=14)
        q = queries(p.T, Hq, 128, torch.bfloat16, 9, 30.0)
        check(*run(p, q, scale=0.2), reference(p, q, scale=0.2), torch.bfloat16, 3000)
        p.v_cache.mul_(12000)
        q = queries(p.T, Hq, 128, torch.bfloat16, 9)
        assert float(p.v_cache.abs().max()) < 65504
        check(*run(p, q), reference(p, q), torch.bfloat16, 3000)
    assert fattn.device_status() == 0
    p.v_cache[int(p.table[0, 0]), 0, 0, 0] = 70000.0
    run(p, q)
    assert fattn.device_status() & 0xff == 5  # FATTN_ERR_RANGE, as attn_fwd
    assert fattn.device_status() == 0


def test_lists_out_of_range_are_reported_and_do_no_harm():
    base = dict(q_lens=[4, 1, 6], kv_lens=[100, 200, 6], Hk=2, d=64, page=16, seed=15)
    p = make_paged(**base)
    q = queries(p.T, 4, 64, torch.bfloat16, 10)
    pools = p.k_cache.cuda(), p.v_cache.cuda()
    fattn.device_status()

    def call(table, cu, kv_len, max_q):
        o, lse = torch.full((p.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(
            (p.T, 4), 7.0, device="cuda")
        fattn.attn_fwd_paged(q.cuda(), *pools, table.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),
                             torch.tensor(kv_len, dtype=torch.int32).cuda(), max_q, out=o, lse=lse)
        return o, lse, fattn.device_status() & 0xff

    want = reference(p, q)
    o, lse, st = call(p.table, p.cu, p.kv_len, 6)
    assert st == 0
    check(o, lse, want, torch.bfloat16, 200)
    # a page outside the pool reads as zeros; the other sequences are right
    for page in (-1, p.k_cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = p.table.clone()
        t[1, 3] = page
        o, lse, st = call(t, p.cu, p.kv_len, 6)
        assert st == 6
        z = make_paged(**base)
        z.k_cache = torch.cat([z.k_cache, torch.zeros_like(z.k_cache[:1])])
        z.v_cache = torch.cat([z.v_cache, torch.zeros_like(z.v_cache[:1])])
        z.table[1, 3] = z.k_cache.shape[0] - 1
        check(o, lse, reference(z, q), torch.bfloat16, 200)
    # lengths past the table's end, negative lengths
    o, lse, st = call(p.table, p.cu, [100, 200, 2 ** 31 - 1], 6)
    assert st == 6
    check(o[:5], lse[:5], tuple(x[:5] for x in want), torch.bfloat16, 200)
    o, lse, st = call(p.table, p.cu, [100, 200, -5], 6)
    assert st == 6 and bool((o[5:] == 0).all()) and bool((lse[5:] == -float("inf")).all())
    # token lists out of order or past the rows: rows that are still some
    # sequence's are written, nothing beyond o
    for cu in ([0, 4, 5, 99], [0, 6, 5, 11], [-4, 4, 5, 11]):
        assert call(p.table, cu, p.kv_len, 6)[2] == 6
    # more new tokens than max_q: only the first max_q rows are served
    o, lse, st = call(p.table, p.cu, p.kv_len, 4)
    assert st == 6 and bool((o[9:] == 7).all())
    check(o[:5], lse[:5], tuple(x[:5] for x in want), torch.bfloat16, 200)
    assert fattn.device_status() == 0


def test_far_pages():
    """Page offsets past 2^31 elements."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB")
    p = make_paged([2, 20], [50, 20], 1, 64, 16, seed=16, spare=0)
    n = p.k_cache.shape[0]
    stride = (1 << 33) // 8 + 4096
    big = torch.zeros(n * stride, dtype=torch.bfloat16, device="cuda")
    kc = torch.as_strided(big, (n, 1, 16, 64), (stride, 1024, 64, 1))
    vc = torch.as_strided(big[2048:], (n, 1, 16, 64), (stride, 1024, 64, 1))
    kc.copy_(p.k_cache)
    vc.copy_(p.v_cache)
    assert (n - 1) * stride > 1 << 32
    q = queries(p.T, 2, 64, torch.bfloat16, 11)
    o, lse = fattn.attn_fwd_paged(q.cuda(), kc, vc, *p.lists(), 20)
    check(o, lse, reference(p, q), torch.bfloat16, 50)


def test_streams_and_replayed_graphs():
    """Two graphs with a workspace each, replayed after the lists, the queries
    and the cache changed; a call on another stream."""
    p = make_paged([1] * 6, [40 * i + 1 for i in range(6)], 2, 128, 16, seed=17, extra_cols=20)
    g = torch.Generator().manual_seed(3)
    table = torch.randint(0, p.k_cache.shape[0], p.table.shape, generator=g, dtype=torch.int32)
    p.table = table
    q = queries(p.T, 8, 128, torch.bfloat16, 12).cuda()
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    lists = p.lists()
    want = fattn.attn_fwd_paged(q, kc, vc, *lists, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fattn.attn_fwd_paged(q, kc, vc, *lists, 1, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs, outs = [], []
    for _ in range(2):
        ws = torch.empty(fattn.paged_workspace_size(8, 2, 128, 1), dtype=torch.uint8, device="cuda")
        o, lse = torch.empty_like(q), torch.empty(p.T, 8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fattn.attn_fwd_paged(q, kc, vc, *lists, 1, workspace=ws, out=o, lse=lse)
        graphs.append(graph)
        outs.append((ws, o, lse))
    lens = [200, 17, 0, 300, 1, 129]
    p.kv_len = lens
    lists[2].copy_(torch.tensor(lens, dtype=torch.int32))
    q.mul_(0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs[0].replay()
    with torch.cuda.stream(side):
        graphs[1].replay()
    torch.cuda.synchronize()
    want = reference(p, q.cpu())
    for _, o, lse in outs:
        check(o, lse, want, torch.bfloat16, 300)
    assert torch.equal(outs[0][1], outs[1][1])
    assert fattn.device_status() == 0


def test_two_calls_at_once():
    """Two streams, a workspace each, both filling the GPU; many times."""
    cases = []
    for seed, (q_lens, kv_lens, d) in enumerate((([1] * 12, [3000 + 17 * i for i in range(12)], 128),
                                                 ([200, 1, 60], [900, 4000, 60], 64))):
        p = make_paged(q_lens, kv_lens, 4, d, 32, seed=30 + seed)
        q = queries(p.T, 8, d, torch.bfloat16, 14 + seed).cuda()
        args = (q, p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(), p.max_q)
        cases.append((args, fattn.attn_fwd_paged(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for args, _, s in cases:
            got.append(fattn.attn_fwd_paged(*args, stream=s))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        want = cases[i % 2][1]
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert fattn.device_status() == 0


def test_a_captured_step_behind_copies_and_a_joined_stream():
    """Copies, the append and the attention in one graph, the queries produced
    on another stream that joins before the attention: the attention is
    launched ahead of its predecessors and has to wait for them."""
    p = make_paged([1] * 4, [300, 40, 129, 700], 2, 128, 16, seed=33)
    g = torch.Generator().manual_seed(1)
    steps = [[torch.randn(4, h, 128, generator=g).to(torch.bfloat16) for h in (8, 2, 2)] for _ in range(6)]
    q, k, v = [torch.zeros_like(t).cuda() for t in steps[0]]
    src = [torch.zeros_like(t).cuda() for t in steps[0]]
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    lists = p.lists()
    o, lse = torch.empty_like(q), torch.empty(4, 8, device="cuda")
    ws = torch.empty(fattn.paged_workspace_size(8, 2, 128, 1), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        k.copy_(src[1])
        v.copy_(src[2])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q.copy_(src[0])
            q.mul_(0.5)
        fattn.kv_append(k, v, kc, vc, *lists)
        main.wait_stream(side)
        fattn.attn_fwd_paged(q, kc, vc, *lists, 1, workspace=ws, out=o, lse=lse)
        q.zero_()
    for step in steps:
        for a, b in zip(src, step):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(4):
            at = p.kv_len[b] - 1
            page = int(p.table[b, at // 16])
            p.k_cache[page, :, at % 16], p.v_cache[page, :, at % 16] = step[1][b], step[2][b]
        check(o, lse, reference(p, step[0] * 0.5), torch.bfloat16, 700)
    assert fattn.device_status() == 0


@pytest.mark.parametrize("d", [64, 96, 128])
def test_agrees_with_the_dense_forward(d):
    """A prompt whose pages are one contiguous buffer, whole and in chunks,
    against attn_fwd on the same tensors: both within their bounds of the same
    reference."""
    H, N = 2, 500
    g = torch.Generator().manual_seed(d)
    q, k, v = [torch.randn(1, H, N, d, generator=g).to(torch.bfloat16) for _ in range(3)]
    o, lse = fattn.attn_fwd(q.cuda(), k.cuda(), v.cuda(), causal=True)
    kc, vc = [torch.cat([t[0], torch.zeros(H, 12, d).bfloat16()], 1).reshape(H, 32, 16, d)
              .transpose(0, 1).contiguous() for t in (k, v)]
    p = make_paged([N], [N], H, d, 16, seed=1)
    p.k_cache, p.v_cache, p.table = kc, vc, torch.arange(32, dtype=torch.int32)[None]
    qt = q[0].transpose(0, 1).contiguous()
    want = reference(p, qt)
    check(o[0].transpose(0, 1), lse[0].T, want, torch.bfloat16, N)
    whole = run(p, qt)
    check(*whole, want, torch.bfloat16, N)
    at = 0
    for n in (1, 130, 69, 300):
        part = make_paged([n], [at + n], H, d, 16, seed=1)
        part.k_cache, part.v_cache, part.table = kc, vc, p.table
        got = run(part, qt[at:at + n])
        check(*got, tuple(x[at:at + n] for x in want), torch.bfloat16, N, "rows %d.." % at)
        at += n
    assert fattn.device_status() == 0


@pytest.mark.parametrize("dtype,d,Hq,Hk,inter", [(torch.bfloat16, 128, 8, 2, False),
                                                 (torch.float16, 64, 3, 3, True)])
def test_serving_steps_together(dtype, d, Hq, Hk, inter):
    """Prompts, then decode steps with a sequence that joins later, in one
    captured graph per kind of step's sizes: qk_norm_rope -> kv_append ->
    attn_fwd_paged, against fp64 from the projections.  q, k are rounded once
    by the norm and the turned k once more in the cache (half a step each:
    scores off by at most 3 half * sum |q k|), then the attention's own
    bounds."""
    page, rot = 16, 32
    g = torch.Generator().manual_seed(21)
    wq, wk = [(1 + 0.2 * torch.randn(d, generator=g)).to(dtype) for _ in range(2)]
    rope = fattn.rope_table(512, rot)
    total = [90, 33, 70]
    joins = [0, 0, 2]
    data = [torch.randn(n, Hq + 2 * Hk, d, generator=g).to(dtype) for n in total]
    # fp64 of the whole sequences
    half = torch.finfo(dtype).eps / 2
    want = []
    for x in data:
        n = x.shape[0]
        ang = rope.cpu()[:n][None, None]
        qn = ref.norm_rope(x[:, :Hq].transpose(0, 1)[None], wq, None, 1e-6, inter)
        kn = ref.norm_rope(x[:, Hq:Hq + Hk].transpose(0, 1)[None], wk, None, 1e-6, inter)
        qn, kn = ref.turn(qn, ang, inter)[0], ref.turn(kn, ang, inter)[0]
        v = x[:, Hq + Hk:].transpose(0, 1).double()
        kn, v = kn.repeat_interleave(Hq // Hk, 0), v.repeat_interleave(Hq // Hk, 0)
        s = qn @ kn.transpose(1, 2) * d ** -0.5
        e = 3 * half * (qn.abs() @ kn.abs().transpose(1, 2)).amax(-1) * d ** -0.5
        s = s.masked_fill(torch.ones(n, n).triu(1).bool(), -float("inf"))
        p = torch.softmax(s, -1)
        want.append((p @ v, p @ v.abs(), e))
    pages = torch.randperm(40, generator=g).int()
    table = torch.stack([pages[i * 8:(i + 1) * 8] for i in range(3)]).cuda()
    kc = torch.full((40, Hk, page, d), float("nan"), dtype=dtype, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    done, step, checked = [0, 0, 0], 0, 0
    cwq, cwk = wq.cuda(), wk.cuda()
    while any(a < b for a, b in zip(done, total)):
        news = [0 if step < joins[i] else min(40 if done[i] == 0 else 1 + step % 3, total[i] - done[i])
                for i in range(3)]
        x = torch.cat([data[i][done[i]:done[i] + news[i]] for i in range(3)]).cuda()
        pos = torch.cat([torch.arange(done[i], done[i] + news[i]) for i in range(3)])
        done = [a + b for a, b in zip(done, news)]
        cu = torch.tensor([0] + news).cumsum(0).int().cuda()
        kv_len = torch.tensor(done, dtype=torch.int32).cuda()
        q = x[:, :Hq].transpose(0, 1)[None]
        k = x[:, Hq:Hq + Hk].transpose(0, 1)[None]
        qo, _ = fattn.qk_norm_rope(q, None, cwq, None, rope, pos.int()[None].cuda(), interleaved=inter)
        _, ko = fattn.qk_norm_rope(None, k, None, cwk, interleaved=inter)  # turned by the append
        fattn.kv_append(ko[0].transpose(0, 1), x[:, Hq + Hk:], kc, vc, table, cu, kv_len, rope=rope,
                        interleaved=inter)
        o, lse = fattn.attn_fwd_paged(qo[0].transpose(0, 1), kc, vc, table, cu, kv_len,
                                      max(max(news), 1))
        o, at = o.double().cpu(), 0
        for i in range(3):
            rows = slice(done[i] - news[i], done[i])
            wo, size, e = (t[:, rows] for t in want[i])
            got = o[at:at + news[i]].transpose(0, 1)
            # e moves p by e and the normaliser by e
            tol = half * wo.abs() + (2.0 ** -11 + 2 * e[..., None] * 1.1 + 2.0 ** -14) * size + 2e-6
            assert bool(((got - wo).abs() <= tol).all()), (step, i)
            at += news[i]
            checked += got.numel()
        step += 1
    assert checked == sum(total) * Hq * d
    assert fattn.device_status() == 0
