"""GPU tests of attn_bwd_cross against the fp64 formula, element by element
within bounds that follow from the roundings: odd sizes, shared heads, ragged
lengths, padding that holds anything, few keys under many queries and the
reverse, small gradients, views, graphs and streams."""
import pytest
import torch

from tests import search_ref as ref
from tests.test_cross_gpu import make
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def dout(q, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(q.shape, generator=g) * size).to(dtype)


def saved(q, k, v, lens, scale):
    """o and lse as a forward pass without errors of its own leaves them."""
    o, lse, *_ = ref.cross(q, k, v, lens, scale)
    return o.to(q.dtype), lse.float()


def run(q, k, v, o, lse, do, lens, **kw):
    kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    return fattn.attn_bwd_cross(*(t.cuda() for t in (q, k, v, o, lse, do)), kv_len=kv_len, **kw)


def verify(got, q, k, v, do, lens, what="", scale=None, o_err=None):
    scale = fattn.default_scale(q.shape[-1]) if scale is None else scale
    want, tol = ref.cross_bwd(q, k, v, do, lens, scale, q.dtype, o_err)
    for name, g, w, t in zip(("dq", "dk", "dv"), got, want, tol):
        g = g.double().cpu()
        assert bool(torch.isfinite(g).all()), "%s %s" % (what, name)
        err = (g - w).abs()
        bad = err > t * (1 + 1e-9)
        assert not bool(bad.any()), "%s %s: %d of %d beyond the bound, worst ratio %.3g" % (
            what, name, int(bad.sum()), bad.numel(), float((err / t.clamp(min=1e-300)).max()))


def both(B, Hq, Hk, Nq, Nk, d, dtype, lens, seed=0, size=1.0, **kw):
    q, k, v = make(B, Hq, Hk, Nq, Nk, d, dtype, seed=seed, lens=lens, **kw)
    do = dout(q, dtype, seed + 1, size)
    scale = fattn.default_scale(d)
    got = run(q, k, v, *saved(q, k, v, lens, scale), do, lens)
    return got, q, k, v, do


CASES = [
    # B, Hq, Hk, Nq, Nk, d, lens
    (1, 1, 1, 1, 1, 64, None),
    (1, 1, 1, 1, 300, 128, None),
    (1, 1, 1, 300, 1, 64, None),
    (1, 2, 2, 128, 128, 64, None),
    (1, 1, 1, 129, 127, 128, None),
    (2, 2, 1, 128, 256, 96, None),
    (3, 12, 4, 333, 501, 64, [501, 128, 77]),
    (2, 3, 3, 200, 260, 96, [260, 129]),
    (4, 3, 3, 129, 257, 128, [0, 257, 127, 256]),     # a sequence without keys
    (2, 16, 1, 40, 50, 64, [50, 0]),                  # sixteen heads share one
    (1, 4, 2, 2000, 77, 64, [77]),                    # one key tile under many queries
    (2, 2, 2, 1500, 154, 128, [154, 51]),
    (1, 1, 1, 20, 3000, 64, None),                    # one query tile, many keys
    (300, 1, 1, 5, 9, 64, [i % 10 for i in range(300)]),
    (7, 40, 20, 130, 200, 64, [200, 1, 128, 129, 60, 0, 199]),   # several units a CTA
    (4, 40, 40, 150, 200, 128, None),
    (1, 1, 1, 1000, 1000, 128, None),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Hq,Hk,Nq,Nk,d,lens", CASES,
                         ids=["B%d_H%d-%d_q%d_k%d_d%d%s" % (*c[:6], "_ragged" if c[6] else "") for c in CASES])
def test_against_the_formula(B, Hq, Hk, Nq, Nk, d, lens, dtype):
    got, q, k, v, do = both(B, Hq, Hk, Nq, Nk, d, dtype, lens, seed=Nq + Nk)
    assert fattn.device_status() == 0
    verify(got, q, k, v, do, lens)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf"), 6e4])
def test_padding_may_hold_anything(fill, dtype):
    lens = [1, 100, 128, 200, 0, 255]
    for d in (64, 96):
        got, q, k, v, do = both(6, 4, 2, 130, 256, d, dtype, lens, seed=4, fill=fill)
        assert fattn.device_status() == 0
        verify(got, q, k, v, do, lens, str(fill))
        for b, n in enumerate(lens):
            assert bool((got[1][b, :, n:] == 0).all()) and bool((got[2][b, :, n:] == 0).all())


@pytest.mark.parametrize("dtype,size", [(torch.float16, 2.0 ** -14), (torch.float16, 2.0 ** -20),
                                        (torch.float16, 500.0), (torch.bfloat16, 1e-20),
                                        (torch.bfloat16, 1e6)])
def test_small_and_large_gradients(dtype, size):
    """dS of a thousand keys is a thousandth of dP: below fp16's normal numbers
    without its scaling."""
    got, q, k, v, do = both(1, 2, 1, 200, 1000, 64, dtype, [1000], seed=5, size=size, scale=0.5)
    verify(got, q, k, v, do, [1000], "size %g" % size)


def test_a_zero_gradient():
    for dtype in (torch.bfloat16, torch.float16):
        got, *_ = both(2, 2, 1, 70, 90, 64, dtype, [90, 30], size=0.0)
        assert all(bool((g == 0).all()) for g in got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_forward_and_backward_together_on_packed_views(dtype):
    """q [B, Nq, Hq, d], keys and values [B, Nk, 2, Hk, d], the forward's own o
    and lse, gradients into one packed [B, Nk, 2, Hk, d] buffer."""
    g = torch.Generator().manual_seed(6)
    B, Hq, Hk, Nq, Nk, d = 3, 6, 2, 170, 150, 128
    lens = [150, 33, 128]
    q = torch.randn(B, Nq, Hq, d, generator=g).to(dtype).transpose(1, 2)
    kv = torch.randn(B, Nk, 2, Hk, d, generator=g).to(dtype)
    do = torch.randn(B, Nq, Hq, d, generator=g).to(dtype).transpose(1, 2)
    k, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    kvg, lg = kv.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    qg, dog = q.cuda(), do.cuda()
    kg, vg = kvg[:, :, 0].transpose(1, 2), kvg[:, :, 1].transpose(1, 2)
    o, lse = fattn.attn_fwd_cross(qg, kg, vg, kv_len=lg, scale=0.1)
    dkv = torch.full((B, Nk, 2, Hk, d), 9.0, dtype=dtype, device="cuda")
    got = fattn.attn_bwd_cross(qg, kg, vg, o, lse, dog, kv_len=lg, scale=0.1,
                               dk=dkv[:, :, 0].transpose(1, 2), dv=dkv[:, :, 1].transpose(1, 2))
    assert fattn.device_status() == 0
    # o as the forward pass is allowed to leave it (its own test's bound)
    wo, wl, size, terms, vmax = ref.cross(q, k, v, lens, 0.1)
    U, half = 2.0 ** -24, torch.finfo(dtype).eps / 2
    e = (d + 6) * U * terms + 2.0 ** -22 + (Nk + 64) * U
    o_err = half * wo.abs() + (1 + half) * ((2.0 ** -11 + 2 * e)[..., None] * size +
                                            Nk * 2.0 ** -25 * vmax[..., None]) + 2.0 ** -25
    verify(got, q, k, v, do, lens, scale=0.1, o_err=o_err)


@pytest.mark.parametrize("empty", ["queries", "keys"])
def test_without_queries_or_keys(empty):
    Nq, Nk = (0, 70) if empty == "queries" else (70, 0)
    q = torch.randn(2, 4, Nq, 64).bfloat16().cuda()
    k = torch.randn(2, 2, Nk, 64).bfloat16().cuda()
    lse = torch.full((2, 4, Nq), -float("inf"), device="cuda")
    outs = [torch.full_like(t, 5) for t in (q, k, k)]
    got = fattn.attn_bwd_cross(q, k, k, torch.zeros_like(q), lse, q, dq=outs[0], dk=outs[1], dv=outs[2])
    assert all(bool((g == 0).all()) for g in got) and fattn.device_status() == 0


@pytest.mark.parametrize("bad", [-1, 301, 2 ** 31 - 1, -2 ** 31])
def test_lengths_out_of_range_are_brought_into_it(bad):
    lens = [min(max(bad, 0), 300), 40]
    q, k, v = make(2, 2, 2, 30, 300, 64, torch.bfloat16, seed=7)
    do = dout(q, torch.bfloat16, 8)
    got = run(q, k, v, *saved(q, k, v, lens, 0.125), do, [bad, 40])
    assert fattn.device_status() & 0xffff == 6 | 12 << 8
    verify(got, q, k, v, do, lens)


def test_equal_calls_give_equal_bits_and_streams_do_not_meet():
    shapes = [(2, 8, 2, 700, 90, 64, [90, 33]), (1, 3, 3, 300, 900, 128, None)]
    sets, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for B, Hq, Hk, Nq, Nk, d, lens in shapes:
        q, k, v = make(B, Hq, Hk, Nq, Nk, d, torch.bfloat16, seed=9, lens=lens)
        do = dout(q, torch.bfloat16, 10)
        kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        sets.append(([t.cuda() for t in (q, k, v, *saved(q, k, v, lens, d ** -0.5), do)], kv_len))
    alone = [fattn.attn_bwd_cross(*a, kv_len=n) for a, n in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [fattn.attn_bwd_cross(*a, kv_len=n, stream=s) for (a, n), s in zip(sets, streams)]
        torch.cuda.synchronize()
        for x, y in zip(got, alone):
            assert all(torch.equal(i, j) for i, j in zip(x, y))
    assert fattn.device_status() == 0


def test_a_captured_call_follows_its_lengths():
    q, k, v = make(2, 4, 2, 200, 300, 64, torch.float16, seed=11)
    do = dout(q, torch.float16, 12)
    lens = torch.tensor([300, 300], dtype=torch.int32, device="cuda")
    t = [x.cuda() for x in (q, k, v, *saved(q, k, v, None, 0.125), do)]
    out = [torch.empty_like(t[i]) for i in (0, 1, 2)]
    ws = torch.empty(fattn.cross_bwd_workspace_size(2, 4, 2, 200, 300, 64), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fattn.attn_bwd_cross(*t, kv_len=lens, dq=out[0], dk=out[1], dv=out[2], workspace=ws)
    for n in ([300, 40], [0, 300], [129, 128]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        o, lse = saved(q, k, v, n, 0.125)
        t[3].copy_(o)
        t[4].copy_(lse)
        graph.replay()
        torch.cuda.synchronize()
        verify(out, q, k, v, do, n, str(n))
    assert fattn.device_status() == 0


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
def test_inputs_changed_in_place(d, dtype):
    """Calls one behind the other on the same buffers, whose contents and lengths
    change before each: none reads what the one before has left in a cache."""
    g = torch.Generator().manual_seed(17)
    B, H, Hk, Nq, Nk = 3, 4, 2, 300, 400
    sets = []
    for i in range(2):
        q, do = ((torch.randn(B, H, Nq, d, generator=g) * (1 + 7 * i)).to(dtype).cuda() for _ in range(2))
        k, v = (torch.randn(B, Hk, Nk, d, generator=g).to(dtype).cuda() for _ in range(2))
        kv_len = torch.tensor([[400, 1, 129], [7, 400, 256]][i], dtype=torch.int32, device="cuda")
        o, lse = fattn.attn_fwd_cross(q, k, v, kv_len)
        ins = (q, k, v, o, lse, do, kv_len)
        sets.append((ins, fattn.attn_bwd_cross(*ins)))
    bufs = [torch.empty_like(t) for t in sets[0][0]]
    outs = [torch.empty_like(t) for t in sets[0][1]]
    ws = torch.empty(fattn.cross_bwd_workspace_size(B, H, Hk, Nq, Nk, d), dtype=torch.uint8, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for n in range(200):
        ins, want = sets[n % 2]
        for to, t in zip(bufs, ins):
            to.copy_(t)
        fattn.attn_bwd_cross(*bufs, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
        for x, y in zip(outs, want):
            wrong += (x != y).sum()
    assert int(wrong) == 0 and fattn.device_status() == 0


@pytest.mark.parametrize("d,Nq,Nk", [(64, 2048, 2048), (64, 2048, 200), (96, 900, 900), (128, 1024, 1024)])
def test_many_calls_in_a_row(d, Nq, Nk):
    """No wait of the pipelines ever runs out, whatever the warps' order: some
    thousand calls of many tiles, the last one's bits the first one's."""
    g = torch.Generator().manual_seed(13)
    q, do = (torch.randn(4, 8, Nq, d, generator=g).bfloat16().cuda() for _ in range(2))
    k, v = (torch.randn(4, 8, Nk, d, generator=g).bfloat16().cuda() for _ in range(2))
    o, lse = fattn.attn_fwd_cross(q, k, v)
    first = fattn.attn_bwd_cross(q, k, v, o, lse, do)
    outs = [torch.empty_like(t) for t in first]
    ws = torch.empty(fattn.cross_bwd_workspace_size(4, 8, 8, Nq, Nk, d), dtype=torch.uint8, device="cuda")
    for _ in range(2000):
        fattn.attn_bwd_cross(q, k, v, o, lse, do, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
    torch.cuda.synchronize()
    assert fattn.device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(first, outs))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("G,Nq,d", [(1, 3, 64), (4, 300, 128), (8, 2000, 64), (2, 77, 96)])
def test_one_key_has_no_gradient_but_its_values(G, Nq, d, dtype):
    """A softmax over one key is 1 whatever q and k are; units whole and split."""
    q, k, v = (t.cuda() for t in make(3, 2 * G, 2, Nq, 40, d, dtype, seed=d, lens=[1, 40, 1]))
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    kv_len = torch.tensor([1, 40, 1], dtype=torch.int32, device="cuda")
    o, lse = fattn.attn_fwd_cross(q, k, v, kv_len)
    dq, dk, dv = fattn.attn_bwd_cross(q, k, v, o, lse, do, kv_len)
    for b in (0, 2):
        assert not dq[b].any() and not dk[b].any() and not dv[b, :, 1:].any()
        # P is 1 in the inputs' type (its exponent is off by some 1e-6), so dv is a sum
        # of G Nq values in fp32, each addition off by at most 2^-23 of all their sizes,
        # and rounded once.
        x = do[b].double().reshape(2, G * Nq, d)
        bound = torch.finfo(dtype).eps / 2 * x.sum(1).abs() + 1.01 * G * Nq * 2 ** -23 * x.abs().sum(1)
        assert bool(((dv[b, :, 0].double() - x.sum(1)).abs() <= bound).all())
    assert bool(dq[1].any()) and bool(dk[1].any()) and fattn.device_status() == 0
