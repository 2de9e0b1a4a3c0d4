"""GPU tests of qk_norm_rope and its backward pass against the fp64 reference:
head dimensions, both element types, both pairings, partial and absent
rotations, absent norms and tensors, strided views, in place, given positions,
and the places where it can go wrong (one token, ragged warps, positions out
of the table, other streams, graphs)."""
import itertools

import pytest
import torch

from tests import serving_ref as ref
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu

EPS = 1e-6
U = 2.0 ** -24  # half a step of fp32, relative

# Bounds, first order in U.  A row's statistic sums d squares (every term
# passes through at most d additions), one division, one addition, rsqrtf (2
# ulp): relative error of r at most (d/2 + 6) U with its square root halving
# the sum's.  The turned element adds a product with the table's angle, the
# folded weight and one fused add: 8 U of the terms' size in all.  The store
# rounds by half a step of the type, relative to the value (2^-25 absolute for
# fp16 subnormals).


def half(dtype):
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def check(got, want, size, d, dtype, what):
    got = got.double().cpu()
    rel = (d / 2 + 14) * U
    tol = half(dtype) * want.abs() + (1 + half(dtype)) * rel * size + floor_of(dtype)
    err = (got - want).abs()
    assert torch.isfinite(got).all(), what
    bad = err > tol * (1 + 1e-9)
    assert not bad.any(), "%s: %d of %d beyond the bound, worst %.3g at tolerance %.3g" % (
        what, int(bad.sum()), bad.numel(), float(err[bad].max()), float(tol[bad].min()))


def make(B, H, N, d, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, H, N, d, generator=g) * scale).to(dtype)


def weights(d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)


def angles_of(rope, positions, B, N):
    if rope is None:
        return None
    pos = torch.arange(N).expand(B, N) if positions is None else positions.long()
    return rope[pos][:, None]


def setup(B, Hq, Hk, N, d, dtype, rot, positions=False, norm=True, seed=0):
    q, k = make(B, Hq, N, d, dtype, seed, 1.7), make(B, Hk, N, d, dtype, seed + 1, 0.6)
    wq = weights(d, dtype, seed + 2) if norm else None
    wk = weights(d, dtype, seed + 3) if norm else None
    rope = ref.rope_rows(max(N, 4096), rot) if rot else None
    pos = None
    if positions:
        g = torch.Generator().manual_seed(seed + 4)
        pos = torch.randint(0, 4096, (B, N), generator=g, dtype=torch.int32)
    return q, k, wq, wk, rope, pos


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


CASES = [
    # B, Hq, Hk, N, d, rot, interleaved, positions, norm
    (1, 1, 1, 1, 64, 64, False, True, True),
    (1, 8, 2, 1, 128, 128, False, True, True),
    (2, 3, 1, 37, 128, 128, False, False, True),
    (3, 5, 5, 33, 64, 32, False, False, True),
    (2, 4, 2, 50, 96, 96, False, True, True),
    (1, 9, 3, 65, 96, 64, True, False, True),
    (2, 6, 2, 21, 256, 256, False, False, True),
    (1, 7, 1, 19, 256, 16, True, True, True),
    (2, 16, 4, 130, 128, 128, True, False, True),
    (2, 2, 2, 40, 64, 0, False, False, True),
    (2, 4, 2, 40, 128, 128, False, True, False),
    (1, 4, 4, 77, 96, 96, True, False, False),
    (1, 33, 1, 300, 64, 48, False, False, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot,inter,positions,norm", CASES)
def test_forward(B, Hq, Hk, N, d, rot, inter, positions, norm, dtype):
    q, k, wq, wk, rope, pos = setup(B, Hq, Hk, N, d, dtype, rot, positions, norm, seed=N + d)
    out = fattn.qk_norm_rope(*cuda(q, k, wq, wk, rope, pos), eps=EPS, interleaved=inter)
    ang = angles_of(rope, pos, B, N)
    for got, x, w, what in zip(out, (q, k), (wq, wk), "qk"):
        want = ref.norm_rope(x, w, ang, EPS, inter)
        size = ref.g_terms(ref.norm_rope(x, w, None, EPS, inter), ang, inter)
        check(got, want, size, d, dtype, what)
    assert fattn.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot,inter,positions,norm", CASES)
def test_backward(B, Hq, Hk, N, d, rot, inter, positions, norm, dtype):
    q, k, wq, wk, rope, pos = setup(B, Hq, Hk, N, d, dtype, rot, positions, norm, seed=N + d + 9)
    gq, gk = make(B, Hq, N, d, dtype, 77), make(B, Hk, N, d, dtype, 78, 3.0)
    out = fattn.qk_norm_rope_bwd(*cuda(gq, gk, q, k, wq, wk, rope, pos), eps=EPS, interleaved=inter)
    ang = angles_of(rope, pos, B, N)
    for i, (g, x, w, H) in enumerate(((gq, q, wq, Hq), (gk, k, wk, Hk))):
        dx, dw, size, dw_size = ref.norm_rope_bwd(g, x, w, ang, EPS, inter)
        # two statistics enter each term, and r three times in the second
        check(out[i], dx, 4 * size, d, dtype, "d" + "qk"[i])
        if w is None:
            assert out[2 + i] is None
            continue
        # Each term carries r's error and the turn's; a lane adds the rows of
        # its heads and items (one item a warp at these sizes), then 4 rows of
        # a warp, 4 warps, and the blocks in fp64.
        rel = (d / 2 + 16 + H + 8) * U
        err = (out[2 + i].double().cpu() - dw).abs()
        assert bool((err <= rel * dw_size + U * dw.abs()).all()), float((err / dw_size).max() / U)
    assert fattn.device_status() == 0


def test_weight_gradient_over_many_rows():
    """More items than the grid has warps: lanes add many rows each."""
    B, H, N, d = 2, 8, 16000, 64
    q, k, wq, wk, rope, pos = setup(B, H, 1, N, d, torch.bfloat16, 64, seed=5)
    gq, gk = make(B, H, N, d, torch.bfloat16, 6), make(B, 1, N, d, torch.bfloat16, 7)
    out = fattn.qk_norm_rope_bwd(*cuda(gq, gk, q, k, wq, wk, rope, pos), eps=EPS)
    again = fattn.qk_norm_rope_bwd(*cuda(gq, gk, q, k, wq, wk, rope, pos), eps=EPS)
    ang = angles_of(rope, pos, B, N)
    warps = 8 * torch.cuda.get_device_properties(0).multi_processor_count * 4
    for i, (g, x, w, h) in enumerate(((gq, q, wq, H), (gk, k, wk, 1))):
        _, dw, _, dw_size = ref.norm_rope_bwd(g, x, w, ang, EPS, False)
        rows_a_lane = -(-B * N * 2 * H // (4 * warps)) * H + H
        err = (out[2 + i].double().cpu() - dw).abs()
        assert bool((err <= (d / 2 + 24 + rows_a_lane) * U * dw_size).all())
        assert torch.equal(out[2 + i], again[2 + i]), "equal calls give equal bits"


def test_gradients_against_differences():
    """<dy, f(x + h u) - f(x - h u)> / 2h of the fp64 forward formula against
    the kernel's <dx, u> and <dw, u>.  Central differences of a smooth
    function: error O(h^2) = 1e-8 of the terms, far below the kernel's bf16
    rounding of dx (2^-9 of each element, random signs)."""
    B, H, N, d, rot = 1, 2, 11, 64, 32
    q, k, wq, wk, rope, pos = setup(B, H, 1, N, d, torch.bfloat16, rot, seed=31)
    gq, gk = make(B, H, N, d, torch.bfloat16, 8), make(B, 1, N, d, torch.bfloat16, 9)
    out = [t.double().cpu() for t in
           fattn.qk_norm_rope_bwd(*cuda(gq, gk, q, k, wq, wk, rope, pos), eps=EPS)]
    ang = angles_of(rope, pos, B, N)
    h = 1e-4
    for i, (g, x, w) in enumerate(((gq, q, wq), (gk, k, wk))):
        for seed in range(3):
            gen = torch.Generator().manual_seed(seed)
            u = torch.randn(x.shape, generator=gen, dtype=torch.float64)
            f = [(g.double() * ref.norm_rope(x.double() + s * h * u, w, ang, EPS, False)).sum()
                 for s in (1, -1)]
            want, got = (f[0] - f[1]) / (2 * h), (out[i] * u).sum()
            tol = half(torch.bfloat16) * (out[i] * u).abs().sum() + 1e-5 * (g.double() * u).abs().sum()
            assert abs(want - got) <= tol
            u = torch.randn(d, generator=gen, dtype=torch.float64)
            f = [(g.double() * ref.norm_rope(x, w.double() + s * h * u, ang, EPS, False)).sum()
                 for s in (1, -1)]
            want, got = (f[0] - f[1]) / (2 * h), (out[2 + i] * u).sum()
            assert abs(want - got) <= 1e-5 * (out[2 + i] * u).abs().sum() + 1e-4


@pytest.mark.parametrize("d,inter", [(128, False), (96, True)])
def test_views_of_a_packed_projection_in_place(d, inter):
    """q and k as windows of one [B, N, (Hq + 2 Hk), d] buffer, turned in
    place: the same bits as apart, the values' window untouched."""
    B, Hq, Hk, N = 2, 6, 2, 45
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(B, N, Hq + 2 * Hk, d, generator=g).to(torch.bfloat16).cuda()
    before = qkv.clone()
    wq, wk = weights(d, torch.bfloat16, 1).cuda(), weights(d, torch.bfloat16, 2).cuda()
    rope = ref.rope_rows(64, 64).cuda()
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hk].transpose(1, 2)
    want = fattn.qk_norm_rope(q.contiguous(), k.contiguous(), wq, wk, rope, eps=EPS, interleaved=inter)
    fattn.qk_norm_rope(q, k, wq, wk, rope, eps=EPS, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, :, Hq + Hk:], before[:, :, Hq + Hk:])
    # the gradients in place of the upstream ones
    dy = torch.randn(B, N, Hq + 2 * Hk, d, generator=g).to(torch.bfloat16).cuda()
    gq, gk = dy[:, :, :Hq].transpose(1, 2), dy[:, :, Hq:Hq + Hk].transpose(1, 2)
    xq, xk = before[:, :, :Hq].transpose(1, 2), before[:, :, Hq:Hq + Hk].transpose(1, 2)
    want = fattn.qk_norm_rope_bwd(gq.contiguous(), gk.contiguous(), xq, xk, wq, wk, rope, eps=EPS,
                                  interleaved=inter)
    got = fattn.qk_norm_rope_bwd(gq, gk, xq, xk, wq, wk, rope, eps=EPS, interleaved=inter, dq=gq,
                                 dk=gk)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_one_tensor_alone_and_no_rows():
    q, k, wq, wk, rope, pos = setup(2, 4, 2, 30, 128, torch.bfloat16, 128, seed=8)
    q, k, wq, wk, rope = cuda(q, k, wq, wk, rope)
    both = fattn.qk_norm_rope(q, k, wq, wk, rope)
    alone_q, none = fattn.qk_norm_rope(q, None, wq, None, rope)
    assert none is None and torch.equal(alone_q, both[0])
    none, alone_k = fattn.qk_norm_rope(None, k, None, wk, rope)
    assert none is None and torch.equal(alone_k, both[1])
    grads = fattn.qk_norm_rope_bwd(q, k, q, k, wq, wk, rope)
    only = fattn.qk_norm_rope_bwd(None, k, None, k, None, wk, rope)
    assert only[0] is None and only[2] is None
    assert torch.equal(only[1], grads[1])
    # The same rows on other warps: each sum within its bound of the exact one.
    kc, wkc = k.cpu(), wk.cpu()
    size = ref.norm_rope_bwd(kc, kc, wkc, angles_of(rope.cpu(), None, 2, 30), 1e-6, False)[3]
    err = (only[3] - grads[3]).double().abs().cpu()
    assert bool((err <= 2 * (128 / 2 + 16 + 2 + 8) * U * size).all())
    # mixed: a norm for q only
    mixed = fattn.qk_norm_rope(q, k, wq, None, rope)
    assert torch.equal(mixed[0], both[0])
    e = q[:, :, :0]
    out = fattn.qk_norm_rope(e, None, wq, None, rope)
    assert out[0].shape == e.shape
    out = fattn.qk_norm_rope_bwd(e, None, e, None, wq, None, rope)
    assert float(out[2].abs().max()) == 0.0


def test_positions_out_of_the_table_are_left_out_and_reported():
    q, k, wq, wk, rope, _ = setup(1, 3, 1, 9, 64, torch.bfloat16, 64, seed=12)
    pos = torch.tensor([[0, 4095, 4096, -1, 7, 2 ** 31 - 1, 8, -2 ** 31, 9]], dtype=torch.int32)
    bad = [2, 3, 5, 7]
    good = [i for i in range(9) if i not in bad]
    args = cuda(q, k, wq, wk, rope, pos)
    q_out, k_out = torch.full_like(args[0], 7.0), torch.full_like(args[1], 7.0)
    fattn.device_status()
    fattn.qk_norm_rope(*args, eps=EPS, q_out=q_out, k_out=k_out)
    assert fattn.device_status() & 0xff == 6
    assert bool((q_out[:, :, bad] == 7).all()) and bool((k_out[:, :, bad] == 7).all())
    safe = pos.clone()
    safe[0, bad] = 0
    want = fattn.qk_norm_rope(*cuda(q, k, wq, wk, rope, safe), eps=EPS)
    assert torch.equal(q_out[:, :, good], want[0][:, :, good])
    # their rows add nothing to the weights' gradients
    out = fattn.qk_norm_rope_bwd(args[0], args[1], *args, eps=EPS)
    assert fattn.device_status() & 0xff == 6
    keep = [args[0][:, :, good].contiguous(), args[1][:, :, good].contiguous()]
    want = fattn.qk_norm_rope_bwd(*keep, *keep, args[2], args[3], args[4],
                                  args[5][:, good].contiguous(), eps=EPS)
    for i in (2, 3):
        size = want[i].abs().max()
        assert float((out[i] - want[i]).abs().max()) <= 64 * U * float(size) * 9
    assert fattn.device_status() == 0


def test_far_rows_and_a_position_of_its_own_per_token():
    """Rows more than 2^32 elements from the base."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB")
    stride = (1 << 31) + 64 * 8
    big = torch.empty(3 * stride + 1024, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (1, 2, 4, 64), (8, 64, stride, 1))
    g = torch.Generator().manual_seed(4)
    vals = torch.randn(1, 2, 4, 64, generator=g).to(torch.bfloat16).cuda()
    x.copy_(vals)
    w = weights(64, torch.bfloat16, 5).cuda()
    rope = ref.rope_rows(16, 64).cuda()
    want = fattn.qk_norm_rope(vals, None, w, None, rope)[0]
    got = fattn.qk_norm_rope(x, None, w, None, rope, q_out=x)[0]
    assert torch.equal(got, want)


def test_other_streams_and_a_replayed_graph():
    q, k, wq, wk, rope, pos = cuda(*setup(2, 4, 2, 60, 128, torch.bfloat16, 128, True, seed=20))
    want = fattn.qk_norm_rope(q, k, wq, wk, rope, pos)
    grads = fattn.qk_norm_rope_bwd(q, k, q, k, wq, wk, rope, pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = fattn.qk_norm_rope(q, k, wq, wk, rope, pos, stream=s)
    got_g = fattn.qk_norm_rope_bwd(q, k, q, k, wq, wk, rope, pos, stream=s)
    raw = fattn.qk_norm_rope(q, k, wq, wk, rope, pos, stream=s.cuda_stream)
    s.synchronize()
    for a, b in itertools.chain(zip(got, want), zip(got_g, grads), zip(raw, want)):
        assert torch.equal(a, b)
    outs = [torch.empty_like(t) for t in (q, k)]
    ws = torch.empty(fattn.qk_norm_rope_bwd_workspace_size(128), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fattn.qk_norm_rope(q, k, wq, wk, rope, pos, q_out=outs[0], k_out=outs[1])
        dg = fattn.qk_norm_rope_bwd(q, k, q, k, wq, wk, rope, pos, workspace=ws)
    q2 = torch.randn_like(q)
    pos2 = torch.randint(0, 4096, pos.shape, dtype=torch.int32, device="cuda")
    q.copy_(q2)
    pos.copy_(pos2)
    graph.replay()
    want = fattn.qk_norm_rope(q, k, wq, wk, rope, pos)
    grads = fattn.qk_norm_rope_bwd(q, k, q, k, wq, wk, rope, pos)
    torch.cuda.synchronize()
    for a, b in itertools.chain(zip(outs, want), zip(dg, grads)):
        assert torch.equal(a, b)


def test_next_to_the_attention_of_a_training_step():
    """norm and rotation -> attn_fwd -> attn_bwd -> their gradients, against
    autograd of the whole in fp64 on the same inputs.  The 16-bit
    intermediates (q, k, o, dq, dk each rounded once, p and ds inside the
    backward) are independent roundings of 2^-9 relative rms each: about ten
    of them give 2^-9 sqrt(10) ~ 0.6 %; held to 2 % in the 2-norm."""
    B, H, N, d = 1, 2, 256, 64
    q, k, wq, wk, rope, _ = setup(B, H, H, N, d, torch.bfloat16, 64, seed=40)
    v, do = make(B, H, N, d, torch.bfloat16, 41), make(B, H, N, d, torch.bfloat16, 42)
    cq, ck, cwq, cwk, crope, cv, cdo = cuda(q, k, wq, wk, rope, v, do)
    nq, nk = fattn.qk_norm_rope(cq, ck, cwq, cwk, crope, eps=EPS)
    o, lse = fattn.attn_fwd(nq, nk, cv, causal=True)
    dnq, dnk, dv = fattn.attn_bwd(nq, nk, cv, o, lse, cdo, causal=True)
    got = fattn.qk_norm_rope_bwd(dnq, dnk, cq, ck, cwq, cwk, crope, eps=EPS)
    leaves = [t.double().requires_grad_() for t in (q, k, wq, wk, v)]
    ang = angles_of(rope, None, B, N)

    def norm(x, w):
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        c, s = ang[..., :32].double(), ang[..., 32:].double()
        return torch.cat([y[..., :32] * c - y[..., 32:] * s, y[..., 32:] * c + y[..., :32] * s], -1)

    x = norm(leaves[0], leaves[2]) @ norm(leaves[1], leaves[3]).transpose(2, 3) * d ** -0.5
    x = x.masked_fill(torch.ones(N, N).triu(1).bool(), float("-inf"))
    (torch.softmax(x, -1) @ leaves[4] * do.double()).sum().backward()
    for a, leaf in zip((got[0], got[1], got[2], got[3], dv), leaves):
        a, b = a.double().cpu(), leaf.grad
        assert float((a - b).norm() / b.norm()) < 0.02
    assert fattn.device_status() == 0
