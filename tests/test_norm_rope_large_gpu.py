"""GPU tests of the loops that training and prompt sizes take: warps of the
backward pass with many rows (the ring of copies wraps, blocks are dealt to q
and k by their rows), items of more heads than a warp holds at a time in the
forward pass.  Against the fp64 formulas, on the GPU."""
import pytest
import torch

from tests import serving_ref as ref
from tests.test_norm_rope_gpu import EPS, U, angles_of, cuda, floor_of, half, setup
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def tokens_a_warp(d):
    return 32 // (d // 16)


def heads_a_item(tokens, heads, d):
    """As the launch chooses them: 4, doubled while the items would still give
    every SM 64 warps."""
    blocks, n = -(-tokens // tokens_a_warp(d)), 4
    while n < heads and blocks * -(-heads // (2 * n)) >= 64 * sms():
        n *= 2
    return n


def rows_a_warp(tokens, Hq, Hk, d):
    """(q, k): the rows of a lane group, at most, with blocks of 4 warps, 4 an
    SM, dealt by the tensors' rows."""
    blocks, total = -(-tokens // tokens_a_warp(d)), 4 * sms()
    q = (total * Hq + (Hq + Hk) // 2) // (Hq + Hk)
    q = min(max(q, 1), total - 1)
    return -(-blocks * Hq // (4 * q)), -(-blocks * Hk // (4 * (total - q)))


def check(got, want, size, d, dtype, what):
    """The bound of the small cases (a row's arithmetic does not depend on how
    many there are)."""
    rel = (d / 2 + 14) * U
    tol = half(dtype) * want.abs() + (1 + half(dtype)) * rel * size + floor_of(dtype)
    err = (got.double() - want).abs()
    bad = ~(err <= tol * (1 + 1e-9))
    assert not bool(bad.any()), "%s: %d of %d beyond the bound, worst ratio %.3g" % (
        what, int(bad.sum()), bad.numel(), float((err / tol).nan_to_num(9e9).max()))


FORWARD = [
    # B, Hq, Hk, N, d, rot, interleaved, positions, dtype
    (2, 11, 2, 20011, 64, 64, False, False, torch.bfloat16),
    (1, 9, 5, 25603, 96, 48, True, True, torch.float16),
    (3, 13, 6, 7001, 128, 128, False, False, torch.float16),
    (1, 7, 6, 10007, 256, 256, False, True, torch.bfloat16),
]


@pytest.mark.parametrize("B,Hq,Hk,N,d,rot,inter,positions,dtype", FORWARD)
def test_forward(B, Hq, Hk, N, d, rot, inter, positions, dtype):
    heads = heads_a_item(B * N, Hq + Hk, d)
    assert heads > 4 and Hq % heads, "more than a warp holds, and a last item of fewer heads"
    q, k, wq, wk, rope, pos = cuda(*setup(B, Hq, Hk, N, d, dtype, 0, positions, seed=d))
    rope = ref.rope_rows(max(N, 4096), rot).cuda()
    out = fattn.qk_norm_rope(q, k, wq, wk, rope, pos, eps=EPS, interleaved=inter)
    ang = angles_of(rope, pos if pos is not None else torch.arange(N, device="cuda").expand(B, N), B, N)
    for got, x, w, what in zip(out, (q, k), (wq, wk), "qk"):
        want = ref.norm_rope(x, w, ang, EPS, inter)
        check(got, want, ref.g_terms(ref.norm_rope(x, w, None, EPS, inter), ang, inter), d, dtype, what)
    assert fattn.device_status() == 0


BACKWARD = [
    # B, Hq, Hk, N, d, rot, interleaved, positions, dtype, in place
    (2, 8, 1, 16000, 64, 64, False, False, torch.bfloat16, False),
    (2, 6, 2, 7001, 96, 96, True, False, torch.float16, True),
    (1, 8, 3, 9001, 128, 128, False, True, torch.float16, False),
    (3, 2, 7, 4001, 128, 32, True, False, torch.bfloat16, False),
    (1, 5, 3, 5003, 256, 256, False, True, torch.bfloat16, True),
]


@pytest.mark.parametrize("B,Hq,Hk,N,d,rot,inter,positions,dtype,in_place", BACKWARD)
def test_backward(B, Hq, Hk, N, d, rot, inter, positions, dtype, in_place):
    rows = rows_a_warp(B * N, Hq, Hk, d)
    assert min(rows) > 3, "the ring of three rows wraps in both tensors' warps"
    q, k, wq, wk, rope, pos = cuda(*setup(B, Hq, Hk, N, d, dtype, 0, positions, seed=d + 1))
    rope = ref.rope_rows(max(N, 4096), rot).cuda()
    g = torch.Generator("cuda").manual_seed(d)
    gq, gk = [torch.randn(x.shape, generator=g, device="cuda").to(dtype) for x in (q, k)]
    keep = gq.clone(), gk.clone()
    extra = dict(dq=gq, dk=gk) if in_place else {}
    out = fattn.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, rope, pos, eps=EPS, interleaved=inter, **extra)
    again = fattn.qk_norm_rope_bwd(*[t.clone() for t in keep], q, k, wq, wk, rope, pos, eps=EPS,
                                   interleaved=inter)
    ang = angles_of(rope, pos if pos is not None else torch.arange(N, device="cuda").expand(B, N), B, N)
    for i, (gr, x, w) in enumerate(((keep[0], q, wq), (keep[1], k, wk))):
        dx, dw, size, dw_size = ref.norm_rope_bwd(gr, x, w, ang, EPS, inter)
        check(out[i], dx, 4 * size, d, dtype, "d" + "qk"[i])
        # Each term carries r's error and the turn's, (d/2 + 16) U; a lane adds
        # its rows, then the rows of a warp's groups are added, four warps, and
        # the blocks with their rounding errors carried along.
        rel = (d / 2 + 16 + rows[i] + tokens_a_warp(d) + 4 + 4) * U
        err = (out[2 + i].double() - dw).abs()
        assert bool((err <= rel * dw_size).all()), float((err / dw_size).max() / U)
        assert torch.equal(out[i], again[i]) and torch.equal(out[2 + i], again[2 + i])
    assert fattn.device_status() == 0


@pytest.mark.parametrize("B,Hq,Hk,N,d", [(2, 8, 1, 11003, 64), (1, 6, 2, 7001, 96), (1, 3, 8, 9001, 128),
                                         (1, 5, 3, 5003, 256), (1, 1, 1, 1, 64), (1, 2, 1, 100, 128)])
def test_weight_gradients_count_every_row(B, Hq, Hk, N, d):
    """x and dy of +-1, eps = 3: r = 1 / sqrt(1 + 3), so dw is half the sum of
    the rows' signs in each column.  r is off by 4 U (rsqrtf: 2 steps) and 3 U
    (the mean); the sums of a lane and on add (rows + groups + 8) U of half the
    number of rows.  A row left out or added twice is half a unit, at least
    twice the bound."""
    g = torch.Generator("cuda").manual_seed(N)

    def signs(H):
        return (torch.randint(0, 2, (B, H, N, d), generator=g, device="cuda") * 2 - 1).bfloat16()

    q, k, gq, gk = signs(Hq), signs(Hk), signs(Hq), signs(Hk)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    out = fattn.qk_norm_rope_bwd(gq, gk, q, k, w, w, eps=3.0)
    rows = rows_a_warp(B * N, Hq, Hk, d)
    for i, (x, gr, H) in enumerate(((q, gq, Hq), (k, gk, Hk))):
        want = (x.float() * gr.float()).sum((0, 1, 2), dtype=torch.float64) / 2
        tol = (max(rows[i], 3) + tokens_a_warp(d) + 8 + 7) * U * B * H * N / 2
        assert tol <= 0.25
        err = (out[2 + i].double() - want).abs()
        assert bool((err <= tol).all()), (float(err.max()), tol)
