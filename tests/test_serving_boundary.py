"""CPU tests of the argument checks of the norm, rotation and cache calls: they
come before any device call, so fake addresses are never dereferenced."""
import ctypes
import os

import pytest
import torch

from tests import serving_ref as ref
from tiled_online_softmax_fwd_gb300 import build as fbuild
from tiled_online_softmax_fwd_gb300 import fattn

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 1 << 20
MB = 1 << 24


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fattn.library_path()):
        fbuild.build()
    return fattn.load()


def arr(*x):
    return (ctypes.c_longlong * len(x))(*x)


def i64(t):
    return None if t is None else arr(*t)


# ------------------------------------------------------------------ norm, rotation
def norm(lib, **kw):
    a = dict(q=A, k=A + MB, q_out=A + 2 * MB, k_out=A + 3 * MB, wq=A + 4 * MB, wk=A + 5 * MB,
             rope=A + 6 * MB, positions=A + 8 * MB, B=1, Hq=4, Hk=2, N=8, d=64, rot=64, max_pos=128,
             qs=(2048, 512, 64), ks=(1024, 512, 64), qos=(2048, 512, 64), kos=(1024, 512, 64),
             eps=1e-6, inter=0, dtype=0)
    a.update(kw)
    return lib.fattn_qk_norm_rope(a["q"], a["k"], a["q_out"], a["k_out"], a["wq"], a["wk"], a["rope"],
                                  a["positions"], a["B"], a["Hq"], a["Hk"], a["N"], a["d"], a["rot"],
                                  a["max_pos"], i64(a["qs"]), i64(a["ks"]), i64(a["qos"]),
                                  i64(a["kos"]), a["eps"], a["inter"], a["dtype"], None)


def test_norm_without_rows_is_a_noop(lib):
    assert norm(lib, N=0, q=0, k=0, q_out=0, k_out=0) == OK
    assert norm(lib, B=0) == OK
    assert norm(lib, Hq=0, Hk=0) == OK


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hk=-2), INVALID), (dict(N=-1), INVALID),
    (dict(d=80), UNSUPPORTED), (dict(d=512), UNSUPPORTED), (dict(dtype=2), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(inter=2), INVALID), (dict(rot=24), INVALID), (dict(rot=80), INVALID),
    (dict(rot=-16), INVALID), (dict(rope=0), INVALID), (dict(max_pos=0), INVALID),
    (dict(rope=A + 6 * MB + 4), INVALID), (dict(positions=A + 8 * MB + 2), INVALID),
    (dict(q=0), INVALID), (dict(q_out=0), INVALID), (dict(k=0), INVALID), (dict(q=A + 8), INVALID),
    (dict(wq=A + 4 * MB + 2), INVALID), (dict(qs=None), INVALID), (dict(kos=None), INVALID),
    (dict(qs=(2048, 508, 64)), INVALID), (dict(qs=(2048, 512, 0)), INVALID),
    (dict(qs=(2048, 512, -64)), INVALID),
    (dict(qos=(2048, 512, 32)), INVALID),          # rows of q_out overlap
    (dict(q_out=A + 64), INVALID),                 # shifted over its input
    (dict(q_out=A, qos=(4096, 1024, 64)), INVALID),  # in place with other strides
    (dict(q_out=A + MB), INVALID),                 # over k
    (dict(k_out=A + 2 * MB), INVALID),             # over q_out
    (dict(q_out=A + 6 * MB), INVALID),             # over the table
    (dict(k_out=A + 8 * MB), INVALID),             # over the positions
    (dict(k_out=A + 4 * MB), INVALID),             # over the weights
    (dict(qs=(2048, 1 << 39, 64)), INVALID),
    (dict(qs=(2048, 1 << 37, 64)), UNSUPPORTED),   # beyond 2^39 bytes
])
def test_norm_refusals(lib, kw, expect):
    assert norm(lib, **kw) == expect


def norm_bwd(lib, **kw):
    a = dict(gq=A + 9 * MB, gk=A + 10 * MB, q=A, k=A + MB, wq=A + 4 * MB, wk=A + 5 * MB,
             rope=A + 6 * MB, positions=0, dq=A + 2 * MB, dk=A + 3 * MB, dwq=A + 11 * MB,
             dwk=A + 12 * MB, B=1, Hq=4, Hk=2, N=8, d=64, rot=64, max_pos=128, s4=(2048, 512, 64),
             s2=(1024, 512, 64), dqs=(2048, 512, 64), eps=1e-6, ws=A + 13 * MB, bytes=MB)
    a.update(kw)
    return lib.fattn_qk_norm_rope_bwd(a["gq"], a["gk"], a["q"], a["k"], a["wq"], a["wk"], a["rope"],
                                      a["positions"], a["dq"], a["dk"], a["dwq"], a["dwk"], a["B"],
                                      a["Hq"], a["Hk"], a["N"], a["d"], a["rot"], a["max_pos"],
                                      i64(a["s4"]), i64(a["s2"]), i64(a["s4"]), i64(a["s2"]),
                                      i64(a["dqs"]), i64(a["s2"]), a["eps"], 0, 0, a["ws"],
                                      a["bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dwq=0), INVALID), (dict(wk=0), INVALID), (dict(d=48), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(gq=0), INVALID), (dict(dk=0), INVALID), (dict(dqs=None), INVALID),
    (dict(dqs=(2048, 512, 56)), INVALID), (dict(dwq=A + 11 * MB + 2), INVALID),
])
def test_norm_backward_refusals(lib, kw, expect):
    assert norm_bwd(lib, **kw) == expect


# ------------------------------------------------------------------ append
def append(lib, **kw):
    a = dict(k=A, v=A + MB, kc=A + 2 * MB, vc=A + 4 * MB, table=A + 6 * MB, cu=A + 7 * MB,
             kv_len=A + 8 * MB, rope=A + 9 * MB, T=5, B=2, Hk=2, d=64, pages=8, page=16, max_pages=4,
             row=4, rot=64, max_pos=64, ks=(128, 64), vs=(128, 64), kcs=(2048, 1024, 64),
             vcs=(2048, 1024, 64), inter=0, dtype=0)
    a.update(kw)
    return lib.fattn_kv_append(a["k"], a["v"], a["kc"], a["vc"], a["table"], a["cu"], a["kv_len"],
                               a["rope"], a["T"], a["B"], a["Hk"], a["d"], a["pages"], a["page"],
                               a["max_pages"], a["row"], a["rot"], a["max_pos"], i64(a["ks"]),
                               i64(a["vs"]), i64(a["kcs"]), i64(a["vcs"]), a["inter"], a["dtype"],
                               None)


def test_append_of_nothing_is_a_noop(lib):
    for kw in (dict(T=0), dict(B=0), dict(Hk=0)):
        assert append(lib, k=0, v=0, kc=0, vc=0, table=0, cu=0, kv_len=0, **kw) == OK


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(Hk=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(d=72), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(page=0), UNSUPPORTED), (dict(pages=-1), INVALID), (dict(pages=0), INVALID),
    (dict(max_pages=-1), INVALID), (dict(page=1 << 20, max_pages=1 << 12), UNSUPPORTED),
    (dict(rot=40), INVALID), (dict(rope=0), INVALID), (dict(inter=-1), INVALID),
    (dict(table=0), INVALID), (dict(cu=0), INVALID), (dict(kv_len=0), INVALID),
    (dict(table=A + 6 * MB + 2), INVALID), (dict(row=3), INVALID), (dict(ks=None), INVALID),
    (dict(vcs=None), INVALID), (dict(k=0), INVALID), (dict(vc=0), INVALID), (dict(kc=A + 2 * MB + 8), INVALID),
    (dict(kcs=(2048, 1024, 32)), INVALID),   # slots overlap
    (dict(kcs=(1024, 1024, 64)), INVALID),   # pages overlap
    (dict(vc=A + 2 * MB), INVALID),          # one pool for both
    (dict(kc=A), INVALID),                   # over the new keys
    (dict(vc=A + 6 * MB), INVALID),          # over the page table
    (dict(kc=A + 9 * MB), INVALID),          # over the rotation table
])
def test_append_refusals(lib, kw, expect):
    assert append(lib, **kw) == expect


# ------------------------------------------------------------------ binding
def test_python_checks_need_no_device():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fattn.qk_norm_rope(x, x)  # CPU tensors
    with pytest.raises(ValueError):
        fattn.qk_norm_rope(None, None)
    with pytest.raises(TypeError):
        fattn.kv_append(None, x, x, x, x, x, x)
    with pytest.raises(ValueError):
        fattn.rope_table(8, 24)


def test_rope_table_is_the_formula():
    got = fattn.rope_table(1 << 12, 32, theta=500000.0, device="cpu")
    assert got.dtype == torch.float32
    want = ref.rope_rows(1 << 12, 32, 500000.0)
    # both round an fp64 cosine once; fp64 powers may differ by an ulp
    assert float((got - want).abs().max()) <= 2.0 ** -24


# ------------------------------------------------------------------ reference
def test_reference_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(2, 3, 5, 64, generator=g, dtype=torch.float64).requires_grad_()
    w = (1 + 0.2 * torch.randn(64, generator=g, dtype=torch.float64)).requires_grad_()
    dy = torch.randn(2, 3, 5, 64, generator=g, dtype=torch.float64)
    ang = ref.rope_rows(16, 32)[torch.randint(0, 16, (2, 5), generator=g)][:, None]
    for inter in (False, True):
        h = 1e-5
        dx, dw, _, _ = ref.norm_rope_bwd(dy, x.detach(), w.detach(), ang, 1e-6, inter)
        u = torch.randn(x.shape, generator=g, dtype=torch.float64)
        f = [float((dy * ref.norm_rope(x.detach() + s * h * u, w.detach(), ang, 1e-6, inter)).sum())
             for s in (1, -1)]
        assert abs((f[0] - f[1]) / (2 * h) - float((dx * u).sum())) < 1e-6
        t = torch.randn(64, generator=g, dtype=torch.float64)
        f = [float((dy * ref.norm_rope(x.detach(), w.detach() + s * h * t, ang, 1e-6, inter)).sum())
             for s in (1, -1)]
        assert abs((f[0] - f[1]) / (2 * h) - float((dw * t).sum())) < 1e-6


# ------------------------------------------------------------------ paged attention
def paged(lib, **kw):
    a = dict(q=A, kc=A + 2 * MB, vc=A + 4 * MB, table=A + 6 * MB, cu=A + 7 * MB, kv_len=A + 8 * MB,
             o=A + 9 * MB, lse=A + 10 * MB, T=5, B=2, Hq=4, Hk=2, d=64, pages=8, page=16, max_pages=4,
             row=4, max_q=3, qs=(256, 64), kcs=(2048, 1024, 64), vcs=(2048, 1024, 64), os=(256, 64),
             scale=0.125, causal=1, dtype=0, ws=A + 64 * MB, bytes=1 << 30)
    a.update(kw)
    return lib.attn_fwd_paged(a["q"], a["kc"], a["vc"], a["table"], a["cu"], a["kv_len"], a["o"],
                              a["lse"], a["T"], a["B"], a["Hq"], a["Hk"], a["d"], a["pages"],
                              a["page"], a["max_pages"], a["row"], a["max_q"], i64(a["qs"]),
                              i64(a["kcs"]), i64(a["vcs"]), i64(a["os"]), a["scale"], a["causal"],
                              a["dtype"], a["ws"], a["bytes"], None)


def test_paged_attention_of_nothing_is_a_noop(lib):
    for kw in (dict(T=0), dict(B=0), dict(Hq=0)):
        assert paged(lib, q=0, kc=0, vc=0, table=0, cu=0, kv_len=0, o=0, lse=0, ws=0, **kw) == OK


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(Hq=-4), INVALID), (dict(Hk=0), INVALID),
    (dict(Hq=5), INVALID), (dict(Hq=258, Hk=2), UNSUPPORTED), (dict(max_q=0), INVALID),
    (dict(d=256), UNSUPPORTED), (dict(d=80), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
    (dict(page=48), UNSUPPORTED), (dict(pages=0), INVALID), (dict(page=1 << 20, max_pages=1 << 12), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(causal=2), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(table=0), INVALID), (dict(cu=0), INVALID),
    (dict(kv_len=A + 8 * MB + 1), INVALID), (dict(row=3), INVALID), (dict(q=0), INVALID),
    (dict(kc=0), INVALID), (dict(vc=A + 4 * MB + 4), INVALID), (dict(o=0), INVALID),
    (dict(lse=0), INVALID), (dict(lse=A + 10 * MB + 2), INVALID), (dict(qs=None), INVALID),
    (dict(os=None), INVALID), (dict(kcs=None), INVALID), (dict(qs=(256, 60)), INVALID),
    (dict(os=(256, 32)), INVALID), (dict(os=(128, 64)), INVALID),  # rows of o overlap
    (dict(o=A), INVALID), (dict(o=A + 64), INVALID),               # over q
    (dict(o=A + 2 * MB), INVALID), (dict(o=A + 4 * MB), INVALID),  # over the caches
    (dict(o=A + 6 * MB), INVALID), (dict(lse=A + 9 * MB), INVALID), (dict(lse=A + 2 * MB), INVALID),
    (dict(lse=A + 7 * MB), INVALID), (dict(kcs=(1 << 39, 1024, 64)), INVALID),
])
def test_paged_attention_refusals(lib, kw, expect):
    assert paged(lib, **kw) == expect


def test_paged_attention_token_indexes_stay_in_32_bits(lib):
    assert paged(lib, T=(1 << 31) - 1) == UNSUPPORTED
    assert paged(lib, T=(1 << 31) - 256) == UNSUPPORTED


def test_workspace_sizes_of_bad_arguments_are_zero(lib):
    for args in ((0, 1, 64, 1), (4, 3, 64, 1), (4, 2, 80, 1), (4, 2, 64, 0), (-1, 1, 64, 1)):
        assert lib.attn_fwd_paged_workspace_size(*args) == 0
    assert lib.fattn_qk_norm_rope_bwd_workspace_size(80) == 0
