"""CPU tests of the argument checks of the tree, page and cross attention calls
(they come before any device call, so fake addresses are never dereferenced),
and of the references that their GPU tests compare with."""
import ctypes
import os

import pytest
import torch

from tests import search_ref as ref
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


def i64(t):
    return None if t is None else (ctypes.c_longlong * len(t))(*t)


# ------------------------------------------------------------------ trees
def tree(lib, **kw):
    a = dict(q=A, kc=A + 2 * MB, vc=A + 4 * MB, table=A + 6 * MB, cu=A + 7 * MB, kv_len=A + 8 * MB,
             mask=A + 11 * MB, o=A + 9 * MB, lse=A + 10 * MB, T=5, B=2, Hq=4, Hk=2, d=64, pages=8, page=16,
             max_pages=4, row=4, max_q=3, words=1, mrow=1, qs=(256, 64), kcs=(2048, 1024, 64),
             vcs=(2048, 1024, 64), os=(256, 64), scale=0.125, dtype=0, ws=A + 64 * MB, bytes=1 << 30)
    a.update(kw)
    return lib.attn_fwd_tree(a["q"], a["kc"], a["vc"], a["table"], a["cu"], a["kv_len"], a["mask"], a["o"],
                             a["lse"], a["T"], a["B"], a["Hq"], a["Hk"], a["d"], a["pages"], a["page"],
                             a["max_pages"], a["row"], a["max_q"], a["words"], a["mrow"], i64(a["qs"]),
                             i64(a["kcs"]), i64(a["vcs"]), i64(a["os"]), a["scale"], a["dtype"], a["ws"],
                             a["bytes"], None)


def test_tree_attention_of_nothing_is_a_noop(lib):
    for kw in (dict(T=0), dict(B=0), dict(Hq=0)):
        assert tree(lib, q=0, kc=0, vc=0, table=0, cu=0, kv_len=0, mask=0, o=0, lse=0, ws=0, **kw) == OK


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(Hk=0), INVALID), (dict(Hq=5), INVALID),
    (dict(Hq=258, Hk=2), UNSUPPORTED), (dict(max_q=0), INVALID), (dict(d=256), UNSUPPORTED),
    (dict(page=24), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(scale=-1.0), INVALID),
    (dict(words=0), INVALID), (dict(words=1, max_q=33), INVALID), (dict(words=-1), INVALID),
    (dict(words=2, mrow=1), INVALID), (dict(mrow=1 << 39), INVALID), (dict(mask=0), INVALID),
    (dict(mask=A + 11 * MB + 2), INVALID), (dict(o=A + 11 * MB), INVALID), (dict(lse=A + 11 * MB), INVALID),
    (dict(q=0), INVALID), (dict(kc=0), INVALID), (dict(o=A), INVALID), (dict(lse=0), INVALID),
    (dict(kv_len=A + 8 * MB + 1), INVALID), (dict(os=(128, 64)), INVALID), (dict(qs=None), INVALID)])
def test_tree_attention_refusals(lib, kw, expect):
    assert tree(lib, **kw) == expect


def tree_mask(lib, **kw):
    a = dict(parents=A, cu=A + MB, kv_len=A + 2 * MB, mask=A + 3 * MB, pos=A + 4 * MB, T=9, B=2, words=1)
    a.update(kw)
    return lib.fattn_tree_mask(*(a[x] for x in ("parents", "cu", "kv_len", "mask", "pos", "T", "B", "words")),
                               None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=0, parents=0, mask=0), OK), (dict(B=0), OK), (dict(T=-1), INVALID), (dict(B=-1), INVALID),
    (dict(words=0), INVALID), (dict(words=(1 << 24) + 1), UNSUPPORTED), (dict(T=2 ** 31 - 1), UNSUPPORTED),
    (dict(parents=0), INVALID), (dict(cu=0), INVALID), (dict(kv_len=0), INVALID), (dict(mask=0), INVALID),
    (dict(pos=0), INVALID), (dict(pos=A + 4 * MB + 2), INVALID), (dict(mask=A + 32), INVALID),
    (dict(pos=A), INVALID), (dict(pos=A + 3 * MB + 32), INVALID), (dict(mask=A + MB), INVALID)])
def test_tree_mask_refusals(lib, kw, expect):
    assert tree_mask(lib, **kw) == expect


# ------------------------------------------------------------------ pages
def keep(lib, **kw):
    a = dict(kc=A + 2 * MB, vc=A + 4 * MB, table=A + 6 * MB, cu=A + 7 * MB, kv_len=A + 8 * MB,
             kept=A + 9 * MB, count=A + 10 * MB, out=A + 11 * MB, B=2, Hk=2, d=64, pages=8, page=16,
             max_pages=4, row=4, m=3, krow=3, kcs=(2048, 1024, 64), vcs=(2048, 1024, 64))
    a.update(kw)
    return lib.fattn_kv_keep(a["kc"], a["vc"], a["table"], a["cu"], a["kv_len"], a["kept"], a["count"],
                             a["out"], a["B"], a["Hk"], a["d"], a["pages"], a["page"], a["max_pages"],
                             a["row"], a["m"], a["krow"], i64(a["kcs"]), i64(a["vcs"]), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=0, kc=0, vc=0, table=0, cu=0, kv_len=0, kept=0, count=0, out=0), OK), (dict(B=-1), INVALID),
    (dict(Hk=-1), INVALID), (dict(m=-1), INVALID), (dict(d=80), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
    (dict(B=2 ** 30), UNSUPPORTED), (dict(table=0), INVALID), (dict(cu=0), INVALID), (dict(kv_len=0), INVALID),
    (dict(kept=0), INVALID), (dict(count=0), INVALID), (dict(out=0), INVALID), (dict(krow=2), INVALID),
    (dict(out=A + 11 * MB + 1), INVALID), (dict(kept=A + 9 * MB + 2), INVALID), (dict(out=A + 9 * MB), INVALID),
    (dict(out=A + 10 * MB), INVALID), (dict(out=A + 7 * MB), INVALID), (dict(out=A + 8 * MB + 4), INVALID),
    (dict(kc=0), INVALID), (dict(vc=A + 4 * MB + 8), INVALID), (dict(kcs=None), INVALID),
    (dict(kcs=(2048, 1024, 32)), INVALID), (dict(vc=A + 2 * MB), INVALID), (dict(kc=A + 9 * MB), INVALID),
    (dict(vc=A + 11 * MB), INVALID), (dict(row=3), INVALID)])
def test_keep_refusals(lib, kw, expect):
    assert keep(lib, **kw) == expect


def fork(lib, **kw):
    a = dict(kc=A + 2 * MB, vc=A + 4 * MB, table=A + 6 * MB, kv_len=A + 7 * MB, refs=A + 8 * MB,
             parents=A + 9 * MB, cu=A + 10 * MB, tout=A + 11 * MB, lout=A + 12 * MB, rout=A + 13 * MB, B=2,
             Hk=2, d=64, pages=8, page=16, max_pages=4, row=4, orow=4, kcs=(2048, 1024, 64),
             vcs=(2048, 1024, 64), ws=A + 64 * MB, bytes=1 << 20)
    a.update(kw)
    return lib.fattn_kv_fork(a["kc"], a["vc"], a["table"], a["kv_len"], a["refs"], a["parents"], a["cu"],
                             a["tout"], a["lout"], a["rout"], a["B"], a["Hk"], a["d"], a["pages"], a["page"],
                             a["max_pages"], a["row"], a["orow"], i64(a["kcs"]), i64(a["vcs"]), a["ws"],
                             a["bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=0, kc=0, table=0, kv_len=0, refs=0, tout=0, lout=0, rout=0, ws=0), OK), (dict(B=-1), INVALID),
    (dict(Hk=-1), INVALID), (dict(d=80), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(B=2 ** 28), UNSUPPORTED), (dict(table=0), INVALID), (dict(kv_len=0), INVALID),
    (dict(refs=0), INVALID), (dict(tout=0), INVALID), (dict(lout=0), INVALID), (dict(rout=0), INVALID),
    (dict(row=3), INVALID), (dict(orow=3), INVALID), (dict(tout=A + 6 * MB, orow=5), INVALID),
    (dict(tout=A + 6 * MB + 16), INVALID), (dict(lout=A + 8 * MB), INVALID), (dict(rout=A + 7 * MB), INVALID),
    (dict(lout=A + 12 * MB + 2), INVALID), (dict(parents=A + 9 * MB + 2), INVALID),
    (dict(cu=A + 10 * MB + 3), INVALID), (dict(lout=A + 9 * MB), INVALID), (dict(tout=A + 10 * MB), INVALID),
    (dict(rout=A + 12 * MB), INVALID), (dict(ws=0), INVALID), (dict(ws=A + 64 * MB + 8), INVALID),
    (dict(bytes=16), INVALID), (dict(ws=A + 6 * MB), INVALID), (dict(ws=A + 13 * MB), INVALID),
    (dict(kc=0), INVALID), (dict(kcs=None), INVALID), (dict(vc=A + 2 * MB), INVALID),
    (dict(kcs=(1024, 1024, 64)), INVALID), (dict(kc=A + 8 * MB), INVALID), (dict(vc=A + 11 * MB), INVALID)])
def test_fork_refusals(lib, kw, expect):
    assert fork(lib, **kw) == expect


# ------------------------------------------------------------------ cross attention
def cross(lib, **kw):
    a = dict(q=A, k=A + 2 * MB, v=A + 4 * MB, kv_len=A + 6 * MB, o=A + 8 * MB, lse=A + 10 * MB, B=2, Hq=4,
             Hk=2, Nq=3, Nk=7, d=64, qs=(768, 192, 64), ks=(896, 448, 64), vs=(896, 448, 64),
             os=(768, 192, 64), scale=0.125, dtype=0, ws=A + 64 * MB, bytes=1 << 30)
    a.update(kw)
    return lib.attn_fwd_cross(a["q"], a["k"], a["v"], a["kv_len"], a["o"], a["lse"], a["B"], a["Hq"], a["Hk"],
                              a["Nq"], a["Nk"], a["d"], i64(a["qs"]), i64(a["ks"]), i64(a["vs"]), i64(a["os"]),
                              a["scale"], a["dtype"], a["ws"], a["bytes"], None)


SHARED = [
    (dict(B=-1), INVALID), (dict(Nq=-1), INVALID), (dict(Nk=-1), INVALID), (dict(Hk=0), INVALID),
    (dict(Hq=5), INVALID), (dict(Hq=258), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(d=80), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(Nk=2 ** 31 - 1), UNSUPPORTED),
    (dict(B=4, Nq=1 << 29), UNSUPPORTED), (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID),
    (dict(o=0), INVALID), (dict(lse=0), INVALID), (dict(kv_len=A + 6 * MB + 2), INVALID),
    (dict(lse=A + 10 * MB + 1), INVALID), (dict(q=A + 8), INVALID), (dict(qs=None), INVALID),
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(os=None), INVALID),
    (dict(qs=(768, 190, 64)), INVALID), (dict(ks=(0, 448, 64)), INVALID), (dict(vs=(896, 448, -64)), INVALID),
]


@pytest.mark.parametrize("kw,expect", SHARED + [
    (dict(os=(768, 192, 32)), INVALID), (dict(o=A), INVALID), (dict(o=A + 64), INVALID),
    (dict(o=A + 2 * MB), INVALID), (dict(o=A + 4 * MB), INVALID), (dict(o=A + 6 * MB), INVALID),
    (dict(lse=A + 8 * MB), INVALID), (dict(lse=A), INVALID), (dict(lse=A + 6 * MB), INVALID),
    (dict(qs=(768, 1 << 38, 64)), UNSUPPORTED), (dict(B=0, q=0, o=0), OK), (dict(Nq=0, q=0, o=0, ws=0), OK)])
def test_cross_refusals(lib, kw, expect):
    assert cross(lib, **kw) == expect


def cross_bwd(lib, **kw):
    a = dict(q=A, k=A + 2 * MB, v=A + 4 * MB, o=A + 8 * MB, lse=A + 10 * MB, do=A + 12 * MB,
             kv_len=A + 6 * MB, dq=A + 14 * MB, dk=A + 16 * MB, dv=A + 18 * MB, B=2, Hq=4, Hk=2, Nq=3, Nk=7,
             d=64, qs=(768, 192, 64), ks=(896, 448, 64), vs=(896, 448, 64), os=(768, 192, 64),
             dos=(768, 192, 64), dqs=(768, 192, 64), dks=(896, 448, 64), dvs=(896, 448, 64), scale=0.125,
             dtype=0, ws=A + 64 * MB, bytes=1 << 30)
    a.update(kw)
    return lib.attn_bwd_cross(*(a[x] for x in ("q", "k", "v", "o", "lse", "do", "kv_len", "dq", "dk", "dv", "B",
                                               "Hq", "Hk", "Nq", "Nk", "d")),
                              *(i64(a[x]) for x in ("qs", "ks", "vs", "os", "dos", "dqs", "dks", "dvs")),
                              a["scale"], a["dtype"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,expect", SHARED + [
    (dict(do=0), INVALID), (dict(dq=0), INVALID), (dict(dk=0), INVALID), (dict(dv=0), INVALID),
    (dict(dos=None), INVALID), (dict(dqs=None), INVALID), (dict(dks=None), INVALID), (dict(dvs=None), INVALID),
    (dict(dqs=(768, 192, 32)), INVALID), (dict(dks=(448, 448, 64)), INVALID), (dict(dq=A), INVALID),
    (dict(dq=A + 12 * MB), INVALID), (dict(dk=A + 2 * MB), INVALID), (dict(dv=A + 4 * MB), INVALID),
    (dict(dk=A + 18 * MB), INVALID), (dict(dv=A + 14 * MB), INVALID), (dict(dq=A + 8 * MB), INVALID),
    (dict(dk=A + 10 * MB), INVALID), (dict(dv=A + 6 * MB), INVALID), (dict(B=0), OK),
    (dict(Nq=0, Nk=0, q=0, k=0, dq=0, dk=0), OK)])
def test_cross_backward_refusals(lib, kw, expect):
    assert cross_bwd(lib, **kw) == expect


def test_workspace_sizes_of_bad_arguments_are_zero(lib):
    assert lib.attn_fwd_cross_workspace_size(4, 3, 5, 64) == 0
    assert lib.attn_fwd_cross_workspace_size(4, 2, 0, 64) == 0
    assert lib.attn_bwd_cross_workspace_size(1, 4, 3, 5, 5, 64) == 0
    assert lib.attn_bwd_cross_workspace_size(1, 4, 2, 5, 5, 256) == 0
    assert lib.fattn_kv_fork_workspace_size(0, 4, 4) == 0
    assert lib.fattn_kv_fork_workspace_size(2, -1, 4) == 0


# ------------------------------------------------------------------ binding
def test_python_checks_need_no_device():
    x = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: fattn.attn_fwd_tree(x[0], x, x, i[None], i, i, i[None], 2),
                 lambda: fattn.tree_mask(i, i, i, 2), lambda: fattn.kv_keep(x, x, i[None], i, i, i[None], i),
                 lambda: fattn.kv_fork(x, x, i[None], i, i), lambda: fattn.attn_fwd_cross(x, x, x),
                 lambda: fattn.attn_bwd_cross(x, x, x, x, x, x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fattn.attn_fwd_tree(None, x, x, i[None], i, i, i[None], 2),
                 lambda: fattn.tree_mask(None, i, i, 2), lambda: fattn.attn_fwd_cross(None, x, x),
                 lambda: fattn.kv_fork(x, x, i[None], None, i)):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ references
def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(0)
    B, Hq, Hk, Nq, Nk, d, lens = 2, 4, 2, 5, 7, 64, [7, 3]
    q, do = (torch.randn(B, Hq, Nq, d, generator=g, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(B, Hk, Nk, d, generator=g, dtype=torch.float64) for _ in range(2))
    grads = ref.cross_bwd(q, k, v, do, lens, 0.2)
    step = 1e-5
    for at, grad in enumerate(grads):
        u = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        f = []
        for sign in (1, -1):
            t = [q, k, v]
            t[at] = t[at] + sign * step * u
            f.append(float((ref.cross(*t, lens, 0.2)[0] * do).sum()))
        assert abs((f[0] - f[1]) / (2 * step) - float((grad * u).sum())) < 1e-6
    assert bool((grads[1][1, :, 3:] == 0).all()) and bool((grads[2][1, :, 3:] == 0).all())


def test_reference_fork_is_a_list_of_tokens():
    """Forty steps of reordered, ended and restarted sequences: the cache holds
    each sequence's tokens, and the counts are those of the entries."""
    g = torch.Generator().manual_seed(1)
    B, page, cols, pages = 5, 16, 8, 60
    kc = torch.zeros(pages, 1, page, 1)
    table, lens, refs = [[-1] * cols for _ in range(B)], [0] * B, [0] * pages
    hist = [[] for _ in range(B)]
    for _ in range(40):
        parents = torch.randint(-1, B, (B,), generator=g).tolist()
        new = torch.randint(0, 4, (B,), generator=g).tolist()
        table, lens, refs, kc, _ = ref.fork(kc, kc.clone(), table, lens, refs, parents, new)
        hist = [list(hist[p]) if p >= 0 else [] for p in parents]
        for b in range(B):
            for _ in range(new[b]):
                x = float(torch.rand(1, generator=g))
                kc[table[b][len(hist[b]) // page], 0, len(hist[b]) % page] = x
                hist[b].append(x)
            assert lens[b] == len(hist[b])
        count = [0] * pages
        for row in table:
            for x in row:
                if x >= 0:
                    count[x] += 1
        assert refs == count
        for b in range(B):
            got = [float(kc[table[b][j // page], 0, j % page]) for j in range(lens[b])]
            assert got == [float(torch.tensor(x)) for x in hist[b]]
