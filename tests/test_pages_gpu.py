"""GPU tests of kv_keep and kv_fork against the plain references: moves inside
and across pages, batches of every size, lists that are wrong, in place and
apart, both pool layouts, pages that run out, graphs, and a whole search."""
import pytest
import torch

from tests import search_ref as ref
from tests.paged import make_paged
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu

KEEP, FORK = 6 | 10 << 8, 6 | 11 << 8


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def same(a, b):
    """Equal bits (the unused slots hold NaN)."""
    return torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16))


def padded(kept, width=None):
    width = max(map(len, kept)) if width is None else width
    return ints([k + [-7] * (width - len(k)) for k in kept]).reshape(len(kept), width)


def random_kept(q_lens, g, share):
    return [[t for t in range(n) if torch.rand(1, generator=g) < share] for n in q_lens]


# ------------------------------------------------------------------ keep
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_lens,kv_lens,Hk,d,page,share", [
    ([1], [1], 1, 64, 16, 1.0), ([1], [40], 2, 128, 16, 0.0), ([6], [6], 1, 96, 16, 0.5),
    ([26, 26, 1, 0], [150, 1100, 9, 5], 8, 128, 16, 0.2), ([40, 33, 64], [64, 640, 65], 2, 256, 16, 0.6),
    ([200, 129], [300, 1000], 3, 64, 128, 0.9), ([700], [2000], 5, 128, 64, 0.4),
    ([1 + i % 30 for i in range(300)], [40 + i for i in range(300)], 1, 64, 32, 0.3)])
def test_keep(q_lens, kv_lens, Hk, d, page, share, dtype):
    p = make_paged(q_lens, kv_lens, Hk, d, page, dtype, seed=sum(kv_lens), fill=float("nan"))
    kept = random_kept(q_lens, torch.Generator().manual_seed(1), share)
    want = ref.keep(p.k_cache, p.v_cache, p.table.tolist(), p.cu, p.kv_len, kept)
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    table, cu, kv_len = p.lists()
    out = fattn.kv_keep(kc, vc, table, cu, kv_len, padded(kept), ints(list(map(len, kept))))
    assert fattn.device_status() == 0
    assert same(kc, want[0]) and same(vc, want[1]) and out.tolist() == want[2]
    assert kv_len.tolist() == list(kv_lens)


def test_keep_in_place_and_in_other_layouts():
    """Lengths in place; caches [pages, slots, 2, heads, d]; a wide kept list
    with rows apart."""
    q_lens, kv_lens = [30, 11], [77, 300]
    p = make_paged(q_lens, kv_lens, 4, 64, 16, torch.bfloat16, seed=5)
    kept = [[0, 3, 9, 20, 29], [2]]
    both = torch.stack([p.k_cache, p.v_cache], 2).permute(0, 3, 2, 1, 4).contiguous().cuda()
    kc, vc = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    table, cu, kv_len = p.lists()
    wide = torch.full((2, 12), -1, dtype=torch.int32, device="cuda")
    wide[:, 4:9] = padded(kept)
    out = fattn.kv_keep(kc, vc, table, cu, kv_len, wide[:, 4:9], ints([5, 1]), kv_len_out=kv_len)
    want = ref.keep(p.k_cache, p.v_cache, p.table.tolist(), p.cu, p.kv_len, kept)
    assert fattn.device_status() == 0 and out is kv_len
    assert same(kc, want[0]) and same(vc, want[1]) and out.tolist() == want[2]


def test_keep_many_heads_in_place_of_lengths():
    """Eight blocks a sequence read the length that one of them overwrites."""
    B = 200
    q_lens, kv_lens = [24] * B, [30 + i % 9 for i in range(B)]
    p = make_paged(q_lens, kv_lens, 8, 128, 16, torch.bfloat16, seed=6)
    kept = random_kept(q_lens, torch.Generator().manual_seed(2), 0.7)
    want = ref.keep(p.k_cache, p.v_cache, p.table.tolist(), p.cu, p.kv_len, kept)
    for _ in range(3):
        kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
        table, cu, kv_len = p.lists()
        fattn.kv_keep(kc, vc, table, cu, kv_len, padded(kept, 24), ints(list(map(len, kept))),
                      kv_len_out=kv_len)
        assert same(kc, want[0]) and same(vc, want[1]) and kv_len.tolist() == want[2]
    assert fattn.device_status() == 0


@pytest.mark.parametrize("what,change", [
    ("order", dict(kept=[3, 2, 5])), ("twice", dict(kept=[1, 1, 4])), ("behind", dict(kept=[0, 2, 8])),
    ("negative", dict(kept=[-1, 2, 3])), ("more than new", dict(count=9)), ("count", dict(count=-1)),
    ("more than the list", dict(count=4)), ("too short", dict(kv_len=7)),
    ("beyond the table", dict(kv_len=49)), ("a page outside", dict(page=-1)),
    ("a page past the pool", dict(page=10 ** 6))])
def test_keep_leaves_a_sequence_with_wrong_lists(what, change):
    """Sequence 1 of three is wrong: it stays as it was, the others move."""
    q_lens, kv_lens = [5, 8, 6], [20, 40, 30]
    p = make_paged(q_lens, kv_lens, 2, 64, 16, torch.bfloat16, seed=7)
    kept = [[1, 4], [0, 2, 5], [3]]
    asked = [kept[0], change.get("kept", kept[1]), kept[2]]
    count = [2, change.get("count", 3), 1]
    lens = [20, change.get("kv_len", 40), 30]
    want = ref.keep(p.k_cache, p.v_cache, p.table.tolist(), p.cu, p.kv_len,
                    [kept[0], list(range(8)), kept[2]])
    if "page" in change:
        p.table[1, 2] = change["page"]  # of its new tokens
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    out = fattn.kv_keep(kc, vc, p.table.cuda(), ints(p.cu), ints(lens), padded(asked, 3), ints(count))
    assert fattn.device_status() & 0xffff == KEEP, what
    assert same(kc, want[0]) and same(vc, want[1])
    assert out.tolist() == [17, lens[1], 25]


# ------------------------------------------------------------------ fork
def state(lens, Hk, d, page, dtype=torch.bfloat16, seed=0, spare=8, shared=(), cols=None):
    """A cache of sequences; `shared`: pairs (a, b) where b's leading whole
    pages are a's."""
    p = make_paged([0] * len(lens), lens, Hk, d, page, dtype, seed=seed, spare=spare)
    cols = p.table.shape[1] + 3 if cols is None else cols
    table = [(r + [-1] * cols)[:cols] for r in p.table.tolist()]
    for a, b in shared:
        n = min(lens[a], lens[b]) // page
        table[b][:n] = table[a][:n]
    refs = [0] * p.k_cache.shape[0]
    for row in table:
        for x in row:
            if x >= 0:
                refs[x] += 1
    return p, table, refs


def run_fork(p, table, lens, refs, parents, new, place=False, **kw):
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    t, l, r = ints(table), ints(lens), ints(refs)
    cu = None if new is None else ints([sum(new[:i]) for i in range(len(new) + 1)])
    if place:
        kw.update(page_table_out=t, kv_len_out=l, page_refs_out=r)
    got = fattn.kv_fork(kc, vc, t, l, r, None if parents is None else ints(parents), cu, **kw)
    return (*got, kc, vc), (t, l, r)


def check_fork(p, table, lens, refs, parents, new, **kw):
    want = ref.fork(p.k_cache, p.v_cache, table, lens, refs,
                    list(range(len(lens))) if parents is None else parents,
                    [0] * len(lens) if new is None else new)
    for place in (False, True):
        got, given = run_fork(p, table, lens, refs, parents, new, place, **kw)
        assert fattn.device_status() == 0
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2]
        assert same(got[3], want[3]) and same(got[4], want[4])
        if not place:
            assert given[0].tolist() == table and given[1].tolist() == lens and given[2].tolist() == refs
    return want


@pytest.mark.parametrize("lens,Hk,d,page,parents,new", [
    ([5], 1, 64, 16, [0], [1]), ([16], 1, 64, 16, [0], [1]), ([0], 2, 128, 16, [-1], [0]),
    ([20, 0, 0], 2, 64, 16, [0, 0, 0], [1, 1, 1]),            # one to three
    ([20, 33, 7], 2, 96, 16, [1, 1, 1], [1, 0, 40]),          # all from the middle
    ([20, 33, 7], 2, 256, 16, [2, 0, 1], [1, 1, 1]),          # a rotation: no copies
    ([32, 48, 16], 8, 128, 16, [1, 1, 2], [1, 1, 1]),         # whole pages only
    ([300, 1, 129, 64], 4, 128, 64, [-1, 2, 2, -1], [0, 5, 1, 200]),
    ([300, 1, 129, 64], 4, 128, 64, None, [1, 127, 0, 300]),  # growth alone
    ([300, 1, 129, 64], 1, 64, 32, [3, 0, -1, -1], None),     # no new tokens
    ([40 + 3 * i for i in range(96)], 2, 64, 16, [(i * 5) % 96 for i in range(96)], [1] * 96),
    ([40 + 3 * i for i in range(96)], 2, 64, 16, [i // 8 * 8 + (i * 3) % 5 for i in range(96)], [1] * 96),
    ([1000 + 7 * i for i in range(40)], 1, 64, 16,            # a cluster's work
     [-1 if i % 7 == 0 else (i * 11) % 40 for i in range(40)], [i % 90 for i in range(40)]),
])
def test_fork(lens, Hk, d, page, parents, new):
    p, table, refs = state(lens, Hk, d, page, seed=len(lens), spare=len(lens) * 3 + 20,
                           cols=max(lens) // page + 22)
    check_fork(p, table, lens, refs, parents, new)


def test_fork_of_sequences_that_share_pages():
    lens = [100, 105, 100, 40, 41]
    p, table, refs = state(lens, 2, 64, 16, seed=3, spare=40, shared=[(0, 1), (0, 2), (3, 4)])
    want = check_fork(p, table, lens, refs, [1, 1, 0, -1, 1], [1, 2, 20, 17, 1])
    count = [0] * len(refs)
    for row in want[0]:
        for x in row:
            if x >= 0:
                count[x] += 1
    assert count == want[2]


def test_fork_keeps_spare_pages_and_fills_holes():
    """Entries behind the last key are the owner's to use; others get theirs new."""
    lens = [20, 20, 20]
    p, table, refs = state(lens, 1, 64, 16, seed=4, spare=12)
    spare = [x for x, r in enumerate(refs) if r == 0][:3]
    table[0][2], table[0][4], table[1][3] = spare
    for x in spare:
        refs[x] = 1
    check_fork(p, table, lens, refs, [0, 0, 2], [30, 30, 5])


def test_pages_given_back_are_given_out_in_the_same_step():
    lens = [64, 64]
    p, table, refs = state(lens, 2, 64, 16, seed=5, spare=0, cols=6)
    # Four are freed, and there are no others: ceil(45 / 16) and one for 67 tokens.
    check_fork(p, table, lens, refs, [-1, 1], [45, 3])


def test_fork_out_of_pages():
    lens = [20, 20]
    p, table, refs = state(lens, 2, 64, 16, seed=6, spare=1, cols=6)
    want = ref.fork(p.k_cache, p.v_cache, table, lens, refs, [0, 0], [1, 50])
    got, _ = run_fork(p, table, lens, refs, [0, 0], [1, 50])
    assert fattn.device_status() & 0xffff == FORK
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2]
    assert same(got[3], want[3]) and same(got[4], want[4])
    assert -1 in got[0].tolist()[1][:5]


@pytest.mark.parametrize("what,change", [
    ("parent past", dict(parents=[0, 3, 2])), ("parent", dict(parents=[0, -2, 2])),
    ("length", dict(lens=[20, -3, 20])), ("long", dict(lens=[20, 10 ** 9, 20])),
    ("entry", dict(entry=10 ** 6)), ("entry", dict(entry=-5)), ("starts", dict(cu=[0, 3, 1, 2])),
    ("too many", dict(cu=[0, 10 ** 9, 10 ** 9, 10 ** 9]))])
def test_fork_reports_and_stays_in_range(what, change):
    lens = change.get("lens", [20, 33, 20])
    p, table, refs = state([20, 33, 20], 2, 64, 16, seed=7, spare=20, cols=8)
    if "entry" in change:
        table[1][1] = change["entry"]
    kc, vc = p.k_cache.cuda(), p.v_cache.cuda()
    got = fattn.kv_fork(kc, vc, ints(table), ints(lens), ints(refs), ints(change.get("parents", [0, 0, 1])),
                        ints(change.get("cu", [0, 1, 2, 3])))
    assert fattn.device_status() & 0xffff == FORK, what
    assert all(-1 <= x < len(refs) for row in got[0].tolist() for x in row)
    assert all(0 <= x <= 8 * 16 for x in got[1].tolist())


def test_fork_of_nothing():
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    got = fattn.kv_fork(kc, kc.clone(), torch.zeros(0, 3, dtype=torch.int32, device="cuda"), ints([]),
                        ints([0] * 4), ints([]), ints([0]))
    assert got[0].shape == (0, 3)


def test_fork_in_a_captured_graph_is_a_beam_search():
    """The lists in place, the step captured once: ten steps of appended tokens
    and reordered beams leave in the cache what a plain list of tokens holds."""
    B, page, cols, pages = 4, 16, 6, 40
    g = torch.Generator().manual_seed(8)
    kc = torch.zeros(pages, 1, page, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    table, lens, refs = ints([[-1] * cols] * B), ints([0] * B), ints([0] * pages)
    parents, cu = ints([-1] * B), ints([0, 1, 2, 3, 4])
    k, v = (torch.zeros(B, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(fattn.kv_fork_workspace_size(B, cols, pages), dtype=torch.uint8, device="cuda")

    def step():
        fattn.kv_fork(kc, vc, table, lens, refs, parents, cu, page_table_out=table, kv_len_out=lens,
                      page_refs_out=refs, workspace=ws)
        fattn.kv_append(k, v, kc, vc, table, cu, lens)

    graph = torch.cuda.CUDAGraph()
    step()
    for t, start in ((table, -1), (lens, 0), (refs, 0)):
        t.fill_(start)
    with torch.cuda.graph(graph):
        step()
    hist = [[] for _ in range(B)]
    for i in range(60):
        par = [-1] * B if i == 0 else torch.randint(0, B, (B,), generator=g).tolist()
        parents.copy_(torch.tensor(par, dtype=torch.int32))
        values = torch.randint(0, 200, (B,), generator=g).tolist()
        for b in range(B):
            k[b], v[b] = float(values[b]), float(-values[b])
        graph.replay()
        hist = [(hist[p] if p >= 0 else []) + [values[b]] for b, p in enumerate(par)]
    torch.cuda.synchronize()
    assert fattn.device_status() == 0
    t = table.tolist()
    for b in range(B):
        assert int(lens[b]) == len(hist[b])
        got = [float(kc[t[b][j // page], 0, j % page, 5]) for j in range(len(hist[b]))]
        assert got == [float(x) for x in hist[b]], b
        assert [float(vc[t[b][j // page], 0, j % page, 9]) for j in range(len(hist[b]))] == [-x for x in got]
    count = [0] * pages
    for row in t:
        for x in row:
            if x >= 0:
                count[x] += 1
    assert refs.tolist() == count


# ------------------------------------------------------------------ a search
def test_a_drafting_loop_gives_the_plain_loops_outputs():
    """Fork (growth), masks, append, tree attention, keep: after every step the
    tree's outputs are those of a plain cache of the kept tokens."""
    from tests.test_paged_gpu import check
    B, Hq, Hk, d, page, cols = 3, 4, 2, 64, 16, 20
    pages = 40
    g = torch.Generator().manual_seed(9)
    kc = torch.full((pages, Hk, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    table, lens, refs = ints([[-1] * cols] * B), ints([0] * B), ints([0] * pages)
    past_k = [torch.zeros(0, Hk, d, dtype=torch.bfloat16) for _ in range(B)]
    past_v = [x.clone() for x in past_k]
    for step in range(6):
        n = [int(x) for x in torch.randint(1, 30, (B,), generator=g)]
        cu = [0, n[0], n[0] + n[1], sum(n)]
        table, lens, refs = fattn.kv_fork(kc, vc, table, lens, refs, None, ints(cu))
        trees = [ref.random_tree(x, g) for x in n]
        q, k, v = (torch.randn(cu[-1], h, d, generator=g).bfloat16() for h in (Hq, Hk, Hk))
        mask, pos = fattn.tree_mask(ints([x for t in trees for x in t]), ints(cu), lens, max(n))
        fattn.kv_append(k.cuda(), v.cuda(), kc, vc, table, ints(cu), lens)
        o, lse = fattn.attn_fwd_tree(q.cuda(), kc, vc, table, ints(cu), lens, mask, max(n))
        kept = [sorted(ref.paths(t)[-1]) for t in trees]
        want, lens_now = [], []
        for b in range(B):
            kb, vb = (torch.cat([past, new[cu[b]:cu[b + 1]]]) for past, new in ((past_k[b], k), (past_v[b], v)))
            L = kb.shape[0]
            one = torch.zeros(1, L, dtype=torch.int32)
            want.append(ref.tree_attention(q[cu[b]:cu[b + 1]], kb.transpose(0, 1)[None],
                                           vb.transpose(0, 1)[None], one, [0, n[b]], [L],
                                           ref.paths(trees[b]), fattn.default_scale(d)))
            base = past_k[b].shape[0]
            assert pos[0, cu[b]:cu[b + 1]].tolist() == [base + len(r) - 1 for r in ref.paths(trees[b])]
            past_k[b], past_v[b] = (torch.cat([x[:base], x[[base + t for t in kept[b]]]]) for x in (kb, vb))
            lens_now.append(base + len(kept[b]))
        check(o, lse, tuple(torch.cat([w[i] for w in want]) for i in range(5)), torch.bfloat16, 200)
        fattn.kv_keep(kc, vc, table, ints(cu), lens, padded(kept), ints(list(map(len, kept))),
                      kv_len_out=lens)
        assert lens.tolist() == lens_now
    assert fattn.device_status() == 0


@pytest.mark.parametrize("B,spare", [(2049, 100), (2500, 36000), (70, 40000)])
def test_fork_of_many_sequences_and_pages(B, spare):
    """More sequences than the lists in shared memory hold, more pages than each
    block counts for itself; free pages before, between and behind those in use."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 70, (B,), generator=g).tolist()
    parents = torch.randint(-1, B, (B,), generator=g).tolist()
    new = torch.randint(0, 40, (B,), generator=g).tolist()
    p, table, refs = state(lens, 1, 64, 16, seed=9, spare=spare + 3 * B, cols=8)
    check_fork(p, table, lens, refs, parents, new)


def test_growth_of_a_long_cache():
    """One sequence of 40000 pages, room for 30000 more: one table row, most of
    the pool."""
    cols = 70001
    p, table, refs = state([40000 * 16 - 5], 1, 64, 16, seed=10, spare=30100, cols=cols)
    check_fork(p, table, [40000 * 16 - 5], refs, None, [30000 * 16])
