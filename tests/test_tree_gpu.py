"""GPU tests of attn_fwd_tree and tree_mask against the fp64 reference: trees of
one token to several hundred, arbitrary masks, rows that see nothing, trees that
begin anywhere in a key tile, grouped heads, both types, whatever lies in unused
slots and mask bits, strides, splits, streams and graphs."""
import pytest
import torch

from tests import search_ref as ref
from tests.paged import make_paged
from tests.test_paged_gpu import check, queries
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def make(q_lens, kv_lens, Hk, d, page, dtype, seed=0, **kw):
    p = make_paged(q_lens, kv_lens, Hk, d, page, dtype, seed=seed, fill=float("nan"), **kw)
    g = torch.Generator().manual_seed(seed + 1)
    trees = [ref.random_tree(n, g) for n in q_lens]
    return p, trees, [row for t in trees for row in ref.paths(t)]


def words_of(p):
    return max((p.max_q + 31) // 32, 1)


def run(p, q, mask, **kw):
    return fattn.attn_fwd_tree(q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(), mask.cuda(),
                               max(p.max_q, 1), **kw)


def reference(p, q, rows, scale=None):
    scale = fattn.default_scale(q.shape[-1]) if scale is None else scale
    return ref.tree_attention(q, p.k_cache, p.v_cache, p.table, p.cu, p.kv_len, rows, scale)


CASES = [
    # q_lens, kv_lens, Hq, Hk, d, page
    ([1], [1], 1, 1, 64, 16),
    ([1], [129], 4, 1, 128, 16),
    ([7], [7], 4, 4, 64, 16),                    # nothing before the tree
    ([8, 8, 8], [128, 135, 136], 4, 1, 128, 32),  # ends at, in and one key into a tile
    ([5, 3, 1, 7], [260, 3, 900, 1300], 12, 4, 96, 64),
    ([26, 26], [150, 1100], 32, 8, 128, 16),
    ([33, 31, 32], [200, 31, 160], 1, 1, 64, 16),  # around a word, around a lane quarter
    ([64, 64], [700, 65], 8, 2, 128, 64),
    ([63, 1, 65, 0, 20], [300, 0, 200, 9, 20], 6, 2, 128, 64),
    ([129], [140], 2, 2, 64, 64),
    ([200, 130], [256, 777], 2, 1, 128, 16),
    ([300, 2], [300, 1024], 3, 1, 96, 128),      # a mask of ten words
    ([3], [300], 128, 1, 64, 16),                # one token a tile
    ([30, 4], [20, 2], 4, 2, 64, 16),            # more new tokens than keys
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk,d,page", CASES,
                         ids=["B%d_q%d_k%d_H%d-%d_d%d_p%d" % (len(c[0]), max(c[0]), max(c[1]), *c[2:])
                              for c in CASES])
def test_against_reference(q_lens, kv_lens, Hq, Hk, d, page, dtype):
    p, _, rows = make(q_lens, kv_lens, Hk, d, page, dtype, seed=sum(kv_lens))
    q = queries(p.T, Hq, d, dtype, 1)
    o, lse = run(p, q, ref.pack(rows, words_of(p)))
    assert fattn.device_status() == 0
    check(o, lse, reference(p, q, rows), dtype, max(kv_lens))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("seen", [0.0, 0.03, 0.5, 1.0])
def test_any_mask(seen, dtype):
    """Bits anywhere, tokens after a row's own among them; rows without a bit
    see the keys before the tree, or nothing where there are none."""
    q_lens, kv_lens = [40, 17, 150, 9], [40, 300, 150, 137]
    p, _, _ = make(q_lens, kv_lens, 2, 64, 16, dtype, seed=3)
    g = torch.Generator().manual_seed(4)
    rows = [{j for j in range(n) if torch.rand(1, generator=g) < seen} for n in q_lens for _ in range(n)]
    q = queries(p.T, 4, 64, dtype, 5)
    o, lse = run(p, q, ref.pack(rows, words_of(p)))
    assert fattn.device_status() == 0
    check(o, lse, reference(p, q, rows), dtype, max(kv_lens), "seen %s" % seen)


def test_bits_and_words_behind_a_tree_do_not_count():
    """Every bit from a sequence's n on is set, in a mask with more words than
    any tree needs, whose rows are apart."""
    p, _, rows = make([5, 37, 64], [300, 90, 128], 2, 128, 32, torch.bfloat16, seed=8)
    n_of = [n for n in (5, 37, 64) for _ in range(n)]
    full = [row | set(range(n, 160)) for row, n in zip(rows, n_of)]
    wide = torch.full((p.T, 9), -1, dtype=torch.int32)
    wide[:, 2:7] = ref.pack(full, 5)
    q = queries(p.T, 4, 128, torch.bfloat16, 6)
    o, lse = run(p, q, wide[:, 2:7])
    assert fattn.device_status() == 0
    check(o, lse, reference(p, q, rows), torch.bfloat16, 300)


def test_hidden_keys_may_be_nan():
    p, _, rows = make([20], [150], 1, 64, 16, torch.bfloat16, seed=9)
    never = [t for t in range(20) if all(t not in r for r in rows[:5])]
    q = queries(p.T, 2, 64, torch.bfloat16, 7)
    want = reference(p, q, rows)
    for t in never:
        pos = 130 + t
        p.k_cache[p.table[0, pos // 16], :, pos % 16] = float("nan")
    o, lse = run(p, q, ref.pack(rows, 1))
    assert fattn.device_status() & 0xff == 5  # rows that see one are NaN
    got = o[:5].double().cpu()
    assert bool(torch.isfinite(got).all())
    part = tuple(x[:5] for x in want)
    check(o[:5], lse[:5], part, torch.bfloat16, 150)


def test_a_causal_mask_gives_the_causal_calls_bits():
    """The same rows seen, the same arithmetic."""
    q_lens, kv_lens = [50, 3, 90], [400, 3, 90]
    p, _, _ = make(q_lens, kv_lens, 2, 128, 32, torch.bfloat16, seed=10)
    rows = [set(range(i + 1)) for n in q_lens for i in range(n)]
    q = queries(p.T, 8, 128, torch.bfloat16, 11)
    o, lse = run(p, q, ref.pack(rows, words_of(p)))
    check(o, lse, reference(p, q, rows), torch.bfloat16, 400)
    o2, lse2 = fattn.attn_fwd_paged(q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(), p.max_q)
    # one unit each, no key tile skipped in either
    assert torch.equal(o[50:53], o2[50:53]) and torch.equal(lse[50:53], lse2[50:53])


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk,d,page", [
    ([24], [40000], 4, 1, 128, 64),                        # one unit over every CTA
    ([64, 20], [20000, 9000], 8, 2, 64, 16),
    ([200], [9000], 4, 2, 128, 128),                       # pairs of tiles, split
    ([1 + i % 40 for i in range(300)], [41 + (i * 37) % 200 for i in range(300)], 2, 1, 64, 16),
])
def test_long_and_many_sequences(q_lens, kv_lens, Hq, Hk, d, page):
    p, _, rows = make(q_lens, kv_lens, Hk, d, page, torch.bfloat16, seed=7, extra_cols=5)
    q = queries(p.T, Hq, d, torch.bfloat16, 2, 2.5)
    mask = ref.pack(rows, words_of(p))
    o, lse = run(p, q, mask)
    again = run(p, q, mask)
    assert fattn.device_status() == 0
    check(o, lse, reference(p, q, rows), torch.bfloat16, max(kv_lens))
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_strides_rows_behind_the_last_sequence_and_a_scale():
    p, _, rows = make([9, 30], [100, 260], 2, 96, 16, torch.float16, seed=12)
    T = p.T + 5
    big = torch.zeros(T, 3, 4, 96, dtype=torch.float16)
    big[:p.T, 1] = queries(p.T, 4, 96, torch.float16, 13)
    q = big[:, 1]
    out = torch.full((T, 8, 96), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T, 4), 7.0, device="cuda")
    mask = torch.cat([ref.pack(rows, 1), torch.full((5, 1), -1, dtype=torch.int32)])
    fattn.attn_fwd_tree(big.cuda()[:, 1], p.k_cache.cuda(), p.v_cache.cuda(), *p.lists(), mask.cuda(),
                        30, scale=0.3, out=out[:, 2:6], lse=lse)
    assert fattn.device_status() == 0
    assert bool((out[p.T:] == 7).all()) and bool((lse[p.T:] == 7).all())
    assert bool((out[:, :2] == 7).all()) and bool((out[:, 6:] == 7).all())
    check(out[:p.T, 2:6], lse[:p.T], reference(p, q[:p.T], rows, 0.3), torch.float16, 260)


# ------------------------------------------------------------------ masks
@pytest.mark.parametrize("q_lens,extra", [([1], 0), ([5, 0, 1, 33], 0), ([64, 31, 32, 200], 40),
                                          ([700, 3], 0), ([3] * 400, 0)])
def test_tree_mask_is_the_paths(q_lens, extra):
    g = torch.Generator().manual_seed(sum(q_lens))
    kv = [n + int(torch.randint(0, 500, (1,), generator=g)) for n in q_lens]
    p, trees, rows = make(q_lens, kv, 1, 64, 16, torch.bfloat16, seed=2)
    max_q = p.max_q + extra
    words = (max_q + 31) // 32
    parents = torch.tensor([x for t in trees for x in t], dtype=torch.int32)
    _, cu, kv_len = p.lists()
    mask, pos = fattn.tree_mask(parents.cuda(), cu, kv_len, max_q)
    assert fattn.device_status() == 0
    assert torch.equal(mask.cpu(), ref.pack(rows, words))
    want = [kv[b] - q_lens[b] + len(r) - 1 for b in range(len(q_lens))
            for r in rows[p.cu[b]:p.cu[b + 1]]]
    assert pos.shape == (1, p.T) and pos[0].tolist() == want


def test_a_tree_beyond_the_shared_memory():
    """5000 tokens: a chain of 130 to every 40th, the others leaves of those."""
    n, g = 5000, torch.Generator().manual_seed(3)
    parents = [i - 40 if i % 40 == 0 else i // 40 * 40 for i in range(n)]
    parents[0] = -1
    mask, pos = fattn.tree_mask(torch.tensor(parents, dtype=torch.int32).cuda(),
                                torch.tensor([0, n], dtype=torch.int32).cuda(),
                                torch.tensor([n + 9], dtype=torch.int32).cuda(), n)
    assert fattn.device_status() == 0
    rows = ref.paths(parents)
    some = torch.randperm(n, generator=g)[:300].tolist() + [0, 1, n - 1]
    assert torch.equal(mask[some].cpu(), ref.pack([rows[i] for i in some], 157))
    assert pos[0].tolist() == [9 + len(r) - 1 for r in rows]


def test_tree_mask_of_a_chain_is_causal():
    n = 150
    parents = torch.arange(-1, n - 1, dtype=torch.int32)
    mask, pos = fattn.tree_mask(parents.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(),
                                torch.tensor([1000], dtype=torch.int32).cuda(), n)
    assert torch.equal(mask.cpu(), ref.pack([set(range(i + 1)) for i in range(n)], 5))
    assert pos[0].tolist() == list(range(850, 1000))


@pytest.mark.parametrize("bad", [3, 4, 99, -2, 2 ** 31 - 1, -2 ** 31])
def test_tree_mask_reports_bad_parents(bad):
    """Token 3's parent is itself, a later token or no token: it is a root."""
    parents = [-1, 0, 1, bad, 3, 2]
    good = [-1, 0, 1, -1, 3, 2]
    mask, pos = fattn.tree_mask(torch.tensor(parents, dtype=torch.int32).cuda(),
                                torch.tensor([0, 6], dtype=torch.int32).cuda(),
                                torch.tensor([16], dtype=torch.int32).cuda(), 6)
    assert fattn.device_status() & 0xffff == 6 | 9 << 8
    rows = ref.paths(good)
    assert torch.equal(mask.cpu(), ref.pack(rows, 1)) and pos[0].tolist() == [10 + len(r) - 1 for r in rows]


@pytest.mark.parametrize("cu", [[1, 3, 6], [0, 7, 6], [0, 4, 9], [0, -1, 6], [0, 3, 2 ** 31 - 1]])
def test_tree_mask_reports_bad_starts(cu):
    parents = torch.full((6,), -1, dtype=torch.int32)
    keep = torch.full((6, 1), 77, dtype=torch.int32, device="cuda")
    fattn.tree_mask(parents.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),
                    torch.tensor([10, 10], dtype=torch.int32).cuda(), 6, mask=keep)
    assert fattn.device_status() & 0xffff == 6 | 9 << 8


def test_tree_mask_skips_what_has_no_word():
    """More tokens than the mask's words: skipped, reported, nothing behind
    the rows touched."""
    parents = torch.arange(-1, 69, dtype=torch.int32)
    mask = torch.full((70, 2), 5, dtype=torch.int32, device="cuda")
    pos = torch.full((1, 70), -9, dtype=torch.int32, device="cuda")
    fattn.tree_mask(parents.cuda(), torch.tensor([0, 70], dtype=torch.int32).cuda(),
                    torch.tensor([100], dtype=torch.int32).cuda(), 64, mask=mask, positions=pos)
    assert fattn.device_status() & 0xffff == 6 | 9 << 8
    assert torch.equal(mask[:64].cpu(), ref.pack([set(range(i + 1)) for i in range(64)], 2))
    assert bool((mask[64:] == 5).all()) and bool((pos[0, 64:] == -9).all())


def test_masks_made_in_a_captured_graph_follow_the_parents():
    p, trees, rows = make([24, 7], [200, 31], 2, 64, 16, torch.bfloat16, seed=14)
    q = queries(p.T, 4, 64, torch.bfloat16, 15)
    args = (q.cuda(), p.k_cache.cuda(), p.v_cache.cuda())
    lists = p.lists()
    parents = torch.full((p.T,), -1, dtype=torch.int32, device="cuda")
    ws = torch.empty(fattn.paged_workspace_size(4, 2, 64, 24), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(args[0]), torch.empty(p.T, 4, device="cuda")
    mask, pos = torch.empty(p.T, 1, dtype=torch.int32, device="cuda"), torch.empty(
        1, p.T, dtype=torch.int32, device="cuda")

    def step():
        fattn.tree_mask(parents, lists[1], lists[2], 24, mask=mask, positions=pos)
        fattn.attn_fwd_tree(*args, *lists, mask, 24, workspace=ws, out=out, lse=lse)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (14, 99):
        g = torch.Generator().manual_seed(seed)
        trees = [ref.random_tree(n, g) for n in (24, 7)]
        rows = [r for t in trees for r in ref.paths(t)]
        parents.copy_(torch.tensor([x for t in trees for x in t], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert fattn.device_status() == 0
        check(out, lse, reference(p, q, rows), torch.bfloat16, 200)


def test_two_trees_at_once_on_two_streams():
    """Workspaces of their own: calls that overlap do not meet."""
    sets, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed, shape in ((20, ([26] * 6, [700 + 90 * i for i in range(6)], 2, 128, 16)),
                        (21, ([60, 200], [3000, 900], 4, 64, 32))):
        p, trees, rows = make(*shape, torch.bfloat16, seed=seed)
        q = queries(p.T, 8, shape[3], torch.bfloat16, seed)
        args = [t.cuda() for t in (q, p.k_cache, p.v_cache)]
        parents = torch.tensor([x for t in trees for x in t], dtype=torch.int32).cuda()
        sets.append((p, q, rows, args, p.lists(), parents))
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for (p, q, rows, args, lists, parents), s in zip(sets, streams):
            mask, _ = fattn.tree_mask(parents, lists[1], lists[2], p.max_q, stream=s)
            got.append(fattn.attn_fwd_tree(*args, *lists, mask, p.max_q, stream=s))
    torch.cuda.synchronize()
    assert fattn.device_status() == 0
    for i, (o, lse) in enumerate(got):
        p, q, rows = sets[i % 2][:3]
        if i < 2:
            check(o, lse, reference(p, q, rows), torch.bfloat16, 3000)
        assert torch.equal(o, got[i % 2][0]) and torch.equal(lse, got[i % 2][1])
