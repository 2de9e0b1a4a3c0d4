"""GPU tests of attn_fwd_paged with NaN and infinite queries and keys: a row
whose scores hold a NaN or +inf is NaN in o and lse, whether its unit is whole
or split over CTAs; a score of -inf takes no part; all other rows are as ever."""
import math

import pytest
import torch

from tests.paged import make_paged
from tests.test_paged_gpu import check, queries, run
from tiled_online_softmax_fwd_gb300 import fattn

pytestmark = pytest.mark.gpu


def expected(p, q, causal=True):
    """As serving_ref.paged_attention, and the rows [T, Hq] with a NaN or +inf
    among their scores.  Scores of -inf (an infinite key against a query of
    the other sign) are left out of the sizes that errors are relative to."""
    T, Hq, d = q.shape
    Hk, page = p.k_cache.shape[1], p.k_cache.shape[2]
    G, scale = Hq // Hk, fattn.default_scale(d)
    o = torch.zeros(T, Hq, d, dtype=torch.float64)
    size = torch.zeros_like(o)
    lse, terms, vmax = [torch.zeros(T, Hq, dtype=torch.float64) for _ in range(3)]
    poisoned = torch.zeros(T, Hq, dtype=torch.bool)
    for b, n in enumerate(p.kv_len):
        t0, t1 = p.cu[b], p.cu[b + 1]
        idx = torch.arange(n)
        rows = p.table[b, idx // page].long()
        for h in range(Hq):
            k = p.k_cache[rows, h // G, idx % page].double()
            v = p.v_cache[rows, h // G, idx % page].double()
            x = q[t0:t1, h].double() @ k.T * scale
            t = q[t0:t1, h].double().abs() @ k.abs().T * scale
            if causal:
                hidden = idx[None, :] > torch.arange(n - (t1 - t0), n)[:, None]
                x, t = x.masked_fill(hidden, -math.inf), t.masked_fill(hidden, 0.0)
            poisoned[t0:t1, h] = (torch.isnan(x) | (x == math.inf)).any(-1)
            t = torch.where(x == -math.inf, 0.0, t)
            y = torch.logsumexp(x, -1)
            w = torch.where(x == -math.inf, 0.0, torch.exp(x - y[:, None]))
            o[t0:t1, h], lse[t0:t1, h], size[t0:t1, h] = w @ v, y, w @ v.abs()
            terms[t0:t1, h], vmax[t0:t1, h] = t.amax(-1), v.abs().max()
    return (o, lse, size, terms, vmax), poisoned


def verify(p, q, dtype, what, causal=True):
    want, poisoned = expected(p, q, causal)
    assert bool(poisoned.any()) and not bool(poisoned.all()), "%s: the case has both kinds" % what
    fattn.device_status()
    o, lse = run(p, q, causal)
    status = fattn.device_status()
    bad = poisoned.cuda()
    assert bool(torch.isnan(o[bad]).all()), "%s: %d of %d elements of o are numbers" % (
        what, int((~torch.isnan(o[bad])).sum()), o[bad].numel())
    assert bool(torch.isnan(lse[bad]).all()), "%s: lse %s" % (what, lse[bad].tolist()[:4])
    good = ~poisoned
    check(o[good.cuda()], lse[good.cuda()], tuple(x[good] for x in want), dtype, max(p.kv_len), what)
    # bf16 reports a row that is not finite; fp16 does not look for one.
    assert status & 0xff == (5 if dtype == torch.bfloat16 else 0), what


def at(p, b, j):
    """Where position j of sequence b lies in the caches."""
    page = p.k_cache.shape[2]
    return int(p.table[b, j // page]), slice(None), j % page


# q_lens, kv_lens, Hq, Hk: units of at most 32 rows, of one tile, of two; the
# short ones lie whole in a CTA, the long ones are split.
UNITS = [([1, 1, 1], [300, 40, 129], 8, 2), ([1, 1], [9000, 200], 8, 2),
         ([50, 3], [300, 40], 4, 2), ([60, 3], [12000, 40], 4, 2),
         ([300, 1], [700, 64], 2, 1), ([300, 1], [14000, 64], 2, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk", UNITS)
def test_a_key_that_is_not_finite(q_lens, kv_lens, Hq, Hk, d, dtype):
    for value in (float("nan"), float("inf"), -float("inf")):
        for j in (0, kv_lens[0] // 2, kv_lens[0] - 5):
            p = make_paged(q_lens, kv_lens, Hk, d, 32, dtype, seed=d + j)
            q = queries(p.T, Hq, d, dtype, 3)
            page, heads, slot = at(p, 0, j)
            p.k_cache[page, heads, slot, 7] = value
            verify(p, q, dtype, "%s at key %d" % (value, j))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk", UNITS)
def test_a_query_that_is_not_finite(q_lens, kv_lens, Hq, Hk, d, dtype):
    """NaN, and an infinity: against hundreds of keys of both signs some score
    is +inf."""
    for value in (float("nan"), float("inf")):
        p = make_paged(q_lens, kv_lens, Hk, d, 16, dtype, seed=d)
        q = queries(p.T, Hq, d, dtype, 4)
        q[q_lens[0] // 2, 1, 3] = value
        q[q_lens[0] - 1, Hq - 1, d - 1] = value
        verify(p, q, dtype, "query %s" % value)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_score_of_a_row_is_not_finite(dtype):
    """NaN at each key of a stretch that covers whole key tiles and whole
    CTAs' shares, and at all keys of one sequence."""
    for j0, j1 in ((0, 5000), (4000, 9000), (8872, 9000), (0, 9000)):
        p = make_paged([1, 2], [9000, 300], 2, 64, 16, dtype, seed=j1)
        q = queries(p.T, 8, 64, dtype, 5)
        for j in range(j0, j1):
            page, heads, slot = at(p, 0, j)
            p.k_cache[page, heads, slot, j % 64] = float("nan")
        verify(p, q, dtype, "NaN at keys %d..%d" % (j0, j1), causal=False)
