"""Timing cases of the operators around drafted, forked and cross-attending
sequences: attention for trees of drafted tokens over a paged cache, keeping a
tree's accepted tokens, forking, growing and freeing the cache's sequences, and
cross attention to an encoder's states (forward and backward).

Each case names one operator and its sizes.  ``run`` makes one pass, either in
plain torch operations in 32 bits (``own`` false) or through the library's
entry points (``own`` true); ``exact`` gives the result in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One tree of drafted tokens for each of a few short conversations,
        # the same tree shape at every step (its masks are made once): latency.
        dict(name="tree_few", op="tree", B=4, Hq=32, Hk=8, d=128, dtype="bf16", q_lo=26, q_hi=26,
             k_lo=150, k_hi=1100, page=16, fresh=False),
        # Trees of 64 tokens for many long conversations (up to 32K keys).
        dict(name="tree_long", op="tree", B=16, Hq=32, Hk=8, d=128, dtype="bf16", q_lo=64, q_hi=64,
             k_lo=12000, k_hi=32768, page=64, fresh=False),
        # Trees drafted anew at each step (the pass makes their masks and
        # positions), ragged, from a single token to 200; one key head a query
        # head, fp16.
        dict(name="tree_fresh_d64", op="tree", B=24, Hq=16, Hk=16, d=64, dtype="fp16", q_lo=1,
             q_hi=200, k_lo=1, k_hi=4096, page=32, fresh=True),
        # The end of a drafting step, few sequences: the drafts were appended,
        # the accepted ones are moved together behind the prefix.
        dict(name="keep_few", op="keep", B=4, Hq=0, Hk=8, d=128, dtype="bf16", q_lo=26, q_hi=26,
             k_lo=150, k_hi=1100, page=16, m_hi=6),
        # The same for a large ragged batch with wider trees.
        dict(name="keep_many", op="keep", B=192, Hq=0, Hk=8, d=128, dtype="bf16", q_lo=20, q_hi=129,
             k_lo=100, k_hi=1500, page=64, m_hi=24),
        # A step of a beam search over two requests: beams continue other
        # beams, and each gets room for its next token.
        dict(name="fork_few", op="fork", B=8, beams=4, Hq=0, Hk=8, d=128, dtype="bf16", k_lo=100,
             k_hi=900, page=16, n_hi=1, ended=0.0),
        # Many requests with several candidates each, some of them ended and
        # their places taken by new prompts.
        dict(name="fork_many", op="fork", B=256, beams=4, Hq=0, Hk=4, d=128, dtype="bf16",
             k_lo=500, k_hi=4000, page=32, n_hi=700, ended=0.1),
        # A decoder's single tokens against an encoder's states.
        dict(name="cross_decode", op="cross", B=32, Hq=16, Hk=16, Nq=1, Nk=1500, d=64, dtype="fp16",
             ragged=True, backward=False),
        # Long targets against long ragged sources, grouped heads.
        dict(name="cross_long", op="cross", B=8, Hq=32, Hk=8, Nq=2048, Nk=4096, d=128,
             dtype="bf16", ragged=True, backward=False),
        # Gradients at small odd sizes.
        dict(name="cross_bwd_odd", op="cross", B=3, Hq=12, Hk=4, Nq=333, Nk=501, d=64,
             dtype="fp16", ragged=True, backward=True),
        # Gradients of many positions that attend to one short text.
        dict(name="cross_bwd_short", op="cross", B=2, Hq=16, Hk=16, Nq=4096, Nk=154, d=64,
             dtype="bf16", ragged=True, backward=True),
        # Gradients of a training batch with long ragged sources.
        dict(name="cross_bwd_long", op="cross", B=4, Hq=16, Hk=16, Nq=2048, Nk=4096, d=128,
             dtype="bf16", ragged=True, backward=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "keep", "fork", "cross", "cross", "cross"])
    case = dict(op=op, d=rng.choice([64, 64, 96, 128, 128]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                Hk=rng.choice([1, 2, 4, 5, 8]))
    if op == "cross":
        group = rng.choice([1, 1, 2, 3, 4])
        nq = 1 if rng.random() < 0.2 else _log_int(rng, 2, 2048)
        case.update(B=_log_int(rng, 1, 16), Hq=case["Hk"] * group, Nq=nq,
                    Nk=_log_int(rng, 1, 4096), ragged=rng.random() < 0.7)
        case["backward"] = nq > 1 and rng.random() < 0.5
        while case["B"] > 1 and case["B"] * case["Hq"] * nq * case["Nk"] > 2 ** 29:
            case["B"] //= 2
        return case
    case["page"] = rng.choice([16, 32, 64, 128])
    if op == "fork":
        beams = rng.choice([1, 2, 3, 4, 5, 8])
        hi = _log_int(rng, 16, 3000)
        case.update(beams=beams, B=beams * _log_int(rng, 1, 96 // beams), Hq=0,
                    k_lo=rng.randint(1, hi), k_hi=hi, n_hi=rng.choice([1, 1, 8, 300]),
                    ended=rng.choice([0.0, 0.1, 0.3]))
        return case
    if op == "keep":
        hi = _log_int(rng, 2, 160)
        case.update(B=_log_int(rng, 1, 64), Hq=0, q_lo=rng.randint(1, hi), q_hi=hi, k_lo=1,
                    k_hi=_log_int(rng, hi, 2500), m_hi=rng.randint(1, 24))
        return case
    hi = _log_int(rng, 2, 256)
    case.update(Hq=case["Hk"] * rng.choice([1, 2, 3, 4, 7, 8]), q_lo=rng.randint(1, hi), q_hi=hi,
                k_lo=1, k_hi=_log_int(rng, hi, 8000), B=_log_int(rng, 1, 12), fresh=rng.random() < 0.5)
    while case["B"] > 1 and case["B"] * case["Hq"] * hi * case["k_hi"] > 2 ** 29:
        case["B"] //= 2
    return case


# ------------------------------------------------------------------ inputs
def _spread(case, lo, hi, count, salt):
    """`count` lengths of the case (not of the seed) in [lo, hi], both taken."""
    g = torch.Generator("cpu").manual_seed(count * 7919 + lo * 31 + hi * 17 + salt)
    u = torch.rand(count, generator=g, dtype=torch.float64)
    if lo * 16 < hi:  # spread over their logarithm: mostly short
        n = (lo * (hi / lo) ** u).round().long()
    else:
        n = lo + (u * (hi - lo + 1)).floor().long()
    n = n.clamp(lo, hi)
    n[-1], n[0] = lo, hi
    return n


def _lengths(case):
    """New tokens and keys (the new ones among them) of each sequence."""
    qlen = _spread(case, case["q_lo"], case["q_hi"], case["B"], 1)
    klen = _spread(case, case["k_lo"], case["k_hi"], case["B"], 2).flip(0)
    return qlen, torch.maximum(klen, qlen)


def _key_lengths(case):
    if not case["ragged"]:
        return torch.full((case["B"],), case["Nk"])
    return _spread(case, max(1, case["Nk"] // 3), case["Nk"], case["B"], 3)


def _starts(lengths):
    return torch.cat([torch.zeros(1, dtype=torch.long), lengths.cumsum(0)])


def _tree(n, rng):
    """Parents of n drafted tokens: each continues one of the six before it."""
    parents = [-1]
    for i in range(1, n):
        parents.append(rng.randint(max(0, i - 6), i - 1))
    return parents


def _fork_lists(case, seed):
    """Sequences in groups of beams that share their prompt's whole pages: the
    lists of a cache as its earlier calls left it, and what is asked next."""
    import random
    rng = random.Random(seed * 1000003 + case["B"])
    B, beams, page = case["B"], case["beams"], case["page"]
    groups = B // beams
    klen = _spread(case, case["k_lo"], case["k_hi"], groups, 4)
    need = torch.div(klen + page - 1, page, rounding_mode="floor").tolist()
    room = max(need) + -(-case["n_hi"] // page) + 1
    table, lens, parents, new, used = [], [], [], [], 0
    for g in range(groups):
        shared = int(klen[g]) * 3 // 4 // page
        first = list(range(used, used + shared))
        used += shared
        gone = rng.random() < case["ended"]
        for i in range(beams):
            own_pages = need[g] - shared
            table.append(first + list(range(used, used + own_pages)))
            used += own_pages
            lens.append(int(klen[g]))
            parents.append(-1 if gone else g * beams + rng.randrange(beams))
            # A new prompt in the place of an ended request, else the next token.
            new.append(rng.randint(1, case["n_hi"]) if gone else 1)
    # Room for each sequence's copied page and new tokens, and some to spare.
    pool = used + used // 8 + B + 8 + sum(-(-n // page) + 1 for n in new)
    order = list(range(pool))
    rng.shuffle(order)
    refs = [0] * pool
    for i, row in enumerate(table):
        for p in row:
            refs[order[p]] += 1
        table[i] = [order[p] for p in row] + [-1] * (room - len(row))
    return dict(table=table, lens=lens, parents=parents, new=new, refs=refs, pool=pool)


def prepare(case, seed):
    import random
    g = torch.Generator("cuda").manual_seed(seed)
    dt, d, B, Hk = DTYPES[case["dtype"]], case["d"], case["B"], case["Hk"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    def ints(x):
        return torch.as_tensor(x, dtype=torch.int32).cuda()

    s = dict(case=dict(case), d=d, dtype=dt)
    if case["op"] == "cross":
        Hq, Nq, Nk = case["Hq"], case["Nq"], case["Nk"]
        # Views of the projections' outputs: [B, tokens, heads, d], keys and
        # values packed; the padding holds whatever the encoder gave it.
        s["q"] = randn(B, Nq, Hq, d).transpose(1, 2)
        kv = randn(B, Nk, 2, Hk, d)
        s["k"], s["v"] = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
        s["kv_len"] = ints(_key_lengths(case)) if case["ragged"] else None
        if case["backward"]:
            s["o"], s["lse"] = _plain_cross(s)  # the forward pass kept these
            s["do"] = randn(B, Nq, Hq, d).transpose(1, 2)
        return s
    page = case["page"]
    if case["op"] == "fork":
        lists = _fork_lists(case, seed)
        s["page_table"], s["kv_len"] = ints(lists["table"]), ints(lists["lens"])
        s["page_refs"], s["parents"] = ints(lists["refs"]), ints(lists["parents"])
        s["cu_q"] = ints(_starts(torch.tensor(lists["new"])))
        s["k_cache"] = randn(lists["pool"], Hk, page, d)
        s["v_cache"] = randn(lists["pool"], Hk, page, d)
        return s
    qlen, klen = _lengths(case)
    T = int(qlen.sum())
    used = (klen + page - 1) // page
    max_pages, total = int(used.max()), int(used.sum())
    pool = total + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    first = _starts(used)[:-1].cuda()
    col = torch.arange(max_pages, device="cuda")
    at = first[:, None] + col
    s["page_table"] = torch.where(col < used.cuda()[:, None], order[at.clamp(max=pool - 1)],
                                  torch.full_like(order[:1], -1)).contiguous()
    s["cu_q"], s["kv_len"] = ints(_starts(qlen)), ints(klen)
    s["max_q"], s["T"] = int(qlen.max()), T
    s["k_cache"], s["v_cache"] = randn(pool, Hk, page, d), randn(pool, Hk, page, d)
    rng = random.Random(seed)
    if case["op"] == "keep":
        kv = randn(T, 2, Hk, d)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        kept, kept_len = [], []
        for n in qlen.tolist():
            m = rng.randint(1, min(n, case["m_hi"]))
            kept.append(sorted([0] + rng.sample(range(1, n), m - 1)) + [-1] * (case["m_hi"] - m))
            kept_len.append(m)
        s["kept"], s["kept_len"] = ints(kept), ints(kept_len)
        return s
    s["q"] = randn(T, case["Hq"], d)
    s["parents"] = ints([p for n in qlen.tolist() for p in _tree(n, rng)])
    if not case["fresh"]:
        s["mask"] = _plain_tree(s)[0]
    return s


# ------------------------------------------------------------------ plain forms
def _token_of(s):
    """Sequence and index in it of each of the T new tokens."""
    t = torch.arange(s["T"], device="cuda")
    cu = s["cu_q"].long()
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b]


def _plain_tree(s):
    """Masks int32 [T, words] (bit j: the token sees its sequence's token j,
    itself and those it continues) and positions int32 [1, T]."""
    n, T = s["max_q"], s["T"]
    words = (n + 31) // 32
    b, i = _token_of(s)
    B = s["cu_q"].numel() - 1
    par = s["parents"].long()
    sees = torch.zeros(B, n, n, device="cuda")
    sees[b, i, i] = 1
    has = par >= 0
    sees[b[has], i[has], par[has]] = 1
    for _ in range(max(1, (n - 1).bit_length())):  # paths of twice the length
        sees = (torch.matmul(sees, sees) > 0).float()
    rows = torch.zeros(T, words * 32, dtype=torch.long, device="cuda")
    rows[:, :n] = sees[b, i].long()
    bits = (rows.reshape(T, words, 32) << torch.arange(32, device="cuda")).sum(-1)
    mask = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).int()
    cu = s["cu_q"].long()
    pos = s["kv_len"].long()[b] - (cu[b + 1] - cu[b]) + rows.sum(-1) - 1
    return mask, pos.int()[None]


def _plain_tree_attn(s, mask):
    c, q = s["case"], s["q"]
    T, Hq, d = q.shape
    B, Hk = c["B"], c["Hk"]
    G, n, page = Hq // Hk, s["max_q"], c["page"]
    pages = s["page_table"].clamp(min=0).long()
    L = pages.shape[1] * page
    k = s["k_cache"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hk, L, d).float()
    v = s["v_cache"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hk, L, d).float()
    cu, klen = s["cu_q"].long(), s["kv_len"].long()
    qlen = cu[1:] - cu[:-1]
    rows = (cu[:-1, None] + torch.arange(n, device="cuda")).clamp(max=T - 1)
    qp = q[rows].float().reshape(B, n, Hk, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, d)
    x = torch.matmul(qp, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    # Key j is the prefix's (seen by all) or the sequence's token j - (L - n).
    t = torch.arange(L, device="cuda") - (klen - qlen)[:, None]
    word = (t.clamp(min=0) // 32).clamp(max=mask.shape[1] - 1)
    bits = torch.gather(mask[rows].long(), 2, word[:, None].expand(B, n, L))
    sees = ((bits >> (t.clamp(min=0) % 32)[:, None]) & 1).bool()
    seen = ((t < 0)[:, None] | sees) & (t < qlen[:, None])[:, None]
    x = x.reshape(B, Hk, G, n, L).masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = torch.exp(x - m)
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(B, Hk, G * n, L), v).reshape(B, Hk, G, n, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l))[..., 0]
    b, i = _token_of(s)
    o = o.permute(0, 3, 1, 2, 4)[b, i].reshape(T, Hq, d).to(q.dtype)
    return o, lse.permute(0, 3, 1, 2)[b, i].reshape(T, Hq).contiguous()


def _plain_keep(s):
    page = s["case"]["page"]
    b, i = _token_of(s)
    cu, klen, table = s["cu_q"].long(), s["kv_len"].long(), s["page_table"].long()
    prefix = klen - (cu[1:] - cu[:-1])
    pos = prefix[b] + i
    at = table[b, pos // page]
    s["k_cache"][at, :, pos % page] = s["k"]
    s["v_cache"][at, :, pos % page] = s["v"]
    kept = s["kept"].long()
    row, j = torch.nonzero(torch.arange(kept.shape[1], device="cuda") < s["kept_len"][:, None],
                           as_tuple=True)
    src, dst = prefix[row] + kept[row, j], prefix[row] + j
    for cache in (s["k_cache"], s["v_cache"]):
        cache[table[row, dst // page], :, dst % page] = cache[table[row, src // page], :, src % page]
    return s["k_cache"], s["v_cache"], (prefix + s["kept_len"]).int()


def _plain_fork(s):
    page = s["case"]["page"]
    old, lens, par = s["page_table"].long(), s["kv_len"].long(), s["parents"].long()
    refs = s["page_refs"].long().clone()
    B, width = old.shape
    me, col = torch.arange(B, device="cuda"), torch.arange(width, device="cuda")
    has, src = par >= 0, par.clamp(min=0)
    # The child that goes on with its parent's own pages: the parent itself,
    # else the first.
    first = torch.full((B,), B, dtype=torch.long, device="cuda")
    first.scatter_reduce_(0, src, torch.where(has, me, torch.full_like(me, B)), "amin")
    first = torch.where(has & (par == me), me, first)
    keeps = has & (first[src] == me)
    base = torch.where(has, lens[src], torch.zeros_like(lens))
    whole = base // page
    table = torch.where((keeps[:, None] | (col < whole[:, None])) & has[:, None], old[src],
                        torch.full_like(old, -1))
    n = s["cu_q"].long()
    total = base + n[1:] - n[:-1]
    want = (total + page - 1) // page
    refs.index_add_(0, old[old >= 0], torch.full_like(old[old >= 0], -1))
    refs.index_add_(0, table[table >= 0], torch.ones_like(table[table >= 0]))
    free = torch.nonzero(refs == 0)[:, 0]
    missing = (table < 0) & (col < want[:, None])
    rank = missing.reshape(-1).long().cumsum(0).reshape(B, width) - 1
    table = torch.where(missing, free[rank.clamp(0, free.numel() - 1)], table)
    refs.index_fill_(0, table[missing], 1)
    copies = torch.nonzero(has & ~keeps & (base % page > 0))[:, 0]
    a, z = old[src[copies], whole[copies]], table[copies, whole[copies]]
    slots = (torch.arange(page, device="cuda") < (base % page)[copies, None])[:, None, :, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[z] = torch.where(slots, cache[a], cache[z])
    return table.int(), total.int(), refs.int(), s["k_cache"], s["v_cache"]


def _cross_scores(s):
    """Scaled scores [B, Hk, G Nq, Nk] in 32 bits, -inf behind a source's end."""
    q, k = s["q"].float(), s["k"].float()
    B, Hq, Nq, d = q.shape
    Hk, Nk = k.shape[1], k.shape[2]
    x = torch.matmul(q.reshape(B, Hk, Hq // Hk * Nq, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    if s["kv_len"] is not None:
        behind = torch.arange(Nk, device="cuda") >= s["kv_len"][:, None]
        x = x.masked_fill(behind[:, None, None], -math.inf)
    return x


def _plain_cross(s):
    x = _cross_scores(s)
    B, Hq, Nq, d = s["q"].shape
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = torch.exp(x - m)
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x, s["v"].float())
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).reshape(B, Hq, Nq, d)
    return o.to(s["dtype"]), (m + torch.log(l)).reshape(B, Hq, Nq)


def _plain_cross_bwd(s):
    q, k, v, do = (s[x].float() for x in ("q", "k", "v", "do"))
    B, Hq, Nq, d = q.shape
    Hk = k.shape[1]
    x = _cross_scores(s)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    g = do.reshape(B, Hk, Hq // Hk * Nq, d)
    dv = torch.matmul(p.transpose(2, 3), g)
    dp = torch.matmul(g, v.transpose(2, 3))
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * (1.0 / math.sqrt(d))
    dq = torch.matmul(ds, k).reshape(B, Hq, Nq, d)
    dk = torch.matmul(ds.transpose(2, 3), q.reshape(B, Hk, Hq // Hk * Nq, d))
    return dq.to(s["dtype"]), dk.to(s["dtype"]), dv.to(s["dtype"])


def run(state):
    s, c = state, state["case"]
    if own:
        from tiled_online_softmax_fwd_gb300 import fattn
        if c["op"] == "tree":
            lists = (s["page_table"], s["cu_q"], s["kv_len"])
            if not c["fresh"]:
                return fattn.attn_fwd_tree(s["q"], s["k_cache"], s["v_cache"], *lists, s["mask"],
                                           s["max_q"])
            mask, positions = fattn.tree_mask(s["parents"], s["cu_q"], s["kv_len"], s["max_q"])
            o, lse = fattn.attn_fwd_tree(s["q"], s["k_cache"], s["v_cache"], *lists, mask, s["max_q"])
            return o, lse, mask, positions
        if c["op"] == "keep":
            fattn.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_q"],
                            s["kv_len"])
            kv_len = fattn.kv_keep(s["k_cache"], s["v_cache"], s["page_table"], s["cu_q"],
                                   s["kv_len"], s["kept"], s["kept_len"])
            return s["k_cache"], s["v_cache"], kv_len
        if c["op"] == "fork":
            table, kv_len, refs = fattn.kv_fork(s["k_cache"], s["v_cache"], s["page_table"],
                                                s["kv_len"], s["page_refs"], s["parents"], s["cu_q"])
            return table, kv_len, refs, s["k_cache"], s["v_cache"]
        if c["backward"]:
            return fattn.attn_bwd_cross(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"],
                                        kv_len=s["kv_len"])
        return fattn.attn_fwd_cross(s["q"], s["k"], s["v"], kv_len=s["kv_len"])
    if c["op"] == "tree":
        if not c["fresh"]:
            return _plain_tree_attn(s, s["mask"])
        mask, positions = _plain_tree(s)
        return (*_plain_tree_attn(s, mask), mask, positions)
    if c["op"] == "keep":
        return _plain_keep(s)
    if c["op"] == "fork":
        return _plain_fork(s)
    return _plain_cross_bwd(s) if c["backward"] else _plain_cross(s)


# ------------------------------------------------------------------ floors
def work(case):
    d, B, Hk = case["d"], case["B"], case["Hk"]
    row = Hk * d * 2  # a token's keys, or its values
    if case["op"] == "cross":
        Hq, Nq = case["Hq"], case["Nq"]
        keys = int(_key_lengths(case).sum())
        q, kv, stats = B * Hq * Nq * d * 2, 2 * keys * row, B * Hq * Nq * 4
        pairs = Hq * Nq * keys
        if case["backward"]:
            grads = 2 * B * case["Nk"] * row  # zeros behind a source's end among them
            return {"bytes": 4 * q + kv + grads + stats, "flops": 10 * d * pairs}
        return {"bytes": 2 * q + kv + stats, "flops": 4 * d * pairs}
    page = case["page"]
    if case["op"] == "fork":
        x = _fork_lists(case, 0)
        kept = sum(len([p for p in r if p >= 0]) for r in x["table"])
        copied = sum(x["lens"][p] % page for b, p in enumerate(x["parents"]) if p >= 0 and p != b and
                     (p in x["parents"][:b] or x["parents"][p] == p))
        return {"bytes": 4 * copied * row + 4 * kept + 4 * B * len(x["table"][0]) + 8 * x["pool"] + 16 * B,
                "flops": 0}
    qlen, klen = _lengths(case)
    tokens = int(qlen.sum())
    plan = 4 * (2 * B + 1) + 4 * int(((klen + page - 1) // page).sum())
    if case["op"] == "keep":
        kept = B * (1 + case["m_hi"]) // 2
        return {"bytes": 4 * tokens * row + 4 * kept * row + plan + 4 * kept + 8 * B, "flops": 0}
    words = (case["q_hi"] + 31) // 32
    pairs = int((qlen * (klen - qlen + 1)).sum())
    made = 12 * tokens if case["fresh"] else 0
    return {"bytes": 2 * int(klen.sum()) * row + tokens * case["Hq"] * (4 * d + 4) +
            4 * tokens * words + plan + made,
            "flops": 4 * d * case["Hq"] * pairs}


# ------------------------------------------------------------------ 64 bits
def _exact_tree(case, s):
    cu, klen, par = s["cu_q"].tolist(), s["kv_len"].tolist(), s["parents"].tolist()
    Hq, Hk, d, page = case["Hq"], case["Hk"], case["d"], case["page"]
    G, T, words = Hq // Hk, s["T"], (s["max_q"] + 31) // 32
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    masks, positions = [], []
    for b in range(case["B"]):
        t0, t1, L = cu[b], cu[b + 1], klen[b]
        n = t1 - t0
        paths = []
        for i in range(n):
            p = par[t0 + i]
            paths.append({i} | (paths[p] if p >= 0 else set()))
            value = sum(1 << j for j in paths[-1])
            masks.append([(x ^ 2 ** 31) - 2 ** 31 for x in
                          ((value >> (32 * w)) & 0xffffffff for w in range(words))])
            positions.append(L - n + len(paths[-1]) - 1)
        hidden = torch.ones(n, n, dtype=torch.bool)
        for i, path in enumerate(paths):
            hidden[i, list(path)] = False
        hidden = torch.cat([torch.zeros(n, L - n, dtype=torch.bool), hidden], 1).cuda()
        at = s["page_table"][b, :(L + page - 1) // page].long()
        for h in range(Hk):
            k = s["k_cache"][at, h].reshape(-1, d)[:L].double()
            v = s["v_cache"][at, h].reshape(-1, d)[:L].double()
            q = s["q"][t0:t1, h * G:(h + 1) * G].double().transpose(0, 1)
            x = (q @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            y = torch.logsumexp(x, -1)
            lse[t0:t1, h * G:(h + 1) * G] = y.T
            out[t0:t1, h * G:(h + 1) * G] = (torch.exp(x - y[..., None]) @ v).transpose(0, 1)
    if not case["fresh"]:
        return out, lse
    return (out, lse, torch.tensor(masks, dtype=torch.int32).cuda(),
            torch.tensor([positions], dtype=torch.int32).cuda())


def _exact_keep(case, s):
    cu, klen, table, page = s["cu_q"].tolist(), s["kv_len"].tolist(), s["page_table"].tolist(), case["page"]
    kept, count = s["kept"].tolist(), s["kept_len"].tolist()
    caches, lens = [s["k_cache"].clone(), s["v_cache"].clone()], []
    at, tokens = [], []  # slot of the pool that ends with each of these tokens
    for b in range(case["B"]):
        n = cu[b + 1] - cu[b]
        ends = kept[b][:count[b]] + list(range(count[b], n))
        for j in range(n):
            slot = klen[b] - n + j
            at.append(table[b][slot // page] * page + slot % page)
            tokens.append(cu[b] + ends[j])
        lens.append(klen[b] - n + count[b])
    at, tokens = torch.tensor(at).cuda(), torch.tensor(tokens).cuda()
    for cache, x in zip(caches, (s["k"], s["v"])):
        cache.transpose(1, 2)[at // page, at % page] = x[tokens]
    return (*caches, torch.tensor(lens, dtype=torch.int32).cuda())


def _exact_fork(case, s):
    old, lens, par = s["page_table"].tolist(), s["kv_len"].tolist(), s["parents"].tolist()
    cu, refs, page, B = s["cu_q"].tolist(), s["page_refs"].tolist(), case["page"], case["B"]
    table, total, copies = [], [], []
    for b in range(B):
        p = par[b]
        base = lens[p] if p >= 0 else 0
        keeps = p >= 0 and (p == b or (par[p] != p and p not in par[:b]))
        table.append([old[p][i] if keeps or (p >= 0 and i < base // page) else -1
                      for i in range(len(old[b]))])
        total.append(base + cu[b + 1] - cu[b])
        if p >= 0 and not keeps and base % page:
            copies.append((b, base // page, old[p][base // page], base % page))
    for rows, by in ((old, -1), (table, 1)):
        for row in rows:
            for x in row:
                if x >= 0:
                    refs[x] += by
    free = iter([x for x, r in enumerate(refs) if r == 0])
    for b in range(B):
        for i in range((total[b] + page - 1) // page):
            if table[b][i] < 0:
                table[b][i] = next(free)
                refs[table[b][i]] = 1
    caches = [s["k_cache"].clone(), s["v_cache"].clone()]
    for b, i, x, slots in copies:
        for cache in caches:
            cache[table[b][i], :, :slots] = cache[x, :, :slots]
    return (*(torch.tensor(x, dtype=torch.int32).cuda() for x in (table, total, refs)), *caches)


def _exact_cross(case, s):
    B, Hq, Hk, Nq, Nk, d = (case[x] for x in ("B", "Hq", "Hk", "Nq", "Nk", "d"))
    f64 = dict(dtype=torch.float64, device="cuda")
    outs = [torch.zeros(B, Hq, Nq, d, **f64), torch.zeros(B, Hq, Nq, **f64)]
    if case["backward"]:
        outs = [outs[0], torch.zeros(B, Hk, Nk, d, **f64), torch.zeros(B, Hk, Nk, d, **f64)]
    for b in range(B):
        n = Nk if s["kv_len"] is None else int(s["kv_len"][b])
        for h in range(Hq):
            q = s["q"][b, h].double()
            k, v = (s[x][b, h * Hk // Hq, :n].double() for x in ("k", "v"))
            x = torch.einsum("id,jd->ij", q, k) / math.sqrt(d)
            y = torch.logsumexp(x, 1)
            p = torch.exp(x - y[:, None])
            o = p @ v
            if not case["backward"]:
                outs[0][b, h], outs[1][b, h] = o, y
                continue
            g = s["do"][b, h].double()
            ds = p * (g @ v.T - (g * o).sum(1, keepdim=True)) / math.sqrt(d)
            outs[0][b, h] = ds @ k
            outs[1][b, h * Hk // Hq, :n] += ds.T @ q
            outs[2][b, h * Hk // Hq, :n] += p.T @ g
    return tuple(outs)


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "keep": _exact_keep, "fork": _exact_fork,
            "cross": _exact_cross}[case["op"]](case, s)
