"""Plain references, on the CPU and in fp64, of the calls around drafted trees,
forked sequences and cross attention, written from the formulas (no kernel
code)."""
import math

import torch


def paths(parents):
    """For each token of one sequence the set of itself and those it continues."""
    out = []
    for i, p in enumerate(parents):
        out.append({i} | (out[p] if p >= 0 else set()))
    return out


def pack(rows, words):
    """int32 [len(rows), words] whose bits are the members of each row's set."""
    mask = torch.zeros(len(rows), words, dtype=torch.int32)
    for r, row in enumerate(rows):
        for w in range(words):
            x = sum(1 << (j - 32 * w) for j in row if 32 * w <= j < 32 * w + 32)
            mask[r, w] = x - (1 << 32) if x >= 1 << 31 else x
    return mask


def random_tree(n, g):
    return [-1 if i == 0 or torch.rand(1, generator=g) < 0.05 else
            int(torch.randint(max(0, i - 5), i, (1,), generator=g)) for i in range(n)]


def softmax_rows(x, v):
    """(o, lse, weighted sizes) of scores x [..., n] over values v [n, d]."""
    y = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(y == -math.inf, torch.zeros_like(y), y)[..., None])
    p = torch.where(x == -math.inf, torch.zeros_like(p), p)
    return p @ v, y, p @ v.abs()


def tree_attention(q, k_cache, v_cache, table, cu, kv_len, rows, scale):
    """As serving_ref.paged_attention (o, lse and the sizes that errors are
    relative to); rows[t]: the set of its sequence's new tokens that token t
    sees."""
    T, Hq, d = q.shape
    Hk, page = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hk
    o = torch.full((T, Hq, d), math.nan, dtype=torch.float64)
    size = torch.zeros((T, Hq, d), dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    terms, vmax = torch.zeros((T, Hq), dtype=torch.float64), torch.zeros((T, Hq), dtype=torch.float64)
    for b in range(len(kv_len)):
        t0, t1, n = cu[b], cu[b + 1], kv_len[b]
        if t1 == t0:
            continue
        if n == 0:
            o[t0:t1], lse[t0:t1] = 0.0, -math.inf
            continue
        idx = torch.arange(n)
        at = table[b, idx // page].long()
        first = n - (t1 - t0)  # of the new tokens; may be negative
        hidden = torch.zeros(t1 - t0, n, dtype=torch.bool)
        for t in range(t0, t1):
            for j in range(max(first, 0), n):
                hidden[t - t0, j] = (j - first) not in rows[t]
        for h in range(Hk):
            k = k_cache[at, h, idx % page].double()
            v = v_cache[at, h, idx % page].double()
            for g in range(G):
                to = (slice(t0, t1), h * G + g)
                x = (q[to].double() @ k.T * scale).masked_fill(hidden, -math.inf)
                o[to], lse[to], size[to] = softmax_rows(x, v)
                terms[to] = (q[to].double().abs() @ k.abs().T * scale).amax(-1)
                vmax[to] = v.abs().max()
    return o, lse, size, terms, vmax


def keep(k_cache, v_cache, table, cu, kv_len, kept):
    """(k_cache, v_cache, lengths) with kept[b] the tokens that stay."""
    kc, vc, lens = k_cache.clone(), v_cache.clone(), []
    page = kc.shape[2]
    for b, n in enumerate(kv_len):
        first = n - (cu[b + 1] - cu[b])
        for j, t in enumerate(kept[b]):
            src, dst = first + t, first + j
            for c, old in ((kc, k_cache), (vc, v_cache)):
                c[table[b][dst // page], :, dst % page] = old[table[b][src // page], :, src % page]
        lens.append(first + len(kept[b]))
    return kc, vc, lens


def fork(k_cache, v_cache, table, lens, refs, parents, new):
    """(table, lens, refs, k_cache, v_cache) afterwards; lists of ints, in
    range.  A page that is not to be had is -1."""
    page, B, cols = k_cache.shape[2], len(table), len(table[0])
    kc, vc, refs = k_cache.clone(), v_cache.clone(), list(refs)
    owner = {}
    for b in range(B):
        if parents[b] >= 0 and (parents[b] == b or parents[b] not in owner):
            owner[parents[b]] = b
    for b in range(B):
        if parents[b] == b:
            owner[b] = b
    out, total, copy = [], [], []
    for b in range(B):
        p = parents[b]
        base = lens[p] if p >= 0 else 0
        mine = p >= 0 and owner[p] == b
        out.append([table[p][c] if p >= 0 and (mine or c < base // page) else -1 for c in range(cols)])
        total.append(base + new[b])
        copy.append((table[p][base // page], base % page) if p >= 0 and not mine and base % page else None)
    for row in table:
        for x in row:
            if x >= 0:
                refs[x] -= 1
    for row in out:
        for x in row:
            if x >= 0:
                refs[x] += 1
    free = [x for x, r in enumerate(refs) if r == 0]
    for b in range(B):
        for c in range((total[b] + page - 1) // page):
            if out[b][c] >= 0:
                continue
            if not free:
                continue
            x = free.pop(0)
            out[b][c], refs[x] = x, 1
            if copy[b] is not None and parents[b] >= 0 and c == lens[parents[b]] // page:
                src, slots = copy[b]
                kc[x, :, :slots], vc[x, :, :slots] = k_cache[src, :, :slots], v_cache[src, :, :slots]
    return out, total, refs, kc, vc


def cross(q, k, v, kv_len, scale):
    """(o, lse, size, terms, vmax) of [B, H, N, d] tensors, each [B, Hq, Nq, ..]."""
    B, Hq, Nq, d = q.shape
    G = Hq // k.shape[1]
    o = torch.zeros(B, Hq, Nq, d, dtype=torch.float64)
    size = torch.zeros_like(o)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64)
    terms, vmax = torch.zeros_like(lse), torch.zeros_like(lse)
    for b in range(B):
        n = k.shape[2] if kv_len is None else kv_len[b]
        if n == 0:
            terms[b] = 0
            continue
        for h in range(Hq):
            kk, vv = k[b, h // G, :n].double(), v[b, h // G, :n].double()
            x = q[b, h].double() @ kk.T * scale
            o[b, h], lse[b, h], size[b, h] = softmax_rows(x, vv)
            terms[b, h] = (q[b, h].double().abs() @ kk.abs().T * scale).amax(-1)
            vmax[b, h] = vv.abs().max()
    return o, lse, size, terms, vmax


def cross_bwd(q, k, v, do, kv_len, scale, dtype=None, o_err=None):
    """(dq, dk, dv) in fp64, and with a type the bounds of a computation that
    rounds as the library says (first order, doubled nowhere):

    h is half a step of the type, U = 2^-24.  A score adds d terms, and lse is
    fp32: P is off by e = (d + 6) U sum|q k| scale + 3 U |lse| + 2^-22 relative,
    then rounded by h (fp16: and 2^-25, below its normal numbers).  dP is off by
    (d + 2) U sum|do v|; D by the rounding of o (o_err, else h |o|) and (d + 2) U
    sum|do o|.  dS = P (dP - D) carries these, e, and its own rounding (fp16:
    scaled to where the largest |do| is at least 1, so 2^-25 of that is its
    floor).  Sums of n terms add (n + 64) U of the terms' sizes, the store h of
    the result (fp16: and 2^-25)."""
    B, Hq, Nq, d = q.shape
    Hk, Nk = k.shape[1], k.shape[2]
    G = Hq // Hk
    out = [torch.zeros(x.shape, dtype=torch.float64) for x in (q, k, v)]
    tol = [torch.zeros_like(x) for x in out]
    U = 2.0 ** -24
    h = torch.finfo(dtype).eps / 2 if dtype is not None else 0.0
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    floor = tiny * float(do.double().abs().max()) if do.numel() else 0.0
    for b in range(B):
        n = Nk if kv_len is None else kv_len[b]
        if n == 0:
            continue
        for hq in range(Hq):
            qq, g = q[b, hq].double(), do[b, hq].double()
            kk, vv = k[b, hq // G, :n].double(), v[b, hq // G, :n].double()
            x = qq @ kk.T * scale
            y = torch.logsumexp(x, -1, keepdim=True)
            p = torch.exp(x - y)
            o = p @ vv
            dp = g @ vv.T
            D = (g * o).sum(-1, keepdim=True)
            ds = p * (dp - D)
            out[0][b, hq] = ds @ kk * scale
            out[1][b, hq // G, :n] += ds.T @ qq * scale
            out[2][b, hq // G, :n] += p.T @ g
            if dtype is None:
                continue
            e = (d + 6) * U * (qq.abs() @ kk.abs().T * scale) + 3 * U * y.abs() + 2.0 ** -22
            p_err = p * (e + h) + tiny
            oe = h * o.abs() if o_err is None else o_err[b, hq]
            d_err = (g.abs() * oe).sum(-1, keepdim=True) + (d + 2) * U * (g * o).abs().sum(-1, keepdim=True)
            dp_err = (d + 2) * U * (g.abs() @ vv.abs().T)
            s_err = ds.abs() * (e + h + 4 * U) + p * (d_err + dp_err) * (1 + h) + floor
            tol[0][b, hq] = scale * (s_err @ kk.abs() + (n + 64) * U * (ds.abs() @ kk.abs()))
            m = G * Nq + 64
            tol[1][b, hq // G, :n] += scale * (s_err.T @ qq.abs() + m * U * (ds.abs().T @ qq.abs()))
            tol[2][b, hq // G, :n] += p_err.T @ g.abs() + m * U * (p.T @ g.abs())
    if dtype is None:
        return out
    return out, [t * (1 + h) + h * x.abs() + tiny for t, x in zip(tol, out)]
