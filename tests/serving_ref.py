"""Plain fp64 references of the norm and rotation, the cache append and the
paged attention, on the CPU, written from the formulas (no kernel code)."""
import math

import torch


def rope_rows(positions: int, rot: int, theta: float = 10000.0):
    """fp32 [positions, rot]: cosines, then sines."""
    rows = torch.empty(positions, rot, dtype=torch.float64)
    for i in range(rot // 2):
        ang = torch.arange(positions, dtype=torch.float64) * theta ** (-2 * i / rot)
        rows[:, i], rows[:, rot // 2 + i] = torch.cos(ang), torch.sin(ang)
    return rows.float()


def pair_of(rot, interleaved):
    """Columns (first, second) of each rotated pair."""
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(x, angles, interleaved, sign=1.0):
    """x [..., d] (fp64) turned by table rows angles [..., rot] times sign."""
    if angles is None:
        return x
    rot = angles.shape[-1]
    a, b = pair_of(rot, interleaved)
    cos, sin = angles[..., :rot // 2].double(), sign * angles[..., rot // 2:].double()
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def norm_rope(x, w, angles, eps, interleaved):
    """x [B, H, N, d] 16-bit; angles [B, 1, N, rot] or None -> fp64."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    return turn(x, angles, interleaved)


def norm_rope_bwd(dy, x, w, angles, eps, interleaved):
    """(dx, dw, size of dx's terms, size of dw's terms) in fp64."""
    g = turn(dy.double(), angles, interleaved, -1.0)
    ga = g_terms(dy, angles, interleaved)
    if w is None:
        return g, None, ga, None
    x, w = x.double(), w.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    size = r * (ga * w.abs() + n.abs() * (ga * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, (g * n).sum((0, 1, 2)), size, (ga * n.abs()).sum((0, 1, 2))


def g_terms(x, angles, interleaved):
    """|x_a cos| + |x_b sin| of each turned element: what its rounding errors
    are relative to."""
    if angles is None:
        return x.double().abs()
    rot = angles.shape[-1]
    a, b = pair_of(rot, interleaved)
    cos, sin = angles[..., :rot // 2].double().abs(), angles[..., rot // 2:].double().abs()
    x = x.double().abs()
    y = x.clone()
    y[..., a] = x[..., a] * cos + x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def append(k, v, k_cache, v_cache, table, cu, kv_len, rope, interleaved):
    """The caches after the append, in fp64, and the mask of written slots
    ([pages, page_size]).  Tokens without a valid place are skipped."""
    kc, vc = k_cache.double(), v_cache.double()
    pages, _, page, _ = kc.shape
    written = torch.zeros(pages, page, dtype=torch.bool)
    for b in range(len(kv_len)):
        for t in range(cu[b], cu[b + 1]):
            pos = kv_len[b] - cu[b + 1] + t
            if pos < 0 or pos // page >= table.shape[1]:
                continue
            p = int(table[b, pos // page])
            if p < 0 or p >= pages or (rope is not None and pos >= rope.shape[0]):
                continue
            row = None if rope is None else rope[pos]
            kc[p, :, pos % page] = turn(k[t].double(), row, interleaved)
            vc[p, :, pos % page] = v[t].double()
            written[p, pos % page] = True
    return kc, vc, written


def paged_attention(q, k_cache, v_cache, table, cu, kv_len, causal, scale):
    """o [T, Hq, d], lse [T, Hq], and what their errors are relative to: the
    weighted sizes sum_j p_j |v_j| [T, Hq, d], each row's largest scale sum_c
    |q_c k_c| [T, Hq] and largest |v| [T, Hq].  All fp64; rows without a
    sequence are NaN."""
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
        idx = torch.arange(n)
        rows = table[b, idx // page].long()
        for h in range(Hk):
            k = k_cache[rows, h, idx % page].double()
            v = v_cache[rows, h, idx % page].double()
            for g in range(G):
                at = (slice(t0, t1), h * G + g)
                x = q[at].double() @ k.T * scale
                if causal:
                    pos = torch.arange(n - (t1 - t0), n)
                    x = x.masked_fill(idx[None, :] > pos[:, None], -math.inf)
                if n == 0:
                    o[at], lse[at] = 0.0, -math.inf
                    continue
                y = torch.logsumexp(x, -1)
                p = torch.exp(x - torch.where(y == -math.inf, 0.0, y)[:, None])
                p = torch.where(x == -math.inf, torch.zeros_like(p), p)
                o[at], lse[at], size[at] = p @ v, y, p @ v.abs()
                terms[at] = (q[at].double().abs() @ k.abs().T * scale).amax(-1)
                vmax[at] = v.abs().max()
    return o, lse, size, terms, vmax
