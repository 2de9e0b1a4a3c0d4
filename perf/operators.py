"""Timing cases of the serving and training operators around the attention
kernels: attention over a paged key/value cache, appending to that cache, and
the per-head norm with position rotation of queries and keys (forward and
backward).

Each case names one operator and its sizes.  ``run`` makes one pass, either in
plain torch operations in 32 bits (``own`` false) or through the library's
entry points (``own`` true); ``exact`` gives the result in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One new token for each of a few short conversations: latency.
        dict(name="attn_decode_few", op="attn", B=4, Hq=32, Hk=8, d=128, dtype="bf16",
             q_lo=1, q_hi=1, k_lo=150, k_hi=1100, page=16, causal=True),
        # One new token for each of many long conversations (up to 32K keys).
        dict(name="attn_decode_long", op="attn", B=16, Hq=32, Hk=8, d=128, dtype="bf16",
             q_lo=1, q_hi=1, k_lo=16000, k_hi=32768, page=64, causal=True),
        # Ragged batch of single tokens, drafted tokens and short chunks, one
        # key head per query head, fp16.
        dict(name="attn_mixed_d64", op="attn", B=24, Hq=16, Hk=16, d=64, dtype="fp16",
             q_lo=1, q_hi=333, k_lo=1, k_hi=4096, page=32, causal=True),
        # A chunk of new tokens against a 16K-key cache (chunked prefill).
        dict(name="attn_chunk_16k", op="attn", B=2, Hq=32, Hk=8, d=128, dtype="bf16",
             q_lo=1900, q_hi=2048, k_lo=16000, k_hi=16384, page=128, causal=True),
        # The decode step's append: one token a sequence.
        dict(name="append_decode", op="append", B=64, Hq=0, Hk=8, d=128, dtype="bf16",
             q_lo=1, q_hi=1, k_lo=1, k_hi=2048, page=16, rot=128, interleaved=False),
        # The prompt's append, ragged prompts of up to 4096 tokens.
        dict(name="append_prompts", op="append", B=24, Hq=0, Hk=8, d=128, dtype="bf16",
             q_lo=500, q_hi=4096, k_lo=500, k_hi=5000, page=64, rot=128, interleaved=False),
        # Drafts and short chunks, partial rotation of neighbouring pairs.
        dict(name="append_chunks_d64", op="append", B=33, Hq=0, Hk=16, d=64, dtype="fp16",
             q_lo=1, q_hi=257, k_lo=1, k_hi=3000, page=32, rot=32, interleaved=True),
        # Norm and rotation of a decode step's queries and keys.
        dict(name="norm_rope_decode", op="norm", B=1, N=16, Hq=32, Hk=8, d=128, dtype="bf16",
             rot=128, interleaved=False, backward=False),
        # The same for a training batch, 16 heads, 4096 tokens.
        dict(name="norm_rope_train", op="norm", B=4, N=4096, Hq=16, Hk=16, d=128, dtype="bf16",
             rot=128, interleaved=False, backward=False),
        # Gradients for one odd-length sequence, grouped heads, fp16, d = 64.
        dict(name="norm_rope_bwd_odd", op="norm", B=1, N=1021, Hq=24, Hk=6, d=64, dtype="fp16",
             rot=64, interleaved=True, backward=True),
        # Gradients for the training batch, and for the same tokens with
        # grouped heads and a partial rotation.
        dict(name="norm_rope_bwd_train", op="norm", B=4, N=4096, Hq=16, Hk=16, d=128,
             dtype="bf16", rot=128, interleaved=False, backward=True),
        dict(name="norm_rope_bwd_grouped", op="norm", B=3, N=4096, Hq=32, Hk=4, d=96,
             dtype="bf16", rot=64, interleaved=False, backward=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "norm", "norm"])
    d = rng.choice([64, 64, 96, 128, 128])
    case = dict(op=op, d=d, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "norm":
        case.update(B=rng.randint(1, 4), N=_log_int(rng, 1, 4096), Hk=rng.choice([1, 2, 4, 5, 8]),
                    rot=16 * rng.randint(0, d // 16), interleaved=rng.random() < 0.4,
                    backward=rng.random() < 0.5)
        case["Hq"] = case["Hk"] * min(rng.choice([1, 2, 3, 4]), 32 // case["Hk"] - 1)
        return case
    case.update(Hk=rng.choice([1, 2, 4, 5, 8]), page=rng.choice([16, 32, 64, 128, 256]))
    if op == "append":
        hi = _log_int(rng, 1, 2048)
        case.update(B=_log_int(rng, 1, 28), Hq=0, q_lo=rng.randint(1, hi), q_hi=hi, k_lo=1,
                    k_hi=_log_int(rng, hi, 4096), rot=16 * rng.randint(0, d // 16),
                    interleaved=rng.random() < 0.4)
        return case
    group = rng.choice([1, 2, 3, 4, 7, 8])
    case.update(Hq=case["Hk"] * group, causal=rng.random() < 0.85)
    kind = rng.choice(["decode", "draft", "mixed", "chunk"])
    if kind == "decode":
        hi = _log_int(rng, 2, 24000)
        case.update(B=_log_int(rng, 1, 16), q_lo=1, q_hi=1, k_lo=rng.randint(1, hi), k_hi=hi)
    elif kind == "draft":
        hi = _log_int(rng, 16, 12000)
        case.update(B=_log_int(rng, 1, 16), q_lo=2, q_hi=9, k_lo=rng.randint(9, hi), k_hi=hi)
    elif kind == "mixed":
        case.update(B=rng.randint(2, 12), q_lo=1, q_hi=rng.randint(2, 300), k_lo=1,
                    k_hi=_log_int(rng, 64, 3000))
    else:
        hi = _log_int(rng, 64, 1500)
        case.update(B=rng.randint(1, 2), q_lo=max(1, hi // 2), q_hi=hi, k_lo=1,
                    k_hi=_log_int(rng, hi, 10000))
    return case


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """New tokens and cached keys (the new ones among them) of each sequence:
    sizes of the case, not of the seed."""
    g = torch.Generator("cpu").manual_seed(case["B"] * 7919 + case["q_hi"] * 31 + case["k_hi"])
    B, q_lo, q_hi, k_lo, k_hi = (case[x] for x in ("B", "q_lo", "q_hi", "k_lo", "k_hi"))
    u = torch.rand(B, generator=g, dtype=torch.float64)
    w = torch.rand(B, generator=g, dtype=torch.float64)
    if q_lo * 16 < q_hi:  # spread over their logarithm: mostly short
        qlen = (q_lo * (q_hi / q_lo) ** u).round().long()
    else:
        qlen = q_lo + (u * (q_hi - q_lo + 1)).floor().long()
    qlen = qlen.clamp(q_lo, q_hi)
    qlen[0] = q_hi
    klen = (k_lo + (w * (k_hi - k_lo + 1)).floor().long()).clamp(k_lo, k_hi)
    klen[-1] = k_hi
    return qlen, torch.maximum(klen, qlen)


def _rope_table(positions, rot):
    """fp32 [positions, rot]: cosines, then sines, of p * 10000^(-2 i / rot)."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    d = case["d"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = dict(case=dict(case), d=d, dtype=dt)
    if case["op"] == "norm":
        B, N, Hq, Hk = (case[x] for x in ("B", "N", "Hq", "Hk"))
        # Projections of unit inputs leave each head with a spread of its own.
        s["q"] = randn(B, Hq, N, d) * 1.5
        s["k"] = randn(B, Hk, N, d) * 0.8
        s["wq"] = (1 + 0.2 * randn(d).float()).to(dt)
        s["wk"] = (1 + 0.2 * randn(d).float()).to(dt)
        s["rope"] = _rope_table(8192, case["rot"]) if case["rot"] else None
        # Decode: a position of its own for each token; training: 0..N-1.
        s["positions"] = (torch.randint(0, 8192, (B, N), generator=g, device="cuda",
                                        dtype=torch.int32) if B == 1 else None)
        if case["backward"]:
            s["dq"], s["dk"] = randn(B, Hq, N, d), randn(B, Hk, N, d)
        return s
    B, Hk, page = case["B"], case["Hk"], case["page"]
    qlen, klen = _lengths(case)
    T = int(qlen.sum())
    used = (klen + page - 1) // page
    max_pages, total = int(used.max()), int(used.sum())
    pool = total + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    first = torch.cat([torch.zeros(1, dtype=torch.long), used.cumsum(0)])[:-1].cuda()
    col = torch.arange(max_pages, device="cuda")
    at = first[:, None] + col
    s["page_table"] = torch.where(col < used.cuda()[:, None], order[at.clamp(max=pool - 1)],
                                  torch.full_like(order[:1], -1)).contiguous()
    s["cu_q"] = torch.cat([torch.zeros(1, dtype=torch.long), qlen.cumsum(0)]).int().cuda()
    s["kv_len"] = klen.int().cuda()
    s["max_q"], s["T"] = int(qlen.max()), T
    s["k_cache"] = randn(pool, Hk, page, d)
    s["v_cache"] = randn(pool, Hk, page, d)
    if case["op"] == "attn":
        s["q"] = randn(T, case["Hq"], d)
    else:
        # Keys and values as they leave one packed projection.
        kv = randn(T, 2, Hk, d)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        s["rope"] = _rope_table(8192, case["rot"]) if case["rot"] else None
    return s


# ------------------------------------------------------------------ plain forms
def _token_of(s):
    """Sequence and index in it of each of the T new tokens."""
    t = torch.arange(s["T"], device="cuda")
    cu = s["cu_q"].long()
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b]


def _rotate(x, cos, sin, rot, interleaved):
    """x [..., d] with cos, sin [..., rot / 2]: pairs (c, c + rot/2), or
    neighbouring pairs."""
    if rot == 0:
        return x
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        h = rot // 2
        a, b = x[..., :h], x[..., h:rot]
        y[..., :h], y[..., h:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _cos_sin(s, pos):
    rot = s["case"]["rot"]
    if rot == 0:
        return None, None
    row = s["rope"][pos]
    return row[..., :rot // 2], row[..., rot // 2:]


def _plain_attn(s):
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
    i, j = torch.arange(n, device="cuda"), torch.arange(L, device="cuda")
    rows = (cu[:-1, None] + i).clamp(max=T - 1)
    qp = q[rows].float().reshape(B, n, Hk, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, d)
    x = torch.matmul(qp, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    last = (klen - qlen)[:, None] + i if c["causal"] else (klen - 1)[:, None].expand(B, n)
    seen = (j <= last[:, :, None]) & (j < klen[:, None, None])
    x = x.reshape(B, Hk, G, n, L).masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = torch.exp(x - m)
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(B, Hk, G * n, L), v).reshape(B, Hk, G, n, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l))[..., 0]
    b, t = _token_of(s)
    o = o.permute(0, 3, 1, 2, 4)[b, t].reshape(T, Hq, d).to(q.dtype)
    return o, lse.permute(0, 3, 1, 2)[b, t].reshape(T, Hq).contiguous()


def _plain_append(s):
    c = s["case"]
    b, i = _token_of(s)
    cu, klen = s["cu_q"].long(), s["kv_len"].long()
    pos = klen[b] - (cu[b + 1] - cu[b]) + i
    cos, sin = _cos_sin(s, pos)
    if c["rot"]:
        cos, sin = cos[:, None], sin[:, None]
    k = _rotate(s["k"].float(), cos, sin, c["rot"], c["interleaved"]).to(s["dtype"])
    page = s["page_table"].long()[b, pos // c["page"]]
    s["k_cache"][page, :, pos % c["page"]] = k
    s["v_cache"][page, :, pos % c["page"]] = s["v"]
    return s["k_cache"], s["v_cache"]


def _norm_angles(s):
    c = s["case"]
    pos = s["positions"]
    pos = torch.arange(c["N"], device="cuda")[None] if pos is None else pos.long()
    cos, sin = _cos_sin(s, pos)
    return (None, None) if cos is None else (cos[:, None], sin[:, None])


def _plain_norm(s):
    c = s["case"]
    cos, sin = _norm_angles(s)

    def one(x, w):
        x = x.float()
        n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return _rotate(n * w.float(), cos, sin, c["rot"], c["interleaved"]).to(s["dtype"])

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _plain_norm_bwd(s):
    c = s["case"]
    cos, sin = _norm_angles(s)

    def one(dy, x, w):
        x, w = x.float(), w.float()
        g = _rotate(dy.float(), cos, None if sin is None else -sin, c["rot"], c["interleaved"])
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        dw = (g * n).sum((0, 1, 2), dtype=torch.float64).float()
        g = g * w
        return (r * (g - n * (g * n).mean(-1, keepdim=True))).to(s["dtype"]), dw

    dq, dwq = one(s["dq"], s["q"], s["wq"])
    dk, dwk = one(s["dk"], s["k"], s["wk"])
    return dq, dk, dwq, dwk


def run(state):
    s, c = state, state["case"]
    if own:
        from tiled_online_softmax_fwd_gb300 import fattn
        if c["op"] == "attn":
            return fattn.attn_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"],
                                        s["cu_q"], s["kv_len"], s["max_q"], causal=c["causal"])
        if c["op"] == "append":
            return fattn.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"],
                                   s["cu_q"], s["kv_len"], rope=s["rope"],
                                   interleaved=c["interleaved"])
        if c["backward"]:
            return fattn.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"],
                                          rope=s["rope"], positions=s["positions"], eps=EPS,
                                          interleaved=c["interleaved"])
        return fattn.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], rope=s["rope"],
                                  positions=s["positions"], eps=EPS,
                                  interleaved=c["interleaved"])
    if c["op"] == "attn":
        return _plain_attn(s)
    if c["op"] == "append":
        return _plain_append(s)
    return _plain_norm_bwd(s) if c["backward"] else _plain_norm(s)


# ------------------------------------------------------------------ floors
def work(case):
    d = case["d"]
    if case["op"] == "norm":
        rows, tokens = case["B"] * case["N"] * (case["Hq"] + case["Hk"]), case["B"] * case["N"]
        passes = 3 if case["backward"] else 2
        angles = (tokens if case["B"] == 1 else case["N"]) * case["rot"] * 4
        return {"bytes": passes * rows * d * 2 + angles + (tokens * 4 if case["B"] == 1 else 0) +
                (4 + 8 * case["backward"]) * d,
                "flops": rows * d * (14 if case["backward"] else 8)}
    qlen, klen = _lengths(case)
    tokens, B = int(qlen.sum()), case["B"]
    plan = 4 * (2 * B + 1) + 4 * int(((klen + case["page"] - 1) // case["page"]).sum())
    if case["op"] == "append":
        touched = tokens * case["Hk"] * d * 2
        return {"bytes": 4 * touched + tokens * case["rot"] * 4 + plan,
                "flops": 3 * tokens * case["Hk"] * case["rot"]}
    pairs = (qlen * klen - (qlen * (qlen - 1) // 2 if case["causal"] else 0)).sum()
    return {"bytes": 2 * int(klen.sum()) * case["Hk"] * d * 2 + 2 * tokens * case["Hq"] * d * 2 +
            tokens * case["Hq"] * 4 + plan,
            "flops": 4 * d * case["Hq"] * int(pairs)}


# ------------------------------------------------------------------ 64 bits
def _exact_turn(x, table, rot, interleaved, sign):
    """x [rows, H, d] in 64 bits, each row's pairs turned by its angle (the
    table's cosines and sines are inputs) times sign, as complex products."""
    if rot == 0:
        return x
    z = torch.complex(table[:, :rot // 2].double(), sign * table[:, rot // 2:].double())[:, None]
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        pairs = torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous()) * z
        turned = torch.stack([pairs.real, pairs.imag], -1).flatten(-2)
    else:
        re, im = head.split(rot // 2, -1)
        pairs = torch.complex(re.contiguous(), im.contiguous()) * z
        turned = torch.cat([pairs.real, pairs.imag], -1)
    return torch.cat([turned, rest], -1)


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "norm":
        B, N, rot = case["B"], case["N"], case["rot"]
        pos = (torch.arange(N, device="cuda").repeat(B) if s["positions"] is None
               else s["positions"].reshape(-1).long())
        table = s["rope"][pos] if rot else None

        def rows(t):  # [B, H, N, d] -> [B N, H, d]
            return t.transpose(1, 2).reshape(B * N, t.shape[1], d).double()

        def back(t):
            return t.reshape(B, N, t.shape[1], d).transpose(1, 2).contiguous()

        outs, sums = [], []
        for name in ("q", "k"):
            x, w = rows(s[name]), s["w" + name].double()
            norm = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
            if not case["backward"]:
                outs.append(back(_exact_turn(x / norm * w, table, rot, case["interleaved"], 1.0)))
                continue
            g = _exact_turn(rows(s["d" + name]), table, rot, case["interleaved"], -1.0)
            sums.append((g * x / norm).sum((0, 1)))
            u = g * w
            outs.append(back(u / norm - x * (u * x).sum(-1, keepdim=True) / (d * norm ** 3)))
        return tuple(outs + sums)
    cu, klen, table = s["cu_q"].tolist(), s["kv_len"].tolist(), s["page_table"].tolist()
    Hk, page = case["Hk"], case["page"]
    if case["op"] == "append":
        k_out, v_out = s["k_cache"].double(), s["v_cache"].double()
        for b in range(case["B"]):
            t0, t1 = cu[b], cu[b + 1]
            first = klen[b] - (t1 - t0)
            angles = s["rope"][first:klen[b]] if case["rot"] else None
            k = _exact_turn(s["k"][t0:t1].double(), angles, case["rot"], case["interleaved"], 1.0)
            at = first
            while at < klen[b]:
                end = min(klen[b], (at // page + 1) * page)
                dst = (table[b][at // page], slice(None), slice(at % page, at % page + end - at))
                k_out[dst] = k[at - first:end - first].transpose(0, 1)
                v_out[dst] = s["v"][t0 + at - first:t0 + end - first].transpose(0, 1).double()
                at = end
        return k_out, v_out
    T, Hq = s["T"], case["Hq"]
    G = Hq // Hk
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        t0, t1, n = cu[b], cu[b + 1], klen[b]
        pages = s["page_table"][b, :(n + page - 1) // page].long()
        for h in range(Hk):
            k = s["k_cache"][pages, h].reshape(-1, d)[:n].double()
            v = s["v_cache"][pages, h].reshape(-1, d)[:n].double()
            q = s["q"][t0:t1, h * G:(h + 1) * G].double().transpose(0, 1)  # [G, rows, d]
            x = q @ k.T / math.sqrt(d)
            if case["causal"]:
                rows = torch.arange(n - (t1 - t0), n, device="cuda")[:, None]
                x = torch.where(torch.arange(n, device="cuda") > rows, -math.inf, x)
            y = torch.logsumexp(x, -1)
            lse[t0:t1, h * G:(h + 1) * G] = y.T
            out[t0:t1, h * G:(h + 1) * G] = (torch.exp(x - y[..., None]) @ v).transpose(0, 1)
    return out, lse
