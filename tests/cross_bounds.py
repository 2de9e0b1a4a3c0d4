"""Bounds of the gradients of cross attention, row by row: what a computation may
be off by that rounds P and dS to the inputs' type, each at a scale of its own."""
import torch

U = 2.0 ** -24
FEW_KEYS = 16  # up to so many, D is worked out from the keys and not from o


def gradients(q, k, v, do, lens, scale, floor, values=False, p_floor=2.0 ** -25):
    """(dq, dk, dv) in fp64 and a bound of each element's error, first order.

    h is half a step of the type.  A score adds d terms, and lse is fp32: P is off
    by e = (d + 6) U sum|q k| scale + 3 U |lse| + 2^-22 relative, then rounded by h
    (fp16: and p_floor, half a step of its subnormal numbers at P's scale).  dP is
    off by (d + 2) U sum|do v|.  D is off by the same of do . o and by o's rounding,
    h |o|; with at most FEW_KEYS keys, where it is the sum of P dP, by e and dP's error
    instead, and by n U of the terms added.  dS = P (dP - D) carries these, e and its
    own rounding: h, and in fp16 `floor` times the norm of the row's do, for dk the
    largest of the key head's rows (`values`: and times the largest norm of a row of
    v), half a step of the subnormal numbers at that scale.  Sums of n terms add
    (n + 64) U of the terms' sizes, the store h of the result (fp16: and 2^-25)."""
    B, Hq, Nq, d = q.shape
    Hk, Nk = k.shape[1], k.shape[2]
    G = Hq // Hk
    half = q.dtype == torch.float16
    h = torch.finfo(q.dtype).eps / 2
    out = [torch.zeros(x.shape, dtype=torch.float64) for x in (q, k, v)]
    tol = [torch.zeros_like(x) for x in out]
    for b in range(B):
        n = Nk if lens is None else lens[b]
        if n == 0:
            continue
        for hq in range(Hq):
            hk = hq // G
            qq, g = q[b, hq].double(), do[b, hq].double()
            kk, vv = k[b, hk, :n].double(), v[b, hk, :n].double()
            x = qq @ kk.T * scale
            y = torch.logsumexp(x, -1, keepdim=True)
            p = torch.exp(x - y)
            dp = g @ vv.T
            D = (p * dp).sum(-1, keepdim=True)
            ds = p * (dp - D)
            out[0][b, hq] = ds @ kk * scale
            out[1][b, hk, :n] += ds.T @ qq * scale
            out[2][b, hk, :n] += p.T @ g
            e = (d + 6) * U * (qq.abs() @ kk.abs().T * scale) + 3 * U * y.abs() + 2.0 ** -22
            p_err = p * (e + h) + (p_floor if half else 0.0)
            dp_err = (d + 2) * U * (g.abs() @ vv.abs().T)
            if n <= FEW_KEYS:
                d_err = (p * (e * dp.abs() + dp_err)).sum(-1, keepdim=True) + \
                    (n + 2) * U * (p * dp.abs()).sum(-1, keepdim=True)
            else:
                o = p @ vv
                d_err = h * (g * o).abs().sum(-1, keepdim=True) + (d + 2) * U * (g * o).abs().sum(-1, keepdim=True)
            s_err = ds.abs() * (e + h + 4 * U) + p * (d_err + dp_err) * (1 + h)
            size = floor * (vv.norm(dim=-1).max() if values else 1.0) if half else 0.0
            row = size * g.norm(dim=-1, keepdim=True)
            head = size * do[b, hk * G:hk * G + G].double().norm(dim=-1).max()
            tol[0][b, hq] = scale * ((s_err + row) @ kk.abs() + (n + 64) * U * (ds.abs() @ kk.abs()))
            m = G * Nq + 64
            tol[1][b, hk, :n] += scale * ((s_err + head).T @ qq.abs() + m * U * (ds.abs().T @ qq.abs()))
            tol[2][b, hk, :n] += p_err.T @ g.abs() + m * U * (p.T @ g.abs())
    return out, [t * (1 + h) + h * x.abs() + (2.0 ** -25 if half else 0.0) for t, x in zip(tol, out)]


def within(got, want, tol, what=""):
    for name, g, w, t in zip(("dq", "dk", "dv"), got, want, tol):
        g = g.double().cpu()
        assert bool(torch.isfinite(g).all()), "%s %s" % (what, name)
        err = (g - w).abs()
        bad = err > t * (1 + 1e-9)
        assert not bool(bad.any()), "%s %s: %d of %d beyond the bound, worst ratio %.3g" % (
            what, name, int(bad.sum()), bad.numel(), float((err / t.clamp(min=1e-300)).max()))
