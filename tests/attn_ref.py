"""Plain fp64 forms of the softmax-attention layer's operators, for the tests: the formulas of
include/gdn.h written out on CPU tensors, with the error bounds that the GPU's roundings allow.

Bounds.  A rounding to bf16 is off by at most half a step, U = 2^-8 of the value.  The kernels round,
besides their results, the weights p of a softmax (before the product with v) and the gradients ds of the
scores (before the products with q and k).  Everything else is fp32: sums of at most a few thousand terms,
whose error stays below F = 1e-4 of the sum of the terms' magnitudes (2^-24 a term, 2^-24 * 1700 terms).
"""
import torch

U = 2.0 ** -8
F = 1e-4


def f64(t):
    return t.detach().cpu().double()


# ---- norm and rotation -----------------------------------------------------------------------------
def norm_rope(x, w, pos, freq, eps=1e-6, interleaved=False, rot_scale=1.0):
    """x [T, H, d] fp64; w [d] or None; pos [T] integers or None; freq [rot / 2] or None."""
    n = x
    if w is not None:
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    if freq is None:
        return n
    h = freq.numel()
    a = pos.double()[:, None, None] * freq.double()
    c, s = rot_scale * torch.cos(a), rot_scale * torch.sin(a)
    y = n.clone()
    i, j = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    y[..., i] = n[..., i] * c - n[..., j] * s
    y[..., j] = n[..., j] * c + n[..., i] * s
    return y


def norm_rope_grad(x, w, pos, freq, g, eps=1e-6, interleaved=False, rot_scale=1.0):
    """(dx, dw or None) by the reverse formula."""
    gn = g.clone()
    if freq is not None:
        h = freq.numel()
        a = pos.double()[:, None, None] * freq.double()
        c, s = rot_scale * torch.cos(a), rot_scale * torch.sin(a)
        i, j = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
        gn[..., i] = g[..., i] * c + g[..., j] * s
        gn[..., j] = g[..., j] * c - g[..., i] * s
    if w is None:
        return gn, None
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dw = (gn * x * r).sum((0, 1))
    gw = gn * w
    return r * (gw - x * r * r * (gw * x).mean(-1, keepdim=True)), dw


# ---- attention ---------------------------------------------------------------------------------------
def visible(n, window):
    """[n, n] mask of a causal sequence."""
    i = torch.arange(n)
    see = i[None, :] <= i[:, None]
    if window:
        see &= i[None, :] > i[:, None] - window
    return see


def attend(q, k, v, see, scale):
    """One head: q [n, d], k and v [m, d], see [n, m].  Returns (o, bound, p); rows that see nothing are 0."""
    s = torch.where(see, scale * (q @ k.T), torch.tensor(-float("inf"), dtype=torch.float64))
    mx = s.amax(-1, keepdim=True)
    e = torch.where(see, torch.exp(s - torch.where(torch.isinf(mx), torch.zeros_like(mx), mx)), torch.zeros_like(s))
    l = e.sum(-1, keepdim=True)
    p = e / torch.where(l > 0, l, torch.ones_like(l))
    o = p @ v
    return o, (U + F) * (p @ v.abs()) + U * o.abs(), p


def attend_grad(q, k, v, see, scale, do):
    """Gradients of attend and their bounds: ((dq, dk, dv), (bq, bk, bv)) for one head."""
    o, _, p = attend(q, k, v, see, scale)
    dp = do @ v.T
    delta = (do * o).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    dq, dk, dv = scale * ds @ k, scale * ds.T @ q, p.T @ do
    # p in o off by U: delta = do . o off by U sum |do| (p |v|), and ds by p times that
    edelta = U * (do.abs() * (p @ v.abs())).sum(-1, keepdim=True)
    mag = p * ((do.abs() @ v.abs().T) + (do.abs() * (p @ v.abs())).sum(-1, keepdim=True))
    eds = U * ds.abs() + p * edelta + F * mag
    return ((dq, dk, dv),
            (scale * eds @ k.abs() + U * dq.abs(), scale * eds.T @ q.abs() + U * dk.abs(),
             (U + F) * (p.T @ do.abs()) + U * dv.abs()))


def packed(q, k, v, cu, scale, window, do=None):
    """Packed sequences, grouped heads: (o, bound) or, with do, (o, bound, grads, bounds)."""
    q, k, v = f64(q), f64(k), f64(v)
    G = q.shape[1] // k.shape[1]
    o, bo = torch.zeros_like(q), torch.zeros_like(q)
    g = [torch.zeros_like(t) for t in (q, k, v)]
    b = [torch.zeros_like(t) for t in (q, k, v)]
    for s in range(len(cu) - 1):
        r = slice(cu[s], cu[s + 1])
        if cu[s] == cu[s + 1]:
            continue
        see = visible(cu[s + 1] - cu[s], window)
        for h in range(q.shape[1]):
            o[r, h], bo[r, h], _ = attend(q[r, h], k[r, h // G], v[r, h // G], see, scale)
            if do is not None:
                gs, bs = attend_grad(q[r, h], k[r, h // G], v[r, h // G], see, scale, f64(do)[r, h])
                for t, (x, y) in enumerate(zip(gs, bs)):
                    at = h if t == 0 else h // G
                    g[t][r, at] += x
                    b[t][r, at] += y
    return (o, bo) if do is None else (o, bo, g, b)


def decode(q, kc, vc, table, ctx, scale, window):
    """One query token a sequence over a paged cache; pages out of range are left out."""
    q, kc, vc = f64(q), f64(kc), f64(vc)
    N, Hq, d = q.shape
    pages, page, Hk, _ = kc.shape
    G = Hq // Hk
    o, b = torch.zeros_like(q), torch.zeros_like(q)
    for n in range(N):
        m = min(max(int(ctx[n]), 0), table.shape[1] * page)
        pos = [p for p in range(max(0, m - window) if window else 0, m) if 0 <= int(table[n, p // page]) < pages]
        if not pos:
            continue
        at = torch.tensor([int(table[n, p // page]) * page + p % page for p in pos])
        k, v = kc.view(-1, Hk, d)[at], vc.view(-1, Hk, d)[at]
        see = torch.ones(1, len(pos), dtype=torch.bool)
        for h in range(Hq):
            o[n, h], b[n, h], _ = (t[0] for t in attend(q[n, h:h + 1], k[:, h // G], v[:, h // G], see, scale))
    return o, b


def within(got, ref, bound, name=""):
    got = f64(got)
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    over = ((got - ref).abs() - bound).max().item() if got.numel() else 0.0
    worst = ((got - ref).abs() / (bound + 1e-30)).max().item() if got.numel() else 0.0
    assert over <= 1e-30, f"{name}: error up to {worst:.3f} of its bound"
    return worst
