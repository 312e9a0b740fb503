"""The drafter-training operators in 64 bits, from their definitions (CPU, torch)."""
import math

import torch

INF = math.inf


def record(x, K, T):
    """x [n, V], T [n]: (top_logits, top_index, tail_lse)."""
    x, T = x.double(), T.double()[:, None]
    v, i = torch.sort(x + 0.0, dim=1, descending=True, stable=True)
    top, idx = v[:, :K], i[:, :K]
    idx = torch.where(top == -INF, -1, idx)
    rest = v[:, K:] / T
    tail = torch.logsumexp(rest, 1) if K < x.shape[1] else torch.full((x.shape[0],), -INF, dtype=torch.double)
    return top, idx, tail


def distill(z, top, idx, tail, label, w, T, kl, tv, ce):
    """Per row: loss, parts, gradient, and `size`, the sum of the magnitudes of
    the gradient's terms (what a relative error of the weights acts on)."""
    n, V = z.shape
    loss, parts = torch.zeros(n, dtype=torch.double), torch.zeros(n, 3, dtype=torch.double)
    grad, size = torch.zeros(n, V, dtype=torch.double), torch.zeros(n, V, dtype=torch.double)
    for r in range(n):
        wr, t = float(w[r]), float(T[r])
        if wr == 0:
            continue
        lq = torch.log_softmax(z[r].double() / t, 0)
        q = lq.exp()
        keep = idx[r] >= 0
        tok, x = idx[r][keep].long(), top[r][keep].double() / t
        tl = -INF if tail is None else float(tail[r])
        lp = torch.log_softmax(torch.cat([x, torch.tensor([tl], dtype=torch.double)]), 0)
        p = lp.exp()
        inside = torch.zeros(V, dtype=torch.bool)
        inside[tok] = True
        qr = q[~inside].sum()
        qb = torch.cat([q[tok], qr[None]])
        lqb = torch.cat([lq[tok], qr.log()[None]])
        has = p > 0
        klv = (p[has] * (lp[has] - lqb[has])).sum()
        tvv = 0.5 * (p - qb).abs().sum()
        y = int(label[r])
        cev = -lq[y] if y >= 0 else torch.tensor(0.0, dtype=torch.double)
        parts[r] = torch.stack([klv, tvv, cev])
        loss[r] = wr * sum(a * b for a, b in ((kl, klv), (tv, tvv), (ce, cev)) if a != 0)
        # through the buckets and the softmax
        share = torch.where(inside, 0.0, q / qr if qr > 0 else torch.zeros_like(q))
        pv = share * p[-1]
        pv[tok] = p[:-1]
        sign = torch.sign(qb - p)
        s = sign[-1].expand(V).clone()
        s[tok] = sign[:-1]
        hot = torch.zeros(V, dtype=torch.double)
        lce = 0.0
        if y >= 0:
            hot[y] = 1.0
            lce = ce
        g = kl * (q - pv) + tv * q * (0.5 * s - 0.5 * (sign * qb).sum()) + lce * (q - hot)
        grad[r] = wr / t * g
        size[r] = abs(wr) / t * (abs(kl) * (q + pv) + abs(tv) * q + abs(lce) * (q + hot))
    return loss, parts, grad, size


def ce_forward(h, w, label):
    l = h.double() @ w.double().t()
    lse = torch.logsumexp(l, 1)
    live = label >= 0
    z = l.gather(1, label.clamp(min=0).long()[:, None])[:, 0]
    zero = torch.zeros((), dtype=torch.double)
    return torch.where(live, lse - z, zero), torch.where(live, lse, zero)


def ce_backward(h, w, label, g, delta=0.0):
    """Gradients, and how far they may be off where the logits less lse are off by
    `delta`.  G = g (p - [v = y]), and p = e^{l - lse} is off by delta p.  That is
    not a share of G: for p_y near 1, G_y = g (p_y - 1) is small while p_y's error
    is not, so |dG| <= 2^-8 |G| (one rounding to bf16) + delta |g| p.  The products
    add |dG| times the other factor's magnitude, and each output is rounded once."""
    h, w, g = h.double().clone(), w.double(), g.double()
    live = (label >= 0) & (g != 0)
    h[~live] = 0
    l = h @ w.t()
    p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True)) * torch.where(live, g, 0.0)[:, None]
    G = p.clone()
    G[torch.arange(len(g)), label.clamp(min=0).long()] -= torch.where(live, g, 0.0)
    off = 2.0 ** -8 * G.abs() + delta * p.abs()
    gh, gw = G @ w, G.t() @ h
    return (gh, gw, off @ w.abs() + 2.0 ** -8 * gh.abs() + 1e-37, off.t() @ h.abs() + 2.0 ** -8 * gw.abs() + 1e-37)
