"""64-bit references of the operators around the routing, with bounds on what
their kernels may be off by.

A sum of squares or of products along a row is made of at most 32 fused
additions in a thread, 5 between lanes and 31 between warps, each off by 2^-24 of
what is added up: below 70 * 2^-24, less than ROW = 2^-17.
"""
from __future__ import annotations

import torch

ROW = 2.0 ** -17


def half_step(t):
    """A rounding to type t is off by at most this, relative to the value."""
    return torch.finfo(t).eps / 2


def inside(got, want, tol, normal=2.0 ** -126):
    """got within tol of want, and its own rounding; infinities and NaN in the same places."""
    g, w = got.double(), want.double()
    fine = torch.isfinite(w)
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    assert torch.equal(g[~fine & ~torch.isnan(w)], w[~fine & ~torch.isnan(w)])
    tol = torch.as_tensor(tol, dtype=torch.float64, device=g.device).expand_as(w)[fine]
    off = (g[fine] - w[fine]).abs() - (tol + half_step(got.dtype) * (w[fine].abs() + tol) + normal)
    bad = ~(off <= 0)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst by {off.max().item():.3g}"


def norm64(x, w, residual, eps):
    """-> (h in its type, y in 64 bits)."""
    h = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    d = h.double()
    y = d * torch.rsqrt(d.square().mean(1, keepdim=True) + eps)
    return h, y if w is None else y * w.double()


def norm_backward64(dy, h, w, dres, eps):
    """-> (dh, its bound, dw, its bound), 64 bits."""
    d, g0 = h.double(), dy.double()
    rs = torch.rsqrt(d.square().mean(1, keepdim=True) + eps)
    n, g = d * rs, g0 if w is None else g0 * w.double()
    mean = (g * n).mean(1, keepdim=True)
    dh = rs * (g - n * mean)
    # rs and the mean are each off by a row's sum, and what follows by a few operations
    tol = 4 * ROW * rs * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dres is not None:
        dh = dh + dres.double()
        tol = tol + 2.0 ** -23 * (dres.double().abs() + dh.abs())
    # a block adds every 152nd row at most, and a column's sum then goes through at most 76 parts (a 16th of 8 * 152) and 15
    # runs of them: each of these additions is off by 2^-24 of what is added up
    dw, T = (g0 * n).sum(0), h.shape[0]
    return dh, tol, dw, (2 * ROW + (T / 152 + 92) * 2.0 ** -24) * (g0 * n).abs().sum(0)


def scores64(l, scoring):
    l = l.double()
    bad = torch.isnan(l)
    if scoring == "sigmoid":
        return torch.where(bad, 0.0, torch.sigmoid(l))
    v = l.masked_fill(bad, -torch.inf)
    mx = v.amax(1, keepdim=True)
    p = torch.where(v == mx, 1.0, torch.exp(v - mx))   # also of infinities
    p = torch.where(bad, 0.0, p)
    return p / p.sum(1, keepdim=True)


def select64(logits, K, *, scoring="softmax", bias=None, num_groups=1, topk_groups=1, group_score="max",
             renormalize=True, scale=1.0):
    """-> (idx, weights in 64 bits), experts one at a time as the definition says."""
    T, E = logits.shape
    l, p = logits.double(), scores64(logits, scoring)
    key = l if bias is None else p + bias.double()
    key = torch.where(torch.isnan(l) | torch.isnan(key), -torch.inf, key)
    if num_groups > 1:
        of = torch.where(key == -torch.inf, -torch.inf, p if bias is None and group_score == "top2" else key)
        of = of.view(T, num_groups, -1)
        best = of.sort(2, descending=True).values
        mark = best[..., 0]
        if group_score == "top2" and of.shape[2] > 1:
            mark = mark + torch.where(best[..., 1] == -torch.inf, 0.0, best[..., 1])
        place = mark.sort(dim=1, descending=True, stable=True).indices.argsort(1)
        key = key.masked_fill((place >= topk_groups).repeat_interleave(E // num_groups, 1), -torch.inf)
    top = key.sort(dim=1, descending=True, stable=True)
    idx, there = top.indices[:, :K], top.values[:, :K] > -torch.inf
    w = torch.where(there, p.gather(1, idx), 0.0)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(there, idx, -1), w * scale


def weights_tol(logits, w):
    """Of fp32 weights: exponentials off by twice their argument's 2^-24 and 2^-22 of themselves, a sum of at most 32
    such, and a handful of operations."""
    l = logits.float().double()
    spread = torch.nan_to_num(l, 0, 0, 0).abs().amax(1, keepdim=True)
    return (100 + 8 * spread) * 2.0 ** -24 * w.abs()


def select_backward64(logits, idx, dw, *, scoring, renormalize, scale):
    l = logits.double().detach().requires_grad_(True)
    p = torch.softmax(l, 1) if scoring == "softmax" else torch.sigmoid(l)
    there = idx >= 0
    c = torch.where(there, p.gather(1, idx.clamp(min=0)), 0.0)
    if renormalize:
        total = c.sum(1, keepdim=True)
        c = c / torch.where(total > 0, total, 1.0)
    (g,) = torch.autograd.grad((c * scale * dw.double()).sum(), l)
    # what is subtracted from one another is off by its own size
    d = (dw.double().abs() * scale * there)
    size = torch.zeros_like(g).scatter_add_(1, idx.clamp(min=0), (d + (d * c).sum(1, keepdim=True)) * there)
    pd = p.detach()
    share = pd / torch.where(there, pd.gather(1, idx.clamp(min=0)), 0.0).sum(1, keepdim=True).clamp(min=1e-300) \
        if renormalize else pd
    tol = (150 + 8 * logits.double().abs().amax(1, keepdim=True)) * 2.0 ** -24 * share * (
        size + ((d * c.detach()).sum(1, keepdim=True) if scoring == "softmax" and not renormalize else 0.0))
    # the reference's own: where the softmax's terms cancel, 64 bits leave a few 2^-53 of what cancels, at most the
    # sum of |d| over the chosen scores' sum, times the score
    total = torch.where(there, pd.gather(1, idx.clamp(min=0)), 0.0).sum(1, keepdim=True)
    tol = tol + 2.0 ** -48 * pd * d.sum(1, keepdim=True) / (torch.where(total > 0, total, 1.0) if renormalize else 1.0)
    return g.detach(), tol.detach()


def lora64(x, ids, a, b, scaling, base):
    """-> (out, bound), 64 bits."""
    M, N = x.shape[0], b.shape[1]
    out = torch.zeros((M, N), dtype=torch.float64, device=x.device) if base is None else base.double().clone()
    tol = 2.0 ** -23 * out.abs()
    for i in range(a.shape[0]):
        rows = torch.nonzero(ids == i)[:, 0]
        if rows.numel() == 0:
            continue
        s = 1.0 if scaling is None else scaling[i].double()
        xs, ai, bi = x[rows].double(), a[i].double(), b[i].double()
        v = xs @ ai.t()
        part = s * (v @ bi.t())
        # the first product's sums (8 * 2^-23 of 128 columns each and 2^-17 in all) and the second's at most 24 steps
        dv = 2.0 ** -17 * (xs.abs() @ ai.abs().t())
        tol[rows] += abs(s) * (dv @ bi.abs().t() + 2.0 ** -17 * (v.abs() @ bi.abs().t())) + 2.0 ** -23 * part.abs()
        out[rows] += part
    return out, tol
