"""Inputs and 64-bit references of the few-token operators' tests.

Tolerances are bounds, not fits.  A product sum of n terms is made of at most
eight matrix steps per group of 128 columns, whose fp32 accumulators may
truncate (8 * 2^-23 of the group's absolute sum), and of at most 64 fp32
additions of groups and slices (64 * 2^-24 of the whole absolute sum):
together below 2^-17 of sum |x||w|.  What follows (activation, planes of h,
weights, output rounding) is added term by term below.
"""
from __future__ import annotations

import torch

import combine_send_counts_gb300 as ep

SUM = 2.0 ** -17


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def w4_random(lead, N, K, group, zeros, g):
    q = torch.randint(0, 256, (*lead, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand((*lead, N, K // group), generator=g, device="cuda") * 0.1 + 0.01).to(torch.bfloat16)
    z = torch.randint(0, 16, s.shape, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return ep.W4(q, s, z, group)


def values64(w):
    """A weight tensor or W4 in 64 bits."""
    if isinstance(w, torch.Tensor):
        return w.double()
    lo, hi = (w.q & 15).double(), torch.div(w.q, 16, rounding_mode="floor").double()
    v = torch.stack((lo, hi), -1).reshape(*w.scale.shape, w.group)
    z = 8.0 if w.zero is None else w.zero.double()[..., None]
    return ((v - z) * w.scale.double()[..., None]).reshape(w.shape)


def moe64(x, idx, wts, w13, w2, rank=0, planes=2):
    """-> (out [T,H], bound on the error before the output's rounding), 64 bits."""
    El, I2, H = w13.shape
    I = I2 // 2
    out = torch.zeros((x.shape[0], H), dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(out)
    for e in range(El):
        toks, ks = torch.nonzero(idx == e + rank * El, as_tuple=True)
        if toks.numel() == 0:
            continue
        a, b = values64(w13[e]), values64(w2[e])
        xs = x[toks].double()
        g, u = xs @ a[:I].t(), xs @ a[I:].t()
        dg, du = SUM * (xs.abs() @ a[:I].abs().t()), SUM * (xs.abs() @ a[I:].abs().t())
        act = g * torch.sigmoid(g)
        h = act * u
        # |silu'| <= 1.1; exp, division, product and the bf16 planes of h
        dh = 1.1 * dg * u.abs() + act.abs() * du + 1.1 * dg * du + h.abs() * (2.0 ** -20 + 2.0 ** (-8 * planes))
        w = wts[toks, ks].double()[:, None]
        out.index_add_(0, toks, w * (h @ b.t()))
        tol.index_add_(0, toks, w.abs() * (dh @ b.abs().t() + (SUM + 2.0 ** -19) * (h.abs() @ b.abs().t())))
    return out, tol


def assert_close(got, want, tol):
    """got (bf16 or fp32) within tol plus its own type's rounding of want."""
    eps = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23
    # below bf16's and fp32's normal range the spacing is absolute
    off = (got.double() - want).abs() - (tol + eps * want.abs() + 2.0 ** -126)
    bad = ~(off <= 0)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside, worst by {off.max().item():.3g}, "
                           f"first at {torch.nonzero(bad)[0].tolist()}")


def routes(T, E, K, g, how="distinct"):
    if how == "distinct":
        idx = torch.rand((T, E), generator=g, device="cuda").topk(K, dim=1).indices
    elif how == "repeats":     # the same expert may stand in several slots of a token
        idx = torch.randint(0, E, (T, K), generator=g, device="cuda")
    elif how == "one":         # every slot names the same expert
        idx = torch.full((T, K), E - 1, device="cuda", dtype=torch.int64)
    elif how == "none":
        idx = torch.full((T, K), -1, device="cuda", dtype=torch.int64)
    elif how == "masked":
        idx = torch.rand((T, E), generator=g, device="cuda").topk(K, dim=1).indices
        idx[torch.rand((T, K), generator=g, device="cuda") < 0.3] = -1
        idx[0] = -1            # one token goes nowhere
    else:
        raise ValueError(how)
    return idx.contiguous(), torch.rand((T, K), generator=g, device="cuda")
