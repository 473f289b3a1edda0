"""Plain 64-bit forms of sliding-window attention with sinks and of rotary positions, and the error
bounds of the kernels' roundings against them.

One rounding to bf16 is off by at most U = 2^-8 relative. The attention kernels round P and dS to bf16
(operands of the matrix products) and every result once; sums, exponentials' arguments, LSE and Delta
are fp32, whose part is covered by E (exponentials good to 7.5e-5 relative, sums of at most a few
thousand terms): the bounds below follow term by term.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8
E = 4e-4  # fp32 arithmetic of a weight: exp2 7.5e-5, its argument (|s| < 64) * 2^-22, sums of <= 4096 terms


def visible(S, W, ns, cu=None, device="cpu"):
    """[S, S] truth values: row i sees key j."""
    i, j = torch.arange(S, device=device).unsqueeze(1), torch.arange(S, device=device)
    lo = torch.zeros(S, dtype=torch.long, device=device)
    for a, b in zip(cu[:-1], cu[1:]) if cu is not None else []:
        lo[a:b] = a
    lo = lo.unsqueeze(1)
    return (j <= i) & (j >= lo) & ((i - j < W) | (j - lo < ns))


def attend(q, k, v, vis):
    """[B, S, H, D] in 64 bits -> (out, lse, P [B, Hq, S, S])."""
    G = q.shape[2] // k.shape[2]
    kk, vv = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, kk) / math.sqrt(q.shape[3])
    s = s.masked_fill(~vis, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse).unsqueeze(-1))
    return torch.einsum("bhij,bjhd->bihd", p, vv), lse.transpose(1, 2), p


def forward_bounds(q, k, v, vis):
    """(out, lse, bound of out, bound of lse). out: the weights' roundings move the weighted mean by at
    most U sum_j p_j |v_j - out| <= U (A + |out|), A = sum_j p_j |v_j|; the result is rounded once more."""
    out, lse, p = attend(q, k, v, vis)
    G = q.shape[2] // k.shape[2]
    A = torch.einsum("bhij,bjhd->bihd", p, v.abs().repeat_interleave(G, 2))
    # scores: D products summed in fp32, each partial sum off by 2^-24 of what it holds at most
    M = torch.einsum("bihd,bjhd->bhij", q.abs(), k.abs().repeat_interleave(G, 2)).amax(-1).transpose(1, 2)
    D, n = q.shape[3], vis.sum(-1).max().item()
    lse_tol = 2.0 ** -24 * (D * M / math.sqrt(D) + 2 * n + 64)
    return out, lse, (U * (1 + U) + E) * (A + out.abs()) + U * out.abs() + 1e-30, lse_tol


FEW = 48  # rows of fewer keys have their dQ corrected for the rounding of out in Delta


def backward(q, k, v, out, lse, do, vis):
    """The gradients with the given lse in 64 bits, (dq, dk, dv), and their bounds. Delta is the exact
    sum_j P dP: the kernel corrects dO . out by the residue of its row, for dK and dV always, for dQ where
    a row has fewer than FEW keys; elsewhere dQ may be off by |Delta - dO . out| |sum_j P k_j|."""
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    kk, vv = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, kk) / math.sqrt(D)
    p = torch.exp(s - lse.transpose(1, 2).unsqueeze(-1)).masked_fill(~vis, 0.0)
    dp = torch.einsum("bihd,bjhd->bhij", do, vv)
    delta = (p * dp).sum(-1, keepdim=True)
    given = (do * out).sum(-1).transpose(1, 2).unsqueeze(-1)
    off = (delta - given).abs()
    ds = p * (dp - delta)
    # dP, Delta and the residue are fp32 sums of D products each
    mag = torch.einsum("bihd,bjhd->bhij", do.abs(), vv.abs()) + (do * out).abs().sum(-1).transpose(1, 2).unsqueeze(-1)
    eps = 2.0 ** -24 * D * p * (mag + (p * mag).sum(-1, keepdim=True))
    ds_tol = (U + E) * ds.abs() + eps
    # dQ takes dS of the given Delta, rounded, then the correction, rounded
    dq_tol = (U + E) * (p * (dp - given).abs() + p * off) + eps
    sc = 1 / math.sqrt(D)

    def group(x):
        return x.view(B, S, Hkv, G, D).sum(3)

    dq = torch.einsum("bhij,bjhd->bihd", ds, kk) * sc
    dk = group(torch.einsum("bhij,bihd->bjhd", ds, q)) * sc
    dv = group(torch.einsum("bhij,bihd->bjhd", p, do))
    left = torch.einsum("bhij,bjhd->bihd", off * p, kk).abs() * sc * (vis.sum(-1) >= FEW).view(1, S, 1, 1)
    tq = (torch.einsum("bhij,bjhd->bihd", dq_tol, kk.abs()) * sc + left) * (1 + U) + U * dq.abs()
    tk = group(torch.einsum("bhij,bihd->bjhd", ds_tol, q.abs())) * sc * (1 + U) + U * dk.abs()
    tv = group(torch.einsum("bhij,bihd->bjhd", p, do.abs())) * (U + E) * (1 + U) + U * dv.abs()
    return (dq, dk, dv), (tq + 1e-30, tk + 1e-30, tv + 1e-30)


def within(got, want, tol):
    """The largest error as a share of its bound (at most 1 when inside)."""
    d = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all()
    return float((d / tol).max()) if d.numel() else 0.0


def rotate(x, positions, inv_freq, axis, paired, inverse):
    """Pairs as complex numbers times exp(i angle), in 64 bits."""
    R = 2 * inv_freq.numel()
    a = positions.double()[axis.long().to(positions.device)].permute(1, 2, 0) * inv_freq.to(positions.device)
    w = torch.polar(torch.ones_like(a), -a if inverse else a).unsqueeze(2)
    y = x.double().clone()
    re, im = (slice(0, R, 2), slice(1, R, 2)) if paired else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(x[..., re].double().contiguous(), x[..., im].double().contiguous()) * w
    y[..., re], y[..., im] = z.real, z.imag
    return y
