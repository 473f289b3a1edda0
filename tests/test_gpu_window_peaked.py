"""dQ of sliding-window attention on rows whose gradient is far smaller than what Delta's rounding makes of it:
one key with nearly all of a row's weight, keys and values with a common part, repeated tokens.

dS_ij = P_ij (dP_ij - Delta_i) sums to 0 over a row. Delta' = dO . out of the bf16 output is off by r_i, and
r_i sum_j P_ij k_j then stands beside a dQ in which the same keys cancel. The bounds here are those of an
exact Delta: what is left are roundings of dS, of the correction's own weights, and of the result."""
import math

import pytest
import torch

from long_context_exact_tma_b200 import api
from window_ref import E, U, backward, forward_bounds, visible, within

pytestmark = pytest.mark.gpu


def draw(kind, S, Hq, Hkv, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (torch.randn((1, S, h, D), generator=g, device="cuda") for h in (Hq, Hkv, Hkv, Hq))
    u = torch.randn(D, generator=g, device="cuda")
    u = u / u.norm()
    if kind == "sink":  # the first token takes 0.3 to 0.999 of a row's weight
        k[:, 0] = 4 * math.sqrt(D) * u
        q += torch.linspace(1.5, 3.2, S, device="cuda").view(1, S, 1, 1) * u
    elif kind == "near":  # a key of the window does: that of the fifth token before
        q = q + 9 / math.sqrt(D) * k.roll(5, 1).repeat_interleave(Hq // Hkv, 2)
    elif kind == "common":  # keys and values with a large common part
        k += 6 * math.sqrt(D) * u
        v += 6 * math.sqrt(D) * u
        q -= (q * u).sum(-1, keepdim=True) * u
    else:  # the same token again and again
        k[:, 200:] = k[:, 200:201]
        v[:, 200:] = v[:, 200:201]
    return tuple(x.to(torch.bfloat16) for x in (q, k, v, do))


def exact_delta(q, k, v, out, lse, do, vis):
    """(dQ, its bound, the dS of the exact Delta, keys by query head), in 64 bits with the given lse."""
    D, G = q.shape[3], q.shape[2] // k.shape[2]
    kk, vv = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, kk) / math.sqrt(D)
    p = torch.exp(s - lse.transpose(1, 2).unsqueeze(-1)).masked_fill(~vis, 0.0)
    dp = torch.einsum("bihd,bjhd->bhij", do, vv)
    delta = (p * dp).sum(-1, keepdim=True)
    given = (do * out).sum(-1).transpose(1, 2).unsqueeze(-1)
    off = (delta - given).abs()
    ds, ds1 = p * (dp - delta), p * (dp - given).abs()
    # dP and Delta are fp32 sums of D products; the residue is one of n terms whose weights are good to 2^-16
    # (2^-22 of an exponential, 2^-24 |argument| < 2^-17)
    mag = torch.einsum("bihd,bjhd->bhij", do.abs(), vv.abs()) + (do * out).abs().sum(-1).transpose(1, 2).unsqueeze(-1)
    n = vis.sum(-1).view(1, 1, -1, 1)
    eps = p * (2.0 ** -24 * D * (mag + (p * mag).sum(-1, keepdim=True)) +
               (2.0 ** -24 * n + 2.0 ** -16) * ds1.sum(-1, keepdim=True))
    tol = (U + E) * (ds1 + p * off) + eps
    dq = torch.einsum("bhij,bjhd->bihd", ds, kk) / math.sqrt(D)
    tq = torch.einsum("bhij,bjhd->bihd", tol, kk.abs()) / math.sqrt(D) * (1 + U) + U * dq.abs() + 1e-30
    return dq, tq, ds, kk


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("W,ns", [(600, 4), (100, 0), (30, 40)])
@pytest.mark.parametrize("kind", ["sink", "near", "common", "same"])
def test_dq_has_the_exact_delta(kind, W, ns, D, cuda):
    S, Hq, Hkv = 900, 4, 2
    q, k, v, do = draw(kind, S, Hq, Hkv, D, seed=S + W)
    vis = visible(S, W, ns, device="cuda")
    out, lse = api.window_attn_fwd(q, k, v, W, ns, check_status=True)
    qd, kd, vd, dd = (x.double() for x in (q, k, v, do))
    o, L, to, tl = forward_bounds(qd, kd, vd, vis)
    assert within(out, o, to) <= 1 and within(lse, L, tl) <= 1
    dq, dk, dv = api.window_attn_bwd(q, k, v, out, lse, do, W, ns, check_status=True)
    want, tol, ds, kk = exact_delta(qd, kd, vd, out.double(), lse.double(), dd, vis)
    assert within(dq, want, tol) <= 1
    (_, wk, wv), (_, tk, tv) = backward(qd, kd, vd, out.double(), lse.double(), dd, vis)
    assert within(dk, wk, tk) <= 1 and within(dv, wv, tv) <= 1
    if kind != "same":
        # The sum of all errors, against that of the same roundings made in 64 bits: dS rounded, the result
        # rounded. The correction's weights, rounded alike, and r_i P_ij within the rounded dS are 2^-8 of
        # those; twice as much would be another error.
        sim = (torch.einsum("bhij,bjhd->bihd", ds.to(torch.bfloat16).double(), kk) / math.sqrt(D)).to(torch.bfloat16)
        assert (dq.double() - want).norm() <= 2 * (sim.double() - want).norm()
