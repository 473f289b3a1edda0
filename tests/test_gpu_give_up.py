"""Attention kernels whose bounded waits run out: the call ends, reports it in the workspace, frees what it
holds, and the next call over the same workspace is right."""
import contextlib

import pytest
import torch

from long_context_exact_tma_b200 import api
from long_context_exact_tma_b200 import binding as B_

pytestmark = pytest.mark.gpu

LIMIT = 2_000_000_000  # the library's own


@contextlib.contextmanager
def wait_limit(ns):
    B_.usp_set_wait_limit_ns(ns)
    try:
        yield
    finally:
        B_.usp_set_wait_limit_ns(LIMIT)


def normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def give_up(call, ws, sites):
    """Whether a call with no patience at all gave up, at one of these kernels' waits."""
    with wait_limit(0):
        call()
    rc, site = B_.usp_workspace_status(ws)
    assert rc in (B_.USP_OK, B_.USP_ERR_TIMEOUT)
    assert rc == B_.USP_OK or site >> 8 in sites, hex(site)
    return rc != B_.USP_OK


CASES = [
    (200, 2, 90),      # the producers' copies are all on their way before anyone waits for one
    (1300, 4, 300),    # an item a CTA, of several tiles
    (4100, 16, 700),   # several items a CTA: the producers wait for the tiles, and the item, before
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,Hq,W", CASES)
def test_window_attention_gives_up_and_goes_on(S, Hq, W, D, cuda):
    B, Hkv, ns = 1, Hq // 2, 40
    q, k, v, do = normal(1, B, S, Hq, D), normal(2, B, S, Hkv, D), normal(3, B, S, Hkv, D), normal(4, B, S, Hq, D)
    ws = torch.empty(B_.usp_window_workspace_size(B, S, Hq, Hkv, D, W, ns, 0, True), dtype=torch.uint8, device="cuda")
    out, lse = api.window_attn_fwd(q, k, v, W, ns, ws=ws, check_status=True)
    grads = api.window_attn_bwd(q, k, v, out, lse, do, W, ns, ws=ws, check_status=True)
    gave_up = [0, 0]
    for _ in range(20):
        gave_up[0] += give_up(lambda: api.window_attn_fwd(q, k, v, W, ns, ws=ws), ws, (0x4,))
        o, l = api.window_attn_fwd(q, k, v, W, ns, ws=ws, check_status=True)
        assert torch.equal(o, out) and torch.equal(l, lse)
        gave_up[1] += give_up(lambda: api.window_attn_bwd(q, k, v, out, lse, do, W, ns, ws=ws), ws, (0x5, 0x6))
        got = api.window_attn_bwd(q, k, v, out, lse, do, W, ns, ws=ws, check_status=True)
        assert all(torch.equal(x, y) for x, y in zip(got, grads))
    if S == 4100:  # (the forward's waits at D = 64 may all end while they are first looked at)
        assert gave_up[1] > 0 and (gave_up[0] > 0 or D == 64), gave_up


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,Hq,P_u,P_r,docs", [
    (256, 2, 1, 2, None),
    (2048, 8, 2, 2, None),
    (2048, 8, 2, 2, [0, 300, 301, 1500, 2048]),   # query tiles without a key tile among the masked walks
])
def test_mesh_attention_gives_up_and_goes_on(S, Hq, P_u, P_r, docs, D, cuda):
    B, Hkv = 1, Hq // 2
    q, do = (normal(s, P_r, P_u, B, S // P_r, Hq // P_u, D) for s in (1, 4))
    k, v = (normal(s, P_r, P_u, B, S // P_r, Hkv // P_u, D) for s in (2, 3))
    ws = api.workspace(max(B_.usp_attn_workspace_size(B, S, Hq, Hkv, D, True, P_u, P_r, 0, x) for x in (0, 1)), cuda)
    if docs is None:
        def fwd(**kw):
            return api.attn_fwd(q, k, v, True, P_u, P_r, ws=ws, **kw)

        def bwd(**kw):
            return api.attn_bwd(q, k, v, out, lse, do, True, P_u, P_r, ws=ws, **kw)
    else:
        cu = torch.tensor(docs, dtype=torch.int32, device="cuda")

        def fwd(**kw):
            return api.attn_fwd_masked(q, k, v, True, P_u, P_r, cu_seqlens=cu, ws=ws, **kw)

        def bwd(**kw):
            return api.attn_bwd_masked(q, k, v, out, lse, do, True, P_u, P_r, cu_seqlens=cu, ws=ws, **kw)
    out, lse = fwd(check_status=True)
    grads = bwd(check_status=True)
    gave_up = 0
    for _ in range(20):
        gave_up += give_up(fwd, ws, (0x1,))
        o, l = fwd(check_status=True)
        assert torch.equal(o, out) and torch.equal(l, lse)
        gave_up += give_up(bwd, ws, (0x2, 0x3))
        assert all(torch.equal(x, y) for x, y in zip(bwd(check_status=True), grads))
    assert gave_up > 0 or S == 256
