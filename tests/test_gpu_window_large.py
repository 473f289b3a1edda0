"""Sliding-window attention over tensors of more than 2^31 elements: the last heads and rows against the same
rows of a problem that holds nothing else."""
import pytest
import torch

from long_context_exact_tma_b200 import api

pytestmark = pytest.mark.gpu


def draw(seed, *shape):
    # drawn in its own type: 2^31 numbers in fp32 would take another 9 GB
    return torch.empty(shape, device="cuda", dtype=torch.bfloat16).normal_(
        generator=torch.Generator(device="cuda").manual_seed(seed))


def close(a, b):
    """The same products; how work items are cut (pairs of row tiles, runs of far queries) may differ, so the fp32
    sums are added in another order and their roundings may fall to the other side: one bf16 step of the value,
    or of a sum of parts 8 times as large."""
    return ((a.double() - b.double()).abs() <= 2.0 ** -7 * b.double().abs() + 2.0 ** -7 * b.double().abs().mean() / 8).all()


def test_more_elements_than_31_bits(cuda):
    B, S, Hkv, G, D, W, ns = 1, 131149, 8, 17, 128, 100, 4
    q, do = draw(1, B, S, Hkv * G, D), draw(2, B, S, Hkv * G, D)
    k, v = draw(3, B, S, Hkv, D), draw(4, B, S, Hkv, D)
    assert q.numel() > 1 << 31
    out, lse = api.window_attn_fwd(q, k, v, W, ns, check_status=True)
    dq, dk, dv = api.window_attn_bwd(q, k, v, out, lse, do, W, ns, check_status=True)
    for g in (0, Hkv - 1):  # all query heads of a kv head, as a problem of their own
        heads, kv = slice(g * G, (g + 1) * G), slice(g, g + 1)
        qs, ds, ks, vs = (x.contiguous() for x in (q[:, :, heads], do[:, :, heads], k[:, :, kv], v[:, :, kv]))
        o, l = api.window_attn_fwd(qs, ks, vs, W, ns)
        assert close(out[:, :, heads], o) and torch.allclose(lse[:, :, heads], l, rtol=0, atol=2.0 ** -20 * 64)
        grads = api.window_attn_bwd(qs, ks, vs, out[:, :, heads].contiguous(), lse[:, :, heads].contiguous(), ds, W, ns)
        for x, y in zip((dq[:, :, heads], dk[:, :, kv], dv[:, :, kv]), grads):
            assert close(x, y)
