"""Rotary positions with several axes on a B200 against complex multiplication in 64 bits."""
import pytest
import torch

from long_context_exact_tma_b200 import api
from window_ref import rotate

pytestmark = pytest.mark.gpu

# The rotated pair is computed in fp32: the angle is off by at most 2^-24 turns * 2 pi / 2 + the sines'
# 2^-20 (bf16 kernel) or 2^-23 (fp32 kernel), the products by 2^-23: ERR * (|x1| + |x2|) in all; then
# one rounding of the result.
ERR = {torch.bfloat16: 2.0 ** -18, torch.float32: 2.0 ** -20}
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def check(got, x, pos, inv, axis, paired, inverse):
    want = rotate(x, pos, inv, axis, paired, inverse)
    mag = rotate(x.double().abs(), torch.zeros_like(pos), inv, axis, paired, False)
    R = 2 * inv.numel()
    both = mag[..., 0:R:2] + mag[..., 1:R:2] if paired else mag[..., :R // 2] + mag[..., R // 2:R]
    tol = want.abs() * ROUND[x.dtype]
    tol[..., :R] += ERR[x.dtype] * (both.repeat_interleave(2, -1) if paired else torch.cat([both, both], -1))
    assert ((got.double() - want).abs() <= tol).all()
    assert torch.equal(got[..., R:], x[..., R:])


def freqs(R, axes):
    f = torch.arange(R // 2, dtype=torch.float64)
    return 500000.0 ** (-2 * f / R), (f % axes).to(torch.int32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("B,S,Hq,Hkv,D,R,axes", [
    (1, 1, 1, 1, 2, 2, 1), (8, 1, 32, 8, 128, 128, 3), (2, 77, 5, 1, 64, 32, 2), (1, 300, 3, 3, 96, 20, 3),
    (1, 33, 2, 2, 65, 64, 1), (2, 1000, 16, 2, 256, 256, 3), (1, 5, 1, 1, 300, 254, 5),
])
def test_rotation(B, S, Hq, Hkv, D, R, axes, paired, dtype, cuda):
    g = torch.Generator(device="cuda").manual_seed(S)
    q = torch.randn((B, S, Hq, D), generator=g, device="cuda").to(dtype)
    k = torch.randn((B, S, Hkv, D), generator=g, device="cuda").to(dtype)
    pos = torch.randint(-5, 2 ** 30, (axes, B, S), generator=g, device="cuda")
    inv, axis = freqs(R, axes)
    for inverse in (False, True):
        for p in (pos, pos.int()):
            yq, yk = api.rope_axes((q, k), p, inv, axis, paired=paired, inverse=inverse)
            check(yq, q, pos, inv, axis, paired, inverse)
            check(yk, k, pos, inv, axis, paired, inverse)


def test_far_positions_of_64_bits(cuda):
    pos = torch.tensor([[[2 ** 40 + 12345, -2 ** 40 - 7]]], device="cuda")
    x = torch.randn((1, 2, 2, 64), device="cuda")
    f = torch.arange(32, dtype=torch.float64)
    # dyadic frequencies, so that the 64-bit reference's product is exact
    inv, axis = 2.0 ** -(f + 1), torch.zeros(32, dtype=torch.int32)
    got = api.rope_axes(x, pos, inv, axis)
    a = (pos.double()[0].unsqueeze(-1) * inv.cuda())
    c, s = torch.cos(a).unsqueeze(2), torch.sin(a).unsqueeze(2)  # argument reduction of doubles
    x1, x2 = x.double().chunk(2, -1)
    want = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)
    # inv / 2 pi is held to 2^-64 of a turn, of which the position makes 2^-24; sines and products 2^-20
    assert ((got.double() - want).abs() <= 2.0 ** -19 * (x1.abs() + x2.abs()).repeat(1, 1, 1, 2) + want.abs() * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_views_in_place_and_broadcast(dtype, cuda):
    B, S, Hq, Hkv, D, axes = 2, 50, 6, 2, 64, 3
    qkv = torch.randn((B, S, Hq + 2 * Hkv, D), device="cuda").to(dtype)
    pos = torch.randint(0, 5000, (axes, B, S), device="cuda")
    inv, axis = freqs(D, axes)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
    yq, yk = api.rope_axes((q, k), pos, inv, axis)
    check(yq, q, pos, inv, axis, False, False)
    check(yk, k, pos, inv, axis, False, False)
    # an odd element offset: rows that are not 16-byte aligned
    flat = torch.randn(B * S * Hq * D + 1, device="cuda").to(dtype)
    odd = flat[1:].view(B, S, Hq, D)
    check(api.rope_axes(odd, pos, inv, axis), odd, pos, inv, axis, False, False)
    # head-major memory
    hm = torch.randn((B, Hq, S, D), device="cuda").to(dtype).transpose(1, 2)
    check(api.rope_axes(hm, pos, inv, axis), hm, pos, inv, axis, False, False)
    # a broadcast input
    one = torch.randn((1, S, Hq, D), device="cuda").to(dtype).expand(B, S, Hq, D)
    check(api.rope_axes(one, pos, inv, axis), one, pos, inv, axis, False, False)
    # in place, through the views; what lies between them stays
    before = qkv.clone()
    r = api.rope_axes((q, k), pos, inv, axis, outs=(q, k))
    assert r[0].data_ptr() == q.data_ptr()
    assert torch.equal(qkv[:, :, :Hq], yq) and torch.equal(qkv[:, :, Hq:Hq + Hkv], yk)
    assert torch.equal(qkv[:, :, Hq + Hkv:], before[:, :, Hq + Hkv:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("paired", [False, True])
def test_alignment_does_not_change_the_result(paired, dtype, cuda):
    B, S, H, D = 2, 700, 9, 64
    x = torch.randn((B, S, H, D), device="cuda").to(dtype)
    odd = torch.empty(x.numel() + 1, dtype=dtype, device="cuda")[1:].view(x.shape).copy_(x)
    pos = torch.randint(-9, 10 ** 6, (2, B, S), device="cuda")
    inv, axis = freqs(48, 2)
    want = api.rope_axes(x, pos, inv, axis, paired=paired)
    assert torch.equal(api.rope_axes(odd, pos, inv, axis, paired=paired), want)
    assert torch.equal(api.rope_axes([odd, x], pos, inv, axis, paired=paired)[1], want)
    assert torch.equal(api.rope_axes(x, pos, inv, axis, paired=paired, outs=x), want)


def test_inverse_is_the_gradient_and_differences(cuda):
    """The gradient of sum(w * rope(x)) is rope(w, inverse): against 64-bit central differences."""
    B, S, H, D = 1, 9, 2, 32
    x, w, dirn = (torch.randn((B, S, H, D), device="cuda", dtype=torch.float64) for _ in range(3))
    pos = torch.randint(0, 4000, (2, B, S), device="cuda")
    inv, axis = freqs(D, 2)
    g = api.rope_axes(w.float(), pos, inv, axis, inverse=True)
    h = 1e-3  # the map is linear: the difference has no truncation error
    diff = (((rotate(x + h * dirn, pos, inv, axis, False, False) - rotate(x - h * dirn, pos, inv, axis, False, False)) * w).sum() / (2 * h))
    bound = 2.0 ** -19 * (w.abs().sum(-1, keepdim=True) * dirn.abs()).sum()
    assert (diff - (g.double() * dirn).sum()).abs() <= bound


def test_stream_and_graph(cuda):
    x = torch.randn((2, 40, 4, 64), device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 5000, (2, 2, 40), device="cuda", dtype=torch.int32)
    inv, axis = freqs(64, 2)
    want = api.rope_axes(x, pos, inv, axis)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.rope_axes(x, pos, inv, axis, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = api.rope_axes(x, pos, inv, axis)
    pos.add_(3)
    graph.replay()
    check(y, x, pos, inv, axis, False, False)
