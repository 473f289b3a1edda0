"""Sliding-window attention with sinks on a B200: forward, backward and the decode form against the
64-bit definition, with the bounds of window_ref.py; documents, odd sizes, graphs, streams, caches."""
import math
import random

import pytest
import torch

from long_context_exact_tma_b200 import api
from window_ref import U, attend, backward, forward_bounds, rotate, visible, within

pytestmark = pytest.mark.gpu


def normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def qkv(B, S, Hq, Hkv, D, seed=0):
    return normal(seed, B, S, Hq, D), normal(seed + 1, B, S, Hkv, D), normal(seed + 2, B, S, Hkv, D)


# B, S, Hq, Hkv, D, window, sinks, documents
CASES = [
    (1, 1, 2, 2, 64, 1, 0, None),
    (1, 2, 2, 1, 128, 1, 1, None),
    (2, 127, 4, 2, 64, 5, 3, None),
    (1, 128, 1, 1, 128, 128, 0, None),
    (1, 129, 3, 1, 64, 64, 4, None),          # odd group: row pairs, an odd last tile
    (1, 200, 6, 2, 128, 1000, 4, None),       # the window covers everything
    (2, 385, 2, 1, 64, 130, 1, None),
    (1, 513, 4, 4, 64, 129, 128, None),       # as many sinks as a tile
    (1, 700, 2, 2, 128, 33, 17, None),
    (1, 1100, 4, 1, 128, 257, 4, None),
    (3, 260, 5, 5, 64, 1, 2, None),           # itself and the sinks
    (1, 1500, 2, 2, 64, 3, 100, None),
    (1, 640, 2, 1, 64, 100, 4, [0, 1, 2, 130, 131, 640]),
    (2, 999, 4, 2, 128, 64, 20, [0, 250, 250, 257, 900, 999]),   # an empty document
    (1, 1300, 3, 3, 64, 200, 3, [0, 100, 1290, 1300]),
    (1, 1024, 2, 2, 64, 50, 128, [0, 384, 512, 1024]),
    (1, 900, 8, 1, 128, 400, 4, list(range(0, 901, 9))),         # documents shorter than a tile
    (1, 500, 2, 2, 64, 1, 100, [0, 88, 500]),                    # two sink tiles of rows of few keys
    (2, 777, 3, 1, 128, 300, 70, [0, 500, 777]),                 # row pairs whose second tile starts behind the sinks
    (1, 650, 1, 1, 64, 140, 5, [0, 129, 300, 650]),
    (1, 2600, 16, 16, 64, 70, 4, [0, 300, 1111, 2600]),          # more work items than SMs: a few left over,
    (2, 1350, 16, 4, 64, 200, 2, None),                          # of row pairs and of head pairs
    (1, 2500, 1, 1, 64, 90, 6, [0] + list(range(60, 560, 5)) + [2300, 2500]),   # a long document among many short ones
]


@pytest.mark.parametrize("B,S,Hq,Hkv,D,W,ns,cu", CASES)
def test_forward_and_backward(B, S, Hq, Hkv, D, W, ns, cu, cuda):
    q, k, v = qkv(B, S, Hq, Hkv, D, seed=S)
    do = normal(S + 3, B, S, Hq, D)
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    vis = visible(S, W, ns, cu, "cuda")
    out, lse = api.window_attn_fwd(q, k, v, W, ns, cu_seqlens=cut, check_status=True)
    qd, kd, vd, dd = (x.double() for x in (q, k, v, do))
    o, L, to, tl = forward_bounds(qd, kd, vd, vis)
    assert within(out, o, to) <= 1 and within(lse, L, tl) <= 1
    got = api.window_attn_bwd(q, k, v, out, lse, do, W, ns, cu_seqlens=cut, check_status=True)
    want, tol = backward(qd, kd, vd, out.double(), lse.double(), dd, vis)
    for name, x, y, t in zip(("dq", "dk", "dv"), got, want, tol):
        assert within(x, y, t) <= 1, name
    again = api.window_attn_bwd(q, k, v, out, lse, do, W, ns, cu_seqlens=cut)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("seed", range(16))
def test_drawn_shapes(seed, cuda):
    """Shapes, windows, sinks and documents drawn over the whole range, the bounds of the listed ones."""
    rng = random.Random(seed)
    for n in range(8):
        D, Hkv, B = rng.choice([64, 128]), rng.choice([1, 2, 3]), rng.choice([1, 2])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5])
        S, W = int(math.exp(rng.uniform(0, math.log(900)))), int(math.exp(rng.uniform(0, math.log(1000))))
        ns = rng.choice([0, 1, 4, rng.randint(0, 128), 128])
        cu = sorted([0, S] + [rng.randint(0, S) for _ in range(rng.randint(1, 8))]) if rng.random() < 0.5 else None
        try:
            test_forward_and_backward(B, S, Hq, Hkv, D, W, ns, cu, cuda)
        except AssertionError as e:
            raise AssertionError((B, S, Hq, Hkv, D, W, ns, cu)) from e


def test_many_short_steps_in_a_row(cuda):
    """Items that are mostly tiles of 16 and 32 sinks, each walked twice, call after call between other
    work: steps short enough for the warps to be two tiles ahead of a delayed product warp. Every call
    ends, and with the first one's result."""
    B, S, Hq, Hkv, D, W, ns = 1, 1500, 4, 2, 64, 1, 128
    cu = torch.tensor([0, 700, 1500], dtype=torch.int32, device="cuda")
    q, k, v = qkv(B, S, Hq, Hkv, D, seed=51)
    do = normal(54, B, S, Hq, D)
    out, lse = api.window_attn_fwd(q, k, v, W, ns, cu_seqlens=cu, check_status=True)
    first = api.window_attn_bwd(q, k, v, out, lse, do, W, ns, cu_seqlens=cu, check_status=True)
    other = torch.randn(512, 512, dtype=torch.float64, device="cuda")
    for _ in range(300):
        other @ other
        got = api.window_attn_bwd(q, k, v, out, lse, do, W, ns, cu_seqlens=cu, check_status=True)
        assert all(torch.equal(x, y) for x, y in zip(first, got))


def test_gradients_against_differences(cuda):
    """Directional derivatives of the 64-bit forward by central differences (h = 1e-5, error O(h^2)
    of a smooth sum) against the kernel's gradients along the same directions."""
    B, S, Hq, Hkv, D, W, ns = 1, 300, 4, 2, 64, 70, 3
    q, k, v = qkv(B, S, Hq, Hkv, D, seed=5)
    do = normal(9, B, S, Hq, D)
    vis = visible(S, W, ns, device="cuda")
    out, lse = api.window_attn_fwd(q, k, v, W, ns)
    got = api.window_attn_bwd(q, k, v, out, lse, do, W, ns)
    x = [t.double() for t in (q, k, v)]
    _, tol = backward(*x, out.double(), lse.double(), do.double(), vis)
    h = 1e-5
    for n in range(3):
        dirn = torch.randn(x[n].shape, dtype=torch.float64, device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(n))

        def loss(s):
            y = list(x)
            y[n] = x[n] + s * dirn
            return (attend(*y, vis)[0] * do.double()).sum()

        diff = (loss(h) - loss(-h)) / (2 * h)
        bound = (tol[n] * dirn.abs()).sum() + 1e-6 * diff.abs()
        assert (diff - (got[n].double() * dirn).sum()).abs() <= bound


def test_large_window_is_plain_causal_attention(cuda):
    """A window of the whole sequence is the framework's own causal attention, within the roundings of both."""
    B, S, H, D = 1, 1024, 4, 128
    q, k, v = qkv(B, S, H, H, D, seed=11)
    out, lse = api.window_attn_fwd(q, k, v, S, 0)
    o2, l2 = api.attn_fwd(*(x.view(1, 1, B, S, H, D) for x in (q, k, v)), True, 1, 1)
    _, _, to, tl = forward_bounds(*(x.double() for x in (q, k, v)), visible(S, S, 0, device="cuda"))
    assert within(out, o2.view_as(out).double(), 2 * to) <= 1
    assert within(lse, l2.view_as(lse).double(), 2 * tl) <= 1


def test_peaked_rows(cuda):
    """One key takes all the weight of later rows (scores up to ~60): a running maximum that grows."""
    B, S, H, D, W, ns = 1, 600, 2, 64, 200, 1
    q, k, v = qkv(B, S, H, H, D, seed=21)
    k[:, 100] = q[:, 300] * 6
    k[:, 0] = q[:, 500] * 7
    vis = visible(S, W, ns, device="cuda")
    out, lse = api.window_attn_fwd(q, k, v, W, ns)
    o, L, to, tl = forward_bounds(q.double(), k.double(), v.double(), vis)
    assert within(out, o, to) <= 1 and within(lse, L, tl) <= 1


def test_outputs_stay_inside_their_rows(cuda):
    """Given outputs inside larger buffers: nothing around them is written."""
    B, S, H, D, W, ns = 1, 131, 2, 64, 40, 2
    q, k, v = qkv(B, S, H, H, D, seed=31)
    n = q.numel()

    def guarded(numel, dtype):
        buf = torch.full((numel + 4096,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[2048:2048 + numel]

    bo, o = guarded(n, torch.bfloat16)
    bl, l = guarded(n // D, torch.float32)
    out, lse = api.window_attn_fwd(q, k, v, W, ns, out=o.view(q.shape), lse=l.view(B, S, H))
    grads = [guarded(n, torch.bfloat16) for _ in range(3)]
    api.window_attn_bwd(q, k, v, out, lse, normal(3, B, S, H, D), W, ns,
                        **{x: g[1].view(q.shape) for x, g in zip(("dq", "dk", "dv"), grads)})
    for buf in [bo, bl] + [g[0] for g in grads]:
        m = buf.numel() - 4096
        assert (buf[:2048] == 7).all() and (buf[2048 + m:] == 7).all()


def test_outputs_aligned_to_16_bytes(cuda):
    """Outputs that start 16 bytes into a line, beside ones at its start: the same values."""
    B, S, H, D, W, ns = 1, 300, 2, 128, 40, 2
    q, k, v = qkv(B, S, H, H, D, seed=35)
    do = normal(38, B, S, H, D)
    want = api.window_attn_fwd(q, k, v, W, ns)
    wg = api.window_attn_bwd(q, k, v, *want, do, W, ns)

    def shifted(x):
        return torch.empty(x.numel() + 8, dtype=x.dtype, device="cuda")[8:].view(x.shape)

    out, lse = api.window_attn_fwd(q, k, v, W, ns, out=shifted(want[0]))
    got = api.window_attn_bwd(q, k, v, out, lse, do, W, ns, dq=shifted(q), dk=shifted(k), dv=shifted(v))
    assert all(x.data_ptr() % 32 == 16 for x in (out, *got))
    assert all(torch.equal(a, b) for a, b in zip((out, lse, *got), (*want, *wg)))


def test_other_stream_and_graph(cuda):
    """The call on a given stream, and captured and replayed on new inputs in the same buffers."""
    B, S, Hq, Hkv, D, W, ns = 2, 500, 4, 2, 64, 100, 4
    q, k, v = qkv(B, S, Hq, Hkv, D, seed=41)
    do = normal(44, B, S, Hq, D)
    want = api.window_attn_fwd(q, k, v, W, ns)
    wg = api.window_attn_bwd(q, k, v, *want, do, W, ns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = api.window_attn_fwd(q, k, v, W, ns, stream=side)
    got = api.window_attn_bwd(q, k, v, out, lse, do, W, ns, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip((out, lse, *got), (*want, *wg)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gl = api.window_attn_fwd(q, k, v, W, ns)
        gg = api.window_attn_bwd(q, k, v, go, gl, do, W, ns)
    for x, seed in ((q, 51), (k, 52), (v, 53)):
        x.copy_(normal(seed, *x.shape))
    graph.replay()
    graph.replay()
    ref = api.window_attn_fwd(q, k, v, W, ns)
    rg = api.window_attn_bwd(q, k, v, *ref, do, W, ns)
    assert all(torch.equal(a, b) for a, b in zip((go, gl, *gg), (*ref, *rg)))


# ---------------------------------------------------------------- decode
def decode_ref(q, k, v, lens, W, ns):
    """Per sequence and token, the 64-bit rows and their bounds."""
    N, n, Hq, D = q.shape
    G = Hq // k.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    to, tl = torch.full_like(out, 1e-30), torch.zeros_like(lse)
    for s, ln in enumerate(lens):
        for t in range(n):
            p = ln - n + t
            if p < 0:
                continue
            j = torch.arange(p + 1, device="cuda")
            j = j[(p - j < W) | (j < ns)]
            kk, vv = (x[s, j].double().repeat_interleave(G, 1) for x in (k, v))
            x = q[s, t].double()
            sc = torch.einsum("hd,jhd->hj", x, kk) / math.sqrt(D)
            w = torch.softmax(sc, -1)
            out[s, t] = torch.einsum("hj,jhd->hd", w, vv)
            lse[s, t] = torch.logsumexp(sc, -1)
            A = torch.einsum("hj,jhd->hd", w, vv.abs())
            M = torch.einsum("hd,jhd->hj", x.abs(), kk.abs()).amax(-1)
            to[s, t] = (U * (1 + U) + 4e-4) * (A + out[s, t].abs()) + U * out[s, t].abs() + 1e-30
            tl[s, t] = 2.0 ** -24 * (math.sqrt(D) * M + 2 * len(j) + 64)
    return out, lse, to, tl


@pytest.mark.parametrize("N,n,cap,Hq,Hkv,D,W,ns", [
    (1, 1, 1, 1, 1, 64, 1, 0),
    (3, 1, 40, 4, 2, 64, 7, 2),
    (2, 1, 300, 8, 1, 128, 1000, 4),
    (9, 3, 129, 6, 2, 64, 33, 5),
    (2, 16, 2500, 4, 4, 128, 700, 128),
    (1, 5, 5000, 24, 3, 128, 5000, 0),
    (2, 1, 9000, 5, 1, 64, 4096, 1),
    (1, 2, 4000, 17, 1, 64, 2048, 3),
    (1, 1, 20000, 8, 2, 128, 20000, 0),      # keys shared out over the SMs
    (3, 2, 40001, 10, 1, 128, 33333, 7),     # of unequal sequences, 20 rows a kv head
    (40, 1, 9000, 3, 1, 64, 9000, 4),        # more sequences than a warp has lanes
])
def test_decode(N, n, cap, Hq, Hkv, D, W, ns, cuda):
    q, k, v = normal(N + cap, N, n, Hq, D), normal(1, N, cap, Hkv, D), normal(2, N, cap, Hkv, D)
    lens = [cap] + [max(0, cap - 1 - 13 * s) for s in range(1, N)]
    if N > 2:
        lens[1], lens[2] = 0, min(n - 1, cap)  # an idle slot; a token before the first
    if N > 30:
        lens = [cap - 211 * s if s % 3 else s for s in range(N)]
    k2, v2 = k.clone(), v.clone()
    for s, ln in enumerate(lens):  # what lies past the cached tokens may be anything
        k2[s, ln:], v2[s, ln:] = math.nan, math.inf
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = api.window_attn_decode(q, k2, v2, cl, W, ns)
    o, L, to, tl = decode_ref(q, k, v, lens, W, ns)
    assert within(out, o, to) <= 1
    none = torch.isinf(L)
    assert torch.equal(none, torch.isinf(lse)) and (lse[none] < 0).all() and (out[none] == 0).all()
    if (~none).any():
        assert within(lse[~none], L[~none], tl[~none]) <= 1
    # another order of the cache in memory
    kt, vt = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k2, v2))
    out2, lse2 = api.window_attn_decode(q, kt, vt, cl, W, ns)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("N,n,cap,Hq,Hkv,D,W,ns", [(5, 2, 700, 8, 2, 64, 100, 4), (2, 1, 30000, 8, 1, 128, 30000, 0)])
def test_decode_captured_and_on_two_streams(N, n, cap, Hq, Hkv, D, W, ns, cuda):
    """Replayed over a cache and lengths that have grown meanwhile, in one launch and with the keys shared
    out; and two calls at once on their own streams."""
    q, k, v = normal(61, N, n, Hq, D), normal(62, N, cap, Hkv, D), normal(63, N, cap, Hkv, D)
    lens = torch.arange(N, dtype=torch.int32, device="cuda") * (cap // N) + 20
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = api.window_attn_decode(q, k, v, lens, W, ns)
    for step in (0, 1, cap // 3):
        lens.add_(step)
        q.copy_(normal(64 + step, *q.shape))
        graph.replay()
        want = api.window_attn_decode(q, k, v, lens, W, ns)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        o, L, to, tl = decode_ref(q, k, v, [min(x, cap) for x in lens.tolist()], W, ns)
        assert within(out, o, to) <= 1 and within(lse, L, tl) <= 1
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    qs = [q, normal(65, *q.shape)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for s in (0, 1):
            got[s].append(api.window_attn_decode(qs[s], k, v, lens, W, ns, stream=streams[s]))
    torch.cuda.synchronize()
    for s in (0, 1):
        want = api.window_attn_decode(qs[s], k, v, lens, W, ns)
        assert all(torch.equal(a, b) for pair in got[s] for a, b in zip(pair, want))


def test_steps_on_two_streams_at_once(cuda):
    """Forward and backward of two problems, call by call on two streams, next to a plain kernel on a third."""
    W, ns = 60, 4
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    probs = [(qkv(1, 1300, 4, 2, 64, seed=71), normal(74, 1, 1300, 4, 64)),
             (qkv(2, 900, 3, 1, 128, seed=75), normal(78, 2, 900, 3, 128))]

    def step(p, stream=None):
        (q, k, v), do = p
        out, lse = api.window_attn_fwd(q, k, v, W, ns, stream=stream)
        return (out, lse, *api.window_attn_bwd(q, k, v, out, lse, do, W, ns, stream=stream))

    want = [step(p) for p in probs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(25):
        for s in (0, 1):
            got[s].append(step(probs[s], streams[s]))
        probs[0][1] + 1
    torch.cuda.synchronize()
    for s in (0, 1):
        assert all(torch.equal(a, b) for r in got[s] for a, b in zip(r, want[s]))


def test_decode_lens_outside_the_cache_are_clamped(cuda):
    q, k, v = normal(1, 2, 1, 2, 64), normal(2, 2, 50, 1, 64), normal(3, 2, 50, 1, 64)
    a = api.window_attn_decode(q, k, v, torch.tensor([50, 0], dtype=torch.int32, device="cuda"), 20, 1)
    b = api.window_attn_decode(q, k, v, torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda"), 20, 1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_decode_past_32_bit_offsets(cuda):
    """The last sequence of a cache of more than 2^31 elements."""
    N, cap, Hkv, D = 5, 1 << 19, 8, 128
    k = torch.empty((N, cap, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 1 << 31
    W, ns = 500, 4
    for x, seed in ((k, 1), (v, 2)):
        x[:, :ns] = normal(seed, N, ns, Hkv, D)
        x[:, cap - W - 1:] = normal(seed + 10, N, W + 1, Hkv, D)
    q = normal(5, N, 1, 2 * Hkv, D)
    out, lse = api.window_attn_decode(q, k, v, torch.full((N,), cap, dtype=torch.int32, device="cuda"), W, ns)
    # the same keys in a short cache
    ks, vs = (torch.cat([x[:, :ns], x[:, cap - W:]], 1) for x in (k, v))
    o, L, to, tl = decode_ref(q, ks, vs, [ns + W] * N, W, ns)
    assert within(out, o, to) <= 1 and within(lse, L, tl) <= 1


def test_rope_then_attention_then_decode(cuda):
    """The operators as a layer uses them: q, k from a fused projection rotated in one launch, attention,
    its backward with the rotation's inverse on the gradients, and the last token again by decoding."""
    B, S, Hq, Hkv, D, W, ns = 2, 333, 4, 2, 64, 90, 2
    qkv_ = normal(61, B, S, Hq + 2 * Hkv, D)
    v = qkv_[:, :, Hq + Hkv:].contiguous()
    f = torch.arange(D // 2, dtype=torch.float64)
    inv, axis = 10000.0 ** (-2 * f / D), (f % 3).to(torch.int32)
    pos = torch.stack([torch.arange(S) + 100000 * b for b in range(B)]).cuda()
    pos = torch.stack([pos, pos // 7, pos % 50]).contiguous()
    q, k = api.rope_axes((qkv_[:, :, :Hq], qkv_[:, :, Hq:Hq + Hkv]), pos, inv, axis)
    out, lse = api.window_attn_fwd(q, k, v, W, ns)
    do = normal(62, B, S, Hq, D)
    dq, dk, dv = api.window_attn_bwd(q, k, v, out, lse, do, W, ns)
    gq, gk = api.rope_axes((dq, dk), pos, inv, axis, inverse=True)
    # the whole against 64-bit autograd: roundings of q, k, out, P, dS and of each gradient twice;
    # relative L2 of each below 4 U (independent roundings; the measured part of each is under U / 2)
    x = qkv_.double().requires_grad_(True)
    rq, rk = (rotate_grad(x[:, :, a:b], pos, inv, axis) for a, b in ((0, Hq), (Hq, Hq + Hkv)))
    o, L, _ = attend(rq, rk, x[:, :, Hq + Hkv:], visible(S, W, ns, device="cuda"))
    (o * do.double()).sum().backward()
    g = x.grad
    for got, want in ((out, o.detach()), (gq, g[:, :, :Hq]), (gk, g[:, :, Hq:Hq + Hkv]), (dv, g[:, :, Hq + Hkv:])):
        assert ((got.double() - want).norm() / want.norm()).item() <= 4 * U
    o1, l1 = api.window_attn_decode(q[:, -1:].contiguous(), k, v, torch.full((B,), S, dtype=torch.int32, device="cuda"),
                                    W, ns)
    _, _, to, tl = forward_bounds(q.double(), k.double(), v.double(), visible(S, W, ns, device="cuda"))
    assert within(o1, out[:, -1:].double(), 2 * to[:, -1:]) <= 1
    assert within(l1, lse[:, -1:].double(), 2 * tl[:, -1:]) <= 1


def rotate_grad(x, pos, inv, axis):
    """The rotation in 64 bits, differentiable."""
    a = pos.double()[axis.long().cuda()].permute(1, 2, 0) * inv.cuda()
    c, s = torch.cos(a).unsqueeze(2), torch.sin(a).unsqueeze(2)
    x1, x2 = x.chunk(2, -1)
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)
