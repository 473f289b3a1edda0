"""Refusals of the window attention, decode and rotary entry points, before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

from long_context_exact_tma_b200 import api
from long_context_exact_tma_b200 import binding as B_

FAKE = 1 << 20  # 16-byte aligned, never dereferenced (validation fails first)
INVALID, UNSUPPORTED, WORKSPACE = B_.USP_ERR_INVALID_ARG, B_.USP_ERR_UNSUPPORTED, B_.USP_ERR_WORKSPACE

BAD_SHAPES = [
    (dict(B=0), INVALID), (dict(S=0), INVALID), (dict(Hq=-1), INVALID), (dict(Hkv=0), INVALID),
    (dict(window=0), INVALID), (dict(sinks=-1), INVALID), (dict(cu=FAKE, n_docs=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(Hkv=3), UNSUPPORTED), (dict(sinks=129), UNSUPPORTED),
    (dict(S=1 << 28, Hq=8), UNSUPPORTED), (dict(S=(1 << 30) + 1, Hq=1, Hkv=1), UNSUPPORTED),
]


def fwd(**kw):
    a = dict(p=[FAKE] * 5, B=1, S=100, Hq=4, Hkv=2, D=64, window=10, sinks=2, cu=None, n_docs=0, ws=FAKE, n=256)
    a.update(kw)
    return B_.usp_window_attn_fwd(*a["p"], *(a[x] for x in ("B", "S", "Hq", "Hkv", "D", "window", "sinks", "cu", "n_docs")),
                                  a["ws"], a["n"], stream=0, check=False)


def bwd(**kw):
    a = dict(p=[FAKE] * 9, B=1, S=100, Hq=4, Hkv=2, D=64, window=10, sinks=2, cu=None, n_docs=0, ws=FAKE, n=1 << 40)
    a.update(kw)
    return B_.usp_window_attn_bwd(*a["p"], *(a[x] for x in ("B", "S", "Hq", "Hkv", "D", "window", "sinks", "cu", "n_docs")),
                                  a["ws"], a["n"], stream=0, check=False)


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_shapes_are_refused(kw, code):
    assert fwd(**kw) == code and B_.usp_last_error()
    assert bwd(**kw) == code


@pytest.mark.parametrize("call,n", [(fwd, 5), (bwd, 9)])
def test_pointers_and_workspaces_are_refused(call, n):
    for x in range(n):
        for bad in (None, FAKE + 8):
            p = [FAKE] * n
            p[x] = bad
            assert call(p=p) == INVALID
    assert call(ws=None) == WORKSPACE
    assert call(ws=FAKE + 8) == WORKSPACE
    assert call(n=255) == WORKSPACE


def test_workspace_sizes():
    ws = B_.usp_window_workspace_size
    assert ws(1, 100, 4, 2, 64, 10, 2, 0, 0) == ws(3, 9000, 64, 1, 128, 99, 128, 7, 0) == B_.USP_WINDOW_FWD_WS
    tables = 2 * 4 * (1 * 4 * 128)
    assert ws(1, 100, 4, 2, 64, 10, 0, 0, 1) == 256 + tables
    assert ws(1, 100, 4, 2, 64, 100, 2, 0, 1) == 256 + tables            # nobody is far from a sink
    part, sums = 4 * 2 * 1 * 2 * 2 * 64, 4 * 2 * 3 * 2 * 2 * 64
    assert ws(1, 100, 4, 2, 64, 10, 2, 3, 1) == 256 + tables + part + sums
    # short documents without end: no sums
    assert ws(1, 100, 4, 2, 64, 10, 2, 5, 1) == ws(1, 100, 4, 2, 64, 10, 2, 100000, 1) == 256 + tables + part
    assert ws(1, 100, 4, 3, 64, 10, 2, 0, 1) == 0 and ws(1, 100, 4, 2, 64, 0, 2, 0, 0) == 0
    assert ws(1, 100, 4, 2, 64, 10, 2, -1, 0) == 0
    wd = B_.usp_window_decode_workspace_size
    assert wd(64, 1, 4096, 32, 8, 128, 1024, 4) == 256                   # enough sequences: one split
    assert wd(1, 1, 131072, 8, 1, 128, 131072, 0) > 256
    assert wd(1, 17, 100, 8, 1, 128, 50, 0) == 0


def decode(**kw):
    a = dict(p=[FAKE] * 6, N=2, n=1, cap=100, Hq=4, Hkv=2, D=64, window=10, sinks=2, ks=(12800, 128, 64),
             vs=(12800, 128, 64), ws=FAKE, nb=1 << 30)
    a.update(kw)
    return B_.usp_window_attn_decode(*a["p"], *(a[x] for x in ("N", "n", "cap", "Hq", "Hkv", "D", "window", "sinks")),
                                     a["ks"], a["vs"], a["ws"], a["nb"], stream=0, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), INVALID), (dict(n=0), INVALID), (dict(cap=0), INVALID), (dict(window=0), INVALID),
    (dict(sinks=-1), INVALID), (dict(D=80), UNSUPPORTED), (dict(Hq=5), UNSUPPORTED), (dict(n=17), UNSUPPORTED),
    (dict(sinks=129), UNSUPPORTED), (dict(ks=(12800, 132, 64)), INVALID), (dict(vs=(-8, 128, 64)), INVALID),
    (dict(N=1 << 24, Hq=64), UNSUPPORTED), (dict(cap=(1 << 30) + 1), UNSUPPORTED),
    # a long cache of one sequence: partials of the splits
    (dict(N=1, Hkv=1, cap=1 << 20, window=1 << 20, ws=None), WORKSPACE),
    (dict(N=1, Hkv=1, cap=1 << 20, window=1 << 20, nb=256), WORKSPACE),
    (dict(N=1, Hkv=1, cap=1 << 20, window=1 << 20, ws=FAKE + 8), WORKSPACE),
])
def test_decode_is_refused(kw, code):
    assert decode(**kw) == code and B_.usp_last_error()


def test_decode_pointers_are_refused():
    for x in range(6):
        for bad in (None, FAKE + 2):
            p = [FAKE] * 6
            p[x] = bad
            assert decode(p=p) == INVALID


def rope(**kw):
    R = kw.get("R", 8)
    inv = kw.pop("inv", torch.ones(max(R // 2, 1), dtype=torch.float64))
    axis = kw.pop("axis", torch.zeros(max(R // 2, 1), dtype=torch.int32))
    a = dict(jobs=[(FAKE, FAKE, 2, (64, 32, 16), (64, 32, 16))], B=1, S=2, D=16, R=8, dtype=B_.USP_BF16, pos=FAKE,
             bits=64, axes=1, paired=0, inverse=0)
    a.update(kw)
    return B_.usp_rope_axes(a["jobs"], a["B"], a["S"], a["D"], a["R"], a["dtype"], a["pos"], a["bits"], a["axes"], inv,
                            axis, a["paired"], a["inverse"], stream=0, check=False)


JOB = (FAKE, FAKE, 2, (64, 32, 16), (64, 32, 16))


@pytest.mark.parametrize("kw,code", [
    (dict(jobs=[]), INVALID), (dict(jobs=[JOB] * 5), INVALID), (dict(B=0), INVALID), (dict(D=0), INVALID),
    (dict(dtype=7), INVALID), (dict(bits=16), INVALID), (dict(pos=FAKE + 4), INVALID), (dict(pos=None), INVALID),
    (dict(axes=0), INVALID), (dict(axes=256), INVALID), (dict(paired=2), INVALID), (dict(inverse=-1), INVALID),
    (dict(R=7), UNSUPPORTED), (dict(R=0), UNSUPPORTED), (dict(R=18), UNSUPPORTED), (dict(R=258, D=512), UNSUPPORTED),
    (dict(inv=torch.tensor([1.0, float("nan"), 1, 1], dtype=torch.float64)), INVALID),
    (dict(axis=torch.tensor([0, 1, 0, 0], dtype=torch.int32)), INVALID),
    (dict(axis=torch.tensor([0, -1, 0, 0], dtype=torch.int32)), INVALID),
    (dict(inv=None), INVALID), (dict(axis=None), INVALID),
    (dict(jobs=[(None,) + JOB[1:]]), INVALID), (dict(jobs=[(FAKE, FAKE + 1) + JOB[2:]]), INVALID),
    (dict(jobs=[(FAKE, FAKE, 0) + JOB[3:]]), INVALID), (dict(jobs=[JOB[:3] + ((64, -32, 16), (64, 32, 16))]), INVALID),
    (dict(jobs=[JOB[:4] + ((64, 32, 0),)]), INVALID),   # the output's heads on top of one another
    (dict(B=2, jobs=[JOB[:4] + ((32, 32, 16),)]), INVALID),              # its sequences' tokens
    (dict(jobs=[JOB[:4] + ((128, 32, 48),)]), INVALID),                  # a head among the next token's
    (dict(jobs=[JOB[:3] + ((64, 16, 32), (64, 32, 16))]), INVALID),      # in place with other strides
    (dict(jobs=[JOB, JOB]), INVALID),                                    # the same tensor twice
    (dict(jobs=[JOB, (FAKE, 2 * FAKE) + JOB[2:]]), INVALID),             # one reads what the other writes
    (dict(jobs=[(2 * FAKE, FAKE) + JOB[2:], (3 * FAKE, 2 * FAKE) + JOB[2:]]), INVALID),
])
def test_rope_is_refused(kw, code):
    assert rope(**kw) == code and B_.usp_last_error()


def test_python_calls_refuse_cpu_tensors_and_types():
    x = torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.window_attn_fwd(x, x, x, 4)
    with pytest.raises(ValueError):
        api.window_attn_bwd(x, x, x, x, x, x, 4)
    with pytest.raises(ValueError):
        api.window_attn_decode(x, x, x, x, 4)
    with pytest.raises(ValueError):
        api.window_attn_fwd(x[0], x, x, 4)
    with pytest.raises(ValueError):
        api._window_size(0, 1)
    with pytest.raises(ValueError):
        api._window_size(1, -1)
    with pytest.raises(TypeError):
        api._window_size(3.5, 0)
    assert api._window_size(1 << 40, 1 << 35) == (0x7FFFFFFF, 0x7FFFFFFF)
    inv, axis = torch.ones(4, dtype=torch.float64), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.rope_axes(x, torch.zeros((1, 1, 8), dtype=torch.int64), inv, axis)
    with pytest.raises(TypeError):
        api.rope_axes(x.half(), torch.zeros((1, 1, 8), dtype=torch.int64), inv, axis)
    with pytest.raises(ValueError):
        api.rope_axes([], None, inv, axis)


def test_rope_job_matches_the_header():
    assert ctypes.sizeof(B_.RopeJob) == 8 + 8 + 8 + 6 * 8 == B_.ROPE_JOB.size
    job = B_.RopeJob(1, 2, 3, 4, 5, 6, 7, 8, 9)
    assert bytes(job) == B_.ROPE_JOB.pack(1, 2, 3, 4, 5, 6, 7, 8, 9)
