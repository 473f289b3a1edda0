"""Torch-facing helpers over the C ABI: allocate outputs and workspaces with
torch (device memory and streams only) and call libusp.so. No arithmetic of
the path happens here.
"""
from __future__ import annotations

import contextlib
import functools
import operator

import torch

from . import binding as B_


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return B_.USP_BF16
    if t.dtype == torch.float32:
        return B_.USP_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _require_cuda(*ts):
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")


def zigzag_shard(x: torch.Tensor, P_u: int, P_r: int, out=None, stream=None) -> torch.Tensor:
    """global [B, S, H, D] -> rank-major [P, B, S/P, H, D]."""
    _require_cuda(x)
    B, S, H, D = x.shape
    P = P_u * P_r
    out = torch.empty((P, B, S // P, H, D), dtype=x.dtype, device=x.device) if out is None else out
    B_.usp_zigzag_shard(x, out, B, S, H, D, _dt(x), P_u, P_r, stream)
    return out


def zigzag_unshard(x: torch.Tensor, P_u: int, P_r: int, out=None, stream=None) -> torch.Tensor:
    """rank-major [P, B, S/P, H, D] -> global [B, S, H, D]."""
    _require_cuda(x)
    P, B, c2, H, D = x.shape
    S = P * c2
    out = torch.empty((B, S, H, D), dtype=x.dtype, device=x.device) if out is None else out
    B_.usp_zigzag_unshard(x, out, B, S, H, D, _dt(x), P_u, P_r, stream)
    return out


def seq2head(x: torch.Tensor, P_u: int, P_r: int, out=None, stream=None) -> torch.Tensor:
    """rank-major [P, B, S/P, H, D] -> head-sharded [P_r, P_u, B, S/P_r, H/P_u, D]."""
    _require_cuda(x)
    P, B, c2, H, D = x.shape
    S = P * c2
    out = (torch.empty((P_r, P_u, B, S // P_r, H // P_u, D), dtype=x.dtype, device=x.device)
           if out is None else out)
    B_.usp_seq2head_permute(x, out, B, S, H, D, _dt(x), P_u, P_r, stream)
    return out


def head2seq(x: torch.Tensor, P_u: int, P_r: int, out=None, stream=None) -> torch.Tensor:
    """head-sharded [P_r, P_u, B, S/P_r, H/P_u, D] -> rank-major [P, B, S/P, H, D]."""
    _require_cuda(x)
    Pr, Pu, B, L, Hl, D = x.shape
    S = L * P_r
    P = P_u * P_r
    out = torch.empty((P, B, S // P, Hl * P_u, D), dtype=x.dtype, device=x.device) if out is None else out
    B_.usp_head2seq_permute(x, out, B, S, Hl * P_u, D, _dt(x), P_u, P_r, stream)
    return out


def seq2head_many(xs, P_u: int, P_r: int, outs=None, stream=None):
    """The seq->head all-to-all of several rank-major tensors [P, B, S/P, H_x, D_x]
    (e.g. Q, K, V) in one launch; returns the head-sharded tensors."""
    _require_cuda(*xs)
    outs = list(outs) if outs is not None else [None] * len(xs)
    jobs = []
    for x_, (x, o) in enumerate(zip(xs, outs)):
        P, B, c2, H, D = x.shape
        if o is None:
            o = torch.empty((P_r, P_u, B, P * c2 // P_r, H // P_u, D), dtype=x.dtype, device=x.device)
            outs[x_] = o
        jobs.append((x, o, H, D, _dt(x)))
    P, B, c2 = xs[0].shape[:3]
    B_.usp_permute_batch(B_.USP_MAP_SEQ2HEAD, jobs, B, P * c2, P_u, P_r, stream)
    return outs


def head2seq_many(xs, P_u: int, P_r: int, outs=None, stream=None):
    """The head->seq regather of several head-sharded tensors (e.g. dQ, dK, dV)
    in one launch; returns the rank-major tensors [P, B, S/P, H_x, D_x]."""
    _require_cuda(*xs)
    outs = list(outs) if outs is not None else [None] * len(xs)
    jobs = []
    P = P_u * P_r
    for x_, (x, o) in enumerate(zip(xs, outs)):
        Pr, Pu, B, L, Hl, D = x.shape
        if o is None:
            o = torch.empty((P, B, L * P_r // P, Hl * P_u, D), dtype=x.dtype, device=x.device)
            outs[x_] = o
        jobs.append((x, o, Hl * P_u, D, _dt(x)))
    Pr, Pu, B, L = xs[0].shape[:4]
    B_.usp_permute_batch(B_.USP_MAP_HEAD2SEQ, jobs, B, L * P_r, P_u, P_r, stream)
    return outs


def to_head_sharded(x, P_u, P_r, stream=None):
    return seq2head(zigzag_shard(x, P_u, P_r, stream=stream), P_u, P_r, stream=stream)


def from_head_sharded(x, P_u, P_r, stream=None):
    return zigzag_unshard(head2seq(x, P_u, P_r, stream=stream), P_u, P_r, stream=stream)


def workspace(nbytes: int, device) -> torch.Tensor:
    n = max(int(nbytes), 256)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def check_workspace(ws: torch.Tensor, stream=None) -> None:
    """Synchronise the stream and raise UspError(USP_ERR_TIMEOUT) if a kernel that
    used `ws` recorded a timed-out device wait (the word is cleared by the read)."""
    rc, site = B_.usp_workspace_status(ws, stream)
    if rc != B_.USP_OK:
        raise B_.UspError(rc, f"device wait timed out (site {site:#x}): {B_.usp_last_error()}")


def attn_fwd(q, k, v, causal: bool, P_u: int, P_r: int, mode: int = B_.USP_MODE_FUSED,
             ws: torch.Tensor | None = None, out=None, lse=None, stream=None, check_status: bool = False):
    """Forward over head-sharded q [P_r, P_u, B, L, Hq/P_u, D], k/v [..., Hkv/P_u, D].
    Returns (out bf16 like q, lse fp32 [P_r, P_u, B, L, Hq/P_u]). With
    check_status=True the call synchronises and raises on a timed-out device wait."""
    _require_cuda(q, k, v)
    Pr, Pu, B, L, Hql, D = q.shape
    Hkv = k.shape[4] * P_u
    Hq = Hql * P_u
    S = L * P_r
    need = B_.usp_attn_workspace_size(B, S, Hq, Hkv, D, causal, P_u, P_r, mode, 0)
    if ws is None:
        ws = workspace(need, q.device)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if lse is None else lse
    B_.usp_attn_fwd(q, k, v, out, lse, B, S, Hq, Hkv, D, causal, P_u, P_r, mode, ws, ws.numel(), stream)
    if check_status:
        check_workspace(ws, stream)
    return out, lse


def attn_bwd(q, k, v, out, lse, dO, causal: bool, P_u: int, P_r: int, ws=None, dq=None, dk=None, dv=None,
             stream=None, check_status: bool = False, grad_dtype=torch.float32):
    """Backward; returns (dQ bf16 like q, dK like k, dV like v), dK and dV in
    grad_dtype: fp32 (usp_attn_bwd) or bf16 (usp_attn_bwd_prepare, _dkdv_bf16 and
    _dq). With check_status=True the call synchronises and raises on a timed-out
    device wait."""
    if grad_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("grad_dtype must be torch.float32 or torch.bfloat16")
    _require_cuda(q, k, v, out, lse, dO)
    Pr, Pu, B, L, Hql, D = q.shape
    Hkv = k.shape[4] * P_u
    Hq = Hql * P_u
    S = L * P_r
    need = B_.usp_attn_workspace_size(B, S, Hq, Hkv, D, causal, P_u, P_r, 0, 1)
    if ws is None:
        ws = workspace(need, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty(k.shape, dtype=grad_dtype, device=k.device) if dk is None else dk
    dv = torch.empty(v.shape, dtype=grad_dtype, device=v.device) if dv is None else dv
    if dk.dtype != grad_dtype or dv.dtype != grad_dtype:
        raise ValueError("dk and dv must have dtype grad_dtype")
    if grad_dtype == torch.float32:
        B_.usp_attn_bwd(q, k, v, out, lse, dO, dq, dk, dv, B, S, Hq, Hkv, D, causal, P_u, P_r, ws, ws.numel(),
                        stream)
    else:
        geo = (B, S, Hq, Hkv, D, causal, P_u, P_r)
        B_.usp_attn_bwd_prepare(out, lse, dO, *geo, ws, ws.numel(), stream)
        B_.usp_attn_bwd_dkdv_bf16(q, k, v, dO, dk, dv, *geo, ws, ws.numel(), stream)
        B_.usp_attn_bwd_dq(q, k, v, dO, dq, *geo, ws, ws.numel(), stream)
    if check_status:
        check_workspace(ws, stream)
    return dq, dk, dv


def attn_fwd_masked(q, k, v, causal: bool, P_u: int, P_r: int, block_mask=None, cu_seqlens=None, ws=None, out=None,
                    lse=None, stream=None, check_status: bool = False):
    """usp_attn_fwd (fused) with a block mask [B, Hq, S/128, S/128] (uint8, CUDA)
    and/or document boundaries cu_seqlens [n_docs + 1] (int32, CUDA), both in
    original positions."""
    _require_cuda(q, k, v)
    Pr, Pu, B, L, Hql, D = q.shape
    Hkv = k.shape[4] * P_u
    Hq = Hql * P_u
    S = L * P_r
    n_docs = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    if ws is None:
        ws = workspace(B_.usp_attn_workspace_size(B, S, Hq, Hkv, D, causal, P_u, P_r, 0, 0), q.device)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if lse is None else lse
    B_.usp_attn_fwd_masked(q, k, v, out, lse, B, S, Hq, Hkv, D, causal, P_u, P_r, block_mask, cu_seqlens, n_docs, ws,
                           ws.numel(), stream)
    if check_status:
        check_workspace(ws, stream)
    return out, lse


def attn_bwd_masked(q, k, v, out, lse, dO, causal: bool, P_u: int, P_r: int, block_mask=None, cu_seqlens=None,
                    ws=None, stream=None, check_status: bool = False):
    """usp_attn_bwd with the masks of attn_fwd_masked; returns (dQ, dK, dV)."""
    _require_cuda(q, k, v, out, lse, dO)
    Pr, Pu, B, L, Hql, D = q.shape
    Hkv = k.shape[4] * P_u
    Hq = Hql * P_u
    S = L * P_r
    n_docs = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    if ws is None:
        ws = workspace(B_.usp_attn_workspace_size(B, S, Hq, Hkv, D, causal, P_u, P_r, 0, 1), q.device)
    dq = torch.empty_like(q)
    dk = torch.empty(k.shape, dtype=torch.float32, device=k.device)
    dv = torch.empty(v.shape, dtype=torch.float32, device=v.device)
    B_.usp_attn_bwd_masked(q, k, v, out, lse, dO, dq, dk, dv, B, S, Hq, Hkv, D, causal, P_u, P_r, block_mask,
                           cu_seqlens, n_docs, ws, ws.numel(), stream)
    if check_status:
        check_workspace(ws, stream)
    return dq, dk, dv


def dilated_attn_fwd(q, k, v, causal: bool, pairs, ws=None, out=None, lse=None, stream=None,
                     check_status: bool = False):
    """LongNet dilated attention over global-layout q [B, S, Hq, D], k/v [B, S, Hkv, D]
    for the (w, r) pairs `pairs`. Returns (out bf16 like q, lse fp32 [B, S, Hq])."""
    _require_cuda(q, k, v)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    if ws is None:
        ws = workspace(B_.usp_dilated_workspace_size(B, S, Hq, D), q.device)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if lse is None else lse
    B_.usp_dilated_attn_fwd(q, k, v, out, lse, B, S, Hq, Hkv, D, causal, pairs, ws, ws.numel(), stream)
    if check_status:
        check_workspace(ws, stream)
    return out, lse


def dilated_attn_bwd(q, k, v, out, lse, dO, causal: bool, pairs, ws=None, stream=None, check_status: bool = False):
    """Backward of dilated_attn_fwd; returns (dQ bf16 like q, dK fp32 like k, dV fp32 like v)."""
    _require_cuda(q, k, v, out, lse, dO)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    if ws is None:
        ws = workspace(B_.usp_dilated_bwd_workspace_size(B, S, Hq, D, pairs), q.device)
    dq = torch.empty_like(q)
    dk = torch.empty(k.shape, dtype=torch.float32, device=k.device)
    dv = torch.empty(v.shape, dtype=torch.float32, device=v.device)
    B_.usp_dilated_attn_bwd(q, k, v, out, lse, dO, dq, dk, dv, B, S, Hq, Hkv, D, causal, pairs, ws, ws.numel(), stream)
    if check_status:
        check_workspace(ws, stream)
    return dq, dk, dv


def lse_merge(o_parts: torch.Tensor, lse_parts: torch.Tensor, out_dtype=torch.bfloat16, stream=None):
    """o_parts [n, rows, D] fp32, lse_parts [n, rows] fp32 -> (out [rows, D], lse [rows])."""
    _require_cuda(o_parts, lse_parts)
    n, rows, D = o_parts.shape
    out = torch.empty((rows, D), dtype=out_dtype, device=o_parts.device)
    lse = torch.empty(rows, dtype=torch.float32, device=o_parts.device)
    B_.usp_lse_merge(o_parts, lse_parts, n, rows, D, out, _dt(out), lse, stream)
    return out, lse


def bwd_preprocess(out: torch.Tensor, dO: torch.Tensor, stream=None) -> torch.Tensor:
    _require_cuda(out, dO)
    D = out.shape[-1]
    rows = out.numel() // D
    delta = torch.empty(out.shape[:-1], dtype=torch.float32, device=out.device)
    B_.usp_bwd_preprocess(out, dO, delta, rows, D, stream)
    return delta


_HERE = contextlib.nullcontext()


# The checks below are on the path of calls that take a few microseconds: device
# numbers instead of device objects, one comparison per property.
def _refuse(name: str, t, dev: int, dtype, shape, contiguous: bool):
    """Says what is wrong with an argument that one of the calls below has turned down."""
    if not isinstance(t, torch.Tensor) or t.get_device() < 0 or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the device of the first one")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _check(name: str, t, dev: int, dtype, shape=None, contiguous: bool = True) -> None:
    """An argument of the calls below: a tensor of CUDA device `dev` with this type and shape."""
    if (not isinstance(t, torch.Tensor) or t.get_device() != dev or dev < 0 or t.dtype is not dtype
            or (shape is not None and t.shape != shape) or (contiguous and not t.is_contiguous())):
        _refuse(name, t, dev, dtype, shape, contiguous)


def _on(dev: int, stream, *inputs):
    """(context, raw stream) of a call on CUDA device `dev`: the device's current stream, or the given
    one. What the call allocates inside the context belongs to that stream; with a given stream the inputs
    are kept from the allocator until its work on them is done."""
    if stream is not None:
        s = torch.cuda.ExternalStream(stream, dev) if isinstance(stream, int) else stream
        if s.device.index != dev:
            raise ValueError("the stream is of another device than the tensors")
        for t in inputs:
            if t is not None:
                t.record_stream(s)
        return torch.cuda.stream(s), s.cuda_stream
    # (torch.cuda.current_stream() builds an object at ten times the price)
    return (_HERE if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev),
            torch._C._cuda_getCurrentRawStream(dev))


def _scratch(ws, nbytes: int, ref: torch.Tensor, dev: int) -> torch.Tensor:
    """The given workspace, or a new one (the calls below clear what they need of it)."""
    if ws is None:
        return ref.new_empty(nbytes, dtype=torch.uint8)
    _check("ws", ws, dev, torch.uint8)
    return ws


def _like(t, name: str, ref: torch.Tensor, dev: int) -> torch.Tensor:
    """The given output, or a new one like ref."""
    if t is None:
        return torch.empty_like(ref)
    _check(name, t, dev, ref.dtype, ref.shape)
    return t


def _lse_of(t, q: torch.Tensor, shape, dev: int) -> torch.Tensor:
    if t is None:  # (the shape as separate numbers: a tuple takes 0.4 us more)
        return q.new_empty(*shape, dtype=torch.float32)
    _check("lse", t, dev, torch.float32, shape)
    return t


def _window_size(window, sinks):
    """The two as C ints: whole numbers, anything past 31 bits as the longest (or too many)."""
    window, sinks = operator.index(window), operator.index(sinks)
    if 1 <= window <= 0x7FFFFFFF and 0 <= sinks <= 0x7FFFFFFF:
        return window, sinks
    if window < 1:
        raise ValueError("window must be at least 1")
    if sinks < 0:
        raise ValueError("sinks must not be negative")
    return min(window, 0x7FFFFFFF), min(sinks, 0x7FFFFFFF)


def _window_geometry(q, k, v, window, sinks, cu_seqlens):
    dev, qs, ks = q.get_device(), q.shape, k.shape
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("q must be [B, S, Hq, D] and k, v [B, S, Hkv, D]")
    B, S, Hq, D = qs
    Hkv = ks[2]
    bf16 = torch.bfloat16
    if not (dev >= 0 and k.get_device() == dev and v.get_device() == dev and q.dtype is bf16 and k.dtype is bf16
            and v.dtype is bf16 and ks[0] == B and ks[1] == S and ks[3] == D and v.shape == ks and q.is_contiguous()
            and k.is_contiguous() and v.is_contiguous()):
        _check("q", q, dev, bf16)
        _check("k", k, dev, bf16, (B, S, Hkv, D))
        _check("v", v, dev, bf16, (B, S, Hkv, D))
    n_docs = 0
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, dev, torch.int32)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be [n_docs + 1]")
        n_docs = cu_seqlens.numel() - 1
    return (B, S, Hq, Hkv, D, *_window_size(window, sinks)), n_docs, dev


def _ws_bytes(n: int, what: str, *geometry) -> int:
    if n == 0:
        raise B_.UspError(B_.USP_ERR_UNSUPPORTED, f"{what}{geometry}: {B_.usp_last_error()}")
    return n


# (pure functions of the sizes)
@functools.lru_cache(maxsize=256)
def _window_ws(*geometry) -> int:
    return _ws_bytes(B_.usp_window_workspace_size(*geometry), "window attention", *geometry)


@functools.lru_cache(maxsize=256)
def _decode_ws(*geometry) -> int:
    return _ws_bytes(B_.usp_window_decode_workspace_size(*geometry), "window decode", *geometry)


def window_attn_fwd(q, k, v, window: int, sinks: int = 0, cu_seqlens=None, ws=None, out=None, lse=None, stream=None,
                    check_status: bool = False):
    """Causal attention with a sliding window and sinks over global-layout q [B, S, Hq, D], k/v
    [B, S, Hkv, D] (bf16): query i sees its own and the window - 1 keys before it, and the first
    `sinks` keys; with cu_seqlens ([n_docs + 1] int32, CUDA) all within its document. Returns
    (out bf16 like q, lse fp32 [B, S, Hq]). Elements must be finite, hidden ones too."""
    geo, n_docs, dev = _window_geometry(q, k, v, window, sinks, cu_seqlens)
    ctx, st = _on(dev, stream, q, k, v, cu_seqlens, ws, out, lse)
    with ctx:
        out = _like(out, "out", q, dev)
        lse = _lse_of(lse, q, geo[:3], dev)
        ws = _scratch(ws, B_.USP_WINDOW_FWD_WS, q, dev)
        B_.usp_window_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), *geo,
                               None if cu_seqlens is None else cu_seqlens.data_ptr(), n_docs, ws.data_ptr(), ws.numel(),
                               st)
        if check_status:
            check_workspace(ws, st)
    return out, lse


def window_attn_bwd(q, k, v, out, lse, dO, window: int, sinks: int = 0, cu_seqlens=None, ws=None, dq=None, dk=None,
                    dv=None, stream=None, check_status: bool = False):
    """Backward of window_attn_fwd from its out and lse; returns (dQ, dK, dV) in bf16, like q, k, v."""
    geo, n_docs, dev = _window_geometry(q, k, v, window, sinks, cu_seqlens)
    _check("out", out, dev, torch.bfloat16, q.shape)
    _check("dO", dO, dev, torch.bfloat16, q.shape)
    _check("lse", lse, dev, torch.float32, geo[:3])
    need = _window_ws(*geo, n_docs, 1)
    ctx, st = _on(dev, stream, q, k, v, out, lse, dO, cu_seqlens, ws, dq, dk, dv)
    with ctx:
        dq = _like(dq, "dq", q, dev)
        dk = _like(dk, "dk", k, dev)
        dv = _like(dv, "dv", v, dev)
        ws = _scratch(ws, need, q, dev)
        B_.usp_window_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                               dO.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *geo,
                               None if cu_seqlens is None else cu_seqlens.data_ptr(), n_docs, ws.data_ptr(), ws.numel(),
                               st)
        if check_status:
            check_workspace(ws, st)
    return dq, dk, dv


def window_attn_decode(q, k_cache, v_cache, lens, window: int, sinks: int = 0, ws=None, out=None, lse=None,
                       stream=None):
    """The attention of window_attn_fwd for the newest n tokens q [N, n, Hq, D] of N sequences whose
    caches k_cache, v_cache [N, cap, Hkv, D] (any strides, the last dimension contiguous) already hold
    them, lens [N] int32 (CUDA) tokens each. Returns (out bf16 like q, lse fp32 [N, n, Hq]); a token at
    a negative position (lens < n: an idle slot) gets out = 0, lse = -inf. Cache rows past lens are
    never read."""
    dev, qs, cs = q.get_device(), q.shape, k_cache.shape
    if len(qs) != 4 or len(cs) != 4:
        raise ValueError("q must be [N, n, Hq, D] and the caches [N, cap, Hkv, D]")
    N, n, Hq, D = qs
    _, cap, Hkv, _ = cs
    bf16 = torch.bfloat16
    if not (dev >= 0 and k_cache.get_device() == dev and v_cache.get_device() == dev and q.dtype is bf16
            and k_cache.dtype is bf16 and v_cache.dtype is bf16 and cs[0] == N and cs[3] == D and v_cache.shape == cs
            and q.is_contiguous()):
        _check("q", q, dev, bf16)
        _check("k_cache", k_cache, dev, bf16, (N, cap, Hkv, D), False)
        _check("v_cache", v_cache, dev, bf16, (N, cap, Hkv, D), False)
    _check("lens", lens, dev, torch.int32, (N,))
    ks, vs = k_cache.stride(), v_cache.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("the last dimension of the caches must be contiguous")
    geo = (N, n, cap, Hq, Hkv, D, *_window_size(window, sinks))
    need = _decode_ws(*geo)
    ctx, st = _on(dev, stream, q, k_cache, v_cache, lens, ws, out, lse)
    with ctx:
        out = _like(out, "out", q, dev)
        lse = _lse_of(lse, q, (N, n, Hq), dev)
        # (the smallest size: the splits join in the launch itself and need none)
        ws = _scratch(ws, need, q, dev) if ws is not None or need > 256 else None
        B_.usp_window_attn_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), lens.data_ptr(),
                                  out.data_ptr(), lse.data_ptr(), *geo, ks[:3], vs[:3],
                                  None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), st)
    return out, lse


def rope_axes(xs, positions, inv_freq, axis, paired: bool = False, inverse: bool = False, outs=None, stream=None):
    """Rotary positions with several axes of the tensors xs (one or a sequence, [B, S, H_x, D], bf16 or
    fp32, any strides with the last dimension contiguous, e.g. q and k sliced from a fused projection),
    in one launch: pair f of every head row turns by positions[axis[f]] * inv_freq[f]. positions
    [n_axes, B, S] int32 or int64 (CUDA); inv_freq [R/2] float64, up to 2^40 radians per step, and axis
    [R/2] int32 on the CPU (R <= D; elements from R on are copied). paired: pairs (2f, 2f + 1) instead of (f, f + R/2). inverse: the
    gradient's map. outs: where to write (may be xs: in place); else new contiguous tensors. Returns the
    list of outputs (one tensor for one tensor)."""
    single = isinstance(xs, torch.Tensor)
    xs = (xs,) if single else xs
    n = len(xs)
    if not 1 <= n <= B_.USP_MAX_ROPE_JOBS:
        raise ValueError(f"one to {B_.USP_MAX_ROPE_JOBS} tensors")
    if outs is not None:
        outs = (outs,) if single else outs
        if len(outs) != n:
            raise ValueError("one output per tensor")
    x0 = xs[0]
    dtype, dev = x0.dtype, x0.get_device()
    dt = _dt(x0)
    if x0.dim() != 4:
        raise ValueError("tensors must be [B, S, H, D]")
    B, S, _, D = x0.shape
    pos_type = positions.dtype
    if pos_type is not torch.int64 and pos_type is not torch.int32:
        raise TypeError("positions must be int32 or int64")
    _check("positions", positions, dev, pos_type)
    pos_shape = positions.shape
    if len(pos_shape) != 3 or pos_shape[1] != B or pos_shape[2] != S:
        raise ValueError(f"positions must be [n_axes, {B}, {S}]")
    if inv_freq.get_device() >= 0 or inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous 1-D float64 tensor on the CPU")
    if axis.get_device() >= 0 or axis.dtype is not torch.int32 or axis.dim() != 1 or not axis.is_contiguous():
        raise ValueError("axis must be a contiguous 1-D int32 tensor on the CPU")
    n_freq = inv_freq.numel()
    if n_freq != axis.numel():
        raise ValueError("inv_freq and axis must have one entry per frequency")
    ctx, st = _on(dev, stream, positions, *xs, *(outs or ()))
    with ctx:
        ys, jobs = [], []
        for j in range(n):
            x = xs[j]
            if x.dim() != 4:
                raise ValueError("tensors must be [B, S, H, D]")
            H = x.shape[2]
            _check("x", x, dev, dtype, (B, S, H, D), False)
            sx = x.stride()
            if outs is None:
                y = (torch.empty_like(x) if x.is_contiguous()
                     else torch.empty_like(x, memory_format=torch.contiguous_format))
                sy = (S * H * D, H * D, D, 1)
            else:
                y = outs[j]
                _check("out", y, dev, dtype, (B, S, H, D), False)
                sy = y.stride()
            if D > 1 and (sx[3] != 1 or sy[3] != 1):
                raise ValueError("the last dimension must be contiguous")
            ys.append(y)
            jobs.append((x.data_ptr(), y.data_ptr(), H, sx[:3], sy[:3]))
        B_.usp_rope_axes(jobs, B, S, D, 2 * n_freq, dt, positions.data_ptr(), 64 if pos_type is torch.int64 else 32,
                         pos_shape[0], inv_freq.data_ptr(), axis.data_ptr(), 1 if paired else 0, 1 if inverse else 0, st)
    return ys[0] if single else ys
