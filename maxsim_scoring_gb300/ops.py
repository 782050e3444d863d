"""PyTorch-facing binding of the MaxSim C ABI: argument marshalling only.

Every function here checks shapes / dtypes, allocates outputs and workspace
with torch on the tensors' device, and calls the entry point of the same name
in libmaxsim.so on that device's current CUDA stream. All arithmetic happens in
the CUDA kernels behind that call. The library launches on the calling thread's
current device: where the tensors are on another one, the call is made with
theirs current.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
from typing import Optional

import torch

from . import _native

_DT = {torch.float16: _native.F16, torch.bfloat16: _native.BF16}
_DT_ANY = {**_DT, torch.float32: _native.F32}
_U8 = torch.uint8


_SIZE_MAX = ctypes.c_size_t(-1).value

# The calling thread's current device (without the initialisation check of
# torch.cuda.current_device: asked only where a CUDA tensor is at hand).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _with_device(index: int, fn, *args, **kwargs):
    """fn(...) with device `index` current."""
    with torch.cuda.device(index):
        return fn(*args, **kwargs)


def _on_tensors_device(fn):
    """fn, run with the device of its first argument current."""
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, **kwargs):
        t = args[0] if args else kwargs.get(first)
        index = t.get_device() if isinstance(t, torch.Tensor) else -1
        if index >= 0 and index != _current_device():
            return _with_device(index, fn, *args, **kwargs)
        return fn(*args, **kwargs)
    return call


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _contig(t: Optional[torch.Tensor], name: str, dtype=None, device=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.contiguous()


def _mask(m: Optional[torch.Tensor], name: str, device):
    if m is None:
        return None
    if m.dtype == torch.bool:
        m = m.to(torch.uint8)
    return _contig(m, name, torch.uint8, device)


def workspace_size(op: int, Nq: int, Lq: int, Nd: int, Ld: int, dim: int) -> int:
    n = _native.lib().maxsim_workspace_size(op, Nq, Lq, Nd, Ld, dim)
    if n == ctypes_size_max():
        raise ValueError("invalid shape for maxsim_workspace_size")
    return int(n)


def ctypes_size_max() -> int:
    return _SIZE_MAX


def _workspace(nbytes: int, device, ws: Optional[torch.Tensor]):
    if nbytes == 0:
        return None, 0
    if ws is not None:
        if ws.device != device or not ws.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError(f"workspace needs {nbytes} bytes")
        return ws, ws.numel() * ws.element_size()
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, nbytes


@_on_tensors_device
def maxsim_fwd(Q: torch.Tensor, D: torch.Tensor, q_mask=None, d_mask=None, *, want_argmax: bool = False,
               scores: Optional[torch.Tensor] = None, argmax: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None):
    """scores [Nq, Nd] (and argmax [Nq*Nd, Lq] int32) for Q [Nq,Lq,d], D [Nd,Ld,d]."""
    if Q.dtype not in _DT or D.dtype != Q.dtype:
        raise TypeError("Q and D must both be float16 or both bfloat16")
    dev = Q.device
    Q, D = _contig(Q, "Q"), _contig(D, "D", device=dev)
    Nq, Lq, dim = Q.shape
    Nd, Ld, dim2 = D.shape
    if dim2 != dim:
        raise ValueError("Q and D embedding dimensions differ")
    qm, dm = _mask(q_mask, "q_mask", dev), _mask(d_mask, "d_mask", dev)
    if scores is None:
        scores = torch.empty((Nq, Nd), dtype=torch.float32, device=dev)
    if want_argmax and argmax is None:
        argmax = torch.empty((Nq * Nd, Lq), dtype=torch.int32, device=dev)
    ws, nbytes = _workspace(workspace_size(_native.OP_FWD, Nq, Lq, Nd, Ld, dim), dev, workspace)
    rc = _native.lib().maxsim_fwd(_ptr(Q), _ptr(D), _DT[Q.dtype], Nq, Lq, Nd, Ld, dim, _ptr(qm), _ptr(dm),
                                  _ptr(scores), _ptr(argmax), _ptr(ws), nbytes, _stream(dev))
    _native.check(rc, "maxsim_fwd")
    return scores, argmax


@_on_tensors_device
def maxsim_fwd_varlen(Q: torch.Tensor, cu_seqlens_q: Optional[torch.Tensor], max_lq: int, D: torch.Tensor,
                      cu_seqlens_d: torch.Tensor, q_mask=None, d_mask=None, *, want_argmax: bool = False,
                      scores: Optional[torch.Tensor] = None, argmax: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None):
    """Packed documents D [total_d, d] with cu_seqlens_d [Nd+1] (int32).

    Q is dense [Nq, max_lq, d] when cu_seqlens_q is None, else packed
    [total_q, d]. Returns scores [Nq, Nd] (and argmax [Nq*Nd, max_lq]).
    """
    if Q.dtype not in _DT or D.dtype != Q.dtype:
        raise TypeError("Q and D must both be float16 or both bfloat16")
    dev = Q.device
    Q, D = _contig(Q, "Q"), _contig(D, "D", device=dev)
    cu_d = _contig(cu_seqlens_d, "cu_seqlens_d", torch.int32, dev)
    cu_q = _contig(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev)
    dim = Q.shape[-1]
    if D.dim() != 2 or D.shape[1] != dim:
        raise ValueError("D must be packed [total_d, dim]")
    Nd = cu_d.numel() - 1
    Nq = (cu_q.numel() - 1) if cu_q is not None else Q.shape[0]
    if cu_q is None and (Q.dim() != 3 or Q.shape[1] != max_lq):
        raise ValueError("dense Q must be [Nq, max_lq, dim]")
    total_d = D.shape[0]
    qm, dm = _mask(q_mask, "q_mask", dev), _mask(d_mask, "d_mask", dev)
    if scores is None:
        scores = torch.empty((Nq, Nd), dtype=torch.float32, device=dev)
    if want_argmax and argmax is None:
        argmax = torch.empty((Nq * Nd, max_lq), dtype=torch.int32, device=dev)
    ws, nbytes = _workspace(workspace_size(_native.OP_FWD_VARLEN, Nq, max_lq, Nd, total_d, dim), dev, workspace)
    rc = _native.lib().maxsim_fwd_varlen(_ptr(Q), _ptr(cu_q), max_lq, _ptr(D), _ptr(cu_d), total_d, _DT[Q.dtype], Nq,
                                         Nd, dim, _ptr(qm), _ptr(dm), _ptr(scores), _ptr(argmax), _ptr(ws), nbytes,
                                         _stream(dev))
    _native.check(rc, "maxsim_fwd_varlen")
    return scores, argmax


@_on_tensors_device
def maxsim_score_pairs_packed(Q: torch.Tensor, cu_seqlens_q: Optional[torch.Tensor], max_lq: int, D: torch.Tensor,
                              cu_seqlens_d: torch.Tensor, pairs: torch.Tensor, q_mask=None, d_mask=None, *,
                              want_argmax: bool = False, scores: Optional[torch.Tensor] = None,
                              argmax: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Scores of the (query, document) pairs `pairs` [num_pairs, 2] (int32)
    over the packed batches of maxsim_fwd_varlen. Returns scores [num_pairs]
    (and argmax [num_pairs, max_lq])."""
    if Q.dtype not in _DT or D.dtype != Q.dtype:
        raise TypeError("Q and D must both be float16 or both bfloat16")
    dev = Q.device
    Q, D = _contig(Q, "Q"), _contig(D, "D", device=dev)
    cu_d = _contig(cu_seqlens_d, "cu_seqlens_d", torch.int32, dev)
    cu_q = _contig(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev)
    pr = _contig(pairs, "pairs", torch.int32, dev)
    if pr.dim() != 2 or pr.shape[1] != 2:
        raise ValueError("pairs must be [num_pairs, 2]")
    dim = Q.shape[-1]
    if D.dim() != 2 or D.shape[1] != dim:
        raise ValueError("D must be packed [total_d, dim]")
    Nd = cu_d.numel() - 1
    Nq = (cu_q.numel() - 1) if cu_q is not None else Q.shape[0]
    if cu_q is None and (Q.dim() != 3 or Q.shape[1] != max_lq):
        raise ValueError("dense Q must be [Nq, max_lq, dim]")
    total_d, n = D.shape[0], pr.shape[0]
    qm, dm = _mask(q_mask, "q_mask", dev), _mask(d_mask, "d_mask", dev)
    if scores is None:
        scores = torch.empty((n,), dtype=torch.float32, device=dev)
    if want_argmax and argmax is None:
        argmax = torch.empty((n, max_lq), dtype=torch.int32, device=dev)
    ws, nbytes = _workspace(workspace_size(_native.OP_SCORE_PAIRS, Nq, max_lq, Nd, n, dim), dev, workspace)
    rc = _native.lib().maxsim_score_pairs_packed(_ptr(Q), _ptr(cu_q), max_lq, _ptr(D), _ptr(cu_d), total_d,
                                                 _DT[Q.dtype], Nq, Nd, dim, _ptr(qm), _ptr(dm), _ptr(pr), n,
                                                 _ptr(scores), _ptr(argmax), _ptr(ws), nbytes, _stream(dev))
    _native.check(rc, "maxsim_score_pairs_packed")
    return scores, argmax


@_on_tensors_device
def maxsim_bwd(Q: torch.Tensor, D: torch.Tensor, argmax: torch.Tensor, grad_scores: torch.Tensor, q_mask=None, *,
               want_dq: bool = True, want_dd: bool = True, want_csr: bool = False,
               dQ: Optional[torch.Tensor] = None, dD: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None):
    """dQ [Nq,Lq,d] f32, dD [Nd,Ld,d] f32 (and the CSR row_ptr / col)."""
    if Q.dtype not in _DT or D.dtype != Q.dtype:
        raise TypeError("Q and D must both be float16 or both bfloat16")
    dev = Q.device
    Q, D = _contig(Q, "Q"), _contig(D, "D", device=dev)
    Nq, Lq, dim = Q.shape
    Nd, Ld, _ = D.shape
    am = _contig(argmax, "argmax", torch.int32, dev)
    g = _contig(grad_scores, "grad_scores", torch.float32, dev)
    if am.numel() != Nq * Nd * Lq or g.numel() != Nq * Nd:
        raise ValueError("argmax must be [Nq*Nd, Lq] and grad_scores [Nq, Nd]")
    qm = _mask(q_mask, "q_mask", dev)
    if dQ is None and want_dq:
        dQ = torch.empty((Nq, Lq, dim), dtype=torch.float32, device=dev)
    if dD is None and want_dd:
        dD = torch.empty((Nd, Ld, dim), dtype=torch.float32, device=dev)
    for t, shape, name in ((dQ, (Nq, Lq, dim), "dQ"), (dD, (Nd, Ld, dim), "dD")):
        if t is not None and (tuple(t.shape) != shape or t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape {shape}")
    row_ptr = torch.empty(Nd * Ld + 1, dtype=torch.int32, device=dev) if want_csr else None
    col = torch.empty(max(1, Nq * Nd * Lq), dtype=torch.int32, device=dev) if want_csr else None
    ws, nbytes = _workspace(workspace_size(_native.OP_BWD, Nq, Lq, Nd, Ld, dim), dev, workspace)
    rc = _native.lib().maxsim_bwd(_ptr(Q), _ptr(D), _DT[Q.dtype], Nq, Lq, Nd, Ld, dim, _ptr(qm), _ptr(am), _ptr(g),
                                  _ptr(dQ), _ptr(dD), _ptr(row_ptr), _ptr(col), _ptr(ws), nbytes, _stream(dev))
    _native.check(rc, "maxsim_bwd")
    return dQ, dD, row_ptr, col


@_on_tensors_device
def maxsim_bwd_varlen(Q: torch.Tensor, cu_seqlens_q: Optional[torch.Tensor], max_lq: int, D: torch.Tensor,
                      cu_seqlens_d: torch.Tensor, max_ld: int, argmax: torch.Tensor, grad_scores: torch.Tensor,
                      q_mask=None, *, want_dq: bool = True, want_dd: bool = True, want_csr: bool = False,
                      workspace: Optional[torch.Tensor] = None):
    """Gradient of maxsim_fwd_varlen: dQ in Q's layout, dD [total_d, d] (f32),
    and optionally the CSR (row_ptr over D's packed rows, col)."""
    if Q.dtype not in _DT or D.dtype != Q.dtype:
        raise TypeError("Q and D must both be float16 or both bfloat16")
    dev = Q.device
    Q, D = _contig(Q, "Q"), _contig(D, "D", device=dev)
    cu_q = _contig(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev)
    cu_d = _contig(cu_seqlens_d, "cu_seqlens_d", torch.int32, dev)
    dim = Q.shape[-1]
    Nq = (cu_q.numel() - 1) if cu_q is not None else Q.shape[0]
    Nd = cu_d.numel() - 1
    total_d = D.shape[0]
    am = _contig(argmax, "argmax", torch.int32, dev)
    g = _contig(grad_scores, "grad_scores", torch.float32, dev)
    if am.numel() != Nq * Nd * max_lq or g.numel() != Nq * Nd:
        raise ValueError("argmax must be [Nq*Nd, max_lq] and grad_scores [Nq, Nd]")
    qm = _mask(q_mask, "q_mask", dev)
    dQ = torch.empty(Q.shape, dtype=torch.float32, device=dev) if want_dq else None
    dD = torch.empty((total_d, dim), dtype=torch.float32, device=dev) if want_dd else None
    row_ptr = torch.empty(total_d + 1, dtype=torch.int32, device=dev) if want_csr else None
    col = torch.empty(max(1, Nq * Nd * max_lq), dtype=torch.int32, device=dev) if want_csr else None
    ws, nbytes = _workspace(workspace_size(_native.OP_BWD_VARLEN, Nq, max_lq, Nd, total_d, dim), dev, workspace)
    rc = _native.lib().maxsim_bwd_varlen(_ptr(Q), _ptr(cu_q), max_lq, _ptr(D), _ptr(cu_d), total_d, max_ld,
                                         _DT[Q.dtype], Nq, Nd, dim, _ptr(qm), _ptr(am), _ptr(g), _ptr(dQ), _ptr(dD),
                                         _ptr(row_ptr), _ptr(col), _ptr(ws), nbytes, _stream(dev))
    _native.check(rc, "maxsim_bwd_varlen")
    return dQ, dD, row_ptr, col


@_on_tensors_device
def maxsim_fwd_int8(Q: torch.Tensor, q_scale: torch.Tensor, D: torch.Tensor, d_scale: torch.Tensor, q_mask=None,
                    d_mask=None, *, want_argmax: bool = False, want_win_dot: bool = False,
                    scores: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """INT8 x INT8 scores [Nq, Nd] with per-token float32 scales."""
    dev = Q.device
    Q = _contig(Q, "Q", torch.int8)
    D = _contig(D, "D", torch.int8, dev)
    qs = _contig(q_scale, "q_scale", torch.float32, dev)
    ds = _contig(d_scale, "d_scale", torch.float32, dev)
    Nq, Lq, dim = Q.shape
    Nd, Ld, _ = D.shape
    qm, dm = _mask(q_mask, "q_mask", dev), _mask(d_mask, "d_mask", dev)
    if scores is None:
        scores = torch.empty((Nq, Nd), dtype=torch.float32, device=dev)
    argmax = torch.empty((Nq * Nd, Lq), dtype=torch.int32, device=dev) if (want_argmax or want_win_dot) else None
    win = torch.empty((Nq * Nd, Lq), dtype=torch.int32, device=dev) if want_win_dot else None
    ws, nbytes = _workspace(workspace_size(_native.OP_FWD_INT8, Nq, Lq, Nd, Ld, dim), dev, workspace)
    rc = _native.lib().maxsim_fwd_int8(_ptr(Q), _ptr(qs), _ptr(D), _ptr(ds), Nq, Lq, Nd, Ld, dim, _ptr(qm), _ptr(dm),
                                       _ptr(scores), _ptr(argmax), _ptr(win), _ptr(ws), nbytes, _stream(dev))
    _native.check(rc, "maxsim_fwd_int8")
    return scores, argmax, win


def _points(P: torch.Tensor, Q: torch.Tensor):
    if P.dim() != 3 or Q.dim() != 3 or P.shape[0] != Q.shape[0] or P.shape[2] != Q.shape[2]:
        raise ValueError("P must be [B, N, dim] and Q [B, M, dim]")
    dev = P.device
    return _contig(P, "P", torch.float32), _contig(Q, "Q", torch.float32, dev), dev


@_on_tensors_device
def chamfer_fwd(P: torch.Tensor, Q: torch.Tensor, *, workspace: Optional[torch.Tensor] = None):
    """Chamfer distance of B pairs of point sets P [B,N,dim], Q [B,M,dim] (f32).

    Returns (loss [B], dist_p [B,N], idx_p [B,N] i32, dist_q [B,M], idx_q [B,M] i32).
    """
    P, Q, dev = _points(P, Q)
    B, N, dim = P.shape
    M = Q.shape[1]
    loss = torch.empty(B, dtype=torch.float32, device=dev)
    dist_p = torch.empty((B, N), dtype=torch.float32, device=dev)
    idx_p = torch.empty((B, N), dtype=torch.int32, device=dev)
    dist_q = torch.empty((B, M), dtype=torch.float32, device=dev)
    idx_q = torch.empty((B, M), dtype=torch.int32, device=dev)
    ws, nbytes = _workspace(workspace_size(_native.OP_CHAMFER_FWD, B, N, M, 0, dim), dev, workspace)
    rc = _native.lib().maxsim_chamfer_fwd(_ptr(P), _ptr(Q), B, N, M, dim, _ptr(dist_p), _ptr(idx_p), _ptr(dist_q),
                                          _ptr(idx_q), _ptr(loss), _ptr(ws), nbytes, _stream(dev))
    _native.check(rc, "maxsim_chamfer_fwd")
    return loss, dist_p, idx_p, dist_q, idx_q


@_on_tensors_device
def chamfer_bwd(P: torch.Tensor, Q: torch.Tensor, idx_p: torch.Tensor, idx_q: torch.Tensor, grad_loss: torch.Tensor,
                *, dP: Optional[torch.Tensor] = None, dQ: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None):
    """(dP [B,N,dim], dQ [B,M,dim]) f32 of sum_b grad_loss[b] * CD(P_b, Q_b)."""
    P, Q, dev = _points(P, Q)
    B, N, dim = P.shape
    M = Q.shape[1]
    ip = _contig(idx_p, "idx_p", torch.int32, dev)
    iq = _contig(idx_q, "idx_q", torch.int32, dev)
    g = _contig(grad_loss, "grad_loss", torch.float32, dev)
    if ip.numel() != B * N or iq.numel() != B * M or g.numel() != B:
        raise ValueError("idx_p must be [B, N], idx_q [B, M] and grad_loss [B]")
    if dP is None:
        dP = torch.empty((B, N, dim), dtype=torch.float32, device=dev)
    if dQ is None:
        dQ = torch.empty((B, M, dim), dtype=torch.float32, device=dev)
    for t, shape, name in ((dP, (B, N, dim), "dP"), (dQ, (B, M, dim), "dQ")):
        if tuple(t.shape) != shape or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape {shape}")
    ws, nbytes = _workspace(workspace_size(_native.OP_CHAMFER_BWD, B, N, M, 0, dim), dev, workspace)
    rc = _native.lib().maxsim_chamfer_bwd(_ptr(P), _ptr(Q), B, N, M, dim, _ptr(ip), _ptr(iq), _ptr(g), _ptr(dP),
                                          _ptr(dQ), _ptr(ws), nbytes, _stream(dev))
    _native.check(rc, "maxsim_chamfer_bwd")
    return dP, dQ


@_on_tensors_device
def maxsim_topk(scores: torch.Tensor, k: int):
    """(values [R, k] f32, indices [R, k] i32): the k largest entries of every
    row of scores [R, n] (f32), descending, the lower index first among ties."""
    s = _contig(scores, "scores", torch.float32)
    if s.dim() != 2:
        raise ValueError("scores must be [rows, n]")
    R, n = s.shape
    idx = torch.empty((R, k), dtype=torch.int32, device=s.device)
    vals = torch.empty((R, k), dtype=torch.float32, device=s.device)
    rc = _native.lib().maxsim_topk(_ptr(s), R, n, k, _ptr(idx), _ptr(vals), _stream(s.device))
    _native.check(rc, "maxsim_topk")
    return vals, idx


@_on_tensors_device
def maxsim_two_stage_topk(Q8: torch.Tensor, q_scale: torch.Tensor, D8: torch.Tensor, d_scale: torch.Tensor,
                          Q16: torch.Tensor, D16: torch.Tensor, k1: int, k: int, *, want_stage1: bool = False,
                          workspace: Optional[torch.Tensor] = None):
    """Two-stage INT8 -> f16 / bf16 top-k: (top_idx [Nq,k] i32, top_scores [Nq,k] f32,
    stage1_scores [Nq,Nd] or None, candidates [Nq,k1] or None)."""
    dev = Q8.device
    Q8 = _contig(Q8, "Q8", torch.int8)
    D8 = _contig(D8, "D8", torch.int8, dev)
    qs = _contig(q_scale, "q_scale", torch.float32, dev)
    ds = _contig(d_scale, "d_scale", torch.float32, dev)
    if Q16.dtype not in _DT or D16.dtype != Q16.dtype:
        raise TypeError("Q16 and D16 must both be float16 or both bfloat16")
    Q16, D16 = _contig(Q16, "Q16", device=dev), _contig(D16, "D16", device=dev)
    Nq, Lq, dim = Q8.shape
    Nd, Ld, _ = D8.shape
    if tuple(Q16.shape) != (Nq, Lq, dim) or tuple(D16.shape) != (Nd, Ld, dim):
        raise ValueError("Q16 / D16 must have the shapes of Q8 / D8")
    top_idx = torch.empty((Nq, k), dtype=torch.int32, device=dev)
    top_scores = torch.empty((Nq, k), dtype=torch.float32, device=dev)
    s8 = torch.empty((Nq, Nd), dtype=torch.float32, device=dev) if want_stage1 else None
    cand = torch.empty((Nq, k1), dtype=torch.int32, device=dev) if want_stage1 else None
    ws, nbytes = _workspace(workspace_size(_native.OP_TWO_STAGE, Nq, Lq, Nd, Ld, dim), dev, workspace)
    rc = _native.lib().maxsim_two_stage_topk(_ptr(Q8), _ptr(qs), _ptr(D8), _ptr(ds), _ptr(Q16), _ptr(D16),
                                             _DT[Q16.dtype], Nq, Lq, Nd, Ld, dim, k1, k, _ptr(top_idx),
                                             _ptr(top_scores), _ptr(s8), _ptr(cand), _ptr(ws), nbytes, _stream(dev))
    _native.check(rc, "maxsim_two_stage_topk")
    return top_idx, top_scores, s8, cand


@_on_tensors_device
def maxsim_fwd_streamed(Q: torch.Tensor, D_host: torch.Tensor, q_mask=None, *, block_docs: int = 20_000,
                        scores: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Scores [Nq, Nd] of a device query batch Q [Nq,Lq,d] against a corpus
    D_host [Nd,Ld,d] in host memory (pin it for copy/compute overlap),
    streamed in blocks of block_docs documents. The copies are asynchronous:
    keep D_host alive and unchanged until the current stream has passed this
    call (synchronise, or wait on an event recorded after it)."""
    if Q.dtype not in _DT or D_host.dtype != Q.dtype:
        raise TypeError("Q and D_host must both be float16 or both bfloat16")
    if D_host.is_cuda or not D_host.is_contiguous():
        raise ValueError("D_host must be a contiguous host tensor")
    dev = Q.device
    Q = _contig(Q, "Q")
    Nq, Lq, dim = Q.shape
    Nd, Ld, _ = D_host.shape
    qm = _mask(q_mask, "q_mask", dev)
    if scores is None:
        scores = torch.empty((Nq, Nd), dtype=torch.float32, device=dev)
    ws, nbytes = _workspace(workspace_size(_native.OP_FWD_STREAMED, Nq, Lq, min(block_docs, max(Nd, 1)), Ld, dim),
                            dev, workspace)
    rc = _native.lib().maxsim_fwd_streamed(_ptr(Q), D_host.data_ptr(), _DT[Q.dtype], Nq, Lq, Nd, Ld, dim, block_docs,
                                           _ptr(qm), _ptr(scores), _ptr(ws), nbytes, _stream(dev))
    _native.check(rc, "maxsim_fwd_streamed")
    return scores


@_on_tensors_device
def maxsim_fwd_varlen_streamed(Q: torch.Tensor, cu_seqlens_q: Optional[torch.Tensor], max_lq: int,
                               D_host: torch.Tensor, cu_seqlens_d_host: torch.Tensor, q_mask=None, *,
                               block_docs: int = 20_000, block_tokens: int = 1 << 22,
                               scores: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Scores [Nq, Nd] of device queries against a packed corpus in host
    memory: D_host [total_d, d] rows and cu_seqlens_d_host [Nd+1] (int32, host),
    streamed in blocks of whole documents. Keep the host tensors alive and
    unchanged until the current stream has passed this call."""
    if Q.dtype not in _DT or D_host.dtype != Q.dtype:
        raise TypeError("Q and D_host must both be float16 or both bfloat16")
    if D_host.is_cuda or cu_seqlens_d_host.is_cuda or not D_host.is_contiguous():
        raise ValueError("D_host and cu_seqlens_d_host must be contiguous host tensors")
    if cu_seqlens_d_host.dtype != torch.int32 or not cu_seqlens_d_host.is_contiguous():
        raise TypeError("cu_seqlens_d_host must be a contiguous int32 host tensor")
    dev = Q.device
    Q = _contig(Q, "Q")
    cu_q = _contig(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev)
    dim = Q.shape[-1]
    Nq = (cu_q.numel() - 1) if cu_q is not None else Q.shape[0]
    Nd = cu_seqlens_d_host.numel() - 1
    total_d = D_host.shape[0]
    qm = _mask(q_mask, "q_mask", dev)
    if scores is None:
        scores = torch.empty((Nq, Nd), dtype=torch.float32, device=dev)
    bd = min(block_docs, max(Nd, 1))
    ws, nbytes = _workspace(workspace_size(_native.OP_FWD_VARLEN_STREAMED, Nq, max_lq, bd, block_tokens, dim), dev,
                            workspace)
    rc = _native.lib().maxsim_fwd_varlen_streamed(_ptr(Q), _ptr(cu_q), max_lq, D_host.data_ptr(),
                                                  cu_seqlens_d_host.data_ptr(), total_d, _DT[Q.dtype], Nq, Nd, dim,
                                                  _ptr(qm), block_docs, block_tokens, _ptr(scores), _ptr(ws), nbytes,
                                                  _stream(dev))
    _native.check(rc, "maxsim_fwd_varlen_streamed")
    return scores


# The handle of a device's current stream, without the Stream object of
# torch.cuda.current_stream (2 us of a small call).
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _rows(t: torch.Tensor, name: str):
    """(tensor, rows, row stride) of a CUDA tensor [..., cols] whose rows the
    library can read in place; copied where its strides do not allow it."""
    shape = t.shape
    if t.is_contiguous():
        if len(shape) == 2:
            return t, shape[0], shape[1]
    else:
        # rows one fixed stride apart (a slice of a wider buffer) are read where they are
        cols = shape[-1]
        ld = t.stride(-2) if len(shape) > 1 else cols
        if cols and t.stride(-1) == 1 and ld >= cols and all(
                t.stride(i) == t.stride(i + 1) * shape[i + 1] for i in range(len(shape) - 2)):
            return t, t.numel() // cols, ld
        t = t.contiguous()
    if not shape:
        raise ValueError(f"{name} must have at least one dimension")
    cols = shape[-1]
    return t, (t.numel() // cols if cols else shape[:-1].numel()), cols


def _device(t: torch.Tensor, name: str) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


def _given(out: torch.Tensor, name: str, shape, dtype, device):
    """The caller's output buffer, checked."""
    if out.shape != shape or out.dtype != dtype or out.device != device or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return out


def quantize_rows(x: torch.Tensor, *, normalize: bool = False, q: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None):
    """(q int8, scale f32): symmetric INT8 codes of x [..., K] (f16 / bf16 / f32)
    with one scale for each row; q * scale[..., None] is the quantised row, or
    with `normalize` the quantised row of unit L2 length."""
    dt = _DT_ANY.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be float16, bfloat16 or float32, got {x.dtype}")
    index, shape, dev = _device(x, "x"), x.shape, x.device
    if index != _current_device():
        return _with_device(index, quantize_rows, x, normalize=normalize, q=q, scale=scale)
    x, rows, ld = _rows(x, "x")
    cols = shape[-1]
    q = torch.empty(shape, dtype=torch.int8, device=dev) if q is None else _given(q, "q", shape, torch.int8, dev)
    scale = (torch.empty(shape[:-1], dtype=torch.float32, device=dev) if scale is None
             else _given(scale, "scale", shape[:-1], torch.float32, dev))
    rc = _native.lib().maxsim_quantize_rows(x.data_ptr(), dt, rows, cols, ld, 1 if normalize else 0, q.data_ptr(),
                                            cols, scale.data_ptr(), _raw_stream(index))
    if rc:
        _native.check(rc, "maxsim_quantize_rows")
    return q, scale


def linear_int8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                bias: Optional[torch.Tensor] = None, *, out_dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """[..., N] in out_dtype: (x @ w.T) * x_scale[..., None] * w_scale + bias for
    int8 x [..., K] with a scale for each row and int8 w [N, K] with a scale for
    each channel (as quantize_rows gives them); x_scale, w_scale and bias [N] f32."""
    dt = _DT_ANY.get(out_dtype)
    if dt is None:
        raise TypeError(f"out_dtype must be float16, bfloat16 or float32, got {out_dtype}")
    if x.dtype is not torch.int8 or w.dtype is not torch.int8:
        raise TypeError("x and w must be int8")
    if x_scale.dtype is not torch.float32 or w_scale.dtype is not torch.float32:
        raise TypeError("x_scale, w_scale and bias must be float32")
    index, shape, channels = _device(x, "x"), x.shape, w.shape
    if index != _current_device():
        return _with_device(index, linear_int8, x, x_scale, w, w_scale, bias, out_dtype=out_dtype, out=out,
                            workspace=workspace)
    if w.get_device() != index or x_scale.get_device() != index or w_scale.get_device() != index:
        raise ValueError("x, w, their scales and bias must be on one device")
    if len(channels) != 2 or not shape or shape[-1] != channels[1]:
        raise ValueError("w must be [N, K] with x's K")
    lead, (N, K), channels = shape[:-1], channels, channels[:1]
    if x_scale.shape != lead or w_scale.shape != channels:
        raise ValueError("x_scale must have x's leading shape, w_scale and bias [N]")
    x, M, ld_x = _rows(x, "x")
    w, _, ld_w = _rows(w, "w")
    if not x_scale.is_contiguous():
        x_scale = x_scale.contiguous()
    if not w_scale.is_contiguous():
        w_scale = w_scale.contiguous()
    pb = None
    if bias is not None:
        if bias.dtype is not torch.float32:
            raise TypeError("x_scale, w_scale and bias must be float32")
        if bias.get_device() != index:
            raise ValueError("x, w, their scales and bias must be on one device")
        if bias.shape != channels:
            raise ValueError("x_scale must have x's leading shape, w_scale and bias [N]")
        if not bias.is_contiguous():
            bias = bias.contiguous()
        pb = bias.data_ptr()
    full, dev = lead + channels, x.device
    out = torch.empty(full, dtype=out_dtype, device=dev) if out is None else _given(out, "out", full, out_dtype, dev)
    px, pw, lib, stream = x.data_ptr(), w.data_ptr(), _native.lib(), _raw_stream(index)
    px_scale, pw_scale, p_out = x_scale.data_ptr(), w_scale.data_ptr(), out.data_ptr()
    # few tokens and small products need no workspace: its size is asked for once a call says that it is missing
    rc = (lib.maxsim_linear_int8(px, ld_x, px_scale, pw, ld_w, pw_scale, pb, M, N, K, dt, p_out, N, None, 0, stream)
          if M <= 32 or M * N * K <= 1 << 29 else _native.ERR_WORKSPACE)
    if rc == _native.ERR_WORKSPACE:
        need = lib.maxsim_workspace_size(_native.OP_LINEAR_INT8, M, N, K, ld_x if px % 16 == 0 else 1,
                                         ld_w if ld_w and pw % 16 == 0 else 1)
        if need == _SIZE_MAX:
            _native.check(2, "maxsim_linear_int8")
        ws, nbytes = _workspace(need, dev, workspace)
        rc = lib.maxsim_linear_int8(px, ld_x, px_scale, pw, ld_w, pw_scale, pb, M, N, K, dt, p_out, N,
                                    None if ws is None else ws.data_ptr(), nbytes, stream)
    if rc:
        _native.check(rc, "maxsim_linear_int8")
    return out


def dropout_fwd(x: torch.Tensor, p: float, seed: int, offset: int = 0, residual: Optional[torch.Tensor] = None, *,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x with each element dropped with probability p (in steps of 2**-16) and
    the kept ones scaled by 1 / (1 - p), plus `residual` where given. The mask
    is a function of (seed, offset) and the element's place alone: the backward
    draws it again, and calls that need independent masks take other offsets."""
    dt = _DT_ANY.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be float16, bfloat16 or float32, got {x.dtype}")
    index, shape, dev = _device(x, "x"), x.shape, x.device
    if index != _current_device():
        return _with_device(index, dropout_fwd, x, p, seed, offset, residual, out=out)
    pr, ld_r = None, 0
    if residual is not None:
        if residual.shape != shape or residual.dtype is not x.dtype or residual.get_device() != index:
            raise ValueError("residual must have x's shape, dtype and device")
        residual, _, ld_r = _rows(residual, "residual")
        pr = residual.data_ptr()
    x, rows, ld = _rows(x, "x")
    cols = shape[-1]
    out = torch.empty(shape, dtype=x.dtype, device=dev) if out is None else _given(out, "out", shape, x.dtype, dev)
    rc = _native.lib().maxsim_dropout_fwd(x.data_ptr(), dt, rows, cols, ld, pr, ld_r, p, seed, offset, out.data_ptr(),
                                          cols, _raw_stream(index))
    if rc:
        _native.check(rc, "maxsim_dropout_fwd")
    return out


def dropout_bwd(grad: torch.Tensor, p: float, seed: int, offset: int = 0, *,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient in x of dropout_fwd(x, p, seed, offset) (that in `residual`
    is grad itself)."""
    dt = _DT_ANY.get(grad.dtype)
    if dt is None:
        raise TypeError(f"grad must be float16, bfloat16 or float32, got {grad.dtype}")
    index, shape, dev = _device(grad, "grad"), grad.shape, grad.device
    if index != _current_device():
        return _with_device(index, dropout_bwd, grad, p, seed, offset, out=out)
    grad, rows, ld = _rows(grad, "grad")
    cols = shape[-1]
    out = (torch.empty(shape, dtype=grad.dtype, device=dev) if out is None
           else _given(out, "out", shape, grad.dtype, dev))
    rc = _native.lib().maxsim_dropout_bwd(grad.data_ptr(), dt, rows, cols, ld, p, seed, offset, out.data_ptr(), cols,
                                          _raw_stream(index))
    if rc:
        _native.check(rc, "maxsim_dropout_bwd")
    return out


def _fp4_rows(q: torch.Tensor, block_scale: torch.Tensor, scale: Optional[torch.Tensor], name: str, block: int, index: int):
    """(pointer, rows, row stride in bytes, block scales' pointer, row scales' pointer, the tensors) of 4-bit rows, checked."""
    if block != 16 and block != 32:
        raise ValueError("block must be 16 or 32")
    if q.dtype is not _U8 or block_scale.dtype is not _U8:
        raise TypeError(f"{name} and its block scales must be uint8")
    if q.get_device() != index or block_scale.get_device() != index:
        raise ValueError(f"{name} and its scales must be on one device with the other operands")
    shape = q.shape
    if not shape or shape[-1] & 15:
        raise ValueError(f"{name} must have rows of whole 16-byte pieces")
    width = shape[-1]
    if width and q.is_contiguous():
        rows, ld = q.numel() // width, width
    else:
        q, rows, ld = _rows(q, name)
    ptr = q.data_ptr()
    if ptr & 15 or (ld & 15 and rows > 1):
        q, ld = q.clone(memory_format=torch.contiguous_format), width
        ptr = q.data_ptr()
    tiles = ((rows + 127) >> 7, (2 * width + 4 * block - 1) // (4 * block), 32, 4, 4)
    if block_scale.shape != tiles:
        raise ValueError(f"{name}'s block scales must be {tiles}, got {tuple(block_scale.shape)}")
    p_block = block_scale.data_ptr()
    if p_block & 15 or not block_scale.is_contiguous():
        block_scale = block_scale.clone(memory_format=torch.contiguous_format)
        p_block = block_scale.data_ptr()
    p_scale = None
    if scale is not None:
        if scale.dtype is not torch.float32:
            raise TypeError(f"{name}'s row scales must be float32")
        if scale.get_device() != index:
            raise ValueError(f"{name} and its scales must be on one device with the other operands")
        if scale.shape != shape[:-1]:
            raise ValueError(f"{name}'s row scales must have its leading shape")
        if not scale.is_contiguous():
            scale = scale.contiguous()
        p_scale = scale.data_ptr()
    return ptr, rows, ld, p_block, p_scale, (q, block_scale, scale)


def quantize_rows_fp4(x: torch.Tensor, *, block: int = 16, q: Optional[torch.Tensor] = None,
                      block_scale: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None):
    """(q, block_scale, scale): rows of x [..., K] (f16 / bf16 / f32) as 4-bit
    floating point (E2M1) with a scale for every `block` values: 16 (E4M3 scales,
    and one f32 power of two for each row) or 32 (E8M0 scales; scale is None).
    q is uint8 [..., ceil(K / 32) * 16], two codes a byte; block_scale is uint8
    [row tiles, words, 32, 4, 4], laid out as the tensor cores read it."""
    dt = _DT_ANY.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be float16, bfloat16 or float32, got {x.dtype}")
    if block != 16 and block != 32:
        raise ValueError("block must be 16 or 32")
    if block == 32 and scale is not None:
        raise ValueError("rows in blocks of 32 have no scale of their own")
    index, shape, dev = _device(x, "x"), x.shape, x.device
    if index != _current_device():
        return _with_device(index, quantize_rows_fp4, x, block=block, q=q, block_scale=block_scale, scale=scale)
    x, rows, ld = _rows(x, "x")
    cols = shape[-1]
    width, tiles = (cols + 31) // 32 * 16, ((rows + 127) // 128, (cols + 4 * block - 1) // (4 * block), 32, 4, 4)
    q_shape = (*shape[:-1], width)
    q = torch.empty(q_shape, dtype=torch.uint8, device=dev) if q is None else _given(q, "q", q_shape, torch.uint8, dev)
    block_scale = (torch.empty(tiles, dtype=torch.uint8, device=dev) if block_scale is None
                   else _given(block_scale, "block_scale", tiles, torch.uint8, dev))
    ps = None
    if block == 16:
        scale = (torch.empty(shape[:-1], dtype=torch.float32, device=dev) if scale is None
                 else _given(scale, "scale", shape[:-1], torch.float32, dev))
        ps = scale.data_ptr()
    rc = _native.lib().maxsim_quantize_rows_fp4(x.data_ptr(), dt, rows, cols, ld, block, q.data_ptr(), width,
                                                block_scale.data_ptr(), ps, _raw_stream(index))
    if rc:
        _native.check(rc, "maxsim_quantize_rows_fp4")
    return q, block_scale, scale


def dequantize_rows_fp4(q: torch.Tensor, block_scale: torch.Tensor, scale: Optional[torch.Tensor] = None, *, block: int = 16,
                        cols: Optional[int] = None, out_dtype: torch.dtype = torch.bfloat16,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The rows [..., cols] in out_dtype that 4-bit rows (as quantize_rows_fp4
    gives them) stand for; without `cols` all that q holds."""
    dt = _DT_ANY.get(out_dtype)
    if dt is None:
        raise TypeError(f"out_dtype must be float16, bfloat16 or float32, got {out_dtype}")
    index, shape, dev = _device(q, "q"), q.shape, q.device
    if index != _current_device():
        return _with_device(index, dequantize_rows_fp4, q, block_scale, scale, block=block, cols=cols, out_dtype=out_dtype, out=out)
    pq, rows, ld, p_block, p_scale, _kept = _fp4_rows(q, block_scale, scale, "q", block, index)
    if cols is None:
        cols = 2 * shape[-1]
    if not 0 <= cols <= 2 * shape[-1] or (cols + 31) // 32 * 16 != shape[-1]:
        raise ValueError(f"rows of {shape[-1]} bytes do not hold {cols} columns")
    full = (*shape[:-1], cols)
    out = torch.empty(full, dtype=out_dtype, device=dev) if out is None else _given(out, "out", full, out_dtype, dev)
    rc = _native.lib().maxsim_dequantize_rows_fp4(pq, ld, p_block, p_scale, rows, cols, block, dt, out.data_ptr(), cols,
                                                  _raw_stream(index))
    if rc:
        _native.check(rc, "maxsim_dequantize_rows_fp4")
    return out


def linear_fp4(x: torch.Tensor, x_block_scale: torch.Tensor, x_scale: Optional[torch.Tensor], w: torch.Tensor,
               w_block_scale: torch.Tensor, w_scale: Optional[torch.Tensor], bias: Optional[torch.Tensor] = None, *,
               block: int = 16, out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """[..., N] in out_dtype: x @ w.T + bias for 4-bit rows x [..., K] and w [N, K]
    with their block scales and row scales (as quantize_rows_fp4 gives them, both
    in blocks of `block`; a row scale of None is 1); bias [N] f32."""
    dt = _DT_ANY.get(out_dtype)
    if dt is None:
        raise TypeError(f"out_dtype must be float16, bfloat16 or float32, got {out_dtype}")
    index, shape, dev = _device(x, "x"), x.shape, x.device
    if index != _current_device():
        return _with_device(index, linear_fp4, x, x_block_scale, x_scale, w, w_block_scale, w_scale, bias, block=block,
                            out_dtype=out_dtype, out=out)
    channels = w.shape
    if len(channels) != 2 or not shape or channels[1] != shape[-1]:
        raise ValueError("w must be [N, bytes] with x's bytes a row")
    N, width = channels
    px, M, ld_x, px_block, px_scale, _kept_x = _fp4_rows(x, x_block_scale, x_scale, "x", block, index)
    pw, _, ld_w, pw_block, pw_scale, _kept_w = _fp4_rows(w, w_block_scale, w_scale, "w", block, index)
    pb = None
    if bias is not None:
        if bias.dtype is not torch.float32:
            raise TypeError("bias must be float32")
        if bias.get_device() != index:
            raise ValueError("bias must be on x's device")
        if bias.shape != (N,):
            raise ValueError("bias must be [N]")
        if not bias.is_contiguous():
            bias = bias.contiguous()
        pb = bias.data_ptr()
    full = (*shape[:-1], N)
    out = torch.empty(full, dtype=out_dtype, device=dev) if out is None else _given(out, "out", full, out_dtype, dev)
    rc = _native.lib().maxsim_linear_fp4(px, ld_x, px_block, px_scale, pw, ld_w, pw_block, pw_scale, pb, M, N, 2 * width, block, dt,
                                         out.data_ptr(), N, _raw_stream(index))
    if rc:
        _native.check(rc, "maxsim_linear_fp4")
    return out


def _logprobs_rows(logits: torch.Tensor, targets: Optional[torch.Tensor], mask: Optional[torch.Tensor], index: int):
    """(pointer, rows, n, row stride, targets' pointer, T, mask's pointer, mask's stride, leading shape, the tensors) of the
    log probabilities' operands, checked."""
    shape = logits.shape
    n = shape[-1] if shape else 0
    if not n:
        raise ValueError("logits must have at least one column")
    lead = shape[:-1]
    T, p_targets = 0, None
    if targets is not None:
        if targets.dtype is not torch.int64:
            if targets.dtype is not torch.int32:
                raise TypeError(f"targets must be int64 or int32, got {targets.dtype}")
            targets = targets.to(torch.int64)
        if targets.get_device() != index:
            raise ValueError("targets must be on logits' device")
        given = targets.shape
        if given == lead:
            T = 1
        elif given[:-1] == lead and len(given) > len(lead):
            T = given[-1]
        else:
            raise ValueError("targets must have logits' leading shape, with one more dimension for several a row")
        if not targets.is_contiguous():
            targets = targets.contiguous()
        p_targets = targets.data_ptr()
    ld_mask, p_mask = 0, None
    if mask is not None:
        if mask.dtype is not torch.bool and mask.dtype is not _U8:
            raise TypeError(f"mask must be bool or uint8, got {mask.dtype}")
        if mask.get_device() != index:
            raise ValueError("mask must be on logits' device")
        if mask.shape == shape and len(shape) > 1:
            mask, _, ld_mask = _rows(mask, "mask")
        elif mask.shape != shape[-1:]:
            raise ValueError("mask must have logits' shape, or be [n] for all rows")
        elif not mask.is_contiguous():
            mask = mask.contiguous()
        p_mask = mask.data_ptr()
    if logits.is_contiguous():
        rows, ld = logits.numel() // n, n
    else:
        logits, rows, ld = _rows(logits, "logits")
    return logits.data_ptr(), rows, n, ld, p_targets, T, p_mask, ld_mask, lead, (logits, targets, mask)


def logprobs_fwd(logits: torch.Tensor, targets: Optional[torch.Tensor], mask: Optional[torch.Tensor] = None, *,
                 scale: float = 1.0, k: int = 0):
    """(logprob, entropy, top_idx, top_logprob, stats) of softmax(scale * logits) over
    the active columns of logits [..., n] (f16 / bf16 / f32): the log probabilities
    of `targets` ([...] or [..., T], -1 for none), each row's entropy, its k <= 64
    largest columns (by descending value, the lower index first among equal ones;
    -1 where there are fewer) with their log probabilities, and what logprobs_bwd
    takes. mask: bool / uint8, logits' shape or [n]; nonzero = active. logprob is
    None without targets; top_idx and top_logprob are None with k = 0."""
    dt = _DT_ANY.get(logits.dtype)
    if dt is None:
        raise TypeError(f"logits must be float16, bfloat16 or float32, got {logits.dtype}")
    index, dev = _device(logits, "logits"), logits.device
    if index != _current_device():
        return _with_device(index, logprobs_fwd, logits, targets, mask, scale=scale, k=k)
    px, rows, n, ld, p_targets, T, p_mask, ld_mask, lead, _kept = _logprobs_rows(logits, targets, mask, index)
    f32, empty = torch.float32, torch.empty
    logprob = top_idx = top_logprob = p_logprob = p_idx = p_top = None
    if targets is not None:
        logprob = empty(targets.shape, dtype=f32, device=dev)
        p_logprob = logprob.data_ptr()
    entropy = empty(lead, dtype=f32, device=dev)
    stats = empty((*lead, 2), dtype=f32, device=dev)
    if k:
        top_idx = empty((*lead, k), dtype=torch.int32, device=dev)
        top_logprob = empty((*lead, k), dtype=f32, device=dev)
        p_idx, p_top = top_idx.data_ptr(), top_logprob.data_ptr()
    rc = _native.lib().maxsim_logprobs_fwd(px, dt, rows, n, ld, p_targets, T, p_mask, ld_mask, scale, k, p_logprob,
                                           entropy.data_ptr(), p_idx, p_top, stats.data_ptr(), _raw_stream(index))
    if rc:
        _native.check(rc, "maxsim_logprobs_fwd")
    return logprob, entropy, top_idx, top_logprob, stats


def _grad(g: Optional[torch.Tensor], name: str, shape, index: int):
    if g is None:
        return None
    if g.dtype is not torch.float32:
        raise TypeError(f"{name} must be float32, got {g.dtype}")
    if g.shape != shape or g.get_device() != index:
        raise ValueError(f"{name} must be {tuple(shape)} on logits' device")
    return g if g.is_contiguous() else g.contiguous()


def logprobs_bwd(logits: torch.Tensor, targets: Optional[torch.Tensor], mask: Optional[torch.Tensor], stats: torch.Tensor,
                 entropy: torch.Tensor, *, grad_logprob: Optional[torch.Tensor] = None,
                 grad_entropy: Optional[torch.Tensor] = None, top_idx: Optional[torch.Tensor] = None,
                 grad_top: Optional[torch.Tensor] = None, scale: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient in logits, in their type, of logprobs_fwd with the same
    arguments, from its stats and entropy and the f32 gradients of its outputs
    (None: zero; grad_top belongs to top_idx). out shares no elements with logits."""
    dt = _DT_ANY.get(logits.dtype)
    if dt is None:
        raise TypeError(f"logits must be float16, bfloat16 or float32, got {logits.dtype}")
    index, shape, dev = _device(logits, "logits"), logits.shape, logits.device
    if index != _current_device():
        return _with_device(index, logprobs_bwd, logits, targets, mask, stats, entropy, grad_logprob=grad_logprob,
                            grad_entropy=grad_entropy, top_idx=top_idx, grad_top=grad_top, scale=scale, out=out)
    px, rows, n, ld, p_targets, T, p_mask, ld_mask, lead, _kept = _logprobs_rows(logits, targets, mask, index)
    stats, entropy = _grad(stats, "stats", (*lead, 2), index), _grad(entropy, "entropy", lead, index)
    if grad_logprob is not None and targets is None:
        raise ValueError("grad_logprob needs targets")
    grad_logprob = _grad(grad_logprob, "grad_logprob", targets.shape if targets is not None else (), index)
    grad_entropy = _grad(grad_entropy, "grad_entropy", lead, index)
    k = 0
    if grad_top is not None:
        if top_idx is None or top_idx.dtype is not torch.int32 or top_idx.get_device() != index or top_idx.shape[:-1] != lead:
            raise ValueError("grad_top needs the int32 top_idx of the forward")
        grad_top = _grad(grad_top, "grad_top", top_idx.shape, index)
        top_idx, k = top_idx.contiguous(), top_idx.shape[-1]
    if out is not None:
        out = _given(out, "out", shape, logits.dtype, dev)
    elif logits.is_contiguous():
        out = torch.empty_like(logits)  # half the time of torch.empty
    else:
        out = torch.empty(shape, dtype=logits.dtype, device=dev)
    rc = _native.lib().maxsim_logprobs_bwd(px, dt, rows, n, ld, p_targets, T, p_mask, ld_mask, scale, stats.data_ptr(),
                                           entropy.data_ptr(), _ptr(grad_logprob), _ptr(grad_entropy), _ptr(top_idx),
                                           _ptr(grad_top), k, out.data_ptr(), n, _raw_stream(index))
    if rc:
        _native.check(rc, "maxsim_logprobs_bwd")
    return out


def device_status(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device status word."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return int(_native.lib().maxsim_device_status(_stream(dev)))


def debug_inject_wait_timeout(limit_ns: int) -> None:
    """Fault-handling test hook: the next forward launch from this process
    waits, in its epilogue, on a barrier nothing arrives at and gives up after
    limit_ns, recording MAXSIM_ERR_TIMEOUT (read it with device_status())."""
    _native.check(_native.lib().maxsim_debug_inject_wait_timeout(int(limit_ns)), "maxsim_debug_inject_wait_timeout")
