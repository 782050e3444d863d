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
