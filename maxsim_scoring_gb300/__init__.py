"""Fused MaxSim (ColBERT / ColPali late interaction) for GB300.

    score[i, j] = sum_s max_t <Q[i, s], D[j, t]>

The compute lives in libmaxsim.so (hand-written sm_103a kernels behind the C
ABI of include/maxsim.h); this package is its PyTorch-facing binding plus an
autograd wrapper.
"""
from .ops import (chamfer_bwd, chamfer_fwd, dequantize_rows_fp4, device_status, dropout_bwd, dropout_fwd,  # noqa: F401
                  linear_fp4, linear_int8, logprobs_bwd, logprobs_fwd,
                  maxsim_bwd, maxsim_bwd_varlen, maxsim_fwd, maxsim_fwd_int8, maxsim_fwd_streamed, maxsim_fwd_varlen,
                  maxsim_fwd_varlen_streamed, maxsim_score_pairs_packed, maxsim_topk, maxsim_two_stage_topk,
                  quantize_rows, quantize_rows_fp4, workspace_size)
from .autograd import chamfer_distance, dropout, logprobs, maxsim, maxsim_varlen  # noqa: F401

__all__ = ["maxsim", "maxsim_varlen", "maxsim_fwd", "maxsim_fwd_varlen", "maxsim_score_pairs_packed", "maxsim_bwd",
           "maxsim_bwd_varlen", "maxsim_fwd_int8", "maxsim_fwd_streamed", "maxsim_fwd_varlen_streamed", "maxsim_topk", "maxsim_two_stage_topk",
           "quantize_rows", "linear_int8", "dropout", "dropout_fwd", "dropout_bwd",
           "quantize_rows_fp4", "dequantize_rows_fp4", "linear_fp4", "logprobs", "logprobs_fwd", "logprobs_bwd",
           "chamfer_fwd", "chamfer_bwd", "chamfer_distance", "workspace_size", "device_status"]
