"""dg: the local compute of expert- and tensor-parallel linear layers on one GB300.

Its operations, each a C-ABI entry point of libdg (include/dg.h) backed by
hand-written sm_103a kernels (tcgen05 UMMA with TMEM accumulators fed by
TMA/mbarrier pipelines):

* gemm_fp8      D = alpha * (A @ B^T) + beta * C, e4m3 inputs, bf16 output
* a2a_ffn       the all-to-all expert-parallel FFN layer (forward, backward,
                autograd), P logical ranks in one GPU's memory; a forward with
                both GEMMs on e4m3 operands (a2a_ffn_forward_fp8)
* tp_swiglu     the SwiGLU column/row-parallel pair over W shards (forward,
                backward, autograd)
* tp_linear     the attention projections (column-parallel QKV, row-parallel
                wo) over W shards (forward, backward, autograd)
* moe_layer     routed SwiGLU experts for few tokens (moe_route, then
                moe_swiglu on bf16 or moe_swiglu_w4 on 4-bit weights; forward)
* w4_linear     a linear on 4-bit weights with group scales for few rows, and
                the quantiser (w4_quantize, w4_dequantize; forward)
* fp8_linear    a linear on block-scaled e4m3 (power-of-two scales) from one row
                to whole prompts, its gradients from 8-bit activations, and the
                quantiser (fp8_quantize, fp8_dequantize; fp8_linear_layer)
* rms_norm      the root-mean-square norm with the residual's addition, its
                result in bf16 or block-scaled e4m3 (forward, backward,
                autograd; fp8_norm_linear_layer joins it with the linear)
* *_keep8       tp_linear_layer and tp_swiglu_layer with their inputs kept in
                8 bits for the backward

The library is loaded lazily on first use and fails loudly if it is missing.
"""
from .ops import (A2AFFN, DG_FFN_COMP_ONLY, DG_FFN_FUSED_GATE, DG_FFN_SEPARATE_GATE, FFN_PARAM_NAMES, TPSwiGLU,
                  a2a_combine,
                  a2a_dispatch, a2a_ffn, a2a_ffn_backward, a2a_ffn_forward, a2a_ffn_forward_fp8,
                  a2a_ffn_fp8_pack_weights, alloc_workspace, debug_wait_timeout, device_status, error_block,
                  ffn_shape, gemm_fp8, tp_swiglu, tp_linear, tp_linear_backward, tp_linear_layer, TPLinear,
                  tp_swiglu_backward, tp_swiglu_layer, trace_begin, trace_end)
from .few import moe_layer, moe_route, moe_swiglu, moe_swiglu_w4, w4_dequantize, w4_linear, w4_quantize
from .fp8 import (FP8Linear, FP8NormLinear, RMSNorm, TPLinearKeep8, TPSwiGLUKeep8, fp8_dequantize, fp8_linear,
                  fp8_linear_backward, fp8_linear_layer, fp8_norm_linear_layer, fp8_quantize, rms_norm,
                  rms_norm_backward, rms_norm_layer, tp_linear_layer_keep8, tp_swiglu_layer_keep8)

__all__ = [
    "A2AFFN", "DG_FFN_COMP_ONLY", "DG_FFN_FUSED_GATE", "DG_FFN_SEPARATE_GATE", "FFN_PARAM_NAMES", "a2a_combine",
    "a2a_dispatch",
    "a2a_ffn", "a2a_ffn_backward", "a2a_ffn_forward", "a2a_ffn_forward_fp8", "a2a_ffn_fp8_pack_weights",
    "alloc_workspace", "debug_wait_timeout", "device_status", "error_block", "ffn_shape", "gemm_fp8", "tp_swiglu",
    "tp_swiglu_backward", "TPSwiGLU", "tp_swiglu_layer", "tp_linear", "tp_linear_backward", "TPLinear",
    "tp_linear_layer", "trace_begin", "trace_end", "moe_layer", "moe_route", "moe_swiglu", "moe_swiglu_w4",
    "w4_dequantize", "w4_linear", "w4_quantize", "FP8Linear", "FP8NormLinear", "RMSNorm", "fp8_dequantize", "fp8_linear",
    "fp8_linear_backward", "fp8_linear_layer", "fp8_norm_linear_layer", "fp8_quantize", "rms_norm", "rms_norm_backward",
    "rms_norm_layer", "TPLinearKeep8", "TPSwiGLUKeep8", "tp_linear_layer_keep8", "tp_swiglu_layer_keep8",
]
