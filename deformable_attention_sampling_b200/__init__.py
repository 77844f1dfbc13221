"""Deformable sampling-aggregation on NVIDIA B200 (sm_100a).

DCNv3 / DCNv4 deformable convolution core and the multi-scale deformable
attention (MSDeformAttn) core, forward and backward, as hand-written CUDA kernels behind a
C interface (include/dcn.h, libdcn_b200.so).  This package is the thin Python
binding: it marshals pointers, sizes and streams and runs nothing itself.

    import deformable_attention_sampling_b200 as dcnb
    out = dcnb.dcn(x, offset, mask)          # torch CUDA tensors, NHWC
    out = dcnb.msda(value, shapes, starts, loc, attn)
    gx, goff, gmask = dcnb.dcn_grad(x, offset, mask, grad_out)
    gv, gloc, gattn = dcnb.msda_grad(value, shapes, starts, loc, attn, grad_out)
    out = dcnb.dynconv(x, weights, K)        # ContMix core: per-pixel K x K kernels

and the operators of the attention block around them, each with its gradient:

    q = dcnb.axial_rope(q, pos, freqs, axis_pairs)        # rotary positions, 1 to 4 axes
    out, saved = dcnb.diff_attn(q, k, v, lam, save=True)  # difference of two softmax maps
    z, h = dcnb.norm_residual(x, y, scale, gate)          # normed, gated residual join
"""
from ._binding import (  # noqa: F401
    ALGO_CODES,
    DCN_ALGO_AUTO,
    DCN_ALGO_BAND,
    DCN_ALGO_GATHER,
    DCN_ALGO_SIMT,
    DCN_ALGO_TENSOR,
    DYNCONV_ALGO_CODES,
    DCN_ERR_CUDA,
    DCN_ERR_INVALID_ARG,
    DCN_ERR_MISALIGNED,
    DCN_ERR_UNSUPPORTED,
    DCN_OK,
    DCN_NORM_POST,
    DCN_NORM_PRE,
    DCN_NORM_RMS,
    DTYPE_CODES,
    LIB_PATH,
    SIGNATURES,
    DcnError,
    axial_rope,
    axial_rope_backward,
    axial_rope_forward,
    axial_rope_grad,
    dcn,
    STATIC_SCRATCH_BYTES,
    dcn_backward,
    dcn_backward_static_scratch,
    dcn_backward_workspace_size,
    dcn_forward,
    dcn_forward_algo,
    dcn_forward_plan,
    PLAN_FIELDS,
    DCN_FLAG_BAD_LEVELS,
    DCN_FLAG_OUT_OF_BOUNDS,
    DCN_FLAG_WAIT_TIMEOUT,
    DEBUG_LIB_PATH,
    dcn_debug_checks,
    dcn_device_flags,
    debug_library,
    dcn_grad,
    dcn_last_cuda_error,
    dcn_launch_count,
    dcn_output_size,
    dcnv4_fused,
    dcnv4_fused_forward,
    dcnv4_fused_forward_algo,
    dcn_status_string,
    dcn_version,
    diff_attn,
    diff_attn_backward,
    diff_attn_backward_workspace_size,
    diff_attn_forward,
    diff_attn_forward_workspace_size,
    diff_attn_grad,
    dtype_code,
    dynconv,
    dynconv_forward,
    dynconv_forward_algo,
    library,
    msda,
    msda_backward,
    msda_backward_workspace_size,
    msda_forward,
    msda_forward_points,
    msda_mask_value,
    msda_points,
    mask_value,
    msda_grad,
    norm_residual,
    norm_residual_backward,
    norm_residual_backward_workspace_size,
    norm_residual_forward,
    norm_residual_grad,
)
