"""ctypes binding of libdcn_b200.so (include/dcn.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C interface.  Pointer arguments may be integers (device
addresses) or objects with a ``data_ptr()`` method (torch tensors); stream
arguments may be None (torch's current stream), an integer handle, or an object
with a ``cuda_stream`` attribute.  A non-OK status raises DcnError.

There is no fallback: when the shared library is missing the first call
raises RuntimeError naming the build command.
"""
import contextlib
import ctypes
import functools
import math
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_lib", "libdcn_b200.so")
DEBUG_LIB_PATH = os.path.join(PKG, "_lib", "libdcn_b200_debug.so")

DCN_OK = 0
DCN_ERR_INVALID_ARG = -1
DCN_ERR_UNSUPPORTED = -2
DCN_ERR_MISALIGNED = -3
DCN_ERR_CUDA = -4
DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2}
DCN_FLAG_WAIT_TIMEOUT = 1
DCN_FLAG_OUT_OF_BOUNDS = 2
DCN_FLAG_BAD_LEVELS = 4
DCN_NORM_RMS = 1
DCN_NORM_POST = 2
DCN_NORM_PRE = 4
# the entry points the debug library holds (the forward calls and the status calls)
DEBUG_SYMBOLS = ("dcn_forward", "dcn_forward_algo", "dcn_forward_plan", "dcnv4_fused_forward",
                 "dcnv4_fused_forward_algo", "msda_forward", "msda_forward_points",
                 "msda_mask_value", "dcn_output_size", "dcn_status_string", "dcn_last_cuda_error",
                 "dcn_launch_count", "dcn_device_flags", "dcn_debug_checks", "dcn_version")
DCN_ALGO_AUTO = 0
DCN_ALGO_GATHER = 1
DCN_ALGO_SIMT = 1
DCN_ALGO_BAND = 2
DCN_ALGO_TENSOR = 3
ALGO_CODES = {"auto": DCN_ALGO_AUTO, "gather": DCN_ALGO_GATHER, "band": DCN_ALGO_BAND}
# dynconv_forward_algo's kernels
DYNCONV_ALGO_CODES = {"auto": DCN_ALGO_AUTO, "simt": DCN_ALGO_SIMT, "tensor": DCN_ALGO_TENSOR}

# every symbol include/dcn.h declares, with its ctypes signature
_VP = ctypes.c_void_p
_I = ctypes.c_int
_LL = ctypes.c_longlong
SIGNATURES = {
    "dcn_forward": (_I, [_VP, _VP, _VP, _VP] + [_I] * 12 + [_VP]),
    "dcn_forward_algo": (_I, [_VP, _VP, _VP, _VP] + [_I] * 13 + [_VP]),
    "dcn_forward_plan": (_I, [_I] * 13 + [ctypes.POINTER(ctypes.c_int)]),
    "dcn_device_flags": (_I, [_I]),
    "dcn_debug_checks": (_I, []),
    "msda_forward": (_I, [_VP] * 6 + [_I] * 7 + [_VP]),
    "msda_forward_points": (_I, [_VP] * 4 + [_I] + [_VP] * 4 + [_I] * 7 + [_VP]),
    "msda_mask_value": (_I, [_VP] * 3 + [_I] * 5 + [_VP]),
    "dcn_backward_workspace_size": (_LL, [_I] * 5),
    "dcn_backward": (_I, [_VP] * 8 + [_LL] + [_I] * 12 + [_VP]),
    "dcn_backward_static_scratch": (_I, [_VP] * 7 + [_I] * 12 + [_VP]),
    "msda_backward_workspace_size": (_LL, [_I] * 5),
    "msda_backward": (_I, [_VP] * 10 + [_LL] + [_I] * 8 + [_VP]),
    "dynconv_forward": (_I, [_VP] * 3 + [_I] * 8 + [_VP]),
    "dynconv_forward_algo": (_I, [_VP] * 3 + [_I] * 9 + [_VP]),
    "dcnv4_fused_forward": (_I, [_VP] * 4 + [_I] * 10 + [_VP]),
    "dcnv4_fused_forward_algo": (_I, [_VP] * 4 + [_I] * 11 + [_VP]),
    "axial_rope_forward": (_I, [_VP] * 5 + [_I] * 6 + [_LL] * 2 + [_I] * 3 + [_VP]),
    "axial_rope_backward": (_I, [_VP] * 7 + [_I] * 6 + [_LL] * 2 + [_I] * 3 + [_VP]),
    "norm_residual_forward": (_I, [_VP] * 10 + [_I, _LL, _I, _I, ctypes.c_float, _I, _VP]),
    "norm_residual_backward_workspace_size": (_LL, [_I, _LL, _I, _I, _I]),
    "norm_residual_backward": (_I, [_VP] * 18 + [_LL, _I, _LL, _I, _I, ctypes.c_float, _I, _VP]),
    "diff_attn_forward_workspace_size": (_LL, [_I] * 8),
    "diff_attn_forward": (_I, [_VP] * 10 + [_LL] + [_I] * 7 + [_LL] * 6 +
                          [ctypes.c_float, _I, _I, _VP]),
    "diff_attn_backward_workspace_size": (_LL, [_I] * 8),
    "diff_attn_backward": (_I, [_VP] * 14 + [_LL] + [_I] * 7 + [_LL] * 6 +
                           [ctypes.c_float, _I, _I, _VP]),
    "dcn_output_size": (_I, [_I] * 5),
    "dcn_status_string": (ctypes.c_char_p, [_I]),
    "dcn_last_cuda_error": (_I, []),
    "dcn_launch_count": (ctypes.c_uint64, []),
    "dcn_version": (_I, []),
}

_lib = None


class DcnError(RuntimeError):
    """A dcn_status_t other than DCN_OK."""

    def __init__(self, status, where):
        self.status = status
        text = _load().dcn_status_string(status).decode()
        detail = ""
        if status == DCN_ERR_CUDA:
            detail = f" (cudaError {_load().dcn_last_cuda_error()})"
        super().__init__(f"{where}: {text}{detail} [status {status}]")


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m deformable_attention_sampling_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def library():
    """The loaded ctypes library (loads it on first use)."""
    return _load()


_debug_lib = None


def debug_library():
    """The debug library (libdcn_b200_debug.so: the forward and status calls
    with device-side address and level-table checks), loaded on first use."""
    global _debug_lib
    if _debug_lib is None:
        if not os.path.exists(DEBUG_LIB_PATH):
            raise RuntimeError(
                f"{DEBUG_LIB_PATH} is missing: build it with "
                "`python -m deformable_attention_sampling_b200.build`")
        lib = ctypes.CDLL(DEBUG_LIB_PATH)
        for name in DEBUG_SYMBOLS:
            res, args = SIGNATURES[name]
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _debug_lib = lib
    return _debug_lib


def _ptr(p):
    if p is None:
        return None
    if isinstance(p, int):
        return p
    return int(p.data_ptr())


def _stream(s):
    if s is None:
        from torch import _C, cuda
        # the raw handle: a Stream object would cost more than the rest of a small call
        return _C._cuda_getCurrentRawStream(cuda.current_device())
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


@functools.lru_cache(maxsize=256)
def _int_tuple(values):
    return (ctypes.c_int * len(values))(*values)


def _int_array(values, n):
    values = tuple(values)
    if len(values) != n:
        raise ValueError(f"expected {n} values, got {len(values)}")
    return _int_tuple(values)


def _check(status, where):
    if status != DCN_OK:
        raise DcnError(status, where)


def dcn_forward(x, offset, mask, out, N, H, W, C, G, kh, kw, stride, pad, dil,
                softmax_flag, dtype, stream=None):
    """C dcn_forward; raises DcnError on a non-OK status."""
    _check(_load().dcn_forward(_ptr(x), _ptr(offset), _ptr(mask), _ptr(out), N, H, W, C, G,
                               kh, kw, stride, pad, dil, softmax_flag, dtype, _stream(stream)),
           "dcn_forward")


def dcn_forward_algo(x, offset, mask, out, N, H, W, C, G, kh, kw, stride, pad, dil,
                     softmax_flag, dtype, algo, stream=None):
    """C dcn_forward_algo (algo: DCN_ALGO_AUTO / _GATHER / _BAND); raises
    DcnError on a non-OK status."""
    _check(_load().dcn_forward_algo(_ptr(x), _ptr(offset), _ptr(mask), _ptr(out), N, H, W, C,
                                    G, kh, kw, stride, pad, dil, softmax_flag, dtype, algo,
                                    _stream(stream)),
           "dcn_forward_algo")


PLAN_FIELDS = ("algo", "rows_per_step", "margin", "ring_rows", "sampler_warps",
               "steps_in_flight", "runs_per_row", "smem_bytes")


def dcn_forward_plan(N, H, W, C, G, kh, kw, stride, pad, dil, softmax_flag, dtype,
                     algo=DCN_ALGO_AUTO, lib=None):
    """C dcn_forward_plan: the kernel dcn_forward_algo runs for this shape and
    the band kernel's launch shape, as a dict over PLAN_FIELDS (host only, no
    GPU needed); raises DcnError on a non-OK status."""
    plan = (ctypes.c_int * 8)()
    _check((lib or _load()).dcn_forward_plan(N, H, W, C, G, kh, kw, stride, pad, dil,
                                             softmax_flag, dtype, algo, plan),
           "dcn_forward_plan")
    return dict(zip(PLAN_FIELDS, list(plan)))


def dcn_device_flags(reset=False, lib=None):
    """C dcn_device_flags: the status word of the current device (DCN_FLAG_*
    bits), cleared when reset; synchronous.  `lib`: the debug library handle
    instead of the release library."""
    r = (lib or _load()).dcn_device_flags(1 if reset else 0)
    if r < 0:
        raise DcnError(r, "dcn_device_flags")
    return r


def dcn_debug_checks(lib=None):
    """1 for the debug library (device-side checks), 0 for the release one."""
    return int((lib or _load()).dcn_debug_checks())


def msda_forward(value, spatial_shapes, level_start, sampling_loc, attn_w, out, N, Lq, M, D,
                 L, K, dtype, stream=None):
    """C msda_forward; raises DcnError on a non-OK status."""
    _check(_load().msda_forward(_ptr(value), _ptr(spatial_shapes), _ptr(level_start),
                                _ptr(sampling_loc), _ptr(attn_w), _ptr(out), N, Lq, M, D, L,
                                K, dtype, _stream(stream)),
           "msda_forward")


def dcn_backward_workspace_size(N, H, W, C, dtype):
    return int(_load().dcn_backward_workspace_size(N, H, W, C, dtype))


def dcn_backward(x, offset, mask, grad_out, grad_x, grad_offset, grad_mask, workspace,
                 workspace_bytes, N, H, W, C, G, kh, kw, stride, pad, dil, softmax_flag, dtype,
                 stream=None):
    """C dcn_backward; raises DcnError on a non-OK status."""
    _check(_load().dcn_backward(_ptr(x), _ptr(offset), _ptr(mask), _ptr(grad_out), _ptr(grad_x),
                                _ptr(grad_offset), _ptr(grad_mask), _ptr(workspace),
                                workspace_bytes, N, H, W, C, G, kh, kw, stride, pad, dil,
                                softmax_flag, dtype, _stream(stream)),
           "dcn_backward")


# bytes of the library's static grad_x accumulator (DCN_STATIC_SCRATCH_BYTES)
STATIC_SCRATCH_BYTES = 16 << 20


def dcn_backward_static_scratch(x, offset, mask, grad_out, grad_x, grad_offset, grad_mask, N, H,
                                W, C, G, kh, kw, stride, pad, dil, softmax_flag, dtype,
                                stream=None):
    """C dcn_backward_static_scratch (no workspace argument; the library's own
    per-device accumulator); raises DcnError on a non-OK status."""
    _check(_load().dcn_backward_static_scratch(
        _ptr(x), _ptr(offset), _ptr(mask), _ptr(grad_out), _ptr(grad_x), _ptr(grad_offset),
        _ptr(grad_mask), N, H, W, C, G, kh, kw, stride, pad, dil, softmax_flag, dtype,
        _stream(stream)), "dcn_backward_static_scratch")


def msda_backward_workspace_size(N, S, M, D, dtype):
    return int(_load().msda_backward_workspace_size(N, S, M, D, dtype))


def msda_backward(value, spatial_shapes, level_start, sampling_loc, attn_w, grad_out,
                  grad_value, grad_loc, grad_attn, workspace, workspace_bytes, N, S, Lq, M, D,
                  L, K, dtype, stream=None):
    """C msda_backward; raises DcnError on a non-OK status."""
    _check(_load().msda_backward(_ptr(value), _ptr(spatial_shapes), _ptr(level_start),
                                 _ptr(sampling_loc), _ptr(attn_w), _ptr(grad_out),
                                 _ptr(grad_value), _ptr(grad_loc), _ptr(grad_attn),
                                 _ptr(workspace), workspace_bytes, N, S, Lq, M, D, L, K, dtype,
                                 _stream(stream)),
           "msda_backward")


def dynconv_forward(x, weights, out, N, H, W, C, G, K, softmax_flag, dtype, stream=None):
    """C dynconv_forward; raises DcnError on a non-OK status."""
    _check(_load().dynconv_forward(_ptr(x), _ptr(weights), _ptr(out), N, H, W, C, G, K,
                                   softmax_flag, dtype, _stream(stream)),
           "dynconv_forward")


def dynconv_forward_algo(x, weights, out, N, H, W, C, G, K, softmax_flag, dtype, algo,
                         stream=None):
    """C dynconv_forward_algo; raises DcnError on a non-OK status."""
    _check(_load().dynconv_forward_algo(_ptr(x), _ptr(weights), _ptr(out), N, H, W, C, G, K,
                                        softmax_flag, dtype, algo, _stream(stream)),
           "dynconv_forward_algo")


def msda_forward_points(value, spatial_shapes, level_start, reference, ref_dim, valid_ratios,
                        offsets, attn_w, out, N, Lq, M, D, L, K, dtype, stream=None):
    """C msda_forward_points; raises DcnError on a non-OK status."""
    _check(_load().msda_forward_points(_ptr(value), _ptr(spatial_shapes), _ptr(level_start),
                                       _ptr(reference), ref_dim, _ptr(valid_ratios),
                                       _ptr(offsets), _ptr(attn_w), _ptr(out), N, Lq, M, D, L,
                                       K, dtype, _stream(stream)),
           "msda_forward_points")


def msda_mask_value(value, mask, out, N, S, M, D, dtype, stream=None):
    """C msda_mask_value; raises DcnError on a non-OK status."""
    _check(_load().msda_mask_value(_ptr(value), _ptr(mask), _ptr(out), N, S, M, D, dtype,
                                   _stream(stream)),
           "msda_mask_value")


def dcnv4_fused_forward(x, w_om, b_om, out, N, H, W, C, G, kh, kw, pad, dil, dtype,
                        stream=None):
    """C dcnv4_fused_forward; raises DcnError on a non-OK status."""
    _check(_load().dcnv4_fused_forward(_ptr(x), _ptr(w_om), _ptr(b_om), _ptr(out), N, H, W, C,
                                       G, kh, kw, pad, dil, dtype, _stream(stream)),
           "dcnv4_fused_forward")


def dcnv4_fused_forward_algo(x, w_om, b_om, out, N, H, W, C, G, kh, kw, pad, dil, dtype, algo,
                             stream=None):
    """C dcnv4_fused_forward_algo; raises DcnError on a non-OK status."""
    _check(_load().dcnv4_fused_forward_algo(_ptr(x), _ptr(w_om), _ptr(b_om), _ptr(out), N, H, W,
                                            C, G, kh, kw, pad, dil, dtype, algo,
                                            _stream(stream)),
           "dcnv4_fused_forward_algo")


def axial_rope_forward(x, pos, freqs, out, axis_pairs, N, L, M, D, A, pos_images, x_image, x_row,
                       interleaved, inverse, dtype, stream=None):
    """C axial_rope_forward (axis_pairs: a sequence of A ints); raises DcnError
    on a non-OK status."""
    _check(_load().axial_rope_forward(_ptr(x), _ptr(pos), _ptr(freqs), _ptr(out),
                                      _int_array(axis_pairs, A), N, L, M, D, A, pos_images,
                                      x_image, x_row, interleaved, inverse, dtype,
                                      _stream(stream)),
           "axial_rope_forward")


def axial_rope_backward(x, pos, freqs, grad_out, grad_x, grad_pos, axis_pairs, N, L, M, D, A,
                        pos_images, x_image, x_row, interleaved, inverse, dtype, stream=None):
    """C axial_rope_backward; raises DcnError on a non-OK status."""
    _check(_load().axial_rope_backward(_ptr(x), _ptr(pos), _ptr(freqs), _ptr(grad_out),
                                       _ptr(grad_x), _ptr(grad_pos), _int_array(axis_pairs, A),
                                       N, L, M, D, A, pos_images, x_image, x_row, interleaved,
                                       inverse, dtype, _stream(stream)),
           "axial_rope_backward")


def norm_residual_forward(x, y, scale, gate, post_weight, post_bias, pre_weight, pre_bias, z, h,
                          N, L, C, flags, eps, dtype, stream=None):
    """C norm_residual_forward; raises DcnError on a non-OK status."""
    _check(_load().norm_residual_forward(_ptr(x), _ptr(y), _ptr(scale), _ptr(gate),
                                         _ptr(post_weight), _ptr(post_bias), _ptr(pre_weight),
                                         _ptr(pre_bias), _ptr(z), _ptr(h), N, L, C, flags, eps,
                                         dtype, _stream(stream)),
           "norm_residual_forward")


def norm_residual_backward_workspace_size(N, L, C, gated, dtype):
    return int(_load().norm_residual_backward_workspace_size(N, L, C, gated, dtype))


def norm_residual_backward(y, z, grad_z, grad_h, scale, gate, post_weight, post_bias, pre_weight,
                           grad_x, grad_y, grad_scale, grad_gate, grad_post_weight,
                           grad_post_bias, grad_pre_weight, grad_pre_bias, workspace,
                           workspace_bytes, N, L, C, flags, eps, dtype, stream=None):
    """C norm_residual_backward; raises DcnError on a non-OK status."""
    _check(_load().norm_residual_backward(
        _ptr(y), _ptr(z), _ptr(grad_z), _ptr(grad_h), _ptr(scale), _ptr(gate), _ptr(post_weight),
        _ptr(post_bias), _ptr(pre_weight), _ptr(grad_x), _ptr(grad_y), _ptr(grad_scale),
        _ptr(grad_gate), _ptr(grad_post_weight), _ptr(grad_post_bias), _ptr(grad_pre_weight),
        _ptr(grad_pre_bias), _ptr(workspace), workspace_bytes, N, L, C, flags, eps, dtype,
        _stream(stream)), "norm_residual_backward")


def diff_attn_forward_workspace_size(N, Lq, Lk, M, Mk, D, Dv, dtype):
    return int(_load().diff_attn_forward_workspace_size(N, Lq, Lk, M, Mk, D, Dv, dtype))


def diff_attn_forward(q, k, v, lam, mask, lengths, out, maps, lse, workspace, workspace_bytes, N,
                      Lq, Lk, M, Mk, D, Dv, q_image, q_row, k_image, k_row, v_image, v_row, scale,
                      causal, dtype, stream=None):
    """C diff_attn_forward; raises DcnError on a non-OK status."""
    _check(_load().diff_attn_forward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(mask), _ptr(lengths), _ptr(out), _ptr(maps),
        _ptr(lse), _ptr(workspace), workspace_bytes, N, Lq, Lk, M, Mk, D, Dv, q_image, q_row,
        k_image, k_row, v_image, v_row, scale, causal, dtype, _stream(stream)),
        "diff_attn_forward")


def diff_attn_backward_workspace_size(N, Lq, Lk, M, Mk, D, Dv, dtype):
    return int(_load().diff_attn_backward_workspace_size(N, Lq, Lk, M, Mk, D, Dv, dtype))


def diff_attn_backward(q, k, v, lam, mask, lengths, maps, lse, grad_out, grad_q, grad_k,
                       grad_v, grad_lam, workspace, workspace_bytes, N, Lq, Lk, M, Mk, D, Dv,
                       q_image, q_row, k_image, k_row, v_image, v_row, scale, causal, dtype,
                       stream=None):
    """C diff_attn_backward; raises DcnError on a non-OK status."""
    _check(_load().diff_attn_backward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(mask), _ptr(lengths), _ptr(maps), _ptr(lse),
        _ptr(grad_out), _ptr(grad_q), _ptr(grad_k), _ptr(grad_v), _ptr(grad_lam),
        _ptr(workspace), workspace_bytes, N, Lq, Lk, M, Mk, D, Dv, q_image, q_row, k_image, k_row,
        v_image, v_row, scale, causal, dtype, _stream(stream)), "diff_attn_backward")


def dcn_output_size(n_in, k, stride, pad, dil):
    return int(_load().dcn_output_size(n_in, k, stride, pad, dil))


def dcn_status_string(status):
    return _load().dcn_status_string(status).decode()


def dcn_last_cuda_error():
    return int(_load().dcn_last_cuda_error())


def dcn_launch_count():
    return int(_load().dcn_launch_count())


def dcn_version():
    return int(_load().dcn_version())


# ------------------------------------------------------------ tensor helpers

def dtype_code(t):
    """dcn_dtype_t of a torch tensor."""
    import torch
    codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    if t.dtype not in codes:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return codes[t.dtype]


def _require(cond, msg):
    if not cond:
        raise ValueError(msg)


def dcn(x, offset, mask, kh=3, kw=3, stride=1, pad=1, dil=1, softmax_flag=0, out=None,
        stream=None, algo="auto"):
    """dcn_forward_algo on torch CUDA tensors; allocates `out` when not given.

    x [N, H, W, C], offset [N, Ho, Wo, G, K, 2], mask [N, Ho, Wo, G, K], all of
    one dtype (float32 / float16 / bfloat16), contiguous, on one CUDA device.
    algo: "auto" (dcn_forward), "gather" or "band".
    """
    import torch
    _require(x.dim() == 4 and mask.dim() == 5 and offset.dim() == 6,
             "expected x [N,H,W,C], offset [N,Ho,Wo,G,K,2], mask [N,Ho,Wo,G,K]")
    N, H, W, C = x.shape
    G = mask.shape[3]
    Ho = dcn_output_size(H, kh, stride, pad, dil)
    Wo = dcn_output_size(W, kw, stride, pad, dil)
    K = kh * kw
    _require(tuple(offset.shape) == (N, Ho, Wo, G, K, 2), "offset has the wrong shape")
    _require(tuple(mask.shape) == (N, Ho, Wo, G, K), "mask has the wrong shape")
    _require(offset.dtype == x.dtype and mask.dtype == x.dtype, "mixed dtypes")
    _require(x.is_cuda and offset.is_cuda and mask.is_cuda, "tensors must be on a CUDA device")
    _require(x.is_contiguous() and offset.is_contiguous() and mask.is_contiguous(),
             "tensors must be contiguous")
    if out is None:
        out = torch.empty((N, Ho, Wo, C), dtype=x.dtype, device=x.device)
    _require(tuple(out.shape) == (N, Ho, Wo, C) and out.dtype == x.dtype and out.is_contiguous(),
             "out has the wrong shape, dtype or layout")
    _require(algo in ALGO_CODES, f"algo must be one of {sorted(ALGO_CODES)}")
    dcn_forward_algo(x, offset, mask, out, N, H, W, C, G, kh, kw, stride, pad, dil,
                     softmax_flag, dtype_code(x), ALGO_CODES[algo], stream)
    return out


def msda(value, spatial_shapes, level_start, sampling_loc, attn_w, out=None, stream=None):
    """msda_forward on torch CUDA tensors; allocates `out` when not given.

    value [N, S, M, D], spatial_shapes [L, 2] int64 (H, W), level_start [L] int64,
    sampling_loc [N, Lq, M, L, K, 2], attn_w [N, Lq, M, L, K].
    """
    import torch
    _require(value.dim() == 4 and attn_w.dim() == 5 and sampling_loc.dim() == 6,
             "expected value [N,S,M,D], loc [N,Lq,M,L,K,2], attn [N,Lq,M,L,K]")
    N, S, M, D = value.shape
    _, Lq, _, L, K = attn_w.shape
    _require(tuple(sampling_loc.shape) == (N, Lq, M, L, K, 2), "sampling_loc has the wrong shape")
    _require(tuple(attn_w.shape[:3]) == (N, Lq, M), "attn_w has the wrong shape")
    _require(tuple(spatial_shapes.shape) == (L, 2) and tuple(level_start.shape) == (L,),
             "spatial_shapes / level_start have the wrong shape")
    _require(spatial_shapes.dtype == torch.int64 and level_start.dtype == torch.int64,
             "spatial_shapes / level_start must be int64")
    _require(sampling_loc.dtype == value.dtype and attn_w.dtype == value.dtype, "mixed dtypes")
    for t in (value, spatial_shapes, level_start, sampling_loc, attn_w):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    if out is None:
        out = torch.empty((N, Lq, M * D), dtype=value.dtype, device=value.device)
    _require(tuple(out.shape) == (N, Lq, M * D) and out.dtype == value.dtype and out.is_contiguous(),
             "out has the wrong shape, dtype or layout")
    msda_forward(value, spatial_shapes, level_start, sampling_loc, attn_w, out, N, Lq, M, D, L,
                 K, dtype_code(value), stream)
    return out


def _workspace(nbytes, device, workspace):
    """A caller-given workspace tensor, or a new one of nbytes (16-byte aligned)."""
    import torch
    if nbytes <= 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes // 4, dtype=torch.float32, device=device)
    _require(workspace.is_cuda and workspace.is_contiguous(), "workspace must be a CUDA tensor")
    _require(workspace.device == device, "workspace must be on the tensors' device")
    have = workspace.numel() * workspace.element_size()
    _require(have >= nbytes, f"workspace holds {have} bytes, {nbytes} needed")
    return workspace, have


def dcn_grad(x, offset, mask, grad_out, kh=3, kw=3, stride=1, pad=1, dil=1, softmax_flag=0,
             workspace=None, stream=None):
    """dcn_backward on torch CUDA tensors: returns (grad_x, grad_offset, grad_mask).

    The float32 accumulator for grad_x of 16-bit data comes from `workspace`
    when given (a CUDA tensor of at least dcn_backward_workspace_size bytes),
    else a new tensor.
    """
    import torch
    _require(x.dim() == 4 and mask.dim() == 5 and offset.dim() == 6,
             "expected x [N,H,W,C], offset [N,Ho,Wo,G,K,2], mask [N,Ho,Wo,G,K]")
    N, H, W, C = x.shape
    G = mask.shape[3]
    Ho = dcn_output_size(H, kh, stride, pad, dil)
    Wo = dcn_output_size(W, kw, stride, pad, dil)
    K = kh * kw
    _require(tuple(offset.shape) == (N, Ho, Wo, G, K, 2), "offset has the wrong shape")
    _require(tuple(mask.shape) == (N, Ho, Wo, G, K), "mask has the wrong shape")
    _require(tuple(grad_out.shape) == (N, Ho, Wo, C), "grad_out has the wrong shape")
    for t in (offset, mask, grad_out):
        _require(t.dtype == x.dtype, "mixed dtypes")
    for t in (x, offset, mask, grad_out):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    code = dtype_code(x)
    ws, ws_bytes = _workspace(dcn_backward_workspace_size(N, H, W, C, code), x.device, workspace)
    gx = torch.empty_like(x)
    goff = torch.empty_like(offset)
    gmask = torch.empty_like(mask)
    dcn_backward(x, offset, mask, grad_out, gx, goff, gmask, ws, ws_bytes, N, H, W, C, G, kh,
                 kw, stride, pad, dil, softmax_flag, code, stream)
    return gx, goff, gmask


def msda_grad(value, spatial_shapes, level_start, sampling_loc, attn_w, grad_out,
              workspace=None, stream=None):
    """msda_backward on torch CUDA tensors: returns (grad_value, grad_loc, grad_attn)."""
    import torch
    N, S, M, D = value.shape
    _, Lq, _, L, K = attn_w.shape
    _require(tuple(sampling_loc.shape) == (N, Lq, M, L, K, 2), "sampling_loc has the wrong shape")
    _require(tuple(grad_out.shape) == (N, Lq, M * D), "grad_out has the wrong shape")
    _require(spatial_shapes.dtype == torch.int64 and level_start.dtype == torch.int64,
             "spatial_shapes / level_start must be int64")
    for t in (sampling_loc, attn_w, grad_out):
        _require(t.dtype == value.dtype, "mixed dtypes")
    for t in (value, spatial_shapes, level_start, sampling_loc, attn_w, grad_out):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    code = dtype_code(value)
    ws, ws_bytes = _workspace(msda_backward_workspace_size(N, S, M, D, code), value.device,
                              workspace)
    gv = torch.empty_like(value)
    gl = torch.empty_like(sampling_loc)
    ga = torch.empty_like(attn_w)
    msda_backward(value, spatial_shapes, level_start, sampling_loc, attn_w, grad_out, gv, gl, ga,
                  ws, ws_bytes, N, S, Lq, M, D, L, K, code, stream)
    return gv, gl, ga


def dynconv(x, weights, K, softmax_flag=1, out=None, stream=None, algo="auto"):
    """dynconv_forward_algo (the ContMix core) on torch CUDA tensors.

    x [N, H, W, C], weights [N, H, W, G, K*K] (tap ky * K + kx), one dtype.
    algo: "auto" (the tensor-core kernel where it applies), "tensor" or "simt".
    """
    import torch
    _require(x.dim() == 4 and weights.dim() == 5, "expected x [N,H,W,C], weights [N,H,W,G,K*K]")
    N, H, W, C = x.shape
    G = weights.shape[3]
    _require(tuple(weights.shape) == (N, H, W, G, K * K), "weights has the wrong shape")
    _require(weights.dtype == x.dtype, "mixed dtypes")
    for t in (x, weights):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    if out is None:
        out = torch.empty_like(x)
    _require(tuple(out.shape) == (N, H, W, C) and out.dtype == x.dtype and out.is_contiguous(),
             "out has the wrong shape, dtype or layout")
    _require(algo in DYNCONV_ALGO_CODES, f"algo must be one of {sorted(DYNCONV_ALGO_CODES)}")
    dynconv_forward_algo(x, weights, out, N, H, W, C, G, K, softmax_flag, dtype_code(x),
                         DYNCONV_ALGO_CODES[algo], stream)
    return out


def msda_points(value, spatial_shapes, level_start, reference, offsets, attn_w,
                valid_ratios=None, out=None, stream=None):
    """msda_forward_points on torch CUDA tensors: reference [N, Lq, 2 or 4],
    offsets [N, Lq, M, L, K, 2], valid_ratios [N, L, 2] or None."""
    import torch
    N, S, M, D = value.shape
    _, Lq, _, L, K = attn_w.shape
    ref_dim = reference.shape[-1]
    _require(tuple(reference.shape) == (N, Lq, ref_dim) and ref_dim in (2, 4),
             "reference must be [N, Lq, 2] or [N, Lq, 4]")
    _require(tuple(offsets.shape) == (N, Lq, M, L, K, 2), "offsets has the wrong shape")
    _require(valid_ratios is None or tuple(valid_ratios.shape) == (N, L, 2),
             "valid_ratios must be [N, L, 2]")
    for t in (value, reference, offsets, attn_w) + ((valid_ratios,) if valid_ratios is not None else ()):
        _require(t.is_cuda and t.is_contiguous() and t.dtype == value.dtype,
                 "tensors must be contiguous CUDA tensors of one dtype")
    if out is None:
        out = torch.empty((N, Lq, M * D), dtype=value.dtype, device=value.device)
    msda_forward_points(value, spatial_shapes, level_start, reference, ref_dim, valid_ratios,
                        offsets, attn_w, out, N, Lq, M, D, L, K, dtype_code(value), stream)
    return out


def mask_value(value, mask, out=None, stream=None):
    """msda_mask_value on torch CUDA tensors (mask [N, S] bool or uint8);
    out=value masks in place."""
    import torch
    N, S, M, D = value.shape
    _require(tuple(mask.shape) == (N, S), "mask must be [N, S]")
    m = mask.to(torch.uint8) if mask.dtype != torch.uint8 else mask
    _require(m.is_cuda and m.is_contiguous() and value.is_contiguous(), "contiguous CUDA tensors")
    if out is None:
        out = torch.empty_like(value)
    msda_mask_value(value, m, out, N, S, M, D, dtype_code(value), stream)
    return out


def dcnv4_fused(x, w_om, b_om=None, groups=4, kh=3, kw=3, pad=1, dil=1, out=None, stream=None,
                algo="auto"):
    """dcnv4_fused_forward_algo on torch CUDA tensors: x [N, H, W, C], w_om
    [G*kh*kw*3, C], b_om [G*kh*kw*3] or None; algo "auto", "gather" or "band"."""
    import torch
    N, H, W, C = x.shape
    J = groups * kh * kw * 3
    _require(tuple(w_om.shape) == (J, C), "w_om must be [G*K*3, C]")
    _require(b_om is None or tuple(b_om.shape) == (J,), "b_om must be [G*K*3]")
    for t in (x, w_om) + ((b_om,) if b_om is not None else ()):
        _require(t.is_cuda and t.is_contiguous() and t.dtype == x.dtype,
                 "tensors must be contiguous CUDA tensors of one dtype")
    if out is None:
        out = torch.empty_like(x)
    _require(algo in ALGO_CODES, f"algo must be one of {sorted(ALGO_CODES)}")
    dcnv4_fused_forward_algo(x, w_om, b_om, out, N, H, W, C, groups, kh, kw, pad, dil,
                             dtype_code(x), ALGO_CODES[algo], stream)
    return out


# ------------------------------------------------ attention-block operators

_HERE = contextlib.nullcontext()


def _scope(t, stream):
    """A context in which the tensor's device and the call's stream are current:
    the launch goes there, and so does the memory that the call allocates (a
    block of the current stream's may still be in use by what runs there)."""
    import torch
    device = t.get_device()
    if stream is None:
        return _HERE if device == torch.cuda.current_device() else torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device=t.device)
    _require(stream.device == t.device, "the stream must be one of the tensors' device")
    return torch.cuda.stream(stream)


def _same_device(first, *rest):
    _require(first.is_cuda, "tensors must be on a CUDA device")
    device = first.get_device()
    for t in rest:
        _require(t is None or t.get_device() == device, "tensors must be on one CUDA device")


def _heads_stride(t, shape, name):
    """(image, token) strides of a [N, L, ...] tensor whose inner dimensions are dense."""
    if t.shape != shape:
        raise ValueError(f"{name} has the wrong shape")
    inner = math.prod(shape[2:])
    if t.is_contiguous():
        return shape[1] * inner, inner
    inner = 1
    for size, stride in zip(reversed(shape[2:]), reversed(t.stride()[2:])):
        _require(size == 1 or stride == inner, f"{name} must be dense in its last dimensions")
        inner *= size
    N, L = shape[:2]
    row = t.stride(1) if L > 1 else inner
    image = t.stride(0) if N > 1 else max(L, 1) * row
    _require((row >= inner and image >= 0) or N * L == 0,
             f"{name} has overlapping tokens or a negative stride")
    return (image, row) if N * L else (L * inner, inner)


def _rope_checks(x, pos, freqs, axis_pairs):
    import torch
    _require(x.dim() == 4 and pos.dim() == 3, "expected x [N,L,M,D], pos [N or 1,L,A]")
    N, L, M, D = x.shape
    A = pos.shape[2]
    _require(pos.shape[0] in (1, N) and pos.shape[1] == L, "pos must be [N or 1, L, A]")
    _require(1 <= A <= 4, "1 to 4 axes")
    _require(len(axis_pairs) == A, "axis_pairs must hold one count per axis")
    _require(all(p >= 0 for p in axis_pairs) and 2 * sum(axis_pairs) <= D,
             "axis_pairs must be non-negative and rotate at most D channels")
    _require(tuple(freqs.shape) == (sum(axis_pairs),), "freqs must hold one value per pair")
    _require(pos.dtype == torch.float32 and freqs.dtype == torch.float32,
             "pos and freqs must be float32")
    _same_device(x, pos, freqs)
    _require(pos.is_contiguous() and freqs.is_contiguous(), "pos and freqs must be contiguous")
    return N, L, M, D, A, _heads_stride(x, (N, L, M, D), "x")


def axial_rope(x, pos, freqs, axis_pairs, interleaved=False, inverse=False, out=None,
               stream=None):
    """Rotary positions over one to four axes (axial_rope_forward).

    x [N, L, M, D] (heads and channels dense; images and tokens may be strided),
    pos [N or 1, L, A] float32, freqs [sum(axis_pairs)] float32; axis_pairs:
    the number of channel pairs each axis turns.  `out` may be x (in place).
    """
    import torch
    N, L, M, D, A, (image, row) = _rope_checks(x, pos, freqs, axis_pairs)
    code = dtype_code(x)
    _require(out is None or (out.shape == x.shape and out.dtype == x.dtype
                             and out.device == x.device and out.is_contiguous()),
             "out has the wrong shape, dtype, device or layout")
    with _scope(x, stream):
        if out is None:
            out = torch.empty((N, L, M, D), dtype=x.dtype, device=x.device)
        axial_rope_forward(x, pos, freqs, out, axis_pairs, N, L, M, D, A, pos.shape[0], image, row,
                           int(bool(interleaved)), int(bool(inverse)), code)
    return out


def axial_rope_grad(x, pos, freqs, axis_pairs, grad_out, interleaved=False, inverse=False,
                    need_pos=True, stream=None):
    """axial_rope_backward: returns (grad_x, grad_pos); grad_pos is None without need_pos."""
    import torch
    N, L, M, D, A, (image, row) = _rope_checks(x, pos, freqs, axis_pairs)
    _require(grad_out.shape == x.shape and grad_out.dtype == x.dtype and grad_out.is_contiguous(),
             "grad_out has the wrong shape, dtype or layout")
    _same_device(x, grad_out)
    code = dtype_code(x)
    with _scope(x, stream):
        gx = torch.empty((N, L, M, D), dtype=x.dtype, device=x.device)
        gp = None
        if need_pos:    # no images: the launch that would fill a shared pos' gradient does not run
            gp = (torch.empty if N else torch.zeros)(pos.shape, dtype=pos.dtype, device=x.device)
        axial_rope_backward(x, pos, freqs, grad_out, gx, gp, axis_pairs, N, L, M, D, A,
                            pos.shape[0], image, row, int(bool(interleaved)), int(bool(inverse)),
                            code)
    return gx, gp


_NORM_FLAGS = {"layer": 0, "rms": DCN_NORM_RMS}


def _norm_checks(rows, factors, norm, post, pre):
    """(N, L, C, flags, dtype code) of dense [N, L, C] tensors and their factors."""
    t = rows[0]
    _require(t.dim() == 3, "expected [N, L, C] tensors")
    N, L, C = t.shape
    _require(norm in _NORM_FLAGS, f"norm must be one of {sorted(_NORM_FLAGS)}")
    _same_device(*rows, *(f for f, _ in factors))
    for r in rows:
        _require(r is None or (r.shape == t.shape and r.dtype == t.dtype and r.is_contiguous()),
                 "row tensors must be contiguous [N, L, C] of one dtype")
    for f, gated in factors:
        shape = (N, C) if gated else (C,)
        _require(f is None or (tuple(f.shape) == shape and f.dtype == t.dtype
                               and f.is_contiguous()),
                 "factors must be contiguous [C] (gate: [N, C]) of the rows' dtype")
    flags = _NORM_FLAGS[norm] | (DCN_NORM_POST if post else 0) | (DCN_NORM_PRE if pre else 0)
    return N, L, C, flags, dtype_code(t)


def norm_residual(x, y, scale=None, gate=None, post_weight=None, post_bias=None, pre_weight=None,
                  pre_bias=None, norm="layer", post=True, pre=True, eps=1e-6, out=None,
                  stream=None):
    """norm_residual_forward: returns (z, h), the joined residual stream and the
    next block's normed input (None without pre).

    z = x + scale * gate * (norm(y) * post_weight + post_bias), h = norm(z) *
    pre_weight + pre_bias; x, y [N, L, C], gate [N, C], the other factors [C].
    norm: "layer" or "rms"; post / pre switch the two norms.  out=x joins in place.
    """
    import torch
    N, L, C, flags, code = _norm_checks(
        (x, y), ((scale, False), (gate, True), (post_weight, False), (post_bias, False),
                 (pre_weight, False), (pre_bias, False)), norm, post, pre)
    _require(out is None or (out.shape == x.shape and out.dtype == x.dtype
                             and out.device == x.device and out.is_contiguous()),
             "out has the wrong shape, dtype, device or layout")
    with _scope(x, stream):
        z = torch.empty_like(x) if out is None else out
        h = torch.empty_like(x) if pre else None
        norm_residual_forward(x, y, scale, gate, post_weight, post_bias, pre_weight, pre_bias, z,
                              h, N, L, C, flags, eps, code)
    return z, h


def norm_residual_grad(y, z, grad_z, grad_h=None, scale=None, gate=None, post_weight=None,
                       post_bias=None, pre_weight=None, pre_bias=None, norm="layer", post=True,
                       pre=True, eps=1e-6, workspace=None, stream=None):
    """norm_residual_backward: returns (grad_x, grad_y, grad_scale, grad_gate,
    grad_post_weight, grad_post_bias, grad_pre_weight, grad_pre_bias), None for
    the factors that are None.  z is norm_residual's first output."""
    import torch
    N, L, C, flags, code = _norm_checks(
        (y, z, grad_z, grad_h),
        ((scale, False), (gate, True), (post_weight, False), (post_bias, False),
         (pre_weight, False), (pre_bias, False)), norm, post, pre)
    _require((grad_h is not None) == bool(pre), "grad_h belongs to pre=True")

    def like(f):
        return None if f is None else torch.empty_like(f)

    with _scope(y, stream):
        gx, gy = torch.empty_like(y), torch.empty_like(y)
        gs, gg, gpw, gpb = like(scale), like(gate), like(post_weight), like(post_bias)
        gqw, gqb = like(pre_weight), like(pre_bias)
        need = norm_residual_backward_workspace_size(N, L, C, 0 if gate is None else 1, code)
        if need < 0:
            raise DcnError(need, "norm_residual_backward_workspace_size")
        ws, ws_bytes = _workspace(need, y.device, workspace)
        norm_residual_backward(y, z, grad_z, grad_h, scale, gate, post_weight, post_bias,
                               pre_weight, gx, gy, gs, gg, gpw, gpb, gqw, gqb, ws, ws_bytes, N, L,
                               C, flags, eps, code)
    return gx, gy, gs, gg, gpw, gpb, gqw, gqb


def _attn_checks(q, k, v, lam, mask, lengths):
    import torch
    _require(q.dim() == 5 and k.dim() == 5 and v.dim() == 4,
             "expected q [N,Lq,M,2,D], k [N,Lk,Mk,2,D], v [N,Lk,Mk,Dv]")
    N, Lq, M, _, D = q.shape
    Lk, Mk, Dv = v.shape[1:]
    _require(Mk > 0 and M % Mk == 0, "the heads must be a multiple of the key / value heads")
    _same_device(q, k, v, lam, mask, lengths)
    for t in (k, v, lam):
        _require(t.dtype == q.dtype, "mixed dtypes")
    strides = (_heads_stride(q, (N, Lq, M, 2, D), "q") + _heads_stride(k, (N, Lk, Mk, 2, D), "k") +
               _heads_stride(v, (N, Lk, Mk, Dv), "v"))
    _require(tuple(lam.shape) == (M,) and lam.is_contiguous(), "lam must be a contiguous [M]")
    if mask is not None:
        _require(tuple(mask.shape) == (N, Lk) and mask.is_contiguous()
                 and mask.dtype in (torch.bool, torch.uint8), "mask must be [N, Lk] bool or uint8")
    _require(lengths is None or (tuple(lengths.shape) == (N,) and lengths.dtype == torch.int32
                                 and lengths.is_contiguous()), "lengths must be [N] int32")
    return (N, Lq, Lk, M, Mk, D, Dv), strides


def diff_attn(q, k, v, lam, mask=None, lengths=None, causal=False, scale=None, save=False,
              out=None, workspace=None, stream=None):
    """diff_attn_forward: out [N, Lq, M, Dv] of differential attention,
    (softmax(scale q_0 k_0^T) - lam softmax(scale q_1 k_1^T)) v.

    q [N, Lq, M, 2, D], k [N, Lk, Mk, 2, D], v [N, Lk, Mk, Dv] (images and
    tokens may be strided), lam [M]; mask [N, Lk], true where a key is hidden;
    lengths [N] int32, the keys in use; causal: the tokens are the last Lq of
    those.  scale: 1 / sqrt(D) unless given.  save=True returns (out, saved)
    with what diff_attn_grad needs.
    """
    import torch
    (N, Lq, Lk, M, Mk, D, Dv), strides = _attn_checks(q, k, v, lam, mask, lengths)
    code = dtype_code(q)
    _require(out is None or (tuple(out.shape) == (N, Lq, M, Dv) and out.dtype == q.dtype
                             and out.device == q.device and out.is_contiguous()),
             "out has the wrong shape, dtype, device or layout")
    maps = lse = None
    with _scope(q, stream):
        if out is None:
            out = torch.empty((N, Lq, M, Dv), dtype=q.dtype, device=q.device)
        if save:
            maps = torch.empty((N, Lq, M, 2, Dv), dtype=torch.float32, device=q.device)
            lse = torch.empty((N, M, 2, Lq), dtype=torch.float32, device=q.device)
        need = diff_attn_forward_workspace_size(N, Lq, Lk, M, Mk, D, Dv, code)
        if need < 0:
            raise DcnError(need, "diff_attn_forward_workspace_size")
        ws, ws_bytes = _workspace(need, q.device, workspace)
        diff_attn_forward(q, k, v, lam, mask, lengths, out, maps, lse, ws, ws_bytes, N, Lq, Lk, M,
                          Mk, D, Dv, *strides, D ** -0.5 if scale is None else scale,
                          int(bool(causal)), code)
    return (out, (maps, lse)) if save else out


def diff_attn_grad(q, k, v, lam, out, saved, grad_out, mask=None, lengths=None, causal=False,
                   scale=None, workspace=None, stream=None):
    """diff_attn_backward: returns (grad_q, grad_k, grad_v, grad_lam), dense;
    saved: the second of what diff_attn(..., save=True) returned for these
    inputs.  out, the first, is not read (the maps' own outputs in `saved` are):
    it may be None, and need not be kept."""
    import torch
    (N, Lq, Lk, M, Mk, D, Dv), strides = _attn_checks(q, k, v, lam, mask, lengths)
    code = dtype_code(q)
    maps, lse = saved
    _same_device(q, out, maps, lse, grad_out)
    for t in (grad_out,) if out is None else (out, grad_out):
        _require(tuple(t.shape) == (N, Lq, M, Dv) and t.dtype == q.dtype and t.is_contiguous(),
                 "out and grad_out must be contiguous [N, Lq, M, Dv] of q's dtype")
    for t, shape in ((maps, (N, Lq, M, 2, Dv)), (lse, (N, M, 2, Lq))):
        _require(tuple(t.shape) == shape and t.dtype == torch.float32 and t.is_contiguous(),
                 "saved must be diff_attn's")
    with _scope(q, stream):
        gq = torch.empty((N, Lq, M, 2, D), dtype=q.dtype, device=q.device)
        gk = torch.empty((N, Lk, Mk, 2, D), dtype=q.dtype, device=q.device)
        gv = torch.empty((N, Lk, Mk, Dv), dtype=q.dtype, device=q.device)
        gl = torch.empty_like(lam)
        need = diff_attn_backward_workspace_size(N, Lq, Lk, M, Mk, D, Dv, code)
        if need < 0:
            raise DcnError(need, "diff_attn_backward_workspace_size")
        ws, ws_bytes = _workspace(need, q.device, workspace)
        diff_attn_backward(q, k, v, lam, mask, lengths, maps, lse, grad_out, gq, gk, gv, gl,
                           ws, ws_bytes, N, Lq, Lk, M, Mk, D, Dv, *strides,
                           D ** -0.5 if scale is None else scale, int(bool(causal)), code)
    return gq, gk, gv, gl
