"""Thin Python binding of the C ABI in include/headloss.h (ctypes).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libheadloss.so.  Tensors are passed as raw device pointers; torch
is used for device memory and streams.  There is no fallback: if the library
is not built, every call raises.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libheadloss.so")

# enum headloss_flag
HEADLOSS_CE = 1 << 0
HEADLOSS_Z = 1 << 1
HEADLOSS_DIST_CE = 1 << 2
HEADLOSS_FKL = 1 << 3
HEADLOSS_RKL = 1 << 4
HEADLOSS_GRPO = 1 << 5
HEADLOSS_GRPO_STATS = 1 << 6
HEADLOSS_ENTROPY = 1 << 7

# enum headloss_dtype
HEADLOSS_FP32, HEADLOSS_BF16, HEADLOSS_FP16 = 0, 1, 2

# enum headloss_fp8
HEADLOSS_E4M3, HEADLOSS_E5M2 = 0, 1

# enum headloss_status
STATUS = {0: "HEADLOSS_OK", 1: "HEADLOSS_ERR_ARG", 2: "HEADLOSS_ERR_DTYPE",
          3: "HEADLOSS_ERR_ALIGN", 4: "HEADLOSS_ERR_MISSING_INPUT", 5: "HEADLOSS_ERR_CUDA",
          6: "HEADLOSS_ERR_TIMEOUT", 7: "HEADLOSS_ERR_LABEL_RANGE", 8: "HEADLOSS_ERR_SIZE"}
HEADLOSS_OK = 0
HEADLOSS_ERR_ARG = 1
HEADLOSS_ERR_DTYPE = 2
HEADLOSS_ERR_ALIGN = 3
HEADLOSS_ERR_MISSING_INPUT = 4
HEADLOSS_ERR_CUDA = 5
HEADLOSS_ERR_TIMEOUT = 6
HEADLOSS_ERR_LABEL_RANGE = 7
HEADLOSS_ERR_SIZE = 8

# enum headloss_slot
SLOTS = ("total", "ce", "z", "dist_ce", "fkl", "rkl", "grpo_loss", "new_logprob_mean",
         "ratio_mean", "clip_frac", "kl_k3", "adv_mean", "adv_std", "entropy_mean", "n_valid",
         "n_clipped")

# Every function declared in the headers under include/.
EXPORTS = ("headloss_create", "headloss_forward_backward", "headloss_get_device_error",
           "headloss_plan", "headloss_force_plan", "headloss_launches_per_call",
           "headloss_destroy", "headloss_strerror", "headloss_version",
           "headloss_forward_backward_noalloc", "headloss_forward_backward_ext",
           "headloss_gspo_seam", "headloss_forward_backward_rowstats",
           "headloss_lmhead_logits", "headloss_lmhead_logits_rowstats",
           "headloss_sample", "headloss_clip_create", "headloss_clip_grads",
           "headloss_clip_destroy", "headloss_fp8_quantize", "headloss_fp8_workspace",
           "headloss_fp8_matmul", "headloss_fp8_linear_workspace", "headloss_fp8_linear",
           "headloss_beam_workspace", "headloss_beam_select",
           "headloss_reorder_create", "headloss_reorder", "headloss_reorder_destroy")


# enum headloss_kernel
HEADLOSS_KERNEL_AUTO, HEADLOSS_KERNEL_RESIDENT, HEADLOSS_KERNEL_STREAM = 0, 1, 2
KERNELS = {0: "auto", 1: "resident", 2: "stream"}


class headloss_call_ext(ctypes.Structure):
    """struct headloss_call_ext: per-call extras (per-token outputs, gradient
    accumulation, the divisor of a split batch)."""
    _fields_ = [("new_logprobs", ctypes.c_void_p), ("row_loss", ctypes.c_void_p),
                ("accumulate", ctypes.c_int), ("divisor", ctypes.c_double),
                ("token_coeff", ctypes.c_void_p)]


class headloss_gradient(ctypes.Structure):
    """struct headloss_gradient: one tensor of a clipping call."""
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


class headloss_state(ctypes.Structure):
    """struct headloss_state: one tensor of beams' states."""
    _fields_ = [("state", ctypes.c_void_p), ("out", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("outer", "positions", "run_bytes", "row_stride",
                                      "outer_stride", "position_stride")]


class headloss_plan_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("kernel", "cluster", "stages", "threads",
                                             "chunk_words")]


class headloss_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_float) for n in
                ("ce", "z", "dist_ce", "fkl", "rkl", "grpo", "entropy", "grad_scale")]


class HeadlossError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_strerror(status)})")


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libheadloss.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with gradient_row_online_gb300.build.build()")
    lib = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    ip = ctypes.POINTER(ctypes.c_int)
    lib.headloss_create.argtypes = [ctypes.c_uint32, ctypes.POINTER(headloss_weights),
                                    ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                    ctypes.c_float, ctypes.POINTER(vp)]
    lib.headloss_create.restype = i32
    lib.headloss_forward_backward.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.headloss_forward_backward.restype = i32
    lib.headloss_get_device_error.argtypes = [vp, vp, ip]
    lib.headloss_get_device_error.restype = i32
    pp = ctypes.POINTER(headloss_plan_desc)
    lib.headloss_plan.argtypes = [vp, i64, i32, pp, ip, ip]
    lib.headloss_plan.restype = i32
    lib.headloss_force_plan.argtypes = [vp, pp]
    lib.headloss_force_plan.restype = i32
    lib.headloss_launches_per_call.argtypes = []
    lib.headloss_launches_per_call.restype = i32
    lib.headloss_destroy.argtypes = [vp]
    lib.headloss_destroy.restype = None
    lib.headloss_strerror.argtypes = [i32]
    lib.headloss_strerror.restype = ctypes.c_char_p
    lib.headloss_version.argtypes = []
    lib.headloss_version.restype = i32
    lib.headloss_forward_backward_noalloc.argtypes = [
        ctypes.c_uint32, ctypes.POINTER(headloss_weights), ctypes.c_float, ctypes.c_float,
        ctypes.c_float, ctypes.c_float, vp, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.headloss_forward_backward_noalloc.restype = i32
    lib.headloss_forward_backward_ext.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp, vp, vp, vp,
                                                  ctypes.POINTER(headloss_call_ext), vp]
    lib.headloss_forward_backward_ext.restype = i32
    lib.headloss_lmhead_logits.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp]
    lib.headloss_lmhead_logits.restype = i32
    lib.headloss_gspo_seam.argtypes = [vp, vp, vp, vp, i64, i64, vp, i32, f32, f32, f32, vp, vp,
                                       vp]
    lib.headloss_gspo_seam.restype = i32
    lib.headloss_lmhead_logits_rowstats.argtypes = [vp, vp, i32, i32, i32, f32, f32, f32, vp, vp,
                                                    vp, vp, vp]
    lib.headloss_lmhead_logits_rowstats.restype = i32
    lib.headloss_forward_backward_rowstats.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp, vp, vp,
                                                       vp, vp, vp, vp, vp, vp]
    lib.headloss_forward_backward_rowstats.restype = i32
    lib.headloss_sample.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp, vp, vp, f32, f32, vp, vp,
                                    vp, vp, vp, vp]
    lib.headloss_sample.restype = i32
    lib.headloss_clip_create.argtypes = [i32, ctypes.POINTER(vp)]
    lib.headloss_clip_create.restype = i32
    lib.headloss_clip_grads.argtypes = [vp, ctypes.POINTER(headloss_gradient), i32, f32, f32, vp,
                                        vp]
    lib.headloss_clip_grads.restype = i32
    lib.headloss_clip_destroy.argtypes = [vp]
    lib.headloss_clip_destroy.restype = None
    lib.headloss_fp8_quantize.argtypes = [vp, i64, i64, i64, i32, i32, vp, i64, vp, i32, vp, i64, vp,
                                          i32, vp]
    lib.headloss_fp8_quantize.restype = i32
    lib.headloss_fp8_workspace.argtypes = [i64, i64, i64]
    lib.headloss_fp8_workspace.restype = i64
    lib.headloss_fp8_matmul.argtypes = [vp, i64, vp, i32, vp, i64, vp, i32, i64, i64, i64, vp, i64, i32,
                                        vp, i64, vp, vp]
    lib.headloss_fp8_matmul.restype = i32
    lib.headloss_fp8_linear_workspace.argtypes = [i64, i64, i64]
    lib.headloss_fp8_linear_workspace.restype = i64
    lib.headloss_fp8_linear.argtypes = [vp, i64, i32, vp, i64, vp, i32, i64, i64, i64, vp, i64, i32, vp,
                                        i64, vp, vp]
    lib.headloss_fp8_linear.restype = i32
    lib.headloss_beam_workspace.argtypes = [i64, i32, i64, i32, i32]
    lib.headloss_beam_workspace.restype = i64
    lib.headloss_beam_select.argtypes = [vp, i64, i32, i64, i64, i32, vp, vp, i64, i32, i32, f32, f32,
                                         vp, vp, vp, vp, vp, i64, vp]
    lib.headloss_beam_select.restype = i32
    lib.headloss_reorder_create.argtypes = [ctypes.POINTER(headloss_state), i32, i32,
                                            ctypes.POINTER(vp)]
    lib.headloss_reorder_create.restype = i32
    lib.headloss_reorder.argtypes = [vp, vp, i64, vp, vp, vp]
    lib.headloss_reorder.restype = i32
    lib.headloss_reorder_destroy.argtypes = [vp]
    lib.headloss_reorder_destroy.restype = None
    _lib = lib
    return lib


def _strerror(status: int) -> str:
    try:
        return load_library().headloss_strerror(status).decode()
    except Exception:
        return "?"


def _check(status: int, where: str):
    if status != HEADLOSS_OK:
        raise HeadlossError(status, where)


def _ptr(a):
    """Device address of a tensor (or an int address, or None)."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


def _stream(stream):
    if stream is None:
        try:
            import torch
            return torch.cuda.current_stream().cuda_stream
        except Exception:
            return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dtype_code(torch_dtype) -> int:
    import torch
    return {torch.float32: HEADLOSS_FP32, torch.bfloat16: HEADLOSS_BF16,
            torch.float16: HEADLOSS_FP16}[torch_dtype]


def make_weights(ce=1.0, z=0.0, dist_ce=0.0, fkl=0.0, rkl=0.0, grpo=1.0, entropy=0.0,
                 grad_scale=1.0) -> headloss_weights:
    return headloss_weights(ce, z, dist_ce, fkl, rkl, grpo, entropy, grad_scale)


def headloss_create(flags: int, weights=None, temperature: float = 1.0, clip_eps: float = 0.2,
                    softcap: float = 0.0, logits_scale: float = 1.0) -> int:
    lib = load_library()
    if isinstance(weights, dict):
        weights = make_weights(**weights)
    h = ctypes.c_void_p()
    w = ctypes.byref(weights) if weights is not None else None
    _check(lib.headloss_create(flags, w, temperature, clip_eps, softcap, logits_scale,
                               ctypes.byref(h)), "headloss_create")
    return h.value


def headloss_forward_backward(h, logits, N, V, dtype, labels, teacher_logits, old_logprobs,
                              advantages, grad_out, scalars_out, stream=None) -> None:
    lib = load_library()
    _check(lib.headloss_forward_backward(h, _ptr(logits), int(N), int(V), int(dtype),
                                         _ptr(labels), _ptr(teacher_logits), _ptr(old_logprobs),
                                         _ptr(advantages), _ptr(grad_out), _ptr(scalars_out),
                                         _stream(stream)), "headloss_forward_backward")


def headloss_forward_backward_ext(h, logits, N, V, dtype, labels, teacher_logits, old_logprobs,
                                  advantages, grad_out, scalars_out, new_logprobs=None,
                                  row_loss=None, accumulate=False, divisor=0.0,
                                  token_coeff=None, stream=None) -> None:
    """The call with its extras: per-row log p(label) and total loss outputs,
    gradient accumulation into grad_out, the divisor of a split batch, and a
    per-token coefficient on the label column (GSPO's, from headloss_gspo_seam)."""
    lib = load_library()
    ext = headloss_call_ext(_ptr(new_logprobs), _ptr(row_loss), int(bool(accumulate)),
                            float(divisor), _ptr(token_coeff))
    _check(lib.headloss_forward_backward_ext(h, _ptr(logits), int(N), int(V), int(dtype),
                                             _ptr(labels), _ptr(teacher_logits),
                                             _ptr(old_logprobs), _ptr(advantages),
                                             _ptr(grad_out), _ptr(scalars_out),
                                             ctypes.byref(ext), _stream(stream)),
           "headloss_forward_backward_ext")


def headloss_forward_backward_noalloc(flags, weights, temperature, clip_eps, softcap,
                                      logits_scale, logits, N, V, dtype, labels, teacher_logits,
                                      old_logprobs, advantages, grad_out, scalars_out,
                                      stream=None) -> None:
    """The allocation-free call (no handle): for callers that must not allocate
    device memory while computing the loss, e.g. inside a CUDA-graph capture."""
    lib = load_library()
    if isinstance(weights, dict):
        weights = make_weights(**weights)
    w = ctypes.byref(weights) if weights is not None else None
    _check(lib.headloss_forward_backward_noalloc(
        flags, w, temperature, clip_eps, softcap, logits_scale, _ptr(logits), int(N), int(V),
        int(dtype), _ptr(labels), _ptr(teacher_logits), _ptr(old_logprobs), _ptr(advantages),
        _ptr(grad_out), _ptr(scalars_out), _stream(stream)), "headloss_forward_backward_noalloc")


def headloss_lmhead_logits(hidden, weight, N, D, V, logits, stats, err, stream=None) -> None:
    """logits = hidden . weight^T and per-(row, 256-column tile) (max, sum exp)
    statistics (include/headloss_lmhead.h); raises HeadlossError on a bad status."""
    _check(load_library().headloss_lmhead_logits(_ptr(hidden), _ptr(weight), int(N), int(D),
                                                 int(V), _ptr(logits), _ptr(stats), _ptr(err),
                                                 _stream(stream)),
           "headloss_lmhead_logits")


def headloss_lmhead_logits_rowstats(hidden, weight, N, D, V, softcap, logits_scale, logits,
                                    row_stats, err, stream=None, temperature=1.0,
                                    row_stats_t=None) -> None:
    """The LM-head GEMM with the loss's per-tile first-pass records, and with
    row_stats_t the tiles' sums at `temperature` (include/headloss_lmhead.h);
    raises HeadlossError on a bad status."""
    _check(load_library().headloss_lmhead_logits_rowstats(
        _ptr(hidden), _ptr(weight), int(N), int(D), int(V), float(softcap), float(logits_scale),
        float(temperature), _ptr(logits), _ptr(row_stats), _ptr(row_stats_t), _ptr(err),
        _stream(stream)), "headloss_lmhead_logits_rowstats")


def headloss_forward_backward_rowstats(h, logits, N, V, dtype, labels, old_logprobs, advantages,
                                       row_stats, grad_out, scalars_out, stream=None,
                                       teacher=None, row_stats_t=None, teacher_stats=None,
                                       new_logprobs=None, row_loss=None, accumulate=False,
                                       divisor=0.0, token_coeff=None) -> None:
    """The loss's gradient pass alone from the GEMMs' row statistics (the
    student's, its sums at the temperature, the teacher's; include/headloss.h),
    with the extras of headloss_forward_backward_ext; raises HeadlossError on a
    bad status."""
    ext = headloss_call_ext(_ptr(new_logprobs), _ptr(row_loss), int(bool(accumulate)),
                            float(divisor), _ptr(token_coeff))
    _check(load_library().headloss_forward_backward_rowstats(
        h, _ptr(logits), int(N), int(V), int(dtype), _ptr(labels), _ptr(teacher),
        _ptr(old_logprobs), _ptr(advantages), _ptr(row_stats), _ptr(row_stats_t),
        _ptr(teacher_stats), _ptr(grad_out), _ptr(scalars_out), ctypes.byref(ext),
        _stream(stream)), "headloss_forward_backward_rowstats")


def headloss_gspo_seam(new_logprobs, old_logprobs, advantages, labels, N, V, seg_offsets, n_seg,
                       clip_eps, weight, grad_scale, token_coeff, scalars_out,
                       stream=None) -> None:
    """GSPO's per-segment seam (include/headloss.h): the sequence ratios and
    the per-token coefficient for the backward call; raises on a bad status."""
    _check(load_library().headloss_gspo_seam(
        _ptr(new_logprobs), _ptr(old_logprobs), _ptr(advantages), _ptr(labels), int(N), int(V),
        _ptr(seg_offsets), int(n_seg), float(clip_eps), float(weight), float(grad_scale),
        _ptr(token_coeff), _ptr(scalars_out), _stream(stream)), "headloss_gspo_seam")


def headloss_sample(logits, N, V, ld, dtype, uniforms, temperature, top_k, top_p, min_p, softcap,
                    logits_scale, tokens, logprobs, draw_logprobs, n_kept, err,
                    stream=None) -> None:
    """One token a row from the head's logits (include/headloss_sample.h); raises
    HeadlossError on a bad status."""
    _check(load_library().headloss_sample(
        _ptr(logits), int(N), int(V), int(ld), int(dtype), _ptr(uniforms), _ptr(temperature),
        _ptr(top_k), _ptr(top_p), _ptr(min_p), float(softcap), float(logits_scale), _ptr(tokens),
        _ptr(logprobs), _ptr(draw_logprobs), _ptr(n_kept), _ptr(err), _stream(stream)),
        "headloss_sample")


def headloss_clip_create(max_grads: int) -> int:
    h = ctypes.c_void_p()
    _check(load_library().headloss_clip_create(int(max_grads), ctypes.byref(h)),
           "headloss_clip_create")
    return h.value


def headloss_clip_grads(h, grads, n_grads, max_norm, inv_scale, stats_out, stream=None) -> None:
    """Global norm and clipping of a list of tensors (include/headloss_clip.h);
    `grads` is an array of headloss_gradient; raises HeadlossError on a bad status."""
    _check(load_library().headloss_clip_grads(h, grads, int(n_grads), float(max_norm),
                                              float(inv_scale), _ptr(stats_out),
                                              _stream(stream)), "headloss_clip_grads")


def headloss_clip_destroy(h) -> None:
    if h:
        load_library().headloss_clip_destroy(h)


def headloss_fp8_quantize(x, rows, cols, ld, dtype, type, q, ldq, scales, block, qt, ldqt, scales_t,
                          block_t, stream=None) -> None:
    """A matrix and / or its transpose in 8 bits (include/headloss_fp8.h); raises
    HeadlossError on a bad status."""
    _check(load_library().headloss_fp8_quantize(
        _ptr(x), int(rows), int(cols), int(ld), int(dtype), int(type), _ptr(q), int(ldq),
        _ptr(scales), int(block), _ptr(qt), int(ldqt), _ptr(scales_t), int(block_t),
        _stream(stream)), "headloss_fp8_quantize")


def headloss_fp8_workspace(M, N, K) -> int:
    return load_library().headloss_fp8_workspace(int(M), int(N), int(K))


def headloss_fp8_matmul(a, lda, a_scales, a_type, b, ldb, b_scales, b_type, M, N, K, out, ldo,
                        out_dtype, workspace, workspace_bytes, err, stream=None) -> None:
    """out = a . b^T of 8-bit matrices (include/headloss_fp8.h); raises HeadlossError on
    a bad status."""
    _check(load_library().headloss_fp8_matmul(
        _ptr(a), int(lda), _ptr(a_scales), int(a_type), _ptr(b), int(ldb), _ptr(b_scales),
        int(b_type), int(M), int(N), int(K), _ptr(out), int(ldo), int(out_dtype),
        _ptr(workspace), int(workspace_bytes), _ptr(err), _stream(stream)),
        "headloss_fp8_matmul")


def headloss_fp8_linear_workspace(M, N, K) -> int:
    return load_library().headloss_fp8_linear_workspace(int(M), int(N), int(K))


def headloss_fp8_linear(x, ldx, dtype, b, ldb, b_scales, b_type, M, N, K, out, ldo, out_dtype, workspace,
                        workspace_bytes, err, stream=None) -> None:
    """out = x . b^T with x quantised on the way (include/headloss_fp8.h); raises HeadlossError
    on a bad status."""
    _check(load_library().headloss_fp8_linear(
        _ptr(x), int(ldx), int(dtype), _ptr(b), int(ldb), _ptr(b_scales), int(b_type), int(M), int(N),
        int(K), _ptr(out), int(ldo), int(out_dtype), _ptr(workspace), int(workspace_bytes), _ptr(err),
        _stream(stream)), "headloss_fp8_linear")


def headloss_beam_workspace(requests, beams, V, dtype, keep) -> int:
    return load_library().headloss_beam_workspace(int(requests), int(beams), int(V), int(dtype),
                                                  int(keep))


def headloss_beam_select(logits, requests, beams, V, ld, dtype, scores, ended, eos, keep, stay,
                         softcap, logits_scale, out_scores, parents, tokens, out_ended, workspace,
                         workspace_bytes, stream=None) -> None:
    """The best continuations of each request's beams (include/headloss_beam.h); raises
    HeadlossError on a bad status."""
    _check(load_library().headloss_beam_select(
        _ptr(logits), int(requests), int(beams), int(V), int(ld), int(dtype), _ptr(scores),
        _ptr(ended), int(eos), int(keep), int(stay), float(softcap), float(logits_scale),
        _ptr(out_scores), _ptr(parents), _ptr(tokens), _ptr(out_ended), _ptr(workspace),
        int(workspace_bytes), _stream(stream)), "headloss_beam_select")


def headloss_reorder_create(states, n: int, beams: int) -> int:
    """A handle for `n` states (an array of headloss_state) of beams."""
    h = ctypes.c_void_p()
    _check(load_library().headloss_reorder_create(states, int(n), int(beams), ctypes.byref(h)),
           "headloss_reorder_create")
    return h.value


def headloss_reorder(h, parents, requests, begin=None, end=None, stream=None) -> None:
    """The beams take their parents' states (include/headloss_beam.h); raises HeadlossError
    on a bad status."""
    _check(load_library().headloss_reorder(h, _ptr(parents), int(requests), _ptr(begin), _ptr(end),
                                           _stream(stream)), "headloss_reorder")


def headloss_reorder_destroy(h) -> None:
    if h:
        load_library().headloss_reorder_destroy(h)


def headloss_get_device_error(h, stream=None) -> int:
    lib = load_library()
    e = ctypes.c_int()
    _check(lib.headloss_get_device_error(h, _stream(stream), ctypes.byref(e)),
           "headloss_get_device_error")
    return e.value


def headloss_plan(h, V: int, dtype: int) -> dict:
    lib = load_library()
    d = headloss_plan_desc()
    ctas, smem = ctypes.c_int(), ctypes.c_int()
    _check(lib.headloss_plan(h, int(V), int(dtype), ctypes.byref(d), ctypes.byref(ctas),
                             ctypes.byref(smem)), "headloss_plan")
    return dict(kernel=KERNELS[d.kernel], cluster=d.cluster, stages=d.stages,
                threads=d.threads, chunk_words=d.chunk_words, ctas=ctas.value,
                smem_bytes=smem.value)


def headloss_force_plan(h, kernel: int = 0, cluster: int = 0, stages: int = 0, threads: int = 0,
                        chunk_words: int = 0) -> None:
    """Pin plan choices (0 = the planner decides); all zero restores the automatic plan."""
    d = headloss_plan_desc(int(kernel), int(cluster), int(stages), int(threads), int(chunk_words))
    _check(load_library().headloss_force_plan(h, ctypes.byref(d)), "headloss_force_plan")


def headloss_launches_per_call() -> int:
    return load_library().headloss_launches_per_call()


def headloss_destroy(h) -> None:
    if h:
        load_library().headloss_destroy(h)


def headloss_strerror(status: int) -> str:
    return load_library().headloss_strerror(int(status)).decode()


def headloss_version() -> int:
    return load_library().headloss_version()


class HeadLoss:
    """A handle plus the call on torch tensors (same semantics as the C ABI)."""

    def __init__(self, flags: int, weights=None, temperature: float = 1.0,
                 clip_eps: float = 0.2, softcap: float = 0.0, logits_scale: float = 1.0):
        self.flags = flags
        self.h = headloss_create(flags, weights, temperature, clip_eps, softcap, logits_scale)

    def __call__(self, logits, labels=None, teacher_logits=None, old_logprobs=None,
                 advantages=None, grad_out=None, scalars_out=None, stream=None,
                 new_logprobs=None, row_loss=None, accumulate=False, divisor=0.0):
        import torch
        N, V = logits.shape
        if scalars_out is None:
            scalars_out = torch.empty(16, dtype=torch.float32, device=logits.device)
        if new_logprobs is None and row_loss is None and not accumulate and not divisor:
            headloss_forward_backward(self.h, logits, N, V, dtype_code(logits.dtype), labels,
                                      teacher_logits, old_logprobs, advantages, grad_out,
                                      scalars_out, stream)
        else:
            headloss_forward_backward_ext(self.h, logits, N, V, dtype_code(logits.dtype), labels,
                                          teacher_logits, old_logprobs, advantages, grad_out,
                                          scalars_out, new_logprobs, row_loss, accumulate,
                                          divisor, stream)
        return scalars_out

    def plan(self, V: int, dtype: int) -> dict:
        return headloss_plan(self.h, V, dtype)

    def force_plan(self, kernel: int = 0, cluster: int = 0, stages: int = 0, threads: int = 0,
                   chunk_words: int = 0) -> None:
        headloss_force_plan(self.h, kernel, cluster, stages, threads, chunk_words)

    def device_error(self, stream=None) -> int:
        return headloss_get_device_error(self.h, stream)

    def close(self):
        if self.h:
            headloss_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_get_raw_stream = _get_device = None


def _raw_stream(device: int) -> int:
    """The current stream's handle, without the Stream object torch would make."""
    global _get_raw_stream
    if _get_raw_stream is None:
        import torch
        _get_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _get_raw_stream(device)


def _current_device() -> int:
    """The device that the library's calls launch on."""
    global _get_device
    if _get_device is None:
        import torch
        _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _get_device()


def _torch_stream(stream, device: int):
    """The torch stream of a `stream` argument (a torch stream or a handle)."""
    import torch
    if not isinstance(stream, int):
        if stream.device.index != device:
            raise ValueError(f"stream: one of cuda:{device} is wanted, not of {stream.device}")
        return stream
    if stream in (0, 1):  # the default stream (NULL, cudaStreamLegacy), which torch has no external for
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(stream, device)


@contextlib.contextmanager
def _on(device: int, stream):
    """`device` and a stream of it (None: its current one) as the current ones."""
    import torch
    with torch.cuda.device(device), torch.cuda.stream(
            None if stream is None else _torch_stream(stream, device)):
        yield


class HeadSampler:
    """headloss_sample on torch tensors: one token a row of `logits` (N x V, unit
    column stride, any row stride), from one uniform a row.

    The settings are per-row tensors (temperature, top_p, min_p fp32; top_k
    int32), numbers for every row, or None (off).  Returns (tokens int64, log p
    at T = 1 of the whole softmax fp32, log p under the distribution drawn from
    fp32, tokens that could be drawn int32); `out` gives the four buffers.  With
    `stream` the call is as under torch.cuda.stream: its own tensors are made there.
    (The error word is made with the sampler, on the stream that is current then.)"""

    def __init__(self, softcap: float = 0.0, logits_scale: float = 1.0, device="cuda"):
        import torch
        self.softcap, self.logits_scale = float(softcap), float(logits_scale)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.device, self.index = self.err.device, self.err.get_device()
        self._call = load_library().headloss_sample
        self._empty = torch.empty
        self._f32, self._i32 = torch.float32, torch.int32
        self._f64, self._i64 = torch.float64, torch.int64
        self._codes = {torch.float32: HEADLOSS_FP32, torch.bfloat16: HEADLOSS_BF16,
                       torch.float16: HEADLOSS_FP16}

    def _given(self, name, a, dtype, N):
        """The address of a setting (None: 0), and what keeps it alive."""
        if a is None:
            return None, None
        if isinstance(a, (int, float)):
            import torch
            a = torch.full((N,), a, dtype=dtype, device=self.device)
        elif (a.dtype is not dtype or a.dim() != 1 or a.numel() != N or
              a.get_device() != self.index or not a.is_contiguous()):
            raise ValueError(f"{name}: a contiguous {dtype} tensor of {N} on {self.device} is "
                             "wanted")
        return a.data_ptr(), a

    def __call__(self, logits, uniforms, temperature=None, top_k=None, top_p=None, min_p=None,
                 out=None, stream=None):
        if stream is not None or _current_device() != self.index:
            with _on(self.index, stream):
                return self(logits, uniforms, temperature, top_k, top_p, min_p, out)
        if (logits.dim() != 2 or logits.get_device() != self.index or logits.shape[1] < 1 or
                (logits.shape[1] > 1 and logits.stride(1) != 1)):
            raise ValueError("logits: an N x V tensor with unit column stride on "
                             f"{self.device} is wanted")
        N, V = logits.shape
        code = self._codes.get(logits.dtype)
        if code is None:
            raise HeadlossError(HEADLOSS_ERR_DTYPE, "headloss_sample")
        if uniforms is None:
            raise HeadlossError(HEADLOSS_ERR_MISSING_INPUT, "headloss_sample")
        given, f32 = self._given, self._f32
        u, _u = given("uniforms", uniforms, self._f64, N)
        t, _t = given("temperature", temperature, f32, N)
        k, _k = given("top_k", top_k, self._i32, N)
        p, _p = given("top_p", top_p, f32, N)
        m, _m = given("min_p", min_p, f32, N)
        if out is None:
            empty, device = self._empty, self.device
            out = (empty(N, dtype=self._i64, device=device), empty(N, dtype=f32, device=device),
                   empty(N, dtype=f32, device=device), empty(N, dtype=self._i32, device=device))
        else:
            for name, a, d in zip(("tokens", "logprobs", "draw_logprobs", "n_kept"), out,
                                  (self._i64, f32, f32, self._i32)):
                given(name, a, d, N)
        status = self._call(logits.data_ptr(), N, V, logits.stride(0) if N > 1 else V, code, u, t,
                            k, p, m, self.softcap, self.logits_scale, out[0].data_ptr(),
                            out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(),
                            self.err.data_ptr(), _raw_stream(self.index))
        if status:
            _check(status, "headloss_sample")
        return out

    def device_error(self, stream=None) -> int:
        """Synchronise `stream`, then read and clear the error word (bit 0: settings
        out of range; bit 1: a copy wait gave up)."""
        with _on(self.index, stream):
            e = int(self.err.item())
            self.err.zero_()
        return e


class GradClipper:
    """headloss_clip_grads on torch tensors: the global norm over `grads` and one
    factor on all of them, into `outs` (None: in place).  The tensors are held;
    `bind` takes others: checks and addresses on the host, about a microsecond a
    tensor, so gradients that keep their buffers from step to step are bound once.
    Calling it returns the device tensor (norm, factor), made on
    `stream` as under torch.cuda.stream."""

    def __init__(self, grads, outs=None, max_grads: int = 0):
        self.h = None
        grads = list(grads)
        self.max_grads = max(int(max_grads), len(grads), 1)
        self.bind(grads, outs)
        self._call = load_library().headloss_clip_grads
        with _on(self.index, None):
            self.h = headloss_clip_create(self.max_grads)

    def bind(self, grads, outs=None) -> None:
        import torch
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if len(outs) != len(grads) or len(grads) > self.max_grads:
            raise ValueError(f"{len(grads)} gradients and {len(outs)} outputs (up to "
                             f"{self.max_grads})")
        codes = {torch.float32: HEADLOSS_FP32, torch.bfloat16: HEADLOSS_BF16,
                 torch.float16: HEADLOSS_FP16}
        if self.h:  # the workspace's device
            index = self.index
        else:
            index = grads[0].get_device() if grads else torch.cuda.current_device()
        for g, o in zip(grads, outs):
            if g.get_device() != index:
                raise ValueError(f"gradients: tensors on cuda:{index} are wanted, not on {g.device}")
            if not g.is_cuda or not g.is_contiguous() or o is not g and (
                    not o.is_contiguous() or o.dtype is not g.dtype or o.shape != g.shape or
                    o.get_device() != g.get_device()):
                raise ValueError("gradients are contiguous CUDA tensors, their outputs of the "
                                 "same type, shape and device")
            if g.dtype not in codes:
                raise HeadlossError(HEADLOSS_ERR_DTYPE, "headloss_clip_grads")
        # the entries of headloss_gradient as four 64-bit words each (dtype in the low half)
        words = array.array("q", bytes(32 * max(1, len(grads))))
        for j, (g, o) in enumerate(zip(grads, outs)):
            words[4 * j] = g.data_ptr()
            words[4 * j + 1] = o.data_ptr()
            words[4 * j + 2] = g.numel()
            words[4 * j + 3] = codes[g.dtype]
        self.grads, self.outs, self.words = grads, outs, words
        self.table = ctypes.cast(words.buffer_info()[0], ctypes.POINTER(headloss_gradient))
        self.index, self.device = index, torch.device("cuda", index)
        self._empty, self._f32 = torch.empty, torch.float32

    def __call__(self, max_norm: float, inv_scale: float = 1.0, stats=None, stream=None):
        if stream is not None or _current_device() != self.index:
            with _on(self.index, stream):
                return self(max_norm, inv_scale, stats)
        if stats is None:
            stats = self._empty(2, dtype=self._f32, device=self.device)
        elif (stats.dtype is not self._f32 or stats.numel() != 2 or
              stats.get_device() != self.index or not stats.is_contiguous()):
            raise ValueError(f"stats: a contiguous {self._f32} tensor of 2 on {self.device} is wanted")
        status = self._call(self.h, self.table, len(self.grads), max_norm, inv_scale,
                            stats.data_ptr(), _raw_stream(self.index))
        if status:
            _check(status, "headloss_clip_grads")
        return stats

    def close(self):
        if self.h:
            headloss_clip_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Fp8Head:
    """The LM head's products in 8 bits with an fp32 scale for each block of 128
    (include/headloss_fp8.h) on torch tensors: `logits`, and with train=True `backward`.

    `weight` (V x D, unit column stride) is quantised once, in 128 x 128 blocks of e4m3;
    `set_weight` does so again after an optimiser's step, into the same buffers (order it
    with calls on other streams; a checkpoint's codes are left, the first time, for buffers of
    the head's own, and kept with the head: a graph captured before goes on with them).
    `grads` is the 8-bit type of the loss's gradient, "e4m3" or "e5m2".  A call's own buffers
    are made on the stream it runs on."""

    _TYPES = {"e4m3": HEADLOSS_E4M3, "e5m2": HEADLOSS_E5M2}

    def __init__(self, weight, train: bool = False, grads: str = "e4m3"):
        V, D = self._matrix("weight", weight, weight.get_device())
        self._setup(V, D, weight, train, grads)
        with _on(self.index, None):
            self._make()
        self.set_weight(weight)

    @classmethod
    def from_quantized(cls, q, scales, train: bool = False, grads: str = "e4m3"):
        """A checkpoint's weight: `q` V x D float8_e4m3fn or float8_e5m2, `scales` fp32
        ceil(V / 128) x ceil(D / 128).  The codes are held without a copy where their
        rows are contiguous and on the 16-byte grid: leave both as they are while the head is used."""
        import torch
        types = {torch.float8_e4m3fn: HEADLOSS_E4M3, torch.float8_e5m2: HEADLOSS_E5M2}
        if q.dim() != 2 or q.dtype not in types or not q.is_cuda or min(q.shape) < 1:
            raise ValueError("q: a V x D float8 tensor on a GPU is wanted")
        V, D = q.shape
        if (scales.dtype is not torch.float32 or scales.get_device() != q.get_device() or
                tuple(scales.shape) != (-(-V // 128), -(-D // 128))):
            raise ValueError(f"scales: an fp32 tensor of {-(-V // 128)} x {-(-D // 128)} on {q.device} "
                             "is wanted")
        self = cls.__new__(cls)
        self._setup(V, D, q, train, grads)
        self.type = types[q.dtype]
        with _on(self.index, None):
            codes = q.view(torch.uint8)
            self.scales, self.held = scales.contiguous(), True
            if codes.is_contiguous() and D % 16 == 0 and codes.data_ptr() % 16 == 0:
                self.q, self.ldq = codes, D
            else:
                self.q, self.ldq = torch.zeros(V, -(-D // 16) * 16, dtype=torch.uint8, device=q.device), -(-D // 16) * 16
                self.q[:, :D].copy_(codes)
            if train:
                self.qt = torch.zeros(D, -(-V // 16) * 16, dtype=torch.uint8, device=q.device)
                self.qt[:, :V].copy_(codes.t())
                self.ldqt, self.scales_t = self.qt.shape[1], self.scales.t().contiguous()
        return self

    def _setup(self, V, D, like, train, grads):
        import torch
        if grads not in self._TYPES:
            raise ValueError('grads: "e4m3" or "e5m2" is wanted')
        self._lib = load_library()
        self.V, self.D, self.train, self.type = V, D, bool(train), HEADLOSS_E4M3
        self.held = False  # a checkpoint's own memory, which is not written to
        self.grads = self._TYPES[grads]
        self.index, self.device = like.get_device(), like.device
        self.weight_dtype = torch.bfloat16
        self._empty, self._u8, self._f32 = torch.empty, torch.uint8, torch.float32
        self._codes = {torch.float32: HEADLOSS_FP32, torch.bfloat16: HEADLOSS_BF16,
                       torch.float16: HEADLOSS_FP16}
        self._needs = {}
        with _on(self.index, None):
            self.err = torch.zeros(1, dtype=torch.int32, device=self.device)

    def _make(self):
        u8, f32, dev = self._u8, self._f32, self.device
        vb, db = -(-self.V // 128), -(-self.D // 128)
        self.ldq = -(-self.D // 16) * 16
        self.q = self._empty(self.V, self.ldq, dtype=u8, device=dev)
        self.scales = self._empty(vb, db, dtype=f32, device=dev)
        if self.train:
            self.ldqt = -(-self.V // 16) * 16
            self.qt = self._empty(self.D, self.ldqt, dtype=u8, device=dev)
            self.scales_t = self._empty(db, vb, dtype=f32, device=dev)

    @staticmethod
    def _matrix(name, a, index):
        import torch
        if (a.dim() != 2 or index < 0 or a.get_device() != index or
                a.dtype not in (torch.float32, torch.bfloat16, torch.float16) or
                (a.shape[1] > 1 and a.stride(1) != 1) or
                (a.shape[0] > 1 and a.stride(0) < a.shape[1])):
            raise ValueError(f"{name}: an fp32, bf16 or fp16 matrix with unit column stride on "
                             f"cuda:{max(index, 0)} is wanted")
        if name == "weight" and min(a.shape) < 1:
            raise ValueError("weight: at least one row and one column are wanted")
        return a.shape

    def _out(self, name, out, rows, cols, dtype):
        if out is None:
            return self._empty(rows, cols, dtype=dtype, device=self.device)
        self._matrix(name, out, self.index)
        if tuple(out.shape) != (rows, cols):
            raise ValueError(f"{name}: {rows} x {cols} is wanted")
        return out

    def _quantize(self, x, type, q=None, ldq=0, scales=None, block=0, qt=None, ldqt=0, scales_t=None,
                  block_t=0):
        rows, cols = x.shape
        status = self._lib.headloss_fp8_quantize(
            x.data_ptr(), rows, cols, x.stride(0) if rows > 1 else cols, self._codes[x.dtype], type, q,
            ldq, scales, block, qt, ldqt, scales_t, block_t, _raw_stream(self.index))
        if status:
            _check(status, "headloss_fp8_quantize")

    def _matmul(self, a, lda, a_scales, a_type, b, ldb, b_scales, b_type, M, N, K, out):
        need = self._needs.get((M, N, K))
        if need is None:
            need = self._needs[M, N, K] = self._lib.headloss_fp8_workspace(M, N, K)
        work = self._empty(need, dtype=self._u8, device=self.device) if need > 0 else None
        status = self._lib.headloss_fp8_matmul(
            a, lda, a_scales, a_type, b, ldb, b_scales, b_type, M, N, K, out.data_ptr(),
            out.stride(0) if M > 1 else N, self._codes[out.dtype],
            work.data_ptr() if work is not None else None, need, self.err.data_ptr(),
            _raw_stream(self.index))
        if status:
            _check(status, "headloss_fp8_matmul")

    def set_weight(self, weight, stream=None) -> None:
        if stream is not None or _current_device() != self.index:
            with _on(self.index, stream):
                return self.set_weight(weight)
        self._matrix("weight", weight, self.index)
        if tuple(weight.shape) != (self.V, self.D):
            raise ValueError(f"weight: {self.V} x {self.D} is wanted")
        if self.held:
            # Kept: the allocator may give freed memory to a stream that does not wait for the calls that read it. And
            # not written to: their type may be another than the new codes'.
            self.checkpoint = self.q, self.scales, *((self.qt, self.scales_t) if self.train else ())
            self._make()
            self.type, self.held = HEADLOSS_E4M3, False
        t, self.weight_dtype = self.train, weight.dtype
        self._quantize(weight, HEADLOSS_E4M3, self.q.data_ptr(), self.ldq, self.scales.data_ptr(), 128,
                       self.qt.data_ptr() if t else None, self.ldqt if t else 0,
                       self.scales_t.data_ptr() if t else None, 128)

    def logits(self, hidden, out=None, dtype=None, stream=None):
        """hidden . weight^T (tokens x V) in `dtype` (None: the hidden states'), into `out`
        if given."""
        if stream is not None or _current_device() != self.index:
            with _on(self.index, stream):
                return self.logits(hidden, out, dtype)
        N, D = self._matrix("hidden", hidden, self.index)
        if D != self.D:
            raise ValueError(f"hidden: {self.D} columns are wanted")
        dtype = dtype or (hidden.dtype if out is None else out.dtype)
        if dtype not in self._codes or (out is not None and out.dtype is not dtype):
            raise ValueError("logits: fp32, bf16 or fp16 and `out` of that type are wanted")
        out = self._out("out", out, N, self.V, dtype)
        if N == 0:
            return out
        need = self._needs.get(N)
        if need is None:
            need = self._needs[N] = self._lib.headloss_fp8_linear_workspace(N, self.V, D)
        work = self._empty(max(need, 0), dtype=self._u8, device=self.device)
        status = self._lib.headloss_fp8_linear(
            hidden.data_ptr(), hidden.stride(0) if N > 1 else D, self._codes[hidden.dtype], self.q.data_ptr(),
            self.ldq, self.scales.data_ptr(), self.type, N, self.V, D, out.data_ptr(),
            out.stride(0) if N > 1 else self.V, self._codes[dtype], work.data_ptr(), need, self.err.data_ptr(),
            _raw_stream(self.index))
        if status:
            _check(status, "headloss_fp8_linear")
        return out

    def backward(self, grad, hidden, grad_hidden=None, grad_weight=None, weight_dtype=None, stream=None):
        """(grad . weight, grad^T . hidden) of the loss's gradient `grad` (tokens x V) and the
        hidden states: tokens x D in the hidden states' type and V x D in `weight_dtype` (None: that
        of the weight last given, a checkpoint's: bf16), into the buffers given.  The gradient and the hidden states of the
        second product are quantised over the tokens."""
        if stream is not None or _current_device() != self.index:
            with _on(self.index, stream):
                return self.backward(grad, hidden, grad_hidden, grad_weight, weight_dtype)
        if not self.train:
            raise ValueError("backward: a head made with train=True is wanted")
        N, V = self._matrix("grad", grad, self.index)
        if V != self.V or tuple(self._matrix("hidden", hidden, self.index)) != (N, self.D):
            raise ValueError(f"grad, hidden: N x {self.V} and N x {self.D} are wanted")
        D = self.D
        weight_dtype = weight_dtype or (self.weight_dtype if grad_weight is None else grad_weight.dtype)
        if weight_dtype not in self._codes or (grad_weight is not None and grad_weight.dtype is not weight_dtype):
            raise ValueError("grad_weight: fp32, bf16 or fp16 and a buffer of that type are wanted")
        grad_hidden = self._out("grad_hidden", grad_hidden, N, D, hidden.dtype)
        grad_weight = self._out("grad_weight", grad_weight, V, D, weight_dtype)
        if N == 0:
            return grad_hidden, grad_weight.zero_()
        vp, np_ = -(-V // 16) * 16, -(-N // 16) * 16
        vb, nb, db = -(-V // 128), -(-N // 128), -(-D // 128)
        sizes = (N * vp, V * np_, D * np_, 4 * N * vb, 4 * V * nb, 4 * db * nb)
        buf = self._empty(sum(-(-s // 16) * 16 for s in sizes), dtype=self._u8, device=self.device)
        at, parts = buf.data_ptr(), []
        for s in sizes:
            parts.append(at)
            at += -(-s // 16) * 16
        gq, gt, xt, gs, gts, xts = parts
        self._quantize(grad, self.grads, gq, vp, gs, 1, gt, np_, gts, 1)
        self._quantize(hidden, HEADLOSS_E4M3, qt=xt, ldqt=np_, scales_t=xts, block_t=128)
        self._matmul(gq, vp, gs, self.grads, self.qt.data_ptr(), self.ldqt, self.scales_t.data_ptr(), self.type,
                     N, D, V, grad_hidden)
        self._matmul(gt, np_, gts, self.grads, xt, np_, xts, HEADLOSS_E4M3, V, D, N, grad_weight)
        return grad_hidden, grad_weight

    def device_error(self, stream=None) -> int:
        """Synchronise `stream`, then read and clear the error word (bit 0: a wait inside a
        product gave up)."""
        with _on(self.index, stream):
            e = int(self.err.item())
            self.err.zero_()
        return e


class BeamSelector:
    """headloss_beam_select on torch tensors: the `keep` (None: `beams`) best continuations of
    each request's `beams` rows of logits.

    Called with logits ((requests * beams) x V, unit column stride, any row stride), the
    beams' scores (requests x beams fp32) and, where hypotheses can end, a bool tensor of
    those that have (requests x beams).  Returns (scores fp32, parents int32, tokens int64,
    ended bool), requests x keep each; `out` gives the four buffers.  `eos` is the token that
    ends a hypothesis (None: none does).  `stay` (keep == beams alone) leaves a beam that goes
    on in its place, so that states that are reordered in place move least."""

    def __init__(self, beams: int, keep=None, softcap: float = 0.0, logits_scale: float = 1.0, eos=None,
                 stay: bool = False, device="cuda"):
        import torch
        self.beams, self.keep = int(beams), int(beams if keep is None else keep)
        self.softcap, self.logits_scale = float(softcap), float(logits_scale)
        self.eos, self.stay = -1 if eos is None else int(eos), int(bool(stay))
        if not 1 <= self.beams <= 64 or not 1 <= self.keep <= 128 or (self.stay and self.keep != self.beams):
            raise ValueError("beams in 1 .. 64 and keep in 1 .. 128 are wanted, and keep == beams with stay")
        device = torch.device(device)
        self.index = device.index if device.index is not None else torch.cuda.current_device()
        self.device = torch.device("cuda", self.index)
        lib = load_library()
        self._call, self._need = lib.headloss_beam_select, lib.headloss_beam_workspace
        self._empty, self._u8, self._bool = torch.empty, torch.uint8, torch.bool
        self._f32, self._i32, self._i64 = torch.float32, torch.int32, torch.int64
        self._codes = {torch.float32: HEADLOSS_FP32, torch.bfloat16: HEADLOSS_BF16,
                       torch.float16: HEADLOSS_FP16}

    def _given(self, name, a, dtype, shape):
        if (a.dtype is not dtype or tuple(a.shape) != shape or a.get_device() != self.index or
                not a.is_contiguous()):
            raise ValueError(f"{name}: a contiguous {dtype} tensor of {shape[0]} x {shape[1]} on "
                             f"{self.device} is wanted")
        return a.data_ptr()

    def __call__(self, logits, scores, ended=None, out=None, stream=None):
        if stream is not None or _current_device() != self.index:
            with _on(self.index, stream):
                return self(logits, scores, ended, out)
        if (logits.dim() != 2 or logits.get_device() != self.index or logits.shape[1] < 1 or
                logits.shape[0] % self.beams or (logits.shape[1] > 1 and logits.stride(1) != 1)):
            raise ValueError(f"logits: a (requests * {self.beams}) x V tensor with unit column stride on "
                             f"{self.device} is wanted")
        N, V = logits.shape
        code = self._codes.get(logits.dtype)
        if code is None:
            raise HeadlossError(HEADLOSS_ERR_DTYPE, "headloss_beam_select")
        R, k = N // self.beams, self.keep
        s = self._given("scores", scores, self._f32, (R, self.beams))
        e = None if ended is None else self._given("ended", ended, self._bool, (R, self.beams))
        if e is not None and self.eos < 0:
            raise ValueError("ended: a selector made with eos is wanted")
        empty, device = self._empty, self.device
        if out is None:
            out = (empty(R, k, dtype=self._f32, device=device), empty(R, k, dtype=self._i32, device=device),
                   empty(R, k, dtype=self._i64, device=device), empty(R, k, dtype=self._bool, device=device))
        else:
            for name, a, d in zip(("scores", "parents", "tokens", "ended"), out,
                                  (self._f32, self._i32, self._i64, self._bool)):
                self._given("out's " + name, a, d, (R, k))
        need = self._need(R, self.beams, V, code, k)
        work = empty(max(need, 0), dtype=self._u8, device=device)
        status = self._call(logits.data_ptr(), R, self.beams, V, logits.stride(0) if N > 1 else V, code, s, e,
                            self.eos, k, self.stay, self.softcap, self.logits_scale, out[0].data_ptr(),
                            out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), work.data_ptr(), need,
                            _raw_stream(self.index))
        if status:
            _check(status, "headloss_beam_select")
        return out


class StateReorder:
    """headloss_reorder on torch tensors: the beams take their parents' states, in place or into
    `outs` (buffers of the same layout).  The tensors are held.

    `states` are tensors of requests * beams rows (or more: those behind stay as they are); one that is
    listed twice is moved once, and a call refuses those that share memory in other ways.  With
    `axis` the dimension of the positions (a cache's): a call's `begin` and `end` (int32, one a
    request) then name the positions to take, say those behind a prompt that the beams share.
    Called with parents (requests x beams int32, as the selection gives them); returns the
    reordered tensors.  The object is kept as long as a graph that holds one of its calls."""

    def __init__(self, states, beams: int, outs=None, axis=None):
        import torch
        self.h = None
        states = list(states)
        outs = states if outs is None else list(outs)
        if not states or len(outs) != len(states) or not 1 <= int(beams) <= 64:
            raise ValueError("at least one state, as many outs, and beams in 1 .. 64 are wanted")
        self.beams, self.axis = int(beams), axis
        self.index = states[0].get_device()
        table = (headloss_state * len(states))()
        self.rows = min(t.shape[0] if t.dim() else 0 for t in states)
        for t, o, entry in zip(states, outs, table):
            if (not t.is_cuda or t.get_device() != self.index or t.dim() < 1 or o.get_device() != self.index or
                    o is not t and (o.dtype is not t.dtype or o.shape != t.shape or o.stride() != t.stride())):
                raise ValueError(f"states: tensors on cuda:{max(self.index, 0)}, and outs of their types, "
                                 "shapes and strides, are wanted")
            entry.state, entry.out = t.data_ptr(), o.data_ptr()
            self._layout(t, entry)
        self.states, self.outs = states, outs
        self.device = torch.device("cuda", self.index)
        self._i32 = torch.int32
        self._call = load_library().headloss_reorder
        live = [e for e, t in zip(table, states) if t.numel()]
        self._moves = bool(live)
        if live:
            with _on(self.index, None):
                self.h = headloss_reorder_create((headloss_state * len(live))(*live), len(live), self.beams)

    def _layout(self, t, entry):
        """Rows, outer dimensions that go as one, positions, and a run of contiguous elements."""
        size, axis = t.element_size(), self.axis
        if any(n > 1 and s <= 0 for n, s in zip(t.shape, t.stride())):
            raise ValueError("states: expanded dimensions are refused")

        def joined(dims):
            """The number and the stride of the elements of `dims`, where they go as one."""
            n, stride = 1, 0
            for d in reversed(dims):
                if t.shape[d] == 1:
                    continue
                if stride and t.stride(d) != n * stride:
                    raise ValueError("states: dimensions before the positions that go as one, and contiguous "
                                     "ones behind them, are wanted")
                stride = stride or t.stride(d)
                n *= t.shape[d]
            return n, stride
        if axis is not None and not 1 <= axis < t.dim():
            raise ValueError("axis: a dimension behind the rows is wanted")
        behind = range(1 if axis is None else axis + 1, t.dim())
        run, stride = joined(list(behind))
        if run > 1 and stride != 1:
            raise ValueError("states: contiguous elements behind the positions are wanted")
        entry.row_stride = t.stride(0) * size
        entry.run_bytes = run * size
        entry.outer, outer_stride = joined(list(range(1, axis))) if axis is not None else (1, 0)
        entry.outer_stride = outer_stride * size
        entry.positions = t.shape[axis] if axis is not None else 1
        entry.position_stride = t.stride(axis) * size if axis is not None else run * size

    def __call__(self, parents, begin=None, end=None, stream=None):
        if stream is not None or _current_device() != self.index:
            with _on(self.index, stream):
                return self(parents, begin, end)
        if (parents.dim() != 2 or parents.shape[1] != self.beams or parents.dtype is not self._i32 or
                parents.get_device() != self.index or not parents.is_contiguous() or
                parents.numel() > self.rows):
            raise ValueError(f"parents: a contiguous int32 tensor of requests x {self.beams} on {self.device}, "
                             f"for {self.rows} rows at most, is wanted")
        R = parents.shape[0]
        if (begin is None) != (end is None) or (begin is not None and self.axis is None):
            raise ValueError("begin and end: both or none, and none for states without positions")
        for name, a in (("begin", begin), ("end", end)):
            if a is not None and (a.dtype is not self._i32 or a.dim() != 1 or a.numel() != R or
                                  a.get_device() != self.index or not a.is_contiguous()):
                raise ValueError(f"{name}: a contiguous int32 tensor of {R} on {self.device} is wanted")
        if self._moves:
            if not self.h:
                raise ValueError("a reordering that is not closed is wanted")
            status = self._call(self.h, parents.data_ptr(), R, begin.data_ptr() if begin is not None else None,
                                end.data_ptr() if end is not None else None, _raw_stream(self.index))
            if status:
                _check(status, "headloss_reorder")
        return self.outs

    def close(self):
        if self.h:
            headloss_reorder_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
