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
           "headloss_clip_destroy")


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
