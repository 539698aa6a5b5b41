"""Python binding of libmpstep, the mixed-precision update step for MI355X.

Argument marshalling only: every entry point forwards to the C ABI declared in
``include/mpstep.h`` (same names, same arguments), and every step of the update
runs in the library's HIP kernels.  PyTorch supplies device memory and streams.
``ModelState`` allocates the buffers of one model with torch and builds the
plan over them; it computes nothing itself.

Importing this module loads ``libmpstep.so``; it raises if the library has not
been built (``python -m optimizer_step_tensor_amd.build`` or
``__graft_entry__.build()``).  There is no fallback implementation.
"""
import ctypes
import os

import torch  # loaded first: libmpstep then binds to torch's HIP runtime

from .build import LIB as _LIB_PATH

MP_BF16 = 0
MP_FP16 = 1
MP_FP32 = 2            # logits only

MP_OK, MP_ERR_INVALID, MP_ERR_ALIGN, MP_ERR_NOMEM, MP_ERR_HIP, MP_ERR_ORDER = range(6)

ENTRY_POINTS = [
    "mp_status_string", "mp_last_error", "mp_abi_version", "mp_token_weights",
    "mp_state_bytes_per_param", "mp_plan_create", "mp_plan_destroy", "mp_plan_info",
    "mp_chunk_layout",
    "mp_gradset_create", "mp_gradset_destroy", "mp_state_create", "mp_state_destroy",
    "mp_state_read", "mp_state_scale_ptr", "mp_accumulate", "mp_unscale_check_norm",
    "mp_adamw_step", "mp_scaler_update", "mp_cast_to_16", "mp_widen_16",
    "mp_state_export", "mp_state_import", "mp_norm_partial", "mp_norm_finish",
    "mp_cast_fp8_blocks", "mp_fp8set_create", "mp_fp8set_destroy", "mp_adamw_step_fp8",
    "mp_gradset_update", "mp_update_step", "mp_token_weights_dev", "mp_accumulate_group",
    "mp_update_step_group", "mp_unscale_check_norm_group", "mp_adamw_step_group",
    "mp_norm_partial_group", "mp_update_step_noalloc", "mp_accumulate_first_counts",
    "mp_target_count", "mp_token_logprob", "mp_token_logprob_grad", "mp_cross_entropy",
    "mp_policy_loss", "mp_preference_loss", "mp_distill_loss",
    "mp_token_score", "mp_token_score_grad", "mp_route", "mp_route_grad", "mp_route_bias_update",
]

MP_STATE_BLOB_BYTES = 256
MP_NOALLOC_MAX_NORM_BLOCKS = 262144
MP_LOSS_WORKSPACE_BYTES = 65536
MP_DISTILL_MAX_K = 1024
MP_PREF_SIGMOID, MP_PREF_SQUARED = range(2)
MP_SCORE_MAX_TOP = 128
MP_SCORE_WORKSPACE_BYTES = 1 << 20
MP_ROUTE_MAX_EXPERTS, MP_ROUTE_MAX_GROUPS, MP_ROUTE_MAX_TOP = 1024, 64, 16
MP_ROUTE_WORKSPACE_BYTES = 4 << 20
MP_ROUTE_SOFTMAX, MP_ROUTE_SIGMOID = range(2)


class MpError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s: %s" % (_name(status), message))
        self.status = status


class ScalerCfg(ctypes.Structure):
    _fields_ = [("init_scale", ctypes.c_float), ("growth", ctypes.c_float),
                ("backoff", ctypes.c_float), ("min_scale", ctypes.c_float),
                ("max_scale", ctypes.c_float), ("interval", ctypes.c_int32),
                ("enabled", ctypes.c_int32)]


class AdamWHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class Stats(ctypes.Structure):
    _fields_ = [("found_inf", ctypes.c_int32), ("skipped", ctypes.c_int32),
                ("good_steps", ctypes.c_int32), ("reserved0", ctypes.c_int32),
                ("step", ctypes.c_int64), ("skipped_total", ctypes.c_int64),
                ("sumsq", ctypes.c_double), ("beta1_pow", ctypes.c_double),
                ("beta2_pow", ctypes.c_double), ("scale", ctypes.c_float),
                ("grad_norm", ctypes.c_float), ("clip_coef", ctypes.c_float),
                ("reserved1", ctypes.c_float)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_
                if not name.startswith("reserved")}


class Logits(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("stride", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("temperature", ctypes.c_float), ("workspace", ctypes.c_void_p)]


class LogitsGrad(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64),
                ("dev_scale", ctypes.c_void_p), ("dev_count", ctypes.c_void_p),
                ("scale", ctypes.c_float)]


class PolicyCfg(ctypes.Structure):
    _fields_ = [("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float),
                ("kl_coef", ctypes.c_float)]


class PreferenceCfg(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("length_mean", ctypes.c_int32),
                ("beta", ctypes.c_float), ("label_smoothing", ctypes.c_float),
                ("margin", ctypes.c_float)]


class Teacher(ctypes.Structure):
    _fields_ = [("values", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("k", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Score(ctypes.Structure):
    _fields_ = [("logp", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("entropy", ctypes.c_void_p),
                ("top_ids", ctypes.c_void_p), ("top_logp", ctypes.c_void_p),
                ("top_values", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("top", ctypes.c_int32)]


class RouteCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("score", "top", "groups", "top_groups", "group_best",
                                              "renormalise")] + [("scale", ctypes.c_float)]


class Routed(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("weights", "ids", "load", "share", "aux",
                                               "workspace")]


_lib = None


def lib():
    """The loaded libmpstep.so (raises RuntimeError when it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libmpstep.so is not built (%s); run __graft_entry__.build()"
                               % _LIB_PATH)
        _lib = _bind(ctypes.CDLL(_LIB_PATH))
    return _lib


def _bind(L):
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    PP = ctypes.POINTER(ctypes.c_void_p)
    sig = {
        "mp_status_string": ([i32], ctypes.c_char_p),
        "mp_last_error": ([], ctypes.c_char_p),
        "mp_abi_version": ([], i32),
        "mp_token_weights": ([i32, P, P], i32),
        "mp_state_bytes_per_param": ([i32, i32], ctypes.c_size_t),
        "mp_plan_create": ([i32, P, i32, PP, PP, PP, PP, PP, P, PP], i32),
        "mp_plan_destroy": ([P], i32),
        "mp_plan_info": ([P, P, P, P, P], i32),
        "mp_chunk_layout": ([i32, P, i32, P, P, P, P, P, i64], i32),
        "mp_gradset_create": ([P, PP, PP], i32),
        "mp_gradset_destroy": ([P], i32),
        "mp_state_create": ([ctypes.POINTER(ScalerCfg), PP], i32),
        "mp_state_destroy": ([P], i32),
        "mp_state_read": ([P, P, P], i32),
        "mp_state_scale_ptr": ([P, PP], i32),
        "mp_accumulate": ([P, P, f32, i32, P], i32),
        "mp_unscale_check_norm": ([P, P, P, f32, i32, f32, P], i32),
        "mp_adamw_step": ([P, P, P, f32, i32, ctypes.POINTER(AdamWHparams), P], i32),
        "mp_scaler_update": ([P, P], i32),
        "mp_cast_to_16": ([P, P, i64, i32, P], i32),
        "mp_widen_16": ([P, P, i64, i32, P], i32),
        "mp_state_export": ([P, P, ctypes.c_size_t, P], i32),
        "mp_state_import": ([P, P, ctypes.c_size_t, P], i32),
        "mp_norm_partial": ([P, P, P, f32, i32, P, P], i32),
        "mp_norm_finish": ([P, P, P, f32, P], i32),
        "mp_cast_fp8_blocks": ([P, P, P, i64, i32, P], i32),
        "mp_fp8set_create": ([P, PP, PP, PP], i32),
        "mp_fp8set_destroy": ([P], i32),
        "mp_adamw_step_fp8": ([P, P, P, f32, i32, ctypes.POINTER(AdamWHparams), P, P], i32),
        "mp_gradset_update": ([P, PP, P], i32),
        "mp_update_step": ([P, P, P, f32, i32, f32, ctypes.POINTER(AdamWHparams), P], i32),
        "mp_update_step_noalloc": ([P, P, P, f32, i32, f32, ctypes.POINTER(AdamWHparams), P],
                                   i32),
        "mp_token_weights_dev": ([i32, P, P, P], i32),
        "mp_accumulate_group": ([P, PP, P, i32, i32, i32, P], i32),
        "mp_accumulate_first_counts": ([P, PP, i32, i32, P, P, P], i32),
        "mp_update_step_group": ([P, P, PP, P, i32, i32, i32, f32, ctypes.POINTER(AdamWHparams),
                                  P], i32),
        "mp_unscale_check_norm_group": ([P, P, PP, P, i32, i32, i32, f32, P], i32),
        "mp_adamw_step_group": ([P, P, PP, P, i32, i32, i32, ctypes.POINTER(AdamWHparams), P],
                                i32),
        "mp_norm_partial_group": ([P, P, PP, P, i32, i32, i32, P, P], i32),
        "mp_target_count": ([i64, P, P, P], i32),
        "mp_token_logprob": ([P, P, P, P, P], i32),
        "mp_token_logprob_grad": ([P, P, P, P, P, P], i32),
        "mp_cross_entropy": ([P, P, P, P, P, P], i32),
        "mp_policy_loss": ([P] * 12, i32),
        "mp_preference_loss": ([P, P, i64] + [P] * 10, i32),
        "mp_distill_loss": ([P, P, P, P, P, P], i32),
        "mp_token_score": ([P, P, P, P], i32),
        "mp_token_score_grad": ([P] * 8, i32),
        "mp_route": ([P] * 6, i32),
        "mp_route_grad": ([P] * 6 + [f32, f32, P, P], i32),
        "mp_route_bias_update": ([i32, i32, P, i32, P, f32, P, P, P], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


def _name(status):
    try:
        return lib().mp_status_string(status).decode()
    except Exception:  # noqa: BLE001 -- naming an error must not raise
        return "status %d" % status


def _check(status):
    if status != MP_OK:
        raise MpError(status, lib().mp_last_error().decode())


def _ptrs(values):
    if values is None:
        return None
    arr = (ctypes.c_void_p * len(values))()
    for i, x in enumerate(values):
        arr[i] = x.data_ptr() if isinstance(x, torch.Tensor) else x
    return ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))


def _addr(x):
    """Device address of a tensor (or an int address); None stays NULL."""
    if x is None:
        return None
    return ctypes.c_void_p(x.data_ptr() if isinstance(x, torch.Tensor) else int(x))


# the current stream's handle without a Stream object around it (2.5 us a call less)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(stream)


# --- the C ABI, one wrapper per entry point -----------------------------------

def mp_status_string(status):
    return lib().mp_status_string(status).decode()


def mp_last_error():
    return lib().mp_last_error().decode()


def mp_abi_version():
    return lib().mp_abi_version()


def mp_token_weights(counts):
    n = (ctypes.c_int64 * len(counts))(*[int(c) for c in counts])
    w = (ctypes.c_float * len(counts))()
    _check(lib().mp_token_weights(len(counts), n, w))
    return list(w)


def mp_token_weights_dev(k, counts, weights_out, stream=None):
    """counts: k int64 on the device; weights_out: k fp32 on the device."""
    _check(lib().mp_token_weights_dev(int(k), _addr(counts), _addr(weights_out),
                                      _stream(stream)))


def mp_state_bytes_per_param(dtype, with_accumulator):
    return lib().mp_state_bytes_per_param(dtype, int(bool(with_accumulator)))


def mp_plan_create(numel, dtype, acc, master, m, v, w16, wd_mult=None):
    n = len(numel)
    ne = (ctypes.c_int64 * n)(*[int(x) for x in numel])
    wd = None if wd_mult is None else (ctypes.c_float * n)(*[float(x) for x in wd_mult])
    out = ctypes.c_void_p()
    _check(lib().mp_plan_create(n, ne, dtype, _ptrs(acc), _ptrs(master), _ptrs(m), _ptrs(v),
                                _ptrs(w16), wd, ctypes.byref(out)))
    return out


def mp_plan_destroy(plan):
    _check(lib().mp_plan_destroy(plan))


def mp_plan_info(plan):
    nt, tot, nc, ce = ctypes.c_int32(), ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
    _check(lib().mp_plan_info(plan, ctypes.byref(nt), ctypes.byref(tot), ctypes.byref(nc),
                              ctypes.byref(ce)))
    return {"n_tensors": nt.value, "total_params": tot.value, "n_chunks": nc.value,
            "chunk_elems": ce.value}


def mp_chunk_layout(numel, n_cus):
    """(chunk_elems, [(tensor, start, len), ...]) of the plan mp_plan_create would build."""
    n = len(numel)
    ne = (ctypes.c_int64 * n)(*[int(x) for x in numel])
    ce, nc = ctypes.c_int32(), ctypes.c_int64()
    _check(lib().mp_chunk_layout(n, ne, n_cus, ctypes.byref(ce), ctypes.byref(nc), None, None,
                                 None, 0))
    t = (ctypes.c_int32 * nc.value)()
    s = (ctypes.c_int64 * nc.value)()
    ln = (ctypes.c_int32 * nc.value)()
    _check(lib().mp_chunk_layout(n, ne, n_cus, None, None, t, s, ln, nc.value))
    return ce.value, list(zip(t, s, ln))


def mp_gradset_create(plan, g16):
    out = ctypes.c_void_p()
    _check(lib().mp_gradset_create(plan, _ptrs(g16), ctypes.byref(out)))
    return out


def mp_gradset_update(gradset, g16, stream=None):
    _check(lib().mp_gradset_update(gradset, _ptrs(g16), _stream(stream)))


def mp_gradset_destroy(gradset):
    _check(lib().mp_gradset_destroy(gradset))


def mp_state_create(cfg):
    out = ctypes.c_void_p()
    _check(lib().mp_state_create(ctypes.byref(cfg), ctypes.byref(out)))
    return out


def mp_state_destroy(state):
    _check(lib().mp_state_destroy(state))


def mp_state_read(state, out_ptr, stream=None):
    """Enqueue the copy of the device state into host memory at out_ptr (72 bytes)."""
    _check(lib().mp_state_read(state, ctypes.c_void_p(out_ptr), _stream(stream)))


def mp_state_scale_ptr(state):
    out = ctypes.c_void_p()
    _check(lib().mp_state_scale_ptr(state, ctypes.byref(out)))
    return out.value


def mp_accumulate(plan, gradset, weight, first, stream=None):
    _check(lib().mp_accumulate(plan, gradset, float(weight), int(bool(first)), _stream(stream)))


def _group(sets, weights):
    """(gradset array, weight pointer, on_device) for the *_group entry points: weights is a
    list of floats (host), or a device fp32 tensor or an int device address where len(sets)
    consecutive fp32 weights are read when the kernels run."""
    arr = (ctypes.c_void_p * len(sets))(*[s.value if isinstance(s, ctypes.c_void_p) else s
                                          for s in sets])
    if isinstance(weights, torch.Tensor):
        if not weights.is_cuda or weights.dtype != torch.float32:
            raise TypeError("device weights must be a CUDA float32 tensor")
        return ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), _addr(weights), 1
    if isinstance(weights, int):
        return ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), _addr(weights), 1
    w = (ctypes.c_float * len(sets))(*[float(x) for x in weights])
    return ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), ctypes.cast(w, ctypes.c_void_p), 0


def mp_accumulate_group(plan, sets, weights, first, stream=None):
    """Accumulate len(sets) resident micro-batches in one pass (see mp_accumulate_group)."""
    arr, w, dev = _group(sets, weights)
    _check(lib().mp_accumulate_group(plan, arr, w, len(sets), dev, int(bool(first)),
                                     _stream(stream)))


def mp_accumulate_first_counts(plan, sets, k, counts, weights_out, stream=None):
    """Token weights from device counts computed inside the first accumulation of sets (see
    the header); weights_out receives all k weights for the later passes."""
    arr = (ctypes.c_void_p * len(sets))(*[x.value if isinstance(x, ctypes.c_void_p) else x
                                          for x in sets])
    _check(lib().mp_accumulate_first_counts(plan, ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)),
                                            len(sets), int(k), _addr(counts), _addr(weights_out),
                                            _stream(stream)))


def mp_unscale_check_norm(plan, state, last, w_last, last_is_first, max_norm, stream=None):
    _check(lib().mp_unscale_check_norm(plan, state, last, float(w_last), int(bool(last_is_first)),
                                       float(max_norm), _stream(stream)))


def mp_adamw_step(plan, state, last, w_last, last_is_first, hp, stream=None):
    _check(lib().mp_adamw_step(plan, state, last, float(w_last), int(bool(last_is_first)),
                               ctypes.byref(hp), _stream(stream)))


def mp_update_step(plan, state, last, w_last, last_is_first, max_norm, hp, stream=None):
    _check(lib().mp_update_step(plan, state, last, float(w_last), int(bool(last_is_first)),
                                float(max_norm), ctypes.byref(hp), _stream(stream)))


def mp_update_step_noalloc(plan, state, last, w_last, last_is_first, max_norm, hp, stream=None):
    """mp_update_step with the norm's scratch in the library's static device array."""
    _check(lib().mp_update_step_noalloc(plan, state, last, float(w_last),
                                        int(bool(last_is_first)), float(max_norm),
                                        ctypes.byref(hp), _stream(stream)))


def mp_unscale_check_norm_group(plan, state, sets, weights, last_is_first, max_norm,
                                stream=None):
    arr, w, dev = _group(sets, weights)
    _check(lib().mp_unscale_check_norm_group(plan, state, arr, w, len(sets), dev,
                                             int(bool(last_is_first)), float(max_norm),
                                             _stream(stream)))


def mp_norm_partial_group(plan, state, sets, weights, last_is_first, partial_out, stream=None):
    arr, w, dev = _group(sets, weights)
    _check(lib().mp_norm_partial_group(plan, state, arr, w, len(sets), dev,
                                       int(bool(last_is_first)), _addr(partial_out),
                                       _stream(stream)))


def mp_adamw_step_group(plan, state, sets, weights, last_is_first, hp, stream=None):
    arr, w, dev = _group(sets, weights)
    _check(lib().mp_adamw_step_group(plan, state, arr, w, len(sets), dev,
                                     int(bool(last_is_first)), ctypes.byref(hp), _stream(stream)))


def mp_update_step_group(plan, state, sets, weights, last_is_first, max_norm, hp, stream=None):
    """mp_update_step with len(sets) resident micro-batches folded in (see the header)."""
    arr, w, dev = _group(sets, weights)
    _check(lib().mp_update_step_group(plan, state, arr, w, len(sets), dev,
                                      int(bool(last_is_first)), float(max_norm),
                                      ctypes.byref(hp), _stream(stream)))


def mp_scaler_update(state, stream=None):
    _check(lib().mp_scaler_update(state, _stream(stream)))


def mp_cast_to_16(src, dst, n, dtype, stream=None):
    _check(lib().mp_cast_to_16(ctypes.c_void_p(src), ctypes.c_void_p(dst), int(n), dtype,
                               _stream(stream)))


def mp_widen_16(src, dst, n, dtype, stream=None):
    _check(lib().mp_widen_16(ctypes.c_void_p(src), ctypes.c_void_p(dst), int(n), dtype,
                             _stream(stream)))


def mp_state_export(state, blob_ptr, blob_bytes=MP_STATE_BLOB_BYTES, stream=None):
    _check(lib().mp_state_export(state, ctypes.c_void_p(blob_ptr), blob_bytes, _stream(stream)))


def mp_state_import(state, blob_ptr, blob_bytes=MP_STATE_BLOB_BYTES, stream=None):
    _check(lib().mp_state_import(state, ctypes.c_void_p(blob_ptr), blob_bytes, _stream(stream)))


def mp_norm_partial(plan, state, last, w_last, last_is_first, partial_out, stream=None):
    _check(lib().mp_norm_partial(plan, state, last, float(w_last), int(bool(last_is_first)),
                                 ctypes.c_void_p(partial_out), _stream(stream)))


def mp_norm_finish(plan, state, sumsq, max_norm, stream=None):
    _check(lib().mp_norm_finish(plan, state, ctypes.c_void_p(sumsq), float(max_norm),
                                _stream(stream)))


def mp_cast_fp8_blocks(src, codes, scales, n, block=16, stream=None):
    _check(lib().mp_cast_fp8_blocks(ctypes.c_void_p(src), ctypes.c_void_p(codes),
                                    ctypes.c_void_p(scales), int(n), int(block), _stream(stream)))


def mp_fp8set_create(plan, codes, scales):
    """codes[i], scales[i]: tensors / device addresses, or None for a tensor that is not cast."""
    out = ctypes.c_void_p()
    _check(lib().mp_fp8set_create(plan, _ptrs(codes), _ptrs(scales), ctypes.byref(out)))
    return out


def mp_fp8set_destroy(fp8set):
    _check(lib().mp_fp8set_destroy(fp8set))


def mp_adamw_step_fp8(plan, state, last, w_last, last_is_first, hp, fp8set, stream=None):
    _check(lib().mp_adamw_step_fp8(plan, state, last, float(w_last), int(bool(last_is_first)),
                                   ctypes.byref(hp), fp8set, _stream(stream)))


# --- losses over vocabulary logits ----------------------------------------------

_LOGITS_DTYPE = {torch.bfloat16: MP_BF16, torch.float16: MP_FP16, torch.float32: MP_FP32}


def _array(x, dtype, n, name, device=None):
    """Device address of a contiguous array of at least n elements: a tensor (checked) or an
    int address; None stays NULL."""
    if x is None or isinstance(x, int):
        return x
    if x.dtype is not dtype:
        raise TypeError("%s must be a %s tensor, not %s" % (name, dtype, x.dtype))
    if x.numel() < n or not x.is_contiguous():
        raise ValueError("%s must be contiguous, with %d elements" % (name, n))
    if x.device != device if device is not None else not x.is_cuda:
        raise ValueError("%s must be on the logits' GPU" % name)
    return x.data_ptr()


def _matrix(x, name):
    if x.dim() != 2 or x.dtype not in _LOGITS_DTYPE:
        raise TypeError("%s must be a 2-D bfloat16, float16 or float32 tensor" % name)
    if not x.is_cuda:
        raise ValueError("%s must be on a GPU" % name)
    (rows, vocab), (stride, inner) = x.shape, x.stride()
    if vocab > 1 and inner != 1:
        raise ValueError("%s: the elements of a row must be adjacent" % name)
    return x.data_ptr(), rows, vocab, stride if rows > 1 else vocab


def logits(x, temperature=1.0, workspace=None):
    """The mp_logits of a 2-D tensor [rows, vocab] (rows may be strided).  workspace: a tensor of
    MP_LOSS_WORKSPACE_BYTES uint8 on its GPU, used where there are few rows.  The struct keeps
    the tensors it describes."""
    data, rows, vocab, stride = _matrix(x, "logits")
    w = _array(workspace, torch.uint8, MP_LOSS_WORKSPACE_BYTES, "workspace", x.device)
    out = Logits(data, rows, vocab, stride, _LOGITS_DTYPE[x.dtype], temperature, w)
    out.torch = (x.dtype, x.device, rows, vocab)
    out.keep = (x, workspace)
    return out


def logits_grad(dx, scale=1.0, dev_scale=None, dev_count=None):
    """The mp_logits_grad that writes to the 2-D tensor dx: the gradient times scale * dev_scale /
    dev_count.  dev_scale: a float32 tensor or the address mp_state_scale_ptr gives; dev_count: an
    int64 tensor (mp_target_count)."""
    data, rows, vocab, stride = _matrix(dx, "the gradient")
    out = LogitsGrad(data, stride, _array(dev_scale, torch.float32, 1, "dev_scale", dx.device),
                     _array(dev_count, torch.int64, 1, "dev_count", dx.device), scale)
    out.torch = (dx.dtype, dx.device, rows, vocab)
    out.keep = (dx, dev_scale, dev_count)
    return out


def policy_cfg(clip_low=0.2, clip_high=0.2, kl_coef=0.0):
    return PolicyCfg(clip_low, clip_high, kl_coef)


def preference_cfg(kind=MP_PREF_SIGMOID, beta=0.1, label_smoothing=0.0, margin=0.0,
                   length_mean=False):
    return PreferenceCfg(kind, int(bool(length_mean)), beta, label_smoothing, margin)


def teacher(values, ids, lse=None):
    """The mp_teacher of two contiguous [rows, k] tensors: logits (bf16, fp16 or fp32) and int64
    ids; lse: rows float32, the teacher's own normaliser at the student's temperature."""
    if values.dim() != 2 or values.dtype not in _LOGITS_DTYPE:
        raise TypeError("teacher values must be a 2-D bfloat16, float16 or float32 tensor")
    if ids.shape != values.shape:
        raise ValueError("teacher values and ids must have the same shape")
    rows, k = values.shape
    out = Teacher(_array(values, values.dtype, rows * k, "teacher values"),
                  _array(ids, torch.int64, rows * k, "teacher ids", values.device),
                  _array(lse, torch.float32, rows, "teacher lse", values.device), k,
                  _LOGITS_DTYPE[values.dtype])
    out.torch = (values.device, rows)
    out.keep = (values, ids, lse)
    return out


def _grad_of(x, grad):
    """byref of a gradient that fits the logits x; None stays NULL."""
    if grad is None:
        return None
    t, have = getattr(grad, "torch", None), getattr(x, "torch", None)
    if t is not None and have is not None and t != have:
        if t[:2] != have[:2]:
            raise TypeError("the gradient must have the logits' type and GPU")
        raise ValueError("the gradient must have the logits' shape")
    return ctypes.byref(grad)


def _place(x):
    """rows and GPU of the logits x (None: made of addresses)."""
    have = getattr(x, "torch", None)
    return x.rows, have[1] if have is not None else None


def _stream_of(stream, device):
    """`stream`, or the current one of the logits' GPU."""
    if stream is None and device is not None and _raw_stream is not None:
        return _raw_stream(device.index)
    return _stream(stream)


_F32, _I64 = torch.float32, torch.int64


def mp_target_count(targets, count, n=None, stream=None):
    """count[0] = how many targets (int64, the first n or all) are >= 0."""
    n = targets.numel() if n is None else int(n)
    if hasattr(targets, "device") and hasattr(count, "device") and targets.device != count.device:
        raise ValueError("targets and count must be on one GPU")
    _check(lib().mp_target_count(n, _array(targets, _I64, n, "targets"),
                                 _array(count, _I64, 1, "count"), _stream(stream)))


def mp_token_logprob(x, targets, logp, lse=None, stream=None):
    """x: logits(...); targets: int64 [rows]; logp and lse: float32 [rows], written."""
    n, d = _place(x)
    _check(lib().mp_token_logprob(ctypes.byref(x), _array(targets, _I64, n, "targets", d),
                                  _array(logp, _F32, n, "logp", d),
                                  _array(lse, _F32, n, "lse", d), _stream_of(stream, d)))


def mp_token_logprob_grad(x, targets, lse, dlogp, grad, stream=None):
    """grad: logits_grad(...), written; lse from mp_token_logprob; dlogp: float32 [rows]."""
    n, d = _place(x)
    _check(lib().mp_token_logprob_grad(ctypes.byref(x), _array(targets, _I64, n, "targets", d),
                                       _array(lse, _F32, n, "lse", d),
                                       _array(dlogp, _F32, n, "dlogp", d), _grad_of(x, grad),
                                       _stream_of(stream, d)))


def mp_cross_entropy(x, targets, weights, loss, grad=None, stream=None):
    """loss: float32 [rows], written; weights: float32 [rows] or None."""
    n, d = _place(x)
    _check(lib().mp_cross_entropy(ctypes.byref(x), _array(targets, _I64, n, "targets", d),
                                  _array(weights, _F32, n, "weights", d),
                                  _array(loss, _F32, n, "loss", d), _grad_of(x, grad),
                                  _stream_of(stream, d)))


def mp_policy_loss(x, targets, old_logp, ref_logp, advantage, weights, cfg, loss, logp=None,
                   kl=None, grad=None, stream=None):
    """Per-row inputs float32 [rows] (ref_logp and weights may be None); cfg: policy_cfg(...);
    loss, logp and kl: float32 [rows], written."""
    n, d = _place(x)
    _check(lib().mp_policy_loss(ctypes.byref(x), _array(targets, _I64, n, "targets", d),
                                _array(old_logp, _F32, n, "old_logp", d),
                                _array(ref_logp, _F32, n, "ref_logp", d),
                                _array(advantage, _F32, n, "advantage", d),
                                _array(weights, _F32, n, "weights", d), ctypes.byref(cfg),
                                _array(loss, _F32, n, "loss", d), _array(logp, _F32, n, "logp", d),
                                _array(kl, _F32, n, "kl", d), _grad_of(x, grad),
                                _stream_of(stream, d)))


def mp_preference_loss(x, targets, n_pairs, seq_start, ref_logp, cfg, loss, seq_logp, logp, lse,
                       dlogp, grad=None, stream=None):
    """seq_start: int64 [2 n_pairs + 1]; ref_logp: float32 [2 n_pairs] or None; cfg:
    preference_cfg(...); loss [n_pairs], seq_logp [2 n_pairs], logp, lse and dlogp [rows]:
    float32, written."""
    (n, d), p = _place(x), int(n_pairs)
    _check(lib().mp_preference_loss(ctypes.byref(x), _array(targets, _I64, n, "targets", d), p,
                                    _array(seq_start, _I64, 2 * p + 1, "seq_start", d),
                                    _array(ref_logp, _F32, 2 * p, "ref_logp", d), ctypes.byref(cfg),
                                    _array(loss, _F32, p, "loss", d),
                                    _array(seq_logp, _F32, 2 * p, "seq_logp", d),
                                    _array(logp, _F32, n, "logp", d), _array(lse, _F32, n, "lse", d),
                                    _array(dlogp, _F32, n, "dlogp", d), _grad_of(x, grad),
                                    _stream_of(stream, d)))


def mp_distill_loss(x, teacher, weights, loss, grad=None, stream=None):
    """teacher: teacher(...); loss: float32 [rows], written; weights: float32 [rows] or None."""
    n, d = _place(x)
    have = getattr(teacher, "torch", None)
    if have is not None and d is not None:
        if have[0] != d:
            raise ValueError("the teacher's entries must be on the logits' GPU")
        if have[1] < n:
            raise ValueError("the teacher must have an entry list for each of %d rows" % n)
    _check(lib().mp_distill_loss(ctypes.byref(x), ctypes.byref(teacher),
                                 _array(weights, _F32, n, "weights", d),
                                 _array(loss, _F32, n, "loss", d), _grad_of(x, grad),
                                 _stream_of(stream, d)))


# --- scores of logits -------------------------------------------------------------

def score(logp=None, lse=None, entropy=None, top_ids=None, top_logp=None, top_values=None,
          workspace=None):
    """The mp_score of float32 [rows] tensors (each may be None) and of the lists: int64 [rows, top]
    ids, float32 [rows, top] log-probabilities and logits.  workspace: MP_SCORE_WORKSPACE_BYTES
    uint8, used where there are few rows.  The struct keeps the tensors it describes."""
    have = [t for t in (logp, lse, entropy, top_ids, top_logp, top_values) if t is not None]
    if not have:
        raise ValueError("a score needs an output")
    rows, d, top = have[0].shape[0], have[0].device, 0
    if top_ids is not None:
        if top_ids.dim() != 2:
            raise ValueError("top_ids must be a [rows, top] tensor")
        top = top_ids.shape[1]
    for t, name in ((top_logp, "top_logp"), (top_values, "top_values")):
        if t is not None and (top_ids is None or t.shape != top_ids.shape):
            raise ValueError("%s must have the shape of top_ids" % name)
    if not have[0].is_cuda:
        raise ValueError("the score must be on a GPU")
    n = rows * top
    out = Score(_array(logp, _F32, rows, "logp", d), _array(lse, _F32, rows, "lse", d),
                _array(entropy, _F32, rows, "entropy", d), _array(top_ids, _I64, n, "top_ids", d),
                _array(top_logp, _F32, n, "top_logp", d),
                _array(top_values, _F32, n, "top_values", d),
                _array(workspace, torch.uint8, MP_SCORE_WORKSPACE_BYTES, "workspace", d), top)
    out.torch = (d, rows)
    out.keep = (logp, lse, entropy, top_ids, top_logp, top_values, workspace)
    return out


def _fits(x, out, what):
    """The rows and the GPU of outputs made of tensors are those of the logits x."""
    have = getattr(out, "torch", None)
    n, d = _place(x)
    if have is not None and d is not None:
        if have[0] != d:
            raise ValueError("%s must be on the logits' GPU" % what)
        if have[1] < n:
            raise ValueError("%s must have %d rows" % (what, n))
    return n, d


def mp_token_score(x, targets, score, stream=None):
    """x: logits(...); targets: int64 [rows], or None; score: score(...), its arrays written."""
    n, d = _fits(x, score, "the score")
    _check(lib().mp_token_score(ctypes.byref(x), _array(targets, _I64, n, "targets", d),
                                ctypes.byref(score), _stream_of(stream, d)))


def mp_token_score_grad(x, targets, lse, entropy, dlogp, dentropy, grad, stream=None):
    """grad: logits_grad(...), written; lse and entropy from mp_token_score; dlogp and dentropy:
    float32 [rows], either may be None."""
    n, d = _place(x)
    _check(lib().mp_token_score_grad(ctypes.byref(x), _array(targets, _I64, n, "targets", d),
                                     _array(lse, _F32, n, "lse", d),
                                     _array(entropy, _F32, n, "entropy", d),
                                     _array(dlogp, _F32, n, "dlogp", d),
                                     _array(dentropy, _F32, n, "dentropy", d), _grad_of(x, grad),
                                     _stream_of(stream, d)))


# --- routing to experts ------------------------------------------------------------

def route_cfg(top, score=MP_ROUTE_SOFTMAX, groups=1, top_groups=1, group_best=1, renormalise=True,
              scale=1.0):
    return RouteCfg(score, top, groups, top_groups, group_best, int(bool(renormalise)), scale)


def routed(weights, ids, load=None, share=None, aux=None, workspace=None):
    """The mp_routed of [tokens, top] tensors, float32 weights and int64 ids, and for training of
    load (int64 [experts + 1]), share (float32 [experts]), aux (float32 [2]) and a workspace of
    MP_ROUTE_WORKSPACE_BYTES uint8.  The struct keeps the tensors it describes."""
    if ids.dim() != 2 or weights.shape != ids.shape:
        raise ValueError("weights and ids must be [tokens, top] tensors")
    if not ids.is_cuda:
        raise ValueError("ids must be on a GPU")
    d, n = ids.device, ids.numel()
    out = Routed(_array(weights, _F32, n, "weights", d), _array(ids, _I64, n, "ids", d),
                 _array(load, _I64, 1, "load", d), _array(share, _F32, 1, "share", d),
                 _array(aux, _F32, 2, "aux", d),
                 _array(workspace, torch.uint8, MP_ROUTE_WORKSPACE_BYTES, "workspace", d))
    out.torch = (d, ids.shape[0])
    out.shape = (ids.shape[1], None if load is None else load.numel(),
                 None if share is None else share.numel())
    out.keep = (weights, ids, load, share, aux, workspace)
    return out


def _mask(mask, n, device):
    """Address of a mask of n torch.bool or uint8."""
    bool_ = isinstance(mask, torch.Tensor) and mask.dtype is torch.bool
    return _array(mask, torch.bool if bool_ else torch.uint8, n, "mask", device)


def mp_route(x, bias, mask, cfg, routed, stream=None):
    """x: logits(...) of [tokens, experts]; bias: float32 [experts] or None; mask: bool or uint8
    [tokens] or None; cfg: route_cfg(...); routed: routed(...), its arrays written."""
    n, d = _fits(x, routed, "what is routed")
    shape = getattr(routed, "shape", None)
    if shape is not None:
        if shape[0] != cfg.top:
            raise ValueError("weights and ids must have %d columns" % cfg.top)
        for have, want, name in ((shape[1], x.vocab + 1, "load"), (shape[2], x.vocab, "share")):
            if have is not None and have < want:
                raise ValueError("%s must have %d elements" % (name, want))
    _check(lib().mp_route(ctypes.byref(x), _array(bias, _F32, x.vocab, "bias", d),
                          _mask(mask, n, d), ctypes.byref(cfg), ctypes.byref(routed),
                          _stream_of(stream, d)))


def mp_route_grad(x, mask, cfg, ids, dweights, load, balance_coef, z_coef, grad, stream=None):
    """ids and dweights: int64 and float32 [tokens, top] (dweights may be None); load: int64
    [experts + 1], or None without auxiliary losses; grad: logits_grad(...), written."""
    n, d = _place(x)
    for t, name in ((ids, "ids"), (dweights, "dweights")):
        if isinstance(t, torch.Tensor) and t.dim() > 1 and t.shape[-1] != cfg.top:
            raise ValueError("%s must have %d columns" % (name, cfg.top))
    _check(lib().mp_route_grad(ctypes.byref(x), _mask(mask, n, d), ctypes.byref(cfg),
                               _array(ids, _I64, n * cfg.top, "ids", d),
                               _array(dweights, _F32, n * cfg.top, "dweights", d),
                               _array(load, _I64, x.vocab + 1, "load", d), float(balance_coef),
                               float(z_coef), _grad_of(x, grad), _stream_of(stream, d)))


def mp_route_bias_update(bias, load, speed, out=None, state=None, stream=None):
    """bias: float32 [experts] or [layers, experts]; load: int64 [..., layers, experts + 1], of any
    number of micro-batches; out: like bias (None: the bias is replaced); state: skipped with its
    step."""
    out = bias if out is None else out
    experts = bias.shape[-1]
    n = bias.numel()
    layers = n // experts if experts else 0
    if load.dim() < bias.dim() or load.shape[-1] != experts + 1 or (
            bias.dim() > 1 and load.shape[-2] != layers) or bias.dim() > 2:
        raise ValueError("load must be [..., layers, experts + 1] for a bias of [layers, experts]")
    if out.shape != bias.shape:
        raise ValueError("out must have the bias's shape")
    total, d = load.numel(), bias.device
    loads = total // (layers * (experts + 1)) if layers else 1
    if bias.dim() == 1:
        layers = 1
    _check(lib().mp_route_bias_update(layers, experts, _array(bias, _F32, n, "bias"), loads,
                                      _array(load, _I64, total, "load", d), float(speed),
                                      _array(out, _F32, n, "out", d), state,
                                      _stream_of(stream, d if bias.is_cuda else None)))


# --- convenience ---------------------------------------------------------------

def scaler_cfg(init_scale=2.0 ** 16, growth=2.0, backoff=0.5, min_scale=1.0, max_scale=2.0 ** 64,
               interval=2000, enabled=True):
    return ScalerCfg(init_scale, growth, backoff, min_scale, max_scale, interval, int(bool(enabled)))


def adamw_hparams(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1):
    return AdamWHparams(lr, beta1, beta2, eps, weight_decay)


def save_state(state, stream=None):
    """The state blob as bytes (enqueues the copy, then waits for the stream)."""
    buf = torch.empty(MP_STATE_BLOB_BYTES, dtype=torch.uint8, pin_memory=True)
    s = stream if stream is not None else torch.cuda.current_stream()
    mp_state_export(state, buf.data_ptr(), MP_STATE_BLOB_BYTES, s)
    s.synchronize()
    return bytes(buf.numpy())


def load_state(state, blob, stream=None):
    buf = ctypes.create_string_buffer(bytes(blob), len(blob))
    mp_state_import(state, ctypes.addressof(buf), len(blob), stream)


def read_stats(state, stream=None):
    """Read the device state (enqueues the copy, then waits for the stream)."""
    buf = torch.empty(ctypes.sizeof(Stats), dtype=torch.uint8, pin_memory=True)
    s = stream if stream is not None else torch.cuda.current_stream()
    mp_state_read(state, buf.data_ptr(), s)
    s.synchronize()
    return Stats.from_buffer_copy(bytes(buf.numpy())).as_dict()


# Tensor starts in the flat layout: a multiple of 64 elements (256 B of fp32, 128 B of a 16-bit
# format).  The library needs 16 bytes; whole cache lines keep the AdamW pass from writing
# partial lines at every tensor edge, which cost it 10% on a list of 4096 ragged tensors.
FLAT_ALIGN_ELEMS = 64


def _align_elems(n):
    return (n + FLAT_ALIGN_ELEMS - 1) // FLAT_ALIGN_ELEMS * FLAT_ALIGN_ELEMS


class ModelState:
    """Device buffers of one model (torch allocations) and the plan over them.

    For each tensor: fp32 master, m, v, the 16-bit weight, and (with_acc) the
    fp32 accumulation buffer.  ``layout="tensor"`` allocates every buffer of
    every tensor separately; ``layout="flat"`` allocates one contiguous buffer
    per kind (Megatron-style flattened buffers) and hands the plan per-tensor
    views into it, each starting on a multiple of ``FLAT_ALIGN_ELEMS`` (64)
    elements.  ``g16`` gradient buffers are the caller's;
    ``grad_buffers`` makes them in the same layout.
    """

    def __init__(self, numels, dtype, with_acc=True, wd_mult=None, device="cuda",
                 layout="tensor"):
        self.numels = [int(n) for n in numels]
        self.dtype = dtype
        self.layout = layout
        self.device = device
        self.t16 = torch.bfloat16 if dtype == MP_BF16 else torch.float16
        self.master = self._alloc(torch.float32)
        self.m = self._alloc(torch.float32, zero=True)
        self.v = self._alloc(torch.float32, zero=True)
        self.w16 = self._alloc(self.t16, zero=True)
        self.acc = self._alloc(torch.float32, zero=True) if with_acc else None
        self.plan = mp_plan_create(self.numels, dtype, self.acc, self.master, self.m, self.v,
                                   self.w16, wd_mult)

    def _alloc(self, dt, zero=False):
        make = torch.zeros if zero else torch.empty
        if self.layout == "tensor":
            return [make(n, dtype=dt, device=self.device) for n in self.numels]
        assert self.layout == "flat", self.layout
        offs, total = [], 0
        for n in self.numels:
            offs.append(total)
            total += _align_elems(n)
        flat = make(total, dtype=dt, device=self.device)
        return [flat[o:o + n] for o, n in zip(offs, self.numels)]

    def grad_buffers(self):
        """One micro-batch's 16-bit gradient buffers, in this model's layout."""
        return self._alloc(self.t16)

    def gradset(self, g16):
        return mp_gradset_create(self.plan, g16)

    def close(self):
        if self.plan:
            mp_plan_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 -- interpreter shutdown
            pass
