"""Unified paged-KV attention forward for GB300 (sm_103a): Python binding.

A thin ctypes layer over the C ABI in include/ua.h (libua.so, built in-tree by
build.py). The functions below carry the C names and only marshal arguments;
every step of the attention runs in the library's CUDA kernels. Importing
succeeds without the library; the first call raises if libua.so was not
built -- there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libua.so")

UA_OK = 0
UA_ERR_INVALID_ARG = -1
UA_ERR_UNSUPPORTED = -2
UA_ERR_CUDA = -3
UA_ERR_WORKSPACE = -4
UA_ERR_DEVICE_TIMEOUT = -5
UA_ERR_BOUNDS = -6
UA_KV_BF16 = 0
UA_KV_FP8_E4M3 = 1
UA_MAX_SPLITS = 128
UA_DECODE_ROWS = 8
UA_PREFILL_ROWS = 256
UA_MIN_SOFTCAP = 2.0 ** -10
UA_MAX_SOFTCAP = 4096.0
UA_ROPE_HALF = 0
UA_ROPE_INTERLEAVED = 1
UA_ROPE_PLAIN = 0
UA_ROPE_LINEAR = 1
UA_ROPE_NTK = 2
UA_ROPE_BANDS = 3
UA_ROPE_YARN = 4
UA_ROPE_MAX_AXES = 4
UA_MIN_BLOCK_SCALE = 2.0 ** -100
UA_MAX_BLOCK_SCALE = 2.0 ** 100

# Every symbol include/ua.h declares.
EXPORTS = (
    "ua_schedule", "ua_plan_create", "ua_plan_create_ex", "ua_forward", "ua_forward_oneshot",
    "ua_plan_get_info", "ua_last_device_error", "ua_plan_destroy", "ua_status_string",
    "ua_gather_kv_debug", "ua_plan_set_profiling", "ua_plan_kernel_times",
    "ua_forward_static_scratch", "ua_plan_set_debug", "ua_append_kv",
    "ua_plan_set_unified_max", "ua_plan_set_prefill_ctas", "ua_plan_set_fp8_products", "ua_forward_host",
    "ua_rope_frequencies", "ua_rope_create", "ua_rope_destroy", "ua_rope_append_kv",
    "ua_plan_set_scores", "ua_plan_create_prefix", "ua_schedule_prefix", "ua_plan_get_batch",
    "ua_plan_create_sinks", "ua_schedule_sinks", "ua_rope_create_axes", "ua_rope_get_axes",
    "ua_rope_append_kv_axes", "ua_plan_set_block_scales",
)


class ua_tile(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("seq", "kv_head", "row0", "nrows", "kv_lo", "kv_hi", "slot", "group")]


class ua_combine_group(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("seq", "kv_head", "row0", "nrows", "slot0", "nsplits", "pad0", "pad1")]


class ua_plan_info(ctypes.Structure):
    _fields_ = [("num_prefill_tiles", ctypes.c_int64), ("num_decode_tiles", ctypes.c_int64),
                ("num_combine_groups", ctypes.c_int64), ("num_slots", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_int64), ("split_tokens", ctypes.c_int32),
                ("num_sms", ctypes.c_int32), ("num_prefill_ctas", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class UAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {ua_status_string(status)} ({status})")


_lib: Optional[ctypes.CDLL] = None

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F = ctypes.c_float
_D = ctypes.c_double
_I32P = ctypes.POINTER(ctypes.c_int32)

_SIGS = {
    "ua_status_string": (ctypes.c_char_p, [_I32]),
    "ua_schedule": (_I32, [_I32P, _I32P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                           _I32, _I32, _I32, ctypes.POINTER(ua_plan_info),
                           ctypes.POINTER(ua_tile), _I64, ctypes.POINTER(ua_tile), _I64,
                           ctypes.POINTER(ua_combine_group), _I64]),
    "ua_plan_create": (_I32, [ctypes.POINTER(_P), _I32P, _I32P, _I32, _I32, _I32, _I32, _I32,
                              _I32, _I32, _I32, _I32, _I32, _P]),
    "ua_plan_create_ex": (_I32, [ctypes.POINTER(_P), _I32P, _I32P, _I32, _I32, _I32, _I32, _I32,
                                 _I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "ua_forward": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _F, _F, _F, _P]),
    "ua_append_kv": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _F, _F, _P]),
    "ua_forward_oneshot": (_I32, [_P, _P, _P, _P, _I32P, _I32P, _P, _P, _P, _I32, _I32, _I32,
                                  _I32, _I32, _I32, _I64, _I32, _I32, _I32, _F, _I32, _I32, _F,
                                  _F, _I32, _P]),
    "ua_forward_host": (_I32, [_P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32,
                               _I32, _I64, _I32, _F, _I32, _I32, _F, _F, _I32, _I32P, _P]),
    "ua_rope_frequencies": (_I32, [_I32, _D, _I32, _D, _D, _D, _D, ctypes.POINTER(_D),
                                   ctypes.POINTER(_F)]),
    "ua_rope_create": (_I32, [ctypes.POINTER(_P), _I32, _I32, ctypes.POINTER(_D), _F]),
    "ua_rope_destroy": (_I32, [_P]),
    "ua_rope_append_kv": (_I32, [_P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P,
                                 _F, _F, _P]),
    "ua_plan_set_scores": (_I32, [_P, _F, _P]),
    "ua_plan_create_prefix": (_I32, [ctypes.POINTER(_P), _I32P, _I32P, _I32P, _I32, _I32, _I32,
                                     _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "ua_schedule_prefix": (_I32, [_I32P, _I32P, _I32P, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                  _I32, _I32, _I32, _I32, ctypes.POINTER(ua_plan_info),
                                  ctypes.POINTER(ua_tile), _I64, ctypes.POINTER(ua_tile), _I64,
                                  ctypes.POINTER(ua_combine_group), _I64]),
    "ua_plan_create_sinks": (_I32, [ctypes.POINTER(_P), _I32P, _I32P, _I32P, _I32, _I32, _I32,
                                    _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "ua_schedule_sinks": (_I32, [_I32P, _I32P, _I32P, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                 _I32, _I32, _I32, _I32, _I32, _I32,
                                 ctypes.POINTER(ua_plan_info), ctypes.POINTER(ua_tile), _I64,
                                 ctypes.POINTER(ua_tile), _I64,
                                 ctypes.POINTER(ua_combine_group), _I64]),
    "ua_rope_create_axes": (_I32, [ctypes.POINTER(_P), _I32, _I32, ctypes.POINTER(_D), _F, _I32,
                                   _I32P]),
    "ua_rope_get_axes": (_I32, [_P, _I32P]),
    "ua_rope_append_kv_axes": (_I32, [_P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64,
                                      _P, _I64, _F, _F, _P]),
    "ua_plan_set_block_scales": (_I32, [_P, _P, _P, _I64]),
    "ua_plan_get_info": (_I32, [_P, ctypes.POINTER(ua_plan_info)]),
    "ua_plan_get_batch": (_I32, [_P, ctypes.POINTER(_I64), _I32P, _I32P, _I32P]),
    "ua_last_device_error": (_I32, [_P, _I32P]),
    "ua_plan_destroy": (_I32, [_P]),
    "ua_gather_kv_debug": (_I32, [_P, _P, _P, _P, _P, _I64, _P, _P, _I64, _P]),
    "ua_plan_set_profiling": (_I32, [_P, _I32]),
    "ua_plan_set_debug": (_I32, [_P, _I32, _I64]),
    "ua_plan_set_unified_max": (_I32, [_P, _I32, _F]),
    "ua_plan_set_prefill_ctas": (_I32, [_P, _I32]),
    "ua_plan_set_fp8_products": (_I32, [_P, _I32]),
    "ua_forward_static_scratch": (_I32, [_P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32,
                                         _I32, _I32, _I64, _I32, _I32, _I32, _F, _I32, _I32, _F,
                                         _F, _I32, _P, _P]),
    "ua_plan_kernel_times": (_I32, [_P, ctypes.POINTER(ctypes.c_float),
                                    ctypes.POINTER(ctypes.c_int64)]),
}


def lib() -> ctypes.CDLL:
    """The loaded libua.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def _check(status: int, where: str):
    if status != UA_OK:
        raise UAError(status, where)


def _i32_array(values):
    vals = [int(v) for v in values]
    return (ctypes.c_int32 * max(1, len(vals)))(*vals)


def _prefix_array(prefix_lens, num_seqs, causal):
    """Host prefix lengths for the C ABI, which knows the prefix mask as causal."""
    lens = list(prefix_lens)
    if not causal:
        raise ValueError("a prefix mask is causal: causal must be 1 with prefix_lens")
    if len(lens) != num_seqs:
        raise ValueError(f"prefix_lens has {len(lens)} entries for {num_seqs} sequences")
    # 2^31 - 1 is as good as any longer one; what is negative stays so
    return _i32_array(max(-1, min(int(x), 2 ** 31 - 1)) for x in lens)


def _sinks(sink_tokens):
    # 2^31 - 1 is as good as any more; what is negative stays so
    return max(-1, min(int(sink_tokens), 2 ** 31 - 1))


def ua_status_string(status: int) -> str:
    return lib().ua_status_string(int(status)).decode()


def ua_schedule(cu_query_lens, kv_lens, num_q_heads, num_kv_heads, head_dim, block_size,
                max_blocks_per_seq, kv_dtype=UA_KV_BF16, causal=1, window=0, num_splits=0,
                num_sms=152, decode_rows_max=-1, prefix_lens=None, sink_tokens=0):
    """Run the CPU scheduler alone; returns (info, prefill, decode, groups) as
    lists of dicts. prefix_lens: a prefix mask (ua_schedule_prefix);
    sink_tokens: first keys that stay visible under the window
    (ua_schedule_sinks). Raises UAError on a rejected problem."""
    cu, kv = _i32_array(cu_query_lens), _i32_array(kv_lens)
    n = len(list(kv_lens))
    info = ua_plan_info()
    args = (cu, kv, n, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
            kv_dtype, causal, window, num_splits, num_sms, decode_rows_max)
    fn = lib().ua_schedule
    if sink_tokens:
        prefix = None if prefix_lens is None else _prefix_array(prefix_lens, n, causal)
        args = (cu, kv, prefix) + args[2:11] + (_sinks(sink_tokens),) + args[11:]
        fn = lib().ua_schedule_sinks
    elif prefix_lens is not None:
        args = (cu, kv, _prefix_array(prefix_lens, n, causal)) + args[2:9] + args[10:]
        fn = lib().ua_schedule_prefix
    _check(fn(*args, ctypes.byref(info), None, 0, None, 0, None, 0), "ua_schedule")
    pre = (ua_tile * max(1, info.num_prefill_tiles))()
    dec = (ua_tile * max(1, info.num_decode_tiles))()
    grp = (ua_combine_group * max(1, info.num_combine_groups))()
    _check(fn(*args, ctypes.byref(info), pre, info.num_prefill_tiles, dec,
              info.num_decode_tiles, grp, info.num_combine_groups), "ua_schedule")

    def rows(arr, n, cls):
        return [{f: getattr(arr[i], f) for f, _ in cls._fields_} for i in range(n)]
    return (info, rows(pre, info.num_prefill_tiles, ua_tile),
            rows(dec, info.num_decode_tiles, ua_tile),
            rows(grp, info.num_combine_groups, ua_combine_group))


def _stream_handle(stream) -> int:
    if stream is None:
        # torch's current stream without the Stream object that
        # torch.cuda.current_stream() builds (0.1 us a call against 3.0)
        import torch
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return int(getattr(stream, "cuda_stream", stream))


def ua_plan_create(cu_query_lens, kv_lens, num_q_heads, num_kv_heads, head_dim, block_size,
                   max_blocks_per_seq, kv_dtype=UA_KV_BF16, causal=1, window=0, num_splits=0,
                   decode_rows_max=-1, stream=None, prefix_lens=None, sink_tokens=0) -> int:
    """Create a plan from host lengths; returns the opaque plan handle.
    prefix_lens: keys of each sequence that all its queries see (a prefix
    mask, ua_plan_create_prefix). sink_tokens: first keys of each sequence that
    stay visible under the window (ua_plan_create_sinks)."""
    cu, kv = _i32_array(cu_query_lens), _i32_array(kv_lens)
    n = len(list(kv_lens))
    h = ctypes.c_void_p()
    if sink_tokens:
        prefix = None if prefix_lens is None else _prefix_array(prefix_lens, n, causal)
        _check(lib().ua_plan_create_sinks(ctypes.byref(h), cu, kv, prefix, n, num_q_heads,
                                          num_kv_heads, head_dim, block_size,
                                          max_blocks_per_seq, kv_dtype, causal, window,
                                          _sinks(sink_tokens), num_splits, decode_rows_max,
                                          _stream_handle(stream)), "ua_plan_create_sinks")
        return h.value
    if prefix_lens is not None:
        _check(lib().ua_plan_create_prefix(ctypes.byref(h), cu, kv,
                                           _prefix_array(prefix_lens, n, causal), n, num_q_heads,
                                           num_kv_heads, head_dim, block_size,
                                           max_blocks_per_seq, kv_dtype, window, num_splits,
                                           decode_rows_max, _stream_handle(stream)),
               "ua_plan_create_prefix")
        return h.value
    _check(lib().ua_plan_create_ex(ctypes.byref(h), cu, kv, n, num_q_heads, num_kv_heads,
                                   head_dim, block_size, max_blocks_per_seq, kv_dtype, causal,
                                   window, num_splits, decode_rows_max, _stream_handle(stream)),
           "ua_plan_create")
    return h.value


def ua_plan_get_info(plan: int) -> ua_plan_info:
    info = ua_plan_info()
    _check(lib().ua_plan_get_info(plan, ctypes.byref(info)), "ua_plan_get_info")
    return info


def ua_forward(plan, q, k_cache, v_cache, out, cu_query_lens, kv_lens, block_tables, num_blocks,
               max_q, max_kv, scale, k_scale=1.0, v_scale=1.0, stream=None):
    """Launch the forward on `stream` (default: torch's current stream).
    Tensor arguments are CUDA tensors (or raw device pointers)."""
    ptr = lambda t: t if isinstance(t, int) else t.data_ptr()
    _check(lib().ua_forward(plan, ptr(q), ptr(k_cache), ptr(v_cache), ptr(out),
                            ptr(cu_query_lens), ptr(kv_lens), ptr(block_tables), int(num_blocks),
                            int(max_q), int(max_kv), float(scale), float(k_scale),
                            float(v_scale), _stream_handle(stream)), "ua_forward")


def ua_append_kv(plan, k_new, v_new, k_cache, v_cache, block_tables, num_blocks, k_scale=1.0,
                 v_scale=1.0, stream=None):
    """Write the step's new K/V rows into the paged cache on `stream` (positions
    from the plan's lengths). Tensor arguments are CUDA tensors (or raw device
    pointers)."""
    ptr = lambda t: t if isinstance(t, int) else t.data_ptr()
    _check(lib().ua_append_kv(plan, ptr(k_new), ptr(v_new), ptr(k_cache), ptr(v_cache),
                              ptr(block_tables), int(num_blocks), float(k_scale),
                              float(v_scale), _stream_handle(stream)), "ua_append_kv")


def ua_rope_frequencies(rotary_dim, base=10000.0, scaling=UA_ROPE_PLAIN, factor=1.0,
                        original_max_position=0.0, low=1.0, high=4.0):
    """(frequencies in radians per position, amplitude) of a rotary configuration."""
    w = (ctypes.c_double * max(1, int(rotary_dim) // 2))()
    m = ctypes.c_float(0.0)
    _check(lib().ua_rope_frequencies(int(rotary_dim), float(base), int(scaling), float(factor),
                                     float(original_max_position), float(low), float(high), w,
                                     ctypes.byref(m)), "ua_rope_frequencies")
    return list(w), m.value


def ua_rope_create(inv_freq, interleaved=False, amplitude=1.0, axes=None) -> int:
    """A rope over 2 * len(inv_freq) elements of each head; returns its handle.
    axes: the position axis of each pair (0 to the number of axes less one;
    None: one axis)."""
    w = [float(x) for x in inv_freq]
    h = ctypes.c_void_p()
    if axes is not None:
        axes = [int(a) for a in axes]
        if len(axes) != len(w):
            raise ValueError(f"axes has {len(axes)} entries for {len(w)} pairs")
        # (an entry out of range stays so)
        _check(lib().ua_rope_create_axes(
            ctypes.byref(h), 2 * len(w), UA_ROPE_INTERLEAVED if interleaved else UA_ROPE_HALF,
            (ctypes.c_double * max(1, len(w)))(*w), float(amplitude),
            min(max(axes, default=0) + 1, 2 ** 31 - 1),
            _i32_array(max(-1, min(a, 2 ** 31 - 1)) for a in axes)), "ua_rope_create_axes")
        return h.value
    _check(lib().ua_rope_create(ctypes.byref(h), 2 * len(w),
                                UA_ROPE_INTERLEAVED if interleaved else UA_ROPE_HALF,
                                (ctypes.c_double * max(1, len(w)))(*w), float(amplitude)),
           "ua_rope_create")
    return h.value


def ua_rope_get_axes(rope: int) -> int:
    """The number of position axes of a rope."""
    n = ctypes.c_int32(0)
    _check(lib().ua_rope_get_axes(rope, ctypes.byref(n)), "ua_rope_get_axes")
    return n.value


def ua_rope_destroy(rope: int):
    _check(lib().ua_rope_destroy(rope), "ua_rope_destroy")


def _token_rows(t, name, tokens, device, bf16):
    """Pointer, row stride, heads and head_dim of a bf16 [tokens, heads, head_dim]
    tensor whose rows are contiguous (their distance is free)."""
    shape, stride = t.shape, t.stride()
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, not on the current CUDA device")
    if len(shape) != 3 or shape[0] != tokens or stride[2] != 1 or t.dtype != bf16 or (
            stride[1] != shape[2] and shape[1] != 1):  # (one head's distance says nothing)
        raise ValueError(f"{name}: a bf16 [tokens, heads, head_dim] tensor with contiguous rows "
                         f"is needed, of q's {tokens} tokens ({t.dtype}, shape {tuple(shape)}, "
                         f"strides {stride})")
    # with one token (or none) the stride is whatever torch holds: any valid one serves
    heads, d = shape[1], shape[2]
    return t.data_ptr(), stride[0] if tokens > 1 else heads * d, heads, d


def ua_rope_append_kv(plan, rope, q, k_new, v_new, q_out, k_cache, v_cache, block_tables,
                      num_blocks, positions=None, k_scale=1.0, v_scale=1.0, stream=None):
    """Rotate the step's q into q_out (q itself: in place), and its new keys
    and values into the paged cache, on `stream`. q, k_new and v_new are
    [tokens, heads, head_dim] CUDA tensors of the plan's heads and at least its
    tokens, whose token rows may be strided. positions: int32 [tokens], or
    [axes, tokens] with a row for each axis of the rope (the rows' distance is
    free)."""
    _rope_append(plan, None, rope, None, q, k_new, v_new, q_out, k_cache, v_cache, block_tables,
                 num_blocks, positions, k_scale, v_scale, stream)


def _rope_append(plan, batch, rope, axes, q, k_new, v_new, q_out, k_cache, v_cache, block_tables,
                 num_blocks, positions, k_scale, v_scale, stream):
    """batch: the plan's (tokens, query heads, KV heads, head_dim), axes: the rope's;
    None to ask them. Returns the stream's handle."""
    import torch
    bf16, shape = torch.bfloat16, q.shape
    n = shape[0]
    dev = torch._C._cuda_getDevice() if q.is_cuda else 0
    qp, qs, qh, qd = _token_rows(q, "q", n, dev, bf16)
    kp, ks, kh, kd = _token_rows(k_new, "k_new", n, dev, bf16)
    vp, vs, vh, vd = _token_rows(v_new, "v_new", n, dev, bf16)
    if q_out.shape != shape or q_out.dtype != bf16 or q_out.get_device() != dev or (
            not q_out.is_contiguous()):
        raise ValueError("q_out: a contiguous tensor of q's shape, type and device is needed")
    pp, p_stride = None, 0
    if positions is not None and positions.dim() == 2:
        axes = ua_rope_get_axes(rope) if axes is None else axes
        rows, step = positions.stride()
        if positions.shape != (axes, n) or positions.dtype != torch.int32 or (
                positions.get_device() != dev or (n > 1 and step != 1)):
            raise ValueError("positions: an int32 tensor [axes of the rope, tokens of q] with "
                             f"contiguous rows, on q's device, is needed ({positions.dtype}, shape "
                             f"{tuple(positions.shape)}, {axes} axes, {n} tokens)")
        if n:
            pp, p_stride = positions.data_ptr(), rows if axes > 1 else n  # (one row has no distance)
            if p_stride < n:
                raise ValueError("positions: rows that overlap (expand() gives such; copy them)")
    elif positions is not None:
        if positions.shape != (n,) or not positions.is_contiguous() or (
                positions.dtype != torch.int32 or positions.get_device() != dev):
            raise ValueError(f"positions: a contiguous int32 tensor of q's {n} tokens, on its "
                             "device, is needed")
        pp = positions.data_ptr()
    # The row distances do not show the library how many heads there are: rows
    # inside a fused projection are as wide as any plan's.
    tokens, hq, hkv, d = ua_plan_get_batch(plan) if batch is None else batch
    if n < tokens or not (qh == hq and kh == vh == hkv and qd == kd == vd == d):
        raise UAError(UA_ERR_INVALID_ARG, f"ua_rope_append_kv: q {tuple(shape)}, k_new "
                      f"{tuple(k_new.shape)}, v_new {tuple(v_new.shape)} on a plan of {tokens} "
                      f"tokens, {hq} query heads, {hkv} KV heads and head_dim {d}")
    handle = _stream_handle(stream)
    if p_stride:
        _check(lib().ua_rope_append_kv_axes(
            plan, rope, qp, qs, kp, ks, vp, vs, q_out.data_ptr(),
            k_cache if isinstance(k_cache, int) else k_cache.data_ptr(),
            v_cache if isinstance(v_cache, int) else v_cache.data_ptr(),
            block_tables if isinstance(block_tables, int) else block_tables.data_ptr(),
            int(num_blocks), pp, p_stride, float(k_scale), float(v_scale), handle),
            "ua_rope_append_kv_axes")
        return handle
    _check(lib().ua_rope_append_kv(
        plan, rope, qp, qs, kp, ks, vp, vs, q_out.data_ptr(),
        k_cache if isinstance(k_cache, int) else k_cache.data_ptr(),
        v_cache if isinstance(v_cache, int) else v_cache.data_ptr(),
        block_tables if isinstance(block_tables, int) else block_tables.data_ptr(),
        int(num_blocks), pp, float(k_scale), float(v_scale), handle), "ua_rope_append_kv")
    return handle


def ua_forward_oneshot(q, k_cache, v_cache, out, cu_query_lens_host, kv_lens_host,
                       cu_query_lens, kv_lens, block_tables, num_q_heads, num_kv_heads,
                       head_dim, block_size, max_blocks_per_seq, num_blocks, kv_dtype, max_q,
                       max_kv, scale, causal=1, window=0, k_scale=1.0, v_scale=1.0,
                       num_splits=0, stream=None):
    ptr = lambda t: t if isinstance(t, int) else t.data_ptr()
    n = len(list(kv_lens_host))
    _check(lib().ua_forward_oneshot(ptr(q), ptr(k_cache), ptr(v_cache), ptr(out),
                                    _i32_array(cu_query_lens_host), _i32_array(kv_lens_host),
                                    ptr(cu_query_lens), ptr(kv_lens), ptr(block_tables), n,
                                    num_q_heads, num_kv_heads, head_dim, block_size,
                                    max_blocks_per_seq, int(num_blocks), kv_dtype, int(max_q),
                                    int(max_kv), float(scale), causal, window, float(k_scale),
                                    float(v_scale), num_splits, _stream_handle(stream)),
           "ua_forward_oneshot")


def ua_forward_host(q_host, out_host, cu_query_lens_host, kv_lens_host, block_tables_host,
                    k_cache, v_cache, num_q_heads, num_kv_heads, head_dim, block_size,
                    num_blocks, kv_dtype, scale, causal=1, window=0, k_scale=1.0, v_scale=1.0,
                    num_splits=0, stream=None) -> int:
    """One step from host buffers (q/out/lengths/page tables on the host, the
    cache on the device); returns the device error word. Host tensors:
    contiguous CPU tensors (bf16 q / out, int32 lengths and page tables),
    pinned for asynchronous copies."""
    n = int(kv_lens_host.shape[0])
    err = ctypes.c_int32(0)
    _check(lib().ua_forward_host(
        q_host.data_ptr(), out_host.data_ptr(), cu_query_lens_host.data_ptr(),
        kv_lens_host.data_ptr(), block_tables_host.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), n, num_q_heads, num_kv_heads, head_dim, block_size,
        int(block_tables_host.shape[1]) if n else 0, num_blocks, kv_dtype, scale, causal, window,
        k_scale, v_scale, num_splits, ctypes.byref(err), _stream_handle(stream)),
        "ua_forward_host")
    return err.value


def ua_plan_get_batch(plan: int):
    """(query tokens, query heads, KV heads, head_dim) of a plan."""
    n, hq, hkv, d = (ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32())
    _check(lib().ua_plan_get_batch(plan, ctypes.byref(n), ctypes.byref(hq), ctypes.byref(hkv),
                                   ctypes.byref(d)), "ua_plan_get_batch")
    return n.value, hq.value, hkv.value, d.value


def ua_last_device_error(plan: int) -> int:
    code = ctypes.c_int32(0)
    _check(lib().ua_last_device_error(plan, ctypes.byref(code)), "ua_last_device_error")
    return code.value


def ua_plan_destroy(plan: int):
    _check(lib().ua_plan_destroy(plan), "ua_plan_destroy")


def ua_gather_kv_debug(plan, k_cache, v_cache, kv_lens, block_tables, num_blocks, k_out, v_out,
                       rows_cap, stream=None):
    ptr = lambda t: t if isinstance(t, int) else t.data_ptr()
    _check(lib().ua_gather_kv_debug(plan, ptr(k_cache), ptr(v_cache), ptr(kv_lens),
                                    ptr(block_tables), int(num_blocks), ptr(k_out), ptr(v_out),
                                    int(rows_cap), _stream_handle(stream)), "ua_gather_kv_debug")


def ua_plan_set_profiling(plan: int, enable: bool):
    _check(lib().ua_plan_set_profiling(plan, 1 if enable else 0), "ua_plan_set_profiling")


def ua_plan_set_debug(plan: int, flags: int, wait_timeout_ns: int = 0):
    """Test aid: flags bit 0 idles the prefill producer (bounded waits run out)."""
    _check(lib().ua_plan_set_debug(plan, int(flags), int(wait_timeout_ns)), "ua_plan_set_debug")


def ua_plan_set_prefill_ctas(plan: int, num_ctas: int = 0):
    """Prefill CTAs of later forwards on this plan (0: the scheduler's count)."""
    _check(lib().ua_plan_set_prefill_ctas(plan, int(num_ctas)), "ua_plan_set_prefill_ctas")


def ua_plan_set_fp8_products(plan: int, enable: bool = True):
    """fp8 tensor-core products for the prefill tiles of an e4m3 cache (later
    forwards on this plan); enable=False restores the staged bf16 path."""
    _check(lib().ua_plan_set_fp8_products(plan, 1 if enable else 0), "ua_plan_set_fp8_products")


def ua_plan_set_unified_max(plan: int, phi=None):
    """Unified max for decode rows (None: off): phi in units of the scaled
    score; rows whose first maximum lies outside its range fall back to the
    running maximum."""
    on = phi is not None
    _check(lib().ua_plan_set_unified_max(plan, int(on), float(phi) if on else 0.0),
           "ua_plan_set_unified_max")


def ua_plan_set_scores(plan: int, softcap=0.0, alibi_slopes=None):
    """Scores capped at softcap (0: none) and lowered by alibi_slopes[head] per
    position of distance (None: none) in later forwards on this plan. The
    slopes (a float32 CUDA tensor) must outlive those forwards."""
    ptr = lambda t: t if isinstance(t, int) else t.data_ptr()
    _check(lib().ua_plan_set_scores(plan, float(softcap),
                                    None if alibi_slopes is None else ptr(alibi_slopes)),
           "ua_plan_set_scores")


def ua_plan_set_block_scales(plan: int, k_scales=None, v_scales=None, num_blocks=0):
    """An e4m3 cache's scales of each physical block and KV head (float32 CUDA
    tensors [num_blocks, num_kv_heads], or raw device pointers; None: one scale
    per tensor again), for later calls on this plan. They must outlive those."""
    ptr = lambda t: t if t is None or isinstance(t, int) else t.data_ptr()
    _check(lib().ua_plan_set_block_scales(plan, ptr(k_scales), ptr(v_scales), int(num_blocks)),
           "ua_plan_set_block_scales")


KERNEL_KINDS = ("prefill", "decode", "combine", "append", "stage")


def ua_plan_kernel_times(plan: int):
    """{kind: (milliseconds, launches)} since the last read (synchronises)."""
    ms = (ctypes.c_float * len(KERNEL_KINDS))()
    n = (ctypes.c_int64 * len(KERNEL_KINDS))()
    _check(lib().ua_plan_kernel_times(plan, ms, n), "ua_plan_kernel_times")
    return {k: (ms[i], n[i]) for i, k in enumerate(KERNEL_KINDS)}


def ua_forward_static_scratch(q, k_cache, v_cache, out, cu_query_lens, kv_lens, block_tables,
                              num_q_heads, num_kv_heads, head_dim, block_size,
                              max_blocks_per_seq, num_blocks, kv_dtype, max_q, max_kv, scale,
                              causal=1, window=0, k_scale=1.0, v_scale=1.0, num_splits=0,
                              device_error=None, stream=None):
    """The forward without any device allocation (scratch in a static device
    array inside libua.so); for callers that may not allocate device memory."""
    ptr = lambda t: t if isinstance(t, int) else t.data_ptr()
    n = int(kv_lens.numel()) if hasattr(kv_lens, "numel") else int(len(kv_lens))
    _check(lib().ua_forward_static_scratch(
        ptr(q), ptr(k_cache), ptr(v_cache), ptr(out), ptr(cu_query_lens), ptr(kv_lens),
        ptr(block_tables), n, num_q_heads, num_kv_heads, head_dim, block_size,
        max_blocks_per_seq, int(num_blocks), kv_dtype, int(max_q), int(max_kv), float(scale),
        causal, window, float(k_scale), float(v_scale), num_splits,
        None if device_error is None else ptr(device_error), _stream_handle(stream)),
        "ua_forward_static_scratch")


class Rope:
    """RAII wrapper around a rope: rotary frequencies (radians per position,
    one per pair), their layout, the amplitude of the rotated pairs, and with
    positions of several axes the axis of each pair."""

    def __init__(self, inv_freq, interleaved=False, amplitude=1.0, axes=None):
        self.handle = None
        self.handle = ua_rope_create(inv_freq, interleaved, amplitude, axes)
        self.num_axes = ua_rope_get_axes(self.handle)

    @classmethod
    def scaled(cls, rotary_dim, base=10000.0, scaling=UA_ROPE_PLAIN, factor=1.0,
               original_max_position=0.0, low=1.0, high=4.0, interleaved=False, axes=None):
        """The rope of a configuration (ua_rope_frequencies)."""
        w, m = ua_rope_frequencies(rotary_dim, base, scaling, factor, original_max_position,
                                   low, high)
        return cls(w, interleaved, m, axes)

    def close(self):
        if self.handle:
            ua_rope_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class Plan:
    """RAII wrapper around a plan handle."""

    _slopes = None  # the forwards read the caller's tensor: kept as long as they may
    _slopes_streams = ()  # streams whose forwards the tensor's memory waits for
    _scales = ()  # the same of the block scales, which the appends write too
    _scales_streams = ()

    def __init__(self, *args, **kwargs):
        """Arguments as ua_plan_create."""
        self.handle = ua_plan_create(*args, **kwargs)
        self.num_tokens, self.num_q_heads, self.num_kv_heads, self.head_dim = (
            ua_plan_get_batch(self.handle))

    @property
    def info(self) -> ua_plan_info:
        return ua_plan_get_info(self.handle)

    def forward(self, q, k_cache, v_cache, out, cu_query_lens, kv_lens, block_tables, num_blocks,
                max_q, max_kv, scale, k_scale=1.0, v_scale=1.0, stream=None):
        handle = _stream_handle(stream)
        ua_forward(self.handle, q, k_cache, v_cache, out, cu_query_lens, kv_lens, block_tables,
                   num_blocks, max_q, max_kv, scale, k_scale, v_scale, handle)
        if self._slopes is not None and handle not in self._slopes_streams:
            if self._record(stream, self._slopes):
                self._slopes_streams += (handle,)
        if self._scales and handle not in self._scales_streams:
            self._scales_used(stream, handle)

    @staticmethod
    def _record(stream, *tensors) -> bool:
        """The tensors' memory waits for the stream's work so far."""
        import torch
        if stream is None:
            stream = torch.cuda.current_stream(tensors[0].device)
        if not isinstance(stream, torch.cuda.Stream):  # (a handle says nothing of its stream's life)
            return False
        for t in tensors:
            t.record_stream(stream)
        return True

    def _scales_used(self, stream, handle):
        if self._record(stream, *self._scales):
            self._scales_streams += (handle,)

    def append_kv(self, k_new, v_new, k_cache, v_cache, block_tables, num_blocks, k_scale=1.0,
                  v_scale=1.0, stream=None):
        handle = _stream_handle(stream)
        ua_append_kv(self.handle, k_new, v_new, k_cache, v_cache, block_tables, num_blocks,
                     k_scale, v_scale, handle)
        if self._scales and handle not in self._scales_streams:
            self._scales_used(stream, handle)

    def rope_append_kv(self, rope, q, k_new, v_new, q_out, k_cache, v_cache, block_tables,
                       num_blocks, positions=None, k_scale=1.0, v_scale=1.0, stream=None):
        if q.shape[0] < self.num_tokens:  # (len(q) takes four times as long)
            raise ValueError(f"q: {q.shape[0]} tokens, the plan has {self.num_tokens}")
        turn, axes = rope, None  # (rope keeps a caller's temporary alive through the call)
        if isinstance(rope, Rope):
            turn, axes = rope.handle, rope.num_axes
        handle = _rope_append(self.handle, (self.num_tokens, self.num_q_heads, self.num_kv_heads,
                                            self.head_dim),
                              turn, axes, q, k_new, v_new, q_out, k_cache, v_cache, block_tables,
                              num_blocks, positions, k_scale, v_scale, stream)
        if self._scales and handle not in self._scales_streams:
            self._scales_used(stream, handle)

    def set_scores(self, softcap=0.0, alibi_slopes=None):
        """ua_plan_set_scores; the plan holds the tensor until the next call, and
        its memory is not given out again before the plan's forwards have run
        on whatever torch streams (the caller keeps it for one on a raw stream
        handle until that has run, and for a graph that captured one until the
        last replay has)."""
        import torch
        if alibi_slopes is not None and (
                alibi_slopes.shape != (self.num_q_heads,) or not alibi_slopes.is_contiguous()
                or alibi_slopes.dtype != torch.float32):
            raise ValueError(f"alibi_slopes: a contiguous float32 tensor of {self.num_q_heads} "
                             "slopes is needed")
        ua_plan_set_scores(self.handle, softcap, alibi_slopes)
        self._slopes, self._slopes_streams = alibi_slopes, ()

    def set_block_scales(self, k_scales=None, v_scales=None):
        """ua_plan_set_block_scales, of float32 tensors [num_blocks, num_kv_heads];
        the plan holds them until the next call, and their memory is not given out
        again before the plan's calls have run (as set_scores' slopes)."""
        import torch
        if (k_scales is None) != (v_scales is None):
            raise ValueError("block scales: those of the keys and of the values, or neither")
        if k_scales is None:
            ua_plan_set_block_scales(self.handle)
            self._scales = self._scales_streams = ()
            return
        for name, x in (("k_scales", k_scales), ("v_scales", v_scales)):
            if x.dim() != 2 or x.shape[1] != self.num_kv_heads or x.shape != k_scales.shape or (
                    x.dtype != torch.float32 or not x.is_contiguous()):
                raise ValueError(f"{name}: a contiguous float32 tensor [num_blocks, "
                                 f"{self.num_kv_heads}] is needed, the same for both ({x.dtype}, "
                                 f"shape {tuple(x.shape)}, strides {x.stride()})")
        ua_plan_set_block_scales(self.handle, k_scales, v_scales, k_scales.shape[0])
        self._scales, self._scales_streams = (k_scales, v_scales), ()

    def last_device_error(self) -> int:
        return ua_last_device_error(self.handle)

    def set_unified_max(self, phi=None):
        ua_plan_set_unified_max(self.handle, phi)

    def close(self):
        if self.handle:
            ua_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
