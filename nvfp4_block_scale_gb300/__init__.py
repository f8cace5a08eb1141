"""GB300-native NVFP4 block quantization: Python binding of libnvfp4_gb300.so.

The functions named like the C ABI (``nvfp4_quantize``, ``nvfp4_dequantize``,
``nvfp4_encode_e2m1``, ``nvfp4_encode_e4m3``, ``nvfp4_status_string``) take
raw device pointers and sizes and return the C status code, exactly as
declared in include/nvfp4.h.  ``quantize`` / ``dequantize`` / ``encode_*``
are conveniences over them that take torch tensors (torch supplies device
memory and the current stream; every step of the computation runs in the
library's CUDA kernels).  There is no fallback: if the library is missing or
fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

from .build import CHECKED_LIB_PATH, LIB_PATH, build as _build

MAX, FOUR_OVER_SIX, CJSO, CJSO_DECOUPLED = 0, 1, 2, 3
MODES = {"max": MAX, "four_over_six": FOUR_OVER_SIX, "cjso": CJSO, "cjso_decoupled": CJSO_DECOUPLED}

NVFP4_OK = 0
NVFP4_GROUP_MAX = 256

# activations of the product's epilogue
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
ACTIVATIONS = {None: ACT_NONE, "none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH,
               "silu": ACT_SILU}
DTYPE_BF16, DTYPE_FP32, DTYPE_E4M3 = 0, 1, 2
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
SCORINGS = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}

_lib = None
_raw_stream = None


class nvfp4_epilogue(ctypes.Structure):
    """The epilogue of nvfp4_linear (include/nvfp4.h)."""
    _fields_ = [("bias", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64), ("activation", ctypes.c_int)]


class nvfp4_kv_cache(ctypes.Structure):
    """A paged key-value cache (include/nvfp4.h)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_page_stride", ctypes.c_int64),
                ("v_page_stride", ctypes.c_int64), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class nvfp4_expert_matrix(ctypes.Structure):
    """One matrix of every expert (include/nvfp4.h)."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("alpha", ctypes.c_void_p),
                ("code_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64), ("alpha_stride", ctypes.c_int64)]


class nvfp4_experts(ctypes.Structure):
    """The experts of nvfp4_moe (include/nvfp4.h)."""
    _fields_ = [("gate", nvfp4_expert_matrix), ("up", nvfp4_expert_matrix), ("down", nvfp4_expert_matrix),
                ("hidden", ctypes.c_int64), ("inner", ctypes.c_int64), ("experts", ctypes.c_int)]


class nvfp4_sampling(ctypes.Structure):
    """The parameters of nvfp4_sample (include/nvfp4.h)."""
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p), ("temperature_all", ctypes.c_float), ("top_k_all", ctypes.c_int),
                ("top_p_all", ctypes.c_float), ("min_p_all", ctypes.c_float)]


class nvfp4_tensor(ctypes.Structure):
    """One descriptor of nvfp4_quantize_grouped (include/nvfp4.h)."""
    _fields_ = [("W", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("alpha", ctypes.c_void_p)]


class Nvfp4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({nvfp4_status_string(status)})")
        self.status = status


def load(path: str | None = None) -> ctypes.CDLL:
    """Loads the CUDA library (building it first if it is absent or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if path is None:
        path = _build()
    if not os.path.exists(path):
        raise ImportError(f"NVFP4 CUDA library not found at {path}")
    L = ctypes.CDLL(path)
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.nvfp4_quantize.argtypes = [vp, i64, i64, ci, ci, vp, vp, vp, vp]
    L.nvfp4_quantize.restype = ci
    L.nvfp4_dequantize.argtypes = [vp, vp, vp, i64, i64, vp, vp]
    L.nvfp4_dequantize.restype = ci
    L.nvfp4_encode_e2m1.argtypes = [vp, i64, vp, vp]
    L.nvfp4_encode_e2m1.restype = ci
    L.nvfp4_encode_e4m3.argtypes = [vp, i64, vp, vp]
    L.nvfp4_encode_e4m3.restype = ci
    L.nvfp4_quantize_grouped.argtypes = [ctypes.POINTER(nvfp4_tensor), ci, ci, ci, vp]
    L.nvfp4_quantize_grouped.restype = ci
    L.nvfp4_gemv.argtypes = [vp, vp, vp, i64, i64, vp, ci, vp, vp]
    L.nvfp4_gemv.restype = ci
    L.nvfp4_gemm.argtypes = [vp, vp, vp, i64, i64, vp, ci, vp, vp]
    L.nvfp4_gemm.restype = ci
    L.nvfp4_linear_workspace_bytes.argtypes = [i64, i64, i64]
    L.nvfp4_linear_workspace_bytes.restype = i64
    L.nvfp4_linear.argtypes = [vp, vp, vp, i64, i64, vp, i64, i64, ctypes.POINTER(nvfp4_epilogue), vp, i64, vp, i64, vp]
    L.nvfp4_linear.restype = ci
    L.nvfp4_kv_append.argtypes = [ctypes.POINTER(nvfp4_kv_cache), vp, ci, i64, i64, ci, vp, vp, vp, i64, i64, i64,
                                  vp, i64, ci, ci, vp, vp]
    L.nvfp4_kv_append.restype = ci
    L.nvfp4_paged_attention_workspace_bytes.argtypes = [ctypes.POINTER(nvfp4_kv_cache), ci]
    L.nvfp4_paged_attention_workspace_bytes.restype = i64
    L.nvfp4_paged_attention.argtypes = [ctypes.POINTER(nvfp4_kv_cache), vp, i64, i64, ci, vp, vp, i64, i64,
                                        ctypes.c_float, i64, vp, vp, vp, i64, vp]
    L.nvfp4_paged_attention.restype = ci
    L.nvfp4_moe_route.argtypes = [vp, i64, i64, vp, ci, i64, i64, ci, vp, ci, ci, ctypes.c_float, ci, vp, vp, vp]
    L.nvfp4_moe_route.restype = ci
    L.nvfp4_moe_workspace_bytes.argtypes = [ctypes.POINTER(nvfp4_experts), i64, ci]
    L.nvfp4_moe_workspace_bytes.restype = i64
    L.nvfp4_moe.argtypes = [ctypes.POINTER(nvfp4_experts), vp, i64, i64, ci, vp, vp, ci, vp, i64, vp, i64, vp, i64, vp]
    L.nvfp4_moe.restype = ci
    L.nvfp4_sample.argtypes = [vp, ci, i64, i64, i64, ctypes.POINTER(nvfp4_sampling), vp, vp, vp, vp]
    L.nvfp4_sample.restype = ci
    L.nvfp4_swizzled_scales_bytes.argtypes = [i64, i64]
    L.nvfp4_swizzled_scales_bytes.restype = i64
    L.nvfp4_swizzle_scales.argtypes = [vp, i64, i64, vp, vp]
    L.nvfp4_swizzle_scales.restype = ci
    L.nvfp4_quantize_noalloc.argtypes = [vp, i64, i64, ci, vp, vp, vp, vp]
    L.nvfp4_quantize_noalloc.restype = ci
    L.nvfp4_profiler_enable.argtypes = [ci]
    L.nvfp4_profiler_enable.restype = ci
    L.nvfp4_profiler_reset.argtypes = []
    L.nvfp4_profiler_reset.restype = ci
    L.nvfp4_profiler_kinds.argtypes = []
    L.nvfp4_profiler_kinds.restype = ci
    L.nvfp4_profiler_get.argtypes = [ci, ctypes.c_char_p, ci, ctypes.POINTER(ctypes.c_int64),
                                     ctypes.POINTER(ctypes.c_double)]
    L.nvfp4_profiler_get.restype = ci
    L.nvfp4_ffma_probe.argtypes = [ci, i64, vp, i64, ctypes.POINTER(ctypes.c_int64), vp]
    L.nvfp4_ffma_probe.restype = ci
    L.nvfp4_test_fail_allocations.argtypes = [ci]
    L.nvfp4_test_fail_allocations.restype = ci
    L.nvfp4_test_first_wait_tries.argtypes = [i64]
    L.nvfp4_test_first_wait_tries.restype = ci
    L.nvfp4_test_small_clusters.argtypes = [ci]
    L.nvfp4_test_small_clusters.restype = ci
    L.nvfp4_checked_build.argtypes = []
    L.nvfp4_checked_build.restype = ci
    L.nvfp4_check_take.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    L.nvfp4_check_take.restype = ci
    L.nvfp4_check_selftest.argtypes = [i64, i64, vp]
    L.nvfp4_check_selftest.restype = ci
    L.nvfp4_status_string.argtypes = [ci]
    L.nvfp4_status_string.restype = ctypes.c_char_p
    _lib = L
    return L


def library_path() -> str:
    return LIB_PATH


def checked_library_path(build: bool = True) -> str:
    """The bounds-checked build (-DNVFP4_CHECKED), built first if asked; load
    it with load(path) before any other call of the process."""
    return _build(checked=True) if build else CHECKED_LIB_PATH


# ---------------------------------------------------------------- C ABI mirror

def nvfp4_quantize(W, rows, cols, mode, iters, codes, scales, alpha, stream) -> int:
    return load().nvfp4_quantize(W, rows, cols, mode, iters, codes, scales, alpha, stream)


def nvfp4_quantize_noalloc(W, rows, cols, mode, codes, scales, alpha, stream) -> int:
    """Allocation-free max-rule / FourOverSix quantize (see include/nvfp4.h):
    for callers that must not let the library allocate device memory."""
    return load().nvfp4_quantize_noalloc(W, rows, cols, mode, codes, scales, alpha, stream)


def nvfp4_quantize_grouped(tensors, count, mode, iters, stream) -> int:
    """`tensors`: a ctypes array of nvfp4_tensor (or None with count 0)."""
    return load().nvfp4_quantize_grouped(tensors, count, mode, iters, stream)


def nvfp4_dequantize(codes, scales, alpha, rows, cols, out, stream) -> int:
    return load().nvfp4_dequantize(codes, scales, alpha, rows, cols, out, stream)


def nvfp4_gemv(codes, scales, alpha, rows, cols, x, batch, y, stream) -> int:
    return load().nvfp4_gemv(codes, scales, alpha, rows, cols, x, batch, y, stream)


def nvfp4_gemm(codes, scales, alpha, rows, cols, x, batch, y, stream) -> int:
    return load().nvfp4_gemm(codes, scales, alpha, rows, cols, x, batch, y, stream)


def nvfp4_linear_workspace_bytes(rows, cols, batch) -> int:
    return load().nvfp4_linear_workspace_bytes(rows, cols, batch)


def nvfp4_linear(codes, scales, alpha, rows, cols, x, x_stride, batch, epilogue, y, y_stride, workspace,
                 workspace_bytes, stream) -> int:
    """`epilogue`: an nvfp4_epilogue (passed by reference) or None."""
    return load().nvfp4_linear(codes, scales, alpha, rows, cols, x, x_stride, batch, epilogue, y, y_stride,
                               workspace, workspace_bytes, stream)


def nvfp4_kv_append(cache, qkv, qkv_dtype, qkv_stride, tokens, q_heads, seq, pos, table, sequences, table_width,
                    table_stride, cos_sin, positions, rotary_dim, interleaved, q_out, stream) -> int:
    """`cache`: an nvfp4_kv_cache (passed by reference)."""
    return load().nvfp4_kv_append(cache, qkv, qkv_dtype, qkv_stride, tokens, q_heads, seq, pos, table, sequences,
                                  table_width, table_stride, cos_sin, positions, rotary_dim, interleaved, q_out,
                                  stream)


def nvfp4_paged_attention_workspace_bytes(cache, q_heads) -> int:
    return load().nvfp4_paged_attention_workspace_bytes(cache, q_heads)


def nvfp4_paged_attention(cache, q, q_stride, sequences, q_heads, lengths, table, table_width, table_stride, scale,
                          window, out, lse, workspace, workspace_bytes, stream) -> int:
    return load().nvfp4_paged_attention(cache, q, q_stride, sequences, q_heads, lengths, table, table_width,
                                        table_stride, scale, window, out, lse, workspace, workspace_bytes, stream)


def nvfp4_moe_route(x, x_stride, tokens, router, router_dtype, router_stride, hidden, experts, bias, scoring, renormalize,
                    scale, top_k, ids, weights, stream) -> int:
    return load().nvfp4_moe_route(x, x_stride, tokens, router, router_dtype, router_stride, hidden, experts, bias, scoring,
                                  renormalize, scale, top_k, ids, weights, stream)


def nvfp4_moe_workspace_bytes(experts, tokens, top_k) -> int:
    """`experts`: an nvfp4_experts (passed by reference)."""
    return load().nvfp4_moe_workspace_bytes(experts, tokens, top_k)


def nvfp4_moe(experts, x, x_stride, tokens, top_k, ids, weights, activation, residual, residual_stride, y, y_stride,
              workspace, workspace_bytes, stream) -> int:
    return load().nvfp4_moe(experts, x, x_stride, tokens, top_k, ids, weights, activation, residual, residual_stride, y,
                            y_stride, workspace, workspace_bytes, stream)


def nvfp4_sample(logits, dtype, stride, rows, vocabulary, sampling, uniform, token, logprob, stream) -> int:
    """`sampling`: an nvfp4_sampling (passed by reference) or None."""
    return load().nvfp4_sample(logits, dtype, stride, rows, vocabulary, sampling, uniform, token, logprob, stream)


def nvfp4_swizzled_scales_bytes(rows, cols) -> int:
    return load().nvfp4_swizzled_scales_bytes(rows, cols)


def nvfp4_swizzle_scales(scales, rows, cols, out, stream) -> int:
    return load().nvfp4_swizzle_scales(scales, rows, cols, out, stream)


def nvfp4_encode_e2m1(v, n, out, stream) -> int:
    return load().nvfp4_encode_e2m1(v, n, out, stream)


def nvfp4_encode_e4m3(v, n, out, stream) -> int:
    return load().nvfp4_encode_e4m3(v, n, out, stream)


def nvfp4_ffma_probe(packed, rounds, sink, sink_floats, fmas, stream) -> int:
    """fp32 FMA throughput probe (instrumentation); `fmas` is a ctypes int64 pointer."""
    return load().nvfp4_ffma_probe(packed, rounds, sink, sink_floats, fmas, stream)


def nvfp4_test_fail_allocations(count) -> int:
    """Test hook: the next `count` scratch allocations fail (out of memory)."""
    return load().nvfp4_test_fail_allocations(int(count))


def nvfp4_test_first_wait_tries(tries) -> int:
    """Test hook: the first bounded device wait gives up after `tries` polls (< 0: normal)."""
    return load().nvfp4_test_first_wait_tries(int(tries))


def nvfp4_test_small_clusters(on) -> int:
    """Test hook: moe_route and sample take clusters of 8 CTAs at most (1), or of the device's own limit (0)."""
    return load().nvfp4_test_small_clusters(int(on))


def nvfp4_checked_build() -> int:
    return load().nvfp4_checked_build()


def nvfp4_check_take(site) -> int:
    """`site`: a ctypes.c_uint32 (byref'd here)."""
    return load().nvfp4_check_take(ctypes.byref(site))


def nvfp4_check_selftest(i, n, stream) -> int:
    return load().nvfp4_check_selftest(int(i), int(n), stream)


def check_take() -> int:
    """The first failed check's site recorded since the last take (0: none);
    waits for the device to be idle.  Always 0 in the normal build."""
    site = ctypes.c_uint32(0)
    st = nvfp4_check_take(site)
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_check_take")
    return int(site.value)


def nvfp4_status_string(status: int) -> str:
    return load().nvfp4_status_string(int(status)).decode()


def nvfp4_profiler_enable(on: int) -> int:
    return load().nvfp4_profiler_enable(int(on))


def nvfp4_profiler_reset() -> int:
    return load().nvfp4_profiler_reset()


def nvfp4_profiler_kinds() -> int:
    return load().nvfp4_profiler_kinds()


def nvfp4_profiler_get(index, name, name_len, launches, total_ms) -> int:
    return load().nvfp4_profiler_get(index, name, name_len, launches, total_ms)


def profiler_report() -> dict:
    """{kernel name: (launches, total device ms)} of the traced launches."""
    n = nvfp4_profiler_kinds()
    if n < 0:
        raise Nvfp4Error(-n, "nvfp4_profiler_kinds")
    out = {}
    for i in range(n):
        buf = ctypes.create_string_buffer(64)
        cnt = ctypes.c_int64()
        ms = ctypes.c_double()
        _check(nvfp4_profiler_get(i, buf, 64, ctypes.byref(cnt), ctypes.byref(ms)), "nvfp4_profiler_get")
        out[buf.value.decode()] = (int(cnt.value), float(ms.value))
    return out


# ------------------------------------------------------------ torch helpers

def fp32_peak_tflops(seconds: float = 0.05, stream=None) -> dict:
    """Measured fp32 FMA peak of the current device (TFLOP/s): the probe
    kernel, scalar and packed, each timed with CUDA events after a warm-up
    launch; the larger of the two is the peak."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    sink = torch.empty(2048 * sms, dtype=torch.float32, device="cuda")
    res = {}
    for packed in (0, 1):
        fmas = ctypes.c_int64()
        rounds = 1 << 12
        for _ in range(12):  # grow until one launch takes about `seconds`
            _check(nvfp4_ffma_probe(packed, rounds, sink.data_ptr(), sink.numel(), ctypes.byref(fmas), s.cuda_stream),
                   "nvfp4_ffma_probe")
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record(s)
            _check(nvfp4_ffma_probe(packed, rounds, sink.data_ptr(), sink.numel(), ctypes.byref(fmas), s.cuda_stream),
                   "nvfp4_ffma_probe")
            e1.record(s)
            e1.synchronize()
            ms = e0.elapsed_time(e1)
            if ms >= seconds * 1e3 or rounds >= (1 << 30):
                break
            rounds = min(1 << 30, rounds * max(2, int(seconds * 1e3 / max(ms, 1e-3))))
        res["packed" if packed else "scalar"] = 2.0 * fmas.value / (ms / 1e3) / 1e12
    res["tflops"] = max(res["scalar"], res["packed"])
    return res


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _empty(shape, dtype, device, stream):
    """An output of a call on `stream` (None: the current one): memory that this
    stream itself last gave up, since work still running on another one may
    hold what that one gave up; and kept from reuse until the current stream,
    on which the caller goes on, has passed the point where it is dropped."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _check(status: int, what: str):
    if status != NVFP4_OK:
        raise Nvfp4Error(status, what)


def quantize(W, mode=MAX, iters: int = 0, out=None, stream=None):
    """Quantizes a contiguous bf16 CUDA tensor [rows, cols] (cols % 16 == 0).

    Returns (codes uint8 [rows, cols/2], scales uint8 [rows, cols/16] holding
    E4M3 bit patterns, alpha float32 [1]), all on W's device.  `out` may pass
    preallocated (codes, scales, alpha) tensors."""
    import torch
    if isinstance(mode, str):
        mode = MODES[mode]
    if W.dtype != torch.bfloat16 or not W.is_cuda or W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D bf16 CUDA tensor")
    rows, cols = W.shape
    if out is None:
        codes = _empty((rows, cols // 2), torch.uint8, W.device, stream)
        scales = _empty((rows, cols // 16), torch.uint8, W.device, stream)
        alpha = _empty(1, torch.float32, W.device, stream)
    else:
        codes, scales, alpha = out
    st = nvfp4_quantize(W.data_ptr(), rows, cols, int(mode), int(iters), codes.data_ptr(), scales.data_ptr(),
                        alpha.data_ptr(), _stream_ptr(stream))
    _check(st, "nvfp4_quantize")
    return codes, scales, alpha


def quantize_grouped(Ws, mode=MAX, iters: int = 0, outs=None, stream=None):
    """Quantizes a list of contiguous 2-D bf16 CUDA tensors with one grouped
    call; returns a list of (codes, scales, alpha) as `quantize` does."""
    import torch
    if isinstance(mode, str):
        mode = MODES[mode]
    res = []
    arr = (nvfp4_tensor * max(1, len(Ws)))()
    for i, W in enumerate(Ws):
        if W.dtype != torch.bfloat16 or not W.is_cuda or W.dim() != 2 or not W.is_contiguous():
            raise ValueError("every W must be a contiguous 2-D bf16 CUDA tensor")
        rows, cols = W.shape
        if outs is None:
            o = (_empty((rows, cols // 2), torch.uint8, W.device, stream),
                 _empty((rows, cols // 16), torch.uint8, W.device, stream),
                 _empty(1, torch.float32, W.device, stream))
        else:
            o = outs[i]
        arr[i] = nvfp4_tensor(W.data_ptr(), rows, cols, o[0].data_ptr(), o[1].data_ptr(), o[2].data_ptr())
        res.append(o)
    _check(nvfp4_quantize_grouped(arr, len(Ws), int(mode), int(iters), _stream_ptr(stream)),
           "nvfp4_quantize_grouped")
    return res


def dequantize(codes, scales, alpha, rows: int, cols: int, out=None, stream=None):
    """Returns the bf16 CUDA tensor [rows, cols] that the NVFP4 tensor encodes."""
    import torch
    if out is None:
        out = _empty((rows, cols), torch.bfloat16, codes.device, stream)
    st = nvfp4_dequantize(codes.data_ptr(), scales.data_ptr(), alpha.data_ptr(), rows, cols, out.data_ptr(),
                          _stream_ptr(stream))
    _check(st, "nvfp4_dequantize")
    return out


def gemv(codes, scales, alpha, rows: int, cols: int, x, out=None, stream=None):
    """y [batch, rows] fp32 = dequantized weights [rows, cols] times the bf16
    activations x [batch, cols] (batch 1..8), on x's device."""
    import torch
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous() or x.shape[1] != cols:
        raise ValueError("x must be a contiguous bf16 CUDA tensor [batch, cols]")
    batch = x.shape[0]
    y = out if out is not None else _empty((batch, rows), torch.float32, x.device, stream)
    _check(nvfp4_gemv(codes.data_ptr(), scales.data_ptr(), alpha.data_ptr(), rows, cols, x.data_ptr(), batch,
                      y.data_ptr(), _stream_ptr(stream)), "nvfp4_gemv")
    return y


def gemm(codes, scales, alpha, rows: int, cols: int, x, out=None, stream=None):
    """As gemv, on the tensor cores, for x [batch, cols] with batch 1..256."""
    import torch
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous() or x.shape[1] != cols:
        raise ValueError("x must be a contiguous bf16 CUDA tensor [batch, cols]")
    batch = x.shape[0]
    y = out if out is not None else _empty((batch, rows), torch.float32, x.device, stream)
    _check(nvfp4_gemm(codes.data_ptr(), scales.data_ptr(), alpha.data_ptr(), rows, cols, x.data_ptr(), batch,
                      y.data_ptr(), _stream_ptr(stream)), "nvfp4_gemm")
    return y


def _on(device, stream):
    """The handle of the stream to launch on."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        _raw_stream = _current_raw()
    return _raw_stream(device.index)


def _current_raw():
    # the current stream's handle without making a Stream object: 0.1 us instead of 3
    try:
        from torch._C import _cuda_getCurrentRawStream
        return _cuda_getCurrentRawStream
    except ImportError:
        import torch
        return lambda index: torch.cuda.current_stream(index).cuda_stream


def _workspace(nbytes: int, device):
    import torch
    if nbytes < 0:
        raise ValueError("invalid shape, or no supported device")
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def _space(workspace, device):
    """Address and size of a caller's workspace, or nothing."""
    if workspace is None:
        return None, 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"a workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.nbytes


def _rows_of(t, batch: int, width: int, what: str):
    import torch
    strides = t.stride()
    if t.dtype is not torch.bfloat16 or not t.is_cuda or t.shape != (batch, width) or (width > 1 and strides[1] != 1):
        raise ValueError(f"{what} must be a bf16 CUDA tensor [{batch}, {width}] with contiguous rows")
    return t.data_ptr(), strides[0] if batch > 1 and width > 0 else (width + 7) // 8 * 8


def linear_workspace(rows: int, cols: int, batch: int, device="cuda"):
    """A workspace for linear() of this shape and up to `batch` vectors, kept by
    the caller from call to call (one per stream that such calls run on)."""
    return _workspace(nvfp4_linear_workspace_bytes(rows, cols, batch), device)


def linear(codes, scales, alpha, rows: int, cols: int, x, bias=None, activation=None, gate=None, residual=None,
           out=None, workspace=None, stream=None):
    """The W4A16 product with its epilogue: bf16 y [batch, rows] =
    residual + gate * activation(W x + bias), W = q * Delta * alpha, for bf16 x
    [batch, cols]; bias [rows], gate and residual [batch, rows] bf16 or None;
    activation: None, "relu", "gelu", "gelu_tanh" or "silu".  x, gate, residual
    and out may have rows further apart than their width; out may be the
    residual.  See nvfp4_linear in include/nvfp4.h."""
    import torch
    if x.dim() == 1:
        x = x.unsqueeze(0)
    batch = x.shape[0]
    xp, xs = _rows_of(x, batch, cols, "x")
    if codes.numel() * 2 != rows * cols or scales.numel() * 16 != rows * cols or not codes.is_contiguous() or \
            not scales.is_contiguous() or codes.element_size() != 1 or scales.element_size() != 1 or \
            not codes.is_cuda or not scales.is_cuda:
        raise ValueError("codes and scales must be contiguous CUDA tensors of bytes that hold [rows, cols] elements")
    if alpha.dtype is not torch.float32 or not alpha.is_cuda or alpha.numel() < 1:
        raise ValueError("alpha must be an fp32 CUDA tensor [1]")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(k for k in ACTIVATIONS if k)}")
    bp = gp = rp = None
    gs = rs = 0
    if bias is not None:
        if bias.dtype is not torch.bfloat16 or not bias.is_cuda or bias.shape != (rows,) or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous bf16 CUDA tensor [rows]")
        bp = bias.data_ptr()
    if gate is not None:
        gp, gs = _rows_of(gate, batch, rows, "gate")
    if residual is not None:
        rp, rs = _rows_of(residual, batch, rows, "residual")
    if out is None:
        out = _empty((batch, rows), torch.bfloat16, x.device, stream)
    yp, ys = _rows_of(out, batch, rows, "out")
    wp, wb = _space(workspace, x.device)
    ep = nvfp4_epilogue(bp, gp, gs, rp, rs, ACTIVATIONS[activation])
    _check((_lib or load()).nvfp4_linear(codes.data_ptr(), scales.data_ptr(), alpha.data_ptr(), rows, cols, xp, xs, batch,
                                         ep, yp, ys, wp, wb, _on(x.device, stream)), "nvfp4_linear")
    return out


class KVCache:
    """A paged key-value cache: k and v bf16 or float8_e4m3fn CUDA tensors
    [pages, kv_heads, page_size, head_dim], contiguous inside a page (the pages
    may lie further apart); k_scale and v_scale [kv_heads] fp32 give the value
    of one unit of an E4M3 cache (None: 1).  The tensors stay the caller's;
    this object is the handle that kv_append and paged_attention take."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        kinds = {torch.bfloat16: DTYPE_BF16, torch.float8_e4m3fn: DTYPE_E4M3}
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in kinds or not k.is_cuda or \
                k.device != v.device:
            raise ValueError("k and v must be alike: bf16 or float8_e4m3fn CUDA tensors "
                             "[pages, kv_heads, page_size, head_dim]")
        pages, heads, size, dim = k.shape
        for t in (k, v):
            if pages > 0 and not t[0].is_contiguous():
                raise ValueError("keys and values must be contiguous inside a page")
        for t in (k_scale, v_scale):
            if t is not None and (k.dtype == torch.bfloat16 or t.dtype != torch.float32 or t.device != k.device or
                                  t.shape != (heads,) or not t.is_contiguous()):
                raise ValueError("scales are for E4M3 caches: contiguous fp32 CUDA tensors [kv_heads]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, size, dim
        self.device = k.device
        page = heads * size * dim
        self.desc = nvfp4_kv_cache(k.data_ptr(), v.data_ptr(), k.stride(0) if pages > 1 else page,
                                   v.stride(0) if pages > 1 else page, pages, size, heads, dim, kinds[k.dtype],
                                   None if k_scale is None else k_scale.data_ptr(),
                                   None if v_scale is None else v_scale.data_ptr())

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page_size: int, head_dim: int, dtype=None, device="cuda", k_scale=None,
              v_scale=None):
        """A cache of uninitialised pages (dtype: torch.bfloat16, the default, or torch.float8_e4m3fn)."""
        import torch
        shape = (pages, kv_heads, page_size, head_dim)
        make = lambda: torch.empty(shape, dtype=dtype or torch.bfloat16, device=device)  # noqa: E731
        return cls(make(), make(), k_scale, v_scale)


def _ints(t, n: int, what: str):
    import torch
    if t.dtype is not torch.int32 or not t.is_cuda or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 CUDA tensor [{n}]")
    return t.data_ptr()


def _table_of(table):
    import torch
    if table.dtype is not torch.int32 or not table.is_cuda or table.dim() != 2:
        raise ValueError("table must be an int32 CUDA tensor [sequences, pages of a sequence]")
    n, width = table.shape
    step, one = table.stride()
    if one != 1 and width > 1:
        raise ValueError("table must have contiguous rows")
    return table.data_ptr(), n, width, step if n > 1 else width


def kv_append(cache: KVCache, qkv, q_heads: int, seq, pos, table, cos_sin=None, interleaved: bool = False, out=None,
              stream=None):
    """Writes the keys and values of new tokens into the cache and returns the
    queries, bf16 [tokens, q_heads, head_dim]; queries and keys are rotated by
    position on the way.  qkv: bf16 or fp32 CUDA [tokens, (q_heads + 2 kv_heads)
    * head_dim]; seq, pos: int32 [tokens] (pos -1: padding); table: int32
    [sequences, pages]; cos_sin: fp32 [positions, rotary_dim], cosines then
    sines (None: no rotation).  See nvfp4_kv_append in include/nvfp4.h."""
    import torch
    dim = cache.head_dim
    width = (q_heads + 2 * cache.kv_heads) * dim
    kind = qkv.dtype
    if (kind is not torch.bfloat16 and kind is not torch.float32) or not qkv.is_cuda or qkv.dim() != 2 or \
            qkv.shape[1] != width or qkv.stride(1) != 1:
        raise ValueError(f"qkv must be a bf16 or fp32 CUDA tensor [tokens, {width}] with contiguous rows")
    tokens = qkv.shape[0]
    sp, pp = _ints(seq, tokens, "seq"), _ints(pos, tokens, "pos")
    tp, sequences, pages, stride = _table_of(table)
    cp, positions, rotary = None, 0, 0
    if cos_sin is not None:
        if cos_sin.dtype is not torch.float32 or not cos_sin.is_cuda or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous fp32 CUDA tensor [positions, rotary_dim]")
        positions, rotary = cos_sin.shape
        cp = cos_sin.data_ptr()
    shape = (tokens, q_heads, dim)
    if out is None:
        out = _empty(shape, torch.bfloat16, cache.device, stream)
    elif out.dtype is not torch.bfloat16 or not out.is_cuda or out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous bf16 CUDA tensor {list(shape)}")
    _check((_lib or load()).nvfp4_kv_append(cache.desc, qkv.data_ptr(), DTYPE_FP32 if kind is torch.float32 else DTYPE_BF16,
                                            qkv.stride(0) if tokens > 1 else width, tokens, q_heads, sp, pp, tp,
                                            sequences, pages, stride, cp, positions, rotary, bool(interleaved),
                                            out.data_ptr(), _on(cache.device, stream)), "nvfp4_kv_append")
    return out


def attention_workspace(cache: KVCache, q_heads: int):
    """A workspace for paged_attention() over this cache, whatever the batch
    and the lengths, kept by the caller from call to call (one per stream)."""
    return _workspace(nvfp4_paged_attention_workspace_bytes(cache.desc, q_heads), cache.device)


def paged_attention(cache: KVCache, q, table, lengths, scale=None, window: int = 0, out=None, return_lse: bool = False,
                    workspace=None, stream=None):
    """Attention of one new token per sequence over the cache: bf16 out like q
    [sequences, q_heads, head_dim], with return_lse also the fp32 log-sum-exp
    [sequences, q_heads].  lengths: int32 [sequences], tokens in the cache with
    the new one (0: an empty row); window: only the last `window` tokens (0:
    all); scale: head_dim ** -0.5 by default.  See nvfp4_paged_attention in
    include/nvfp4.h."""
    import torch
    shape, strides, dim = q.shape, q.stride(), cache.head_dim
    if q.dtype is not torch.bfloat16 or not q.is_cuda or len(shape) != 3 or shape[2] != dim or strides[2] != 1 or \
            (shape[1] > 1 and strides[1] != dim):
        raise ValueError("q must be a bf16 CUDA tensor [sequences, q_heads, head_dim] with contiguous sequences")
    n, heads, _ = shape
    tp, sequences, pages, stride = _table_of(table)
    if sequences != n:
        raise ValueError("table must have one row per sequence")
    lp = _ints(lengths, n, "lengths")
    lse = None
    if out is None:
        out = _empty(shape, torch.bfloat16, cache.device, stream)
    elif out.dtype is not torch.bfloat16 or not out.is_cuda or out.shape != shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 CUDA tensor shaped like q")
    if return_lse:
        lse = _empty((n, heads), torch.float32, cache.device, stream)
    wp, wb = _space(workspace, cache.device)
    _check((_lib or load()).nvfp4_paged_attention(
        cache.desc, q.data_ptr(), strides[0] if n > 1 else heads * dim, n, heads, lp, tp, pages, stride,
        dim ** -0.5 if scale is None else scale, window, out.data_ptr(), None if lse is None else lse.data_ptr(), wp, wb,
        _on(cache.device, stream)), "nvfp4_paged_attention")
    return (out, lse) if return_lse else out


def moe_route(x, router, top_k: int, scoring: str = "softmax", renormalize: bool = True, bias=None, scale: float = 1.0,
              stream=None):
    """The router of a mixture-of-experts layer: (ids int32, weights fp32), both
    [tokens, top_k], of each token's top_k experts in descending order of their
    scores, for bf16 x [tokens, hidden] and a bf16 or fp32 router [experts,
    hidden] (rows may lie further apart than their width).  scoring "softmax":
    chosen by the logits, weighted by their softmax over all experts;
    "sigmoid": chosen by sigmoid(logit) + bias (fp32 [experts] or None), weighted
    by the sigmoid.  renormalize: a token's weights sum to 1; scale multiplies
    them.  See nvfp4_moe_route in include/nvfp4.h."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be a bf16 CUDA tensor [tokens, hidden]")
    tokens, hidden = x.shape
    xp, xs = _rows_of(x, tokens, hidden, "x")
    kind = router.dtype
    if (kind is not torch.bfloat16 and kind is not torch.float32) or router.device != x.device or router.dim() != 2 or \
            router.shape[1] != hidden or (hidden > 1 and router.stride(1) != 1):
        raise ValueError(f"router must be a bf16 or fp32 tensor [experts, {hidden}] with contiguous rows on x's device")
    experts = router.shape[0]
    if scoring not in SCORINGS:
        raise ValueError(f"scoring must be one of {sorted(SCORINGS)}")
    bp = None
    if bias is not None:
        if scoring != "sigmoid" or bias.dtype is not torch.float32 or bias.device != x.device or \
                bias.shape != (experts,) or not bias.is_contiguous():
            raise ValueError("bias goes with sigmoid: a contiguous fp32 tensor [experts] on x's device")
        bp = bias.data_ptr()
    ids = _empty((tokens, top_k), torch.int32, x.device, stream)
    weights = _empty((tokens, top_k), torch.float32, x.device, stream)
    _check((_lib or load()).nvfp4_moe_route(
        xp, xs, tokens, router.data_ptr(), DTYPE_FP32 if kind is torch.float32 else DTYPE_BF16,
        router.stride(0) if experts > 1 else (hidden + 7) // 8 * 8, hidden, experts, bp, SCORINGS[scoring], bool(renormalize),
        scale, top_k, ids.data_ptr(), weights.data_ptr(), _on(x.device, stream)), "nvfp4_moe_route")
    return ids, weights


class Experts:
    """The quantized experts of a mixture-of-experts layer: up, down and (None:
    none) gate are each (codes, scales, alpha) of all experts: codes CUDA bytes
    [experts, rows, cols/2] and scales [experts, rows, cols/16], contiguous
    inside an expert (the experts may lie further apart), alpha fp32 [experts].
    gate and up are [inner, hidden] matrices, down [hidden, inner].  The tensors
    stay the caller's; this object is the handle that moe() takes."""

    def __init__(self, up, down, gate=None):
        import torch
        codes = up[0]
        if codes.dim() != 3 or not codes.is_cuda:
            raise ValueError("codes must be CUDA tensors [experts, rows, cols / 2]")
        n, inner, half = codes.shape
        hidden = 2 * half

        def matrix(m, rows, cols, what):
            c, s, a = m
            if c.shape != (n, rows, cols // 2) or s.shape != (n, rows, cols // 16) or c.element_size() != 1 or \
                    s.element_size() != 1 or c.device != codes.device or s.device != codes.device or \
                    (n > 0 and not (c[0].is_contiguous() and s[0].is_contiguous())):
                raise ValueError(f"{what}: codes and scales must be CUDA bytes [{n}, {rows}, {cols // 2}] and "
                                 f"[{n}, {rows}, {cols // 16}], contiguous inside an expert")
            if a.dtype is not torch.float32 or a.device != codes.device or a.dim() < 1 or a.shape[0] != n or \
                    a.numel() != n:
                raise ValueError(f"{what}: alpha must be an fp32 tensor [{n}] on the codes' device")
            return nvfp4_expert_matrix(c.data_ptr(), s.data_ptr(), a.data_ptr(), c.stride(0), s.stride(0), a.stride(0))

        self.tensors = (up, down, gate)
        self.experts, self.hidden, self.inner, self.device = n, hidden, inner, codes.device
        self.desc = nvfp4_experts(nvfp4_expert_matrix() if gate is None else matrix(gate, inner, hidden, "gate"),
                                  matrix(up, inner, hidden, "up"), matrix(down, hidden, inner, "down"), hidden, inner, n)

    @classmethod
    def quantize(cls, up, down, gate=None, mode=MAX, iters: int = 0, stream=None):
        """Experts quantized from contiguous bf16 CUDA tensors up [experts, inner,
        hidden], down [experts, hidden, inner] and gate like up (or None), all
        in one grouped call."""
        import torch
        ws, outs, parts = [], [], []
        for w in (up, down, gate):
            if w is None:
                parts.append(None)
                continue
            n, rows, cols = w.shape
            part = (_empty((n, rows, cols // 2), torch.uint8, w.device, stream),
                    _empty((n, rows, cols // 16), torch.uint8, w.device, stream), _empty(n, torch.float32, w.device, stream))
            ws += list(w)
            outs += [(part[0][i], part[1][i], part[2][i:i + 1]) for i in range(n)]
            parts.append(part)
        quantize_grouped(ws, mode, iters, outs, stream)
        return cls(*parts)


def moe_workspace(experts: Experts, tokens: int, top_k: int):
    """A workspace for moe() of up to `tokens` tokens, kept by the caller from
    call to call (one per stream that such calls run on)."""
    return _workspace(nvfp4_moe_workspace_bytes(experts.desc, tokens, top_k), experts.device)


def moe(experts: Experts, x, ids, weights, activation="silu", residual=None, out=None, workspace=None, stream=None):
    """The experts' products of a mixture-of-experts layer: bf16 y [tokens,
    hidden] = residual + sum over a token's slots of weights * down(act(gate x) *
    up x) (without a gate: down(act(up x))), for bf16 x [tokens, hidden] and the
    slots' experts and weights, int32 and fp32 [tokens, top_k], as moe_route
    gives them; an id outside [0, experts) adds nothing (-1: padding).  x,
    residual and out may have rows further apart than their width; out may be
    the residual or x.  See nvfp4_moe in include/nvfp4.h."""
    import torch
    tokens, top_k = ids.shape
    if ids.dtype is not torch.int32 or not ids.is_contiguous() or ids.device != experts.device or \
            weights.dtype is not torch.float32 or weights.shape != ids.shape or not weights.is_contiguous() or \
            weights.device != experts.device:
        raise ValueError("ids and weights must be contiguous int32 and fp32 tensors [tokens, top_k] on the experts' device")
    hidden = experts.hidden
    xp, xs = _rows_of(x, tokens, hidden, "x")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(k for k in ACTIVATIONS if k)}")
    rp, rs = (None, 0) if residual is None else _rows_of(residual, tokens, hidden, "residual")
    if out is None:
        out = _empty((tokens, hidden), torch.bfloat16, experts.device, stream)
    yp, ys = _rows_of(out, tokens, hidden, "out")
    if not experts.device == x.device == out.device == (x if residual is None else residual).device:
        raise ValueError("x, residual and out must be on the experts' device")
    wp, wb = _space(workspace, experts.device)
    _check((_lib or load()).nvfp4_moe(experts.desc, xp, xs, tokens, top_k, ids.data_ptr(), weights.data_ptr(),
                                      ACTIVATIONS[activation], rp, rs, yp, ys, wp, wb, _on(experts.device, stream)),
           "nvfp4_moe")
    return out


def _setting(v, off, rows: int, kind, device, what: str):
    """A sampling parameter: the address of a tensor [rows], or nothing and one value."""
    import torch
    if isinstance(v, torch.Tensor):
        if v.dtype is not kind or v.shape != (rows,) or v.device != device or not v.is_contiguous():
            raise ValueError(f"{what} must be a number or a contiguous {kind} tensor [{rows}] on the logits' device")
        return v.data_ptr(), off
    return None, off if v is None else v


def sample(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None, return_logprob: bool = False,
           stream=None):
    """The next token of each row of logits (bf16 or fp32 [rows, vocabulary], rows
    may lie further apart than their width): int32 [rows], with return_logprob
    also the fp32 logarithm of its probability among the tokens that stay.
    uniform: fp32 [rows] random numbers in [0, 1).  temperature (1), top_k (all),
    top_p (1), min_p (0): a number, a tensor [rows] (fp32; top_k int32) or None.
    temperature 0 takes the largest; logits of -inf are masked, and a row of
    them gives -1.  See nvfp4_sample in include/nvfp4.h."""
    import torch
    kind = logits.dtype
    if (kind is not torch.bfloat16 and kind is not torch.float32) or not logits.is_cuda or logits.dim() != 2 or \
            (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a bf16 or fp32 CUDA tensor [rows, vocabulary] with contiguous rows")
    rows, vocabulary = logits.shape
    device = logits.device
    if uniform.dtype is not torch.float32 or uniform.shape != (rows,) or uniform.device != device or \
            not uniform.is_contiguous():
        raise ValueError(f"uniform must be a contiguous fp32 tensor [{rows}] on the logits' device")
    tp, t = _setting(temperature, 1.0, rows, torch.float32, device, "temperature")
    kp, k = _setting(top_k, 0, rows, torch.int32, device, "top_k")
    k = max(min(k, vocabulary), 0)
    pp, p = _setting(top_p, 1.0, rows, torch.float32, device, "top_p")
    mp, m = _setting(min_p, 0.0, rows, torch.float32, device, "min_p")
    token = _empty((rows,), torch.int32, device, stream)
    logprob = _empty((rows,), torch.float32, device, stream) if return_logprob else None
    _check((_lib or load()).nvfp4_sample(
        logits.data_ptr(), DTYPE_FP32 if kind is torch.float32 else DTYPE_BF16,
        logits.stride(0) if rows > 1 else vocabulary, rows, vocabulary, nvfp4_sampling(tp, kp, pp, mp, t, k, p, m),
        uniform.data_ptr(), token.data_ptr(), None if logprob is None else logprob.data_ptr(), _on(device, stream)),
        "nvfp4_sample")
    return (token, logprob) if return_logprob else token


def swizzle_scales(scales, rows: int, cols: int, stream=None):
    """The [rows, cols/16] scales in the tensor-core tile layout (flat uint8)."""
    import torch
    out = _empty(nvfp4_swizzled_scales_bytes(rows, cols), torch.uint8, scales.device, stream)
    _check(nvfp4_swizzle_scales(scales.data_ptr(), rows, cols, out.data_ptr(), _stream_ptr(stream)),
           "nvfp4_swizzle_scales")
    return out


def encode_e2m1(v, stream=None):
    import torch
    out = _empty(v.shape, torch.uint8, v.device, stream)
    _check(nvfp4_encode_e2m1(v.data_ptr(), v.numel(), out.data_ptr(), _stream_ptr(stream)), "nvfp4_encode_e2m1")
    return out


def encode_e4m3(v, stream=None):
    import torch
    out = _empty(v.shape, torch.uint8, v.device, stream)
    _check(nvfp4_encode_e4m3(v.data_ptr(), v.numel(), out.data_ptr(), _stream_ptr(stream)), "nvfp4_encode_e4m3")
    return out
