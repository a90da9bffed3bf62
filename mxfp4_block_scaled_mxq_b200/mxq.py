"""Thin Python binding of libmxq (the C ABI in include/mxq.h).

Argument marshalling only: every step of the quantized linear layer runs in the
library's sm_100a kernels.  Functions named ``mxq_*`` mirror the C entry points one
for one (device buffers may be given as torch CUDA tensors or raw integer device
pointers); the lower-case helpers below them allocate the output tensors and call
the ``mxq_*`` functions.  There is no fallback: if the shared library is missing or
the device is not an sm_100 GPU, calls raise.
"""

from __future__ import annotations

import ctypes
import functools
import inspect
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxq.so")

MXQ_OK = 0
STATUS_NAMES = {0: "MXQ_OK", 1: "MXQ_ERR_INVALID_ARG", 2: "MXQ_ERR_SHAPE", 3: "MXQ_ERR_ALIGN",
                4: "MXQ_ERR_UNSUPPORTED", 5: "MXQ_ERR_CUDA", 6: "MXQ_ERR_TIMEOUT"}
MXQ_SCALE_OCP, MXQ_SCALE_UOS = 0, 1
MXQ_ACT_MXFP4, MXQ_ACT_FP8_E4M3 = 0, 1
MXQ_NORM_HEAD, MXQ_NORM_ROW = 0, 1
MXQ_ROPE_HALVES, MXQ_ROPE_PAIRS = 0, 1
MXQ_KV_BF16, MXQ_KV_FP8_E4M3 = 0, 1
MXQ_PREC_W4A4, MXQ_PREC_W4A4_TRANSFORM, MXQ_PREC_W4A8, MXQ_PREC_BF16 = 0, 1, 2, 3

EXPORTED = ("mxq_status_string", "mxq_sf_bytes", "mxq_quantize_act", "mxq_pack_weight", "mxq_gemm_w4a4",
            "mxq_gemm_w4a8", "mxq_dequant_mxfp4", "mxq_qdq_act", "mxq_channel_absmax", "mxq_smooth_factors",
            "mxq_quantize_smooth", "mxq_sqnr_accumulate", "mxq_sqnr_db", "mxq_select_precision", "mxq_attn_padded_keys",
            "mxq_attn_code_poly", "mxq_quantize_vt",
            "mxq_attention_mxfp4", "mxq_qk_norm_rope", "mxq_kv_append", "mxq_attention_paged_workspace_bytes",
            "mxq_attention_paged", "mxq_linear_workspace_bytes", "mxq_linear_w4a4", "mxq_linear_w4a4_static",
            "mxq_debug_poll", "mxq_selftest_wait_timeout")


class MxqError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class NormRope(ctypes.Structure):
    """mxq_norm_rope: norm weights and epsilon, rotation table and style."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_rows", ctypes.c_int64), ("rot", ctypes.c_int64), ("eps", ctypes.c_float),
                ("span", ctypes.c_int), ("style", ctypes.c_int)]


class PagedKVArgs(ctypes.Structure):
    """mxq_paged_kv: buffers, sizes, strides (elements) and format of a paged cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("heads", ctypes.c_int64), ("d", ctypes.c_int64),
                ("stride_page", ctypes.c_int64), ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64),
                ("fmt", ctypes.c_int), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class PagedBatchArgs(ctypes.Structure):
    """mxq_paged_batch: row offsets, lengths and pages of a batch of sequences."""
    _fields_ = [("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("batch", ctypes.c_int64), ("max_pages", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libmxq.so from the package directory (built by ``build.py``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"libmxq.so not built ({_LIB_PATH}); run `python -m mxfp4_block_scaled_mxq_b200.build`")
    L = ctypes.CDLL(_LIB_PATH)
    P, I64, I32, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.mxq_status_string.argtypes = [I32]
    L.mxq_status_string.restype = ctypes.c_char_p
    L.mxq_sf_bytes.argtypes = [I64, I64]
    L.mxq_sf_bytes.restype = I64
    L.mxq_quantize_act.argtypes = [P, I64, I64, I64, I32, I32, I32, F32, P, P, P]
    L.mxq_quantize_act.restype = I32
    L.mxq_pack_weight.argtypes = [P, I64, I64, I64, I32, I32, P, P, P]
    L.mxq_pack_weight.restype = I32
    L.mxq_gemm_w4a4.argtypes = [P, P, P, P, I64, I64, I64, F32, P, P, I64, P]
    L.mxq_gemm_w4a4.restype = I32
    L.mxq_gemm_w4a8.argtypes = [P, F32, P, P, I64, I64, I64, P, P, I64, P]
    L.mxq_gemm_w4a8.restype = I32
    L.mxq_dequant_mxfp4.argtypes = [P, P, I64, I64, P, I64, P]
    L.mxq_dequant_mxfp4.restype = I32
    L.mxq_qdq_act.argtypes = [P, I64, I64, I64, I32, I32, I32, F32, P, I64, P]
    L.mxq_qdq_act.restype = I32
    L.mxq_channel_absmax.argtypes = [P, I64, I64, I64, I32, I32, P, P]
    L.mxq_channel_absmax.restype = I32
    L.mxq_smooth_factors.argtypes = [P, P, I64, F32, P, P, P]
    L.mxq_smooth_factors.restype = I32
    L.mxq_quantize_smooth.argtypes = [P, I64, I64, I64, I32, I32, P, P, P, P]
    L.mxq_quantize_smooth.restype = I32
    L.mxq_sqnr_accumulate.argtypes = [P, I64, P, I64, I64, I64, I32, P, P]
    L.mxq_sqnr_accumulate.restype = I32
    L.mxq_sqnr_db.argtypes = [ctypes.c_double, ctypes.c_double]
    L.mxq_sqnr_db.restype = ctypes.c_double
    L.mxq_select_precision.argtypes = [ctypes.c_double] * 4
    L.mxq_select_precision.restype = I32
    L.mxq_attn_padded_keys.argtypes = [I64]
    L.mxq_attn_padded_keys.restype = I64
    L.mxq_quantize_vt.argtypes = [P, I64, I64, I64, I32, P, P, P]
    L.mxq_quantize_vt.restype = I32
    L.mxq_attn_code_poly.argtypes = [P]
    L.mxq_attn_code_poly.restype = None
    L.mxq_attention_mxfp4.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, I32, P, I64, P]
    L.mxq_attention_mxfp4.restype = I32
    L.mxq_qk_norm_rope.argtypes = [P, I64, I64, P, I64, I64, P, I64, P, I64, I64, P, I64, P, P]
    L.mxq_qk_norm_rope.restype = I32
    L.mxq_kv_append.argtypes = [P, P, P, I64, P, I64, P, I64, P, I64, I64, P, I64, P]
    L.mxq_kv_append.restype = I32
    L.mxq_attention_paged_workspace_bytes.argtypes = [I64] * 5
    L.mxq_attention_paged_workspace_bytes.restype = I64
    L.mxq_attention_paged.argtypes = [P, I64, I64, I64, P, P, I32, I64, F32, P, I64, P, I64, P]
    L.mxq_attention_paged.restype = I32
    L.mxq_linear_workspace_bytes.argtypes = [I64, I64]
    L.mxq_linear_workspace_bytes.restype = I64
    L.mxq_linear_w4a4.argtypes = [P, I64, I64, I64, I32, P, P, I64, F32, P, P, I64, P, I64, P]
    L.mxq_linear_w4a4.restype = I32
    L.mxq_linear_w4a4_static.argtypes = [P, I64, I64, I64, I32, P, P, I64, F32, P, P, I64, P]
    L.mxq_linear_w4a4_static.restype = I32
    L.mxq_debug_poll.argtypes = []
    L.mxq_debug_poll.restype = I32
    L.mxq_selftest_wait_timeout.argtypes = [P]
    L.mxq_selftest_wait_timeout.restype = I32
    _lib = L
    return L


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("libmxq takes device buffers: got a CPU tensor")
    if not t.is_contiguous():
        raise ValueError("libmxq buffers must be contiguous (use the leading-dimension argument for strides)")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != MXQ_OK:
        raise MxqError(status, where)


# ------------------------------------------------------------------ C entry points
def mxq_status_string(status: int) -> str:
    return lib().mxq_status_string(int(status)).decode()


def mxq_sf_bytes(rows: int, K: int) -> int:
    return int(lib().mxq_sf_bytes(int(rows), int(K)))


def mxq_quantize_act(x, M, K, ldx, fmt, rule, hadamard128, act_scale, q_out, sf_out, stream=None) -> None:
    _check(lib().mxq_quantize_act(_ptr(x), int(M), int(K), int(ldx), int(fmt), int(rule), int(bool(hadamard128)),
                                  float(act_scale), _ptr(q_out), _ptr(sf_out), _stream(stream)), "mxq_quantize_act")


def mxq_pack_weight(w, N, K, ldw, rule, hadamard128, codes_out, sf_out, stream=None) -> None:
    _check(lib().mxq_pack_weight(_ptr(w), int(N), int(K), int(ldw), int(rule), int(bool(hadamard128)),
                                 _ptr(codes_out), _ptr(sf_out), _stream(stream)), "mxq_pack_weight")


def mxq_gemm_w4a4(a_codes, a_sf, b_codes, b_sf, M, N, K, alpha, bias, d, ldd, stream=None) -> None:
    _check(lib().mxq_gemm_w4a4(_ptr(a_codes), _ptr(a_sf), _ptr(b_codes), _ptr(b_sf), int(M), int(N), int(K),
                               float(alpha), _ptr(bias), _ptr(d), int(ldd), _stream(stream)), "mxq_gemm_w4a4")


def mxq_gemm_w4a8(a_e4m3, act_scale, b_codes, b_sf, M, N, K, bias, d, ldd, stream=None) -> None:
    _check(lib().mxq_gemm_w4a8(_ptr(a_e4m3), float(act_scale), _ptr(b_codes), _ptr(b_sf), int(M), int(N), int(K),
                               _ptr(bias), _ptr(d), int(ldd), _stream(stream)), "mxq_gemm_w4a8")


def mxq_dequant_mxfp4(codes, sf, rows, K, out, ldo, stream=None) -> None:
    _check(lib().mxq_dequant_mxfp4(_ptr(codes), _ptr(sf), int(rows), int(K), _ptr(out), int(ldo), _stream(stream)),
           "mxq_dequant_mxfp4")


def mxq_qdq_act(x, M, K, ldx, fmt, rule, hadamard128, act_scale, out, ldo, stream=None) -> None:
    _check(lib().mxq_qdq_act(_ptr(x), int(M), int(K), int(ldx), int(fmt), int(rule), int(bool(hadamard128)),
                             float(act_scale), _ptr(out), int(ldo), _stream(stream)), "mxq_qdq_act")


def mxq_channel_absmax(x, rows, K, ldx, hadamard128, accumulate, amax_out, stream=None) -> None:
    _check(lib().mxq_channel_absmax(_ptr(x), int(rows), int(K), int(ldx), int(bool(hadamard128)),
                                    int(bool(accumulate)), _ptr(amax_out), _stream(stream)), "mxq_channel_absmax")


def mxq_smooth_factors(amax_x, amax_w, K, alpha, lambda_out, inv_lambda_out, stream=None) -> None:
    _check(lib().mxq_smooth_factors(_ptr(amax_x), _ptr(amax_w), int(K), float(alpha), _ptr(lambda_out),
                                    _ptr(inv_lambda_out), _stream(stream)), "mxq_smooth_factors")


def mxq_quantize_smooth(x, rows, K, ldx, rule, hadamard128, chan_scale, codes_out, sf_out, stream=None) -> None:
    _check(lib().mxq_quantize_smooth(_ptr(x), int(rows), int(K), int(ldx), int(rule), int(bool(hadamard128)),
                                     _ptr(chan_scale), _ptr(codes_out), _ptr(sf_out), _stream(stream)),
           "mxq_quantize_smooth")


def mxq_sqnr_accumulate(y, ldy, ref, ldr, M, N, accumulate, acc, stream=None) -> None:
    _check(lib().mxq_sqnr_accumulate(_ptr(y), int(ldy), _ptr(ref), int(ldr), int(M), int(N), int(bool(accumulate)),
                                     _ptr(acc), _stream(stream)), "mxq_sqnr_accumulate")


def mxq_sqnr_db(signal: float, noise: float) -> float:
    return float(lib().mxq_sqnr_db(float(signal), float(noise)))


def mxq_select_precision(sqnr_plain_db: float, sqnr_transform_db: float, high_db: float, low_db: float) -> int:
    return int(lib().mxq_select_precision(float(sqnr_plain_db), float(sqnr_transform_db), float(high_db),
                                          float(low_db)))


def mxq_attn_padded_keys(S_kv: int) -> int:
    return int(lib().mxq_attn_padded_keys(int(S_kv)))


def mxq_attn_code_poly() -> list[float]:
    """{1, a1, a2, a3}: the FP32 cubic the attention kernel decides the numerators' codes with."""
    c = (ctypes.c_float * 4)()
    lib().mxq_attn_code_poly(c)
    return [float(x) for x in c]


def mxq_quantize_vt(v, S, HD, ldv, rule, codes_out, sf_out, stream=None) -> None:
    _check(lib().mxq_quantize_vt(_ptr(v), int(S), int(HD), int(ldv), int(rule), _ptr(codes_out), _ptr(sf_out),
                                 _stream(stream)), "mxq_quantize_vt")


def mxq_attention_mxfp4(q_codes, q_sf, k_codes, k_sf, vt_codes, vt_sf, S_q, S_kv, H, d, rule, out, ldo,
                        stream=None) -> None:
    _check(lib().mxq_attention_mxfp4(_ptr(q_codes), _ptr(q_sf), _ptr(k_codes), _ptr(k_sf), _ptr(vt_codes),
                                     _ptr(vt_sf), int(S_q), int(S_kv), int(H), int(d), int(rule), _ptr(out),
                                     int(ldo), _stream(stream)), "mxq_attention_mxfp4")


def mxq_qk_norm_rope(cfg: NormRope, T, d, q, Hq, ldq, q_out, ldqo, k, Hk, ldk, k_out, ldko, positions,
                     stream=None) -> None:
    _check(lib().mxq_qk_norm_rope(ctypes.byref(cfg), T, d, _ptr(q), Hq, ldq, _ptr(q_out), ldqo, _ptr(k), Hk, ldk,
                                  _ptr(k_out), ldko, _ptr(positions), _stream(stream)), "mxq_qk_norm_rope")


def mxq_kv_append(cfg: NormRope, cache: PagedKVArgs, batch: PagedBatchArgs, T, k, ldk, v, ldv, q, Hq, ldq, q_out, ldqo,
                  stream=None) -> None:
    _check(lib().mxq_kv_append(ctypes.byref(cfg), ctypes.byref(cache), ctypes.byref(batch), T, _ptr(k), ldk, _ptr(v),
                               ldv, _ptr(q), Hq, ldq, _ptr(q_out), ldqo, _stream(stream)), "mxq_kv_append")


def mxq_attention_paged_workspace_bytes(T: int, batch: int, Hq: int, heads: int, d: int) -> int:
    return int(lib().mxq_attention_paged_workspace_bytes(T, batch, Hq, heads, d))


def mxq_attention_paged(q, T, Hq, ldq, cache: PagedKVArgs, batch: PagedBatchArgs, causal, window, scale, workspace,
                        workspace_bytes, out, ldo, stream=None) -> None:
    _check(lib().mxq_attention_paged(_ptr(q), T, Hq, ldq, ctypes.byref(cache), ctypes.byref(batch), int(bool(causal)),
                                     window, scale, _ptr(workspace), workspace_bytes, _ptr(out), ldo, _stream(stream)),
           "mxq_attention_paged")


def mxq_linear_workspace_bytes(M: int, K: int) -> int:
    return int(lib().mxq_linear_workspace_bytes(int(M), int(K)))


def mxq_linear_w4a4(x, M, K, ldx, rule, w_codes, w_sf, N, alpha, bias, workspace, workspace_bytes, d, ldd,
                    stream=None) -> None:
    _check(lib().mxq_linear_w4a4(_ptr(x), int(M), int(K), int(ldx), int(rule), _ptr(w_codes), _ptr(w_sf), int(N),
                                 float(alpha), _ptr(bias), _ptr(workspace), int(workspace_bytes), _ptr(d), int(ldd),
                                 _stream(stream)), "mxq_linear_w4a4")


def mxq_linear_w4a4_static(x, M, K, ldx, rule, w_codes, w_sf, N, alpha, bias, d, ldd, stream=None) -> None:
    _check(lib().mxq_linear_w4a4_static(_ptr(x), int(M), int(K), int(ldx), int(rule), _ptr(w_codes), _ptr(w_sf),
                                        int(N), float(alpha), _ptr(bias), _ptr(d), int(ldd), _stream(stream)),
           "mxq_linear_w4a4_static")


def mxq_debug_poll() -> int:
    return int(lib().mxq_debug_poll())


def mxq_selftest_wait_timeout(stream=None) -> None:
    _check(lib().mxq_selftest_wait_timeout(_stream(stream)), "mxq_selftest_wait_timeout")


# ------------------------------------------------------------------ allocating helpers
def _on_stream(fn):
    """Runs an allocating helper with its `stream` argument as torch's current stream.

    The caching allocator hands a freed block out again only after the work queued on the
    stream that allocated it, so tensors the helper allocates (outputs and temporaries such
    as the quantised activations of linear_w4a4) then stay valid for as long as the kernels
    the helper queued on `stream` read or write them, whatever stream the caller is on."""
    place = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        stream = args[place] if len(args) > place else kwargs.get("stream")
        if stream is None:
            return fn(*args, **kwargs)
        s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
        with torch.cuda.stream(s):
            return fn(*args, **kwargs)

    return wrapper


def _bf16_2d(x: torch.Tensor, name: str) -> torch.Tensor:
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{name}: expected a 2-D bfloat16 CUDA tensor")
    if x.stride(1) != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    _on_current_device(x, name)
    return x


def _on_current_device(x: torch.Tensor, name: str) -> None:
    """The library launches on the current CUDA device; a tensor on another device would
    be read through the wrong context, so it is refused here."""
    cur = torch.cuda.current_device()
    if x.device.index is not None and x.device.index != cur:
        raise ValueError(f"{name}: tensor on {x.device} but the current CUDA device is cuda:{cur} "
                         f"(run the call under torch.cuda.device({x.device.index}))")


@_on_stream
def quantize_act(x: torch.Tensor, rule: int = MXQ_SCALE_OCP, hadamard128: bool = False, out=None, stream=None):
    """Dynamic MXFP4 quantisation of X[M][K] -> (codes [M][K/2] uint8, sf uint8[mxq_sf_bytes(M, K)])."""
    x = _bf16_2d(x, "x")
    M, K = x.shape
    if out is None:
        out = (torch.empty(M, K // 2, dtype=torch.uint8, device=x.device),
               torch.empty(mxq_sf_bytes(M, K), dtype=torch.uint8, device=x.device))
    q, sf = out
    mxq_quantize_act(x.data_ptr(), M, K, x.stride(0), MXQ_ACT_MXFP4, rule, hadamard128, 1.0, q, sf, stream)
    return q, sf


@_on_stream
def quantize_act_fp8(x: torch.Tensor, act_scale: float, out=None, stream=None) -> torch.Tensor:
    """Static FP8 E4M3 quantisation of X[M][K] with per-tensor scale s -> uint8 [M][K]."""
    x = _bf16_2d(x, "x")
    M, K = x.shape
    q = torch.empty(M, K, dtype=torch.uint8, device=x.device) if out is None else out
    mxq_quantize_act(x.data_ptr(), M, K, x.stride(0), MXQ_ACT_FP8_E4M3, MXQ_SCALE_OCP, False, act_scale, q, None,
                     stream)
    return q


@_on_stream
def pack_weight(w: torch.Tensor, rule: int = MXQ_SCALE_OCP, hadamard128: bool = False, stream=None):
    """Offline MXFP4 packing of W[N][K] -> (codes [N][K/2] uint8, sf uint8[mxq_sf_bytes(N, K)])."""
    w = _bf16_2d(w, "w")
    N, K = w.shape
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=w.device)
    sf = torch.empty(mxq_sf_bytes(N, K), dtype=torch.uint8, device=w.device)
    mxq_pack_weight(w.data_ptr(), N, K, w.stride(0), rule, hadamard128, codes, sf, stream)
    return codes, sf


def _out_bf16(M: int, N: int, device) -> torch.Tensor:
    """[M][N] BF16 view of a buffer whose rows are padded to a multiple of 8 elements
    (the output's row stride must be a multiple of 16 bytes)."""
    ldd = (N + 7) // 8 * 8
    return torch.empty(M, ldd, dtype=torch.bfloat16, device=device)[:, :N]


@_on_stream
def gemm_w4a4(a_codes, a_sf, b_codes, b_sf, M, N, K, alpha=1.0, bias=None, out=None, stream=None) -> torch.Tensor:
    """D[M][N] (BF16) = alpha * deq(A) deq(B)^T + bias, on the tensor cores."""
    d = _out_bf16(M, N, a_codes.device) if out is None else out
    mxq_gemm_w4a4(a_codes, a_sf, b_codes, b_sf, M, N, K, alpha, bias, d.data_ptr(), d.stride(0), stream)
    return d


@_on_stream
def gemm_w4a8(a_e4m3, act_scale, b_codes, b_sf, M, N, K, bias=None, out=None, stream=None) -> torch.Tensor:
    """D[M][N] (BF16) = act_scale * e4m3(A) deq(B)^T + bias, on the tensor cores."""
    d = _out_bf16(M, N, a_e4m3.device) if out is None else out
    mxq_gemm_w4a8(a_e4m3, act_scale, b_codes, b_sf, M, N, K, bias, d.data_ptr(), d.stride(0), stream)
    return d


@_on_stream
def dequant_mxfp4(codes: torch.Tensor, sf: torch.Tensor, K: int, out=None, stream=None) -> torch.Tensor:
    """MXFP4 codes [rows][K/2] + swizzled scales -> BF16 [rows][K] (exact values)."""
    rows = codes.shape[0]
    o = _out_bf16(rows, K, codes.device) if out is None else out
    mxq_dequant_mxfp4(codes, sf, rows, K, o.data_ptr(), o.stride(0), stream)
    return o


@_on_stream
def qdq_act(x: torch.Tensor, fmt: int = MXQ_ACT_MXFP4, rule: int = MXQ_SCALE_OCP, hadamard128: bool = False,
            act_scale: float = 1.0, out=None, stream=None) -> torch.Tensor:
    """BF16 dequant(quant(X)) with the activation quantiser's arithmetic (fake quantisation)."""
    x = _bf16_2d(x, "x")
    M, K = x.shape
    o = _out_bf16(M, K, x.device) if out is None else out
    mxq_qdq_act(x.data_ptr(), M, K, x.stride(0), fmt, rule, hadamard128, act_scale, o.data_ptr(), o.stride(0),
                stream)
    return o


@_on_stream
def channel_absmax(x: torch.Tensor, hadamard128: bool = False, out=None, accumulate: bool = False,
                   stream=None) -> torch.Tensor:
    """Per-channel max |x R| over the rows (FP32 [K]); accumulate merges into `out`."""
    x = _bf16_2d(x, "x")
    rows, K = x.shape
    o = torch.empty(K, dtype=torch.float32, device=x.device) if out is None else out
    mxq_channel_absmax(x.data_ptr(), rows, K, x.stride(0), hadamard128, accumulate, o, stream)
    return o


@_on_stream
def smooth_factors(amax_x: torch.Tensor, amax_w: torch.Tensor, alpha: float = 0.5, stream=None):
    """SmoothQuant (lambda, 1/lambda) from the channel maxima of activations and weights."""
    K = amax_x.numel()
    lam = torch.empty(K, dtype=torch.float32, device=amax_x.device)
    inv = torch.empty_like(lam)
    mxq_smooth_factors(amax_x, amax_w, K, alpha, lam, inv, stream)
    return lam, inv


@_on_stream
def quantize_smooth(x: torch.Tensor, chan_scale: torch.Tensor, rule: int = MXQ_SCALE_OCP,
                    hadamard128: bool = False, out=None, stream=None):
    """MXFP4 codes + scales of (x R) * chan_scale (per channel): 1/lambda for activations,
    lambda for weights."""
    x = _bf16_2d(x, "x")
    rows, K = x.shape
    if out is None:
        out = (torch.empty(rows, K // 2, dtype=torch.uint8, device=x.device),
               torch.empty(mxq_sf_bytes(rows, K), dtype=torch.uint8, device=x.device))
    q, sf = out
    mxq_quantize_smooth(x.data_ptr(), rows, K, x.stride(0), rule, hadamard128, chan_scale, q, sf, stream)
    return q, sf


@_on_stream
def quantize_vt(v: torch.Tensor, rule: int = MXQ_SCALE_UOS, out=None, stream=None):
    """V [S][H*d] -> V^T MXFP4 (codes [H*d][Sp/2], scales) with 32-key blocks."""
    v = _bf16_2d(v, "v")
    S, HD = v.shape
    Sp = mxq_attn_padded_keys(S)
    if out is None:
        out = (torch.empty(HD, Sp // 2, dtype=torch.uint8, device=v.device),
               torch.empty(mxq_sf_bytes(HD, Sp), dtype=torch.uint8, device=v.device))
    mxq_quantize_vt(v.data_ptr(), S, HD, v.stride(0), rule, out[0], out[1], stream)
    return out


@_on_stream
def attention_mxfp4(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, H: int, rule: int = MXQ_SCALE_UOS,
                    out=None, stream=None) -> torch.Tensor:
    """MXFP4 attention with UOS / PNQ: q [Sq][H*d], k, v [Skv][H*d] BF16 -> O [Sq][H*d] BF16.
    Quantises Q, K (blocks along d) and V (blocks along the keys), then one attention launch."""
    Sq, HD = q.shape
    Skv = k.shape[0]
    d = HD // H
    qc, qs = quantize_act(q, rule, False, stream=stream)
    kc, ks = quantize_act(k, rule, False, stream=stream)
    vc, vs = quantize_vt(v, rule, stream=stream)
    o = _out_bf16(Sq, HD, q.device) if out is None else out
    mxq_attention_mxfp4(qc, qs, kc, ks, vc, vs, Sq, Skv, H, d, rule, o.data_ptr(), o.stride(0), stream)
    return o


@_on_stream
def linear_w4a4(x: torch.Tensor, w_codes, w_sf, N: int, rule: int = MXQ_SCALE_OCP, hadamard128: bool = False,
                bias=None, stream=None) -> torch.Tensor:
    """The quantized linear layer: dynamic MXFP4 quantisation of X, then the W4A4 GEMM."""
    M, K = x.shape
    q, sf = quantize_act(x, rule, hadamard128, stream=stream)
    return gemm_w4a4(q, sf, w_codes, w_sf, M, N, K, 1.0, bias, stream=stream)


def linear_workspace(M: int, K: int, device) -> torch.Tensor:
    """A workspace for linear_w4a4_ws (the quantised activations)."""
    return torch.empty(mxq_linear_workspace_bytes(M, K), dtype=torch.uint8, device=device)


@_on_stream
def linear_w4a4_ws(x: torch.Tensor, w_codes, w_sf, N: int, rule: int = MXQ_SCALE_OCP, alpha: float = 1.0,
                   bias=None, workspace=None, out=None, stream=None) -> torch.Tensor:
    """The quantized linear layer in one call of the C ABI (quantised activations in `workspace`)."""
    x = _bf16_2d(x, "x")
    M, K = x.shape
    ws = linear_workspace(M, K, x.device) if workspace is None else workspace
    d = _out_bf16(M, N, x.device) if out is None else out
    mxq_linear_w4a4(x.data_ptr(), M, K, x.stride(0), rule, w_codes, w_sf, N, alpha, bias, ws, ws.numel(),
                    d.data_ptr(), d.stride(0), stream)
    return d


@_on_stream
def linear_w4a4_static(x: torch.Tensor, w_codes, w_sf, N: int, rule: int = MXQ_SCALE_OCP, alpha: float = 1.0,
                       bias=None, out=None, stream=None) -> torch.Tensor:
    """The quantized linear layer with the library's own fixed scratch (no allocation by the call)."""
    x = _bf16_2d(x, "x")
    M, K = x.shape
    d = _out_bf16(M, N, x.device) if out is None else out
    mxq_linear_w4a4_static(x.data_ptr(), M, K, x.stride(0), rule, w_codes, w_sf, N, alpha, bias, d.data_ptr(),
                           d.stride(0), stream)
    return d


@_on_stream
def linear_w4a8(x: torch.Tensor, act_scale: float, w_codes, w_sf, N: int, bias=None, stream=None) -> torch.Tensor:
    """The W4A8 layer: static FP8 quantisation of X, then the W4A8 GEMM."""
    M, K = x.shape
    q = quantize_act_fp8(x, act_scale, stream=stream)
    return gemm_w4a8(q, act_scale, w_codes, w_sf, M, N, K, bias, stream=stream)


# ------------------------------------------------------------------ queries and keys, paged cache
def _operand(x: torch.Tensor, cur: int, name: str) -> None:
    """_bf16_2d in a few cheap checks: a generated token's whole layer is some tens of microseconds."""
    if x.dtype is not torch.bfloat16 or x.dim() != 2 or x.get_device() != cur or x.stride(1) != 1:
        _bf16_2d(x, name)


def _current(x: torch.Tensor, name: str) -> int:
    """The current device, once x is known to be on one."""
    if not x.is_cuda:
        raise ValueError(f"{name}: expected a 2-D bfloat16 CUDA tensor")
    return torch.cuda.current_device()


def _here(x: torch.Tensor, dev: int, name: str) -> None:
    """Refuses x unless it is on device `dev`, the current one or that of the tensors it belongs to."""
    if x.get_device() != dev:
        if not x.is_cuda:
            raise ValueError(f"{name}: expected a CUDA tensor")
        raise ValueError(f"{name}: tensor on {x.device}, expected one on cuda:{dev}")


def _width(x: torch.Tensor, heads: int, d: int, name: str) -> None:
    if heads < 1 or x.shape[1] != heads * d:
        raise ValueError(f"{name}: {x.shape[1]} columns are not {heads} heads of {d}")


def _int32(x: torch.Tensor, shape: tuple, cur: int, name: str) -> int:
    if x.dtype is not torch.int32 or x.shape != shape or not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 CUDA tensor of shape {shape}")
    _here(x, cur, name)
    return x.data_ptr()


def _weight(w: torch.Tensor, n: int, cur: int, name: str) -> int:
    if w.dtype is not torch.bfloat16 or w.numel() != n or not w.is_contiguous():
        raise ValueError(f"{name}: expected {n} contiguous bfloat16 values")
    _here(w, cur, name)
    return w.data_ptr()


def _norm_rope(Hq, Hk, d, q_weight, k_weight, eps, span, table, style, cur) -> NormRope:
    qw = None if q_weight is None else _weight(q_weight, Hq * d if span == MXQ_NORM_ROW else d, cur, "q_weight")
    kw = None if k_weight is None else _weight(k_weight, Hk * d if span == MXQ_NORM_ROW else d, cur, "k_weight")
    if table is None:
        return NormRope(qw, kw, None, 0, 0, eps, span, style)
    if table.dtype is not torch.float32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table: expected a contiguous float32 tensor [positions][rot]")
    _here(table, cur, "table")
    return NormRope(qw, kw, table.data_ptr(), *table.shape, eps, span, style)


def rope_table(positions: int | torch.Tensor, rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """FP32 [positions][rot]: cos, then sin, of position * base^(-2 i / rot), the angles in 64 bits.
    `positions`: how many (0, 1, 2, ...), or a 1-D tensor of positions (one row of the table each)."""
    pos = torch.arange(positions, device=device) if isinstance(positions, int) else positions.to(device)
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = pos.to(torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)


class PagedKV:
    """A paged key / value cache: k and v [pages][page_size][heads][d], BF16 or E4M3 (float8_e4m3fn or
    uint8), with contiguous heads; other orders of the dimensions are views with other strides.
    k_scale, v_scale: static scales of an E4M3 cache."""

    __slots__ = ("k", "v", "args")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0):
        shape, strides, dtype = k.shape, k.stride(), k.dtype
        if len(shape) != 4 or v.shape != shape or v.stride() != strides or v.dtype is not dtype:
            raise ValueError("k, v: expected two [pages][page_size][heads][d] tensors alike in shape, strides and type")
        if dtype is torch.bfloat16:
            fmt = MXQ_KV_BF16
        elif dtype is torch.float8_e4m3fn or dtype is torch.uint8:
            fmt = MXQ_KV_FP8_E4M3
        else:
            raise ValueError("k, v: expected bfloat16, float8_e4m3fn or uint8")
        if not k.is_cuda or v.get_device() != k.get_device() or strides[3] != 1:
            raise ValueError("k, v: expected CUDA tensors of one device, with contiguous heads")
        self.k, self.v = k, v
        self.args = PagedKVArgs(k.data_ptr(), v.data_ptr(), *shape, strides[0], strides[1], strides[2], fmt, k_scale,
                                v_scale)


def paged_kv(pages: int, page_size: int, heads: int, d: int, fmt: int = MXQ_KV_BF16, k_scale: float = 1.0,
             v_scale: float = 1.0, device="cuda") -> PagedKV:
    """Allocates a cache (its contents are undefined until tokens are appended)."""
    dtype = torch.bfloat16 if fmt == MXQ_KV_BF16 else torch.float8_e4m3fn
    k, v = (torch.empty(pages, page_size, heads, d, dtype=dtype, device=device) for _ in range(2))
    return PagedKV(k, v, k_scale, v_scale)


class PagedBatch:
    """The sequences of a call: cu_q [batch + 1], kv_len [batch] and block_table [batch][max_pages], int32 on
    one GPU (see mxq_paged_batch).  Holds the tensors: their contents may change between calls."""

    __slots__ = ("cu_q", "kv_len", "block_table", "args")

    def __init__(self, cu_q: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor):
        if block_table.dim() != 2:
            raise ValueError("block_table: expected [batch][max_pages]")
        batch, max_pages = block_table.shape
        dev = cu_q.get_device()  # the others are on it too: a call checks cu_q alone
        self.args = PagedBatchArgs(_int32(cu_q, (batch + 1,), dev, "cu_q"), _int32(kv_len, (batch,), dev, "kv_len"),
                                   _int32(block_table, (batch, max_pages), dev, "block_table"), batch, max_pages)
        self.cu_q, self.kv_len, self.block_table = cu_q, kv_len, block_table


def _out_heads(out, x: torch.Tensor, cur: int, name: str) -> torch.Tensor:
    if out is None:
        return torch.empty_like(x)
    _operand(out, cur, name)
    if out.shape != x.shape:
        raise ValueError(f"{name}: expected shape {tuple(x.shape)}")
    return out


@_on_stream
def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, Hq: int, Hk: int, q_weight=None, k_weight=None, eps: float = 1e-6,
                 span: int = MXQ_NORM_HEAD, table=None, positions=None, style: int = MXQ_ROPE_HALVES, q_out=None,
                 k_out=None, stream=None):
    """Norm (where weights are given) and rotation (where a table is given) of q [T][Hq*d] and k
    [T][Hk*d] -> (q_out, k_out).  positions: int32 [T], or None for 0, 1, 2, ...; a row whose position is
    outside the table is not written.  q_out=q, k_out=k work in place."""
    cur = _current(q, "q")
    _operand(q, cur, "q")
    _operand(k, cur, "k")
    T = q.shape[0]
    d = q.shape[1] // Hq if Hq > 0 else 0
    _width(q, Hq, d, "q")
    _width(k, Hk, d, "k")
    if k.shape[0] != T:
        raise ValueError("q, k: expected the same number of rows")
    cfg = _norm_rope(Hq, Hk, d, q_weight, k_weight, eps, span, table, style, cur)
    pos = None if positions is None else _int32(positions, (T,), cur, "positions")
    qo, ko = _out_heads(q_out, q, cur, "q_out"), _out_heads(k_out, k, cur, "k_out")
    mxq_qk_norm_rope(cfg, T, d, q.data_ptr(), Hq, q.stride(0), qo.data_ptr(), qo.stride(0), k.data_ptr(), Hk,
                     k.stride(0), ko.data_ptr(), ko.stride(0), pos, stream)
    return qo, ko


@_on_stream
def kv_append(k: torch.Tensor, v: torch.Tensor, cache: PagedKV, batch: PagedBatch, k_weight=None, eps: float = 1e-6,
              span: int = MXQ_NORM_HEAD, table=None, style: int = MXQ_ROPE_HALVES, q=None, q_weight=None, q_out=None,
              stream=None):
    """Norm and rotation of the new keys k [T][heads*d] at their sequences' positions, keys and values
    into the cache; with q [T][Hq*d] also its norm and rotation -> q_out (else None)."""
    cur = _current(k, "k")
    a = cache.args
    d, heads, T = a.d, a.heads, k.shape[0]
    _operand(k, cur, "k")
    _operand(v, cur, "v")
    _width(k, heads, d, "k")
    _width(v, heads, d, "v")
    _here(cache.k, cur, "cache")
    _here(batch.cu_q, cur, "batch")
    if v.shape[0] != T or (q is not None and q.shape[0] != T):
        raise ValueError("k, v, q: expected the same number of rows")
    if q is None:
        cfg = _norm_rope(0, heads, d, None, k_weight, eps, span, table, style, cur)
        mxq_kv_append(cfg, a, batch.args, T, k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0), None, 0, 0, None, 0,
                      stream)
        return None
    _operand(q, cur, "q")
    Hq = q.shape[1] // d
    _width(q, Hq, d, "q")
    cfg = _norm_rope(Hq, heads, d, q_weight, k_weight, eps, span, table, style, cur)
    qo = _out_heads(q_out, q, cur, "q_out")
    mxq_kv_append(cfg, a, batch.args, T, k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0), q.data_ptr(), Hq,
                  q.stride(0), qo.data_ptr(), qo.stride(0), stream)
    return qo


def attention_paged_workspace(T: int, batch: int, Hq: int, heads: int, d: int, device) -> torch.Tensor:
    """A workspace for attention_paged."""
    n = mxq_attention_paged_workspace_bytes(T, batch, Hq, heads, d)
    if n < 0:
        raise ValueError("attention_paged_workspace: invalid sizes (d 64 or 128, Hq a multiple of heads)")
    return torch.empty(n, dtype=torch.uint8, device=device)


@_on_stream
def attention_paged(q: torch.Tensor, Hq: int, cache: PagedKV, batch: PagedBatch, causal: bool = True, window: int = 0,
                    scale: float | None = None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of the new tokens' queries q [T][Hq*d] over their sequences' cached keys and values
    -> O [T][Hq*d] BF16.  scale: d^-1/2 by default.  Rows of no sequence are not written."""
    cur = _current(q, "q")
    a, b = cache.args, batch.args
    d, T = a.d, q.shape[0]
    _operand(q, cur, "q")
    _width(q, Hq, d, "q")
    _here(cache.k, cur, "cache")
    _here(batch.cu_q, cur, "batch")
    if workspace is None:
        workspace = attention_paged_workspace(T, b.batch, Hq, a.heads, d, q.device)
    else:
        _here(workspace, cur, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace: expected a contiguous tensor")
    o = _out_heads(out, q, cur, "out")
    mxq_attention_paged(q.data_ptr(), T, Hq, q.stride(0), a, b, causal, window, d ** -0.5 if scale is None else scale,
                        workspace, workspace.numel() * workspace.element_size(), o.data_ptr(), o.stride(0), stream)
    return o
