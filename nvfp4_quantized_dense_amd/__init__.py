"""MI355X-native NVFP4 dense MLP: Python binding of libnvfp4_mi355x.so.

Argument marshalling only: every step of the path runs in the HIP library
(include/nvfp4.h). PyTorch supplies device memory (tensors) and the stream
(the current torch stream unless one is given). The library must have been
built (``python -m nvfp4_quantized_dense_amd.build``); importing this module
without it fails loudly, there is no other implementation.
"""
import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4_mi355x.so")

NVFP4_OK = 0
NVFP4_ERR_INVALID_ARG = -1
NVFP4_ERR_UNSUPPORTED = -2
NVFP4_ERR_HIP = -3
DTYPE_BF16, DTYPE_F32 = 0, 1
MODE_W4A4, MODE_W4A16, MODE_W4A4_DYN, MODE_W4A16_AWQ = 0, 1, 2, 3
REPACK_PLAIN, REPACK_SWIGLU = 0, 1
ROPE_HALVES, ROPE_NEIGHBOURS = 0, 1
ROPE_AXES = 16  # at most
POOL_NO_PAGES, POOL_NO_TABLE, POOL_NO_ROWS = 1, 2, 4
PATH_AUTO, PATH_GEMV, PATH_STREAM, PATH_TILED, PATH_TILED64, PATH_MID = 0, 1, 2, 3, 4, 5

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_sz = ctypes.c_size_t
_f32 = ctypes.c_float
_f64 = ctypes.c_double

# name -> (restype, argtypes); the exported C ABI.
SIGNATURES = {
    "nvfp4_last_error": (ctypes.c_char_p, []),
    "nvfp4_set_path": (_int, [_int]),
    "nvfp4_calibrate": (_int, [_vp, _int, _i64, _vp, _vp, _vp]),
    "nvfp4_quantize": (_int, [_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp]),
    "nvfp4_quantize_per_token": (_int, [_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp]),
    "nvfp4_repack_bytes": (_sz, [_int, _i64, _i64]),
    "nvfp4_packed_bytes": (_sz, [_int, _i64, _i64]),
    "nvfp4_repack_weight": (_int, [_int, _vp, _vp, _i64, _i64, _vp, _vp]),
    "nvfp4_unpack_weight": (_int, [_int, _vp, _i64, _i64, _vp, _vp, _vp]),
    "nvfp4_gemm": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _int, _vp]),
    "gemm_swiglu_nvfp4_quant": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "nvfp4_gemm_rowscale": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _int, _vp]),
    "gemm_swiglu_nvfp4_quant_rowscale": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp,
                                                _vp, _vp]),
    "gemm_swiglu": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _int, _vp]),
    "silu_mul_nvfp4_quant": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "nvfp4_prescale_bf16": (_int, [_vp, _vp, _i64, _i64, _vp, _vp]),
    "mlp_forward_w4a16_awq": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _int,
                                     _vp]),
    "nvfp4_grouped_gemm": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _int, _vp]),
    "mlp_workspace_bytes": (_sz, [_int, _i64, _i64, _i64]),
    "mlp_workspace_status": (_vp, [_vp, _sz]),
    "nvfp4_set_decode_wait_test": (_int, [_int, _int]),
    "mlp_forward": (_int, [_int, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                           _vp, _int, _vp]),
    "add_rmsnorm_nvfp4_quant": (_int, [_vp, _int, _vp, _int, _vp, _int, _f64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "add_rmsnorm_nvfp4_quant_per_token": (_int, [_vp, _int, _vp, _int, _vp, _int, _f64, _i64, _i64, _vp, _vp, _vp, _vp,
                                                 _vp]),
    "nvfp4_dequantize": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _int, _vp]),
    "nvfp4_kv_cache_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "nvfp4_kv_write": (_int, [_vp, _vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp]),
    "nvfp4_kv_read": (_int, [_vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _int, _vp]),
    "nvfp4_kv_attention_workspace_bytes": (_sz, [_i64] * 7),
    "nvfp4_kv_attention": (_int, [_vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _vp,
                                  _i64, _f32, _i64, _vp, _vp, _vp, _sz, _vp, _int, _vp, _vp]),
    "nvfp4_kv_pool_bytes": (_sz, [_i64]),
    "nvfp4_kv_pool_reset": (_int, [_vp, _i64, _vp]),
    "nvfp4_kv_advance": (_int, [_vp, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "nvfp4_rope": (_int, [_vp, _int, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _int, _f64, _vp, _int, _i64, _vp]),
    "nvfp4_rope_kv_write": (_int, [_vp, _i64, _i64, _vp, _vp, _int, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _int, _f64,
                                   _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _int, _i64, _vp]),
    "nvfp4_tree_mask": (_int, [_vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp]),
    "nvfp4_kv_attention_masked": (_int, [_vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _vp,
                                         _i64, _f32, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp, _int, _vp, _vp]),
    "mlp_forward_noalloc": (_int, [_int, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _vp]),
}

_LIB = None


def lib():
    """The loaded C library (ctypes.CDLL) with typed entry points."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build the HIP library first "
                "(python -m nvfp4_quantized_dense_amd.build); there is no fallback path")
        cdll = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(cdll, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = cdll
    return _LIB


class Nvfp4Error(RuntimeError):
    def __init__(self, name, code, msg):
        super().__init__(f"{name} failed ({code}): {msg}")
        self.code = code


def _check(name, code):
    if code != NVFP4_OK:
        raise Nvfp4Error(name, code, lib().nvfp4_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


_gpu = False  # a GPU has been seen: it does not go away


def _stream(stream):
    """The stream's handle. The current one is asked for without building a Stream object (0.1 us, not 3.5)."""
    global _gpu
    if stream is None:
        if not _gpu:
            if not torch.cuda.is_available():
                return None
            torch.cuda.init()
            _gpu = True
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on(stream):
    """Context in which torch allocates and fills what a call on `stream` uses: on the stream itself, so that the
    kernel comes after the fill, and the memory, once released, goes to work that comes after the kernel."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


_F32 = torch.float32
_DTYPE_CODES = {torch.bfloat16: DTYPE_BF16, _F32: DTYPE_F32}


def _dtype_code(dt):
    code = _DTYPE_CODES.get(dt)
    if code is None:
        raise ValueError(f"unsupported dtype {dt}")
    return code


def _dense(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def set_path(path: int) -> int:
    prev = lib().nvfp4_set_path(int(path))
    if prev < 0:
        _check("nvfp4_set_path", prev)
    return prev


def nvfp4_calibrate(x, g=None, g_inv=None, stream=None):
    """(g, g_inv): 1-element fp32 device tensors with g = amax(|x|)/2688."""
    _dense(x, "x")
    g = torch.empty(1, dtype=torch.float32, device=x.device) if g is None else g
    g_inv = torch.empty(1, dtype=torch.float32, device=x.device) if g_inv is None else g_inv
    _check("nvfp4_calibrate", lib().nvfp4_calibrate(_ptr(x), _dtype_code(x.dtype), x.numel(),
                                                    _ptr(g), _ptr(g_inv), _stream(stream)))
    return g, g_inv


def nvfp4_quantize(x, g_inv, codes=None, scales=None, stream=None):
    """x [M, K] bf16/f32 -> (codes uint8 [M, K/2], scales uint8 [M, K/16])."""
    _dense(x, "x")
    M, K = x.shape
    if codes is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((M, K // 16), dtype=torch.uint8, device=x.device)
    _check("nvfp4_quantize", lib().nvfp4_quantize(_ptr(x), _dtype_code(x.dtype), M, K, _ptr(g_inv),
                                                  _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def nvfp4_quantize_per_token(x, codes=None, scales=None, row_g=None, stream=None):
    """x [M, K] bf16/f32 -> (codes [M, K/2], scales [M, K/16], row_g fp32 [M]), each row
    quantized with its own global scale row_g[t] = amax(|x[t]|)/2688."""
    _dense(x, "x")
    M, K = x.shape
    if codes is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((M, K // 16), dtype=torch.uint8, device=x.device)
    if row_g is None:
        row_g = torch.empty(M, dtype=torch.float32, device=x.device)
    _check("nvfp4_quantize_per_token",
           lib().nvfp4_quantize_per_token(_ptr(x), _dtype_code(x.dtype), M, K, _ptr(codes), _ptr(scales),
                                          _ptr(row_g), _stream(stream)))
    return codes, scales, row_g


def nvfp4_repack_bytes(kind, R, C) -> int:
    return int(lib().nvfp4_repack_bytes(int(kind), int(R), int(C)))


nvfp4_packed_bytes = nvfp4_repack_bytes


def nvfp4_repack_weight(kind, codes, scales, packed=None, stream=None):
    """Canonical NVFP4 weight (codes [R, C/2], scales [R, C/16]) -> packed uint8."""
    _dense(codes, "codes"); _dense(scales, "scales")
    R, C = codes.shape[0], codes.shape[1] * 2
    nbytes = nvfp4_repack_bytes(kind, R, C)
    if packed is None:
        packed = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=codes.device)
    _check("nvfp4_repack_weight", lib().nvfp4_repack_weight(int(kind), _ptr(codes), _ptr(scales), R, C,
                                                            _ptr(packed), _stream(stream)))
    return packed


def nvfp4_unpack_weight(kind, packed, R, C, stream=None):
    codes = torch.empty((R, C // 2), dtype=torch.uint8, device=packed.device)
    scales = torch.empty((R, C // 16), dtype=torch.uint8, device=packed.device)
    _check("nvfp4_unpack_weight", lib().nvfp4_unpack_weight(int(kind), _ptr(packed), R, C, _ptr(codes),
                                                            _ptr(scales), _stream(stream)))
    return codes, scales


def nvfp4_gemm(mode, a, a_scales, w_packed, N, K, alpha, out=None, out_dtype=torch.float32,
               stream=None):
    """out [M, N] = alpha * A @ W^T. W4A4: a = codes [M, K/2] + a_scales; W4A16: a = bf16 [M, K]."""
    _dense(a, "a")
    M = a.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _check("nvfp4_gemm", lib().nvfp4_gemm(int(mode), _ptr(a), _ptr(a_scales), _ptr(w_packed), M, N, K,
                                          _ptr(alpha), _ptr(out), _dtype_code(out.dtype),
                                          _stream(stream)))
    return out


def gemm_swiglu_nvfp4_quant(a_codes, a_scales, w_gu_packed, I, K, alpha, g2_inv, h_codes=None,
                            h_scales=None, stream=None):
    """Fused gate_up GEMM + SiLU(gate)*up + NVFP4 quantize -> (h_codes, h_scales)."""
    _dense(a_codes, "a_codes")
    M = a_codes.shape[0]
    if h_codes is None:
        h_codes = torch.empty((M, I // 2), dtype=torch.uint8, device=a_codes.device)
    if h_scales is None:
        h_scales = torch.empty((M, I // 16), dtype=torch.uint8, device=a_codes.device)
    _check("gemm_swiglu_nvfp4_quant",
           lib().gemm_swiglu_nvfp4_quant(_ptr(a_codes), _ptr(a_scales), _ptr(w_gu_packed), M, I, K,
                                         _ptr(alpha), _ptr(g2_inv), _ptr(h_codes), _ptr(h_scales),
                                         _stream(stream)))
    return h_codes, h_scales


def nvfp4_gemm_rowscale(a_codes, a_scales, row_g, w_packed, N, K, g_w, out=None,
                        out_dtype=torch.float32, stream=None):
    """W4A4 out [M, N] = g_w * row_g[t] * (A @ W^T) with per-token activation scales."""
    _dense(a_codes, "a_codes")
    M = a_codes.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a_codes.device)
    _check("nvfp4_gemm_rowscale",
           lib().nvfp4_gemm_rowscale(_ptr(a_codes), _ptr(a_scales), _ptr(row_g), _ptr(w_packed), M, N, K,
                                     _ptr(g_w), _ptr(out), _dtype_code(out.dtype), _stream(stream)))
    return out


def gemm_swiglu_nvfp4_quant_rowscale(a_codes, a_scales, row_g, w_gu_packed, I, K, g_w, g2_inv,
                                     h_codes=None, h_scales=None, stream=None):
    """gemm_swiglu_nvfp4_quant with per-token activation scales row_g."""
    _dense(a_codes, "a_codes")
    M = a_codes.shape[0]
    if h_codes is None:
        h_codes = torch.empty((M, I // 2), dtype=torch.uint8, device=a_codes.device)
    if h_scales is None:
        h_scales = torch.empty((M, I // 16), dtype=torch.uint8, device=a_codes.device)
    _check("gemm_swiglu_nvfp4_quant_rowscale",
           lib().gemm_swiglu_nvfp4_quant_rowscale(_ptr(a_codes), _ptr(a_scales), _ptr(row_g), _ptr(w_gu_packed),
                                                  M, I, K, _ptr(g_w), _ptr(g2_inv), _ptr(h_codes),
                                                  _ptr(h_scales), _stream(stream)))
    return h_codes, h_scales


def gemm_swiglu(mode, a, a_scales, w_gu_packed, I, K, alpha, h=None, h_dtype=torch.bfloat16,
                stream=None):
    """gate_up GEMM + SiLU(gate)*up -> h [M, I] (bf16 or f32)."""
    _dense(a, "a")
    M = a.shape[0]
    if h is None:
        h = torch.empty((M, I), dtype=h_dtype, device=a.device)
    _check("gemm_swiglu", lib().gemm_swiglu(int(mode), _ptr(a), _ptr(a_scales), _ptr(w_gu_packed), M, I, K,
                                            _ptr(alpha), _ptr(h), _dtype_code(h.dtype), _stream(stream)))
    return h


def silu_mul_nvfp4_quant(gate_up, g_inv, masked_m=None, codes=None, scales=None, stream=None):
    """gate_up bf16 [E, M, 2I] (or [M, 2I] as one expert) -> (codes [E, M, I/2],
    scales [E, M, I/16]) of SiLU(gate) * up, expert e quantized with g_inv[e];
    rows t >= masked_m[e] (int32 device tensor [E]) are not written."""
    _dense(gate_up, "gate_up")
    gu = gate_up if gate_up.dim() == 3 else gate_up.unsqueeze(0)
    E, M, I2 = gu.shape
    I = I2 // 2
    # The caller's outputs are of the current stream; the kernel's is the one that clears them.
    if codes is None:
        codes = torch.empty((E, M, I // 2), dtype=torch.uint8, device=gu.device)
        with _on(stream):
            codes.zero_()
    if scales is None:
        scales = torch.empty((E, M, I // 16), dtype=torch.uint8, device=gu.device)
        with _on(stream):
            scales.zero_()
    _check("silu_mul_nvfp4_quant",
           lib().silu_mul_nvfp4_quant(_ptr(gu), E, M, I, _ptr(masked_m), _ptr(g_inv), _ptr(codes), _ptr(scales),
                                      _stream(stream)))
    return codes, scales


def mlp_workspace_bytes(mode, M, H, I) -> int:
    return int(lib().mlp_workspace_bytes(int(mode), int(M), int(H), int(I)))


STATUS_DECODE_WAIT_EXPIRED = 1


def mlp_workspace_status(ws):
    """The workspace's status word as a 1-element int32 view of ws (its last
    4 bytes, the address the library computes)."""
    n = ws.numel() * ws.element_size()
    addr = lib().mlp_workspace_status(_ptr(ws), n)
    if not addr:
        raise ValueError("workspace too small for a status word")
    off = addr - ws.data_ptr()
    return ws.view(torch.uint8)[off:off + 4].view(torch.int32)


def set_decode_wait_test(withhold: bool, spin_limit: int = 0):
    """Test hook: the calling thread's single-launch decodes withhold their
    records, so every bounded wait gives up after spin_limit polls."""
    _check("nvfp4_set_decode_wait_test", lib().nvfp4_set_decode_wait_test(int(bool(withhold)), int(spin_limit)))


def mlp_forward(mode, x, w_gu_packed, alpha_gu, w_d_packed, alpha_d, I, g1_inv=None, g2_inv=None,
                ws=None, out=None, out_dtype=torch.float32, stream=None):
    """Dense MLP forward: x bf16 [M, H] -> out [M, H]."""
    _dense(x, "x")
    M, H = x.shape
    nws = mlp_workspace_bytes(mode, M, H, I)
    if ws is None:
        with _on(stream):
            ws = torch.zeros(max(nws, 1), dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((M, H), dtype=out_dtype, device=x.device)
    _check("mlp_forward", lib().mlp_forward(int(mode), _ptr(x), M, H, I, _ptr(w_gu_packed), _ptr(alpha_gu),
                                            _ptr(w_d_packed), _ptr(alpha_d), _ptr(g1_inv), _ptr(g2_inv),
                                            _ptr(ws), ws.numel() * ws.element_size(), _ptr(out),
                                            _dtype_code(out.dtype), _stream(stream)))
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20


def mlp_forward_noalloc(mode, x, w_gu_packed, alpha_gu, w_d_packed, alpha_d, I, g1_inv=None, g2_inv=None,
                        out=None, out_dtype=torch.float32, stream=None):
    """mlp_forward on the library's own per-GPU scratch (no workspace
    argument; the library allocates nothing). Pass `out` to allocate nothing
    here either. Calls that overlap on one GPU race."""
    _dense(x, "x")
    M, H = x.shape
    if out is None:
        out = torch.empty((M, H), dtype=out_dtype, device=x.device)
    _check("mlp_forward_noalloc",
           lib().mlp_forward_noalloc(int(mode), _ptr(x), M, H, I, _ptr(w_gu_packed), _ptr(alpha_gu), _ptr(w_d_packed),
                                     _ptr(alpha_d), _ptr(g1_inv), _ptr(g2_inv), _ptr(out), _dtype_code(out.dtype),
                                     _stream(stream)))
    return out


def nvfp4_prescale_bf16(x, s, out=None, stream=None):
    """AWQ pre-quant scaling: bf16(x * s) per input channel; x bf16 [M, K], s bf16 [K]."""
    _dense(x, "x"); _dense(s, "s")
    M, K = x.shape
    if out is None:
        out = torch.empty_like(x)
    _check("nvfp4_prescale_bf16", lib().nvfp4_prescale_bf16(_ptr(x), _ptr(s), M, K, _ptr(out), _stream(stream)))
    return out


def mlp_forward_w4a16_awq(x, w_gu_packed, g_gu, s_gu, w_d_packed, g_d, s_d, I, ws=None, out=None,
                          out_dtype=torch.float32, stream=None):
    """W4A16 MLP forward with AWQ pre-quant scales s_gu [H] and s_d [I] (bf16)."""
    _dense(x, "x")
    M, H = x.shape
    nws = mlp_workspace_bytes(MODE_W4A16_AWQ, M, H, I)
    if ws is None:
        with _on(stream):
            ws = torch.zeros(max(nws, 1), dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((M, H), dtype=out_dtype, device=x.device)
    _check("mlp_forward_w4a16_awq",
           lib().mlp_forward_w4a16_awq(_ptr(x), M, H, I, _ptr(w_gu_packed), _ptr(g_gu), _ptr(s_gu), _ptr(w_d_packed),
                                       _ptr(g_d), _ptr(s_d), _ptr(ws), ws.numel() * ws.element_size(), _ptr(out),
                                       _dtype_code(out.dtype), _stream(stream)))
    return out


def nvfp4_grouped_gemm(mode, a, a_scales, w_packed, N, K, alpha, masked_m=None, out=None, out_dtype=torch.float32,
                       stream=None):
    """Grouped (expert) GEMM: a [E, M, K/2] codes (+ a_scales [E, M, K/16]) or
    bf16 [E, M, K]; w_packed: E packed [N, K] weights back to back; alpha [E];
    masked_m int32 [E] or None. Returns out [E, M, N] (rows past masked_m
    keep what out held)."""
    _dense(a, "a")
    E, M = a.shape[0], a.shape[1]
    if out is None:
        out = torch.empty((E, M, N), dtype=out_dtype, device=a.device)
    _check("nvfp4_grouped_gemm",
           lib().nvfp4_grouped_gemm(int(mode), _ptr(a), _ptr(a_scales), _ptr(w_packed), E, M, N, K, _ptr(masked_m),
                                    _ptr(alpha), _ptr(out), _dtype_code(out.dtype), _stream(stream)))
    return out


def _scalar(t, name):
    """The address of a global scale, which the kernels read as one fp32 number."""
    if t.dtype is not _F32 or t.numel() != 1:
        raise ValueError(f"{name} must be one fp32 number")
    return t.data_ptr()


def _not_on_gpu():
    raise ValueError("all tensors must be on the GPU")


def _norm_outputs(x, w, residual, residual_out, codes, scales):
    M, K = x.shape
    if w.numel() != K:
        raise ValueError(f"w must have {K} elements")
    z = x if residual is None else residual
    if residual is not None and residual.shape != x.shape:
        raise ValueError("residual must have x's shape")
    if residual_out is None:
        residual_out = torch.empty_like(z)
    elif residual_out.shape != x.shape or residual_out.dtype != z.dtype:
        raise ValueError("residual_out must have the residual's shape and type")
    if not (x.is_contiguous() and w.is_contiguous() and z.is_contiguous() and residual_out.is_contiguous()):
        raise ValueError("x, w, residual and residual_out must be contiguous")
    if codes is None:
        codes = torch.empty(M, K // 2, dtype=torch.uint8, device=x.device)
    elif codes.nbytes != M * (K // 2) or not codes.is_contiguous():
        raise ValueError(f"codes must be contiguous, uint8 [{M}, {K // 2}]")
    if scales is None:
        scales = torch.empty(M, K // 16, dtype=torch.uint8, device=x.device)
    elif scales.nbytes != M * (K // 16) or not scales.is_contiguous():
        raise ValueError(f"scales must be contiguous, uint8 [{M}, {K // 16}]")
    if not (x.is_cuda and w.is_cuda and z.is_cuda and residual_out.is_cuda and codes.is_cuda and scales.is_cuda):
        _not_on_gpu()
    return M, K, _dtype_code(z.dtype), residual_out, codes, scales


def add_rmsnorm_nvfp4_quant(x, w, g_inv, residual=None, eps=1e-6, residual_out=None, codes=None, scales=None, stream=None):
    """z = x + residual, y = RMSnorm(z) * w, NVFP4(y) with g_inv: x [M, K] and residual bf16 or f32
    (residual None: z = x), w [K] -> (codes [M, K/2], scales [M, K/16], z). residual_out may be residual."""
    g = _scalar(g_inv, "g_inv")
    M, K, rd, residual_out, codes, scales = _norm_outputs(x, w, residual, residual_out, codes, scales)
    if not g_inv.is_cuda:
        _not_on_gpu()
    _check("add_rmsnorm_nvfp4_quant",
           lib().add_rmsnorm_nvfp4_quant(x.data_ptr(), _dtype_code(x.dtype), _ptr(residual), rd, w.data_ptr(),
                                         _dtype_code(w.dtype), eps, M, K, g, residual_out.data_ptr(),
                                         codes.data_ptr(), scales.data_ptr(), _stream(stream)))
    return codes, scales, residual_out


def add_rmsnorm_nvfp4_quant_per_token(x, w, residual=None, eps=1e-6, residual_out=None, codes=None, scales=None,
                                      row_g=None, stream=None):
    """add_rmsnorm_nvfp4_quant with each row's own global scale -> (codes, scales, z, row_g fp32 [M])."""
    if row_g is None:
        row_g = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    elif row_g.numel() != x.shape[0] or row_g.dtype != torch.float32 or not row_g.is_contiguous():
        raise ValueError(f"row_g must be contiguous, fp32 [{x.shape[0]}]")
    M, K, rd, residual_out, codes, scales = _norm_outputs(x, w, residual, residual_out, codes, scales)
    if not row_g.is_cuda:
        _not_on_gpu()
    _check("add_rmsnorm_nvfp4_quant_per_token",
           lib().add_rmsnorm_nvfp4_quant_per_token(x.data_ptr(), _dtype_code(x.dtype), _ptr(residual), rd, w.data_ptr(),
                                                   _dtype_code(w.dtype), eps, M, K, residual_out.data_ptr(),
                                                   codes.data_ptr(), scales.data_ptr(), row_g.data_ptr(), _stream(stream)))
    return codes, scales, residual_out, row_g


def nvfp4_dequantize(codes, scales, g=None, row_g=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """The numbers of codes [M, K/2] and scales [M, K/16] under the global scale g (1 element) or row_g [M]."""
    _dense(codes, "codes"); _dense(scales, "scales")
    M, K = codes.shape
    K *= 2
    if out is None:
        out = torch.empty(M, K, dtype=out_dtype, device=codes.device)
    elif out.numel() != M * K or not out.is_contiguous():
        raise ValueError(f"out must be contiguous, [{M}, {K}]")
    if codes.element_size() != 1 or scales.element_size() != 1 or scales.numel() * 16 != M * K:
        raise ValueError(f"scales must be [{M}, {K // 16}], a byte each as codes")
    g_at = None if g is None else _scalar(g, "g")
    if row_g is not None and (row_g.dtype is not _F32 or row_g.numel() != M or not row_g.is_contiguous()):
        raise ValueError(f"row_g must be contiguous, fp32 [{M}]")
    if not (codes.is_cuda and scales.is_cuda and out.is_cuda and (g is None or g.is_cuda) and (row_g is None or row_g.is_cuda)):
        _not_on_gpu()
    _check("nvfp4_dequantize", lib().nvfp4_dequantize(codes.data_ptr(), scales.data_ptr(), M, K, g_at, _ptr(row_g),
                                                      out.data_ptr(), _dtype_code(out.dtype), _stream(stream)))
    return out


def nvfp4_kv_cache_bytes(pages, page_size, heads, head_dim) -> int:
    return int(lib().nvfp4_kv_cache_bytes(int(pages), int(page_size), int(heads), int(head_dim)))


def nvfp4_kv_cache(pages, page_size, heads, head_dim, device=None):
    """A paged cache of one layer: uint8 [pages, heads, page_size / 16, 18 * head_dim], contents unset."""
    if nvfp4_kv_cache_bytes(pages, page_size, heads, head_dim) == 0:
        raise ValueError(lib().nvfp4_last_error().decode())
    return torch.empty((pages, heads, page_size // 16, 18 * head_dim), dtype=torch.uint8, device=device)


def _cache_sizes(cache):
    """(pages, page_size, heads, head_dim) of a cache tensor."""
    shape = cache.shape
    if len(shape) != 4 or cache.dtype is not torch.uint8 or shape[3] % 18:
        raise ValueError("cache must be uint8 [pages, heads, page_size / 16, 18 * head_dim]")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    return shape[0], 16 * shape[2], shape[1], shape[3] // 18


def _token_rows(t, name, heads, dim):
    """(tokens, token stride) of t [tokens, heads, dim], whose heads and channels must be dense."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}]")
    T = shape[0]
    row, head, channel = t.stride()
    if T and (channel != 1 or (heads > 1 and head != dim)):
        raise ValueError(f"{name}: heads and channels must be dense")
    return T, row if T > 1 else heads * dim


def _list(t, name, dtype):
    """t, checked to be a dense tensor of dtype."""
    if t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype}")
    return t


def nvfp4_kv_write(k, v, slots, k_g_inv, v_g_inv, cache, stream=None):
    """Quantizes k, v [T, heads, head_dim] (token stride free) into the cache's slots (int64 [T];
    page * page_size + place, outside the cache: skipped). Returns the cache."""
    pages, page_size, heads, dim = _cache_sizes(cache)
    T, ks = _token_rows(k, "k", heads, dim)
    Tv, vs = _token_rows(v, "v", heads, dim)
    if k.dtype is not v.dtype or T != Tv or _list(slots, "slots", torch.int64).numel() != T:
        raise ValueError("k, v and slots must have one type and length")
    kg, vg = _scalar(k_g_inv, "k_g_inv"), _scalar(v_g_inv, "v_g_inv")
    if not (k.is_cuda and v.is_cuda and slots.is_cuda and k_g_inv.is_cuda and v_g_inv.is_cuda and cache.is_cuda):
        _not_on_gpu()
    _check("nvfp4_kv_write",
           lib().nvfp4_kv_write(k.data_ptr(), v.data_ptr(), _dtype_code(k.dtype), T, ks, vs, slots.data_ptr(),
                                kg, vg, cache.data_ptr(), pages, page_size, heads, dim,
                                _stream(stream)))
    return cache


def nvfp4_kv_read(cache, slots, k_g, v_g, k=None, v=None, dtype=torch.bfloat16, stream=None):
    """The cache's numbers at slots (int64 [T]) -> (k, v) [T, heads, head_dim], zeros for slots outside it."""
    pages, page_size, heads, dim = _cache_sizes(cache)
    T = _list(slots, "slots", torch.int64).numel()
    shape = (T, heads, dim)
    if k is None:
        k = torch.empty(T, heads, dim, dtype=dtype, device=cache.device)
    elif k.shape != shape or not k.is_contiguous():
        raise ValueError(f"k must be contiguous, {shape}")
    if v is None:
        v = torch.empty_like(k)
    elif v.shape != shape or v.dtype is not k.dtype or not v.is_contiguous():
        raise ValueError(f"v must be contiguous, {shape}, of k's type")
    kg, vg = _scalar(k_g, "k_g"), _scalar(v_g, "v_g")
    if not (k.is_cuda and v.is_cuda and slots.is_cuda and k_g.is_cuda and v_g.is_cuda and cache.is_cuda):
        _not_on_gpu()
    _check("nvfp4_kv_read",
           lib().nvfp4_kv_read(cache.data_ptr(), pages, page_size, heads, dim, slots.data_ptr(), T, kg, vg,
                               k.data_ptr(), v.data_ptr(), _dtype_code(k.dtype), _stream(stream)))
    return k, v


def _same_gpu(first, *others):
    """All of them (or None) on the current GPU, whose stream the call is on."""
    at = first.get_device()
    for t in others:
        if t is not None and t.get_device() != at:
            at = min(at, t.get_device(), -1) if at < 0 or t.get_device() < 0 else None
            break
    if at is not None and at < 0:
        _not_on_gpu()
    if at is None or at != torch._C._cuda_getDevice():
        raise ValueError(f"all tensors must be on the current GPU, cuda:{torch._C._cuda_getDevice()}")


POOL_HEAD = 4  # words of a pool before its stack


def nvfp4_kv_pool_bytes(pages) -> int:
    return int(lib().nvfp4_kv_pool_bytes(int(pages)))


def _pool_pages(pool):
    if _list(pool, "pool", torch.int32).dim() != 1 or pool.numel() <= POOL_HEAD:
        raise ValueError(f"pool must be int32 [{POOL_HEAD} + pages]")
    return pool.numel() - POOL_HEAD


def nvfp4_kv_pool(pages, device="cuda", stream=None):
    """The pool of a cache's pages, all of them free: int32 [4 + pages]; [0] counts the free ones, [1] is the status
    (POOL_*: why requests were refused since it was last 0)."""
    if nvfp4_kv_pool_bytes(pages) == 0:
        raise ValueError(lib().nvfp4_last_error().decode())
    with _on(stream):
        pool = torch.empty(POOL_HEAD + pages, dtype=torch.int32, device=device)
    return nvfp4_kv_pool_reset(pool, stream)


def nvfp4_kv_pool_reset(pool, stream=None):
    """All pages free again, page 0 the next. Returns the pool."""
    pages = _pool_pages(pool)
    _same_gpu(pool)
    _check("nvfp4_kv_pool_reset", lib().nvfp4_kv_pool_reset(pool.data_ptr(), pages, _stream(stream)))
    return pool


def nvfp4_kv_advance(counts, seq_lens, block_table, pool, page_size, tokens, position_offsets=None, slots=None, positions=None,
                     q_offsets=None, stream=None):
    """counts int32 [B] tokens come to the sequences (or go, below 0): seq_lens int32 [B], block_table int32 [B, width] and
    the pool are brought up to date, in place. Returns (slots int64 [tokens], positions int32 [tokens], q_offsets int32 [B + 1])
    of the new tokens' rows; rows past them have slot -1. position_offsets int32 [B] is added to the positions."""
    pages = _pool_pages(pool)
    B = _list(counts, "counts", torch.int32).numel()
    if _list(seq_lens, "seq_lens", torch.int32).numel() != B:
        raise ValueError("counts and seq_lens must have one length")
    table = block_table.shape
    if len(table) != 2 or block_table.dtype is not torch.int32 or table[0] != B:
        raise ValueError("block_table must be int32 [sequences, width]")
    width = table[1]
    table_stride, entry = block_table.stride()
    if B and width > 1 and entry != 1:
        raise ValueError("block_table must have dense rows")
    if position_offsets is not None and _list(position_offsets, "position_offsets", torch.int32).numel() != B:
        raise ValueError("position_offsets must have one element a sequence")
    dev = counts.device
    if slots is None:
        slots = torch.empty(tokens, dtype=torch.int64, device=dev)
    elif _list(slots, "slots", torch.int64).numel() != tokens:
        raise ValueError(f"slots must be int64 [{tokens}]")
    if positions is None:
        positions = torch.empty(tokens, dtype=torch.int32, device=dev)
    elif _list(positions, "positions", torch.int32).numel() != tokens:
        raise ValueError(f"positions must be int32 [{tokens}]")
    if q_offsets is None:
        q_offsets = torch.empty(B + 1, dtype=torch.int32, device=dev)
    elif _list(q_offsets, "q_offsets", torch.int32).numel() != B + 1:
        raise ValueError("q_offsets must have one more element than seq_lens")
    _same_gpu(counts, seq_lens, block_table, pool, position_offsets, slots, positions, q_offsets)
    _check("nvfp4_kv_advance",
           lib().nvfp4_kv_advance(counts.data_ptr(), B, seq_lens.data_ptr(), block_table.data_ptr(),
                                  table_stride if B > 1 else width, width, page_size, pool.data_ptr(), pages, tokens,
                                  _ptr(position_offsets), q_offsets.data_ptr(), slots.data_ptr(), positions.data_ptr(),
                                  _stream(stream)))
    return slots, positions, q_offsets


def nvfp4_rope_axes(sections, interleaved=False, device="cuda"):
    """The axis of each frequency, int32 [sum(sections)]: sections[a] frequencies of axis a, in one run each or, interleaved,
    the axes in turn until each has its share."""
    left, axes = list(sections), []
    if interleaved:
        while any(left):
            for a, n in enumerate(left):
                if n:
                    axes.append(a)
                    left[a] -= 1
    else:
        for a, n in enumerate(left):
            axes += [a] * n
    return torch.tensor(axes, dtype=torch.int32, device=device)


def _rope_plan(positions, inv_freq, axes, T, dim):
    """(axis stride, axes, rotary channels) of a rotation of T tokens."""
    n = _list(inv_freq, "inv_freq", _F32).numel()
    if 2 * n > dim:
        raise ValueError(f"inv_freq must have at most {dim // 2} elements")
    if axes is not None and _list(axes, "axes", torch.int32).numel() != n:
        raise ValueError("axes must have one element a frequency")
    shape = positions.shape
    if positions.dtype is not torch.int32 or len(shape) not in (1, 2) or shape[-1] != T or (T > 1 and positions.stride(-1) != 1):
        raise ValueError(f"positions must be int32 [{T}] or [axes, {T}], each axis dense")
    if len(shape) == 1:  # of all axes alike
        return 0, 1 if axes is None else ROPE_AXES, 2 * n
    return positions.stride(0) if shape[0] > 1 else 0, shape[0], 2 * n


def nvfp4_rope(x, positions, inv_freq, axes=None, pairs=ROPE_HALVES, factor=1.0, out=None, out_dtype=None, stream=None):
    """x [T, heads, head_dim] (bf16 or f32, token stride free) turned by its positions (int32 [axes, T], or [T]: of all axes):
    frequency i of inv_freq (fp32 [rotary / 2]) with the positions of axis axes[i] (int32 [rotary / 2]; None: the first),
    cosine and sine times factor, channels paired by `pairs`. Frequencies of an axis below 0 or past the positions' (16 of
    [T]) turn nothing. Returns out (x's type by default; may be x)."""
    shape = x.shape
    if len(shape) != 3:
        raise ValueError("x must be [tokens, heads, head_dim]")
    T, xs = _token_rows(x, "x", shape[1], shape[2])
    step, count, rotary = _rope_plan(positions, inv_freq, axes, T, shape[2])
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or x.dtype, device=x.device)
    To, os_ = _token_rows(out, "out", shape[1], shape[2])
    if To != T:
        raise ValueError("out must have x's shape")
    _same_gpu(x, positions, inv_freq, axes, out)
    _check("nvfp4_rope",
           lib().nvfp4_rope(x.data_ptr(), _dtype_code(x.dtype), xs, T, shape[1], shape[2], positions.data_ptr(), step, count,
                            inv_freq.data_ptr(), _ptr(axes), rotary, pairs, factor, out.data_ptr(), _dtype_code(out.dtype), os_,
                            _stream(stream)))
    return out


def nvfp4_rope_kv_write(q, k, v, positions, inv_freq, slots, k_g_inv, v_g_inv, cache, axes=None, pairs=ROPE_HALVES, factor=1.0,
                        q_out=None, stream=None):
    """nvfp4_rope of q [T, heads_q, head_dim] and k, and nvfp4_kv_write of the turned k and of v, in one launch; q, k and v of
    one type. Returns the turned queries (bf16 unless q_out is given, which may be q)."""
    pages, page_size, heads, dim = _cache_sizes(cache)
    if len(q.shape) != 3:
        raise ValueError("q must be [tokens, heads_q, head_dim]")
    heads_q = q.shape[1]
    T, qs = _token_rows(q, "q", heads_q, dim)
    Tk, ks = _token_rows(k, "k", heads, dim)
    Tv, vs = _token_rows(v, "v", heads, dim)
    if q.dtype is not k.dtype or k.dtype is not v.dtype or T != Tk or T != Tv or _list(slots, "slots", torch.int64).numel() != T:
        raise ValueError("q, k, v and slots must have one type and length")
    step, count, rotary = _rope_plan(positions, inv_freq, axes, T, dim)
    if q_out is None:
        q_out = torch.empty(T, heads_q, dim, dtype=torch.bfloat16, device=q.device)
    To, os_ = _token_rows(q_out, "q_out", heads_q, dim)
    if To != T:
        raise ValueError("q_out must have q's shape")
    kg, vg = _scalar(k_g_inv, "k_g_inv"), _scalar(v_g_inv, "v_g_inv")
    _same_gpu(q, k, v, positions, inv_freq, slots, k_g_inv, v_g_inv, cache, axes, q_out)
    _check("nvfp4_rope_kv_write",
           lib().nvfp4_rope_kv_write(q.data_ptr(), qs, heads_q, k.data_ptr(), v.data_ptr(), _dtype_code(q.dtype), T, ks, vs,
                                     positions.data_ptr(), step, count, inv_freq.data_ptr(), _ptr(axes), rotary, pairs, factor,
                                     slots.data_ptr(), kg, vg, cache.data_ptr(), pages, page_size, heads, dim, q_out.data_ptr(),
                                     _dtype_code(q_out.dtype), os_, _stream(stream)))
    return q_out


def nvfp4_tree_mask(parents, q_offsets, max_q, positions=None, tree=None, stream=None):
    """The masks of drafted trees for nvfp4_kv_attention: int64 [T, ceil(max_q / 64)], a bit for itself and each ancestor.
    parents int32 [T]: the number of a token's parent in its sequence's draft (below 0: none); q_offsets int32 [B + 1] (None:
    max_q tokens each). positions int32 [T] become the first row's of a sequence plus the depth, in place."""
    T = _list(parents, "parents", torch.int32).numel()
    if q_offsets is None:
        B = T // max_q if max_q > 0 else 0
        if T != B * max_q:
            raise ValueError("without q_offsets parents must have max_q elements a sequence")
    else:
        B = _list(q_offsets, "q_offsets", torch.int32).numel() - 1
    if tree is None:
        tree = torch.empty(T, max(1, (max_q + 63) // 64), dtype=torch.int64, device=parents.device)
    elif len(tree.shape) != 2 or _list(tree, "tree", torch.int64).shape[0] != T:
        raise ValueError(f"tree must be int64 [{T}, words]")
    if positions is not None and _list(positions, "positions", torch.int32).numel() != T:
        raise ValueError(f"positions must be int32 [{T}]")
    _same_gpu(parents, q_offsets, tree, positions)
    _check("nvfp4_tree_mask", lib().nvfp4_tree_mask(parents.data_ptr(), T, B, _ptr(q_offsets), max_q, tree.data_ptr(),
                                                    tree.shape[1], _ptr(positions), _stream(stream)))
    return tree


def nvfp4_kv_attention_workspace_bytes(T, B, heads_q, heads, head_dim, max_q, max_len) -> int:
    """Bytes of ws for all attention calls of at most these sizes (never less for larger ones)."""
    return lib().nvfp4_kv_attention_workspace_bytes(T, B, heads_q, heads, head_dim, max_q, max_len)


ATTENTION_COUNTER_BYTES = 4096


def nvfp4_kv_attention(q, cache, block_table, seq_lens, k_g, v_g, q_offsets=None, max_q=None, max_len=None, scale=None,
                       window=0, ws=None, out=None, out_dtype=torch.bfloat16, lse=None, return_lse=False, stream=None, sinks=0,
                       tree=None):
    """Causal attention of q bf16 [T, heads_q, head_dim] (token stride free) over the cache.

    block_table int32 [B, width], seq_lens int32 [B]; sequence b's queries are q[q_offsets[b]:q_offsets[b + 1]]
    (int32 [B + 1]; None: T / B each) at its last positions; rows of no sequence are not written. max_q, max_len:
    bounds known on the host (default: T / B or T, and the table's width). scale: 1 / sqrt(head_dim) by default; window: visible keys of a query (0: all),
    sinks: first keys that stay visible behind it. tree int64 [T, words] (nvfp4_tree_mask): a sequence's queries are a drafted
    tree, whose query sees the drafted keys of its bits and all keys in front of them (max_q at most 64 words, 4096, and at
    most the window).
    ws: workspace whose first 4096 bytes are zero the first time; allocated if None. out_dtype fp32 computes with
    probabilities of 22 bits, bf16 with 11. Returns out (and lse)."""
    pages, page_size, heads, dim = _cache_sizes(cache)
    shape = q.shape
    if len(shape) != 3 or q.dtype is not torch.bfloat16:
        raise ValueError("q must be bf16 [tokens, heads_q, head_dim]")
    heads_q = shape[1]
    T, qs = _token_rows(q, "q", heads_q, dim)
    B = _list(seq_lens, "seq_lens", torch.int32).numel()
    table = block_table.shape
    if len(table) != 2 or block_table.dtype is not torch.int32 or table[0] != B:
        raise ValueError("block_table must be int32 [sequences, width]")
    width = table[1]
    table_stride, entry = block_table.stride()
    if width > 1 and entry != 1:
        raise ValueError("block_table must have dense rows")
    if q_offsets is not None and _list(q_offsets, "q_offsets", torch.int32).numel() != B + 1:
        raise ValueError("q_offsets must have one more element than seq_lens")
    if max_q is None:
        max_q = T if q_offsets is not None else (T // B if B else 0)
    if max_len is None:
        max_len = width * page_size
    if scale is None:
        scale = dim ** -0.5
    if out is None:
        out = torch.empty(T, heads_q, dim, dtype=out_dtype, device=q.device)
    elif out.shape != shape or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape")
    if lse is None:
        if return_lse:
            lse = torch.empty(T, heads_q, dtype=torch.float32, device=q.device)
    elif _list(lse, "lse", torch.float32).numel() != T * heads_q:
        raise ValueError("lse must be fp32 [tokens, heads_q]")
    words = 0
    if tree is not None:
        if len(tree.shape) != 2 or _list(tree, "tree", torch.int64).shape[0] != T or tree.shape[1] < 1:
            raise ValueError(f"tree must be int64 [{T}, words]")
        words = tree.shape[1]
    kg, vg = _scalar(k_g, "k_g"), _scalar(v_g, "v_g")
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    if not (q.is_cuda and cache.is_cuda and block_table.is_cuda and seq_lens.is_cuda and k_g.is_cuda and v_g.is_cuda and
            out.is_cuda and (q_offsets is None or q_offsets.is_cuda) and (lse is None or lse.is_cuda) and
            (ws is None or ws.is_cuda)):
        _not_on_gpu()
    if ws is None:
        n = nvfp4_kv_attention_workspace_bytes(T, B, heads_q, heads, dim, max_q, max_len)
        with _on(stream):
            ws = torch.empty(max(n, ATTENTION_COUNTER_BYTES), dtype=torch.uint8, device=q.device)
            ws[:ATTENTION_COUNTER_BYTES].zero_()
    if sinks or tree is not None:
        _same_gpu(q, cache, block_table, seq_lens, k_g, v_g, q_offsets, tree, out, lse, ws)
        _check("nvfp4_kv_attention_masked",
               lib().nvfp4_kv_attention_masked(q.data_ptr(), qs, T, B, heads_q, _ptr(q_offsets), max_q, cache.data_ptr(), pages,
                                               page_size, heads, dim, block_table.data_ptr(), table_stride if B > 1 else width,
                                               width, seq_lens.data_ptr(), max_len, scale, window, sinks, _ptr(tree), words, kg,
                                               vg, ws.data_ptr(), ws.nbytes, out.data_ptr(), _dtype_code(out.dtype), _ptr(lse),
                                               _stream(stream)))
        return out if lse is None else (out, lse)
    _check("nvfp4_kv_attention",
           lib().nvfp4_kv_attention(q.data_ptr(), qs, T, B, heads_q, _ptr(q_offsets), max_q, cache.data_ptr(), pages,
                                    page_size, heads, dim, block_table.data_ptr(), table_stride if B > 1 else width, width,
                                    seq_lens.data_ptr(), max_len, scale, window, kg, vg, ws.data_ptr(),
                                    ws.nbytes, out.data_ptr(), _dtype_code(out.dtype), _ptr(lse), _stream(stream)))
    return out if lse is None else (out, lse)
