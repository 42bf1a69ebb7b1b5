"""Thin Python binding of the C ABI declared in include/pmn.h.

Each function here has the name of its C entry point without the `pmn_`
prefix and does argument marshalling only: it allocates outputs with torch
(device memory), passes raw device pointers and the current CUDA stream to
libpmn.so, and raises on a non-zero status.  Every step of the computation
runs in the library's CUDA kernels; there is no fallback path -- if the
library is missing or fails to load, every call raises.
"""
import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpmn.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = 0, 1, 2, 3, 4
IN_BF16, IN_BF16_SWIGLU = 0, 1
OUTER_PER_ROW, OUTER_PER_GROUP = 0, 1
ROUND_SR, ROUND_RN = 0, 1
OUT_BF16, OUT_F32, OUT_RHT_S2F6, OUT_SWIGLU_BF16 = 0, 1, 2, 3
GROUP_M, GROUP_K = 0, 1
STATE_F32, STATE_MXFP8 = 0, 1
DEVERR_WAIT_TIMEOUT = 1
DEVERR_BAD_OFFSETS = 2

# Stochastic-rounding stream tags of the expert layer's saved tensors.
TAG_X, TAG_H, TAG_W1, TAG_W2 = 1, 2, 3, 4

_P, _I64, _U64, _U32, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int
_F, _D = ctypes.c_float, ctypes.c_double


class AdamWTensor(ctypes.Structure):
    """pmn_adamw_tensor"""
    _fields_ = [("param", _P), ("copy", _P), ("grad", _P), ("m", _P), ("v", _P), ("m_scales", _P), ("v_scales", _P),
                ("n", _I64)]


SIGNATURES = {
    "pmn_version": ([], _I),
    "pmn_status_string": ([_I], ctypes.c_char_p),
    "pmn_get_device_error": ([_P, _P], _I),
    "pmn_set_wait_limit_ns": ([_U64], _U64),
    "pmn_wait_selftest": ([_U64, _P], _I),
    "pmn_nvfp4_quantize": ([_P, _I64, _I64, _I64, _I, _I, _I64, _I, _P, _P, _P, _P, _P, _I64, _P], _I),
    "pmn_nvfp4_quantize_workspace_bytes": ([_I, _I64, _I64], _I64),
    "pmn_nvfp4_quantize_per_group_noalloc": ([_P, _I64, _I64, _I64, _I, _P, _P, _P, _P], _I),
    "pmn_requant_transpose_sr_mxfp8": ([_P, _P, _P, _I, _I64, _I64, _I64, _U64, _U32, _I, _P, _P, _P], _I),
    "pmn_mxfp8_quantize_both": ([_P, _I64, _I64, _P, _P, _P, _P, _P], _I),
    "pmn_requant_transpose_sr_nvfp4": ([_P, _P, _P, _I, _I64, _I64, _I64, _U64, _U32, _I, _P, _P, _P, _P], _I),
    "pmn_mxfp8_quantize": ([_P, _I64, _I64, _I, _P, _P, _P], _I),
    "pmn_mxfp8_quantize_swiglu": ([_P, _I64, _I64, _P, _P, _P, _P], _I),
    "pmn_grouped_gemm_nvfp4": ([_P, _P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _P, _P], _I),
    "pmn_w1_gemm_swiglu_nvfp4": ([_P, _P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _P, _P, _P, _P, _P], _I),
    "pmn_w2_gemm_rht_s2f6": ([_P, _P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _U64, _P, _P, _P, _P], _I),
    "pmn_rht_s2f6_quantize": ([_P, _I64, _I64, _U64, _P, _P, _P], _I),
    "pmn_combine_receive_s2f6": ([_P, _P, _I64, _I64, _U64, _P, _P, _I64, _I, _I, _P, _P], _I),
    "pmn_gemm_mxfp8": ([_P, _P, _P, _P, _P, _I, _I, _I64, _I64, _I64, _I, _P, _P], _I),
    "pmn_add_rmsnorm_mxfp8": ([_P, _I64, _P, _I64, _I, _P, _I64, _I64, _F, _P, _P, _P, _P, _P, _P], _I),
    "pmn_add_rmsnorm_backward": ([_P, _P, _I, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P], _I),
    "pmn_add_rmsnorm_backward_workspace_bytes": ([_I64, _I64], _I64),
    "pmn_w1_gemm_swiglu_mxfp8": ([_P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P], _I),
    "pmn_dh_gemm_swiglu_backward_mxfp8": ([_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P], _I),
    "pmn_adamw_step": ([ctypes.POINTER(AdamWTensor), _I, _I, _I, _I, _D, _D, _D, _D, _D, _I64, _P, _U64, _P], _I),
}

_lib = None


class PmnError(RuntimeError):
    pass


def lib():
    """The loaded libpmn.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise PmnError("libpmn.so not built: run precision_moe_numerics_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _check(st, what):
    if st != OK:
        msg = lib().pmn_status_string(st).decode()
        raise PmnError("%s failed: %s (%d)" % (what, msg, st))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, dtype=None):
    if not t.is_cuda:
        raise PmnError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise PmnError("tensor must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise PmnError("expected %s, got %s" % (dtype, t.dtype))
    return t


def version():
    return lib().pmn_version()


def get_device_error(stream=None):
    err = ctypes.c_int32(0)
    _check(lib().pmn_get_device_error(_stream(stream), ctypes.byref(err)), "get_device_error")
    return err.value


def set_wait_limit_ns(ns):
    """Sets the limit of the library's bounded device waits; returns the previous one."""
    return lib().pmn_set_wait_limit_ns(int(ns))


def wait_selftest(limit_ns, stream=None):
    _check(lib().pmn_wait_selftest(int(limit_ns), _stream(stream)), "wait_selftest")


def nvfp4_quantize_workspace_bytes(outer_mode, rows, rows_per_group=0):
    n = lib().pmn_nvfp4_quantize_workspace_bytes(outer_mode, rows, rows_per_group)
    if n < 0:
        raise PmnError("nvfp4_quantize_workspace_bytes: invalid arguments")
    return n


# ------------------------------------------------------------------ quantisation
def nvfp4_quantize(x, cols=None, four_over_six=False, outer_mode=OUTER_PER_ROW, rows_per_group=None,
                   swiglu=False, want_h=False, out=None, workspace=None, stream=None):
    """bf16 [rows, ldx] -> (codes u8 [rows, cols/2], scales u8 [rows, cols/16], outer f32[, h bf16]).

    swiglu: x holds gate | up halves of width `cols`; h = silu(gate) * up is quantised.
    workspace: the per-group kernel's scratch (uint8 device tensor of at least
    nvfp4_quantize_workspace_bytes(...) bytes); allocated here when None."""
    _dev(x, torch.bfloat16)
    rows, ldx = x.shape
    if cols is None:
        cols = ldx // 2 if swiglu else ldx
    dev = x.device
    if out is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
        n_outer = rows if outer_mode == OUTER_PER_ROW else rows // rows_per_group
        outer = torch.empty((n_outer,), dtype=torch.float32, device=dev)
    else:
        codes, scales, outer = out
    h = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev) if want_h else None
    if workspace is None and outer_mode == OUTER_PER_GROUP:
        workspace = torch.empty((max(1, nvfp4_quantize_workspace_bytes(outer_mode, rows, rows_per_group or 0)),),
                                dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().pmn_nvfp4_quantize(_ptr(x), rows, cols, ldx, IN_BF16_SWIGLU if swiglu else IN_BF16, outer_mode,
                                  rows_per_group or 0, int(four_over_six), _ptr(codes), _ptr(scales), _ptr(outer),
                                  _ptr(h), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "nvfp4_quantize")
    return (codes, scales, outer, h) if want_h else (codes, scales, outer)


def nvfp4_quantize_per_group_noalloc(x, rows_per_group, four_over_six=False, out=None, stream=None):
    """As nvfp4_quantize(x, outer_mode=OUTER_PER_GROUP, ...), through the entry point whose scratch is a
    fixed device array (no allocation inside the call)."""
    _dev(x, torch.bfloat16)
    rows, cols = x.shape
    dev = x.device
    if out is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
        outer = torch.empty((rows // rows_per_group,), dtype=torch.float32, device=dev)
    else:
        codes, scales, outer = out
    st = lib().pmn_nvfp4_quantize_per_group_noalloc(_ptr(x), rows, cols, rows_per_group, int(four_over_six),
                                                    _ptr(codes), _ptr(scales), _ptr(outer), _stream(stream))
    _check(st, "nvfp4_quantize_per_group_noalloc")
    return codes, scales, outer


def requant_transpose_sr_mxfp8(codes, scales, outer, outer_per_row, batch, rows, cols, seed, tag,
                               stochastic=True, out=None, stream=None):
    """NVFP4 [batch, rows, cols] -> MXFP8 transposed (u8 [batch, cols, rows], u8 [batch, cols, rows/32])."""
    _dev(codes, torch.uint8)
    _dev(scales, torch.uint8)
    _dev(outer, torch.float32)
    if out is None:
        q = torch.empty((batch, cols, rows), dtype=torch.uint8, device=codes.device)
        sc = torch.empty((batch, cols, rows // 32), dtype=torch.uint8, device=codes.device)
    else:
        q, sc = out
    st = lib().pmn_requant_transpose_sr_mxfp8(_ptr(codes), _ptr(scales), _ptr(outer),
                                              OUTER_PER_ROW if outer_per_row else OUTER_PER_GROUP, batch, rows,
                                              cols, seed, tag, ROUND_SR if stochastic else ROUND_RN, _ptr(q),
                                              _ptr(sc), _stream(stream))
    _check(st, "requant_transpose_sr_mxfp8")
    return q, sc


def requant_transpose_sr_nvfp4(codes, scales, outer, outer_per_row, batch, rows, cols, seed, tag,
                               stochastic=True, out=None, stream=None):
    """NVFP4 [batch, rows, cols] -> NVFP4 of the transpose with stochastic
    rounding (u8 codes [batch, cols, rows/2], u8 E4M3 [batch, cols, rows/16],
    f32 outer [batch]): the FP4 backward's requantisation."""
    _dev(codes, torch.uint8)
    _dev(scales, torch.uint8)
    _dev(outer, torch.float32)
    if out is None:
        q = torch.empty((batch, cols, rows // 2), dtype=torch.uint8, device=codes.device)
        sc = torch.empty((batch, cols, rows // 16), dtype=torch.uint8, device=codes.device)
        g = torch.empty((batch,), dtype=torch.float32, device=codes.device)
    else:
        q, sc, g = out
    st = lib().pmn_requant_transpose_sr_nvfp4(_ptr(codes), _ptr(scales), _ptr(outer),
                                              OUTER_PER_ROW if outer_per_row else OUTER_PER_GROUP, batch, rows,
                                              cols, seed, tag, ROUND_SR if stochastic else ROUND_RN, _ptr(q),
                                              _ptr(sc), _ptr(g), _stream(stream))
    _check(st, "requant_transpose_sr_nvfp4")
    return q, sc, g


def mxfp8_quantize(x, transpose=False, out=None, stream=None):
    """bf16 [rows, cols] -> MXFP8 with RN (u8 values, u8 E8M0 scales), optionally transposed."""
    _dev(x, torch.bfloat16)
    rows, cols = x.shape
    if out is None:
        shp = (cols, rows) if transpose else (rows, cols)
        q = torch.empty(shp, dtype=torch.uint8, device=x.device)
        sc = torch.empty((shp[0], shp[1] // 32), dtype=torch.uint8, device=x.device)
    else:
        q, sc = out
    _check(lib().pmn_mxfp8_quantize(_ptr(x), rows, cols, int(transpose), _ptr(q), _ptr(sc), _stream(stream)),
           "mxfp8_quantize")
    return q, sc


def mxfp8_quantize_both(x, out=None, out_t=None, stream=None):
    """bf16 [rows, cols] -> (MXFP8 rowwise (u8 [rows, cols], u8 [rows, cols/32]),
    MXFP8 of the transpose (u8 [cols, rows], u8 [cols, rows/32])) in one pass."""
    _dev(x, torch.bfloat16)
    rows, cols = x.shape
    dev = x.device
    if out is None:
        out = (torch.empty((rows, cols), dtype=torch.uint8, device=dev),
               torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev))
    if out_t is None:
        out_t = (torch.empty((cols, rows), dtype=torch.uint8, device=dev),
                 torch.empty((cols, rows // 32), dtype=torch.uint8, device=dev))
    st = lib().pmn_mxfp8_quantize_both(_ptr(x), rows, cols, _ptr(out[0]), _ptr(out[1]), _ptr(out_t[0]),
                                       _ptr(out_t[1]), _stream(stream))
    _check(st, "mxfp8_quantize_both")
    return out, out_t


def mxfp8_quantize_swiglu(y, want_h=False, out=None, stream=None):
    """bf16 y [rows, 2f] (gate | up) -> MXFP8 (RN) of h = silu(gate) * up
    (u8 values [rows, f], u8 E8M0 scales [rows, f/32][, bf16 h])."""
    _dev(y, torch.bfloat16)
    rows, f2 = y.shape
    f = f2 // 2
    if out is None:
        q = torch.empty((rows, f), dtype=torch.uint8, device=y.device)
        sc = torch.empty((rows, f // 32), dtype=torch.uint8, device=y.device)
    else:
        q, sc = out
    h = torch.empty((rows, f), dtype=torch.bfloat16, device=y.device) if want_h else None
    _check(lib().pmn_mxfp8_quantize_swiglu(_ptr(y), rows, f, _ptr(q), _ptr(sc), _ptr(h), _stream(stream)),
           "mxfp8_quantize_swiglu")
    return (q, sc, h) if want_h else (q, sc)


def rht_s2f6_quantize(x, seed, out=None, stream=None):
    _dev(x, torch.float32)
    rows, cols = x.shape
    if out is None:
        q = torch.empty((rows, cols), dtype=torch.int8, device=x.device)
        sc = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
    else:
        q, sc = out
    _check(lib().pmn_rht_s2f6_quantize(_ptr(x), rows, cols, seed, _ptr(q), _ptr(sc), _stream(stream)),
           "rht_s2f6_quantize")
    return q, sc


def combine_receive_s2f6(payload, seed, row_index, gates, out_dtype=torch.bfloat16, out=None, stream=None):
    """payload = (int8 [rows, cols], E8M0 uint8 [rows, cols/32]) in routed
    order; row_index int32 [tokens, k], gates float32 [tokens, k] -> the
    token rows [tokens, cols] (bf16 or float32)."""
    q, sc = payload
    _dev(q, torch.int8)
    _dev(sc, torch.uint8)
    _dev(row_index, torch.int32)
    _dev(gates, torch.float32)
    rows, cols = q.shape
    tokens, k = row_index.shape
    if tuple(gates.shape) != (tokens, k) or tuple(sc.shape) != (rows, cols // 32):
        raise PmnError("combine_receive_s2f6: shape mismatch")
    kind = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}[out_dtype]
    if out is None:
        out = torch.empty((tokens, cols), dtype=out_dtype, device=q.device)
    _check(lib().pmn_combine_receive_s2f6(_ptr(q), _ptr(sc), rows, cols, seed, _ptr(row_index), _ptr(gates),
                                          tokens, k, kind, _ptr(out), _stream(stream)),
           "combine_receive_s2f6")
    return out


# ------------------------------------------------------------------ GEMMs
def grouped_gemm_nvfp4(a, b, offsets, out_dtype=torch.bfloat16, swiglu=False, out=None, stream=None):
    """a = (codes [T, K/2], scales [T, K/16], outer [T]); b = (codes [E, N, K/2],
    scales [E, N, K/16], outer [E]); offsets int32 [E+1] on the device.
    swiglu: the bf16 h = silu(gate) * up [T, N/2] of the float32 product
    (gate = the first N/2 rows of each B_e, up = the last N/2)."""
    ac, asc, ao = a
    bc, bsc, bo = b
    _dev(offsets, torch.int32)
    T = ac.shape[0]
    E, N = bc.shape[0], bc.shape[1]
    K = ac.shape[1] * 2
    kind = OUT_SWIGLU_BF16 if swiglu else (OUT_BF16 if out_dtype == torch.bfloat16 else OUT_F32)
    if out is None:
        out = torch.empty((T, N // 2 if swiglu else N), dtype=torch.bfloat16 if swiglu else out_dtype,
                          device=ac.device)
    st = lib().pmn_grouped_gemm_nvfp4(_ptr(ac), _ptr(asc), _ptr(ao), _ptr(bc), _ptr(bsc), _ptr(bo), _ptr(offsets),
                                      E, T, N, K, kind, _ptr(out), _stream(stream))
    _check(st, "grouped_gemm_nvfp4")
    return out


def w1_gemm_swiglu_nvfp4(a, b, offsets, four_over_six=True, out=None, h=None, stream=None):
    """w1 GEMM with SwiGLU in its epilogue, then NVFP4 (per token, 4/6) of h.
    a = NVFP4 rows (codes [T, K/2], scales [T, K/16], outer [T]); b = NVFP4 W1
    (codes [E, 2F, K/2], scales [E, 2F, K/16], outer [E]) with gate rows first.
    Returns (codes u8 [T, F/2], scales u8 [T, F/16], outer f32 [T]); `h` (bf16
    [T, F], allocated here when None) receives h itself."""
    ac, asc, ao = a
    bc, bsc, bo = b
    _dev(offsets, torch.int32)
    T = ac.shape[0]
    E, F2 = bc.shape[0], bc.shape[1]
    F = F2 // 2
    K = ac.shape[1] * 2
    dev = ac.device
    if out is None:
        out = (torch.empty((T, F // 2), dtype=torch.uint8, device=dev),
               torch.empty((T, F // 16), dtype=torch.uint8, device=dev),
               torch.empty((T,), dtype=torch.float32, device=dev))
    if h is None:
        h = torch.empty((T, F), dtype=torch.bfloat16, device=dev)
    _dev(h, torch.bfloat16)
    c, sc, g = out
    st = lib().pmn_w1_gemm_swiglu_nvfp4(_ptr(ac), _ptr(asc), _ptr(ao), _ptr(bc), _ptr(bsc), _ptr(bo), _ptr(offsets),
                                        E, T, F, K, int(four_over_six), _ptr(h), _ptr(c), _ptr(sc), _ptr(g),
                                        _stream(stream))
    _check(st, "w1_gemm_swiglu_nvfp4")
    return out


def w2_gemm_rht_s2f6(a, b, offsets, seed, out=None, debug_acc=None, stream=None):
    """(q int8 [T, N], scales u8 [T, N/32]); debug_acc: optional float32 [T, N] that receives the
    epilogue's input (the scaled accumulator) on the expert segments' rows."""
    ac, asc, ao = a
    bc, bsc, bo = b
    _dev(offsets, torch.int32)
    T = ac.shape[0]
    E, N = bc.shape[0], bc.shape[1]
    K = ac.shape[1] * 2
    if out is None:
        q = torch.empty((T, N), dtype=torch.int8, device=ac.device)
        sc = torch.empty((T, N // 32), dtype=torch.uint8, device=ac.device)
    else:
        q, sc = out
    if debug_acc is not None:
        _dev(debug_acc, torch.float32)
    st = lib().pmn_w2_gemm_rht_s2f6(_ptr(ac), _ptr(asc), _ptr(ao), _ptr(bc), _ptr(bsc), _ptr(bo), _ptr(offsets), E,
                                    T, N, K, seed, _ptr(q), _ptr(sc),
                                    _ptr(debug_acc) if debug_acc is not None else None, _stream(stream))
    _check(st, "w2_gemm_rht_s2f6")
    return q, sc


def gemm_mxfp8(a, a_sc, b, b_sc, offsets, group_mode, out_dtype=torch.float32, out=None, stream=None):
    """GROUP_M: a [M, K], b [G, N, K] -> [M, N];  GROUP_K: a [M, Kt], b [N, Kt] -> [G, M, N]."""
    _dev(offsets, torch.int32)
    G = offsets.numel() - 1
    M, K = a.shape
    N = b.shape[-2]
    kind = OUT_BF16 if out_dtype == torch.bfloat16 else OUT_F32
    if out is None:
        shp = (M, N) if group_mode == GROUP_M else (G, M, N)
        out = torch.empty(shp, dtype=out_dtype, device=a.device)
    st = lib().pmn_gemm_mxfp8(_ptr(a), _ptr(a_sc), _ptr(b), _ptr(b_sc), _ptr(offsets), G, group_mode, M, N, K, kind,
                              _ptr(out), _stream(stream))
    _check(st, "gemm_mxfp8")
    return out


# ------------------------------------------------------------------ around the MXFP8 layers
_KINDS = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}


def _kind(t, what):
    k = _KINDS.get(t.dtype)
    if k is None:
        raise PmnError("%s must be bfloat16 or float32, got %s" % (what, t.dtype))
    return k


# A launch goes to the current GPU whatever its stream's handle says (the default stream's is the same on every one),
# so a call's tensors and its stream have to be there: `gpu` below is the current one's number.  (torch.cuda's own
# functions look for the library first, and current_stream() builds an object: 3 us of a call that takes 2 us on the GPU.)
def _launch_stream(what, stream, gpu):
    """the raw handle of `stream`, or of the current stream"""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(gpu)
    if stream.device_index != gpu:
        raise PmnError("%s: the stream is of cuda:%d, the current GPU is cuda:%d" % (what, stream.device_index, gpu))
    return stream.cuda_stream


def _at(t):
    return None if t is None else t.data_ptr()


def _empty(shape, dtype, device, stream):
    """memory that the call's stream may write at once: another stream's pool may hand out a block that its own
    kernels still use, and take this one back while the call still runs"""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(t, what, gpu, dtype=None):
    """2-D tensor on the current GPU whose rows are contiguous (any row pitch); returns its pitch in elements"""
    if t.get_device() != gpu or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise PmnError("%s must be a 2-D tensor on the current GPU (cuda:%d) with contiguous rows" % (what, gpu))
    if dtype is not None and t.dtype != dtype:
        raise PmnError("%s: expected %s, got %s" % (what, dtype, t.dtype))
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _shaped(t, shape, dtype, what, gpu):
    """a dense tensor of this shape and type on the current GPU (an output or operand that the kernels index by it)"""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != gpu or not t.is_contiguous():
        raise PmnError("%s must be a dense %s tensor of shape %s on the current GPU (cuda:%d)" % (what, dtype, (shape,), gpu))
    return t


def _mxfp8_out(out, rows, cols, device, stream, gpu, what="out"):
    if out is None:
        return (_empty((rows, cols), torch.uint8, device, stream), _empty((rows, cols // 32), torch.uint8, device, stream))
    _shaped(out[0], (rows, cols), torch.uint8, what, gpu)
    _shaped(out[1], (rows, cols // 32), torch.uint8, what + " scales", gpu)
    return out


def add_rmsnorm_mxfp8(x, residual, weight, eps=1e-6, out=None, res_out=None, y=None, rstd=None, want_y=False,
                      want_rstd=False, stream=None):
    """r = x + residual (in the residual's type; r = x where residual is None), y = r * rstd * weight, MXFP8 of y.

    x bf16 [rows, cols], residual None or bf16 / float32 [rows, cols] (both may be row-strided views), weight
    bf16 [cols].  Returns ((u8 values, u8 E8M0 scales), r or None, y or None, rstd or None); y (bf16) and rstd
    (float32) are written where they are passed in or wanted."""
    gpu = torch._C._cuda_getDevice()
    ldx = _rows(x, "x", gpu, torch.bfloat16)
    rows, cols = x.shape
    dev = x.device
    _shaped(weight, (cols,), torch.bfloat16, "weight", gpu)
    ldr, kind = 0, OUT_BF16
    if residual is not None:
        ldr, kind = _rows(residual, "residual", gpu), _kind(residual, "residual")
        if residual.shape != x.shape:
            raise PmnError("residual must have x's shape")
        if res_out is None:
            res_out = _empty((rows, cols), residual.dtype, dev, stream)
        else:
            _shaped(res_out, (rows, cols), residual.dtype, "res_out", gpu)
    elif res_out is not None:
        raise PmnError("res_out without a residual")
    out = _mxfp8_out(out, rows, cols, dev, stream, gpu)
    if y is not None:
        _shaped(y, (rows, cols), torch.bfloat16, "y", gpu)
    elif want_y:
        y = _empty((rows, cols), torch.bfloat16, dev, stream)
    if rstd is not None:
        _shaped(rstd, (rows,), torch.float32, "rstd", gpu)
    elif want_rstd:
        rstd = _empty((rows,), torch.float32, dev, stream)
    raw = _launch_stream("add_rmsnorm_mxfp8", stream, gpu)
    _check(lib().pmn_add_rmsnorm_mxfp8(_at(x), ldx, _at(residual), ldr, kind, _at(weight), rows, cols, eps,
                                       _at(res_out), _at(out[0]), _at(out[1]), _at(y), _at(rstd), raw),
           "add_rmsnorm_mxfp8")
    return out, res_out, y, rstd


def add_rmsnorm_backward_workspace_bytes(rows, cols):
    n = lib().pmn_add_rmsnorm_backward_workspace_bytes(rows, cols)
    if n < 0:
        raise PmnError("add_rmsnorm_backward_workspace_bytes: invalid arguments")
    return n


def add_rmsnorm_backward(dy, r, rstd, weight, dres=None, dr=None, dx=None, dw=None, want_dx=False, workspace=None,
                         stream=None):
    """Gradients of add_rmsnorm_mxfp8's y: (dr in r's type, dx bf16 or None, dw float32 [cols]).

    dy bf16 [rows, cols]; r bf16 or float32 [rows, cols]; dres (r's type) is added to dr, which is the gradient of
    x and of the residual.  dx: dr rounded to bf16 (float32 r only).  workspace: uint8 device tensor of at least
    add_rmsnorm_backward_workspace_bytes(rows, cols) bytes, allocated here when None."""
    rows, cols = dy.shape
    dev, gpu = dy.device, torch._C._cuda_getDevice()
    _shaped(dy, (rows, cols), torch.bfloat16, "dy", gpu)
    kind = _kind(r, "r")
    _shaped(r, (rows, cols), r.dtype, "r", gpu)
    _shaped(rstd, (rows,), torch.float32, "rstd", gpu)
    _shaped(weight, (cols,), torch.bfloat16, "weight", gpu)
    if dres is not None:
        _shaped(dres, (rows, cols), r.dtype, "dres", gpu)
    dr = _empty(r.shape, r.dtype, dev, stream) if dr is None else _shaped(dr, (rows, cols), r.dtype, "dr", gpu)
    if dx is not None:
        _shaped(dx, (rows, cols), torch.bfloat16, "dx", gpu)
    elif want_dx:
        dx = _empty((rows, cols), torch.bfloat16, dev, stream)
    dw = _empty((cols,), torch.float32, dev, stream) if dw is None else _shaped(dw, (cols,), torch.float32, "dw", gpu)
    if workspace is None:
        workspace = _empty((add_rmsnorm_backward_workspace_bytes(rows, cols),), torch.uint8, dev, stream)
    elif workspace.get_device() != gpu or not workspace.is_contiguous():
        raise PmnError("workspace must be a dense tensor on the current GPU (cuda:%d)" % gpu)
    raw = _launch_stream("add_rmsnorm_backward", stream, gpu)
    _check(lib().pmn_add_rmsnorm_backward(_at(dy), _at(r), kind, _at(rstd), _at(weight), _at(dres), rows, cols,
                                          _at(dr), _at(dx), _at(dw), _at(workspace),
                                          workspace.numel() * workspace.element_size(), raw),
           "add_rmsnorm_backward")
    return dr, dx, dw


def _gated_operands(a, b, offsets, what, gpu):
    """checks of the operands both directions share; (rows, k, experts, rows of B per expert)"""
    aq, asc = a
    bq, bsc = b
    if aq.dim() != 2 or bq.dim() != 3 or aq.shape[1] != bq.shape[2]:
        raise PmnError("%s: a is [rows, k], b is [experts, n, k]" % what)
    rows, k = aq.shape
    experts, n = bq.shape[0], bq.shape[1]
    for t, shape in ((aq, (rows, k)), (asc, (rows, k // 32)), (bq, (experts, n, k)), (bsc, (experts, n, k // 32))):
        _shaped(t, shape, torch.uint8, what + ": an operand", gpu)
    _shaped(offsets, (experts + 1,), torch.int32, what + ": offsets", gpu)
    return rows, k, experts, n


def w1_gemm_swiglu_mxfp8(a, b, offsets, out=None, out_t=None, y=None, want_t=False, want_y=False, stream=None):
    """The gated projection in one kernel: MXFP8 of h = silu(X . Wg^T) * (X . Wu^T).

    a = MXFP8 rows (u8 [T, K], u8 [T, K/32]); b = MXFP8 W1 (u8 [E, 2F, K], u8 [E, 2F, K/32]), gate rows first;
    offsets int32 [E+1] on the device.  Returns (h, h_t or None, y or None): h = (u8 [T, F], u8 [T, F/32]); h_t =
    MXFP8 of h^T along the rows (u8 [F, T], u8 [F, T/32]; offsets and T multiples of 32), y = bf16 [T, 2F], both
    written where they are passed in or wanted (a training step's backward pass needs them)."""
    gpu = torch._C._cuda_getDevice()
    rows, k, experts, f2 = _gated_operands(a, b, offsets, "w1_gemm_swiglu_mxfp8", gpu)
    if f2 % 2:
        raise PmnError("w1_gemm_swiglu_mxfp8: b holds as many gate as up rows, got %d in all" % f2)
    f, dev = f2 // 2, a[0].device
    out = _mxfp8_out(out, rows, f, dev, stream, gpu)
    if out_t is not None or want_t:
        out_t = _mxfp8_out(out_t, f, rows, dev, stream, gpu, "out_t")
    if y is not None:
        _shaped(y, (rows, f2), torch.bfloat16, "y", gpu)
    elif want_y:
        y = _empty((rows, f2), torch.bfloat16, dev, stream)
    t, tsc = out_t if out_t is not None else (None, None)
    raw = _launch_stream("w1_gemm_swiglu_mxfp8", stream, gpu)
    _check(lib().pmn_w1_gemm_swiglu_mxfp8(_at(a[0]), _at(a[1]), _at(b[0]), _at(b[1]), _at(offsets), experts,
                                          rows, f, k, _at(out[0]), _at(out[1]), _at(t), _at(tsc), _at(y), raw),
           "w1_gemm_swiglu_mxfp8")
    return out, out_t, y


def dh_gemm_swiglu_backward_mxfp8(a, b, y, offsets, out=None, out_t=None, stream=None):
    """Backward of the gated projection as far as its pre-activations: dH = dY . W2, then MXFP8 of dY1 =
    [dgate | dup] and of dY1^T.

    a = MXFP8 dY (u8 [T, D], u8 [T, D/32]); b = MXFP8 W2^T (u8 [E, F, D], u8 [E, F, D/32]); y = bf16 [T, 2F] of the
    forward.  Returns ((u8 [T, 2F], u8 [T, 2F/32]), (u8 [2F, T], u8 [2F, T/32])): the operands of the dX and dW1
    GEMMs.  offsets and T are multiples of 32."""
    gpu = torch._C._cuda_getDevice()
    rows, k, experts, f = _gated_operands(a, b, offsets, "dh_gemm_swiglu_backward_mxfp8", gpu)
    _shaped(y, (rows, 2 * f), torch.bfloat16, "y", gpu)
    dev = a[0].device
    out = _mxfp8_out(out, rows, 2 * f, dev, stream, gpu)
    out_t = _mxfp8_out(out_t, 2 * f, rows, dev, stream, gpu, "out_t")
    raw = _launch_stream("dh_gemm_swiglu_backward_mxfp8", stream, gpu)
    _check(lib().pmn_dh_gemm_swiglu_backward_mxfp8(_at(a[0]), _at(a[1]), _at(b[0]), _at(b[1]), _at(y),
                                                   _at(offsets), experts, rows, f, k, _at(out[0]), _at(out[1]),
                                                   _at(out_t[0]), _at(out_t[1]), raw),
           "dh_gemm_swiglu_backward_mxfp8")
    return out, out_t


class AdamWTensors:
    """The tensors of adamw_step, checked and laid out once.

    params: GPU tensors, all bf16 or all float32; grads: all bf16 or all float32, of the same lengths; m, v: float32
    tensors, or (uint8 E4M3, uint8 E8M0 per 32) pairs of m and of sqrt(v) -- adamw_states() makes zero ones; copies:
    bf16 tensors that receive the updated float32 params, or None.  Any shapes; the kernels see flat tensors.  The
    object keeps references to the tensors, and their storage must stay where it is: a loop whose gradients get new
    storage every step makes a new object every step (4 us a tensor on the host)."""

    def __init__(self, params, grads, m, v, copies=None):
        params, grads, m, v = list(params), list(grads), list(m), list(v)
        copies = [None] * len(params) if copies is None else list(copies)
        if len({len(params), len(grads), len(m), len(v), len(copies)}) != 1:
            raise PmnError("AdamWTensors: lists of different lengths")
        kinds = {(_kind(p, "param"), _kind(g, "grad"), isinstance(a, (tuple, list)), isinstance(b, (tuple, list)))
                 for p, g, a, b in zip(params, grads, m, v)}
        if len(kinds) > 1 or any(a != b for _, _, a, b in kinds):
            raise PmnError("AdamWTensors: one type of params, one of grads and one of states")
        self.param_kind, self.grad_kind, eight, _ = next(iter(kinds), (OUT_F32, OUT_F32, False, False))
        self.state_kind = STATE_MXFP8 if eight else STATE_F32
        self.table = (AdamWTensor * max(1, len(params)))()
        self.count = len(params)
        self.device = params[0].get_device() if params else None  # of every tensor
        self.tensors = (params, grads, m, v, copies)
        for t, p, g, a, b, c in zip(self.table, params, grads, m, v, copies):
            n = p.numel()
            q = list(a) + list(b) if eight else [a, b]
            sizes = [n, (n + 31) // 32, n, (n + 31) // 32] if eight else [n, n]
            if len(q) != len(sizes):
                raise PmnError("AdamWTensors: an MXFP8 state is a (values, scales) pair")
            for x, k in zip(q, sizes):
                _dev(x, torch.uint8 if eight else torch.float32)
                if x.numel() != k:
                    raise PmnError("AdamWTensors: a state has %d elements, expected %d" % (x.numel(), k))
            _dev(p), _dev(g)
            if g.numel() != n or (c is not None and (_dev(c, torch.bfloat16).numel() != n or p.dtype != torch.float32)):
                raise PmnError("AdamWTensors: grads and copies have their params' lengths, copies are of float32 params")
            if any(x is not None and x.get_device() != self.device for x in [p, g, c] + q):
                raise PmnError("AdamWTensors: tensors of one step on one GPU")
            t.param, t.grad, t.n = p.data_ptr(), g.data_ptr(), n
            t.copy = None if c is None else c.data_ptr()
            if eight:
                t.m, t.m_scales, t.v, t.v_scales = [x.data_ptr() for x in q]
            else:
                t.m, t.v = [x.data_ptr() for x in q]


def adamw_states(params, mxfp8=False):
    """Zero states (m, v) for AdamWTensors: float32, or (E4M3, E8M0) pairs (byte 0 is the value 0)."""
    def one(p):
        n = p.numel()
        if not mxfp8:
            return torch.zeros((n,), dtype=torch.float32, device=p.device)
        return (torch.zeros((n,), dtype=torch.uint8, device=p.device),
                torch.zeros(((n + 31) // 32,), dtype=torch.uint8, device=p.device))
    return [one(p) for p in params], [one(p) for p in params]


def adamw_step(tensors, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, seed=0, grad_scale=None,
               stream=None):
    """One AdamW step (decoupled weight decay) over the tensors of an AdamWTensors object, in place; step counts
    from 1.  grad_scale: None, or a float32 GPU tensor of one element that the gradients are multiplied by.  bf16
    params and MXFP8 states are rounded stochastically with bits that follow from seed, step and position."""
    gpu = torch._C._cuda_getDevice()
    if tensors.device not in (None, gpu):
        raise PmnError("adamw_step: the tensors are on cuda:%d, the current GPU is cuda:%d" % (tensors.device, gpu))
    if grad_scale is not None:
        if grad_scale.numel() != 1:
            raise PmnError("grad_scale must have one element")
        _shaped(grad_scale, grad_scale.shape, torch.float32, "grad_scale", gpu)
    raw = _launch_stream("adamw_step", stream, gpu)
    _check(lib().pmn_adamw_step(tensors.table, tensors.count, tensors.param_kind, tensors.grad_kind,
                                tensors.state_kind, lr, beta1, beta2, eps, weight_decay, step, _at(grad_scale),
                                seed, raw),
           "adamw_step")
