"""Binding of the C ABI declared in include/tg_gemm.h, through ctypes and, for
what a layer calls several times a step, through csrc/calls.c where it was built.

Argument marshalling only: every step of the GEMM runs in the CUDA kernels
of ``libtg_gemm.so``.  Torch is used for device memory and streams.  If the
library is missing, the first call raises; there is no fallback.
"""
import contextlib
import ctypes
import os
import threading

LIB_NAME = "libtg_gemm.so"
_HERE = os.path.dirname(os.path.abspath(__file__))

EPI_NONE, EPI_RELU = 0, 1
F32_FFMA, F32_TF32 = 0, 1

STATUS = {0: "TG_OK", 1: "TG_ERR_INVALID_ARG", 2: "TG_ERR_ALIGNMENT",
          3: "TG_ERR_UNSUPPORTED", 4: "TG_ERR_CUDA", 5: "TG_ERR_TIMEOUT",
          6: "TG_ERR_NO_DEVICE"}

# Every symbol include/tg_gemm.h declares.
EXPORTS = ("tg_gemm_f32", "tg_gemm_f16", "tg_gemm_bf16", "tg_gemm_w4a16", "tg_gemm_wfp4",
           "tg_gemm_f16_ex", "tg_gemm_bf16_ex", "tg_gemm_bf16_small_m_static",
           "tg_gemm_sp24_f16", "tg_gemm_sp24_bf16",
           "tg_quant_i8", "tg_gemm_w8a8", "tg_gemm_grouped_f16", "tg_gemm_grouped_bf16",
           "tg_gemm_grouped_wgrad_f16", "tg_gemm_grouped_wgrad_bf16", "tg_gemm_grouped_w8a8",
           "tg_expert_sort_scratch", "tg_expert_sort", "tg_expert_gather", "tg_expert_combine",
           "tg_expert_combine_grad",
           "tg_quant_mxfp4", "tg_dequant_mxfp4", "tg_expert_quant_mxfp4", "tg_gemm_mxfp4",
           "tg_gemm_grouped_mxfp4", "tg_expert_route", "tg_expert_route_grad",
           "tg_tune_set", "tg_tune_builtin", "tg_tune_query",
           "tg_status_string", "tg_last_device_status", "tg_num_sms")

# Tuning table (include/tg_gemm.h: tg_tune_rule): operations and kernel paths.
OPS = {"bf16": 0, "f16": 1, "w4a16": 2, "wfp4": 3, "f32_ffma": 4, "f32_tf32": 5}
PATHS = {"auto": 0, "cuda_core": 1, "small_m": 2, "cta_pair": 3, "one_cta": 4}


class TuneRule(ctypes.Structure):
    """tg_tune_rule: which kernel family and launch shape a call uses."""
    _fields_ = [("op", ctypes.c_int32), ("path", ctypes.c_int32),
                ("m_lo", ctypes.c_int64), ("m_hi", ctypes.c_int64),
                ("n_lo", ctypes.c_int64), ("n_hi", ctypes.c_int64),
                ("ctas", ctypes.c_int32), ("group_m", ctypes.c_int32),
                ("splits", ctypes.c_int32), ("stages", ctypes.c_int32)]

_lib = None
_lock = threading.Lock()


class TgError(RuntimeError):
    """A non-OK tg_status returned by the library."""

    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}")


def lib_path():
    return os.path.join(_HERE, LIB_NAME)


def load_library():
    """Load libtg_gemm.so (built in-tree) and declare its signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = lib_path()
        if not os.path.exists(path):
            raise ImportError(f"{LIB_NAME} is not built (expected at {path}); "
                              "run tiled_dense_gemm_tma_b200/build.py")
        lib = ctypes.CDLL(path)
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        lib.tg_gemm_f32.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, ci, ci, vp]
        for name in ("tg_gemm_f16", "tg_gemm_bf16", "tg_gemm_bf16_small_m_static"):
            getattr(lib, name).argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, ci, vp]
        for name in ("tg_gemm_w4a16", "tg_gemm_wfp4"):
            getattr(lib, name).argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, ci,
                                           vp, i64, ci, vp]
        for name in ("tg_gemm_sp24_f16", "tg_gemm_sp24_bf16"):
            getattr(lib, name).argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, ci, vp]
            getattr(lib, name).restype = ci
        for name in ("tg_gemm_f16_ex", "tg_gemm_bf16_ex"):
            getattr(lib, name).argtypes = [i64, i64, i64, vp, i64, ci, vp, i64, ci, vp, i64, ci, vp]
        for name in ("tg_gemm_f32", "tg_gemm_f16", "tg_gemm_bf16", "tg_gemm_w4a16",
                     "tg_gemm_wfp4", "tg_gemm_f16_ex", "tg_gemm_bf16_ex",
                     "tg_gemm_bf16_small_m_static", "tg_last_device_status"):
            getattr(lib, name).restype = ci
        lib.tg_quant_i8.argtypes = [i64, i64, vp, i64, ci, vp, i64, vp, vp]
        lib.tg_gemm_w8a8.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, ci, vp, vp, i64, ci, ci, vp]
        for name in ("tg_gemm_grouped_f16", "tg_gemm_grouped_bf16"):
            getattr(lib, name).argtypes = [i64, i64, i64, ci, vp, i64, vp, vp, i64, i64, ci,
                                           vp, i64, ci, vp]
        for name in ("tg_gemm_grouped_wgrad_f16", "tg_gemm_grouped_wgrad_bf16"):
            getattr(lib, name).argtypes = [i64, i64, i64, ci, vp, i64, vp, i64, vp, vp, i64, i64, vp]
        lib.tg_gemm_grouped_w8a8.argtypes = [i64, i64, i64, ci, vp, i64, vp, vp, vp, i64, i64, ci,
                                             vp, i64, vp, i64, ci, ci, vp]
        lib.tg_expert_sort_scratch.argtypes = [i64, ci]
        lib.tg_expert_sort_scratch.restype = i64
        lib.tg_expert_sort.argtypes = [i64, ci, ci, vp, ci, vp, vp, vp, vp, vp]
        lib.tg_expert_gather.argtypes = [i64, ci, i64, ci, vp, i64, vp, vp, vp, vp, i64, vp, vp]
        lib.tg_expert_combine.argtypes = [i64, ci, i64, ci, vp, i64, vp, vp, vp, vp, i64, vp]
        lib.tg_expert_combine_grad.argtypes = [i64, ci, i64, ci, vp, i64, vp, i64, vp, vp, vp,
                                               vp, i64, vp, vp]
        lib.tg_quant_mxfp4.argtypes = [i64, i64, vp, i64, ci, vp, i64, vp, i64, vp]
        lib.tg_dequant_mxfp4.argtypes = [i64, i64, vp, i64, vp, i64, vp, i64, ci, vp]
        lib.tg_expert_quant_mxfp4.argtypes = [i64, ci, i64, vp, i64, ci, vp, vp, vp, i64, vp, i64, vp]
        lib.tg_gemm_mxfp4.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, ci, ci, vp]
        lib.tg_gemm_grouped_mxfp4.argtypes = [i64, i64, i64, ci, vp, i64, vp, i64, vp, vp, i64, i64,
                                              vp, i64, i64, vp, i64, ci, ci, vp]
        cf = ctypes.c_float
        lib.tg_expert_route.argtypes = [i64, ci, vp, i64, ci, vp, ci, ci, ci, ci, ci, cf, vp, vp, vp]
        lib.tg_expert_route_grad.argtypes = [i64, ci, vp, i64, ci, ci, ci, ci, cf, vp, vp, vp, i64, vp]
        for name in ("tg_quant_mxfp4", "tg_dequant_mxfp4", "tg_expert_quant_mxfp4", "tg_gemm_mxfp4",
                     "tg_gemm_grouped_mxfp4", "tg_expert_route", "tg_expert_route_grad"):
            getattr(lib, name).restype = ci
        for name in ("tg_quant_i8", "tg_gemm_w8a8", "tg_gemm_grouped_f16", "tg_gemm_grouped_bf16",
                     "tg_gemm_grouped_wgrad_f16", "tg_gemm_grouped_wgrad_bf16",
                     "tg_gemm_grouped_w8a8", "tg_expert_sort", "tg_expert_gather",
                     "tg_expert_combine", "tg_expert_combine_grad"):
            getattr(lib, name).restype = ci
        lib.tg_status_string.argtypes = [ci]
        lib.tg_status_string.restype = ctypes.c_char_p
        lib.tg_last_device_status.argtypes = [vp]
        lib.tg_num_sms.argtypes = []
        lib.tg_num_sms.restype = ci
        lib.tg_tune_set.argtypes = [ctypes.POINTER(TuneRule), ci]
        lib.tg_tune_set.restype = ci
        lib.tg_tune_builtin.argtypes = [ctypes.POINTER(TuneRule), ci]
        lib.tg_tune_builtin.restype = ci
        lib.tg_tune_query.argtypes = [ci, i64, i64, ctypes.POINTER(TuneRule)]
        lib.tg_tune_query.restype = ci
        _lib = lib
        return lib


def _stream_handle(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _require_cuda(device, *named):
    """Every tensor on `device`, a CUDA device: the kernels run on the device
    that holds the operands and take raw device pointers."""
    for t, n in named:
        if not t.is_cuda:
            raise ValueError(f"{n} must be a CUDA tensor")
        if t.device != device:
            raise ValueError(f"{n} is on {t.device}, the operands on {device}")


def _device_ctx(t):
    """Make t's device current for the call (the library launches on the
    current device; the default stream is that device's current stream)."""
    if not t.is_cuda:
        return contextlib.nullcontext()
    import torch
    return torch.cuda.device(t.device)


def _ld(t, name):
    """Row pitch (elements) of a row-major 2-D tensor view."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    return t.stride(0)


def _check(code, what):
    if code != 0:
        raise TgError(code, what)


def empty_out(M, N, dtype, device):
    """An M x N output view whose row pitch is a multiple of 16 bytes."""
    import torch
    per = 16 // torch.tensor([], dtype=dtype).element_size()
    ld = max(per, -(-N // per) * per)
    return torch.empty((M, ld), dtype=dtype, device=device)[:, :N]


def _mk(A, B, C, dtype, out_dtype, trans_a=False, trans_b=False):
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    M, K = A.shape[::-1] if trans_a else A.shape
    K2, N = B.shape[::-1] if trans_b else B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    for t, n in ((A, "A"), (B, "B")):
        if t.dtype != dtype:
            raise TypeError(f"{n} must be {dtype}")
    _require_cuda(A.device, (A, "A"), (B, "B"))
    if C is None:
        C = empty_out(M, N, out_dtype, A.device)
    elif C.shape != (M, N) or C.dtype != out_dtype:
        raise ValueError("C has the wrong shape or dtype")
    _require_cuda(A.device, (C, "C"))
    return M, N, K, C


def gemm_f32(A, B, C=None, relu=False, mode=F32_FFMA, stream=None):
    """C = epi(A @ B) for float32 CUDA tensors; mode F32_FFMA or F32_TF32."""
    import torch
    lib = load_library()
    M, N, K, C = _mk(A, B, C, torch.float32, torch.float32)
    with _device_ctx(A):
        code = lib.tg_gemm_f32(M, N, K, A.data_ptr(), _ld(A, "A"), B.data_ptr(), _ld(B, "B"),
                               C.data_ptr(), _ld(C, "C"), EPI_RELU if relu else EPI_NONE,
                               mode, _stream_handle(stream))
    _check(code, "tg_gemm_f32")
    return C


def _gemm16(name, dtype, A, B, C, relu, stream, trans_a, trans_b):
    lib = load_library()
    M, N, K, C = _mk(A, B, C, dtype, dtype, trans_a, trans_b)
    epi = EPI_RELU if relu else EPI_NONE
    with _device_ctx(A):
        if trans_a or trans_b:
            name += "_ex"
            code = getattr(lib, name)(M, N, K, A.data_ptr(), _ld(A, "A"), int(trans_a),
                                      B.data_ptr(), _ld(B, "B"), int(trans_b),
                                      C.data_ptr(), _ld(C, "C"), epi, _stream_handle(stream))
        else:
            code = getattr(lib, name)(M, N, K, A.data_ptr(), _ld(A, "A"), B.data_ptr(),
                                      _ld(B, "B"), C.data_ptr(), _ld(C, "C"), epi,
                                      _stream_handle(stream))
    _check(code, name)
    return C


def gemm_f16(A, B, C=None, relu=False, stream=None, trans_a=False, trans_b=False):
    """C = epi(op(A) @ op(B)) for float16 CUDA tensors, fp32 accumulation.

    op(A) = A, or A.T when trans_a (A then holds the K x M matrix); op(B) =
    B, or B.T when trans_b (B then holds N x K)."""
    import torch
    return _gemm16("tg_gemm_f16", torch.float16, A, B, C, relu, stream, trans_a, trans_b)


def gemm_bf16(A, B, C=None, relu=False, stream=None, trans_a=False, trans_b=False):
    """C = epi(op(A) @ op(B)) for bfloat16 CUDA tensors, fp32 accumulation
    (op as in gemm_f16)."""
    import torch
    return _gemm16("tg_gemm_bf16", torch.bfloat16, A, B, C, relu, stream, trans_a, trans_b)


def _row_major(t):
    return t.stride(1) == 1 or t.shape[1] <= 1


def _stored(u):
    """How the logical 2-D matrix u reaches the kernels: (storage, transposed)
    with u == storage or u == storage.T and the storage row-major.  A
    transposed view (e.g. W.T of a row-major W) needs no copy.  Where both
    readings hold, the one with a 16-byte row pitch wins, the plain one
    first; a view that is neither is copied to a contiguous tensor."""
    cands = []
    if _row_major(u) and u.stride(0) >= u.shape[1]:
        cands.append((u, False))
    v = u.t()
    if _row_major(v) and v.stride(0) >= v.shape[1]:
        cands.append((v, True))
    for st, tr in cands:
        if (st.stride(0) * st.element_size()) % 16 == 0:
            return st, tr
    if cands:
        return cands[0]
    return u.contiguous(), False


def _autograd_matmul():
    import torch

    class _Matmul(torch.autograd.Function):
        """C = A @ B on this library's 16-bit kernels, with the backward
        products dA = dC @ B^T and dB = A^T @ dC.  Every operand, the
        gradient included, is passed as it is stored: a transposed view
        becomes a transposed-operand call, not a copy."""

        @staticmethod
        def forward(ctx, A, B):
            ctx.save_for_backward(A, B)
            fn = gemm_bf16 if A.dtype == torch.bfloat16 else gemm_f16
            a, ta = _stored(A)
            b, tb = _stored(B)
            return fn(a, b, trans_a=ta, trans_b=tb)

        @staticmethod
        def backward(ctx, dC):
            A, B = ctx.saved_tensors
            fn = gemm_bf16 if A.dtype == torch.bfloat16 else gemm_f16
            g, tg = _stored(dC)
            dA = dB = None
            if ctx.needs_input_grad[0]:
                x, tx = _stored(B.t())
                dA = fn(g, x, trans_a=tg, trans_b=tx)
            if ctx.needs_input_grad[1]:
                y, ty = _stored(A.t())
                dB = fn(y, g, trans_a=ty, trans_b=tg)
            return dA, dB

    return _Matmul


_MATMUL = None


def matmul(A, B):
    """Differentiable C = A @ B for 2-D float16 / bfloat16 CUDA tensors.

    A and B may be row-major or transposed views of row-major storage (such
    as W.T for a linear layer's out x in weight W); both reach the kernels
    without a copy."""
    global _MATMUL
    if _MATMUL is None:
        _MATMUL = _autograd_matmul()
    return _MATMUL.apply(A, B)


def gemm_w4a16(A, Bq, scales, N, C=None, group_size=128, relu=False, stream=None):
    """C = epi(A @ W), W[k, n] = q[k, n] * scales[k // group_size, n].

    A: M x K float16; Bq: K x ldbq uint8 (packed, low nibble = even column);
    scales: (K // group_size) x N float16; N: number of output columns.
    """
    import torch
    lib = load_library()
    if A.dtype != torch.float16 or scales.dtype != torch.float16 or Bq.dtype != torch.uint8:
        raise TypeError("A and scales must be float16, Bq uint8")
    if A.dim() != 2 or Bq.dim() != 2 or scales.dim() != 2:
        raise ValueError("A, Bq and scales must be 2-D")
    M, K = A.shape
    if Bq.shape[0] != K:
        raise ValueError("Bq must have K rows")
    _require_cuda(A.device, (A, "A"), (Bq, "Bq"), (scales, "scales"))
    if C is None:
        C = empty_out(M, N, torch.float16, A.device)
    elif C.shape != (M, N) or C.dtype != torch.float16:
        raise ValueError("C has the wrong shape or dtype")
    _require_cuda(A.device, (C, "C"))
    with _device_ctx(A):
        code = lib.tg_gemm_w4a16(M, N, K, A.data_ptr(), _ld(A, "A"), Bq.data_ptr(),
                                 _ld(Bq, "Bq"), scales.data_ptr(), _ld(scales, "scales"),
                                 group_size, C.data_ptr(), _ld(C, "C"),
                                 EPI_RELU if relu else EPI_NONE, _stream_handle(stream))
    _check(code, "tg_gemm_w4a16")
    return C


def gemm_wfp4(A, Bq, scales, N, C=None, block_size=32, relu=False, stream=None):
    """C = epi(A @ W), W[k, n] = e2m1(code[k, n]) * 2^(scales[k // 32, n] - 127).

    A: M x K bfloat16; Bq: K x ldbq uint8 (E2M1 codes, low nibble = even
    column); scales: ceil(K / 32) x N uint8 E8M0 exponents; N: number of
    output columns.  C is M x N bfloat16.
    """
    import torch
    lib = load_library()
    if A.dtype != torch.bfloat16 or Bq.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError("A must be bfloat16, Bq and scales uint8")
    if A.dim() != 2 or Bq.dim() != 2 or scales.dim() != 2:
        raise ValueError("A, Bq and scales must be 2-D")
    M, K = A.shape
    if Bq.shape[0] != K:
        raise ValueError("Bq must have K rows")
    _require_cuda(A.device, (A, "A"), (Bq, "Bq"), (scales, "scales"))
    if C is None:
        C = empty_out(M, N, torch.bfloat16, A.device)
    elif C.shape != (M, N) or C.dtype != torch.bfloat16:
        raise ValueError("C has the wrong shape or dtype")
    _require_cuda(A.device, (C, "C"))
    with _device_ctx(A):
        code = lib.tg_gemm_wfp4(M, N, K, A.data_ptr(), _ld(A, "A"), Bq.data_ptr(), _ld(Bq, "Bq"),
                                scales.data_ptr(), _ld(scales, "scales"), block_size,
                                C.data_ptr(), _ld(C, "C"), EPI_RELU if relu else EPI_NONE,
                                _stream_handle(stream))
    _check(code, "tg_gemm_wfp4")
    return C


def gemm_sp24(Ac, E, B, C=None, relu=False, stream=None):
    """C = epi(A @ B) for a 2:4 structured-sparse A given compressed.

    Ac: M x K/2 float16 or bfloat16 (the two kept values of every chunk of 4
    consecutive k, in increasing k); E: M x ceil(K/8) uint8 position codes
    (per chunk 4 bits, bits 0-1 / 2-3 = positions of the first / second kept
    value, even chunk in the low nibble); B: K x N of Ac's dtype.  K is taken
    from B and must be a multiple of 4.
    """
    import torch
    lib = load_library()
    if Ac.dtype not in (torch.float16, torch.bfloat16) or B.dtype != Ac.dtype:
        raise TypeError("Ac and B must be float16 or bfloat16, the same")
    if E.dtype != torch.uint8:
        raise TypeError("E must be uint8")
    if Ac.dim() != 2 or E.dim() != 2 or B.dim() != 2:
        raise ValueError("Ac, E and B must be 2-D")
    K, N = B.shape
    M = Ac.shape[0]
    if Ac.shape[1] != K // 2 or E.shape[0] != M or E.shape[1] < (K + 7) // 8:
        raise ValueError("Ac must be M x K/2 and E M x ceil(K/8)")
    _require_cuda(Ac.device, (Ac, "Ac"), (E, "E"), (B, "B"))
    if C is None:
        C = empty_out(M, N, Ac.dtype, Ac.device)
    elif C.shape != (M, N) or C.dtype != Ac.dtype:
        raise ValueError("C has the wrong shape or dtype")
    _require_cuda(Ac.device, (C, "C"))
    name = "tg_gemm_sp24_bf16" if Ac.dtype == torch.bfloat16 else "tg_gemm_sp24_f16"
    with _device_ctx(Ac):
        code = getattr(lib, name)(M, N, K, Ac.data_ptr(), _ld(Ac, "Ac"), E.data_ptr(), _ld(E, "E"),
                                  B.data_ptr(), _ld(B, "B"), C.data_ptr(), _ld(C, "C"),
                                  EPI_RELU if relu else EPI_NONE, _stream_handle(stream))
    _check(code, name)
    return C


def gemm_bf16_small_m_static(A, B, C=None, relu=False, stream=None):
    """bf16 GEMM for M <= 128 whose scratch is a fixed device array of the
    library: the call never allocates device memory (C must then be given
    by a caller that cannot allocate)."""
    import torch
    lib = load_library()
    M, N, K, C = _mk(A, B, C, torch.bfloat16, torch.bfloat16)
    with _device_ctx(A):
        code = lib.tg_gemm_bf16_small_m_static(M, N, K, A.data_ptr(), _ld(A, "A"), B.data_ptr(),
                                               _ld(B, "B"), C.data_ptr(), _ld(C, "C"),
                                               EPI_RELU if relu else EPI_NONE,
                                               _stream_handle(stream))
    _check(code, "tg_gemm_bf16_small_m_static")
    return C


# ------------------------------------------------------ 8-bit linear layers

TYPE_F16, TYPE_BF16, TYPE_F32 = 0, 1, 2


def _type16(dtype, name):
    import torch
    if dtype == torch.bfloat16:
        return TYPE_BF16
    if dtype == torch.float16:
        return TYPE_F16
    raise TypeError(f"{name} must be float16 or bfloat16")


_fns = {}


def _calls():
    """What calls the entry points of the sections below: the module _tg_calls where
    it was built (a call through ctypes converts its 10 to 20 arguments in 1.5 us,
    this one in 0.2), else the library itself."""
    lib = load_library()
    try:
        from . import _tg_calls
    except ImportError:
        return _PlainCalls(lib)
    return _tg_calls


class _PlainCalls:
    """The entry points through ctypes.  What does not fit an int becomes the
    nearest that does, as in _tg_calls: ctypes would cut it to its lowest 32 bits."""

    def __init__(self, lib):
        self._library = lib

    def __getattr__(self, name):
        fn = getattr(self._library, name)
        narrow = [kind is ctypes.c_int for kind in fn.argtypes]

        def call(*args):
            return fn(*[max(-1 << 31, min((1 << 31) - 1, a)) if n else a for a, n in zip(args, narrow, strict=True)])

        setattr(self, name, call)
        return call


def _launch(name, device, stream, *args):
    """Call the entry point on `device` (made current where it is not) and on
    `stream`, by default that device's current stream; raise on an error.  The
    calls of this section go through here: they are made once per layer and
    token step, where the host's time per call is what a user waits for."""
    fn = _fns.get(name)
    if fn is None:
        import torch
        _fns["stream"], _fns["device"] = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        fn = _fns[name] = getattr(_calls(), name)
    index = device.index
    if stream is None:
        stream = _fns["stream"](index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _fns["device"]() == index:
        code = fn(*args, stream)
    else:
        import torch
        with torch.cuda.device(index):
            code = fn(*args, stream)
    if code:
        raise TgError(code, name)


def _rows_out(M, N, dtype, device):
    """(a new M x N tensor, its row pitch), the pitch a multiple of 16 bytes.
    empty_strided is the cheapest of torch's allocations on the host."""
    import torch
    per = 16 // dtype.itemsize
    ld = max(per, -(-N // per) * per)
    return torch.empty_strided((M, N), (ld, 1), dtype=dtype, device=device), ld


def _vector_out(n, dtype, device):
    import torch
    return torch.empty_strided((n,), (1,), dtype=dtype, device=device)


def _pitch(t, name):
    """Row pitch (elements) of a row-major 2-D tensor or of the matrices of a
    3-D one; for fewer than two rows, whose stride says nothing, the row
    length rounded up to 16 bytes."""
    shape, strides = t.shape, t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    if shape[-2] > 1:
        return strides[-2]
    per = 16 // t.element_size()
    return max(per, -(-shape[-1] // per) * per)


def _plane(t):
    """Elements between the matrices of a 3-D tensor."""
    return t.stride(0) if t.shape[0] > 1 else 0


def _one_device(device, tensors, names):
    """As _require_cuda, naming the tensors only where something is wrong."""
    for t in tensors:
        if t.device != device or not t.is_cuda:
            _require_cuda(device, *zip(tensors, names.split(", ")))


def _vector(t, n, dtype, name):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n}")


def _memory_of(stream, device):
    """Allocate for `stream`, not the current one: a block that is free on the
    current stream may still be in use there when another one writes it."""
    import torch
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device) if stream
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


def _out(C, M, N, dtype, device, stream):
    """(C, its row pitch), C made for `stream` where it is None."""
    if C is None:
        if stream is None:
            return _rows_out(M, N, dtype, device)
        with _memory_of(stream, device):
            return _rows_out(M, N, dtype, device)
    if C.shape != (M, N) or C.dtype != dtype:
        raise ValueError("C has the wrong shape or dtype")
    return C, _pitch(C, "C")


def quant_i8(X, Q=None, scales=None, stream=None):
    """Rows of X (M x K, float16 / bfloat16) to signed 8-bit integers with one
    float32 scale per row: scale = max|x| / 127, q = round(x * 127 / max|x|),
    ties to even.  Returns (Q, scales).  A row of zeros gets scale 0; a row
    with an infinity or a NaN gets scale NaN."""
    import torch
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    kind = _type16(X.dtype, "X")
    M, K = X.shape
    device = X.device
    if Q is None:
        Q, ldq = _out(None, M, K, torch.int8, device, stream)
    elif Q.shape != (M, K) or Q.dtype != torch.int8:
        raise ValueError("Q has the wrong shape or dtype")
    else:
        ldq = _pitch(Q, "Q")
    if scales is None:
        if stream is None:
            scales = _vector_out(M, torch.float32, device)
        else:
            with _memory_of(stream, device):
                scales = _vector_out(M, torch.float32, device)
    else:
        _vector(scales, M, torch.float32, "scales")
    _one_device(device, (Q, scales), "Q, scales")
    _launch("tg_quant_i8", device, stream, M, K, X.data_ptr(), _pitch(X, "X"), kind,
            Q.data_ptr(), ldq, scales.data_ptr())
    return Q, scales


def gemm_w8a8(A, row_scales, B, col_scales, C=None, out_dtype=None, relu=False, stream=None,
              trans_b=False):
    """C = epi((A @ W) * row_scales[:, None] * col_scales) for int8 A (M x K)
    and W: B is K x N, or N x K with trans_b.  The scales are float32 vectors
    of M and N.  C is float16 or bfloat16 (out_dtype, by default C's or
    bfloat16).  A NaN (of a row's scale) stays one, also with relu."""
    import torch
    if A.dtype != torch.int8 or B.dtype != torch.int8:
        raise TypeError("A and B must be int8")
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    M, K = A.shape
    if trans_b:
        N, K2 = B.shape
    else:
        K2, N = B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    _vector(row_scales, M, torch.float32, "row_scales")
    _vector(col_scales, N, torch.float32, "col_scales")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if C is None else C.dtype
    kind = _type16(out_dtype, "C")
    device = A.device
    C, ldc = _out(C, M, N, out_dtype, device, stream)
    _one_device(device, (B, row_scales, col_scales, C), "B, row_scales, col_scales, C")
    _launch("tg_gemm_w8a8", device, stream, M, N, K, A.data_ptr(), _pitch(A, "A"),
            row_scales.data_ptr(), B.data_ptr(), _pitch(B, "B"), int(trans_b),
            col_scales.data_ptr(), C.data_ptr(), ldc, kind, EPI_RELU if relu else EPI_NONE)
    return C


# ------------------------------------------------------- experts' operators

class ExpertPlan:
    """Where expert_sort put each choice.

    offsets: int32 [E + 1], the rows of expert e are offsets[e]:offsets[e + 1],
    dropped choices follow from offsets[E] on; pos: int32 [tokens, topk], the
    row of each choice; src: int32 [tokens * topk], the flat choice of each
    row (None where a plan is made by hand: nothing here reads it)."""
    __slots__ = ("_offsets", "_pos", "_src")

    def __init__(self, offsets, pos, src=None):
        import torch
        if offsets.dtype != torch.int32 or pos.dtype != torch.int32:
            raise TypeError("a plan's tensors must be int32")
        if offsets.dim() != 1 or offsets.shape[0] < 2 or pos.dim() != 2 or pos.shape[1] < 1 or \
                not offsets.is_contiguous() or not pos.is_contiguous():
            raise ValueError("a plan has a vector of offsets and a tokens x topk matrix pos, "
                             "both contiguous")
        _one_device(offsets.device, (pos,), "pos")
        self._offsets, self._pos, self._src = offsets, pos, src

    @property
    def offsets(self):
        return self._offsets

    @property
    def pos(self):
        return self._pos

    @property
    def src(self):
        return self._src

    @property
    def num_experts(self):
        return self._offsets.shape[0] - 1

    @property
    def tokens(self):
        return self._pos.shape[0]

    @property
    def topk(self):
        return self._pos.shape[1]

    def _kept(self):
        """Address of the number of kept choices."""
        o = self._offsets
        return o.data_ptr() + 4 * (o.shape[0] - 1)


_scratch = {}            # bytes of scratch the sort asks for, by size


def expert_sort(ids, num_experts):
    """Stable sort of the choices ids (tokens x topk, int32 or int64) by
    expert, as an ExpertPlan.  Numbers outside 0..num_experts - 1 are dropped
    choices."""
    import torch
    if ids.dim() != 2:
        raise ValueError("ids must be 2-D (tokens x topk)")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be int32 or int64")
    device = ids.device
    _one_device(device, (ids,), "ids")
    T, k = ids.shape
    if k < 1:
        raise ValueError("ids must hold at least one choice per token")
    n = T * k
    need = _scratch.get((n, num_experts))
    if need is None:
        if len(_scratch) > 1000:
            _scratch.clear()
        need = load_library().tg_expert_sort_scratch(n, num_experts)
        _scratch[n, num_experts] = need
    if need < 0:
        raise ValueError("expert_sort takes 1 to 1024 experts and fewer than 2^31 choices")
    ids = ids.contiguous()
    # one allocation, each part on a 16-byte boundary: offsets, pos, src, scratch
    E1 = num_experts + 1
    at_pos = -(-E1 // 4) * 4
    at_src = at_pos + -(-n // 4) * 4
    at_scratch = at_src + -(-n // 4) * 4
    buf = _vector_out(at_scratch + need // 4, torch.int32, device)
    base = buf.data_ptr()
    _launch("tg_expert_sort", device, None, T, k, num_experts, ids.data_ptr(), ids.element_size(),
            base, base + 4 * at_pos, base + 4 * at_src, base + 4 * at_scratch if need else None)
    plan = ExpertPlan.__new__(ExpertPlan)
    plan._offsets = buf[:E1]
    plan._pos = buf.as_strided((T, k), (k, 1), at_pos)
    plan._src = buf[at_src:at_src + n]
    return plan


def _gather(X, plan, scales=None):
    import torch
    pos = plan._pos
    T, k = pos.shape
    if X.dim() != 2 or X.shape[0] != T:
        raise ValueError("X must have one row per token of the plan")
    if X.dtype not in (torch.float16, torch.bfloat16, torch.int8):
        raise TypeError("X must be float16, bfloat16 or int8")
    X = _aligned_rows(X)
    H, device = X.shape[1], X.device
    out, ldo = _rows_out(T * k, H, X.dtype, device)
    ss = None
    if scales is not None:
        _vector(scales, T, torch.float32, "scales")
        ss = _vector_out(T * k, torch.float32, device)
        _one_device(device, (scales,), "scales")
    _one_device(device, (pos,), "the plan")
    _launch("tg_expert_gather", device, None, T, k, H, X.element_size(), X.data_ptr(),
            _pitch(X, "X"), None if ss is None else scales.data_ptr(), pos.data_ptr(),
            plan._kept(), out.data_ptr(), ldo, None if ss is None else ss.data_ptr())
    return out if ss is None else (out, ss)


def _check_weights(weights, T, k, device):
    import torch
    if weights.dtype != torch.float32:
        raise TypeError("weights must be float32")
    if weights.shape != (T, k):
        raise ValueError("weights must be tokens x topk")
    _one_device(device, (weights,), "weights")
    return weights.contiguous()


def _combine(Y, plan, weights):
    pos = plan._pos
    T, k = pos.shape
    if Y.dim() != 2 or Y.shape[0] != T * k:
        raise ValueError("the sorted rows must be one per choice of the plan")
    kind = _type16(Y.dtype, "the sorted rows")
    Y = _aligned_rows(Y)
    H, device = Y.shape[1], Y.device
    if weights is not None:
        weights = _check_weights(weights, T, k, device)
    out, ldo = _rows_out(T, H, Y.dtype, device)
    _one_device(device, (pos,), "the plan")
    _launch("tg_expert_combine", device, None, T, k, H, kind, Y.data_ptr(), _pitch(Y, "Y"),
            pos.data_ptr(), plan._kept(), None if weights is None else weights.data_ptr(),
            out.data_ptr(), ldo)
    return out


def _combine_grad(Y, weights, g, plan):
    import torch
    pos = plan._pos
    T, k = pos.shape
    H, device = Y.shape[1], Y.device
    weights = weights.contiguous()
    dY, ldd = _rows_out(T * k, H, Y.dtype, device)
    dw = torch.empty_strided((T, k), (k, 1), dtype=torch.float32, device=device)
    _one_device(device, (g,), "the gradient")
    _launch("tg_expert_combine_grad", device, None, T, k, H, _type16(Y.dtype, "Y"), Y.data_ptr(),
            _pitch(Y, "Y"), g.data_ptr(), _pitch(g, "the gradient"), pos.data_ptr(), plan._kept(),
            weights.data_ptr(), dY.data_ptr(), ldd, dw.data_ptr())
    return dY, dw


def _aligned_rows(t):
    """Rows as the kernels take them: t itself where it is row-major with a
    16-byte pitch and base, else a copy.  Autograd hands out expanded and
    oddly pitched gradients that the caller has no say in, and an elementwise
    operation between two of the differentiable operators gives a dense result
    for a pitched one."""
    (rows, cols), (down, across) = t.shape, t.stride()
    if (across == 1 or cols <= 1) and t.data_ptr() % 16 == 0 and \
            (rows <= 1 or (down >= cols and down * t.element_size() % 16 == 0)):
        return t
    out, _ = _rows_out(rows, cols, t.dtype, t.device)
    return out.copy_(t)


def _offsets_of(groups):
    import torch
    if isinstance(groups, ExpertPlan):
        return groups._offsets
    offsets = groups
    if offsets.dtype != torch.int32:
        raise TypeError("offsets must be int32")
    if offsets.dim() != 1 or offsets.shape[0] < 2 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous vector of E + 1")
    return offsets


def gemm_grouped(A, groups, B, C=None, relu=False, stream=None, trans_b=False):
    """C[r] = epi(A[r] @ W[e]) for the rows r of group e: A is M x K (float16
    or bfloat16), W is B (E x K x N), or with trans_b stored E x N x K; groups
    is an ExpertPlan or its offsets.  Rows behind the last group are zero."""
    offsets = _offsets_of(groups)
    E = offsets.shape[0] - 1
    kind = _type16(A.dtype, "A")
    if B.dtype != A.dtype:
        raise TypeError("A and B must have one dtype")
    if A.dim() != 2 or B.dim() != 3 or B.shape[0] != E:
        raise ValueError("A must be 2-D and B one matrix per group")
    M, K = A.shape
    K2, N = (B.shape[2], B.shape[1]) if trans_b else B.shape[1:]
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    device = A.device
    C, ldc = _out(C, M, N, A.dtype, device, stream)
    _one_device(device, (B, offsets, C), "B, offsets, C")
    name = "tg_gemm_grouped_bf16" if kind == TYPE_BF16 else "tg_gemm_grouped_f16"
    _launch(name, device, stream, M, N, K, E, A.data_ptr(), _pitch(A, "A"), offsets.data_ptr(),
            B.data_ptr(), _pitch(B, "B"), _plane(B), int(trans_b), C.data_ptr(), ldc,
            EPI_RELU if relu else EPI_NONE)
    return C


def gemm_grouped_wgrad(A, G, groups, C=None, stream=None):
    """C[e] = A_e^T @ G_e over the rows of each group (float16 or bfloat16, A
    M x K, G M x N, C E x K x N): the gradient of gemm_grouped's W for the
    gradient G of its rows.  A group without rows gets zeros."""
    import torch
    offsets = _offsets_of(groups)
    E = offsets.shape[0] - 1
    kind = _type16(A.dtype, "A")
    if G.dtype != A.dtype:
        raise TypeError("A and G must have one dtype")
    if A.dim() != 2 or G.dim() != 2 or A.shape[0] != G.shape[0]:
        raise ValueError("A and G must be 2-D with the same rows")
    (M, K), N = A.shape, G.shape[1]
    if C is None:
        per = 16 // A.element_size()
        ld = max(per, -(-N // per) * per)
        with contextlib.nullcontext() if stream is None else _memory_of(stream, A.device):
            C = torch.empty_strided((E, K, N), (K * ld, ld, 1), dtype=A.dtype, device=A.device)
    elif C.shape != (E, K, N) or C.dtype != A.dtype:
        raise ValueError("C has the wrong shape or dtype")
    _one_device(A.device, (G, offsets, C), "G, offsets, C")
    name = "tg_gemm_grouped_wgrad_bf16" if kind == TYPE_BF16 else "tg_gemm_grouped_wgrad_f16"
    _launch(name, A.device, stream, M, N, K, E, A.data_ptr(), _pitch(A, "A"), G.data_ptr(),
            _pitch(G, "G"), offsets.data_ptr(), C.data_ptr(), _pitch(C, "C"), _plane(C))
    return C


def gemm_grouped_w8a8(A, row_scales, groups, B, col_scales, C=None, out_dtype=None, relu=False,
                      stream=None, trans_b=False):
    """gemm_grouped on 8-bit rows and weights: int8 A (M x K) with float32
    row_scales (M), int8 B (E x K x N, or E x N x K with trans_b) with float32
    col_scales (E x N); sum and scales as gemm_w8a8."""
    import torch
    offsets = _offsets_of(groups)
    E = offsets.shape[0] - 1
    if A.dtype != torch.int8 or B.dtype != torch.int8:
        raise TypeError("A and B must be int8")
    if A.dim() != 2 or B.dim() != 3 or B.shape[0] != E:
        raise ValueError("A must be 2-D and B one matrix per group")
    M, K = A.shape
    K2, N = (B.shape[2], B.shape[1]) if trans_b else B.shape[1:]
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    _vector(row_scales, M, torch.float32, "row_scales")
    if col_scales.dtype != torch.float32:
        raise TypeError("col_scales must be float32")
    if col_scales.shape != (E, N) or (N > 1 and col_scales.stride(1) != 1):
        raise ValueError("col_scales must be one row-major row of N per group")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if C is None else C.dtype
    kind = _type16(out_dtype, "C")
    device = A.device
    C, ldc = _out(C, M, N, out_dtype, device, stream)
    _one_device(device, (B, row_scales, col_scales, offsets, C), "B, row_scales, col_scales, offsets, C")
    _launch("tg_gemm_grouped_w8a8", device, stream, M, N, K, E, A.data_ptr(), _pitch(A, "A"),
            row_scales.data_ptr(), offsets.data_ptr(), B.data_ptr(), _pitch(B, "B"), _plane(B),
            int(trans_b), col_scales.data_ptr(), _plane(col_scales), C.data_ptr(), ldc, kind,
            EPI_RELU if relu else EPI_NONE)
    return C


def _stored3(W):
    """How the logical E x K x N weights reach the kernels: (storage,
    transposed) with W[e] == storage[e] or its transpose and the storage's
    matrices row-major; a view that is neither is copied.  Where both readings
    hold, the one with a 16-byte row pitch wins, the plain one first."""
    if W.dim() != 3:
        raise ValueError("W must be 3-D (experts x K x N)")
    E, K, N = W.shape
    se, sk, sn = W.stride()
    apart = E <= 1 or se > 0
    plain = apart and (sn == 1 or N <= 1) and (K <= 1 or sk >= N)
    trans = apart and (sk == 1 or K <= 1) and (N <= 1 or sn >= K)
    per = 16 // W.element_size()
    if plain and (K <= 1 or sk % per == 0):
        return W, False
    if trans and (N <= 1 or sn % per == 0):
        return W.transpose(1, 2), True
    if plain:
        return W, False
    if trans:
        return W.transpose(1, 2), True
    return _pitched_copy3(W), False


def _aligned3(w):
    """Row-major matrices as the kernels take them: w itself, or a copy where
    its base, row pitch or plane is no multiple of 16 bytes."""
    per = 16 // w.element_size()
    E, rows, _ = w.shape
    plane, down, _ = w.stride()
    if w.data_ptr() % 16 or (rows > 1 and down % per) or (E > 1 and plane % per):
        return _pitched_copy3(w)
    return w


def _pitched_copy3(W):
    """A row-major copy whose row pitch is a multiple of 16 bytes."""
    import torch
    per = 16 // W.element_size()
    E, K, N = W.shape
    ld = -(-N // per) * per
    copy = torch.empty_strided((E, K, N), (K * ld, ld, 1), dtype=W.dtype, device=W.device)
    return copy.copy_(W)


def _product_grads(A, W, offsets, g, needed):
    """The gradients of expert_matmul from operands of any layout."""
    A = _aligned_rows(A)
    w, tr = _stored3(W)
    w = _aligned3(w)
    dA = gemm_grouped(g, offsets, w, trans_b=not tr) if needed[0] else None
    dW = None
    if needed[1]:
        dW = (gemm_grouped_wgrad(g, A, offsets).transpose(1, 2) if tr
              else gemm_grouped_wgrad(A, g, offsets))
    return dA, dW, None


def _expert_functions():
    import torch

    def once():
        # a backward that itself records a graph would lose the kernels' part
        if torch.is_grad_enabled():
            raise RuntimeError("the experts' operators are differentiable once")

    class _Gather(torch.autograd.Function):
        """Xs[pos[i]] = X[i // topk]; the gradient adds each token's rows."""

        @staticmethod
        def forward(ctx, X, plan):
            ctx.plan = plan
            ctx.save_for_backward(plan._offsets, plan._pos)      # for the check on changes in place
            return _gather(X, plan)

        @staticmethod
        def backward(ctx, g):
            once()
            ctx.saved_tensors
            return _combine(g, ctx.plan, None), None

    class _Combine(torch.autograd.Function):
        """Y[t] = sum_j w[t, j] Ys[pos[t, j]], with both gradients."""

        @staticmethod
        def forward(ctx, Ys, weights, plan):
            ctx.plan = plan
            ctx.save_for_backward(Ys if weights is not None else None, weights, plan._offsets,
                                  plan._pos)
            return _combine(Ys, plan, weights)

        @staticmethod
        def backward(ctx, g):
            once()
            Ys, weights, _, _ = ctx.saved_tensors
            if weights is None:
                return _gather(g, ctx.plan), None, None
            dY, dw = _combine_grad(_aligned_rows(Ys), weights, _aligned_rows(g), ctx.plan)
            return (dY if ctx.needs_input_grad[0] else None,
                    dw if ctx.needs_input_grad[1] else None, None)

    class _Product(torch.autograd.Function):
        """C[r] = A[r] @ W[e], with dA = dC W[e]^T and dW[e] = A_e^T dC_e;
        the weights are read, and their gradient is written, as stored."""

        @staticmethod
        def forward(ctx, A, W, offsets):
            ctx.save_for_backward(A, W, offsets)
            w, tr = _stored3(W)
            w = _aligned3(w)
            a = _aligned_rows(A) if A.dim() == 2 else A
            C = gemm_grouped(a, offsets, w, trans_b=tr)
            # what backward reads again, as checked for the call above
            own = a is A and w.data_ptr() == W.data_ptr()
            ctx.strides = (A.stride(), W.stride()) if own else None
            ctx.layout = (C.shape[0], C.shape[1], A.shape[1], w.shape[0], _pitch(a, "A"),
                          _pitch(w, "W"), _plane(w), tr)
            return C

        @staticmethod
        def backward(ctx, g):
            once()
            A, W, offsets = ctx.saved_tensors
            g = _aligned_rows(g)
            if (A.stride(), W.stride()) != ctx.strides:
                # operands that were copied, or tensors that a saved-tensor hook gave back
                # in another layout than it took
                return _product_grads(A, W, offsets, g, ctx.needs_input_grad)
            M, N, K, E, lda, ldb, plane, tr = ctx.layout
            device, dtype = A.device, A.dtype
            ldg = _pitch(g, "the gradient")
            kind = "bf16" if dtype == torch.bfloat16 else "f16"
            dA = dW = None
            if ctx.needs_input_grad[0]:
                dA, ldd = _rows_out(M, K, dtype, device)
                _launch("tg_gemm_grouped_" + kind, device, None, M, K, N, E, g.data_ptr(), ldg,
                        offsets.data_ptr(), W.data_ptr(), ldb, plane,
                        int(not tr), dA.data_ptr(), ldd, EPI_NONE)
            if ctx.needs_input_grad[1]:
                # (A, K) and (g, N) change places for weights stored N x K
                x, ldx, k, y, ldy, n = (g, ldg, N, A, lda, K) if tr else (A, lda, K, g, ldg, N)
                ld = -(-n // 8) * 8
                dW = torch.empty_strided((E, k, n), (k * ld, ld, 1), dtype=dtype, device=device)
                _launch("tg_gemm_grouped_wgrad_" + kind, device, None, M, n, k, E, x.data_ptr(),
                        ldx, y.data_ptr(), ldy, offsets.data_ptr(), dW.data_ptr(), ld, k * ld)
                if tr:
                    dW = dW.transpose(1, 2)
            return dA, dW, None

    return _Gather, _Combine, _Product


_EXPERT = None


def _expert(i):
    global _EXPERT
    if _EXPERT is None:
        _EXPERT = _expert_functions()
    return _EXPERT[i]


def expert_gather(X, plan, scales=None):
    """The rows of X (tokens x H) sorted by expert: row plan.pos[t, j] is X[t];
    the rows of dropped choices are zero.  X is float16, bfloat16
    (differentiable) or int8; with scales (int8 rows only: float32, one per
    token) returns (rows, their scales).  Rows that are not row-major or do not
    start on 16-byte boundaries (a dense X of a width that is no multiple of 8, or
    16 for int8) are copied to such ones first."""
    if scales is not None:
        import torch
        if X.dtype != torch.int8:
            raise TypeError("scales go with int8 rows")
        return _gather(X, plan, scales)
    return _expert(0).apply(X, plan)


def expert_combine(Ys, plan, weights=None):
    """Sorted rows back to tokens: Y[t] = sum_j weights[t, j] *
    Ys[plan.pos[t, j]] over the kept choices, summed in float32 in the order of
    j.  Ys is float16 or bfloat16, weights float32 (tokens x topk; all 1 where
    None).  Differentiable in Ys and weights.  Rows that do not start on 16-byte
    boundaries are copied as in expert_gather."""
    return _expert(1).apply(Ys, weights, plan)


def expert_matmul(Xs, W, groups):
    """Differentiable experts' product: row r of group e times W[e].

    Xs: M x K sorted rows (float16 or bfloat16); W: E x K x N, or a transposed
    view of E x N x K storage (W.transpose(1, 2)), which needs no copy; groups:
    an ExpertPlan or its offsets.  Rows behind the last group are zero and get
    zero gradient.  Operands whose rows do not start on 16-byte boundaries (dense
    ones of widths that are no multiple of 8; the results here have padded rows)
    are copied first, in backward again; gemm_grouped refuses them."""
    return _expert(2).apply(Xs, W, _offsets_of(groups))


# ------------------------------------------- microscaled 4-bit floating point

# These calls are made several times a layer and token step, so that their checks
# read each property once, and say what is wrong only where something is.

_torch = None


def _get_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _row_pitch(t, rows, cols, name):
    """_pitch of a matrix of bytes (of the last two dimensions), quickly where it is
    dense and has more than one row, or one of whole 16 bytes."""
    return cols if t.is_contiguous() and (rows > 1 or (cols and cols % 16 == 0)) else _pitch(t, name)


def _check_blocks(q, scales, dims, name):
    """What is wrong with codes and their scales: uint8, `dims` dimensions, the
    same rows, one scale for every 16 bytes."""
    import torch
    if q.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError(f"{name} and its scales must be uint8")
    if q.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D")
    if q.shape[:-1] != scales.shape[:-1]:
        raise ValueError(f"{name} and its scales must have the same rows")
    if scales.shape[-1] != (q.shape[-1] + 15) // 16:
        raise ValueError(f"{name} needs one scale for every 16 bytes of a row")


def _bytes_out(t, M, N, device, name):
    """The row pitch of t, a given M x N matrix of bytes."""
    import torch
    if t.shape != (M, N) or t.dtype != torch.uint8:
        raise ValueError(f"{name} has the wrong shape or dtype")
    _one_device(device, (t,), name)
    return _pitch(t, name)


def _values_out(C, M, N, out_dtype, device, stream):
    """(C, its type, its row pitch): C made where it is None, of out_dtype, by
    default bfloat16."""
    torch = _torch or _get_torch()
    if C is None and stream is None:
        dtype = torch.bfloat16 if out_dtype is None else out_dtype
        kind = TYPE_BF16 if dtype is torch.bfloat16 else _type16(dtype, "C")
        ldc = (N + 7) // 8 * 8 or 8
        return torch.empty_strided((M, N), (ldc, 1), dtype=dtype, device=device), kind, ldc
    if out_dtype is None:
        out_dtype = torch.bfloat16 if C is None else C.dtype
    kind = _type16(out_dtype, "C")
    C, ldc = _out(C, M, N, out_dtype, device, stream)
    return C, kind, ldc


def quant_mxfp4(X, plan=None, Q=None, scales=None, stream=None):
    """Rows of X (M x K, float16 / bfloat16) to microscaled 4-bit floating
    point (MXFP4): E2M1 codes, two to a byte along the row, and an E8M0 scale for
    every 32 values, 2^(floor(log2(max|x|)) - 2); round to nearest even, above 6
    scales 6.  Returns (Q, scales), uint8 M x ceil(K / 2) and M x ceil(K / 32).  A
    block with an infinity or a NaN gets scale 255, which stands for NaN.

    With a plan of expert_sort the rows are sorted by expert on the way, as
    expert_gather does: row plan.pos[t, j] of the results is X[t], the rows of
    dropped choices are zero.  Rows of X that do not start on 16-byte boundaries
    are copied to such ones first."""
    if stream is not None:
        with _memory_of(stream, X.device):
            return _quant_mxfp4(X, plan, Q, scales, stream)
    return _quant_mxfp4(X, plan, Q, scales, None)


def _quant_mxfp4(X, plan, Q, scales, stream):
    torch = _torch or _get_torch()
    dtype = X.dtype
    kind = TYPE_BF16 if dtype is torch.bfloat16 else _type16(dtype, "X")
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    M, K = X.shape
    device = X.device
    rows = M
    if plan is not None:
        T, k = plan._pos.shape
        if M != T:
            raise ValueError("X must have one row per token of the plan")
        rows = T * k
        _one_device(device, (plan._pos,), "the plan")
    if not X.is_cuda:
        _require_cuda(device, (X, "X"))
    at = X.data_ptr()
    if K % 8 == 0 and at % 16 == 0 and X.is_contiguous():
        ldx = K
    else:
        X = _aligned_rows(X)
        at, ldx = X.data_ptr(), _pitch(X, "X")
    wide, blocks = (K + 1) // 2, (K + 31) // 32
    # rows of codes on 128-byte lines, of scales on 32-byte sectors, where that adds
    # little: 3000 x 5000 x 4000 takes 41 us so, 45 with rows 2000 bytes apart
    if Q is None:
        ldq = (wide + 127) // 128 * 128 if wide > 512 else (wide + 15) // 16 * 16 or 16
        Q = torch.empty_strided((rows, wide), (ldq, 1), dtype=torch.uint8, device=device)
    else:
        ldq = _bytes_out(Q, rows, wide, device, "Q")
    if scales is None:
        lds = (blocks + 31) // 32 * 32 if blocks > 32 else (blocks + 15) // 16 * 16 or 16
        scales = torch.empty_strided((rows, blocks), (lds, 1), dtype=torch.uint8, device=device)
    else:
        lds = _bytes_out(scales, rows, blocks, device, "scales")
    if plan is None:
        _launch("tg_quant_mxfp4", device, stream, M, K, at, ldx, kind, Q.data_ptr(), ldq, scales.data_ptr(), lds)
    else:
        _launch("tg_expert_quant_mxfp4", device, stream, T, k, K, at, ldx, kind, plan._pos.data_ptr(),
                plan._kept(), Q.data_ptr(), ldq, scales.data_ptr(), lds)
    return Q, scales


def dequant_mxfp4(Q, scales, K=None, C=None, out_dtype=None, stream=None):
    """The M x K values of codes and scales as quant_mxfp4 gives them, each
    rounded once to out_dtype (float16 or bfloat16, by default C's or bfloat16).
    K defaults to all that Q holds."""
    torch = _torch or _get_torch()
    u8 = torch.uint8
    if Q.dim() != 2 or Q.dtype is not u8 or scales.dtype is not u8:
        _check_blocks(Q, scales, 2, "Q")
    M, pairs = Q.shape
    blocks = (pairs + 15) // 16
    if scales.shape != (M, blocks):
        _check_blocks(Q, scales, 2, "Q")
    if K is None:
        K = 2 * pairs
    elif (K + 1) // 2 != pairs:
        raise ValueError("Q must have ceil(K / 2) bytes a row")
    device = Q.device
    C, kind, ldc = _values_out(C, M, K, out_dtype, device, stream)
    _one_device(device, (scales, C), "scales, C")
    _launch("tg_dequant_mxfp4", device, stream, M, K, Q.data_ptr(), _row_pitch(Q, M, pairs, "Q"),
            scales.data_ptr(), _row_pitch(scales, M, blocks, "scales"), C.data_ptr(), ldc, kind)
    return C


def gemm_mxfp4(A, a_scales, B, b_scales, C=None, out_dtype=None, relu=False, stream=None):
    """C = epi(A @ W.T) for A (M x K) and the weights W (N x K), both microscaled
    4-bit floating point as quant_mxfp4 gives it: codes uint8 M x K/2 and N x
    K/2, scales uint8 M x ceil(K / 32) and N x ceil(K / 32).  fp32 accumulation; C
    is float16 or bfloat16 (out_dtype, by default C's or bfloat16).  A NaN (of a
    scale) stays one, also with relu.  Quantised rows of odd length end in a zero
    half byte, which adds nothing."""
    torch = _torch or _get_torch()
    u8 = torch.uint8
    if A.dim() != 2 or B.dim() != 2 or A.dtype is not u8 or a_scales.dtype is not u8 or \
            B.dtype is not u8 or b_scales.dtype is not u8:
        _check_blocks(A, a_scales, 2, "A")
        _check_blocks(B, b_scales, 2, "B")
    (M, pairs), (N, pairs2) = A.shape, B.shape
    if pairs != pairs2:
        raise ValueError(f"inner dimensions differ: {2 * pairs} vs {2 * pairs2}")
    blocks = (pairs + 15) // 16
    if a_scales.shape != (M, blocks) or b_scales.shape != (N, blocks):
        _check_blocks(A, a_scales, 2, "A")
        _check_blocks(B, b_scales, 2, "B")
    device = A.device
    C, kind, ldc = _values_out(C, M, N, out_dtype, device, stream)
    _same_gpu(A, a_scales, B, b_scales, C, "A, a_scales, B, b_scales, C")
    _launch("tg_gemm_mxfp4", device, stream, M, N, 2 * pairs, A.data_ptr(), _row_pitch(A, M, pairs, "A"),
            a_scales.data_ptr(), _row_pitch(a_scales, M, blocks, "a_scales"),
            B.data_ptr(), _row_pitch(B, N, pairs, "B"), b_scales.data_ptr(),
            _row_pitch(b_scales, N, blocks, "b_scales"), C.data_ptr(), ldc, kind, EPI_RELU if relu else EPI_NONE)
    return C


def gemm_grouped_mxfp4(A, a_scales, groups, B, b_scales, C=None, out_dtype=None, relu=False,
                       stream=None):
    """gemm_mxfp4 over groups of rows: row r of group e times W[e].T, the weights
    B uint8 E x N x K/2 with scales E x N x ceil(K / 32); groups is an ExpertPlan
    or its offsets.  Rows behind the last group are zero."""
    torch = _torch or _get_torch()
    u8 = torch.uint8
    offsets = _offsets_of(groups)
    E = offsets.shape[0] - 1
    if A.dim() != 2 or B.dim() != 3 or b_scales.dim() != 3 or A.dtype is not u8 or a_scales.dtype is not u8 or \
            B.dtype is not u8 or b_scales.dtype is not u8:
        _check_blocks(A, a_scales, 2, "A")
        _check_blocks(B, b_scales, 3, "B")
    (M, pairs), (E2, N, pairs2) = A.shape, B.shape
    if E2 != E:
        raise ValueError("B must hold one matrix per group")
    if pairs != pairs2:
        raise ValueError(f"inner dimensions differ: {2 * pairs} vs {2 * pairs2}")
    blocks = (pairs + 15) // 16
    if a_scales.shape != (M, blocks) or b_scales.shape != (E, N, blocks):
        _check_blocks(A, a_scales, 2, "A")
        _check_blocks(B, b_scales, 3, "B")
    device = A.device
    C, kind, ldc = _values_out(C, M, N, out_dtype, device, stream)
    _one_device(device, (offsets,), "offsets")
    _same_gpu(A, a_scales, B, b_scales, C, "A, a_scales, B, b_scales, C")
    _launch("tg_gemm_grouped_mxfp4", device, stream, M, N, 2 * pairs, E, A.data_ptr(),
            _row_pitch(A, M, pairs, "A"), a_scales.data_ptr(), _row_pitch(a_scales, M, blocks, "a_scales"),
            offsets.data_ptr(), B.data_ptr(), _row_pitch(B, N, pairs, "B"), _plane(B), b_scales.data_ptr(),
            _row_pitch(b_scales, N, blocks, "b_scales"), _plane(b_scales), C.data_ptr(), ldc, kind,
            EPI_RELU if relu else EPI_NONE)
    return C


def _same_gpu(a, b, c, d, e, names):
    """All five on a's device, a GPU."""
    index = a.get_device()
    if b.get_device() != index or c.get_device() != index or d.get_device() != index or \
            e.get_device() != index or index < 0:
        _require_cuda(a.device, *zip((a, b, c, d, e), names.split(", ")))


# ------------------------------------------------------------------ routing

SCORES = {"softmax": 0, "sigmoid": 1}


def _logits(x, T, E):
    """(x, its type, its row pitch), x copied where it is not row-major."""
    torch = _torch or _get_torch()
    dtype = x.dtype
    kind = TYPE_F32 if dtype is torch.float32 else _type16(dtype, "logits other than float32")
    if x.is_contiguous():
        return x, kind, E
    down, across = x.stride()
    if T <= 1 or E <= 1 or across != 1 or down < E:
        x = x.contiguous()
        down = E
    return x, kind, down


def _route(logits, topk, bias, score, groups, keep, renorm, scale):
    torch = _torch or _get_torch()
    T, E = logits.shape
    device = logits.device
    x, kind, ldl = _logits(logits, T, E)
    ids = torch.empty_strided((T, topk), (topk, 1), dtype=torch.int32, device=device)
    weights = torch.empty_strided((T, topk), (topk, 1), dtype=torch.float32, device=device)
    at_bias = None
    if bias is not None:
        _vector(bias, E, torch.float32, "bias")
        _one_device(device, (bias,), "bias")
        at_bias = bias.data_ptr()
    if not x.is_cuda:
        _require_cuda(device, (x, "logits"))
    _launch("tg_expert_route", device, None, T, E, x.data_ptr(), ldl, kind, at_bias, score, groups, keep,
            topk, renorm, scale, ids.data_ptr(), weights.data_ptr())
    return ids, weights


def _route_function():
    import torch
    grad_enabled = torch.is_grad_enabled

    class _Route(torch.autograd.Function):
        """Experts and weights of each token; the weights' gradient reaches the
        logits, the choice has none."""

        @staticmethod
        def forward(ctx, logits, args):
            ids, weights = _route(logits, *args)
            ctx.args = args
            ctx.save_for_backward(logits, ids)
            ctx.mark_non_differentiable(ids)
            ctx.set_materialize_grads(False)
            return ids, weights

        @staticmethod
        def backward(ctx, _, g):
            if grad_enabled():
                raise RuntimeError("the experts' operators are differentiable once")
            if g is None:
                return None, None
            logits, ids = ctx.saved_tensors
            if not ids.is_contiguous():                 # from a saved-tensor hook
                ids = ids.contiguous()
            topk, _, score, _, _, renorm, scale = ctx.args
            T, E = logits.shape
            x, kind, ldl = _logits(logits, T, E)
            if not g.is_contiguous():
                g = g.contiguous()
            device = x.device
            if g.device != device:
                _one_device(device, (g,), "the gradient")
            d = torch.empty_strided((T, E), (E, 1), dtype=x.dtype, device=device)
            _launch("tg_expert_route_grad", device, None, T, E, x.data_ptr(), ldl, kind, score, topk, renorm,
                    scale, ids.data_ptr(), g.data_ptr(), d.data_ptr(), E)
            return d, None

    return _Route.apply


_ROUTE = None


def expert_route(logits, topk, *, bias=None, score="softmax", groups=1, topk_groups=None,
                 renorm=True, scale=1.0):
    """The experts of each token and their weights from the router's logits
    (tokens x E, float32, float16 or bfloat16): (ids, weights), int32 and float32
    tokens x topk, as expert_sort and expert_combine take them.

    The scores are softmax(logits) or sigmoid(logits).  The topk highest are
    chosen in falling order, ties to the lower number; a bias (float32, E, finite
    or minus infinity) is added to the scores for the choice alone.  With groups
    (of E / groups consecutive experts) the choice is made in the topk_groups of
    them (by default all) whose two highest (biased) scores sum highest.  Weights
    are scale times the chosen scores, divided by their sum with renorm.  A logit
    or bias of minus infinity is never chosen; where fewer than topk are left, the
    rest are -1 (dropped choices) and weigh 0.  A logit of NaN or plus infinity
    makes its row's weights NaN.  At most 1024 experts, 32 choices and 32 groups.
    Differentiable in the logits."""
    global _ROUTE
    torch = _torch or _get_torch()
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D (tokens x experts)")
    kind = SCORES.get(score)
    if kind is None:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    if topk < 1:
        raise ValueError("topk must be at least 1")
    args = (topk, bias, kind, groups, groups if topk_groups is None else topk_groups, 1 if renorm else 0, scale)
    # without a graph to record, the autograd function would only cost time; inside
    # a level of forward mode it refuses a tensor that has a tangent
    if not (logits.requires_grad and torch.is_grad_enabled()) and torch.autograd.forward_ad._current_level < 0:
        return _route(logits, *args)
    if _ROUTE is None:
        _ROUTE = _route_function()
    return _ROUTE(logits, args)


def last_device_status(stream=None):
    """Synchronise the stream and return (and clear) the device status word."""
    return load_library().tg_last_device_status(_stream_handle(stream))


_MAX_I64 = (1 << 63) - 1


def _rule_of(d):
    """A TuneRule from a dict: op and path by name or number, ranges default
    to everything, knobs to 0 (the library's default)."""
    op = OPS.get(d["op"], d["op"])
    path = PATHS.get(d.get("path", 0), d.get("path", 0))
    return TuneRule(op, path, d.get("m_lo", 1), d.get("m_hi", _MAX_I64), d.get("n_lo", 1),
                    d.get("n_hi", _MAX_I64), d.get("ctas", 0), d.get("group_m", 0),
                    d.get("splits", 0), d.get("stages", 0))


def _dict_of(r):
    return {f: getattr(r, f) for f, _ in TuneRule._fields_}


def tune_set(rules):
    """Install run-time tuning rules (list of dicts, see _rule_of), consulted
    before the built-in ones; an empty list clears them."""
    lib = load_library()
    arr = (TuneRule * max(1, len(rules)))(*[_rule_of(d) for d in rules])
    _check(lib.tg_tune_set(arr, len(rules)), "tg_tune_set")


def tune_builtin():
    """The built-in tuning rules, as dicts."""
    lib = load_library()
    n = lib.tg_tune_builtin(None, 0)
    arr = (TuneRule * max(1, n))()
    lib.tg_tune_builtin(arr, n)
    return [_dict_of(arr[i]) for i in range(n)]


def tune_query(op, M, N):
    """The rule a call of `op` (name or number) with these M and N uses."""
    lib = load_library()
    r = TuneRule()
    _check(lib.tg_tune_query(OPS.get(op, op), M, N, ctypes.byref(r)), "tg_tune_query")
    return _dict_of(r)
