"""Python binding of libttq.so: the C ABI of include/ttq.h and include/ttq_kv.h,
one function per entry point with the same name.  Argument marshalling only -- every step of
the TTQ layer runs in the library's CUDA kernels; torch supplies device
memory and the current stream.  There is no fallback: if the library is
missing or the tensors are not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "libttq.so")

TTQ_OK = 0
TTQ_ERR_INVALID_ARG = 1
TTQ_ERR_UNSUPPORTED = 2
TTQ_ERR_CUDA = 3
TTQ_ERR_NONFINITE = 4
TTQ_ERR_TIMEOUT = 5
TTQ_ERR_WORKSPACE = 6

TTQ_F32 = 0
TTQ_BF16 = 1
TTQ_F16 = 2

TTQ_QSCHEME_ASYMMETRIC = 0
TTQ_QSCHEME_SYMMETRIC = 1
TTQ_QSCHEME_FP8_E4M3 = 2

TTQ_FLAG_NONFINITE = 0x1
TTQ_FLAG_SCALE_OVERFLOW = 0x2
TTQ_FLAG_TIMEOUT = 0x4
TTQ_FLAG_X_RANGE = 0x8
TTQ_FLAG_RANK_DEFICIENT = 0x10
TTQ_FLAG_BAD_INDEX = 0x20

# C signatures, in the order of include/ttq.h and include/ttq_kv.h
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [("status", _SZ), ("D", _SZ), ("D_rsqrt", _SZ), ("partial", _SZ), ("codes", _SZ),
                ("scales", _SZ), ("zeros", _SZ), ("ax", _SZ), ("xh", _SZ), ("xb", _SZ), ("ab", _SZ),
                ("wq", _SZ), ("total", _SZ), ("splits", _I64), ("ax_ld", _I64), ("axp", _SZ),
                ("D_sqrt", _SZ), ("ypart", _SZ), ("tickets", _SZ), ("ax_splits", _I64)]


class _CacheStruct(ctypes.Structure):   # ttq_kv_cache
    _fields_ = [("pages", _P), ("num_pages", _I64), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("bits", ctypes.c_int32), ("group", ctypes.c_int32),
                ("scheme", ctypes.c_int32), ("D_k", _P), ("D_v", _P), ("D_k_rsqrt", _P), ("D_v_rsqrt", _P)]


class _BatchStruct(ctypes.Structure):   # ttq_kv_batch
    _fields_ = [("page_table", _P), ("table_stride", _I64), ("kv_len", _P), ("cu_new", _P), ("batch", _I64),
                ("rows", _I64), ("max_new", _I64)]


_CACHE = ctypes.POINTER(_CacheStruct)
_BATCH = ctypes.POINTER(_BatchStruct)

SIGNATURES = {
    "ttq_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _INT, _INT, _INT]),
    "ttq_workspace_get_layout": (_INT, [_I64, _I64, _I64, _I64, _INT, _INT, _INT,
                                        ctypes.POINTER(WorkspaceLayout)]),
    "ttq_workspace_init": (_INT, [_P, _SZ, _P]),
    "ttq_act_norm": (_INT, [_P, _INT, _I64, _I64, _F, _F, _F, _P, _P, _P, _SZ, _P]),
    "ttq_act_norm_noalloc": (_INT, [_P, _INT, _I64, _I64, _F, _F, _F, _P, _P, _P]),
    "ttq_act_norm_scale": (_INT, [_P, _INT, _I64, _I64, _F, _F, _F, _P, _P, _P, _P, _SZ, _P]),
    "ttq_quantize_weight": (_INT, [_P, _INT, _I64, _I64, _P, _INT, _INT, _P, _P, _P, _P, _SZ, _P]),
    "ttq_quantize_dequant_weight": (_INT, [_P, _INT, _I64, _I64, _P, _INT, _INT, _P, _P, _P, _P, _P,
                                           _SZ, _P]),
    "ttq_quantize_weight_ex": (_INT, [_P, _INT, _I64, _I64, _P, _INT, _INT, _INT, _P, _P, _P, _P, _P,
                                      _SZ, _P]),
    "ttq_linear_forward_ex": (_INT, [_P, _P, _P, _P, _INT, _I64, _I64, _I64, _I64, _F, _F, _F, _INT,
                                     _INT, _INT, _P, _INT, _P, _SZ, _P]),
    "ttq_dequantized_gemm": (_INT, [_P, _P, _I64, _I64, _I64, _P, _INT, _P, _SZ, _P]),
    "ttq_dequantized_gemm_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "ttq_scale_activations": (_INT, [_P, _INT, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "ttq_dequant_gemm": (_INT, [_P, _P, _P, _P, _P, _P, _P, _INT, _I64, _I64, _I64, _I64, _INT, _INT,
                                _P, _INT, _P, _SZ, _P]),
    "ttq_linear_forward": (_INT, [_P, _P, _P, _P, _INT, _I64, _I64, _I64, _I64, _F, _F, _F, _INT, _INT,
                                  _P, _INT, _P, _SZ, _P]),
    "ttq_linear_forward_kernels": (_INT, [_INT, _I64, _I64, _I64, _I64, _F, _INT, _INT, _INT,
                                          ctypes.POINTER(ctypes.c_int)]),
    "ttq_testing_wait_timeout": (_INT, [_INT, ctypes.c_uint64, _INT, _P, _SZ, _P]),
    "ttq_testing_kv_page_of": (_I64, [_INT, _I64]),
    "ttq_quantize_gemm": (_INT, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _INT, _INT, _P, _P, _P,
                                 _P, _INT, _P, _SZ, _P]),
    "ttq_get_status": (_INT, [_P, ctypes.POINTER(ctypes.c_uint32)]),
    "ttq_status_from_flags": (_INT, [ctypes.c_uint32]),
    "ttq_lowrank_workspace_size": (_SZ, [_I64, _I64, _I64, _I64]),
    "ttq_lowrank_init": (_INT, [_P, _INT, _I64, _I64, _I64, _I64, _INT, _P, _P, _P, _P, _P, _SZ, _P]),
    "ttq_kv_page_bytes": (_SZ, [_INT, _INT, _INT, _INT, _INT]),
    "ttq_kv_write": (_INT, [_CACHE, _BATCH, _P, _I64, _I64, _P, _I64, _I64, _INT, _P, _SZ, _P]),
    "ttq_kv_read": (_INT, [_CACHE, _BATCH, _P, _P, _INT, _P, _SZ, _P]),
    "ttq_kv_attention_workspace_size": (_SZ, [_INT, _INT, _INT, _I64, _I64, _I64]),
    "ttq_kv_attention": (_INT, [_CACHE, _BATCH, _P, _I64, _I64, _INT, _I64, _F, _F, _I64, _P, _P, _INT, _P, _SZ,
                                _P]),
    "ttq_status_string": (ctypes.c_char_p, [_INT]),
    "ttq_version": (ctypes.c_char_p, []),
}

_lib = None


class TTQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status) if _lib else status} ({status})")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBRARY):
            raise RuntimeError(f"libttq.so not found at {LIBRARY}; build it with "
                               "`python -m test_weight_quantization_ttq_b200.build`")
        L = ctypes.CDLL(LIBRARY)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(st: int) -> str:
    return lib().ttq_status_string(int(st)).decode()


def _check(st: int, where: str) -> None:
    if st != TTQ_OK:
        raise TTQError(st, where)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TTQ_F32
    if t.dtype == torch.bfloat16:
        return TTQ_BF16
    if t.dtype == torch.float16:
        return TTQ_F16
    raise TypeError(f"unsupported dtype {t.dtype} (float32, bfloat16 or float16)")


def _dev(t: torch.Tensor | None, name: str) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    cur = torch.cuda.current_device()
    if t.device.index is not None and t.device.index != cur:
        raise ValueError(f"{name} is on {t.device}; the library runs on the current device cuda:{cur}")
    return t.data_ptr()


# The C ABI takes bare pointers and sizes, so the sizes it is given must
# describe the tensors behind the pointers: the checks below run before any
# device work and raise instead of letting a kernel read or write past a
# buffer.
_F32 = (torch.float32,)
_F16 = (torch.float16,)
_FLOAT_IN = (torch.float32, torch.bfloat16)


def _matrix(t: torch.Tensor | None, name: str, rows=None, cols=None, dtypes=None) -> None:
    """t (when given) is 2-D, rows x cols where those are given, of one of `dtypes`."""
    if t is None:
        return
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    if (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        want = (rows if rows is not None else "*", cols if cols is not None else "*")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {want}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {list(dtypes)}")


def _vector(t: torch.Tensor | None, name: str, n: int) -> None:
    """t (when given) holds exactly n float32 values (D, D^{-1/2})."""
    if t is None:
        return
    if t.dtype != torch.float32 or t.numel() != n:
        raise ValueError(f"{name} must hold {n} float32 values, got {t.numel()} {t.dtype}")


def _room(t: torch.Tensor | None, name: str, nbytes: int) -> None:
    """t (when given) spans at least nbytes (packed codes, binary16 scales)."""
    if t is None:
        return
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} spans {t.numel() * t.element_size()} bytes, needs {nbytes}")


def _qsizes(d: int, bits: int, group: int, where: str) -> tuple[int, int]:
    """(code bytes, scale bytes) of one row of W."""
    if bits < 1 or group < 1:
        raise TTQError(TTQ_ERR_INVALID_ARG, where)
    return d * bits // 32 * 4, d // group * 2


def _lowrank_pair(A: torch.Tensor | None, B: torch.Tensor | None) -> int:
    """r of the low-rank term: A [r][d] and B [d'][r] are given together."""
    if (A is None) != (B is None):
        raise ValueError("A and B of the low-rank term are given together or not at all")
    return 0 if A is None else A.shape[0]


def _nbytes(ws: torch.Tensor) -> int:
    return ws.numel() * ws.element_size()


def _stream(stream) -> int | None:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream or None


# the current stream's handle without building a torch.cuda.Stream (which
# costs 3 us, as much as a launch), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, device: int) -> int | None:
    if stream is None and _raw_stream is not None:
        return _raw_stream(device) or None
    return _stream(stream)


# ------------------------------------------------------------- workspace
def ttq_workspace_size(d, dp, T, r, bits, group, dtype=TTQ_BF16) -> int:
    return int(lib().ttq_workspace_size(d, dp, T, r, bits, group, dtype))


def ttq_workspace_get_layout(d, dp, T, r, bits, group, dtype=TTQ_BF16) -> WorkspaceLayout:
    out = WorkspaceLayout()
    _check(lib().ttq_workspace_get_layout(d, dp, T, r, bits, group, dtype, ctypes.byref(out)),
           "ttq_workspace_get_layout")
    return out


def ttq_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _check(lib().ttq_workspace_init(_dev(ws, "ws"), _nbytes(ws), _stream(stream)), "ttq_workspace_init")


def new_workspace(d, dp, T, r, bits, group, dtype=TTQ_BF16, device="cuda", stream=None) -> torch.Tensor:
    """A zero-initialised workspace (uint8 tensor) for this shape."""
    n = ttq_workspace_size(d, dp, T, r, bits, group, dtype)
    if n == 0:
        raise TTQError(TTQ_ERR_INVALID_ARG, "ttq_workspace_size")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ttq_workspace_init(ws, stream)
    return ws


def ttq_get_status(ws: torch.Tensor) -> tuple[int, int]:
    """(status, raw flag bits) of the workspace; synchronise the stream first."""
    flags = ctypes.c_uint32(0)
    st = lib().ttq_get_status(_dev(ws, "ws"), ctypes.byref(flags))
    return int(st), int(flags.value)


def ttq_status_from_flags(flags: int) -> int:
    """The status a set of TTQ_FLAG_* bits stands for (host only)."""
    return int(lib().ttq_status_from_flags(int(flags) & 0xFFFFFFFF))


# ---------------------------------------------------------- entry points
def _quant_outputs(dp, d, D, bits, group, codes, scales, zeros, W_hat, where) -> None:
    cb, sb = _qsizes(d, bits, group, where)
    _vector(D, "D", d)
    _room(codes, "codes", dp * cb)
    _room(scales, "scales", dp * sb)
    _room(zeros, "zeros", dp * sb)
    _matrix(W_hat, "W_hat", dp, d, _F16)


def ttq_act_norm(X, p, lam, alpha, ws=None, D=None, D_rsqrt=None, stream=None, copy_out=True):
    """D[i] = (||X[:, i]||_p + lambda)^alpha and D^{-1/2}; X is [T][d].
    With copy_out=False nothing is copied out: D and D^{-1/2} are returned
    as views of the workspace, where the entry point writes them."""
    _matrix(X, "X", dtypes=_FLOAT_IN)
    T, d = X.shape
    _vector(D, "D", d)
    _vector(D_rsqrt, "D_rsqrt", d)
    if ws is None:
        ws = new_workspace(d, 0, T, 0, 4, 32, _dtype_code(X), X.device, stream)
    if not copy_out:
        _check(lib().ttq_act_norm(_dev(X, "X"), _dtype_code(X), d, T, p, lam, alpha, None, None,
                                  _dev(ws, "ws"), _nbytes(ws), _stream(stream)), "ttq_act_norm")
        L = ttq_workspace_get_layout(d, 0, T, 0, 4, 32, _dtype_code(X))
        return (ws[L.D: L.D + 4 * d].view(torch.float32), ws[L.D_rsqrt: L.D_rsqrt + 4 * d].view(torch.float32))
    if D is None:
        D = torch.empty(d, dtype=torch.float32, device=X.device)
    if D_rsqrt is None:
        D_rsqrt = torch.empty(d, dtype=torch.float32, device=X.device)
    _check(lib().ttq_act_norm(_dev(X, "X"), _dtype_code(X), d, T, p, lam, alpha, _dev(D, "D"),
                              _dev(D_rsqrt, "D_rsqrt"), _dev(ws, "ws"), _nbytes(ws), _stream(stream)),
           "ttq_act_norm")
    return D, D_rsqrt


def ttq_act_norm_scale(X, p, lam, alpha, ws=None, D=None, D_rsqrt=None, Xs=None, stream=None,
                       copy_out=True):
    """D, D^{-1/2} and Xs [T][d] binary16 = X * D^{-1/2} in one pass over X.
    With copy_out=False, D and D^{-1/2} are not given to the entry point and
    are returned as views of the workspace, where it writes them."""
    _matrix(X, "X", dtypes=_FLOAT_IN)
    T, d = X.shape
    _vector(D, "D", d)
    _vector(D_rsqrt, "D_rsqrt", d)
    _matrix(Xs, "Xs", T, d, _F16)
    if ws is None:
        ws = new_workspace(d, 0, T, 0, 4, 32, _dtype_code(X), X.device, stream)
    if Xs is None:
        Xs = torch.empty((T, d), dtype=torch.float16, device=X.device)
    if copy_out:
        if D is None:
            D = torch.empty(d, dtype=torch.float32, device=X.device)
        if D_rsqrt is None:
            D_rsqrt = torch.empty(d, dtype=torch.float32, device=X.device)
        dptr, drptr = _dev(D, "D"), _dev(D_rsqrt, "D_rsqrt")
    else:
        dptr = drptr = None
    _check(lib().ttq_act_norm_scale(_dev(X, "X"), _dtype_code(X), d, T, p, lam, alpha, dptr, drptr,
                                    _dev(Xs, "Xs"), _dev(ws, "ws"), _nbytes(ws), _stream(stream)),
           "ttq_act_norm_scale")
    if not copy_out:
        L = ttq_workspace_get_layout(d, 0, T, 0, 4, 32, _dtype_code(X))
        D = ws[L.D: L.D + 4 * d].view(torch.float32)
        D_rsqrt = ws[L.D_rsqrt: L.D_rsqrt + 4 * d].view(torch.float32)
    return D, D_rsqrt, Xs


def ttq_linear_forward_kernels(d, dp, T, r=0, p=2.0, dtype=TTQ_BF16, bits=4, group=128,
                               scheme=TTQ_QSCHEME_ASYMMETRIC) -> int:
    """Kernels one ttq_linear_forward(_ex) call of these sizes and this code
    scheme enqueues on the current device."""
    n = ctypes.c_int(0)
    _check(lib().ttq_linear_forward_kernels(dtype, d, dp, T, r, p, bits, group, scheme, ctypes.byref(n)),
           "ttq_linear_forward_kernels")
    return n.value


def ttq_act_norm_noalloc(X, p, lam, alpha, D=None, D_rsqrt=None, stream=None):
    """ttq_act_norm without a workspace: the library's own fixed scratch array
    is used (d <= 16384; calls overlapping on the GPU race)."""
    _matrix(X, "X", dtypes=_FLOAT_IN)
    T, d = X.shape
    _vector(D, "D", d)
    _vector(D_rsqrt, "D_rsqrt", d)
    if D is None:
        D = torch.empty(d, dtype=torch.float32, device=X.device)
    if D_rsqrt is None:
        D_rsqrt = torch.empty(d, dtype=torch.float32, device=X.device)
    _check(lib().ttq_act_norm_noalloc(_dev(X, "X"), _dtype_code(X), d, T, p, lam, alpha, _dev(D, "D"),
                                      _dev(D_rsqrt, "D_rsqrt"), _stream(stream)),
           "ttq_act_norm_noalloc")
    return D, D_rsqrt


def ttq_quantize_weight(W, D, bits, group, ws=None, codes=None, scales=None, zeros=None, stream=None):
    """codes [d'][d*bits/32] uint32, scales/zeros [d'][d/group] binary16 bits (int16 storage)."""
    _matrix(W, "W", dtypes=_FLOAT_IN)
    dp, d = W.shape
    _quant_outputs(dp, d, D, bits, group, codes, scales, zeros, None, "ttq_quantize_weight")
    dev = W.device
    if ws is None:
        ws = new_workspace(d, 0, 0, 0, bits, group, _dtype_code(W), dev, stream)
    if codes is None:
        codes = torch.empty((dp, d * bits // 32), dtype=torch.int32, device=dev)
    if scales is None:
        scales = torch.empty((dp, d // group), dtype=torch.int16, device=dev)
    if zeros is None:
        zeros = torch.empty((dp, d // group), dtype=torch.int16, device=dev)
    _check(lib().ttq_quantize_weight(_dev(W, "W"), _dtype_code(W), dp, d, _dev(D, "D"), bits, group,
                                     _dev(codes, "codes"), _dev(scales, "scales"), _dev(zeros, "zeros"),
                                     _dev(ws, "ws"), _nbytes(ws), _stream(stream)),
           "ttq_quantize_weight")
    return codes, scales, zeros


def ttq_quantize_weight_ex(W, D, bits, group, scheme, ws=None, codes=None, scales=None, zeros=None,
                           W_hat=None, stream=None, with_codes=True):
    """Codes, scales and zeros under the given TTQ_QSCHEME_*; W_hat (binary16
    s (q - z), optional) is written when given.  With with_codes=False (and
    W_hat given) only W_hat is written and (None, None, None) is returned."""
    _matrix(W, "W", dtypes=_FLOAT_IN)
    dp, d = W.shape
    _quant_outputs(dp, d, D, bits, group, codes, scales, zeros, W_hat, "ttq_quantize_weight_ex")
    dev = W.device
    if ws is None:
        ws = new_workspace(d, 0, 0, 0, bits, group, _dtype_code(W), dev, stream)
    if not with_codes:
        if W_hat is None:
            raise ValueError("ttq_quantize_weight_ex: with_codes=False needs W_hat")
        _check(lib().ttq_quantize_weight_ex(
            _dev(W, "W"), _dtype_code(W), dp, d, _dev(D, "D"), bits, group, scheme, None, None, None,
            _dev(W_hat, "W_hat"), _dev(ws, "ws"), _nbytes(ws), _stream(stream)), "ttq_quantize_weight_ex")
        return None, None, None
    if codes is None:
        codes = torch.empty((dp, d * bits // 32), dtype=torch.int32, device=dev)
    if scales is None:
        scales = torch.empty((dp, d // group), dtype=torch.int16, device=dev)
    if zeros is None:
        zeros = torch.empty((dp, d // group), dtype=torch.int16, device=dev)
    _check(lib().ttq_quantize_weight_ex(
        _dev(W, "W"), _dtype_code(W), dp, d, _dev(D, "D"), bits, group, scheme, _dev(codes, "codes"),
        _dev(scales, "scales"), _dev(zeros, "zeros"), _dev(W_hat, "W_hat"), _dev(ws, "ws"), _nbytes(ws),
        _stream(stream)), "ttq_quantize_weight_ex")
    return codes, scales, zeros


def ttq_quantize_dequant_weight(W, D, bits, group, ws=None, codes=None, scales=None, zeros=None,
                                W_hat=None, stream=None, with_codes=True):
    """ttq_quantize_weight plus W_hat [d'][d] binary16 (torch.float16) = s (q - z).
    With with_codes=False only W_hat is written (codes, scales, zeros are None)."""
    _matrix(W, "W", dtypes=_FLOAT_IN)
    dp, d = W.shape
    _quant_outputs(dp, d, D, bits, group, codes, scales, zeros, W_hat, "ttq_quantize_dequant_weight")
    dev = W.device
    if ws is None:
        ws = new_workspace(d, 0, 0, 0, bits, group, _dtype_code(W), dev, stream)
    if W_hat is None:
        W_hat = torch.empty((dp, d), dtype=torch.float16, device=dev)
    if not with_codes:
        _check(lib().ttq_quantize_dequant_weight(
            _dev(W, "W"), _dtype_code(W), dp, d, _dev(D, "D"), bits, group, None, None, None,
            _dev(W_hat, "W_hat"), _dev(ws, "ws"), _nbytes(ws), _stream(stream)),
            "ttq_quantize_dequant_weight")
        return None, None, None, W_hat
    if codes is None:
        codes = torch.empty((dp, d * bits // 32), dtype=torch.int32, device=dev)
    if scales is None:
        scales = torch.empty((dp, d // group), dtype=torch.int16, device=dev)
    if zeros is None:
        zeros = torch.empty((dp, d // group), dtype=torch.int16, device=dev)
    if W_hat is None:
        W_hat = torch.empty((dp, d), dtype=torch.float16, device=dev)
    _check(lib().ttq_quantize_dequant_weight(
        _dev(W, "W"), _dtype_code(W), dp, d, _dev(D, "D"), bits, group, _dev(codes, "codes"),
        _dev(scales, "scales"), _dev(zeros, "zeros"), _dev(W_hat, "W_hat"), _dev(ws, "ws"),
        _nbytes(ws), _stream(stream)), "ttq_quantize_dequant_weight")
    return codes, scales, zeros, W_hat


def ttq_dequantized_gemm(W_hat, Xs, ws=None, Y=None, y_dtype=torch.bfloat16, stream=None):
    """Y [T][d'] = W_hat Xs^T from a binary16 dequantised weight and binary16 X D^{-1/2}."""
    _matrix(W_hat, "W_hat", dtypes=_F16)
    dp, d = W_hat.shape
    _matrix(Xs, "Xs", cols=d, dtypes=_F16)
    T = Xs.shape[0]
    _matrix(Y, "Y", T, dp, _FLOAT_IN)
    if ws is None:
        # room for the forward's K split of this shape, so the result is its bits
        nbytes = max(4096, int(lib().ttq_dequantized_gemm_workspace_size(d, dp, T)))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=W_hat.device)
        ttq_workspace_init(ws, stream)
    if Y is None:
        Y = torch.empty((T, dp), dtype=y_dtype, device=W_hat.device)
    _check(lib().ttq_dequantized_gemm(_dev(W_hat, "W_hat"), _dev(Xs, "Xs"), d, dp, T, _dev(Y, "Y"),
                                      _dtype_code(Y), _dev(ws, "ws"), _nbytes(ws), _stream(stream)),
           "ttq_dequantized_gemm")
    return Y


def ttq_scale_activations(X, D_rsqrt, ws=None, Xs=None, stream=None):
    """Xs [T][d] binary16 (torch.float16) = X * D^{-1/2}, the product's B operand."""
    _matrix(X, "X", dtypes=_FLOAT_IN + _F16)
    T, d = X.shape
    _vector(D_rsqrt, "D_rsqrt", d)
    _matrix(Xs, "Xs", T, d, _F16)
    if ws is None:
        ws = new_workspace(d, 0, 0, 0, 4, 32, TTQ_BF16, X.device, stream)
    if Xs is None:
        Xs = torch.empty((T, d), dtype=torch.float16, device=X.device)
    _check(lib().ttq_scale_activations(_dev(X, "X"), _dtype_code(X), d, T, _dev(D_rsqrt, "D_rsqrt"),
                                       _dev(Xs, "Xs"), _dev(ws, "ws"), _nbytes(ws), _stream(stream)),
           "ttq_scale_activations")
    return Xs


def ttq_dequant_gemm(codes, scales, zeros, D_rsqrt, X, A, B, bits, group, ws=None, Y=None,
                     y_dtype=None, stream=None):
    """Y [T][d'] = W_hat X (+ B (A X)) from quantised weights; Y in y_dtype
    (default: the dtype of X, or of a given Y)."""
    _matrix(X, "X", dtypes=_FLOAT_IN + _F16)
    T, d = X.shape
    dp = codes.shape[0]
    r = _lowrank_pair(A, B)
    cb, sb = _qsizes(d, bits, group, "ttq_dequant_gemm")
    _room(codes, "codes", dp * cb)
    _room(scales, "scales", dp * sb)
    _room(zeros, "zeros", dp * sb)
    _vector(D_rsqrt, "D_rsqrt", d)
    _matrix(A, "A", r, d, (X.dtype,))
    _matrix(B, "B", dp, r, (X.dtype,))
    _matrix(Y, "Y", T, dp, _FLOAT_IN)
    dt = _dtype_code(X)
    if ws is None:
        ws = new_workspace(d, dp, T, r, bits, group, dt, X.device, stream)
    if Y is None:
        Y = torch.empty((T, dp), dtype=y_dtype or (torch.bfloat16 if dt == TTQ_F16 else X.dtype),
                        device=X.device)
    _check(lib().ttq_dequant_gemm(_dev(codes, "codes"), _dev(scales, "scales"), _dev(zeros, "zeros"),
                                  _dev(D_rsqrt, "D_rsqrt"), _dev(X, "X"), _dev(A, "A"), _dev(B, "B"), dt,
                                  d, dp, T, r, bits, group, _dev(Y, "Y"), _dtype_code(Y), _dev(ws, "ws"),
                                  _nbytes(ws), _stream(stream)),
           "ttq_dequant_gemm")
    return Y


TTQ_TESTING_WAIT_MBARRIER = 0


def ttq_testing_wait_timeout(kind, limit_ns, blocks, ws, stream=None) -> None:
    """Test hook: `blocks` blocks each make one wait of `kind` that cannot
    complete, with a limit of limit_ns; they set TTQ_FLAG_TIMEOUT in ws."""
    _check(lib().ttq_testing_wait_timeout(kind, limit_ns, blocks, _dev(ws, "ws"), _nbytes(ws),
                                          _stream(stream)), "ttq_testing_wait_timeout")


def ttq_testing_kv_page_of(page_size, block) -> int:
    """Test hook (host only): the page, counted along its sequence, of a block of 16 positions, as the cache's kernels
    find it; -1 for arguments out of range."""
    return int(lib().ttq_testing_kv_page_of(page_size, block))


def ttq_quantize_gemm(W, D, Xs, A, B, X, bits, group, ws=None, Y=None, y_dtype=torch.bfloat16,
                      codes=None, scales=None, zeros=None, stream=None):
    """Steps (2)-(3) in one pass over bf16 W [d'][d] for T <= 16 tokens:
    Y [T][d'] = Q[W D^{1/2}] Xs (+ B (A X)), Xs the binary16 X D^{-1/2}
    [T][d]; A [r][d], B [d'][r], X [T][d] bf16 for the low-rank term.
    codes/scales/zeros: None, or all three buffers to receive the codes."""
    _matrix(Xs, "Xs", dtypes=_F16)
    T, d = Xs.shape
    _matrix(W, "W", cols=d, dtypes=(torch.bfloat16,))
    dp = W.shape[0]
    _vector(D, "D", d)
    r = _lowrank_pair(A, B)
    _matrix(A, "A", r, d, (torch.bfloat16,))
    _matrix(B, "B", dp, r, (torch.bfloat16,))
    if r > 0:
        _matrix(X, "X", T, d, (torch.bfloat16,))
    given = [t is not None for t in (codes, scales, zeros)]
    if any(given) and not all(given):
        raise TTQError(TTQ_ERR_INVALID_ARG, "ttq_quantize_gemm: codes, scales and zeros go together")
    if all(given):
        cb, sb = _qsizes(d, bits, group, "ttq_quantize_gemm")
        _room(codes, "codes", dp * cb)
        _room(scales, "scales", dp * sb)
        _room(zeros, "zeros", dp * sb)
    _matrix(Y, "Y", T, dp, _FLOAT_IN)
    if ws is None:
        ws = new_workspace(d, dp, T, r, bits, group, TTQ_BF16, W.device, stream)
    if Y is None:
        Y = torch.empty((T, dp), dtype=y_dtype, device=W.device)
    _check(lib().ttq_quantize_gemm(_dev(W, "W"), _dev(D, "D"), _dev(Xs, "Xs"), _dev(A, "A"), _dev(B, "B"),
                                   _dev(X if r > 0 else None, "X"), d, dp, T, r, bits, group,
                                   _dev(codes, "codes"), _dev(scales, "scales"), _dev(zeros, "zeros"),
                                   _dev(Y, "Y"), _dtype_code(Y), _dev(ws, "ws"), _nbytes(ws),
                                   _stream(stream)),
           "ttq_quantize_gemm")
    return Y


def ttq_linear_forward(X, W, A, B, p, lam, alpha, bits, group, ws=None, Y=None, y_dtype=None,
                       stream=None, scheme=None):
    """The TTQ linear layer: Y [T][d'] = Q[W D^{1/2}] D^{-1/2} X + B (A X);
    Y in y_dtype (default: the dtype of X, or of a given Y).  scheme: None
    (ttq_linear_forward) or a TTQ_QSCHEME_* code (ttq_linear_forward_ex)."""
    _matrix(X, "X", dtypes=_FLOAT_IN)
    T, d = X.shape
    _matrix(W, "W", cols=d, dtypes=(X.dtype,))
    dp = W.shape[0]
    r = _lowrank_pair(A, B)
    _matrix(A, "A", r, d, (X.dtype,))
    _matrix(B, "B", dp, r, (X.dtype,))
    _matrix(Y, "Y", T, dp, _FLOAT_IN)
    dt = _dtype_code(X)
    if ws is None:
        ws = new_workspace(d, dp, T, r, bits, group, dt, X.device, stream)
    if Y is None:
        Y = torch.empty((T, dp), dtype=y_dtype or X.dtype, device=X.device)
    args = (_dev(X, "X"), _dev(W, "W"), _dev(A, "A"), _dev(B, "B"), dt, d, dp, T, r, p, lam, alpha, bits,
            group)
    tail = (_dev(Y, "Y"), _dtype_code(Y), _dev(ws, "ws"), _nbytes(ws), _stream(stream))
    if scheme is None:
        _check(lib().ttq_linear_forward(*args, *tail), "ttq_linear_forward")
    else:
        _check(lib().ttq_linear_forward_ex(*args, scheme, *tail), "ttq_linear_forward_ex")
    return Y


def ttq_lowrank_workspace_size(dp, d, r, oversample) -> int:
    return int(lib().ttq_lowrank_workspace_size(dp, d, r, oversample))


def ttq_lowrank_init(W, r, Omega, power_iters=2, ws=None, B=None, A=None, W_res=None,
                     residual=True, stream=None):
    """Static low-rank factors of W [d'][d] (float32 or bf16): B [d'][r],
    A [r][d] from a randomised truncated SVD with the Gaussian test matrix
    Omega [d][r + oversample] (float32), and W_res = W - B A (when
    `residual`).  Returns (B, A, W_res or None)."""
    _matrix(W, "W", dtypes=_FLOAT_IN)
    dp, d = W.shape
    _matrix(Omega, "Omega", d, None, _F32)
    _matrix(B, "B", dp, r, (W.dtype,))
    _matrix(A, "A", r, d, (W.dtype,))
    _matrix(W_res, "W_res", dp, d, (W.dtype,))
    l = Omega.shape[1]
    oversample = l - r
    dt = _dtype_code(W)
    if ws is None:
        n = ttq_lowrank_workspace_size(dp, d, r, oversample)
        if n == 0:
            raise TTQError(TTQ_ERR_INVALID_ARG, "ttq_lowrank_workspace_size")
        ws = torch.empty(n, dtype=torch.uint8, device=W.device)
        ttq_workspace_init(ws, stream)
    if B is None:
        B = torch.empty((dp, r), dtype=W.dtype, device=W.device)
    if A is None:
        A = torch.empty((r, d), dtype=W.dtype, device=W.device)
    if W_res is None and residual:
        W_res = torch.empty_like(W)
    _check(lib().ttq_lowrank_init(_dev(W, "W"), dt, dp, d, r, oversample, power_iters, _dev(Omega, "Omega"),
                                  _dev(B, "B"), _dev(A, "A"), _dev(W_res, "W_res"), _dev(ws, "ws"),
                                  _nbytes(ws), _stream(stream)),
           "ttq_lowrank_init")
    return B, A, W_res


def workspace_views(ws: torch.Tensor, d, dp, T, r, bits, group, dtype=TTQ_BF16) -> dict:
    """Views of the intermediates a forward call leaves in its workspace."""
    L = ttq_workspace_get_layout(d, dp, T, r, bits, group, dtype)

    def view(off, n, dt):
        itemsize = torch.empty((), dtype=dt).element_size()
        return ws[off: off + n * itemsize].view(dt)

    out = {"D": view(L.D, d, torch.float32), "D_rsqrt": view(L.D_rsqrt, d, torch.float32)}
    if dp > 0:
        out["codes"] = view(L.codes, dp * (d * bits // 32), torch.int32).view(dp, -1)
        out["scales"] = view(L.scales, dp * (d // group), torch.int16).view(dp, -1)
        out["zeros"] = view(L.zeros, dp * (d // group), torch.int16).view(dp, -1)
        out["xh"] = view(L.xh, T * d, torch.float16).view(T, d)
        if L.wq:
            out["wq"] = view(L.wq, dp * d, torch.float16).view(dp, d)
    return out


# --------------------------------------------- the quantised key/value cache
_ROW_TYPES = (torch.float32, torch.bfloat16, torch.float16)


def _ints(t: torch.Tensor, name: str, shape) -> None:
    """t is int32 of this shape (None: any size there)."""
    if t.dtype != torch.int32:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.int32")
    if t.dim() != len(shape) or any(w is not None and w != s for w, s in zip(shape, t.shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple('*' if w is None else w for w in shape)}")


def _rows_of(t: torch.Tensor, name: str, rows: int, heads, head_dim: int) -> tuple:
    """The strides of t, which is [rows][heads][head_dim] with contiguous channels (heads None: any number)."""
    if t.dtype not in _ROW_TYPES:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {list(_ROW_TYPES)}")
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != rows or shape[2] != head_dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {(rows, '*' if heads is None else heads, head_dim)}")
    if strides[2] != 1:
        raise ValueError(f"the channels of {name} must be contiguous, got strides {strides}")
    return strides


def _strided(t: torch.Tensor, name: str, rows: int, heads: int, strides: tuple, device: int) -> tuple:
    """(pointer, row stride, head stride) of a row tensor on this device."""
    if t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{device}, got {t.device}")
    at = t.data_ptr()
    # the stride of a size that is not walked along says nothing
    row, head = strides[0] if rows > 1 else 0, strides[1] if heads > 1 else 0
    if row % 8 or head % 8 or at % 16:
        raise ValueError(f"the rows of {name} must be 16-byte aligned: strides {strides} are not multiples of 8 "
                         "elements, or its first element is not at a 16-byte boundary")
    return at, row, head


def _on(t: torch.Tensor | None, name: str, device: int) -> int | None:
    """Pointer of a contiguous tensor on this device (None stays None)."""
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An uninitialised tensor of the stream that the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_rows(rows, heads, head_dim, dtype, device, stream) -> torch.Tensor:
    """An uninitialised row tensor of the stream that the call runs on."""
    if stream is None:    # with strides: 1 us less of host time
        return torch.empty_strided((rows, heads, head_dim), (heads * head_dim, head_dim, 1), dtype=dtype, device=device)
    return _empty((rows, heads, head_dim), dtype, device, stream)


class _Handle:
    """A C struct built from the public attributes at the first call, after checking them, and again after one of them
    was assigned."""
    _struct = None

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if not name.startswith("_"):
            object.__setattr__(self, "_struct", None)

    def _keep(self, struct, device):
        self._ref, self._device = ctypes.byref(struct), device
        self._struct = struct     # last: another thread takes the struct for built from here on


class KVCache(_Handle):
    """A quantised key/value cache (ttq_kv_cache): `pages` uint8 [num_pages][ttq_kv_page_bytes(...)] (new_kv_cache
    makes it) and its format; D_k, D_v and their inverse square roots float32 [kv_heads][head_dim] or None, as
    ttq_act_norm gives them for rows of K and V.  It keeps the tensors; attributes may be assigned, and count from the
    next call on."""

    def __init__(self, pages, page_size, kv_heads, head_dim, bits, group, scheme=TTQ_QSCHEME_ASYMMETRIC, D_k=None,
                 D_v=None, D_k_rsqrt=None, D_v_rsqrt=None):
        self.pages, self.page_size, self.kv_heads, self.head_dim = pages, page_size, kv_heads, head_dim
        self.bits, self.group, self.scheme = bits, group, scheme
        self.D_k, self.D_v, self.D_k_rsqrt, self.D_v_rsqrt = D_k, D_v, D_k_rsqrt, D_v_rsqrt
        self._check()

    def _check(self):
        pages, n = self.pages, ttq_kv_page_bytes(self.page_size, self.kv_heads, self.head_dim, self.bits, self.group)
        if pages.dtype != torch.uint8 or pages.dim() != 2 or pages.shape[1] != n:
            raise ValueError(f"pages must be uint8 [num_pages][{n}], got {pages.dtype} {tuple(pages.shape)}")
        for name in ("D_k", "D_v", "D_k_rsqrt", "D_v_rsqrt"):
            _vector(getattr(self, name), name, self.kv_heads * self.head_dim)
        for a, b, name in ((self.D_k, self.D_k_rsqrt, "k"), (self.D_v, self.D_v_rsqrt, "v")):
            if (a is None) != (b is None):
                raise ValueError(f"D_{name} and D_{name}_rsqrt are given together or not at all")

    def _arg(self):
        """(the C struct, its device), which is the current one."""
        if self._struct is None:
            self._check()
            self._keep(_CacheStruct(_dev(self.pages, "pages"), self.pages.shape[0], self.page_size, self.kv_heads,
                                    self.head_dim, self.bits, self.group, self.scheme, _dev(self.D_k, "D_k"),
                                    _dev(self.D_v, "D_v"), _dev(self.D_k_rsqrt, "D_k_rsqrt"),
                                    _dev(self.D_v_rsqrt, "D_v_rsqrt")), self.pages.get_device())
        elif self._device != torch.cuda.current_device():
            raise ValueError(f"pages is on {self.pages.device}; the library runs on the current device "
                             f"cuda:{torch.cuda.current_device()}")
        return self._ref, self._device


class KVBatch(_Handle):
    """The rows of a call (ttq_kv_batch): sequence i has rows cu_new[i] .. cu_new[i + 1] - 1, its last positions of
    kv_len[i]; page_table int32 [batch][pages], kv_len int32 [batch], cu_new int32 [batch + 1] (device tensors whose
    contents may change between calls), `rows` rows in the row tensors, at most max_new of any sequence.  Attributes
    may be assigned, and count from the next call on."""

    def __init__(self, page_table, kv_len, cu_new, rows, max_new):
        self.page_table, self.kv_len, self.cu_new, self.rows, self.max_new = page_table, kv_len, cu_new, rows, max_new
        self._check()

    def _check(self):
        _ints(self.kv_len, "kv_len", (None,))
        n = self.kv_len.shape[0]
        _ints(self.cu_new, "cu_new", (n + 1,))
        _ints(self.page_table, "page_table", (n, None))
        if self.rows < 0 or self.max_new < 0:
            raise ValueError(f"rows and max_new must not be negative, got {self.rows} and {self.max_new}")

    def _arg(self, device):
        if self._struct is None:
            self._check()
            self._keep(_BatchStruct(_on(self.page_table, "page_table", device), self.page_table.shape[1],
                                    _on(self.kv_len, "kv_len", device), _on(self.cu_new, "cu_new", device),
                                    self.kv_len.shape[0], self.rows, self.max_new), device)
        if self._device != device:
            raise ValueError(f"the batch is on {self.kv_len.device}, the cache on cuda:{device}")
        return self._ref


def ttq_kv_page_bytes(page_size, kv_heads, head_dim, bits, group) -> int:
    """Bytes of one page of a key/value cache (raises if the format is not built)."""
    n = int(lib().ttq_kv_page_bytes(page_size, kv_heads, head_dim, bits, group))
    if n == 0:
        raise TTQError(TTQ_ERR_UNSUPPORTED, "ttq_kv_page_bytes")
    return n


def new_kv_cache(num_pages, page_size, kv_heads, head_dim, bits, group, scheme=TTQ_QSCHEME_ASYMMETRIC, device="cuda",
                 **statistics) -> KVCache:
    """A KVCache of num_pages uninitialised pages."""
    n = ttq_kv_page_bytes(page_size, kv_heads, head_dim, bits, group)
    return KVCache(torch.empty((num_pages, n), dtype=torch.uint8, device=device), page_size, kv_heads, head_dim, bits,
                   group, scheme, **statistics)


def ttq_kv_attention_workspace_size(head_dim, bits, group, heads, kv_heads, max_new) -> int:
    """Workspace bytes of ttq_kv_attention (0: not built)."""
    return int(lib().ttq_kv_attention_workspace_size(head_dim, bits, group, heads, kv_heads, max_new))


def new_kv_workspace(cache, batch, heads=None, stream=None) -> torch.Tensor:
    """An initialised workspace for the cache's entry points: for ttq_kv_attention with `heads` query heads (None:
    only ttq_kv_write and ttq_kv_read) and batches of at most batch.max_new rows a sequence."""
    n = 4096
    if heads is not None and batch.max_new <= 64:
        n = max(n, ttq_kv_attention_workspace_size(cache.head_dim, cache.bits, cache.group, heads, cache.kv_heads,
                                                   batch.max_new))
    ws = _empty(n, torch.uint8, cache.pages.device, stream)
    ttq_workspace_init(ws, stream)
    return ws


def ttq_kv_write(cache, batch, K, V, ws=None, stream=None) -> None:
    """Quantises the rows of K and V [rows][kv_heads][head_dim] into the cache (one type; rows and heads may be
    strided, as slices of a fused projection are)."""
    rows, heads = batch.rows, cache.kv_heads
    k_strides = _rows_of(K, "K", rows, heads, cache.head_dim)
    v_strides = _rows_of(V, "V", rows, heads, cache.head_dim)
    if K.dtype != V.dtype:
        raise TypeError(f"K and V have different dtypes {K.dtype} and {V.dtype}")
    c, device = cache._arg()
    b = batch._arg(device)
    if ws is None:
        ws = new_kv_workspace(cache, batch, None, stream)
    _check(lib().ttq_kv_write(c, b, *_strided(K, "K", rows, heads, k_strides, device),
                              *_strided(V, "V", rows, heads, v_strides, device), _dtype_code(K),
                              _on(ws, "ws", device), ws.nbytes, _stream_on(stream, device)), "ttq_kv_write")


def ttq_kv_read(cache, batch, K=None, V=None, dtype=None, ws=None, stream=None):
    """The dequantised rows (K, V), each [rows][kv_heads][head_dim] in `dtype` (default bf16, or that of a given
    tensor).  Rows in no sequence are left as they are (uninitialised in a new tensor)."""
    for t, name in ((K, "K"), (V, "V")):
        if t is not None:
            _rows_of(t, name, batch.rows, cache.kv_heads, cache.head_dim)
            if dtype is not None and t.dtype != dtype:
                raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
            dtype = t.dtype
    dtype = dtype or torch.bfloat16
    if dtype not in _ROW_TYPES:
        raise TypeError(f"unsupported dtype {dtype} (float32, bfloat16 or float16)")
    c, device = cache._arg()
    b = batch._arg(device)
    if K is None:
        K = _empty_rows(batch.rows, cache.kv_heads, cache.head_dim, dtype, cache.pages.device, stream)
    if V is None:
        V = _empty_rows(batch.rows, cache.kv_heads, cache.head_dim, dtype, cache.pages.device, stream)
    if ws is None:
        ws = new_kv_workspace(cache, batch, None, stream)
    _check(lib().ttq_kv_read(c, b, _on(K, "K", device), _on(V, "V", device), _dtype_code(K), _on(ws, "ws", device),
                             ws.nbytes, _stream_on(stream, device)), "ttq_kv_read")
    return K, V


def ttq_kv_attention(cache, batch, Q, scale, softcap=0.0, window=0, tree=None, ws=None, Y=None, y_dtype=None,
                     stream=None):
    """Y [rows][heads][head_dim]: attention of the batch's rows of Q (strided like K of ttq_kv_write) over the cache,
    causal among a sequence's own rows, or by `tree` (int64 [rows]: bit k of a row's mask is set iff it sees the
    sequence's k-th new row; bits beyond its rows stand for nothing).  softcap: scores are softcap tanh(t / softcap); window: positions seen, 0 for all."""
    q_strides = _rows_of(Q, "Q", batch.rows, None, cache.head_dim)
    heads = Q.shape[1]
    if heads % cache.kv_heads or heads == 0:
        raise ValueError(f"{heads} query heads are not a multiple of the cache's {cache.kv_heads} heads")
    if tree is not None:
        if tree.dtype != torch.int64:
            raise TypeError(f"tree has dtype {tree.dtype}, expected torch.int64")
        if tree.dim() != 1 or tree.shape[0] != batch.rows:
            raise ValueError(f"tree has shape {tuple(tree.shape)}, expected ({batch.rows},)")
    if Y is not None:
        _rows_of(Y, "Y", batch.rows, heads, cache.head_dim)
        if y_dtype is not None and Y.dtype != y_dtype:
            raise TypeError(f"Y has dtype {Y.dtype}, expected {y_dtype}")
    y_dtype = Y.dtype if Y is not None else (y_dtype or Q.dtype)
    if y_dtype not in _ROW_TYPES:
        raise TypeError(f"unsupported dtype {y_dtype} (float32, bfloat16 or float16)")
    c, device = cache._arg()
    b = batch._arg(device)
    q = _strided(Q, "Q", batch.rows, heads, q_strides, device)
    if Y is None:
        Y = _empty_rows(batch.rows, heads, cache.head_dim, y_dtype, Q.device, stream)
    if ws is None:
        ws = new_kv_workspace(cache, batch, heads, stream)
    _check(lib().ttq_kv_attention(c, b, *q, _dtype_code(Q), heads, scale, softcap, window, _on(tree, "tree", device),
                                  _on(Y, "Y", device), _dtype_code(Y), _on(ws, "ws", device), ws.nbytes,
                                  _stream_on(stream, device)), "ttq_kv_attention")
    return Y
