"""ctypes binding of ``libgemm_epi.so`` (the C ABI in include/gemm_epi.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, then their ``data_ptr()`` and the current CUDA stream are passed
to the C function of the same name. All arithmetic happens in the library's
kernels; if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

F16, BF16 = 0, 1
BIAS, RELU_BIAS, RELU_AUX_BIAS, DRELU_BGRAD, GELU_BIAS, WGRAD, NONE, GELU_AUX_BIAS = 0, 1, 2, 3, 4, 5, 6, 7
EPILOGS = {"BIAS": BIAS, "RELU_BIAS": RELU_BIAS, "RELU_AUX_BIAS": RELU_AUX_BIAS, "DRELU_BGRAD": DRELU_BGRAD,
           "GELU_BIAS": GELU_BIAS, "WGRAD": WGRAD, "NONE": NONE, "GELU_AUX_BIAS": GELU_AUX_BIAS}
DTYPES = {torch.float16: F16, torch.bfloat16: BF16}

OK = 0
ERR_INVALID_ARG = -1
ERR_MISALIGNED = -2
ERR_EPILOG_MISMATCH = -3
ERR_CUDA = -4
ERR_TIMEOUT = -5
ERR_UNSUPPORTED = -6

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgemm_epi.so")

EXPORTED = ["gemm_epi_plan", "gemm_epi_execute", "drelu_bgrad_execute", "gemm_epi_free", "gemm_epi_last_error",
            "gemm_epi_query", "gemm_epi_status", "gemm_epi_unfused_execute", "drelu_bgrad_unfused_execute",
            "drelu_bgrad_execute_noalloc", "gemm_epi_wgrad_execute", "gemm_epi_set_bias_f32", "gemm_epi_plan_ex",
            "gemm_epi_grouped_plan", "gemm_epi_grouped_execute", "gemm_epi_grouped_drelu_bgrad_execute",
            "gemm_epi_grouped_wgrad_execute", "gemm_epi_mx_scales_bytes", "gemm_epi_mx_quantize",
            "gemm_epi_mx_dequantize", "gemm_epi_mx_plan", "gemm_epi_mx_execute", "gemm_epi_gated_plan",
            "gemm_epi_gated_execute", "gemm_epi_dgated_execute", "gemm_epi_w4_bytes", "gemm_epi_w4_scales",
            "gemm_epi_w4_quantize", "gemm_epi_w4_pack", "gemm_epi_w4_dequantize", "gemm_epi_w4_plan",
            "gemm_epi_w4_execute"]
GATED_EPILOGS = {"GATED": 8, "DGATED": 9, "GATED_AUX": 10}  # gemm_epi_gated_epilog
ACTS = {"SILU": 0, "GELU": 1, "RELU": 2}  # gemm_epi_act
MX_TRANSPOSED = 1  # GEMM_EPI_MX_TRANSPOSED
FLAG_W_NK = 1  # GEMM_EPI_FLAG_W_NK
FLAG_OUT_F32 = 2  # GEMM_EPI_FLAG_OUT_F32
FLAG_NO_DBIAS = 4  # GEMM_EPI_FLAG_NO_DBIAS

NOALLOC_SCRATCH_BYTES = 4 << 20  # GEMM_EPI_NOALLOC_SCRATCH_BYTES


class GemmEpiError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"gemm_epi error {code}: {msg}")
        self.code = code


class Info(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("epilog", ctypes.c_int), ("kernel", ctypes.c_int),
                ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int), ("tile_k", ctypes.c_int),
                ("stages", ctypes.c_int), ("split_k", ctypes.c_int), ("grid", ctypes.c_int),
                ("launches", ctypes.c_int), ("num_sms", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


_lib = None


def lib() -> ctypes.CDLL:
    """Load the library (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m gemm_epilogues_tcgen05_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.gemm_epi_plan.restype = vp
        L.gemm_epi_plan.argtypes = [i64, i64, i64, ci, ci]
        L.gemm_epi_plan_ex.restype = vp
        L.gemm_epi_plan_ex.argtypes = [i64, i64, i64, ci, ci, ctypes.c_uint32]
        L.gemm_epi_execute.restype = ci
        L.gemm_epi_execute.argtypes = [vp] * 7
        L.drelu_bgrad_execute.restype = ci
        L.drelu_bgrad_execute.argtypes = [vp] * 7
        L.gemm_epi_free.restype = None
        L.gemm_epi_free.argtypes = [vp]
        L.gemm_epi_last_error.restype = ctypes.c_char_p
        L.gemm_epi_last_error.argtypes = []
        L.gemm_epi_query.restype = ci
        L.gemm_epi_query.argtypes = [vp, ctypes.POINTER(Info)]
        L.gemm_epi_status.restype = ci
        L.gemm_epi_status.argtypes = [vp]
        L.gemm_epi_unfused_execute.restype = ci
        L.gemm_epi_unfused_execute.argtypes = [vp] * 9
        L.drelu_bgrad_unfused_execute.restype = ci
        L.drelu_bgrad_unfused_execute.argtypes = [vp] * 8
        L.drelu_bgrad_execute_noalloc.restype = ci
        L.drelu_bgrad_execute_noalloc.argtypes = [i64, i64, i64, ci] + [vp] * 6
        L.gemm_epi_set_bias_f32.restype = ci
        L.gemm_epi_set_bias_f32.argtypes = [vp, ci]
        L.gemm_epi_wgrad_execute.restype = ci
        L.gemm_epi_wgrad_execute.argtypes = [vp] * 6
        L.gemm_epi_grouped_plan.restype = vp
        L.gemm_epi_grouped_plan.argtypes = [i64, i64, i64, i64, ci, ci, ctypes.c_uint32]
        L.gemm_epi_grouped_execute.restype = ci
        L.gemm_epi_grouped_execute.argtypes = [vp] * 8
        L.gemm_epi_grouped_drelu_bgrad_execute.restype = ci
        L.gemm_epi_grouped_drelu_bgrad_execute.argtypes = [vp] * 8
        L.gemm_epi_grouped_wgrad_execute.restype = ci
        L.gemm_epi_grouped_wgrad_execute.argtypes = [vp] * 7
        L.gemm_epi_mx_scales_bytes.restype = i64
        L.gemm_epi_mx_scales_bytes.argtypes = [i64] * 4
        L.gemm_epi_mx_quantize.restype = ci
        L.gemm_epi_mx_quantize.argtypes = [i64, i64, i64, ci, ctypes.c_uint32, vp, vp, i64, vp, vp, vp]
        L.gemm_epi_mx_dequantize.restype = ci
        L.gemm_epi_mx_dequantize.argtypes = [i64, i64, i64, ci, ctypes.c_uint32, vp, vp, vp, i64, vp, vp]
        L.gemm_epi_mx_plan.restype = vp
        L.gemm_epi_mx_plan.argtypes = [i64, i64, i64, i64, ci, ci, ctypes.c_uint32]
        L.gemm_epi_mx_execute.restype = ci
        L.gemm_epi_mx_execute.argtypes = [vp] * 9
        L.gemm_epi_gated_plan.restype = vp
        L.gemm_epi_gated_plan.argtypes = [i64, i64, i64, ci, ci, ci, ctypes.c_uint32]
        L.gemm_epi_gated_execute.restype = ci
        L.gemm_epi_gated_execute.argtypes = [vp] * 7
        L.gemm_epi_dgated_execute.restype = ci
        L.gemm_epi_dgated_execute.argtypes = [vp] * 7
        for size in (L.gemm_epi_w4_bytes, L.gemm_epi_w4_scales):
            size.restype = i64
            size.argtypes = [i64] * 4
        L.gemm_epi_w4_quantize.restype = ci
        L.gemm_epi_w4_quantize.argtypes = [i64] * 4 + [ci] + [vp] * 5
        L.gemm_epi_w4_pack.restype = ci
        L.gemm_epi_w4_pack.argtypes = [i64] * 4 + [vp] * 7
        L.gemm_epi_w4_dequantize.restype = ci
        L.gemm_epi_w4_dequantize.argtypes = [i64] * 4 + [ci, ctypes.c_uint32] + [vp] * 5
        L.gemm_epi_w4_plan.restype = vp
        L.gemm_epi_w4_plan.argtypes = [i64] * 4 + [ci, ci, ci, ctypes.c_uint32]
        L.gemm_epi_w4_execute.restype = ci
        L.gemm_epi_w4_execute.argtypes = [vp] * 8
        _lib = L
    return _lib


def gemm_epi_last_error() -> str:
    return lib().gemm_epi_last_error().decode()


def _check(rc: int):
    if rc != OK:
        raise GemmEpiError(rc, gemm_epi_last_error())


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t, shape, dtype, name) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on_stream(stream, device):
    """The stream that a call will use, as the current one: outputs that a
    convenience allocates belong to it. (Memory from another stream's pool may
    still be read or written by work that waits on that stream.)"""
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_ptr(stream)
        # (ExternalStream takes 0 for no handle at all, and gives a new stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on_stream(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _zeros(shape, dtype, device, stream):
    if stream is None:
        return torch.zeros(shape, dtype=dtype, device=device)
    with _on_stream(stream, device):
        return torch.zeros(shape, dtype=dtype, device=device)


def gemm_epi_plan(T: int, N: int, K: int, dtype, epilog, flags: int = 0) -> int:
    """Raw handle (int) from the C gemm_epi_plan_ex; raises on error."""
    if isinstance(dtype, torch.dtype):
        dtype = DTYPES[dtype]
    if isinstance(epilog, str):
        epilog = EPILOGS[epilog]
    h = lib().gemm_epi_plan_ex(T, N, K, dtype, epilog, flags)
    if not h:
        raise GemmEpiError(ERR_INVALID_ARG, gemm_epi_last_error())
    return h


def gemm_epi_free(handle) -> None:
    lib().gemm_epi_free(handle)


def drelu_bgrad_execute_noalloc(dY2, W2, aux, dZ, dbias, stream=None):
    """DRELU_BGRAD without a plan and without any device allocation.

    For callers that may not allocate device memory (a host framework that
    owns the device's memory, or an enqueue callback that must not call
    cudaMalloc because it can synchronise the device). The column partials
    live in the library's fixed 4 MiB static scratch, shared by every call:
    calls that overlap on the GPU race, so keep them on one stream. The first
    call on a device does a one-time set-up; make it before any stream
    capture. If the kernel's watchdog fires, dbias comes back as NaN.
    """
    T, K = dY2.shape
    N = W2.shape[1]
    dt = dY2.dtype
    args = (_ptr(dY2, (T, K), dt, "dY2"), _ptr(W2, (K, N), dt, "W2"),
            _ptr(aux, (T, (N + 31) // 32), torch.int32, "aux"), _ptr(dZ, (T, N), dt, "dZ"),
            _ptr(dbias, (N,), torch.float32, "dbias"))
    _check(lib().drelu_bgrad_execute_noalloc(T, N, K, DTYPES[dt], *args, _stream_ptr(stream)))


class Plan:
    """A plan for one (T, N, K, dtype, epilog); execute any number of times."""

    def __init__(self, T: int, N: int, K: int, dtype: torch.dtype, epilog: str | int, w_nk: bool = False,
                 out_f32: bool = False):
        """w_nk: the weight (W, or W2 of DRELU_BGRAD) is N x K, K contiguous.
        out_f32: the output (Y, dZ or dW) is fp32."""
        self.T, self.N, self.K = T, N, K
        self.out_dtype = torch.float32 if out_f32 else dtype
        self.w_shape = (N, K) if w_nk else (K, N)
        self.dtype = dtype
        self.epilog = EPILOGS[epilog] if isinstance(epilog, str) else epilog
        self.aux_words = (N + 31) // 32
        self.bias_dtype = dtype
        self.handle = gemm_epi_plan(T, N, K, dtype, self.epilog,
                                    (FLAG_W_NK if w_nk else 0) | (FLAG_OUT_F32 if out_f32 else 0))

    def aux_spec(self):
        """Shape and dtype of the forward's auxiliary output: the mask words
        (T x ceil(N/32) int32) for RELU_AUX_BIAS, the pre-activation (T x N,
        the plan's 16-bit type) for GELU_AUX_BIAS, None otherwise."""
        if self.epilog == RELU_AUX_BIAS:
            return (self.T, self.aux_words), torch.int32
        if self.epilog == GELU_AUX_BIAS:
            return (self.T, self.N), self.dtype
        return None

    def _aux(self, aux):
        spec = self.aux_spec() or ((self.T, self.aux_words), torch.int32)
        return _ptr(aux, spec[0], spec[1], "aux")

    def set_bias_f32(self, on: bool = True):
        """Read the forward bias as fp32 (True) or in the plan's 16-bit type (False)."""
        _check(lib().gemm_epi_set_bias_f32(self.handle, 1 if on else 0))
        self.bias_dtype = torch.float32 if on else self.dtype

    # life cycle ----------------------------------------------------------
    def free(self):
        if self.handle:
            gemm_epi_free(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.free()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass

    def info(self) -> dict:
        inf = Info()
        _check(lib().gemm_epi_query(self.handle, ctypes.byref(inf)))
        return inf.as_dict()

    def status(self) -> int:
        """OK, or ERR_TIMEOUT if a kernel of this plan gave up a wait (after a sync)."""
        return lib().gemm_epi_status(self.handle)

    # calls -------------------------------------------------------------
    def gemm_epi_execute(self, X, W, bias, Y, aux=None, stream=None):
        T, N, K, dt = self.T, self.N, self.K, self.dtype
        args = (_ptr(X, (T, K), dt, "X"), _ptr(W, self.w_shape, dt, "W"), _ptr(bias, (N,), self.bias_dtype, "bias"),
                _ptr(Y, (T, N), self.out_dtype, "Y"), self._aux(aux))
        _check(lib().gemm_epi_execute(self.handle, *args, _stream_ptr(stream)))

    def drelu_bgrad_execute(self, dY2, W2, aux, dZ, dbias, stream=None):
        T, N, K, dt = self.T, self.N, self.K, self.dtype
        args = (_ptr(dY2, (T, K), dt, "dY2"), _ptr(W2, self.w_shape, dt, "W2"),
                _ptr(aux, (T, self.aux_words), torch.int32, "aux"), _ptr(dZ, (T, N), self.out_dtype, "dZ"),
                _ptr(dbias, (N,), torch.float32, "dbias"))
        _check(lib().drelu_bgrad_execute(self.handle, *args, _stream_ptr(stream)))

    def gemm_epi_wgrad_execute(self, X, dZ, dW, dbias=None, stream=None):
        """WGRAD plan: dW (K x N) = X^T . dZ; dbias (K floats, optional) = sum over t of X."""
        T, N, K, dt = self.T, self.N, self.K, self.dtype
        args = (_ptr(X, (T, K), dt, "X"), _ptr(dZ, (T, N), dt, "dZ"),
                _ptr(dW, (K, N), self.out_dtype, "dW"),
                _ptr(dbias, (K,), torch.float32, "dbias"))
        _check(lib().gemm_epi_wgrad_execute(self.handle, *args, _stream_ptr(stream)))

    def gemm_epi_unfused_execute(self, X, W, bias, T1, T2, Y, aux=None, stream=None):
        T, N, K, dt = self.T, self.N, self.K, self.dtype
        args = (_ptr(X, (T, K), dt, "X"), _ptr(W, self.w_shape, dt, "W"), _ptr(bias, (N,), self.bias_dtype, "bias"),
                _ptr(T1, (T, N), dt, "T1"), _ptr(T2, (T, N), dt, "T2"), _ptr(Y, (T, N), self.out_dtype, "Y"),
                self._aux(aux))
        _check(lib().gemm_epi_unfused_execute(self.handle, *args, _stream_ptr(stream)))

    def drelu_bgrad_unfused_execute(self, dY2, W2, aux, G, dZ, dbias, stream=None):
        T, N, K, dt = self.T, self.N, self.K, self.dtype
        args = (_ptr(dY2, (T, K), dt, "dY2"), _ptr(W2, self.w_shape, dt, "W2"),
                _ptr(aux, (T, self.aux_words), torch.int32, "aux"), _ptr(G, (T, N), dt, "G"),
                _ptr(dZ, (T, N), self.out_dtype, "dZ"), _ptr(dbias, (N,), torch.float32, "dbias"))
        _check(lib().drelu_bgrad_unfused_execute(self.handle, *args, _stream_ptr(stream)))

    # prebuilt calls: (fn, args) so that fn(*args) enqueues the C call with no
    # per-call argument checking (for tight launch loops; check rc yourself)
    def execute_call(self, X, W, bias, Y, aux=None, stream=None):
        T, N, K, dt = self.T, self.N, self.K, self.dtype
        args = (self.handle, _ptr(X, (T, K), dt, "X"), _ptr(W, self.w_shape, dt, "W"), _ptr(bias, (N,), self.bias_dtype, "bias"),
                _ptr(Y, (T, N), self.out_dtype, "Y"), self._aux(aux), _stream_ptr(stream))
        return lib().gemm_epi_execute, args

    def drelu_bgrad_call(self, dY2, W2, aux, dZ, dbias, stream=None):
        T, N, K, dt = self.T, self.N, self.K, self.dtype
        args = (self.handle, _ptr(dY2, (T, K), dt, "dY2"), _ptr(W2, self.w_shape, dt, "W2"),
                _ptr(aux, (T, self.aux_words), torch.int32, "aux"), _ptr(dZ, (T, N), self.out_dtype, "dZ"),
                _ptr(dbias, (N,), torch.float32, "dbias"), _stream_ptr(stream))
        return lib().drelu_bgrad_execute, args

    def wgrad_call(self, X, dZ, dW, dbias=None, stream=None):
        T, N, K, dt = self.T, self.N, self.K, self.dtype
        args = (self.handle, _ptr(X, (T, K), dt, "X"), _ptr(dZ, (T, N), dt, "dZ"),
                _ptr(dW, (K, N), self.out_dtype, "dW"),
                _ptr(dbias, (K,), torch.float32, "dbias"), _stream_ptr(stream))
        return lib().gemm_epi_wgrad_execute, args

    def unfused_call(self, X, W, bias, T1, T2, Y, aux=None, stream=None):
        T, N, K, dt = self.T, self.N, self.K, self.dtype
        args = (self.handle, _ptr(X, (T, K), dt, "X"), _ptr(W, self.w_shape, dt, "W"), _ptr(bias, (N,), self.bias_dtype, "bias"),
                _ptr(T1, (T, N), dt, "T1"), _ptr(T2, (T, N), dt, "T2"), _ptr(Y, (T, N), self.out_dtype, "Y"),
                self._aux(aux), _stream_ptr(stream))
        return lib().gemm_epi_unfused_execute, args

    def drelu_bgrad_unfused_call(self, dY2, W2, aux, G, dZ, dbias, stream=None):
        T, N, K, dt = self.T, self.N, self.K, self.dtype
        args = (self.handle, _ptr(dY2, (T, K), dt, "dY2"), _ptr(W2, self.w_shape, dt, "W2"),
                _ptr(aux, (T, self.aux_words), torch.int32, "aux"), _ptr(G, (T, N), dt, "G"),
                _ptr(dZ, (T, N), self.out_dtype, "dZ"), _ptr(dbias, (N,), torch.float32, "dbias"), _stream_ptr(stream))
        return lib().drelu_bgrad_unfused_execute, args

    # conveniences that allocate their outputs on the call's stream (allocation
    # happens in torch, outside the library; the library call allocates nothing)
    def forward(self, X, W, bias, stream=None):
        Y = _empty((self.T, self.N), self.out_dtype, X.device, stream)
        spec = self.aux_spec()
        aux = _empty(*spec, X.device, stream) if spec else None
        self.gemm_epi_execute(X, W, bias, Y, aux, stream)
        return Y, aux

    def backward(self, dY2, W2, aux, stream=None):
        dZ = _empty((self.T, self.N), self.out_dtype, dY2.device, stream)
        dbias = _empty((self.N,), torch.float32, dY2.device, stream)
        self.drelu_bgrad_execute(dY2, W2, aux, dZ, dbias, stream)
        return dZ, dbias

    def wgrad(self, X, dZ, with_dbias=False, stream=None):
        dW = _empty((self.K, self.N), self.out_dtype, X.device, stream)
        dbias = _empty((self.K,), torch.float32, X.device, stream) if with_dbias else None
        self.gemm_epi_wgrad_execute(X, dZ, dW, dbias, stream)
        return (dW, dbias) if with_dbias else dW


def _raw_stream(index: int, stream) -> int:
    """The stream's handle; without one, the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream_ptr(stream)


def _ptr_on(index: int, t, shape, dtype, name) -> int:
    """_ptr of a tensor that must be on CUDA device ``index``: one test for the
    tensor that is right (these checks are most of a small call's host time);
    _ptr says what is wrong with another."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    _ptr(t, shape, dtype, name)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


class _DevicePlan(Plan):
    """What plans bound to one device share: tensors are checked to be on it,
    and the default stream is its current one."""

    def _own(self, handle):
        self.handle = handle
        if not handle:
            raise GemmEpiError(ERR_INVALID_ARG, gemm_epi_last_error())
        self.index = torch.cuda.current_device()

    def _p(self, t, shape, dtype, name):
        if t is None:
            return None
        return _ptr_on(self.index, t, shape, dtype, name)

    def _s(self, stream) -> int:
        return _raw_stream(self.index, stream)


class GroupedPlan(_DevicePlan):
    """A plan for E products over rows sorted by expert: expert e owns rows
    ``offsets[e] .. offsets[e+1] - 1`` of X (T rows in all), where ``offsets``
    is an int32 CUDA tensor of E + 1 entries that only the kernel reads.

    W is E x K x N (``w_nk``: E x N x K), bias E x N, dW E x K x N, dbias E x N
    (DRELU_BGRAD) or E x K (WGRAD). Rows outside every expert are left as they
    were in Y, dZ and aux; an expert without rows gets zeros in dW and dbias.
    Tensors must be on the device that was current when the plan was made; the
    default stream is that device's current one."""

    def __init__(self, E: int, T: int, N: int, K: int, dtype: torch.dtype, epilog: str | int, w_nk: bool = False,
                 out_f32: bool = False):
        self.E, self.T, self.N, self.K = E, T, N, K
        self.out_dtype = torch.float32 if out_f32 else dtype
        self.w_shape = (E, N, K) if w_nk else (E, K, N)
        self.dtype = self.bias_dtype = dtype
        self.epilog = EPILOGS[epilog] if isinstance(epilog, str) else epilog
        self.aux_words = (N + 31) // 32
        self._shapes = ((T, K), (E, N), (E + 1,), (T, N), (T, self.aux_words), (E, K, N), (E, K))
        self._own(lib().gemm_epi_grouped_plan(E, T, N, K, DTYPES[dtype], self.epilog,
                                              (FLAG_W_NK if w_nk else 0) | (FLAG_OUT_F32 if out_f32 else 0)))

    def _aux(self, aux):
        spec = self.aux_spec() or ((self.T, self.aux_words), torch.int32)
        return self._p(aux, spec[0], spec[1], "aux")

    def gemm_epi_grouped_execute(self, X, W, bias, offsets, Y, aux=None, stream=None):
        i, dt, (xs, bs, os, ys, *_) = self.index, self.dtype, self._shapes
        _check(lib().gemm_epi_grouped_execute(
            self.handle, _ptr_on(i, X, xs, dt, "X"), _ptr_on(i, W, self.w_shape, dt, "W"),
            None if bias is None else _ptr_on(i, bias, bs, self.bias_dtype, "bias"),
            _ptr_on(i, offsets, os, torch.int32, "offsets"), _ptr_on(i, Y, ys, self.out_dtype, "Y"),
            None if aux is None else self._aux(aux), self._s(stream)))

    def gemm_epi_grouped_drelu_bgrad_execute(self, dY2, W2, aux, offsets, dZ, dbias, stream=None):
        i, dt, (xs, bs, os, ys, ms, *_) = self.index, self.dtype, self._shapes
        _check(lib().gemm_epi_grouped_drelu_bgrad_execute(
            self.handle, _ptr_on(i, dY2, xs, dt, "dY2"), _ptr_on(i, W2, self.w_shape, dt, "W2"),
            _ptr_on(i, aux, ms, torch.int32, "aux"), _ptr_on(i, offsets, os, torch.int32, "offsets"),
            _ptr_on(i, dZ, ys, self.out_dtype, "dZ"), _ptr_on(i, dbias, bs, torch.float32, "dbias"), self._s(stream)))

    def gemm_epi_grouped_wgrad_execute(self, X, dZ, offsets, dW, dbias=None, stream=None):
        i, dt, (xs, _, os, ys, _, ws, db) = self.index, self.dtype, self._shapes
        _check(lib().gemm_epi_grouped_wgrad_execute(
            self.handle, _ptr_on(i, X, xs, dt, "X"), _ptr_on(i, dZ, ys, dt, "dZ"),
            _ptr_on(i, offsets, os, torch.int32, "offsets"), _ptr_on(i, dW, ws, self.out_dtype, "dW"),
            None if dbias is None else _ptr_on(i, dbias, db, torch.float32, "dbias"), self._s(stream)))

    # conveniences that allocate their outputs (rows outside every expert: zeros)
    def forward(self, X, W, bias, offsets, stream=None):
        Y = _zeros((self.T, self.N), self.out_dtype, X.device, stream)
        spec = self.aux_spec()
        aux = _zeros(*spec, X.device, stream) if spec else None
        self.gemm_epi_grouped_execute(X, W, bias, offsets, Y, aux, stream)
        return Y, aux

    def backward(self, dY2, W2, aux, offsets, stream=None):
        dZ = _zeros((self.T, self.N), self.out_dtype, dY2.device, stream)
        dbias = _empty((self.E, self.N), torch.float32, dY2.device, stream)
        self.gemm_epi_grouped_drelu_bgrad_execute(dY2, W2, aux, offsets, dZ, dbias, stream)
        return dZ, dbias

    def wgrad(self, X, dZ, offsets, with_dbias=False, stream=None):
        dW = _empty((self.E, self.K, self.N), self.out_dtype, X.device, stream)
        dbias = _empty((self.E, self.K), torch.float32, X.device, stream) if with_dbias else None
        self.gemm_epi_grouped_wgrad_execute(X, dZ, offsets, dW, dbias, stream)
        return (dW, dbias) if with_dbias else dW


def mx_scales_bytes(rows: int, cols: int, batch: int = 1, groups: int | None = None) -> int:
    """Bytes of the scales of ``batch`` microscaled matrices (or of rows in ``groups`` groups)."""
    n = lib().gemm_epi_mx_scales_bytes(batch, rows, cols, groups or 0)
    if n < 0:
        raise GemmEpiError(ERR_INVALID_ARG, gemm_epi_last_error())
    return n


def _mx_args(values, name, q, scales, offsets, transposed):
    """Check one quantisation call's tensors (``values``: the 16-bit or fp32
    side): device, batch, rows, cols, groups and the four pointers."""
    if not isinstance(values, torch.Tensor) or values.dim() not in (2, 3):
        raise ValueError(f"{name} must be a tensor of 2 or 3 dimensions")
    if not values.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    shape = values.shape
    flat = len(shape) == 2
    batch = 1 if flat else shape[0]
    rows, cols = (shape[-1], shape[-2]) if transposed else (shape[-2], shape[-1])
    if rows < 1 or cols < 32 or cols % 32 or batch < 1:
        raise ValueError(f"bad shape {tuple(shape)} of {name}: rows >= 1 and a multiple of 32 columns")
    index = values.get_device()
    if offsets is None:
        groups, tiles, po = 0, batch * ((rows + 127) // 128), None
    else:
        groups = offsets.numel() - 1
        tiles = rows // 128 + min(groups, rows)
        po = _ptr_on(index, offsets, (groups + 1,), torch.int32, "offsets")
        if groups < 1:
            raise ValueError("offsets must have at least 2 entries")
    pq = _ptr_on(index, q, (rows, cols // 2) if flat else (batch, rows, cols // 2), torch.uint8, "q")
    ps = _ptr_on(index, scales, (tiles * ((cols + 127) // 128) * 512,), torch.uint8, "scales")
    return index, batch, rows, cols, groups, _ptr_on(index, values, shape, values.dtype, name), pq, ps, po


def _on_device(index, fn, *args):
    """One call with device ``index`` current (the quantisation entry points run on the current device)."""
    if index == torch.cuda.current_device():
        _check(fn(*args))
    else:
        with torch.cuda.device(index):
            _check(fn(*args))


def gemm_epi_mx_quantize(src, q, scales, offsets=None, transposed=False, stream=None):
    """Quantise src (rows x cols, or batch x rows x cols; 16-bit) to microscaled
    4 bits: q (... x cols / 2, uint8) and scales (uint8, ``mx_scales_bytes``).
    transposed: src is (batch x) cols x rows. offsets: int32, rows in groups."""
    index, batch, rows, cols, groups, px, pq, ps, po = _mx_args(src, "src", q, scales, offsets, transposed)
    dtype = DTYPES.get(src.dtype)
    if dtype is None:
        raise ValueError(f"src has dtype {src.dtype}, expected float16 or bfloat16")
    _on_device(index, lib().gemm_epi_mx_quantize, batch, rows, cols, dtype, MX_TRANSPOSED if transposed else 0, px, po,
               groups, pq, ps, _raw_stream(index, stream))


def gemm_epi_mx_dequantize(q, scales, out, offsets=None, stream=None):
    """The values that q and scales stand for, into out (float16, bfloat16 or float32)."""
    index, batch, rows, cols, groups, px, pq, ps, po = _mx_args(out, "out", q, scales, offsets, False)
    f32 = out.dtype is torch.float32
    dtype = BF16 if f32 else DTYPES.get(out.dtype)
    if dtype is None:
        raise ValueError(f"out has dtype {out.dtype}, expected float16, bfloat16 or float32")
    _on_device(index, lib().gemm_epi_mx_dequantize, batch, rows, cols, dtype, FLAG_OUT_F32 if f32 else 0, pq, ps, po,
               groups, px, _raw_stream(index, stream))


def mx_quantize(src, offsets=None, transposed=False, stream=None):
    """gemm_epi_mx_quantize with allocated outputs, cleared first: (q, scales).
    A loop that keeps its buffers calls gemm_epi_mx_quantize itself."""
    rows, cols = (src.shape[-1], src.shape[-2]) if transposed else src.shape[-2:]
    q = _zeros((*src.shape[:-2], rows, cols // 2), torch.uint8, src.device, stream)
    n = mx_scales_bytes(rows, cols, src.shape[0] if src.dim() == 3 else 1, None if offsets is None else offsets.numel() - 1)
    scales = _zeros((n,), torch.uint8, src.device, stream)
    gemm_epi_mx_quantize(src, q, scales, offsets, transposed, stream)
    return q, scales


class MxPlan(_DevicePlan):
    """A plan for Y = epilog(X . W^T) of microscaled 4-bit operands: X T x K, W
    N x K (E given: E weights, rows grouped by expert as in GroupedPlan);
    epilog BIAS, RELU_BIAS, GELU_BIAS or NONE; Y and bias of ``dtype``."""

    def __init__(self, T: int, N: int, K: int, dtype: torch.dtype, epilog: str | int, E: int | None = None,
                 out_f32: bool = False):
        self.E, self.T, self.N, self.K = E, T, N, K
        self.out_dtype = torch.float32 if out_f32 else dtype
        self.dtype = self.bias_dtype = dtype
        self.epilog = EPILOGS[epilog] if isinstance(epilog, str) else epilog
        self._own(lib().gemm_epi_mx_plan(E or 0, T, N, K, DTYPES[dtype], self.epilog, FLAG_OUT_F32 if out_f32 else 0))
        self.x_scales = mx_scales_bytes(T, K, groups=E)
        self.w_scales = mx_scales_bytes(N, K, batch=E or 1)

    def gemm_epi_mx_execute(self, Xq, Xs, Wq, Ws, bias, Y, offsets=None, stream=None):
        """Operands as ``mx_quantize`` makes them; bias N (or E x N) values, or None for NONE."""
        E, T, N, K, u8 = self.E, self.T, self.N, self.K, torch.uint8
        w_shape = (N, K // 2) if Wq.dim() == 2 and E in (None, 1) else (E or 1, N, K // 2)
        b_shape = (N,) if bias is not None and bias.dim() == 1 and E in (None, 1) else (E or 1, N)
        _check(lib().gemm_epi_mx_execute(
            self.handle, self._p(Xq, (T, K // 2), u8, "Xq"), self._p(Xs, (self.x_scales,), u8, "Xs"),
            self._p(Wq, w_shape, u8, "Wq"), self._p(Ws, (self.w_scales,), u8, "Ws"),
            self._p(bias, b_shape, self.bias_dtype, "bias"),
            None if offsets is None else self._p(offsets, ((E or 0) + 1,), torch.int32, "offsets"),
            self._p(Y, (T, N), self.out_dtype, "Y"), self._s(stream)))

    def forward(self, Xq, Xs, Wq, Ws, bias, offsets=None, stream=None):
        Y = _zeros((self.T, self.N), self.out_dtype, Xq.device, stream)
        self.gemm_epi_mx_execute(Xq, Xs, Wq, Ws, bias, Y, offsets, stream)
        return Y


class GatedPlan(_DevicePlan):
    """A plan for a gated layer: Z = X . W + bias (2N columns, the gate's first),
    H = act(Z[:, :N]) * Z[:, N:], with act "SILU", "GELU" or "RELU".

    epilog "GATED": H. "GATED_AUX": H and Z (T x 2N, 16-bit), which the backward
    reads. "DGATED": dZ (T x 2N) from dY (T x K), W2 (K x N) and Z, and the bias
    gradient (2N), for which the plan holds a workspace unless ``dbias`` is False.
    W is K x 2N (``w_nk``: 2N x K; W2: N x K); ``out_f32``: H or dZ
    is fp32. bias may be None. Tensors must be on the device that was current
    when the plan was made; the default stream is that device's current one."""

    def __init__(self, T: int, N: int, K: int, dtype: torch.dtype, epilog: str = "GATED", act: str = "SILU",
                 w_nk: bool = False, out_f32: bool = False, dbias: bool = True):
        self.T, self.N, self.K = T, N, K
        self.out_dtype = torch.float32 if out_f32 else dtype
        self.dtype = self.bias_dtype = dtype
        self.epilog = GATED_EPILOGS[epilog] if isinstance(epilog, str) else epilog
        cols = N if self.epilog == GATED_EPILOGS["DGATED"] else 2 * N
        self.w_shape = (cols, K) if w_nk else (K, cols)
        self._shapes = ((T, K), (T, N), (T, 2 * N), (2 * N,))
        self._own(lib().gemm_epi_gated_plan(T, N, K, DTYPES[dtype], self.epilog, ACTS[act] if isinstance(act, str) else act,
                                            (FLAG_W_NK if w_nk else 0) | (FLAG_OUT_F32 if out_f32 else 0) |
                                            (FLAG_NO_DBIAS if not dbias else 0)))

    def aux_spec(self):
        return (self._shapes[2], self.dtype) if self.epilog == GATED_EPILOGS["GATED_AUX"] else None

    def gemm_epi_gated_execute(self, X, W, bias, H, aux=None, stream=None):
        i, dt, (xs, hs, zs, bs) = self.index, self.dtype, self._shapes
        _check(lib().gemm_epi_gated_execute(
            self.handle, _ptr_on(i, X, xs, dt, "X"), _ptr_on(i, W, self.w_shape, dt, "W"),
            None if bias is None else _ptr_on(i, bias, bs, self.bias_dtype, "bias"),
            _ptr_on(i, H, hs, self.out_dtype, "H"), None if aux is None else _ptr_on(i, aux, zs, dt, "aux"),
            self._s(stream)))

    def gemm_epi_dgated_execute(self, dY, W2, aux, dZ, dbias=None, stream=None):
        i, dt, (xs, _, zs, bs) = self.index, self.dtype, self._shapes
        _check(lib().gemm_epi_dgated_execute(
            self.handle, _ptr_on(i, dY, xs, dt, "dY"), _ptr_on(i, W2, self.w_shape, dt, "W2"),
            _ptr_on(i, aux, zs, dt, "aux"), _ptr_on(i, dZ, zs, self.out_dtype, "dZ"),
            None if dbias is None else _ptr_on(i, dbias, bs, torch.float32, "dbias"), self._s(stream)))

    # conveniences that allocate their outputs on the call's stream
    def forward(self, X, W, bias=None, stream=None):
        H = _empty((self.T, self.N), self.out_dtype, X.device, stream)
        spec = self.aux_spec()
        aux = _empty(*spec, X.device, stream) if spec else None
        self.gemm_epi_gated_execute(X, W, bias, H, aux, stream)
        return H, aux

    def backward(self, dY, W2, aux, with_dbias=False, stream=None):
        dZ = _empty((self.T, 2 * self.N), self.out_dtype, dY.device, stream)
        dbias = _empty((2 * self.N,), torch.float32, dY.device, stream) if with_dbias else None
        self.gemm_epi_dgated_execute(dY, W2, aux, dZ, dbias, stream)
        return (dZ, dbias) if with_dbias else dZ


def w4_empty(N: int, K: int, dtype: torch.dtype, group: int = 128, zeros: bool = False, batch: int = 1, device=None,
             stream=None):
    """Uninitialised (q, scales, zeros or None) of ``batch`` weights of N x K held in 4 bits
    with a scale (and zero point) for each ``group`` columns. All three are flat."""
    nq, ns = lib().gemm_epi_w4_bytes(batch, N, K, group), lib().gemm_epi_w4_scales(batch, N, K, group)
    if nq < 0 or ns < 0:
        raise GemmEpiError(ERR_INVALID_ARG, gemm_epi_last_error())
    device = torch.device("cuda") if device is None else device
    return (_empty((nq,), torch.uint8, device, stream), _empty((ns,), dtype, device, stream),
            _empty((ns,), torch.uint8, device, stream) if zeros else None)


def _w4_args(values, name, q, scales, zeros, group, dtype, cols):
    """Check one call's tensors: ``values`` is (batch x) N x ``cols(shape)`` on the device of all;
    device, batch, N, K and the pointers of values, q, scales, zeros."""
    if not isinstance(values, torch.Tensor) or values.dim() not in (2, 3):
        raise ValueError(f"{name} must be a tensor of 2 or 3 dimensions")
    if not values.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    index, batch, N, K = values.get_device(), 1 if values.dim() == 2 else values.shape[0], values.shape[-2], cols(values.shape)
    if group in (32, 64, 128):  # (the sizes here: two calls of the library less; it checks the shape)
        tiles = batch * ((N + 31) // 32) * ((K + 127) // 128)
        nq, ns = 2048 * tiles, 32 * (128 // group) * tiles
    else:
        nq, ns = lib().gemm_epi_w4_bytes(batch, N, K, group), -1
    if nq < 0 or ns < 0:
        raise GemmEpiError(ERR_INVALID_ARG, gemm_epi_last_error())
    return (index, batch, N, K, _ptr_on(index, values, values.shape, values.dtype, name),
            _ptr_on(index, q, (nq,), torch.uint8, "q"), _ptr_on(index, scales, (ns,), dtype, "scales"),
            None if zeros is None else _ptr_on(index, zeros, (ns,), torch.uint8, "zeros"))


def gemm_epi_w4_quantize(W, q, scales, zeros=None, group=128, stream=None):
    """Quantise W (N x K or batch x N x K, 16-bit) to 4 bits: q, scales (W's type) and, if given, zeros."""
    dtype = DTYPES.get(getattr(W, "dtype", None))
    if dtype is None:
        raise ValueError("W must be a float16 or bfloat16 tensor")
    index, batch, N, K, pw, pq, ps, pz = _w4_args(W, "W", q, scales, zeros, group, W.dtype, lambda s: s[-1])
    _on_device(index, lib().gemm_epi_w4_quantize, batch, N, K, group, dtype, pw, pq, ps, pz, _raw_stream(index, stream))


def gemm_epi_w4_dequantize(q, scales, zeros, out, group=128, stream=None):
    """The values that q, scales and zeros (or None) stand for, into out (the scales' type, or float32)."""
    dtype = DTYPES.get(getattr(scales, "dtype", None))
    if dtype is None or getattr(out, "dtype", None) not in (scales.dtype, torch.float32):
        raise ValueError("scales must be float16 or bfloat16, and out of that type or float32")
    index, batch, N, K, po, pq, ps, pz = _w4_args(out, "out", q, scales, zeros, group, scales.dtype, lambda s: s[-1])
    _on_device(index, lib().gemm_epi_w4_dequantize, batch, N, K, group, dtype,
               FLAG_OUT_F32 if out.dtype is torch.float32 else 0, pq, ps, pz, po, _raw_stream(index, stream))


def gemm_epi_w4_pack(codes, src_scales, src_zeros, q, scales, zeros=None, stream=None):
    """Row-major codes ((batch x) N x K / 2 bytes, the lower column in the low 4 bits), scales ((batch x)
    N x K / group) and zeros (the same, uint8 of 0 .. 127, or None) to the product's layout. A group
    whose zero point is 128 or more gets a NaN scale."""
    if getattr(src_scales, "dtype", None) not in DTYPES or getattr(codes, "dtype", None) is not torch.uint8:
        raise ValueError("codes must be uint8, scales float16 or bfloat16")
    K, groups = 2 * codes.shape[-1], src_scales.shape[-1]
    group = K // groups if groups else 0
    if (src_zeros is None) != (zeros is None):
        raise ValueError("zeros on one side alone")
    index, batch, N, K, pc, pq, ps, pz = _w4_args(codes, "codes", q, scales, zeros, group, src_scales.dtype,
                                                  lambda s: 2 * s[-1])
    shape = (*codes.shape[:-1], K // group)
    sc = _ptr_on(index, src_scales, shape, src_scales.dtype, "scales")
    sz = None if src_zeros is None else _ptr_on(index, src_zeros, shape, torch.uint8, "zeros")
    _on_device(index, lib().gemm_epi_w4_pack, batch, N, K, group, pc, sc, sz, pq, ps, pz, _raw_stream(index, stream))


def w4_quantize(W, group=128, zeros=False, stream=None):
    """gemm_epi_w4_quantize with allocated outputs: (q, scales, zeros or None)."""
    out = w4_empty(W.shape[-2], W.shape[-1], W.dtype, group, zeros, W.shape[0] if W.dim() == 3 else 1, W.device, stream)
    gemm_epi_w4_quantize(W, *out, group=group, stream=stream)
    return out


def w4_pack(codes, scales, zeros=None, stream=None):
    """gemm_epi_w4_pack with allocated outputs: (q, scales, zeros or None)."""
    K, groups = 2 * codes.shape[-1], scales.shape[-1]
    out = w4_empty(codes.shape[-2], K, scales.dtype, K // groups if groups else 0, zeros is not None,
                   codes.shape[0] if codes.dim() == 3 else 1, codes.device, stream)
    gemm_epi_w4_pack(codes, scales, zeros, *out, stream=stream)
    return out


class W4Plan(_DevicePlan):
    """A plan for Y = epilog(X . W^T) of few 16-bit rows (T <= 256) and a weight held in 4
    bits with a scale for each ``group`` columns (w4_quantize, w4_pack): epilog BIAS,
    RELU_BIAS, GELU_BIAS or NONE, or "GATED": two weights of N rows (a batch of two, the
    gate's first), H = act(X . W0^T) * (X . W1^T) with act "SILU", "GELU" or "RELU"."""

    def __init__(self, T: int, N: int, K: int, dtype: torch.dtype, epilog: str | int, group: int = 128, act: str = "SILU",
                 out_f32: bool = False):
        self.T, self.N, self.K, self.group = T, N, K, group
        self.out_dtype = torch.float32 if out_f32 else dtype
        self.dtype = self.bias_dtype = dtype
        self.epilog = {**EPILOGS, **GATED_EPILOGS}[epilog] if isinstance(epilog, str) else epilog
        gated = self.epilog == GATED_EPILOGS["GATED"]
        self._own(lib().gemm_epi_w4_plan(T, N, K, group, DTYPES[dtype], self.epilog,
                                         ACTS[act] if isinstance(act, str) else act, FLAG_OUT_F32 if out_f32 else 0))
        batch = 2 if gated else 1
        self._shapes = ((T, K), (lib().gemm_epi_w4_bytes(batch, N, K, group),),
                        (lib().gemm_epi_w4_scales(batch, N, K, group),), (batch * N,), (T, N))

    def aux_spec(self):
        return None

    def gemm_epi_w4_execute(self, X, q, scales, zeros, bias, Y, stream=None):
        """q, scales and zeros (None: 8 everywhere) as w4_quantize and w4_pack make them; bias
        N (gated: 2N) values, or None for NONE and GATED."""
        i, dt, (xs, qs, ss, bs, ys) = self.index, self.dtype, self._shapes
        _check(lib().gemm_epi_w4_execute(
            self.handle, _ptr_on(i, X, xs, dt, "X"), _ptr_on(i, q, qs, torch.uint8, "q"),
            _ptr_on(i, scales, ss, dt, "scales"), None if zeros is None else _ptr_on(i, zeros, ss, torch.uint8, "zeros"),
            None if bias is None else _ptr_on(i, bias, bs, self.bias_dtype, "bias"),
            _ptr_on(i, Y, ys, self.out_dtype, "Y"), self._s(stream)))

    def forward(self, X, q, scales, zeros=None, bias=None, stream=None):
        Y = _empty((self.T, self.N), self.out_dtype, X.device, stream)
        self.gemm_epi_w4_execute(X, q, scales, zeros, bias, Y, stream)
        return Y
