"""quantized_weight_linear_gb300 -- Python binding of libqlin (quantized linear forward on GB300).

The library (``libqlin.so``, built from ``csrc/`` for sm_103a) implements
Y = X . W_hat^T for three compressed weight formats -- W4 g128 (GPTQ page),
SpQR 3-bit g16 with fp16 outliers (SpQR page) and SmoothQuant W8A8
(SmoothQuant page) -- behind a C ABI declared in ``include/qlin.h``.  This module
only marshals arguments: it loads the library with ctypes, mirrors its entry
points under the same names, and offers ``QLinear``, which uses PyTorch for device
memory and streams.  Every step of the forward runs in the library's kernels;
there is no other code path, and importing the package fails loudly if the
library is missing.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlin.so")

QLIN_OK = 0
QLIN_ERR_INVALID_ARG = 1
QLIN_ERR_UNSUPPORTED = 2
QLIN_ERR_CUDA = 3
QLIN_ERR_WORKSPACE = 4
QLIN_ERR_TIMEOUT = 5
QLIN_ERR_NOT_BOUND = 6

FMT_W4G128 = 1
FMT_SPQR = 2
FMT_W8A8 = 3

KV_INT8 = 1
KV_E4M3 = 2
KV_BLOCK = 16  # tokens of a cache block (one key and one value scale per block and head)

#: every entry point include/qlin.h declares
EXPORTED_SYMBOLS = (
    "qlin_pack_w4g128", "qlin_pack_w4g128_gptq", "qlin_pack_spqr", "qlin_pack_w8", "qlin_device_bytes",
    "qlin_workspace_bytes",
    "qlin_bind", "qlin_attach", "qlin_set_workspace", "qlin_forward", "qlin_forward_host", "qlin_act_quant",
    "qlin_forward_acc", "qlin_dequant_device", "qlin_poll_status", "qlin_export", "qlin_info",
    "qlin_destroy", "qlin_status_string", "qlin_sm_count", "qlin_debug_wait_timeout", "qlin_forward_spqr_static",
    "qlin_poll_static_status", "qlin_import",
    "qlin_kv_workspace_bytes", "qlin_kv_init_workspace", "qlin_kv_append", "qlin_kv_read", "qlin_kv_attend",
    "qlin_kv_poll_status",
)


class QlinError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class LayerInfo(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("nnz", ctypes.c_int64),
                ("packed_bytes", ctypes.c_int64), ("bits_per_param", ctypes.c_double),
                ("device_bytes", ctypes.c_int64), ("alpha", ctypes.c_float), ("outlier_frac", ctypes.c_float)]


class Canonical(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("codes", "scale", "zero", "codes3", "qs3", "qz3", "stats", "rowptr",
                                               "col", "val", "qw", "sw", "s", "s_inv", "perm")]


class KvCacheStruct(ctypes.Structure):
    _fields_ = [("code", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


class KvBatchStruct(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("total_q", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("max_kv", ctypes.c_int32), ("pages_width", ctypes.c_int32), ("pages_stride", ctypes.c_int64),
                ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("pages", ctypes.c_void_p)]


class HeadsStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class RopeStruct(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("n_pos", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Loads libqlin.so (raises if it was not built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libqlin.so not found at {LIB_PATH}; build it with "
                              "`python -m quantized_weight_linear_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        H = ctypes.c_void_p
        sig = {
            "qlin_pack_w4g128": ([vp, i32, i32, ctypes.POINTER(H)], i32),
            "qlin_pack_w4g128_gptq": ([vp, i32, i32, vp, i32, ctypes.c_double, i32, ctypes.POINTER(H)], i32),
            "qlin_pack_spqr": ([vp, i32, i32, f32, ctypes.POINTER(H)], i32),
            "qlin_pack_w8": ([vp, i32, i32, vp, f32, ctypes.POINTER(H)], i32),
            "qlin_device_bytes": ([H, ctypes.POINTER(sz)], i32),
            "qlin_workspace_bytes": ([H, i32, ctypes.POINTER(sz)], i32),
            "qlin_bind": ([H, vp, sz, vp], i32),
            "qlin_attach": ([H, vp, sz], i32),
            "qlin_set_workspace": ([H, vp, sz, i32, vp], i32),
            "qlin_forward": ([H, vp, vp, i32, vp], i32),
            "qlin_forward_host": ([H, vp, vp, vp, vp, i32, vp], i32),
            "qlin_act_quant": ([H, vp, vp, vp, i32, vp], i32),
            "qlin_forward_acc": ([H, vp, vp, i32, vp], i32),
            "qlin_dequant_device": ([H, vp, vp], i32),
            "qlin_poll_status": ([H, vp], i32),
            "qlin_export": ([H, ctypes.POINTER(Canonical)], i32),
            "qlin_info": ([H, ctypes.POINTER(LayerInfo)], i32),
            "qlin_destroy": ([H], None),
            "qlin_status_string": ([i32], ctypes.c_char_p),
            "qlin_sm_count": ([], i32),
            "qlin_debug_wait_timeout": ([vp, i32, vp], i32),
            "qlin_forward_spqr_static": ([H, vp, vp, i32, vp], i32),
            "qlin_poll_static_status": ([vp], i32),
            "qlin_import": ([i32, i32, i32, ctypes.POINTER(Canonical), ctypes.POINTER(H)], i32),
            "qlin_kv_workspace_bytes": ([vp, ctypes.POINTER(sz)], i32),
            "qlin_kv_init_workspace": ([vp, sz, vp], i32),
            "qlin_kv_append": ([vp, vp, vp, vp, vp, i32, vp, vp, vp, vp], i32),
            "qlin_kv_read": ([vp, vp, vp, vp, vp, vp], i32),
            "qlin_kv_attend": ([vp, vp, vp, i32, f32, i32, i32, vp, vp, vp, sz, vp], i32),
            "qlin_kv_poll_status": ([vp, vp], i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
        return L


def status_string(status: int) -> str:
    return lib().qlin_status_string(status).decode()


def _check(status: int, what: str):
    if status != QLIN_OK:
        raise QlinError(status, what)


def _f32(a) -> np.ndarray:
    return np.ascontiguousarray(a, dtype=np.float32)


def _vp(x) -> ctypes.c_void_p:
    """Pointer of a numpy array, a torch tensor, an int address or None."""
    if x is None:
        return ctypes.c_void_p(None)
    if isinstance(x, int):
        return ctypes.c_void_p(x)
    if isinstance(x, np.ndarray):
        return ctypes.c_void_p(x.ctypes.data)
    return ctypes.c_void_p(x.data_ptr())


def _stream(s) -> ctypes.c_void_p:
    if s is None:
        try:
            import torch
            if torch.cuda.is_available():
                return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        except Exception:  # pragma: no cover
            pass
        return ctypes.c_void_p(None)
    if isinstance(s, int):
        return ctypes.c_void_p(s)
    return ctypes.c_void_p(s.cuda_stream)


class Handle:
    """Owns a qlin_handle (host object); destroyed with the Python object."""

    def __init__(self, ptr: ctypes.c_void_p):
        self.ptr = ptr
        self._info = None

    def __del__(self):
        if getattr(self, "ptr", None) and self.ptr.value:
            try:
                lib().qlin_destroy(self.ptr)
            except Exception:  # pragma: no cover
                pass
            self.ptr = ctypes.c_void_p(None)

    @property
    def info(self) -> LayerInfo:
        if self._info is None:
            inf = LayerInfo()
            _check(lib().qlin_info(self.ptr, ctypes.byref(inf)), "qlin_info")
            self._info = inf
        return self._info


# -------------------------------------------------------------------------------- C ABI mirror

def qlin_pack_w4g128(W) -> Handle:
    W = _f32(W)
    h = ctypes.c_void_p()
    _check(lib().qlin_pack_w4g128(_vp(W), W.shape[0], W.shape[1], ctypes.byref(h)), "qlin_pack_w4g128")
    return Handle(h)


def qlin_pack_w4g128_gptq(W, Xcal, damp: float = 0.01, act_order: bool = False) -> Handle:
    W = _f32(W)
    X = _f32(Xcal)
    if X.ndim != 2 or X.shape[1] != W.shape[1]:
        raise ValueError("Xcal must be [S, K] with the layer's K")
    h = ctypes.c_void_p()
    _check(lib().qlin_pack_w4g128_gptq(_vp(W), W.shape[0], W.shape[1], _vp(X), X.shape[0], float(damp),
                                       int(bool(act_order)), ctypes.byref(h)), "qlin_pack_w4g128_gptq")
    return Handle(h)


def qlin_pack_spqr(W, outlier_frac: float) -> Handle:
    W = _f32(W)
    h = ctypes.c_void_p()
    _check(lib().qlin_pack_spqr(_vp(W), W.shape[0], W.shape[1], float(outlier_frac), ctypes.byref(h)),
           "qlin_pack_spqr")
    return Handle(h)


def qlin_pack_w8(W, act_absmax, alpha: float) -> Handle:
    W = _f32(W)
    a = _f32(act_absmax)
    h = ctypes.c_void_p()
    _check(lib().qlin_pack_w8(_vp(W), W.shape[0], W.shape[1], _vp(a), float(alpha), ctypes.byref(h)), "qlin_pack_w8")
    return Handle(h)


def qlin_device_bytes(h: Handle) -> int:
    n = ctypes.c_size_t()
    _check(lib().qlin_device_bytes(h.ptr, ctypes.byref(n)), "qlin_device_bytes")
    return n.value


def qlin_workspace_bytes(h: Handle, max_M: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().qlin_workspace_bytes(h.ptr, max_M, ctypes.byref(n)), "qlin_workspace_bytes")
    return n.value


def qlin_bind(h: Handle, dev_weights, nbytes: int, stream=None):
    _check(lib().qlin_bind(h.ptr, _vp(dev_weights), nbytes, _stream(stream)), "qlin_bind")


def qlin_attach(h: Handle, dev_weights, nbytes: int):
    _check(lib().qlin_attach(h.ptr, _vp(dev_weights), nbytes), "qlin_attach")


def qlin_set_workspace(h: Handle, dev_ws, nbytes: int, max_M: int, stream=None):
    _check(lib().qlin_set_workspace(h.ptr, _vp(dev_ws), nbytes, max_M, _stream(stream)), "qlin_set_workspace")


def qlin_forward(h: Handle, X, Y, M: int, stream=None):
    _check(lib().qlin_forward(h.ptr, _vp(X), _vp(Y), M, _stream(stream)), "qlin_forward")


def qlin_forward_spqr_static(h: Handle, X, Y, M: int, stream=None):
    """SpQR decode forward (1 <= M <= 16) that uses the library's fixed scratch array instead
    of a workspace: for callers that may not allocate device memory (see include/qlin.h)."""
    _check(lib().qlin_forward_spqr_static(h.ptr, _vp(X), _vp(Y), M, _stream(stream)), "qlin_forward_spqr_static")


def qlin_poll_static_status(stream=None) -> int:
    """Status of the qlin_forward_spqr_static calls on the current device since the last poll
    (waits for the stream; QLIN_OK or QLIN_ERR_TIMEOUT)."""
    return lib().qlin_poll_static_status(_stream(stream))


def qlin_forward_host(h: Handle, X_host, Y_host, X_dev, Y_dev, M: int, stream=None):
    _check(lib().qlin_forward_host(h.ptr, _vp(X_host), _vp(Y_host), _vp(X_dev), _vp(Y_dev), M, _stream(stream)),
           "qlin_forward_host")


def qlin_act_quant(h: Handle, X, qx, sx, M: int, stream=None):
    _check(lib().qlin_act_quant(h.ptr, _vp(X), _vp(qx), _vp(sx), M, _stream(stream)), "qlin_act_quant")


def qlin_forward_acc(h: Handle, X, acc, M: int, stream=None):
    _check(lib().qlin_forward_acc(h.ptr, _vp(X), _vp(acc), M, _stream(stream)), "qlin_forward_acc")


def qlin_dequant_device(h: Handle, out, stream=None):
    _check(lib().qlin_dequant_device(h.ptr, _vp(out), _stream(stream)), "qlin_dequant_device")


def qlin_poll_status(h: Handle, stream=None) -> int:
    return lib().qlin_poll_status(h.ptr, _stream(stream))


def qlin_sm_count() -> int:
    return lib().qlin_sm_count()


def qlin_debug_wait_timeout(status_dev, limit_us: int, stream=None):
    _check(lib().qlin_debug_wait_timeout(_vp(status_dev), limit_us, _stream(stream)), "qlin_debug_wait_timeout")


def qlin_export(h: Handle) -> dict:
    """Copies of the canonical packed arrays (layouts in include/qlin.h)."""
    c = Canonical()
    _check(lib().qlin_export(h.ptr, ctypes.byref(c)), "qlin_export")
    inf = h.info
    N, K, nnz = inf.N, inf.K, inf.nnz

    def arr(ptr, dtype, shape):
        count = int(np.prod(shape))
        if ptr is None or count == 0:
            return np.zeros(shape, dtype=dtype)
        buf = (ctypes.c_char * (count * np.dtype(dtype).itemsize)).from_address(ptr)
        return np.frombuffer(buf, dtype=dtype).reshape(shape).copy()

    if inf.format == FMT_W4G128:
        out = {"codes": arr(c.codes, np.uint32, (N, K // 8)),
               "scale": arr(c.scale, np.uint16, (N, K // 128)).view(np.float16),
               "zero": arr(c.zero, np.uint16, (N, K // 128)).view(np.float16)}
        if c.perm:  # act-order
            out["perm"] = arr(c.perm, np.int32, (K,))
        return out
    if inf.format == FMT_SPQR:
        return {"codes": arr(c.codes3, np.uint8, (N, 3 * K // 8)),
                "qs_bits": arr(c.qs3, np.uint8, (N, 3 * (K // 16) // 8)),
                "qz_bits": arr(c.qz3, np.uint8, (N, 3 * (K // 16) // 8)),
                "stats": arr(c.stats, np.uint16, (N, K // 256, 4)).view(np.float16),
                "rowptr": arr(c.rowptr, np.int32, (N + 1,)),
                "col": arr(c.col, np.int16, (nnz,)),
                "val": arr(c.val, np.uint16, (nnz,)).view(np.float16)}
    return {"qw": arr(c.qw, np.int8, (N, K)), "sw": arr(c.sw, np.float32, (N,)),
            "s": arr(c.s, np.float32, (K,)), "s_inv": arr(c.s_inv, np.float32, (K,))}


# canonical array names per format, with their dtypes (the dict qlin_export returns)
_CANONICAL = {
    FMT_W4G128: {"codes": np.uint32, "scale": np.float16, "zero": np.float16},
    FMT_SPQR: {"codes": np.uint8, "qs_bits": np.uint8, "qz_bits": np.uint8, "stats": np.float16,
               "rowptr": np.int32, "col": np.int16, "val": np.float16},
    FMT_W8A8: {"qw": np.int8, "sw": np.float32, "s": np.float32, "s_inv": np.float32},
}
_FIELD = {"codes3": "codes", "qs3": "qs_bits", "qz3": "qz_bits"}  # struct field -> dict key (SpQR)


def qlin_import(fmt: int, N: int, K: int, arrays: dict) -> Handle:
    """A handle from canonical arrays (a qlin_export dict or a loaded checkpoint); no quantization."""
    if fmt not in _CANONICAL:
        raise ValueError(f"unknown format {fmt}")
    keep = {k: np.ascontiguousarray(arrays[k], dtype=dt) for k, dt in _CANONICAL[fmt].items()}
    c = Canonical()
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p).value if a.size else None
    if fmt == FMT_W4G128:
        c.codes, c.scale, c.zero = ptr(keep["codes"]), ptr(keep["scale"]), ptr(keep["zero"])
        if arrays.get("perm") is not None:  # act-order
            keep["perm"] = np.ascontiguousarray(arrays["perm"], dtype=np.int32)
            c.perm = ptr(keep["perm"])
    elif fmt == FMT_SPQR:
        c.codes3, c.qs3, c.qz3 = ptr(keep["codes"]), ptr(keep["qs_bits"]), ptr(keep["qz_bits"])
        c.stats, c.rowptr, c.col, c.val = ptr(keep["stats"]), ptr(keep["rowptr"]), ptr(keep["col"]), ptr(keep["val"])
    else:
        c.qw, c.sw, c.s, c.s_inv = ptr(keep["qw"]), ptr(keep["sw"]), ptr(keep["s"]), ptr(keep["s_inv"])
    h = ctypes.c_void_p()
    _check(lib().qlin_import(int(fmt), int(N), int(K), ctypes.byref(c), ctypes.byref(h)), "qlin_import")
    return Handle(h)


# -------------------------------------------------------------------------------- torch front end

class QLinear:
    """A packed layer resident on one GPU; tensors come from PyTorch, compute from libqlin."""

    def __init__(self, handle: Handle):
        self.handle = handle
        inf = handle.info
        self.format, self.N, self.K = inf.format, inf.N, inf.K
        self.weights = None
        self.workspace = None
        self.max_M = 0

    @classmethod
    def from_w4g128(cls, W):
        return cls(qlin_pack_w4g128(W))

    @classmethod
    def from_w4g128_gptq(cls, W, Xcal, damp: float = 0.01, act_order: bool = False):
        return cls(qlin_pack_w4g128_gptq(W, Xcal, damp, act_order))

    @classmethod
    def from_spqr(cls, W, outlier_frac: float = 0.01):
        return cls(qlin_pack_spqr(W, outlier_frac))

    @classmethod
    def from_w8(cls, W, act_absmax, alpha: float = 0.85):
        return cls(qlin_pack_w8(W, act_absmax, alpha))

    def to(self, device="cuda", max_M: int = 16, stream=None):
        import torch
        nb = qlin_device_bytes(self.handle)
        self.weights = torch.empty(nb + 256, dtype=torch.uint8, device=device)
        w = self.weights[(-self.weights.data_ptr()) % 256:][:nb]
        qlin_bind(self.handle, w.data_ptr(), nb, stream)
        self.set_max_M(max_M, device, stream)
        return self

    def set_max_M(self, max_M: int, device="cuda", stream=None):
        import torch
        wb = qlin_workspace_bytes(self.handle, max_M)
        self.workspace = torch.empty(wb + 256, dtype=torch.uint8, device=device)
        ws = self.workspace[(-self.workspace.data_ptr()) % 256:][:wb]
        qlin_set_workspace(self.handle, ws.data_ptr(), wb, max_M, stream)
        self.max_M = max_M

    def _here(self, *tensors):
        """The library launches on the current device: the layer and its tensors have to be there."""
        import torch
        device = torch._C._cuda_getDevice()
        for x in (self.weights, *tensors):
            if x is not None and x.get_device() != device:
                raise ValueError(f"the current device is cuda:{device}, the layer or a tensor is on {x.device}")

    def __call__(self, X, out=None, stream=None):
        import torch
        self._here(X, out)
        assert X.dtype == torch.bfloat16 and X.is_contiguous() and X.shape[-1] == self.K
        M = X.shape[0]
        Y = out if out is not None else torch.empty((M, self.N), dtype=torch.bfloat16, device=X.device)
        qlin_forward(self.handle, X, Y, M, stream)
        return Y

    def forward_host(self, X_host, Y_host, X_dev, Y_dev, stream=None):
        self._here(X_dev, Y_dev)
        qlin_forward_host(self.handle, X_host, Y_host, X_dev, Y_dev, X_host.shape[0], stream)
        return Y_host

    def act_quant(self, X, stream=None):
        import torch
        self._here(X)
        M = X.shape[0]
        qx = torch.empty((M, self.K), dtype=torch.int8, device=X.device)
        sx = torch.empty((M,), dtype=torch.float32, device=X.device)
        qlin_act_quant(self.handle, X, qx, sx, M, stream)
        return qx, sx

    def forward_acc(self, X, stream=None):
        import torch
        self._here(X)
        M = X.shape[0]
        acc = torch.empty((M, self.N), dtype=torch.int32, device=X.device)
        qlin_forward_acc(self.handle, X, acc, M, stream)
        return acc

    def dequant_device(self, stream=None):
        import torch
        self._here()
        dt = torch.int8 if self.format == FMT_W8A8 else torch.float32
        out = torch.empty((self.N, self.K), dtype=dt, device=self.weights.device)
        qlin_dequant_device(self.handle, out, stream)
        return out

    def poll_status(self, stream=None) -> int:
        return qlin_poll_status(self.handle, stream)

    def export(self) -> dict:
        return qlin_export(self.handle)

    def save(self, path) -> None:
        """Writes the canonical packed arrays (the qlin_export layouts) to an .npz checkpoint."""
        np.savez(path, format=np.int32(self.format), N=np.int32(self.N), K=np.int32(self.K), **self.export())

    @classmethod
    def load(cls, path):
        """A layer from a checkpoint written by save(); the weights are not requantized."""
        with np.load(path) as z:
            fmt, N, K = int(z["format"]), int(z["N"]), int(z["K"])
            arrays = {k: z[k] for k in _CANONICAL.get(fmt, {})}
            if "perm" in z.files:
                arrays["perm"] = z["perm"]
            return cls(qlin_import(fmt, N, K, arrays))


# ------------------------------------------------------------------- 8-bit key/value cache

_KV_CODES = {"int8": KV_INT8, "e4m3": KV_E4M3}


class Rope:
    """Rotation tables: cos, sin fp32 [positions, rot_dim / 2] on the device (contiguous)."""

    def __init__(self, cos, sin, interleaved: bool = False):
        import torch
        if cos.shape != sin.shape or cos.dim() != 2:
            raise ValueError("cos and sin must both be [positions, rot_dim / 2]")
        for x in (cos, sin):
            if x.dtype != torch.float32 or not x.is_contiguous() or not x.is_cuda:
                raise ValueError("cos and sin must be contiguous fp32 device tensors")
        self.cos, self.sin, self.interleaved, self.index = cos, sin, bool(interleaved), cos.get_device()
        if sin.get_device() != self.index:
            raise ValueError("cos and sin must be on one device")
        self.struct = RopeStruct(cos.data_ptr(), sin.data_ptr(), cos.shape[0], 2 * cos.shape[1], int(self.interleaved))
        self.ref = ctypes.addressof(self.struct)


class KVBatch:
    """The sequences of one step, shared by all layers: q_start int32 [n + 1], kv_len int32 [n]
    and pages int32 [n, columns] on the device (a row's columns adjacent); total_q, max_q and
    max_kv are what the host knows of them (rows of the step, most rows of a sequence, longest
    sequence: a hint, which the present kernels do not need).  The kernels read the tensors when they run."""

    def __init__(self, q_start, kv_len, pages, total_q: int, max_q: int, max_kv: int):
        import torch
        n = kv_len.shape[0]
        for x in (q_start, kv_len, pages):
            if x.dtype != torch.int32 or not x.is_cuda:
                raise ValueError("q_start, kv_len and pages must be int32 device tensors")
        if q_start.shape != (n + 1,) or kv_len.dim() != 1 or pages.dim() != 2 or pages.shape[0] != n:
            raise ValueError("expected q_start [n + 1], kv_len [n], pages [n, columns]")
        if not q_start.is_contiguous() or not kv_len.is_contiguous() or (pages.shape[1] > 1 and pages.stride(1) != 1):
            raise ValueError("q_start, kv_len and the rows of pages must be contiguous")
        self.q_start, self.kv_len, self.pages, self.index = q_start, kv_len, pages, q_start.get_device()
        if kv_len.get_device() != self.index or pages.get_device() != self.index:
            raise ValueError("q_start, kv_len and pages must be on one device")
        self.n_seqs, self.total_q, self.max_q, self.max_kv = n, int(total_q), int(max_q), int(max_kv)
        stride = max(pages.stride(0), pages.shape[1]) if n > 1 else pages.shape[1]
        if n > 1 and pages.stride(0) < pages.shape[1]:
            raise ValueError("the rows of pages overlap")
        self.struct = KvBatchStruct(n, self.total_q, self.max_q, self.max_kv, pages.shape[1], stride,
                                    q_start.data_ptr(), kv_len.data_ptr(), pages.data_ptr())
        self.ref = ctypes.addressof(self.struct)


def _allocate_on(stream, make):
    """make() with its tensors belonging to `stream` (as a call takes it; None: the current one): memory that
    kernels queued elsewhere still use is not handed out to it."""
    import torch
    if stream is None:
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream).value or 0)
    with torch.cuda.stream(stream):
        return make()


class KVWorkspace:
    """Device workspace of cache calls (status word, counters, partial results) in a uint8 tensor: cleared
    when it is made, on `stream`, and not by the caches that are given it."""

    def __init__(self, memory, stream=None):
        import torch
        self.memory, self.index = memory, memory.get_device()
        if torch._C._cuda_getDevice() != self.index:
            raise ValueError("the workspace is not on the current device")
        self.ptr = memory.data_ptr() + (-memory.data_ptr()) % 256
        self.nbytes = memory.data_ptr() + memory.numel() - self.ptr
        on = torch._C._cuda_getCurrentRawStream(self.index) if stream is None else _stream(stream)
        _check(lib().qlin_kv_init_workspace(self.ptr, max(self.nbytes, 0), on), "qlin_kv_init_workspace")


class KVCache:
    """A paged 8-bit key/value cache of one layer and the attention over it (layouts and
    semantics in include/qlin.h).

    codes uint8 [n_pages, n_heads, 2, page_tokens * head_dim], scales fp32
    [n_pages, n_heads, page_tokens / 16, 2], both on the device; KVCache.empty allocates them.  That
    device has to be the current one in every call.  A call runs on `stream` (default: the current one),
    to which the tensors that it makes belong; the stream waits for the caller's inputs if the caller says so.
    A cache is not safe for concurrent calls from several threads.  Calls that share a workspace
    must not overlap on the GPU; caches whose calls follow one another (the layers of a model) can
    share one: KVCache(..., workspace=first.workspace), a KVWorkspace.  Their status is shared too.  A
    plain uint8 tensor is taken as fresh memory and cleared."""

    def __init__(self, codes, scales, code: str = "int8", workspace=None, stream=None):
        import torch
        if code not in _KV_CODES:
            raise ValueError(f"code must be one of {sorted(_KV_CODES)}")
        if codes.dtype != torch.uint8 or scales.dtype != torch.float32 or codes.dim() != 4 or scales.dim() != 4 or \
                codes.shape[2] != 2 or scales.shape[3] != 2 or codes.shape[:2] != scales.shape[:2]:
            raise ValueError("expected codes uint8 [n_pages, n_heads, 2, page_tokens * head_dim] and "
                             "scales fp32 [n_pages, n_heads, page_tokens / 16, 2]")
        if not codes.is_contiguous() or not scales.is_contiguous() or not codes.is_cuda or not scales.is_cuda:
            raise ValueError("codes and scales must be contiguous device tensors")
        self.codes, self.scales, self.code = codes, scales, code
        self.n_pages, self.n_heads = codes.shape[0], codes.shape[1]
        self.page_tokens = scales.shape[2] * KV_BLOCK
        if self.page_tokens == 0 or codes.shape[3] % self.page_tokens:
            raise ValueError("codes and scales do not describe the same pages")
        self.head_dim = codes.shape[3] // self.page_tokens
        # what every call needs, looked up once (a decoding step's calls are a few microseconds)
        self._lib, self._device, self._index = lib(), codes.device, codes.get_device()
        self._bf16, self._f32, self._empty, self._scale = torch.bfloat16, torch.float32, torch.empty, self.head_dim ** -0.5
        self._raw_stream, self._current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        self._args = (HeadsStruct(), HeadsStruct(), HeadsStruct())  # k, v, q of the call being made
        self._arg_refs = tuple(ctypes.addressof(x) for x in self._args)
        self.struct = KvCacheStruct(_KV_CODES[code], self.n_pages, self.n_heads, self.head_dim, self.page_tokens,
                                    codes.data_ptr(), scales.data_ptr())
        self.ref = ctypes.addressof(self.struct)
        self._on(stream)  # refuses another device's
        n = ctypes.c_size_t()
        _check(lib().qlin_kv_workspace_bytes(self.ref, ctypes.byref(n)), "qlin_kv_workspace_bytes")
        self.ws_bytes = n.value
        if workspace is None:
            workspace = _allocate_on(stream, lambda: torch.empty(n.value + 256, dtype=torch.uint8, device=codes.device))
        if scales.get_device() != self._index or (workspace.index if isinstance(workspace, KVWorkspace) else
                                                  workspace.get_device()) != self._index:
            raise ValueError("codes, scales and workspace must be on one device")
        if not isinstance(workspace, KVWorkspace):
            if (-workspace.data_ptr()) % 256 + n.value > workspace.numel():
                raise ValueError("workspace too small")
            workspace = KVWorkspace(workspace, stream)
        if workspace.nbytes < n.value:
            raise ValueError("workspace too small")
        self.workspace, self.ws = workspace, workspace.ptr

    @classmethod
    def empty(cls, n_pages: int, n_heads: int, head_dim: int, page_tokens: int = 64, code: str = "int8", device="cuda",
              workspace=None, stream=None):
        import torch
        codes, scales = _allocate_on(stream, lambda: (
            torch.empty((n_pages, n_heads, 2, page_tokens * head_dim), dtype=torch.uint8, device=device),
            torch.empty((n_pages, n_heads, page_tokens // KV_BLOCK, 2), dtype=torch.float32, device=device)))
        return cls(codes, scales, code, workspace, stream)

    def _heads(self, h, x, n_heads, rows, what):
        """Checks per-head rows and describes them in h; returns the number of heads."""
        shape = x.shape
        if x.dtype is not self._bf16 or len(shape) != 3 or shape[0] != rows or shape[2] != self.head_dim or \
                (n_heads is not None and shape[1] != n_heads) or x.get_device() != self._index:
            raise ValueError(f"{what} must be bf16 [{rows}, {n_heads or 'heads'}, {self.head_dim}] on the cache's device, "
                             f"got {x.dtype} {tuple(shape)} on {x.device}")
        stride = x.stride()
        if stride[2] != 1:
            raise ValueError(f"{what}: the elements of a head must be adjacent")
        h.data, h.token_stride, h.head_stride = x.data_ptr(), stride[0], stride[1]
        return shape[1]

    def _out(self, x, shape, dtype, what, stream):
        if x is None:
            if stream is not None:
                return _allocate_on(stream, lambda: self._empty(shape, dtype=dtype, device=self._device))
            return self._empty(shape, dtype=dtype, device=self._device)
        if x.dtype is not dtype or tuple(x.shape) != shape or not x.is_contiguous() or x.get_device() != self._index:
            raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {shape} on the cache's device")
        return x

    def _on(self, stream):
        """The stream's handle; by default the current one of the cache's device, which has to be the
        current device: the library launches on that one."""
        if self._current_device() != self._index:
            raise ValueError(f"the current device is cuda:{self._current_device()}, the cache is on cuda:{self._index}: "
                             f"call it under torch.cuda.device({self._index})")
        if stream is None:
            return self._raw_stream(self._index)
        if getattr(stream, "device_index", self._index) != self._index:
            raise ValueError("the stream is on another device than the cache")
        return _stream(stream)

    def _same_device(self, x, what):
        if x.index != self._index:
            raise ValueError(f"the {what} is on another device than the cache")

    def append(self, batch: KVBatch, k, v, q=None, rope: Rope = None, q_out=None, stream=None):
        """Stores the step's keys and values (bf16 [total_q, n_heads, head_dim], any token and
        head strides that are multiples of 8); keys and the queries q are rotated by rope.
        Returns the rotated queries [total_q, heads, head_dim], or None without q."""
        rows, ks, vs, qs = batch.total_q, *self._args
        on = self._on(stream)
        self._same_device(batch, "batch")
        self._heads(ks, k, self.n_heads, rows, "k")
        self._heads(vs, v, self.n_heads, rows, "v")
        if rope is not None:
            self._same_device(rope, "rope")
            rope = rope.ref
        if q is None:
            q_ref, nq, qo, q_ptr = None, 0, None, None
        else:
            q_ref, nq = self._arg_refs[2], self._heads(qs, q, None, rows, "q")
            qo = self._out(q_out, (rows, nq, self.head_dim), self._bf16, "q_out", stream)
            q_ptr = qo.data_ptr()
        st = self._lib.qlin_kv_append(self.ref, batch.ref, self._arg_refs[0], self._arg_refs[1], q_ref, nq, q_ptr, rope,
                                      self.ws, on)
        if st:
            raise QlinError(st, "qlin_kv_append")
        return qo

    def read(self, batch: KVBatch, stream=None):
        """The cached keys and values of the batch's tokens, bf16 [total_q, n_heads, head_dim] each."""
        on = self._on(stream)
        self._same_device(batch, "batch")
        shape = (batch.total_q, self.n_heads, self.head_dim)
        k, v = self._out(None, shape, self._bf16, "k", stream), self._out(None, shape, self._bf16, "v", stream)
        st = self._lib.qlin_kv_read(self.ref, batch.ref, k.data_ptr(), v.data_ptr(), self.ws, on)
        if st:
            raise QlinError(st, "qlin_kv_read")
        return k, v

    def attend(self, batch: KVBatch, q, scale: float = None, window: int = 0, sinks: int = 0, out=None, lse=None,
               return_lse: bool = False, stream=None):
        """Attention of the step's (rotated) queries, bf16 [total_q, heads, head_dim], over the
        cache.  window > 0: a query sees the last `window` positions up to its own and the first
        `sinks` ones.  scale defaults to head_dim ** -0.5.  Returns the output (and with
        return_lse the log-sum-exp of every row, fp32 [total_q, heads])."""
        rows = batch.total_q
        on = self._on(stream)
        self._same_device(batch, "batch")
        nq = self._heads(self._args[2], q, None, rows, "q")
        o = self._out(out, (rows, nq, self.head_dim), self._bf16, "out", stream)
        lse_ptr = None
        if lse is not None or return_lse:
            lse = self._out(lse, (rows, nq), self._f32, "lse", stream)
            lse_ptr = lse.data_ptr()
        st = self._lib.qlin_kv_attend(self.ref, batch.ref, self._arg_refs[2], nq, self._scale if scale is None else scale,
                                      window, sinks, o.data_ptr(), lse_ptr, self.ws, self.ws_bytes, on)
        if st:
            raise QlinError(st, "qlin_kv_attend")
        return o if lse is None else (o, lse)

    def poll_status(self, stream=None) -> int:
        """Waits for the stream; QLIN_OK, QLIN_ERR_INVALID_ARG (a bad index was met since the
        last poll) or QLIN_ERR_TIMEOUT."""
        return self._lib.qlin_kv_poll_status(self.ws, self._on(stream))


def build(force: bool = False) -> str:
    from .build import build as _b
    return _b(force=force)
