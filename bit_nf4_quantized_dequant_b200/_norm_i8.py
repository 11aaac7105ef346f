"""ctypes binding of ``include/qlora_i8.h``: the RMS norm and the 8-bit integer
linear. As in ``_binding``, every function maps onto one C entry point and
allocates what the caller does not pass; no step of the computation runs here.

Shapes, types, devices and contiguity are checked here, since the C side only
sees pointers: a tensor that does not fit raises ``ValueError`` before the call.
"""

from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch

from . import _binding

__all__ = [
    "I8Matrix", "SYMBOLS_I8", "i8_quantize", "i8_dequantize", "rmsnorm_fwd", "rmsnorm_bwd", "rmsnorm_workspace",
    "i8_linear_fwd", "i8_linear_dx", "i8_linear_workspace",
]

# every symbol include/qlora_i8.h declares
SYMBOLS_I8 = [
    "qlora_i8_quantize", "qlora_i8_dequantize", "qlora_rmsnorm_fwd", "qlora_rmsnorm_workspace", "qlora_rmsnorm_bwd",
    "qlora_i8_linear_fwd", "qlora_i8_linear_workspace", "qlora_i8_linear_dx",
]

_BF16, _F32, _I8 = torch.bfloat16, torch.float32, torch.int8
_TYPE = {_BF16: 0, _F32: 1}
_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = _binding.library()
        P, I32, I64, F, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        PSZ = ctypes.POINTER(SZ)
        for name, args in (
                ("qlora_i8_quantize", [P, I32, I64, I64, P, P, P, P]),
                ("qlora_i8_dequantize", [P, P, I64, I64, P, P]),
                ("qlora_rmsnorm_fwd", [P, P, I32, P, I32, F, I64, I64, P, P, P, P, P]),
                ("qlora_rmsnorm_workspace", [I64, I64, PSZ]),
                ("qlora_rmsnorm_bwd", [P, P, I32, P, I32, F, P, I64, I64, P, P, P, P, SZ, P]),
                ("qlora_i8_linear_fwd", [P, P, I64, P, P, I64, I64, P, P, I32, P, P, P]),
                ("qlora_i8_linear_workspace", [I64, I64, I64, PSZ]),
                ("qlora_i8_linear_dx", [P, I64, P, P, I64, I64, P, P, I32, P, P, SZ, P, P])):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        _lib = lib
    return _lib


def _need(t, name, dtype, shape, dev):
    """A contiguous tensor of this type (or one of these) and shape on CUDA device `dev`: its address."""
    if ((t.dtype is dtype or (dtype.__class__ is tuple and t.dtype in dtype)) and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    dtypes = dtype if isinstance(dtype, tuple) else (dtype,)
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")
    raise ValueError(f"{name}: not contiguous")


def _opt(t, name, dtype, shape, dev):
    return None if t is None else _need(t, name, dtype, shape, dev)


def _device(t, name):
    """The device of a call: that of its first tensor, which has to be the current one."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: on {t.device}, expected a CUDA device")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    return dev


@functools.lru_cache(maxsize=4096)
def _bytes(size, dev, *shape):
    """A workspace's size on device `dev` (the current one), which goes by its SM count and the shape alone."""
    return size(*shape)


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected a matrix")
    return t.shape


def _raw(stream, dev):
    """The handle of the stream to launch on: the given one, or the device's current one."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(like, shape, dtype, stream):
    """Memory on the device of `like`, from the current stream's pool; where another stream uses it, that is recorded."""
    t = like.new_empty(shape, dtype=dtype)
    if stream is not None and stream.cuda_stream != torch._C._cuda_getCurrentRawStream(t.get_device()):
        stream.wait_stream(torch.cuda.current_stream())   # the memory may still be in use here
        t.record_stream(stream)
    return t


_check = _binding._check


@dataclass
class I8Matrix:
    """Int8 rows: codes int8 [rows, cols] and one fp32 scale a row [rows]."""
    codes: torch.Tensor
    scale: torch.Tensor

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda"):
        return cls(torch.empty((rows, cols), dtype=_I8, device=device),
                   torch.empty(rows, dtype=_F32, device=device))


def _need_i8(q, name, shape, dev):
    return (_need(q.codes, name + ".codes", _I8, shape, dev),
            _need(q.scale, name + ".scale", _F32, shape[:1], dev))


def i8_quantize(X, col_scale=None, out: I8Matrix | None = None, stream=None) -> I8Matrix:
    """Int8 rows of X [M, K] (bf16 or fp32), or of X * col_scale[K]."""
    M, K = shape = _matrix(X, "X")
    dev = _device(X, "X")
    x = _need(X, "X", (_BF16, _F32), shape, dev)
    if out is None:
        out = I8Matrix(_empty(X, shape, _I8, stream), _empty(X, (M,), _F32, stream))
    codes, scale = _need_i8(out, "out", shape, dev)
    _check(_library().qlora_i8_quantize(x, _TYPE[X.dtype], M, K, _opt(col_scale, "col_scale", _F32, (K,), dev),
                                        codes, scale, _raw(stream, dev)), "qlora_i8_quantize")
    return out


def i8_dequantize(q: I8Matrix, out=None, stream=None):
    """codes * scale as bf16 [M, K]."""
    M, K = shape = _matrix(q.codes, "codes")
    dev = _device(q.codes, "codes")
    codes, scale = _need_i8(q, "q", shape, dev)
    if out is None:
        out = _empty(q.codes, shape, _BF16, stream)
    _check(_library().qlora_i8_dequantize(codes, scale, M, K, _need(out, "out", _BF16, shape, dev), _raw(stream, dev)),
           "qlora_i8_dequantize")
    return out


def rmsnorm_fwd(X, weight, eps: float, residual=None, H=None, Y=None, q: I8Matrix | None = None,
                want_H: bool = True, stream=None):
    """RMS norm of h = X + residual (either may be None). Returns (Y, H, q): the
    outputs that are passed are written; Y (bf16) is allocated when neither Y nor
    q (int8 rows) is passed, H (the stream's type) when both X and residual are
    given and want_H."""
    first = residual if residual is not None else X
    if first is None:
        raise ValueError("X or residual is needed")
    M, K = shape = _matrix(first, "residual" if residual is not None else "X")
    dev = _device(first, "residual" if residual is not None else "X")
    ht = _BF16 if residual is None else residual.dtype
    x = _opt(X, "X", _BF16, shape, dev)
    r = _opt(residual, "residual", (_BF16, _F32), shape, dev)
    w = _need(weight, "weight", (_BF16, _F32), (K,), dev)
    if Y is None and q is None:
        Y = _empty(first, shape, _BF16, stream)
    if H is None and want_H and X is not None and residual is not None:
        H = _empty(first, shape, ht, stream)
    codes, scale = (None, None) if q is None else _need_i8(q, "q", shape, dev)
    _check(_library().qlora_rmsnorm_fwd(x, r, _TYPE[ht], w, _TYPE[weight.dtype], eps, M, K,
                                        _opt(H, "H", ht, shape, dev), _opt(Y, "Y", _BF16, shape, dev),
                                        codes, scale, _raw(stream, dev)), "qlora_rmsnorm_fwd")
    return Y, H, q


def rmsnorm_workspace(M: int, K: int) -> int:
    b = ctypes.c_size_t()
    _check(_library().qlora_rmsnorm_workspace(M, K, ctypes.byref(b)), "qlora_rmsnorm_workspace")
    return b.value


def rmsnorm_bwd(dY, H, weight, eps: float, dres=None, dH=None, dX=None, dW=None, ws=None, want_dW: bool = True,
                stream=None, want_dH: bool = True):
    """(dH, dX, dW): the gradient of the stream h in its type (None without
    want_dH, for a first block's norm with dX passed), its bf16 copy (only when
    dX is passed) and the weight's (fp32, or None without want_dW)."""
    M, K = shape = _matrix(dY, "dY")
    dev = _device(dY, "dY")
    ht = H.dtype
    dy = _need(dY, "dY", _BF16, shape, dev)
    h = _need(H, "H", (_BF16, _F32), shape, dev)
    w = _need(weight, "weight", (_BF16, _F32), (K,), dev)
    dr = _opt(dres, "dres", ht, shape, dev)
    if dH is None and want_dH:
        dH = _empty(dY, shape, ht, stream)
    if dW is None and want_dW:
        dW = _empty(dY, (K,), _F32, stream)
    if dW is not None and ws is None:
        need = _bytes(rmsnorm_workspace, dev, M, K)
        ws = _empty(dY, (need,), torch.uint8, stream) if need else None
    _check(_library().qlora_rmsnorm_bwd(dy, h, _TYPE[ht], w, _TYPE[weight.dtype], eps, dr, M, K,
                                        _opt(dH, "dH", ht, shape, dev), _opt(dX, "dX", _BF16, shape, dev),
                                        _opt(dW, "dW", _F32, (K,), dev), *_space(ws, dev), _raw(stream, dev)),
           "qlora_rmsnorm_bwd")
    return dH, dX, dW


def _space(ws, dev):
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: a contiguous buffer on cuda:{dev} is expected")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _adapter(act, act_name, w, w_name, M, features, rank_first, dev):
    """Addresses and rank of an optional adapter term, both factors or neither:
    act [M, r] and w [features, r], or [r, features] with rank_first."""
    if act is None and w is None:
        return None, None, 0
    if act is None or w is None:
        raise ValueError(f"{act_name} and {w_name} go together")
    r = _matrix(act, act_name)[1]
    return (_need(act, act_name, _BF16, (M, r), dev),
            _need(w, w_name, _BF16, (r, features) if rank_first else (features, r), dev), r)


def i8_linear_fwd(W: I8Matrix, X: I8Matrix, sU=None, B=None, Y=None, status=None, stream=None):
    """Y [M, N] = (X codes . W codes^T) * X.scale * W.scale + sU B^T, bf16."""
    M, K = xs = _matrix(X.codes, "X.codes")
    N, _ = _matrix(W.codes, "W.codes")
    dev = _device(X.codes, "X.codes")
    xq, sx = _need_i8(X, "X", xs, dev)
    wq, sw = _need_i8(W, "W", (N, K), dev)
    u, b, r = _adapter(sU, "sU", B, "B", M, N, False, dev)
    if Y is None:
        Y = _empty(X.codes, (M, N), _BF16, stream)
    _check(_library().qlora_i8_linear_fwd(xq, sx, M, wq, sw, N, K, u, b, r, _need(Y, "Y", _BF16, (M, N), dev),
                                          _opt(status, "status", torch.int32, (1,), dev), _raw(stream, dev)),
           "qlora_i8_linear_fwd")
    return Y


def i8_linear_workspace(M: int, N: int, K: int) -> int:
    b = ctypes.c_size_t()
    _check(_library().qlora_i8_linear_workspace(M, N, K, ctypes.byref(b)), "qlora_i8_linear_workspace")
    return b.value


def i8_linear_dx(W: I8Matrix, dY, sT=None, A=None, dX=None, ws=None, status=None, stream=None):
    """dX [M, K] of the 8-bit linear: int8 rows of dY * W.scale through W's codes, + sT A."""
    M, N = ys = _matrix(dY, "dY")
    _, K = _matrix(W.codes, "W.codes")
    dev = _device(dY, "dY")
    dy = _need(dY, "dY", _BF16, ys, dev)
    wq, sw = _need_i8(W, "W", (N, K), dev)
    t, a, r = _adapter(sT, "sT", A, "A", M, K, True, dev)
    if dX is None:
        dX = _empty(dY, (M, K), _BF16, stream)
    if ws is None:
        ws = _empty(dY, (_bytes(i8_linear_workspace, dev, M, N, K),), torch.uint8, stream)
    _check(_library().qlora_i8_linear_dx(dy, M, wq, sw, N, K, t, a, r, _need(dX, "dX", _BF16, (M, K), dev),
                                         *_space(ws, dev), _opt(status, "status", torch.int32, (1,), dev),
                                         _raw(stream, dev)), "qlora_i8_linear_dx")
    return dX
