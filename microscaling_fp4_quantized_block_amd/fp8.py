"""Block-128 FP8 operators of libmxfp4 (E4M3 elements, one E8M0 scale per 128
contraction elements of a row): quantization, the matrix product, RMS norm with
the residual's addition and an FP8 output, the gated feed-forward projections,
and their gradients.  Layouts, formulas and errors are those of
``include/mxfp4.h``; this module marshals arguments.
"""
from __future__ import annotations

import ctypes
from operator import attrgetter
from typing import Optional

import torch

from . import _check, _nbytes, lib

# the current stream's handle of a device index (torch.cuda.current_stream() builds a Stream object, 2 us a call)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty = torch.empty_strided   # (a quarter less host time a call than torch.empty)

_byref = ctypes.byref

ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
C_TYPE = {torch.float32: 0, torch.bfloat16: 1}


class Fp8TensorStruct(ctypes.Structure):
    """Mirror of the C struct mxfp4_fp8_tensor."""
    _fields_ = [("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("scale_ld", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


def _declare():
    i32, i64, vp, sz, f32 = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    T, S = ctypes.POINTER(Fp8TensorStruct), ctypes.POINTER(sz)
    for name, args in {
            "tensor_bytes": [i64, i64, S, S],
            "quantize": [vp, i64, i64, i64, i32, i32, T, vp],
            "dequantize": [T, vp, i64, vp],
            "gemm_workspace_bytes": [T, T, S],
            "gemm": [T, T, vp, i64, i32, vp, sz, vp],
            "rmsnorm": [vp, i64, i64, i64, vp, i64, vp, f32, T, vp, i64, vp, i64, vp, vp],
            "rmsnorm_backward_workspace_bytes": [i64, i64, S],
            "rmsnorm_backward": [vp, i64, i64, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp, sz, vp],
            "gated_workspace_bytes": [T, T, i64, i32, S],
            "gated": [T, T, i64, i32, T, vp, i64, vp, vp, i64, vp, sz, vp],
            "gated_backward_workspace_bytes": [i64, i64, T, T, S],
            "gated_backward": [vp, i64, vp, vp, i64, i64, i64, i32, T, T, vp, i64, vp, i64, i32, T, vp, sz, vp]}.items():
        f = getattr(lib, "mxfp4_fp8_" + name)
        f.restype, f.argtypes = i32, args


_declare()


def _up(n: int, to: int) -> int:
    return (n + to - 1) // to * to


class Fp8Tensor:
    """A contraction-major FP8 matrix [rows, k].

    codes:  uint8 [rows, >= k rounded up to 128] (zeros from k on)
    scales: uint8 [k / 128 rounded up, >= rows]
    pair:   for two matrices in one (the gated block's weights, the columns
            each has, or the rows): their own length; each is padded to 128
    Rows may be strided by multiples of 16 bytes; both live on one GPU.  The
    library reads a descriptor made from the fields, so they cannot be set again.
    """
    __slots__ = ("_rows", "_k", "_codes", "_scales", "pair", "_device", "_struct")
    rows, k, codes, scales, device = (property(attrgetter(f)) for f in ("_rows", "_k", "_codes", "_scales", "_device"))

    def __init__(self, rows: int, k: int, codes: torch.Tensor, scales: torch.Tensor, pair: Optional[int] = None):
        kp, blocks = _up(k, 128), _up(k, 128) // 128
        for name, t in (("codes", codes), ("scales", scales)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or t.dim() != 2 or not t.is_cuda:
                raise ValueError(f"{name} must be a 2-D uint8 tensor on a GPU")
            if t.numel() and (t.stride(1) != 1 or t.stride(0) % 16 or t.data_ptr() % 16):
                raise ValueError(f"{name} must have unit stride along its last dimension, and 16-byte aligned rows")
        if rows < 0 or k < 0 or codes.shape[0] != rows or codes.shape[1] < kp:
            raise ValueError(f"codes have shape {tuple(codes.shape)}, expected [{rows}, {kp}]")
        if scales.shape[0] != blocks or scales.shape[1] < rows:
            raise ValueError(f"scales have shape {tuple(scales.shape)}, expected [{blocks}, >= {rows}]")
        if scales.device != codes.device:
            raise ValueError("codes and scales must live on one device")
        # the row stride of a single row is not a stride: any that is long enough will do
        ld = codes.stride(0) if rows > 1 else _up(codes.shape[1], 16)
        scale_ld = scales.stride(0) if blocks > 1 else _up(scales.shape[1], 16)
        if codes.numel() and scales.numel() and (ld < kp or scale_ld < rows):
            raise ValueError("rows of codes or scales overlap")
        self._set(rows, k, codes, scales, pair, ld, scale_ld)

    def _set(self, rows, k, codes, scales, pair, ld, scale_ld):
        self._rows, self._k, self._codes, self._scales, self.pair = rows, k, codes, scales, pair
        self._device = codes.device
        self._struct = Fp8TensorStruct(rows, k, ld, scale_ld, codes.data_ptr() or None, scales.data_ptr() or None)

    def elements(self) -> torch.Tensor:
        """The elements [rows, k] (a view)."""
        c = self.codes if self.codes.shape[1] == self.k else self.codes[:, :self.k]
        return c.view(torch.float8_e4m3fn)

    def exponents(self) -> torch.Tensor:
        """The scales [blocks, rows] (a view)."""
        s = self.scales if self.scales.shape[1] == self.rows else self.scales[:, :self.rows]
        return s.view(torch.float8_e8m0fnu)


def empty_fp8(rows: int, k: int, device, pair: Optional[int] = None) -> Fp8Tensor:
    """An Fp8Tensor for a quantizer to fill."""
    kp, pitch = _up(k, 128), _up(rows, 16)
    q = Fp8Tensor.__new__(Fp8Tensor)
    q._set(rows, k, _empty((rows, kp), (kp, 1), dtype=torch.uint8, device=device),
           _empty((kp // 128, pitch), (pitch, 1), dtype=torch.uint8, device=device), pair, kp, pitch)
    return q


def _matrix(t: torch.Tensor, name: str, shape=None, device=None, dtype=torch.bfloat16) -> int:
    """Checks a matrix argument; returns its row stride (at least its width)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D {dtype} tensor on a GPU")
    R, C = t.shape
    ld, one = t.stride()
    if shape is not None and (R, C) != shape:
        raise ValueError(f"{name} has shape {(R, C)}, expected {shape}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must live on {device}")
    if one != 1 and C > 1 and R:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    if ld < C:
        if R > 1:
            raise ValueError(f"{name}'s rows overlap")
        ld = C   # (the stride of a single row is not one)
    return ld or 1


def _vector(t: torch.Tensor, name: str, n: int, dtype, device) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != (n,) or t.device != device:
        raise ValueError(f"{name} must be a {dtype} vector of {n} elements on {device}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")


def _fp8(q, name: str, rows=None, k=None, device=None) -> Fp8Tensor:
    if not isinstance(q, Fp8Tensor):
        raise ValueError(f"{name} must be an Fp8Tensor")
    if (rows is not None and q.rows != rows) or (k is not None and q.k != k):
        raise ValueError(f"{name} is [{q.rows}, {q.k}], expected [{q.rows if rows is None else rows}, "
                         f"{q.k if k is None else k}]")
    if device is not None and q.device != device:
        raise ValueError(f"{name} must live on {device}")
    return q


def _room(need: int, workspace: Optional[torch.Tensor], device):
    """(tensor, its bytes) of a caller's workspace, or a new one of the size needed."""
    if workspace is None:
        return (_empty((need,), (1,), dtype=torch.uint8, device=device), need) if need else (None, 0)
    return workspace, _nbytes(workspace, device)


def _launch(device: torch.device, f, *args) -> None:
    """f(*args, stream) on the device's current stream.  Kernels go to the current device (the default stream's
    handle is the same on all of them), which may be another one than the operands'."""
    if device.index == _current_device():
        _check(f(*args, _raw_stream(device.index)))
    else:
        with torch.cuda.device(device):
            _check(f(*args, _raw_stream(device.index)))


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def mxfp4_fp8_tensor_bytes(rows: int, k: int):
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.mxfp4_fp8_tensor_bytes(rows, k, _byref(cb), _byref(sb)))
    return cb.value, sb.value


def mxfp4_fp8_quantize(x: torch.Tensor, axis: int = 1, block_rows: int = 1,
                       out: Optional[Fp8Tensor] = None) -> Fp8Tensor:
    """FP8 of bf16 x [R, C]: axis=1 along C (result [R, C]), axis=0 along R
    (result [C, R]).  block_rows=128 gives each 128 x 128 block of x one scale."""
    ldx = _matrix(x, "x")
    R, C = x.shape
    rows, k = (R, C) if axis == 1 else (C, R)
    if out is None:
        out = empty_fp8(rows, k, x.device)
    else:
        _fp8(out, "out", rows, k, x.device)
    _launch(x.device, lib.mxfp4_fp8_quantize, x.data_ptr(), R, C, ldx, int(axis), int(block_rows), _byref(out._struct))
    return out


def mxfp4_fp8_quantize_pair(gate: torch.Tensor, up: torch.Tensor, axis: int = 1) -> Fp8Tensor:
    """The gated block's two bf16 weights [n, k] in one operand, with a scale
    per 128 x 128 block: axis=1 one under the other ([2 np, k], for
    mxfp4_fp8_gated), axis=0 transposed and side by side ([k, 2 np], for its
    gradient), np = n rounded up to 128."""
    _matrix(gate, "gate")
    _matrix(up, "up", gate.shape, gate.device)
    n, k = gate.shape
    np_, kp = _up(n, 128), _up(k, 128)
    if axis == 1:
        q = empty_fp8(2 * np_, k, gate.device, pair=n)
        if np_ != n:
            q.codes[n:np_] = 0
            q.codes[np_ + n:] = 0
            q.scales[:, n:np_] = 0
            q.scales[:, np_ + n:] = 0
        parts = [Fp8Tensor(n, k, q.codes[i * np_:i * np_ + n], q.scales[:, i * np_:i * np_ + n]) for i in (0, 1)]
    elif axis == 0:
        q = empty_fp8(k, 2 * np_, gate.device, pair=n)
        parts = [Fp8Tensor(k, n, q.codes[:, i * np_:(i + 1) * np_],
                           q.scales[i * (np_ // 128):(i + 1) * (np_ // 128)]) for i in (0, 1)]
    else:
        raise ValueError("axis must be 0 or 1")
    if n and k:
        for part, w in zip(parts, (gate, up)):
            mxfp4_fp8_quantize(w, axis=axis, block_rows=128, out=part)
    return q


def mxfp4_fp8_dequantize(q: Fp8Tensor) -> torch.Tensor:
    """The binary32 values of q [rows, k]."""
    _fp8(q, "q")
    y = torch.empty((q.rows, q.k), dtype=torch.float32, device=q.device)
    _launch(q.device, lib.mxfp4_fp8_dequantize, _byref(q._struct), _p(y), max(q.k, 1))
    return y


def mxfp4_fp8_gemm_workspace_bytes(A: Fp8Tensor, B: Fp8Tensor) -> int:
    b = ctypes.c_size_t()
    _check(lib.mxfp4_fp8_gemm_workspace_bytes(_byref(A._struct), _byref(B._struct), _byref(b)))
    return b.value


def mxfp4_fp8_gemm(A: Fp8Tensor, B: Fp8Tensor, dtype: torch.dtype = torch.bfloat16,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C = A B^T [A.rows, B.rows] as float32 or bfloat16, accumulated in binary32
    registers by a matrix instruction that cuts products to 13 binary places
    below the largest of eight neighbours (include/mxfp4.h has the bound): float32
    results are good to about 1.5e-5 of the root of the sum of their squared
    products, where a binary32 product would be good to 1e-7."""
    _fp8(A, "A")
    _fp8(B, "B", device=A.device)
    if out is not None:
        dtype = out.dtype
    if dtype not in C_TYPE:
        raise ValueError("the result is float32 or bfloat16")
    if out is None:
        out = _empty((A.rows, B.rows), (B.rows, 1), dtype=dtype, device=A.device)
        ldc = B.rows
    else:
        ldc = _matrix(out, "out", (A.rows, B.rows), A.device, dtype)
    ws, ws_bytes = _room(mxfp4_fp8_gemm_workspace_bytes(A, B), workspace, A.device)
    _launch(A.device, lib.mxfp4_fp8_gemm, _byref(A._struct), _byref(B._struct), out.data_ptr(), ldc, C_TYPE[dtype],
            _p(ws), ws_bytes)
    return out


def mxfp4_fp8_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                      residual: Optional[torch.Tensor] = None, train: bool = False, out: Optional[Fp8Tensor] = None,
                      sum_out: Optional[torch.Tensor] = None):
    """(q, r): r = bf16(x + residual) (x itself without a residual) and q the FP8
    of its RMS norm times weight; train=True: (q, r, y, rstd) with the norm in
    bf16 and the rows' 1 / rms too.  sum_out (x or residual themselves, if
    they may be overwritten) receives r."""
    ldx = _matrix(x, "x")
    T, H = shape = tuple(x.shape)
    dev = x.device
    _vector(weight, "weight", H, torch.bfloat16, dev)
    ldr = lds = 0
    if residual is not None:
        ldr = _matrix(residual, "residual", shape, dev)
        if sum_out is None:
            sum_out, lds = _empty(shape, (H, 1), dtype=torch.bfloat16, device=dev), H
        else:
            lds = _matrix(sum_out, "sum_out", shape, dev)
    elif sum_out is not None:
        raise ValueError("sum_out goes with a residual")
    if out is None:
        out = empty_fp8(T, H, dev)
    else:
        _fp8(out, "out", T, H, dev)
    y = _empty(shape, (H, 1), dtype=torch.bfloat16, device=dev) if train else None
    rstd = _empty((T,), (1,), dtype=torch.float32, device=dev) if train else None
    _launch(dev, lib.mxfp4_fp8_rmsnorm, x.data_ptr(), T, H, ldx, _p(residual), ldr, weight.data_ptr(), eps,
            _byref(out._struct), _p(sum_out), lds, _p(y), H, _p(rstd))
    r = x if residual is None else sum_out
    return (out, r, y, rstd) if train else (out, r)


def mxfp4_fp8_rmsnorm_backward_workspace_bytes(T: int, H: int) -> int:
    b = ctypes.c_size_t()
    _check(lib.mxfp4_fp8_rmsnorm_backward_workspace_bytes(T, H, _byref(b)))
    return b.value


def mxfp4_fp8_rmsnorm_backward(dy: torch.Tensor, r: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                               dres: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None):
    """(dx, dw) of mxfp4_fp8_rmsnorm for bf16 dy, with the r, weight and rstd of
    the forward pass: dx (bf16, the gradient of x and of the residual) has dres,
    the gradient that reaches r past the norm, added; dw is float32."""
    ldd = _matrix(dy, "dy")
    T, H = shape = tuple(dy.shape)
    dev = dy.device
    ldr = _matrix(r, "r", shape, dev)
    _vector(weight, "weight", H, torch.bfloat16, dev)
    _vector(rstd, "rstd", T, torch.float32, dev)
    lde = 0 if dres is None else _matrix(dres, "dres", shape, dev)
    if out is None:
        out, ldx = _empty(shape, (H, 1), dtype=torch.bfloat16, device=dev), H
    else:
        ldx = _matrix(out, "out", shape, dev)
    dw = _empty((H,), (1,), dtype=torch.float32, device=dev)
    ws, ws_bytes = _room(mxfp4_fp8_rmsnorm_backward_workspace_bytes(T, H), workspace, dev)
    _launch(dev, lib.mxfp4_fp8_rmsnorm_backward, dy.data_ptr(), T, H, ldd, r.data_ptr(), ldr, weight.data_ptr(),
            rstd.data_ptr(), _p(dres), lde, out.data_ptr(), ldx, dw.data_ptr(), _p(ws), ws_bytes)
    return out, dw


def _pair(w: Fp8Tensor, name: str) -> int:
    if w.pair is None:
        raise ValueError(f"{name} must hold a pair of weights (mxfp4_fp8_quantize_pair)")
    return w.pair


def _act(act: str) -> int:
    if act not in ACT:
        raise ValueError(f"act must be one of {sorted(ACT)}")
    return ACT[act]


def mxfp4_fp8_gated_workspace_bytes(x: Fp8Tensor, w: Fp8Tensor, fp8_out: bool = True) -> int:
    b = ctypes.c_size_t()
    _check(lib.mxfp4_fp8_gated_workspace_bytes(_byref(x._struct), _byref(w._struct), _pair(w, "w"), int(fp8_out),
                                               _byref(b)))
    return b.value


def mxfp4_fp8_gated(x: Fp8Tensor, w: Fp8Tensor, act: str = "silu", train: bool = False, dtype=None, out=None,
                    workspace: Optional[torch.Tensor] = None):
    """h = act(x Wg^T) * (x Wu^T) [x.rows, n], w the pair of weights: as an
    Fp8Tensor (quantized from binary32; the projections are as exact as
    mxfp4_fp8_gemm's sums), or in bf16 with dtype=torch.bfloat16.  train=True: (h, g, u), the two projections in bf16 for
    the backward pass."""
    _fp8(x, "x")
    _fp8(w, "w", device=x.device)
    n, T, dev = _pair(w, "w"), x.rows, x.device
    if dtype not in (None, torch.bfloat16):
        raise ValueError("the result is FP8 (dtype=None) or bfloat16")
    fp8 = dtype is None
    ldh = n
    if out is None:
        out = empty_fp8(T, n, dev) if fp8 else torch.empty((T, n), dtype=torch.bfloat16, device=dev)
    elif fp8:
        _fp8(out, "out", T, n, dev)
    else:
        ldh = _matrix(out, "out", (T, n), dev)
    g = torch.empty((T, n), dtype=torch.bfloat16, device=dev) if train else None
    u = torch.empty((T, n), dtype=torch.bfloat16, device=dev) if train else None
    ws, ws_bytes = _room(mxfp4_fp8_gated_workspace_bytes(x, w, fp8), workspace, dev)
    _launch(dev, lib.mxfp4_fp8_gated, _byref(x._struct), _byref(w._struct), n, _act(act),
            _byref(out._struct) if fp8 else None, None if fp8 else out.data_ptr(), ldh, _p(g), _p(u), n, _p(ws),
            ws_bytes)
    return (out, g, u) if train else out


def mxfp4_fp8_gated_backward_workspace_bytes(T: int, wt: Fp8Tensor, xt: Fp8Tensor) -> int:
    b = ctypes.c_size_t()
    _check(lib.mxfp4_fp8_gated_backward_workspace_bytes(T, _pair(wt, "wt"), _byref(wt._struct), _byref(xt._struct),
                                                        _byref(b)))
    return b.value


def mxfp4_fp8_gated_backward(dh: torch.Tensor, g: torch.Tensor, u: torch.Tensor, wt: Fp8Tensor, xt: Fp8Tensor,
                             act: str = "silu", dtype: torch.dtype = torch.float32, want_ht: bool = False,
                             workspace: Optional[torch.Tensor] = None):
    """(dx, dwg, dwu) of mxfp4_fp8_gated for bf16 dh [T, n]: g and u from the
    forward pass, wt the weights transposed (mxfp4_fp8_quantize_pair, axis=0), xt
    the input quantized along the tokens (mxfp4_fp8_quantize, axis=0).  dx is
    bf16, dwg and dwu [n, H] are of dtype (float32 or bfloat16; their sums are as
    exact as mxfp4_fp8_gemm's).  want_ht=True:
    the FP8 transpose [n, T] of h too, which the down projection's weight
    gradient multiplies."""
    ldd = _matrix(dh, "dh")
    T, n = shape = tuple(dh.shape)
    dev = dh.device
    ldgu = _matrix(g, "g", shape, dev)
    if _matrix(u, "u", shape, dev) != ldgu and T > 1:   # (the stride of a single row is not one)
        raise ValueError("g and u must have the same row stride")
    _fp8(wt, "wt", device=dev)
    _fp8(xt, "xt", wt.rows, T, dev)
    if _pair(wt, "wt") != n:
        raise ValueError(f"wt holds weights of {wt.pair} rows, expected {n}")
    if dtype not in C_TYPE:
        raise ValueError("the weights' gradients are float32 or bfloat16")
    H, np_ = wt.rows, _up(n, 128)
    dx = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    dw = torch.empty((2 * np_, H), dtype=dtype, device=dev)
    ht = empty_fp8(n, T, dev) if want_ht else None
    ws, ws_bytes = _room(mxfp4_fp8_gated_backward_workspace_bytes(T, wt, xt), workspace, dev)
    _launch(dev, lib.mxfp4_fp8_gated_backward, dh.data_ptr(), ldd, g.data_ptr(), u.data_ptr(), ldgu, T, n, _act(act),
            _byref(wt._struct), _byref(xt._struct), _p(dx), max(H, 1), _p(dw), max(H, 1), C_TYPE[dtype],
            _byref(ht._struct) if want_ht else None, _p(ws), ws_bytes)
    got = (dx, dw[:n], dw[np_:np_ + n])
    return got + (ht,) if want_ht else got
