"""Binding of the e4m3 block-128 product (include/f8.h): argument marshalling only."""
from __future__ import annotations

import ctypes

import torch

from ._args import device_of, dtype_of, native, pointer
from ._lib import _check, _empty, _stream, lib

F8 = torch.float8_e4m3fn
F8_EXPORTS = ("f8_quantize_rows", "f8_quantize_cols", "f8_quantize_weights", "f8_transpose_weights", "f8_gemm",
              "f8_linear_work_bytes", "f8_linear", "f8_linear_backward_work_bytes", "f8_linear_backward")
_funcs = None


def _f8():
    global _funcs
    if _funcs is None:
        L = lib()
        P, I, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
        L.f8_quantize_rows.argtypes = [I, I, I, P, LL, P, P, P]
        L.f8_quantize_cols.argtypes = [I, I, I, P, LL, P, P, P]
        L.f8_quantize_weights.argtypes = [I, I, I, P, P, P, P]
        L.f8_transpose_weights.argtypes = [I, I, P, P, P, P, P]
        L.f8_gemm.argtypes = [I, I, I, I, P, P, P, P, P, P]
        for name in F8_EXPORTS[:5]:
            getattr(L, name).restype = I
        _funcs = L
    return _funcs


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _rows(x, what: str):
    """A matrix with contiguous rows, which may be a slice of a wider one: (GPU, dtype, M, K, address, row stride)."""
    dev = device_of(x, what)
    dt = dtype_of(x, what)
    if x.dim() != 2 or x.shape[0] < 1 or x.shape[1] < 1:
        raise ValueError(f"{what}: expected a matrix [rows][columns], got {tuple(x.shape)}")
    M, K = x.shape
    stride = x.stride(0) if M > 1 else K
    if (K > 1 and x.stride(1) != 1) or stride < K:
        raise ValueError(f"{what}: the values of a row must be contiguous and rows must not overlap")
    return dev, dt, M, K, x.data_ptr(), stride


def f8_quantize_act(x: torch.Tensor, stream=None):
    """x [M][K] float32 or bfloat16 (rows may be strided) -> (codes e4m3 [M][Kp], scales float32 [Kp/128][M]),
    Kp = K rounded up to 128: one scale for each 1 x 128 block."""
    dev, dt, M, K, px, stride = _rows(x, "x")
    kb = _blocks(K)
    xq = _empty(stream, (M, kb * 128), F8, x.device)
    xs = _empty(stream, (kb, M), torch.float32, x.device)
    _check(_f8().f8_quantize_rows(M, K, dt, px, stride, xq.data_ptr(), xs.data_ptr(), _stream(stream)),
           "f8_quantize_rows")
    return xq, xs


def f8_quantize_act_t(x: torch.Tensor, stream=None):
    """x [M][K] -> (codes e4m3 [K][Mp], scales float32 [Mp/128][K]): transposed, one scale for each channel's block
    of 128 tokens (the weight gradient's operands)."""
    dev, dt, M, K, px, stride = _rows(x, "x")
    mb = _blocks(M)
    xt = _empty(stream, (K, mb * 128), F8, x.device)
    xts = _empty(stream, (mb, K), torch.float32, x.device)
    _check(_f8().f8_quantize_cols(M, K, dt, px, stride, xt.data_ptr(), xts.data_ptr(), _stream(stream)),
           "f8_quantize_cols")
    return xt, xts


def f8_quantize_weights(w: torch.Tensor, stream=None):
    """w [N][K] float32 or bfloat16 -> (codes e4m3 [N][Kp], scales float32 [Np/128][Kp/128]), 128 x 128 blocks."""
    dev = device_of(w, "w")
    dt = dtype_of(w, "w")
    N, K = w.shape
    pw = pointer(w, dev, (N, K), w.dtype, "w")
    wq = _empty(stream, (N, _blocks(K) * 128), F8, w.device)
    ws = _empty(stream, (_blocks(N), _blocks(K)), torch.float32, w.device)
    _check(_f8().f8_quantize_weights(N, K, dt, pw, wq.data_ptr(), ws.data_ptr(), _stream(stream)),
           "f8_quantize_weights")
    return wq, ws


def f8_transpose_weights(wq: torch.Tensor, ws: torch.Tensor, K: int, stream=None):
    """Codes [N][Kp] and scales of f8_quantize_weights -> (codes [K][Np], scales [Kp/128][Np/128]): what
    f8_linear_backward reads."""
    dev = device_of(wq, "wq")
    N = wq.shape[0]
    kb, nb = _blocks(K), _blocks(N)
    pq = pointer(wq, dev, (N, kb * 128), F8, "wq")
    ps = pointer(ws, dev, (nb, kb), torch.float32, "ws")
    wqt = _empty(stream, (K, nb * 128), F8, wq.device)
    wst = _empty(stream, (kb, nb), torch.float32, wq.device)
    _check(_f8().f8_transpose_weights(N, K, pq, ps, wqt.data_ptr(), wst.data_ptr(), _stream(stream)),
           "f8_transpose_weights")
    return wqt, wst


def f8_gemm(xq, xs, wq, ws, out=None, dtype=torch.float32, stream=None):
    """Product of codes: xq [M][Kp], xs [Kp/128][M], wq [N][Kp], ws [Np/128][Kp/128] -> y [M][N] (dtype)."""
    dev = device_of(xq, "xq")
    M, Kp = xq.shape
    N, kb = wq.shape[0], _blocks(Kp)
    if out is None:
        out = _empty(stream, (M, N), dtype, xq.device)
    _check(_f8().f8_gemm(M, Kp, N, dtype_of(out, "out"), pointer(xq, dev, (M, Kp), F8, "xq"),
                         pointer(xs, dev, (kb, M), torch.float32, "xs"), pointer(wq, dev, (N, Kp), F8, "wq"),
                         pointer(ws, dev, (_blocks(N), kb), torch.float32, "ws"),
                         pointer(out, dev, (M, N), out.dtype, "out"), _stream(stream)), "f8_gemm")
    return out


def f8_linear(x, wq, ws, out=None, work=None, stream=None):
    """x [M][K] float32 or bfloat16 (rows may be strided), quantized per 1 x 128 block, times the weights of
    f8_quantize_weights -> y [M][N] in x's dtype. One launch for a few rows, two otherwise."""
    return native().f8_linear(x, wq, ws, out, work, stream)


def f8_linear_backward(dy, x, wqt, wst, dx=None, dw=None, need_dx=True, need_dw=True, work=None, stream=None):
    """Gradients of f8_linear: dy [M][N], x [M][K] (same dtype), weights of f8_transpose_weights -> (dx [M][K] in x's
    dtype, dw [N][K] in x's dtype). dx takes dy quantized per 1 x 128 block along N, dw takes dy and x quantized per
    block of 128 tokens; a dw that is given decides on its dtype (float32 or bfloat16). With need_dx or need_dw False
    that gradient is None (and wqt, wst or x may be None)."""
    return native().f8_linear_backward(dy, x, wqt, wst, dx, dw, need_dx, need_dw, work, stream)
