"""The linear layer in 8-bit floating point: torch tensors -> include/sgemm_fp8.h.

    q, s        = quantize_fp8(x, block=(1, 128))             # or (128, 1), (128, 128)
    qr, sr, qc, sc = quantize_fp8_both(x)                     # (1, 128) and (128, 1) in one pass
    y           = gemm_fp8(qx, sx, qw, sw, transB=True)       # x @ w.T
    o           = rms_norm_fp8(x, w, residual=r)              # o.q, o.scale, o.h
    dx, dw      = rms_norm_backward(dy, h, w, rstd, dh=dh)

An 8-bit matrix is a torch.float8_e4m3fn or torch.float8_e5m2 tensor with a
float32 tensor of one scale per block; an element stands for q * s.  Blocks
span 128 elements along the inner dimension of the product that reads them and
1 or 128 along the outer one.  The 8-bit tensors made here have rows that start
on 16-byte boundaries (a row stride rounded up to 16), which is what the fast
kernels read; any other layout gives the same results.

All matrices are 2-D CUDA tensors with unit column stride and any row stride.
Every function runs on ``stream`` (a torch.cuda.Stream; what it allocates then
belongs to that stream) or on torch's current stream, and returns once its work
is queued.  Nothing here computes; there is no CPU fallback.  The usual calls
(plain tensors of the current device, its current stream) are marshalled by the
extension module _fp8_torch where it has been built; it hands back what it does
not take, and the code here checks everything and says what is wrong.  Its outputs come straight from the caching
allocator: dispatch modes and torch.utils.deterministic's filling do not see them.
"""
import collections
import ctypes

import torch

from ._binding import SgemmError, _current_raw_stream, _op, load_library

BLOCK = 128
_BLOCKS = ((1, BLOCK), (BLOCK, 1), (BLOCK, BLOCK))
TYPE_F32, TYPE_BF16, TYPE_F16, TYPE_E4M3, TYPE_E5M2 = 0, 1, 2, 8, 9
_FLOAT = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16, torch.float16: TYPE_F16}
_FP8 = {torch.float8_e4m3fn: TYPE_E4M3, torch.float8_e5m2: TYPE_E5M2}
_F32 = {torch.float32: TYPE_F32}
_SAME = {code: {dtype: code} for dtype, code in _FLOAT.items()}
_WEIGHT = {code: _F32 | same for code, same in _SAME.items()}   # a norm's weights: float32 or its input's type

RmsNormFp8 = collections.namedtuple("RmsNormFp8", "q scale h y rstd")
RmsNormFp8.__doc__ = """What rms_norm_fp8 returns: the quantised norm and its scales, h = x + residual
(None without a residual), and, with training=True, the norm y in x's type and rstd."""

_lib = None
_usual = None   # the extension module, once the library is loaded
_I64, _VP, _INT, _F = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        lib.sgemm_fp8.argtypes = [_INT, _INT, _I64, _I64, _I64, _F, _VP, _INT, _I64, _VP, _I64, _INT,
                                  _VP, _INT, _I64, _VP, _I64, _INT, _F, _VP, _INT, _I64, _VP]
        lib.sgemm_fp8_quantize.argtypes = [_I64, _I64, _VP, _INT, _I64, _VP, _INT, _I64, _VP, _I64, _INT, _INT, _VP]
        lib.sgemm_fp8_quantize_both.argtypes = [_I64, _I64, _VP, _INT, _I64, _INT, _VP, _I64, _VP, _I64, _VP, _I64,
                                                _VP, _I64, _VP]
        lib.sgemm_rms_norm_fp8.argtypes = [_I64, _I64, _F, _VP, _I64, _VP, _I64, _INT, _VP, _INT, _VP, _I64, _VP,
                                           _I64, _VP, _INT, _I64, _VP, _I64, _VP, _VP]
        lib.sgemm_rms_norm_backward.argtypes = [_I64, _I64, _VP, _I64, _VP, _I64, _INT, _VP, _INT, _VP, _VP, _I64,
                                                _VP, _I64, _VP, _VP, ctypes.c_size_t, _VP]
        for f in (lib.sgemm_fp8, lib.sgemm_fp8_quantize, lib.sgemm_fp8_quantize_both, lib.sgemm_rms_norm_fp8,
                  lib.sgemm_rms_norm_backward):
            f.restype = _INT
        lib.sgemm_fp8_select_form.argtypes = [_INT, _INT, _I64, _I64, _I64, _VP, _I64, _VP, _I64, _INT, _F, _VP, _INT,
                                              _I64, ctypes.POINTER(_INT)]
        lib.sgemm_fp8_select_form.restype = _INT
        lib.sgemm_rms_norm_backward_workspace.argtypes = [_I64, _I64]
        lib.sgemm_rms_norm_backward_workspace.restype = ctypes.c_size_t
        global _usual
        try:
            from . import _fp8_torch
        except ImportError:   # not built (or for another torch)
            _usual = None
        else:
            _fp8_torch.bind(*(ctypes.cast(f, _VP).value for f in (
                lib.sgemm_fp8, lib.sgemm_fp8_quantize, lib.sgemm_fp8_quantize_both, lib.sgemm_rms_norm_fp8,
                lib.sgemm_rms_norm_backward, lib.sgemm_rms_norm_backward_workspace, lib.sgemm_sandwich_norm_fp8,
                lib.sgemm_sandwich_norm_backward, lib.sgemm_sandwich_norm_backward_workspace, lib.sgemm_swiglu_fp8,
                lib.sgemm_swiglu_backward_fp8, lib.sgemm_fp8_requantize)))
            _usual = _fp8_torch
        _lib = lib
    return _lib


def _raise(where, status):
    if status != 0:
        raise SgemmError(status, where)


# ------------------------------------------------------------------ the C ABI
# (same names and arguments, pointers as ints, raising SgemmError)
def sgemm_fp8(transA, transB, M, N, K, alpha, A, typeA, lda, SA, ldsa, blockA, B, typeB, ldb, SB, ldsb, blockB, beta,
              C, typeC, ldc, stream=None):
    """C = alpha*op(A)*op(B) + beta*C with block-scaled 8-bit A and B."""
    _raise("sgemm_fp8", _library().sgemm_fp8(_op(transA), _op(transB), M, N, K, alpha, A, typeA, lda, SA, ldsa, blockA,
                                             B, typeB, ldb, SB, ldsb, blockB, beta, C, typeC, ldc, stream))


FP8_FORMS = ("few_16", "few_32", "few_64", "half", "tile", "loaded", "pair", "pair_staged", "pair_bulk")


def sgemm_fp8_select_form(transA, transB, M, N, K, A, lda, B, ldb, blockB, beta, C, typeC, ldc):
    """(name of the form, CTAs sharing a tile) that sgemm_fp8 would run, or None if it would multiply nothing."""
    split = _INT(0)
    form = _library().sgemm_fp8_select_form(_op(transA), _op(transB), M, N, K, A, lda, B, ldb, blockB, beta, C, typeC,
                                            ldc, ctypes.byref(split))
    return None if form < 0 else (FP8_FORMS[form], split.value)


def sgemm_fp8_quantize(rows, cols, X, typeX, ldx, Q, typeQ, ldq, S, lds, block_rows, block_cols, stream=None):
    """Q, S = X quantised in blocks of block_rows x block_cols."""
    _raise("sgemm_fp8_quantize", _library().sgemm_fp8_quantize(rows, cols, X, typeX, ldx, Q, typeQ, ldq, S, lds,
                                                               block_rows, block_cols, stream))


def sgemm_fp8_quantize_both(rows, cols, X, typeX, ldx, typeQ, QR, ldqr, SR, ldsr, QC, ldqc, SC, ldsc, stream=None):
    """X quantised in 1 x 128 and in 128 x 1 blocks."""
    _raise("sgemm_fp8_quantize_both",
           _library().sgemm_fp8_quantize_both(rows, cols, X, typeX, ldx, typeQ, QR, ldqr, SR, ldsr, QC, ldqc, SC, ldsc,
                                              stream))


def sgemm_rms_norm_fp8(rows, cols, eps, X, ldx, R, ldr, typeX, W, typeW, H, ldh, Y, ldy, Q, typeQ, ldq, S, lds, T,
                       stream=None):
    """RMS norm of X + R with an 8-bit output (R, H, Y, T may be None)."""
    _raise("sgemm_rms_norm_fp8", _library().sgemm_rms_norm_fp8(rows, cols, eps, X, ldx, R, ldr, typeX, W, typeW, H, ldh,
                                                               Y, ldy, Q, typeQ, ldq, S, lds, T, stream))


def sgemm_rms_norm_backward(rows, cols, DY, lddy, H, ldh, typeX, W, typeW, T, DH, lddh, DX, lddx, DW, workspace,
                            workspace_bytes, stream=None):
    """Gradient of the norm (DH, DW and, without DW, workspace may be None)."""
    _raise("sgemm_rms_norm_backward",
           _library().sgemm_rms_norm_backward(rows, cols, DY, lddy, H, ldh, typeX, W, typeW, T, DH, lddh, DX, lddx, DW,
                                              workspace, workspace_bytes, stream))


def sgemm_rms_norm_backward_workspace(rows, cols) -> int:
    """Bytes of workspace that sgemm_rms_norm_backward needs."""
    return _library().sgemm_rms_norm_backward_workspace(rows, cols)


# ------------------------------------------------------------------ torch
def _mat(t, name, types):
    """(pointer, rows, cols, ld, type, device) of a 2-D CUDA tensor with unit column stride."""
    try:
        rows, cols = t.shape
        ld, st1 = t.stride()
        code = types[t.dtype]
    except (AttributeError, KeyError, ValueError):
        raise TypeError(f"{name} must be a 2-D tensor of {' or '.join(str(d) for d in types)}") from None
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if st1 != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    if ld < cols or ld < 1:
        if rows > 1:
            raise ValueError(f"{name} has overlapping rows")
        ld = cols if cols > 0 else 1
    return t.data_ptr(), rows, cols, ld, code, dev


def _vec(t, name, n, types):
    """(pointer, type, device) of a contiguous 1-D CUDA tensor of n elements."""
    try:
        (size,) = t.shape
        code = types[t.dtype]
    except (AttributeError, KeyError, ValueError):
        raise TypeError(f"{name} must be a 1-D tensor of {' or '.join(str(d) for d in types)}") from None
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if size != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must hold {n} contiguous elements")
    return t.data_ptr(), code, dev


def _one_device(*devs):
    for d in devs:
        if d != devs[0]:
            raise ValueError("tensors are on different devices")


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(stream, dev):
    """The context in which a call allocates and runs, or None if that is the current one."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"stream is of cuda:{stream.device.index}, the tensors are on cuda:{dev}")
        return torch.cuda.stream(stream)
    return None if dev == _current_device() else torch.cuda.device(dev)


def _cdiv(a, b):
    return -(-a // b)


def _empty_fp8(rows, cols, dtype, dev):
    """(tensor, ld): rows on 16-byte boundaries."""
    ld = max((cols + 15) // 16 * 16, 1)
    return torch.empty_strided((rows, cols), (ld, 1), dtype=dtype, device=dev), ld


def _fp8_type(dtype):
    if dtype not in _FP8:
        raise TypeError(f"dtype must be {' or '.join(str(d) for d in _FP8)}")
    return _FP8[dtype]


def quantize_fp8(x, block=(1, BLOCK), dtype=torch.float8_e4m3fn, stream=None):
    """(q, scale) of a float32, bfloat16 or float16 matrix in blocks of (1, 128), (128, 1) or (128, 128):
    scale = max(max|x| / F, 2^-126) per block, q = x / scale rounded to `dtype`."""
    if _usual is not None and stream is None and dtype in _FP8 and block in _BLOCKS:
        r = _usual.quantize(x, *block, _FP8[dtype])
        if r is not None:
            return r
    px, rows, cols, ldx, tx, dev = _mat(x, "x", _FLOAT)
    tq = _fp8_type(dtype)
    br, bc = block
    if (br, bc) not in _BLOCKS:
        raise ValueError("block must be (1, 128), (128, 1) or (128, 128)")
    ctx = _on(stream, dev)
    if ctx is not None:
        with ctx:
            return quantize_fp8(x, block, dtype)
    q, ldq = _empty_fp8(rows, cols, dtype, x.device)
    sr, sc = _cdiv(rows, br), _cdiv(cols, bc)
    s = torch.empty((sr, sc), dtype=torch.float32, device=x.device)
    st = (_lib or _library()).sgemm_fp8_quantize(rows, cols, px, tx, ldx, q.data_ptr(), tq, ldq, s.data_ptr(), sc or 1,
                                                 br, bc, _current_raw_stream(dev))
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_quantize")
    return q, s


def quantize_fp8_both(x, dtype=torch.float8_e4m3fn, stream=None):
    """(q_rows, scale_rows, q_cols, scale_cols): x in (1, 128) and in (128, 1) blocks, in one pass over it."""
    if _usual is not None and stream is None and dtype in _FP8:
        r = _usual.quantize_both(x, _FP8[dtype])
        if r is not None:
            return r
    px, rows, cols, ldx, tx, dev = _mat(x, "x", _FLOAT)
    tq = _fp8_type(dtype)
    ctx = _on(stream, dev)
    if ctx is not None:
        with ctx:
            return quantize_fp8_both(x, dtype)
    qr, ldqr = _empty_fp8(rows, cols, dtype, x.device)
    qc, ldqc = _empty_fp8(rows, cols, dtype, x.device)
    kr, kc = _cdiv(cols, BLOCK), _cdiv(rows, BLOCK)
    sr = torch.empty((rows, kr), dtype=torch.float32, device=x.device)
    sc = torch.empty((kc, cols), dtype=torch.float32, device=x.device)
    st = (_lib or _library()).sgemm_fp8_quantize_both(rows, cols, px, tx, ldx, tq, qr.data_ptr(), ldqr, sr.data_ptr(),
                                                      kr or 1, qc.data_ptr(), ldqc, sc.data_ptr(), cols or 1,
                                                      _current_raw_stream(dev))
    if st != 0:
        raise SgemmError(st, "sgemm_fp8_quantize_both")
    return qr, sr, qc, sc


def _scales(s, name, outer, kb, inner_rows):
    """(pointer, ld, block, device) of an operand's scales; the block along the outer dimension follows from the
    shape."""
    ps, r, c, ld, _, dev = _mat(s, name, _F32)
    o, k = (c, r) if inner_rows else (r, c)
    if k == kb:
        if o == outer:
            return ps, ld, 1, dev
        if o == (outer + 127) // 128:
            return ps, ld, BLOCK, dev
    raise ValueError(f"{name} is {r} x {c}: one scale is wanted for each block of 128 along the inner dimension "
                     f"({kb}) times each 1 or 128 along the outer one ({outer} or {_cdiv(outer, BLOCK)})")


def gemm_fp8(A, A_scale, B, B_scale, C=None, alpha=1.0, beta=0.0, transA=False, transB=False, out_dtype=None,
             stream=None):
    """C = alpha * op(A) @ op(B) + beta * C with 8-bit A and B (float8_e4m3fn or float8_e5m2, each its own).

    A, B are in stored layout (A is K x M when transA, B is N x K when transB), and so are their scales: one per
    128 elements along K and per 1 or 128 along M or N.  C is float32, bfloat16 or float16; if it is None a new
    M x N tensor of ``out_dtype`` (default bfloat16) is returned (beta must then be 0).
    """
    if _usual is not None and stream is None:
        tc = TYPE_BF16 if out_dtype is None else _FLOAT.get(out_dtype)
        if tc is not None and (C is None or out_dtype is None or getattr(C, "dtype", None) == out_dtype):
            r = _usual.product(A, A_scale, B, B_scale, C, alpha, beta, transA, transB, tc)
            if r is not None:
                return r
    pa, ra, ca, lda, fa, dev = _mat(A, "A", _FP8)
    pb, rb, cb, ldb, fb, devb = _mat(B, "B", _FP8)
    M, K = (ca, ra) if transA else (ra, ca)
    Kb, N = (cb, rb) if transB else (rb, cb)
    if K != Kb:
        raise ValueError(f"inner dimensions differ: {K} vs {Kb}")
    kb = (K + 127) // 128
    psa, ldsa, ba, devsa = _scales(A_scale, "A_scale", M, kb, transA)
    psb, ldsb, bb, devsb = _scales(B_scale, "B_scale", N, kb, not transB)
    if not dev == devb == devsa == devsb:
        raise ValueError("tensors are on different devices")
    ctx = _on(stream, dev)
    if ctx is not None:
        with ctx:
            return gemm_fp8(A, A_scale, B, B_scale, C, alpha, beta, transA, transB, out_dtype)
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        if out_dtype is None:
            out_dtype = torch.bfloat16
        elif out_dtype not in _FLOAT:
            raise TypeError(f"out_dtype must be {' or '.join(str(d) for d in _FLOAT)}")
        C = torch.empty((M, N), dtype=out_dtype, device=A.device)
        pc, ldc, tc = C.data_ptr(), N or 1, _FLOAT[out_dtype]
    else:
        if out_dtype is not None and out_dtype != C.dtype:
            raise TypeError(f"C is {C.dtype}, out_dtype {out_dtype}")
        pc, rc, cc, ldc, tc, devc = _mat(C, "C", _FLOAT)
        if rc != M or cc != N:
            raise ValueError(f"C must be {M} x {N}")
        _one_device(dev, devc)
    st = (_lib or _library()).sgemm_fp8(1 if transA else 0, 1 if transB else 0, M, N, K, alpha, pa, fa, lda, psa, ldsa,
                                        ba, pb, fb, ldb, psb, ldsb, bb, beta, pc, tc, ldc, _current_raw_stream(dev))
    if st != 0:
        raise SgemmError(st, "sgemm_fp8")
    return C


def rms_norm_fp8(x, weight, residual=None, eps=1e-6, dtype=torch.float8_e4m3fn, training=False, stream=None):
    """RMS norm of x + residual, quantised in (1, 128) blocks: RmsNormFp8(q, scale, h, y, rstd).

    h = x + residual in x's type (None without a residual: h is x).  With training=True also y, the norm in x's
    type, and rstd = 1 / sqrt(mean(h^2) + eps) per row, which rms_norm_backward wants (not set for rows without
    elements).  `weight` is float32 or of x's type."""
    if _usual is not None and stream is None and dtype in _FP8:
        r = _usual.norm(x, weight, residual, eps, _FP8[dtype], training)
        if r is not None:
            return RmsNormFp8._make(r)
    px, rows, cols, ldx, tx, dev = _mat(x, "x", _FLOAT)
    tq = _fp8_type(dtype)
    pw, tw, devw = _vec(weight, "weight", cols, _WEIGHT[tx])
    pr, ldr, devr = None, 0, dev
    if residual is not None:
        pr, rr, rc, ldr, _, devr = _mat(residual, "residual", _SAME[tx])
        if rr != rows or rc != cols:
            raise ValueError(f"residual must be {rows} x {cols}")
    if not dev == devw == devr:
        raise ValueError("tensors are on different devices")
    ctx = _on(stream, dev)
    if ctx is not None:
        with ctx:
            return rms_norm_fp8(x, weight, residual, eps, dtype, training)
    q, ldq = _empty_fp8(rows, cols, dtype, x.device)
    kb = _cdiv(cols, BLOCK)
    s = torch.empty((rows, kb), dtype=torch.float32, device=x.device)
    h = y = t = ph = py = pt = None
    if residual is not None:
        h = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
        ph = h.data_ptr()
    if training:
        y = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
        t = torch.empty((rows,), dtype=torch.float32, device=x.device)
        py, pt = y.data_ptr(), t.data_ptr()
    ld = cols or 1
    st = (_lib or _library()).sgemm_rms_norm_fp8(rows, cols, eps, px, ldx, pr, ldr, tx, pw, tw, ph, ld, py, ld,
                                                 q.data_ptr(), tq, ldq, s.data_ptr(), kb or 1, pt,
                                                 _current_raw_stream(dev))
    if st != 0:
        raise SgemmError(st, "sgemm_rms_norm_fp8")
    return RmsNormFp8(q, s, h, y, t)


def rms_norm_backward(dy, h, weight, rstd, dh=None, stream=None):
    """(dx, dweight) of y = h * rstd * weight: dx (the gradient of x and of the residual alike, `dh` added to it)
    in h's type, dweight in weight's.  `dh` is the gradient that reaches h along the residual path."""
    if _usual is not None and stream is None:
        r = _usual.norm_backward(dy, h, weight, rstd, dh)
        if r is not None:
            return r
    pd, rows, cols, lddy, tx, dev = _mat(dy, "dy", _FLOAT)
    ph, hr, hc, ldh, _, devh = _mat(h, "h", _SAME[tx])
    if hr != rows or hc != cols:
        raise ValueError(f"h must be {rows} x {cols}")
    pw, tw, devw = _vec(weight, "weight", cols, _WEIGHT[tx])
    pt, _, devt = _vec(rstd, "rstd", rows, _F32)
    pg, lddh, devg = None, 0, dev
    if dh is not None:
        pg, gr, gc, lddh, _, devg = _mat(dh, "dh", _SAME[tx])
        if gr != rows or gc != cols:
            raise ValueError(f"dh must be {rows} x {cols}")
    _one_device(dev, devh, devw, devt, devg)
    ctx = _on(stream, dev)
    if ctx is not None:
        with ctx:
            return rms_norm_backward(dy, h, weight, rstd, dh)
    lib = _lib or _library()
    dx = torch.empty((rows, cols), dtype=dy.dtype, device=dy.device)
    dw = torch.empty((cols,), dtype=weight.dtype, device=dy.device)
    need = lib.sgemm_rms_norm_backward_workspace(rows, cols)
    ws = torch.empty((need // 4,), dtype=torch.float32, device=dy.device)
    st = lib.sgemm_rms_norm_backward(rows, cols, pd, lddy, ph, ldh, tx, pw, tw, pt, pg, lddh, dx.data_ptr(), cols or 1,
                                     dw.data_ptr(), ws.data_ptr(), need, _current_raw_stream(dev))
    if st != 0:
        raise SgemmError(st, "sgemm_rms_norm_backward")
    return dx, dw
