"""What stands around the products of a gated block in 8-bit floating point: torch tensors -> include/sgemm_fp8_block.h.

    o = sandwich_norm_fp8(a, x, post_weight, weight, gate=gate)    # o.q, o.scale: the next product's operand; o.h
    g = sandwich_norm_backward(dy, o.a8, o.h8, post_weight, weight, o.post_rstd, o.rstd, gate=gate, dh=dh)
    o = swiglu_fp8(gate, up)                                       # o.q, o.scale: the down projection's operand
    g = swiglu_backward_fp8(dy, o.gate8, o.up8)                    # operands of the gradients' products
    q, s = requantize_fp8(q, s)                                    # (1, 128) blocks -> (128, 1) blocks

A checkpoint is a matrix in 8 bits as quantize_fp8 makes it in (1, 128) blocks, a pair (q, scale): half the memory of a
16-bit matrix between the forward and the backward pass.  Where the backward functions take a matrix that the forward
pass had, they take it or its checkpoint.

Tensors, streams and errors are as in module fp8: 2-D CUDA tensors with unit column stride and any row stride, every
function runs on ``stream`` or torch's current stream and returns once its work is queued, nothing here computes.  The
matrices made here have rows that start on 16-byte (8-bit) or 32-byte boundaries: a row stride rounded up to 16.  An 8-bit
matrix and its scales may share one allocation, and so may all that a call returns for the backward pass, the gradients of
weights and of a gate for all rows, or everything else that a call makes if that is a megabyte at most: what shares one is
freed when the last of it is.
"""
import collections
import ctypes

import torch

from . import fp8
from ._binding import SgemmError, _current_raw_stream
from .fp8 import BLOCK, _FLOAT, _FP8, _SAME, _WEIGHT, _F32, _cdiv, _empty_fp8, _fp8_type, _mat, _on, _one_device, _vec

E4M3 = torch.float8_e4m3fn

SandwichNormFp8 = collections.namedtuple("SandwichNormFp8", "q scale h post_rstd rstd a8 h8")
SandwichNormFp8.__doc__ = """What sandwich_norm_fp8 returns: the quantised norm and its scales, h, with training=True
post_rstd and rstd, and with checkpoint=... a8 and h8, the pairs (q, scale) of a and h in 8 bits (else None)."""
SandwichNormGrad = collections.namedtuple("SandwichNormGrad", "da dx dpost_weight dweight dgate")
SandwichNormGrad.__doc__ = """What sandwich_norm_backward returns (dgate None without a gate)."""
SwigluFp8 = collections.namedtuple("SwigluFp8", "q scale gate8 up8")
SwigluFp8.__doc__ = """What swiglu_fp8 returns: the quantised unit and its scales, and with checkpoint=... gate8 and up8,
the pairs (q, scale) of gate and up in 8 bits (else None)."""
SwigluGradFp8 = collections.namedtuple("SwigluGradFp8", "q_rows scale_rows q_cols scale_cols y_cols y_scale")
SwigluGradFp8.__doc__ = """What swiglu_backward_fp8 returns: [dgate | dup] in (1, 128) and in (128, 1) blocks, and the
unit y in (128, 1) blocks."""

_lib = None
_I64, _VP, _INT, _F = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float


def _library():
    global _lib
    if _lib is None:
        lib = fp8._library()
        lib.sgemm_sandwich_norm_fp8.argtypes = [
            _I64, _I64, _F, _F, _VP, _I64, _VP, _I64, _INT, _VP, _VP, _INT, _VP, _I64, _INT, _I64, _VP, _I64, _VP, _INT,
            _I64, _VP, _I64, _VP, _VP, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _I64, _INT, _VP]
        lib.sgemm_sandwich_norm_backward.argtypes = [
            _I64, _I64, _F, _VP, _I64, _VP, _I64, _INT, _VP, _INT, _I64, _VP, _I64, _VP, _INT, _I64, _VP, _I64, _VP, _VP,
            _INT, _VP, _I64, _INT, _I64, _VP, _VP, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _I64, _VP, ctypes.c_size_t, _VP]
        lib.sgemm_swiglu_fp8.argtypes = [_I64, _I64, _VP, _I64, _VP, _I64, _INT, _VP, _INT, _I64, _VP, _I64, _VP, _I64,
                                         _VP, _I64, _VP, _I64, _VP, _I64, _INT, _VP]
        lib.sgemm_swiglu_backward_fp8.argtypes = [
            _I64, _I64, _VP, _I64, _INT, _VP, _INT, _I64, _VP, _I64, _VP, _INT, _I64, _VP, _I64, _INT, _VP, _I64, _VP,
            _I64, _VP, _I64, _VP, _I64, _INT, _VP, _I64, _VP, _I64, _VP]
        lib.sgemm_fp8_requantize.argtypes = [_I64, _I64, _VP, _INT, _I64, _VP, _I64, _VP, _INT, _I64, _VP, _I64, _VP]
        for f in (lib.sgemm_sandwich_norm_fp8, lib.sgemm_sandwich_norm_backward, lib.sgemm_swiglu_fp8,
                  lib.sgemm_swiglu_backward_fp8, lib.sgemm_fp8_requantize):
            f.restype = _INT
        lib.sgemm_sandwich_norm_backward_workspace.argtypes = [_I64, _I64]
        lib.sgemm_sandwich_norm_backward_workspace.restype = ctypes.c_size_t
        _lib = lib
    return _lib


def _raise(where, status):
    if status != 0:
        raise SgemmError(status, where)


# ------------------------------------------------------------------ the C ABI
# (same names and arguments, pointers as ints, raising SgemmError)
def sgemm_sandwich_norm_fp8(rows, cols, eps, residual_scale, A, lda, X, ldx, typeX, WP, W, typeW, GATE, ldgate, typeGate,
                            group_rows, H, ldh, Q, typeQ, ldq, S, lds, TP, T, QA, ldqa, SA, ldsa, QH, ldqh, SH, ldsh,
                            typeKeep, stream=None):
    """Norm of A, gate, residual X, norm with an 8-bit output (GATE, TP, T, QA with SA, QH with SH may be None)."""
    _raise("sgemm_sandwich_norm_fp8", _library().sgemm_sandwich_norm_fp8(
        rows, cols, eps, residual_scale, A, lda, X, ldx, typeX, WP, W, typeW, GATE, ldgate, typeGate, group_rows, H, ldh,
        Q, typeQ, ldq, S, lds, TP, T, QA, ldqa, SA, ldsa, QH, ldqh, SH, ldsh, typeKeep, stream))


def sgemm_sandwich_norm_backward(rows, cols, residual_scale, DY, lddy, DH, lddh, typeX, A, typeA, lda, SA, ldsa, H, typeH,
                                 ldh, SH, ldsh, WP, W, typeW, GATE, ldgate, typeGate, group_rows, TP, T, DA, ldda, DX,
                                 lddx, DWP, DW, DGATE, lddgate, workspace, workspace_bytes, stream=None):
    """Its gradient (DH, SA, SH, GATE, DWP, DW, DGATE and, without those three, workspace may be None)."""
    _raise("sgemm_sandwich_norm_backward", _library().sgemm_sandwich_norm_backward(
        rows, cols, residual_scale, DY, lddy, DH, lddh, typeX, A, typeA, lda, SA, ldsa, H, typeH, ldh, SH, ldsh, WP, W,
        typeW, GATE, ldgate, typeGate, group_rows, TP, T, DA, ldda, DX, lddx, DWP, DW, DGATE, lddgate, workspace,
        workspace_bytes, stream))


def sgemm_sandwich_norm_backward_workspace(rows, cols) -> int:
    """Bytes of workspace that sgemm_sandwich_norm_backward needs."""
    return _library().sgemm_sandwich_norm_backward_workspace(rows, cols)


def sgemm_swiglu_fp8(rows, cols, G, ldg, U, ldu, typeX, Q, typeQ, ldq, S, lds, QG, ldqg, SG, ldsg, QU, ldqu, SU, ldsu,
                     typeKeep, stream=None):
    """The gated unit with an 8-bit output (QG with SG, QU with SU may be None)."""
    _raise("sgemm_swiglu_fp8", _library().sgemm_swiglu_fp8(rows, cols, G, ldg, U, ldu, typeX, Q, typeQ, ldq, S, lds, QG,
                                                           ldqg, SG, ldsg, QU, ldqu, SU, ldsu, typeKeep, stream))


def sgemm_swiglu_backward_fp8(rows, cols, DY, lddy, typeX, G, typeG, ldg, SG, ldsg, U, typeU, ldu, SU, ldsu, typeZ, QR,
                              ldqr, SR, ldsr, QC, ldqc, SC, ldsc, typeY, QY, ldqy, SY, ldsy, stream=None):
    """Its gradient in both quantisations, and the unit in 128 x 1 blocks (SG and SU are None for G, U of typeX)."""
    _raise("sgemm_swiglu_backward_fp8", _library().sgemm_swiglu_backward_fp8(
        rows, cols, DY, lddy, typeX, G, typeG, ldg, SG, ldsg, U, typeU, ldu, SU, ldsu, typeZ, QR, ldqr, SR, ldsr, QC,
        ldqc, SC, ldsc, typeY, QY, ldqy, SY, ldsy, stream))


def sgemm_fp8_requantize(rows, cols, QX, typeX, ldqx, SX, ldsx, Q, typeQ, ldq, S, lds, stream=None):
    """1 x 128 blocks (QX, SX) -> 128 x 1 blocks (Q, S)."""
    _raise("sgemm_fp8_requantize", _library().sgemm_fp8_requantize(rows, cols, QX, typeX, ldqx, SX, ldsx, Q, typeQ, ldq,
                                                                   S, lds, stream))


# ------------------------------------------------------------------ torch
def _like(t, name, rows, cols, types):
    """_mat() of a matrix that must be rows x cols."""
    m = _mat(t, name, types)
    if m[1] != rows or m[2] != cols:
        raise ValueError(f"{name} must be {rows} x {cols}")
    return m


def _kept(k, name, rows, cols, types):
    """(pointer, type, ld, scales' pointer or None, their ld, device) of a matrix or its checkpoint."""
    if not isinstance(k, tuple):
        p, _, _, ld, code, dev = _like(k, name, rows, cols, types)
        return p, code, ld, None, 1, dev
    if len(k) != 2:
        raise TypeError(f"{name} must be a matrix or a pair (q, scale)")
    p, _, _, ld, code, dev = _like(k[0], name, rows, cols, _FP8)
    ps, _, _, lds, _, devs = _like(k[1], f"{name}'s scales", rows, _cdiv(cols, BLOCK), _F32)
    _one_device(dev, devs)
    return p, code, ld, ps, lds, dev


def _gate(gate, rows, cols, types):
    """(pointer, ld, type, rows that share one, device): of one row for all, or of one for every rows / gate.rows."""
    if getattr(gate, "ndim", 0) == 1:
        p, code, dev = _vec(gate, "gate", cols, types)
        return p, max(cols, 1), code, max(rows, 1), dev
    p, groups, gc, ld, code, dev = _mat(gate, "gate", types)
    if gc != cols or (rows % groups if groups else rows):
        raise ValueError(f"gate must have {cols} columns and a number of rows that divides {rows}")
    return p, ld, code, max(rows // groups, 1) if groups else 1, dev


def _empty_rows(rows, cols, like):
    """(tensor of like's type, ld): rows on 32-byte boundaries."""
    ld = max((cols + 15) // 16 * 16, 1)
    return torch.empty_strided((rows, cols), (ld, 1), dtype=like.dtype, device=like.device), ld


def _checkpoint(rows, cols, dtype, dev):
    q, ld = _empty_fp8(rows, cols, dtype, dev)
    return (q, torch.empty((rows, _cdiv(cols, BLOCK)), dtype=torch.float32, device=dev)), ld


def sandwich_norm_fp8(a, x, post_weight, weight, gate=None, residual_scale=1.0, eps=1e-6, dtype=E4M3, training=False,
                      checkpoint=None, stream=None):
    """The norm behind a block, its gate, the residual and the norm in front of the next block, quantised in (1, 128)
    blocks: SandwichNormFp8(q, scale, h, post_rstd, rstd, a8, h8) of

        h = residual_scale * x + gate * (rmsnorm(a) * post_weight),     y = rmsnorm(h) * weight

    `a` is the block's output, `x` the residual stream, both of one type; h is of it too.  `gate` is a vector for all
    rows, or a matrix with one row for each of as many equal runs of consecutive rows (sequences, say; one row each if
    it has a's number of rows).  post_weight, weight and gate are float32 or of a's type.  With training=True also
    post_rstd and rstd, which sandwich_norm_backward wants (not set for rows without elements); with `checkpoint` an
    8-bit type also the checkpoints of a and h in it."""
    if fp8._usual is not None and stream is None and dtype in _FP8:
        r = fp8._usual.sandwich_norm(a, x, post_weight, weight, gate, residual_scale, eps, _FP8[dtype], training,
                                     -1 if checkpoint is None else _fp8_type(checkpoint))
        if r is not None:
            return SandwichNormFp8._make(r)
    px, rows, cols, lda, tx, dev = _mat(a, "a", _FLOAT)
    pr, _, _, ldx, _, devx = _like(x, "x", rows, cols, _SAME[tx])
    tq = _fp8_type(dtype)
    tk = _fp8_type(checkpoint) if checkpoint is not None else tq
    pwp, twp, devwp = _vec(post_weight, "post_weight", cols, _WEIGHT[tx])
    pw, tw, devw = _vec(weight, "weight", cols, _WEIGHT[tx])
    if twp != tw:
        raise TypeError("post_weight and weight must be of one type")
    pg, ldg, tg, group, devg = (None, 1, tx, 1, dev) if gate is None else _gate(gate, rows, cols, _WEIGHT[tx])
    _one_device(dev, devx, devwp, devw, devg)
    ctx = _on(stream, dev)
    if ctx is not None:
        with ctx:
            return sandwich_norm_fp8(a, x, post_weight, weight, gate, residual_scale, eps, dtype, training, checkpoint)
    q, ldq = _empty_fp8(rows, cols, dtype, a.device)
    kb = _cdiv(cols, BLOCK)
    s = torch.empty((rows, kb), dtype=torch.float32, device=a.device)
    h, ld = _empty_rows(rows, cols, a)
    tp = t = a8 = h8 = ptp = pt = None
    keep = [None, 1, None, 1] * 2
    if training:
        tp, t = (torch.empty((rows,), dtype=torch.float32, device=a.device) for _ in range(2))
        ptp, pt = tp.data_ptr(), t.data_ptr()
    if checkpoint is not None:
        a8, ldk = _checkpoint(rows, cols, checkpoint, a.device)
        h8, _ = _checkpoint(rows, cols, checkpoint, a.device)
        keep = [v for k in (a8, h8) for v in (k[0].data_ptr(), ldk, k[1].data_ptr(), kb or 1)]
    _raise("sgemm_sandwich_norm_fp8", (_lib or _library()).sgemm_sandwich_norm_fp8(
        rows, cols, eps, residual_scale, px, lda, pr, ldx, tx, pwp, pw, tw, pg, ldg, tg, group, h.data_ptr(), ld,
        q.data_ptr(), tq, ldq, s.data_ptr(), kb or 1, ptp, pt, *keep, tk, _current_raw_stream(dev)))
    return SandwichNormFp8(q, s, h, tp, t, a8, h8)


def sandwich_norm_backward(dy, a, h, post_weight, weight, post_rstd, rstd, gate=None, residual_scale=1.0, dh=None,
                           stream=None):
    """The gradient of sandwich_norm_fp8's y: SandwichNormGrad(da, dx, dpost_weight, dweight, dgate).

    `a` and `h` are the forward pass's matrices (of dy's type) or checkpoints of them, post_rstd and rstd what it
    returned; `dh` is the gradient that reaches h along the residual path.  da and dx are in dy's type, the others in
    those of what they are gradients of; dgate is summed over the rows that share a row of the gate."""
    if fp8._usual is not None and stream is None:
        r = fp8._usual.sandwich_norm_backward(dy, a, h, post_weight, weight, post_rstd, rstd, gate, residual_scale, dh)
        if r is not None:
            return SandwichNormGrad._make(r)
    pd, rows, cols, lddy, tx, dev = _mat(dy, "dy", _FLOAT)
    pa, ta, lda, psa, ldsa, deva = _kept(a, "a", rows, cols, _SAME[tx])
    ph, th, ldh, psh, ldsh, devh = _kept(h, "h", rows, cols, _SAME[tx])
    pwp, twp, devwp = _vec(post_weight, "post_weight", cols, _WEIGHT[tx])
    pw, tw, devw = _vec(weight, "weight", cols, _WEIGHT[tx])
    if twp != tw:
        raise TypeError("post_weight and weight must be of one type")
    ptp, _, devtp = _vec(post_rstd, "post_rstd", rows, _F32)
    pt, _, devt = _vec(rstd, "rstd", rows, _F32)
    pg, ldg, tg, group, devg = (None, 1, tx, 1, dev) if gate is None else _gate(gate, rows, cols, _WEIGHT[tx])
    pdh, lddh, devdh = None, 1, dev
    if dh is not None:
        pdh, _, _, lddh, _, devdh = _like(dh, "dh", rows, cols, _SAME[tx])
    _one_device(dev, deva, devh, devwp, devw, devtp, devt, devg, devdh)
    ctx = _on(stream, dev)
    if ctx is not None:
        with ctx:
            return sandwich_norm_backward(dy, a, h, post_weight, weight, post_rstd, rstd, gate, residual_scale, dh)
    lib = _lib or _library()
    (da, ld), (dx, _) = (_empty_rows(rows, cols, dy) for _ in range(2))
    dwp, dw = (torch.empty((cols,), dtype=weight.dtype, device=dy.device) for _ in range(2))
    dg = None
    if gate is not None:
        dg = torch.empty_like(gate) if gate.dim() == 1 else _empty_rows(len(gate), cols, gate)[0]
    need = lib.sgemm_sandwich_norm_backward_workspace(rows, cols)
    ws = torch.empty((need // 4,), dtype=torch.float32, device=dy.device)
    if dg is not None and rows == 0:
        dg.zero_()   # a sum over no rows
    _raise("sgemm_sandwich_norm_backward", lib.sgemm_sandwich_norm_backward(
        rows, cols, residual_scale, pd, lddy, pdh, lddh, tx, pa, ta, lda, psa, ldsa, ph, th, ldh, psh, ldsh, pwp, pw, tw,
        pg, ldg, tg, group, ptp, pt, da.data_ptr(), ld, dx.data_ptr(), ld, dwp.data_ptr(), dw.data_ptr(),
        dg.data_ptr() if dg is not None and rows else None, ld, ws.data_ptr(), need, _current_raw_stream(dev)))
    return SandwichNormGrad(da, dx, dwp, dw, dg)


def swiglu_fp8(gate, up, dtype=E4M3, checkpoint=None, stream=None):
    """The gated unit y = silu(gate) * up, quantised in (1, 128) blocks: SwigluFp8(q, scale, gate8, up8).

    gate and up are of one type (the halves of one product's output, say).  With `checkpoint` an 8-bit type also the
    checkpoints of both in it, which swiglu_backward_fp8 takes."""
    if fp8._usual is not None and stream is None and dtype in _FP8:
        r = fp8._usual.swiglu(gate, up, _FP8[dtype], -1 if checkpoint is None else _fp8_type(checkpoint))
        if r is not None:
            return SwigluFp8._make(r)
    pg, rows, cols, ldg, tx, dev = _mat(gate, "gate", _FLOAT)
    pu, _, _, ldu, _, devu = _like(up, "up", rows, cols, _SAME[tx])
    _one_device(dev, devu)
    tq = _fp8_type(dtype)
    tk = _fp8_type(checkpoint) if checkpoint is not None else tq
    ctx = _on(stream, dev)
    if ctx is not None:
        with ctx:
            return swiglu_fp8(gate, up, dtype, checkpoint)
    q, ldq = _empty_fp8(rows, cols, dtype, gate.device)
    kb = _cdiv(cols, BLOCK)
    s = torch.empty((rows, kb), dtype=torch.float32, device=gate.device)
    g8 = u8 = None
    keep = [None, 1, None, 1] * 2
    if checkpoint is not None:
        g8, ldk = _checkpoint(rows, cols, checkpoint, gate.device)
        u8, _ = _checkpoint(rows, cols, checkpoint, gate.device)
        keep = [v for k in (g8, u8) for v in (k[0].data_ptr(), ldk, k[1].data_ptr(), kb or 1)]
    _raise("sgemm_swiglu_fp8", (_lib or _library()).sgemm_swiglu_fp8(
        rows, cols, pg, ldg, pu, ldu, tx, q.data_ptr(), tq, ldq, s.data_ptr(), kb or 1, *keep, tk,
        _current_raw_stream(dev)))
    return SwigluFp8(q, s, g8, u8)


def swiglu_backward_fp8(dy, gate, up, dtype=E4M3, y_dtype=E4M3, stream=None):
    """The gradient of silu(gate) * up as operands of the products that follow: SwigluGradFp8(q_rows, scale_rows, q_cols,
    scale_cols, y_cols, y_scale).

    gate and up are the forward pass's matrices (of dy's type) or both checkpoints of one type.  q_rows and q_cols hold
    [dgate | dup] in `dtype`, each half as wide as cols rounded up to a multiple of 128 and zero behind its cols columns:
    the operand of a product with both projections' weights in one matrix, or by halves (q[:, :cols] and
    q[:, q.shape[1] // 2:][:, :cols], the scales likewise) of one with each.  y_cols is y in `y_dtype`, for the weight
    gradient of the projection that read it."""
    if fp8._usual is not None and stream is None and dtype in _FP8 and y_dtype in _FP8:
        r = fp8._usual.swiglu_backward(dy, gate, up, _FP8[dtype], _FP8[y_dtype])
        if r is not None:
            return SwigluGradFp8._make(r)
    pd, rows, cols, lddy, tx, dev = _mat(dy, "dy", _FLOAT)
    pg, tg, ldg, psg, ldsg, devg = _kept(gate, "gate", rows, cols, _SAME[tx])
    pu, tu, ldu, psu, ldsu, devu = _kept(up, "up", rows, cols, _SAME[tx])
    if tg != tu:
        raise TypeError("gate and up must be both matrices or both checkpoints of one type")
    _one_device(dev, devg, devu)
    tz, ty = _fp8_type(dtype), _fp8_type(y_dtype)
    ctx = _on(stream, dev)
    if ctx is not None:
        with ctx:
            return swiglu_backward_fp8(dy, gate, up, dtype, y_dtype)
    kb, rb = _cdiv(cols, BLOCK), _cdiv(rows, BLOCK)
    wide, ld = 2 * kb * BLOCK, max(2 * kb * BLOCK, 1)
    qr, qc = (torch.empty((rows, wide), dtype=dtype, device=dy.device) for _ in range(2))
    sr, sc, sy = (torch.empty(n, dtype=torch.float32, device=dy.device) for n in ((rows, 2 * kb), (rb, wide), (rb, cols)))
    qy, ldqy = _empty_fp8(rows, cols, y_dtype, dy.device)
    _raise("sgemm_swiglu_backward_fp8", (_lib or _library()).sgemm_swiglu_backward_fp8(
        rows, cols, pd, lddy, tx, pg, tg, ldg, psg, ldsg, pu, tu, ldu, psu, ldsu, tz, qr.data_ptr(), ld, sr.data_ptr(),
        2 * kb or 1, qc.data_ptr(), ld, sc.data_ptr(), ld, ty, qy.data_ptr(), ldqy, sy.data_ptr(), cols or 1,
        _current_raw_stream(dev)))
    return SwigluGradFp8(qr, sr, qc, sc, qy, sy)


def requantize_fp8(q, scale, dtype=None, stream=None):
    """(q, scale) in (128, 1) blocks of what a matrix in (1, 128) blocks stands for, in `dtype` (default: q's): a weight
    gradient's operand from the rows that the forward pass multiplied with."""
    if fp8._usual is not None and stream is None:
        to = _FP8.get(getattr(q, "dtype", None) if dtype is None else dtype, -1)
        r = fp8._usual.requantize(q, scale, to) if to >= 0 else None
        if r is not None:
            return r
    pq, rows, cols, ldq, tx, dev = _mat(q, "q", _FP8)
    ps, _, _, lds, _, devs = _like(scale, "scale", rows, _cdiv(cols, BLOCK), _F32)
    _one_device(dev, devs)
    dtype = q.dtype if dtype is None else dtype
    tq = _fp8_type(dtype)
    ctx = _on(stream, dev)
    if ctx is not None:
        with ctx:
            return requantize_fp8(q, scale, dtype)
    o, ldo = _empty_fp8(rows, cols, dtype, q.device)
    s = torch.empty((_cdiv(rows, BLOCK), cols), dtype=torch.float32, device=q.device)
    _raise("sgemm_fp8_requantize", (_lib or _library()).sgemm_fp8_requantize(
        rows, cols, pq, tx, ldq, ps, lds, o.data_ptr(), tq, ldo, s.data_ptr(), cols or 1, _current_raw_stream(dev)))
    return o, s
