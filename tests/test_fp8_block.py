"""What stands around a gated block's products in 8-bit floating point: the norms around a block with gate and residual,
the gated unit, their gradients, and kept rows as a weight gradient's operand, each against its definition in 64 bits.

Tolerances, with u = 2^-24 (FP32 rounding), derived where they are used:
  sums      over a row: at most 72 additions in a thread and 10 after it; over rows: at most 34 in a CTA, 38 over CTAs
            and 5 after that.  With the roundings of what is added all of them lose at most 2^-17 of the sum of
            magnitudes (128 u).
  norms     t is within 2^-17 relative for given h; what h is off by comes on top, and is carried through to y.
  gradient  the formula's sums, each off by 2^-17 of its magnitudes, carried through likewise.
  unit      __expf is off by 2 + 1.173 |g| units in the last place and __fdividef by 2 (CUDA's documented bounds).
            What the kernels do lies within these: ex2.approx is off by 2^-22 and its argument g log2(e), rounded twice, by
            |g| 1.32 u of the result, together at most 4 u + 1.32 |g| u, and a unit in the last place is u at least, 2 u at
            most; rcp.approx is off by one unit.
  q, s      a value that is off by E and its block's by at most E* has a scale off by E* / F and a q within half a step
            of the 8-bit type plus E / s.
These hold for the 32-bit value; rounding to the output type is monotone, so the output lies between the bounds' own
roundings (`within`).
"""
import pytest
import torch

from .test_fp8 import B, E4M3, E5M2, FLOATS, FMAX, U, cdiv, rng, sg, clean_status, spread, strided, ulp8, within  # noqa: F401

gpu = pytest.mark.gpu
SUM = 2.0 ** -17


def close_quantised(q, s, want, E, br, bc):
    """q, s against the values `want` (64 bits), each known up to E."""
    rows, cols = want.shape
    F = FMAX[q.dtype]

    def block_max(v):
        p = v.new_zeros(cdiv(rows, br) * br, cdiv(cols, bc) * bc)
        p[:rows, :cols] = v
        return p.view(cdiv(rows, br), br, cdiv(cols, bc), bc).abs().amax((1, 3))
    least = (block_max(want) / F).clamp_min(2.0 ** -126)
    assert q.shape == want.shape and s.shape == least.shape
    assert ((s.double() - least).abs() <= block_max(E) / F + 2 * U * least).all()
    S = spread(s, br, bc, rows, cols)
    v, e = want / S, E / S
    lim = ulp8(v.abs() + e, q.dtype) / 2 + e + 4 * U * v.abs()
    assert ((q.double() - v).abs() <= lim).all()


def same(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def same_rows(a, b, rows):
    a, b = (v.contiguous().view(torch.uint8).view(len(rows), -1)[rows] for v in (a, b))
    return torch.equal(a, b)


def randn(shape, seed, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=rng(seed), device="cuda") * scale).to(dtype)


def gate_of(kind, rows, cols, dtype, seed):
    """None, a vector, one row each, or one for each of `kind` runs of rows."""
    if kind == "none":
        return None
    g = randn(cols if kind == "one" else (rows if kind == "each" else kind, cols), seed)
    return g.to(dtype)


def gate_rows(gate, rows):
    """The gate of every row in 64 bits."""
    if gate is None:
        return 1.0
    g = gate.double()
    return g[None, :] if g.dim() == 1 else g.repeat_interleave(rows // g.shape[0], 0)


def mean_square(v):
    return v.square().mean(1, keepdim=True)


# ---------------------------------------------------------------- norms around a block
def forward_bounds(a, x, wp, w, gate, rho, eps):
    """tp, h, t, y in 64 bits and what the kernel's may be off by."""
    a, x, wp, w = (v.double() for v in (a, x, wp, w))
    tp = 1 / (mean_square(a) + eps).sqrt()
    u = a * tp * wp * gate_rows(gate, a.shape[0])
    h = rho * x + u
    Eh = (SUM + 4 * U) * u.abs() + U * (h.abs() + (rho * x).abs())
    t = 1 / (mean_square(h) + eps).sqrt()
    # |mean (h + e)^2 - mean h^2| <= 2 |h| |e| + |e|^2 in the mean; half of it relative to mean h^2 + eps reaches t
    et = SUM + ((Eh * h.abs()).mean(1, keepdim=True) + mean_square(Eh)) * t.square()
    y = h * t * w
    Ey = Eh * (t * w).abs() + y.abs() * (et + 4 * U)
    return tp, h, Eh, t, et, y, Ey


# a row a warp; a row a CTA of up to 1024 threads; two chunks a thread (16-bit types from 1216 rows on); longer rows
NORM_SHAPES = [(1, 1), (1, 128), (7, 5), (129, 127), (19, 512), (1, 4096), (300, 1000), (700, 520), (612, 1024), (40, 2100),
               (305, 4097), (612, 8192), (1217, 4104), (1217, 5128), (1300, 8192), (5, 16384), (3, 16392), (2, 33000)]


@gpu
@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("gate", ["none", "one", "each"])
def test_norms(sg, shape, dtype, gate):  # noqa: F811
    rows, cols = shape
    a, x = randn(shape, 1, dtype, 3.0), randn(shape, 2, dtype)
    wp, w = 1 + randn(cols, 3, scale=0.1), 1 + randn(cols, 4, scale=0.1)
    if gate == "each":
        wp, w = wp.to(dtype), w.to(dtype)
    g = gate_of(gate, rows, cols, torch.float32 if gate == "one" else dtype, 5)
    rho, eps = 0.75, 1e-5
    o = sg.sandwich_norm_fp8(a, x, wp, w, gate=g, residual_scale=rho, eps=eps, training=True, checkpoint=E5M2)
    tp, h, Eh, t, et, y, Ey = forward_bounds(a, x, wp, w, g, rho, eps)
    assert o.h.dtype == dtype and within(o.h, h, Eh)
    assert ((o.post_rstd.double()[:, None] - tp).abs() <= SUM * tp).all()
    assert ((o.rstd.double()[:, None] - t).abs() <= et * t).all()
    close_quantised(o.q, o.scale, y, Ey, 1, B)
    close_quantised(*o.h8, h, Eh, 1, B)
    for got, want in zip(o.a8, sg.quantize_fp8(a, dtype=E5M2)):
        assert same(got, want)
    bare = sg.sandwich_norm_fp8(a, x, wp, w, gate=g, residual_scale=rho, eps=eps)
    assert bare.post_rstd is bare.rstd is bare.a8 is bare.h8 is None
    for got, want in zip(bare[:3], o[:3]):
        assert same(got, want)


@gpu
@pytest.mark.parametrize("groups,each", [(1, 5), (5, 1), (3, 7), (2, 400), (40, 33)])
def test_a_gate_for_each_run_of_rows(sg, groups, each):  # noqa: F811
    """A gate row for every run is the same as the run by itself with its gate for all."""
    rows, cols = groups * each, 392
    a, x = randn((rows, cols), 11, torch.bfloat16), randn((rows, cols), 12, torch.bfloat16)
    wp, w, g = randn(cols, 13), randn(cols, 14), randn((groups, cols), 15)
    o = sg.sandwich_norm_fp8(a, x, wp, w, gate=g, training=True)
    tp, h, Eh, t, et, y, Ey = forward_bounds(a, x, wp, w, g, 1.0, 1e-6)
    assert within(o.h, h, Eh)
    close_quantised(o.q, o.scale, y, Ey, 1, B)
    for i in range(groups if rows < 600 else 0):   # (more rows are laid over threads otherwise)
        part = slice(i * each, (i + 1) * each)
        alone = sg.sandwich_norm_fp8(a[part], x[part], wp, w, gate=g[i], training=True)
        for got, want in zip(o[:5], alone[:5]):
            assert same(got[part], want)


def gradient_bounds(dy, dh, a, h, wp, w, gate, tp, t, rho):
    """The gradient in 64 bits, {name: (value, what the kernel's may be off by)}; a, h: 64 bits, off by u if kept."""
    rows, cols = dy.shape
    dy, wp, w, tp, t = dy.double(), wp.double(), w.double(), tp.double()[:, None], t.double()[:, None]
    dh = torch.zeros_like(dy) if dh is None else dh.double()
    gr = gate_rows(gate, rows)
    g, p = dy * w, gr * wp * a
    mean = lambda v: v.mean(1, keepdim=True)   # noqa: E731
    k = t.square() * mean(g * h)
    Ek = (SUM + 8 * U) * t.square() * mean((g * h).abs())
    H = t * (g - h * k) + dh
    EH = t * h.abs() * Ek + 8 * U * (t * (g.abs() + (h * k).abs()) + dh.abs())
    v = H * gr * wp
    kp = tp.square() * mean(v * a)
    SP, SR = mean((t * g.abs() + dh.abs()) * p.abs()), mean((h * p).abs())
    Ekp = tp.square() * ((SUM + 8 * U) * (SP + (t * k).abs() * SR) + t * Ek * SR)
    da = tp * (v - a * kp)
    Eda = tp * ((gr * wp).abs() * EH + a.abs() * Ekp + 8 * U * (v.abs() + (a * kp).abs())) if gate is not None else \
        tp * (wp.abs() * EH + a.abs() * Ekp + 8 * U * (v.abs() + (a * kp).abs()))
    n, En = H * a * tp, EH * a.abs() * tp
    dw, dwp = dy * h * t, n * gr
    Edwp = En * (gr.abs() if gate is not None else 1.0)
    out = {"da": (da, Eda), "dx": (rho * H, abs(rho) * EH + U * (rho * H).abs()),
           "dpost_weight": (dwp.sum(0), (SUM * dwp.abs() + Edwp).sum(0)),
           "dweight": (dw.sum(0), SUM * dw.abs().sum(0))}
    if gate is not None:
        parts = 1 if gate.dim() == 1 else gate.shape[0]
        per = lambda v: v.view(parts, rows // parts, cols).sum(1).view(gate.shape)   # noqa: E731
        out["dgate"] = (per(n * wp), per((SUM * n.abs() + En) * wp.abs()))
    return out


def check_gradient(got, want):
    for name, (value, lim) in want.items():
        assert within(getattr(got, name), value, lim), name


# CTAs of one to four warps, clusters of one, two, four and eight, longer rows; one row a cluster and many
GRADIENT_SHAPES = [(1, 1), (1, 128), (7, 5), (129, 127), (1, 4096), (300, 1000), (2500, 250), (2600, 264), (612, 1032), (700, 2048),
                   (700, 2056), (305, 4097), (700, 4096), (460, 8192), (5, 8200), (310, 8201), (150, 16384), (4, 16392), (310, 16400)]


@gpu
@pytest.mark.parametrize("shape", GRADIENT_SHAPES)
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("gate,keep", [("none", "tensors"), ("one", "e4m3"), ("each", "e5m2"), ("one", "types"), ("each", "a"),
                                       ("none", "h")])
def test_norms_gradient(sg, shape, dtype, gate, keep):  # noqa: F811
    """From the tensors, from checkpoints of one type or of two, and from one of each."""
    rows, cols = shape
    a, h = randn(shape, 21, dtype, 3.0), randn(shape, 22, dtype)
    dy, dh = randn(shape, 23, dtype), randn(shape, 24, dtype)
    wp, w = 1 + randn(cols, 25, scale=0.1), 1 + randn(cols, 26, scale=0.1)
    if gate == "each":
        wp, w = wp.to(dtype), w.to(dtype)
    g = gate_of(gate, rows, cols, torch.float32 if gate == "one" else dtype, 27)
    tp, t = (1 / (mean_square(v.float())[:, 0] + 1e-6).sqrt() for v in (a, h))
    if gate == "none":
        dh = None
    kept = {"e4m3": (E4M3, E4M3), "e5m2": (E5M2, E5M2), "types": (E4M3, E5M2), "a": (E4M3, None), "h": (None, E5M2),
            "tensors": (None, None)}[keep]
    A, H = (v if k is None else sg.quantize_fp8(v, dtype=k) for v, k in zip((a, h), kept))
    va, vh = (v[0].double() * spread(v[1], 1, B, rows, cols) if isinstance(v, tuple) else v.double() for v in (A, H))
    got = sg.sandwich_norm_backward(dy, A, H, wp, w, tp, t, gate=g, residual_scale=0.5, dh=dh)
    assert got.da.dtype == got.dx.dtype == dtype and got.dweight.dtype == got.dpost_weight.dtype == w.dtype
    assert (got.dgate is None) == (g is None)
    check_gradient(got, gradient_bounds(dy, dh, va, vh, wp, w, g, tp, t, 0.5))


@gpu
@pytest.mark.parametrize("groups,each", [(1, 3), (2, 1), (3, 7), (2, 800), (5, 611), (40, 33), (900, 2), (7, 152), (1300, 1)])
@pytest.mark.parametrize("cols", [250, 4096, 8200, 16400])
def test_gradient_of_gates_of_runs(sg, groups, each, cols):  # noqa: F811
    """Runs that lie in one CTA's rows, that end inside them, and that span several."""
    shape, dtype = (groups * each, cols), torch.bfloat16
    if groups * each * cols > 1 << 23:
        pytest.skip("covered by the smaller ones")
    a, h, dy, dh = (randn(shape, 31 + i, dtype) for i in range(4))
    wp, w, g = randn(cols, 35), randn(cols, 36), randn((groups, cols), 37)
    tp, t = (1 / (mean_square(v.float())[:, 0] + 1e-6).sqrt() for v in (a, h))
    got = sg.sandwich_norm_backward(dy, a, h, wp, w, tp, t, gate=g, dh=dh)
    check_gradient(got, gradient_bounds(dy, dh, a.double(), h.double(), wp, w, g, tp, t, 1.0))


@gpu
def test_norms_gradient_against_differences(sg):  # noqa: F811
    """sum(y dy) + sum(h dh) changes along a direction as the gradients say: central differences of the 64-bit formula
    at two steps, the larger one's distance from the smaller one bounding their own error (it is four times it)."""
    rows, cols, rho, eps = 24, 200, 0.5, 1e-6
    a, x, dy, dh = (randn((rows, cols), 41 + i) for i in range(4))
    wp, w, g = randn(cols, 45), randn(cols, 46), randn((4, cols), 47)
    o = sg.sandwich_norm_fp8(a, x, wp, w, gate=g, residual_scale=rho, eps=eps, training=True)
    got = sg.sandwich_norm_backward(dy, a, o.h, wp, w, o.post_rstd, o.rstd, gate=g, residual_scale=rho, dh=dh)

    def value(a, x, wp, w, g):
        _, h, _, _, _, y, _ = forward_bounds(a, x, wp, w, g, rho, eps)
        return (y * dy.double()).sum() + (h * dh.double()).sum()
    at = [v.double() for v in (a, x, wp, w, g)]
    bounds = gradient_bounds(dy, dh, a.double(), o.h.double(), wp, w, g, o.post_rstd, o.rstd, rho)
    for i, name in enumerate(("da", "dx", "dpost_weight", "dweight", "dgate")):
        for seed in range(3):
            d = randn(at[i].shape, 50 + seed).double()
            slope = []
            for step in (1e-4, 2e-4):
                ends = [value(*at[:i], at[i] + e * d, *at[i + 1:]) for e in (step, -step)]
                slope.append((ends[0] - ends[1]) / (2 * step))
            along = (getattr(got, name).double() * d).sum()
            # the gradient's own bound; tp, t and h rounded to FP32 add as much again
            lim = 2 * (bounds[name][1] * d.abs()).sum() + 2 * SUM * (bounds[name][0] * d).abs().sum()
            assert (along - slope[0]).abs() <= lim + (slope[1] - slope[0]).abs(), name


@gpu
def test_norms_of_empty_and_special_rows(sg):  # noqa: F811
    """Padding (rows of zeros) stays finite; a row with a NaN or an infinity reaches itself and the sums only."""
    rows, cols = 260, 1000
    a, x, dy, dh = (randn((rows, cols), 61 + i, torch.bfloat16) for i in range(4))
    for v in (a, x, dy, dh):
        v[7:9] = 0
    wp, w, g = randn(cols, 65), randn(cols, 66), randn(cols, 67)
    o = sg.sandwich_norm_fp8(a, x, wp, w, gate=g, training=True, checkpoint=E4M3)
    for v in (o.h, o.q, o.a8[0], o.h8[0]):
        assert (v[7:9].float() == 0).all()
    assert (o.scale[7:9] == 2.0 ** -126).all() and torch.isfinite(o.rstd).all()
    clean = sg.sandwich_norm_backward(dy, a, o.h, wp, w, o.post_rstd, o.rstd, gate=g, dh=dh)
    assert all(torch.isfinite(v).all() for v in clean) and (clean.da[7:9] == 0).all() and (clean.dx[7:9] == 0).all()
    rest = torch.arange(rows, device="cuda") != 100
    for bad in (float("nan"), float("inf"), -float("inf")):
        for which in (0, 1):
            b = [a.clone(), x.clone()]
            b[which][100, 333] = bad
            p = sg.sandwich_norm_fp8(*b, wp, w, gate=g, training=True, checkpoint=E4M3)
            assert not torch.isfinite(p.scale[100, 2]) and not torch.isfinite(p.h[100, 333].float())
            assert not torch.isfinite(p.h8[1][100, 2])
            for got, want in zip((*p[:5], *p.a8, *p.h8), (*o[:5], *o.a8, *o.h8)):
                assert same_rows(got, want, rest)
            d = dy.clone()
            d[100, 333] = bad
            q = sg.sandwich_norm_backward(d, a, o.h, wp, w, o.post_rstd, o.rstd, gate=g, dh=dh)
            assert not torch.isfinite(q.da[100].float()).any() and not torch.isfinite(q.dweight[333])
            assert same_rows(q.da, clean.da, rest) and same_rows(q.dx, clean.dx, rest)
    one = torch.arange(cols, device="cuda") != 333
    assert same(q.dweight[one], clean.dweight[one])


@gpu
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 8), (1, 1), (0, 5)])
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("cols", [141, 1000, 8264])
def test_norms_strides(sg, pad, offset, dtype, cols):  # noqa: F811
    """Any row stride and base, with NaN beyond every row's end."""
    rows = 30
    a, x, dy, dh = (randn((rows, cols), 71 + i, dtype) for i in range(4))
    wp, w, g = randn(cols, 75), randn(cols, 76), randn((3, cols), 77, dtype)
    odd = lambda v: strided(v[None] if v.dim() == 1 else v, pad, offset).view(v.shape) if v.dim() == 1 else strided(v, pad, offset)  # noqa: E731
    up = [strided(v, -cols % 16) for v in (a, x, dy, dh, g)]
    want = sg.sandwich_norm_fp8(up[0], up[1], wp, w, gate=up[4], training=True, checkpoint=E4M3)
    got = sg.sandwich_norm_fp8(odd(a), odd(x), odd(wp), odd(w), gate=odd(g), training=True, checkpoint=E4M3)
    for p, q in zip((*got[:5], *got.a8, *got.h8), (*want[:5], *want.a8, *want.h8)):
        assert same(p, q)
    for kept in (False, True):
        A, H = (want.a8, want.h8) if kept else (up[0], want.h)
        oddly = lambda k: tuple(odd(v) for v in k) if kept else odd(k)   # noqa: E731
        first = sg.sandwich_norm_backward(up[2], A, H, wp, w, want.post_rstd, want.rstd, gate=up[4], dh=up[3])
        again = sg.sandwich_norm_backward(odd(dy), oddly(A), oddly(H), odd(wp), odd(w), want.post_rstd, want.rstd,
                                          gate=odd(g), dh=odd(dh))
        for p, q in zip(again, first):
            assert same(p, q)


@gpu
def test_norms_write_their_outputs_only(sg):  # noqa: F811
    """Outputs with odd row strides through the C entry: what lies between their rows is left as it was."""
    rows, cols, kb = 9, 301, 3
    a, x = randn((rows, cols), 81), randn((rows, cols), 82)
    wp, w = randn(cols, 83), randn(cols, 84)
    want = sg.sandwich_norm_fp8(a, x, wp, w, training=True, checkpoint=E4M3)
    f = lambda n: torch.full((rows, n + 3), -5.0, device="cuda")     # noqa: E731
    b = lambda n: torch.full((rows, n + 3), 0x55, dtype=torch.uint8, device="cuda")   # noqa: E731
    h, s, sa, sh, q, qa, qh = f(cols), f(kb), f(kb), f(kb), b(cols), b(cols), b(cols)
    sg.sgemm_sandwich_norm_fp8(rows, cols, 1e-6, 1.0, a.data_ptr(), cols, x.data_ptr(), cols, 0, wp.data_ptr(), w.data_ptr(),
                               0, None, 0, 0, 0, h.data_ptr(), cols + 3, q.data_ptr(), 8, cols + 3, s.data_ptr(), kb + 3,
                               None, None, qa.data_ptr(), cols + 3, sa.data_ptr(), kb + 3, qh.data_ptr(), cols + 3,
                               sh.data_ptr(), kb + 3, 8, torch.cuda.current_stream().cuda_stream)
    for got, ref, left in ((h, want.h, -5), (s, want.scale, -5), (sa, want.a8[1], -5), (sh, want.h8[1], -5),
                           (q, want.q, 0x55), (qa, want.a8[0], 0x55), (qh, want.h8[0], 0x55)):
        n = ref.shape[1]
        assert torch.equal(got[:, :n], ref.view(got.dtype)) and (got[:, n:] == left).all()
    for k in range(2):   # one of the checkpoints and of the statistics alone
        q1, s1, t1 = b(cols), f(kb), f(rows)[0]
        one = [(q1.data_ptr(), cols + 3, s1.data_ptr(), kb + 3), (None, 0, None, 0)]
        stat = [t1.data_ptr(), None]
        sg.sgemm_sandwich_norm_fp8(rows, cols, 1e-6, 1.0, a.data_ptr(), cols, x.data_ptr(), cols, 0, wp.data_ptr(),
                                   w.data_ptr(), 0, None, 0, 0, 0, h.data_ptr(), cols + 3, q.data_ptr(), 8, cols + 3,
                                   s.data_ptr(), kb + 3, stat[k], stat[1 - k], *one[k], *one[1 - k], 8,
                                   torch.cuda.current_stream().cuda_stream)
        ref8, reft = (want.a8, want.post_rstd) if k == 0 else (want.h8, want.rstd)
        assert torch.equal(q1[:, :cols], ref8[0].view(torch.uint8)) and torch.equal(s1[:, :kb], ref8[1])
        assert torch.equal(t1[:rows], reft) and (t1[rows:] == -5).all() and (q1[:, cols:] == 0x55).all()
        assert torch.equal(h[:, :cols], want.h) and torch.equal(q[:, :cols], want.q.view(torch.uint8))
    dy = randn((rows, cols), 85)
    ref = sg.sandwich_norm_backward(dy, a, x, wp, w, want.post_rstd, want.rstd)
    da, dx = f(cols), f(cols)
    need = sg.sgemm_sandwich_norm_backward_workspace(rows, cols)
    ws = torch.full((need // 4 + 1,), 7.0, device="cuda")
    sg.sgemm_sandwich_norm_backward(rows, cols, 1.0, dy.data_ptr(), cols, None, 0, 0, a.data_ptr(), 0, cols, None, 0,
                                    x.data_ptr(), 0, cols, None, 0, wp.data_ptr(), w.data_ptr(), 0, None, 0, 0, 0,
                                    want.post_rstd.data_ptr(), want.rstd.data_ptr(), da.data_ptr(), cols + 3, dx.data_ptr(),
                                    cols + 3, None, None, None, 0, None, 0, torch.cuda.current_stream().cuda_stream)
    for got, w_ in ((da, ref.da), (dx, ref.dx)):
        assert torch.equal(got[:, :cols], w_) and (got[:, cols:] == -5).all()
    for k in range(2):   # one of the sums alone
        out = torch.full((cols + 1,), -5.0, device="cuda")
        sg.sgemm_sandwich_norm_backward(rows, cols, 1.0, dy.data_ptr(), cols, None, 0, 0, a.data_ptr(), 0, cols, None, 0,
                                        x.data_ptr(), 0, cols, None, 0, wp.data_ptr(), w.data_ptr(), 0, None, 0, 0, 0,
                                        want.post_rstd.data_ptr(), want.rstd.data_ptr(), da.data_ptr(), cols + 3,
                                        dx.data_ptr(), cols + 3, *((out.data_ptr(), None) if k else (None, out.data_ptr())),
                                        None, 0, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert torch.equal(out[:cols], (ref.dpost_weight if k else ref.dweight)) and out[cols] == -5 and ws[-1] == 7


# ---------------------------------------------------------------- the gated unit
def unit_bounds(g, u):
    """p, y and dy's factors of g and u in 64 bits with what the kernel's may be off by."""
    p = torch.sigmoid(g)
    m = torch.sigmoid(-g)                                   # 1 - p
    Ep = p * U * (2 * m * (2 + 1.173 * g.abs()) + 6) + torch.where(g < -87, 2.0 ** -125, 0.0)
    y = g * p * u
    Ey = (g * u).abs() * Ep + 3 * U * y.abs()
    fu = g * p                                              # of du
    Eu = g.abs() * Ep + U * fu.abs()
    slope = p + fu * m                                      # of silu
    Es = Ep + Eu * m + fu.abs() * (Ep + U) + 4 * U * (p + fu.abs() * m)
    return y, Ey, fu, Eu, slope, Es


UNIT_SHAPES = [(1, 1), (1, 128), (7, 5), (128, 128), (129, 127), (1, 4096), (300, 1000), (257, 129), (1000, 1013)]


@gpu
@pytest.mark.parametrize("shape", UNIT_SHAPES)
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("to", [E4M3, E5M2])
def test_unit(sg, shape, dtype, to):  # noqa: F811
    g, u = randn(shape, 101, dtype, 3.0), randn(shape, 102, dtype)
    o = sg.swiglu_fp8(g, u, dtype=to, checkpoint=E4M3)
    y, Ey, *_ = unit_bounds(g.double(), u.double())
    close_quantised(o.q, o.scale, y, Ey, 1, B)
    for k, v in ((o.gate8, g), (o.up8, u)):
        for got, want in zip(k, sg.quantize_fp8(v)):
            assert same(got, want)
    bare = sg.swiglu_fp8(g, u, dtype=to)
    assert bare.gate8 is bare.up8 is None and same(bare.q, o.q) and same(bare.scale, o.scale)


def halves(o, cols):
    """dgate and dup of [dgate | dup] both ways, after a look at what lies between."""
    wide = o.q_rows.shape[1] // 2
    assert wide == cdiv(cols, B) * B
    for q in (o.q_rows, o.q_cols):
        pad = q.view(torch.uint8).view(len(q), 2, wide)[:, :, cols:]
        assert (pad == 0).all()
    parts = []
    for at in (0, wide):
        own = slice(at, at + cols)
        parts.append((o.q_rows[:, own], o.scale_rows[:, at // B:(at + wide) // B], o.q_cols[:, own], o.scale_cols[:, own]))
    return parts


@gpu
@pytest.mark.parametrize("shape", UNIT_SHAPES)
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("keep", [None, E4M3, E5M2])
def test_unit_gradient(sg, shape, dtype, keep):  # noqa: F811
    rows, cols = shape
    g, u, dy = randn(shape, 111, dtype, 3.0), randn(shape, 112, dtype), randn(shape, 113, dtype, 0.01)
    G, U_ = (g, u) if keep is None else (sg.quantize_fp8(g, dtype=keep), sg.quantize_fp8(u, dtype=keep))
    vg, vu = (v.double() if keep is None else v[0].double() * spread(v[1], 1, B, rows, cols) for v in (G, U_))
    if keep is not None:   # q * scale is rounded to FP32
        vg, vu = vg.float().double(), vu.float().double()
    o = sg.swiglu_backward_fp8(dy, G, U_, dtype=E4M3 if keep == E4M3 else E5M2, y_dtype=E5M2 if keep == E5M2 else E4M3)
    y, Ey, fu, Eu, slope, Es = unit_bounds(vg, vu)
    d = dy.double()
    want = ((d * vu * slope, (d * vu).abs() * (Es + 3 * U * slope.abs())), (d * fu, d.abs() * (Eu + U * fu.abs())))
    for (qr, sr, qc, sc), (value, E) in zip(halves(o, cols), want):
        close_quantised(qr, sr, value, E, 1, B)
        close_quantised(qc, sc, value, E, B, 1)
    close_quantised(o.y_cols, o.y_scale, y, Ey, B, 1)


@gpu
def test_unit_gradient_against_differences(sg):  # noqa: F811
    """The gradient's values (128 x 1 blocks of one row: q is F, and q * scale the FP32 value) against central differences
    of the 64-bit formula; the logistic function's error, up to 30 u here, is within 1e-5."""
    g, u = torch.linspace(-12, 12, 257, device="cuda")[None], randn((1, 257), 121)
    o = sg.swiglu_backward_fp8(torch.ones_like(g), g, u, dtype=E4M3)
    G, V = g.double(), u.double()
    f = lambda g, u: g / (1 + (-g).exp()) * u   # noqa: E731
    for (_, _, qc, sc), slope in zip(halves(o, 257), ((f(G + 1e-5, V) - f(G - 1e-5, V)) / 2e-5, f(G, torch.ones_like(V)))):
        got = qc.double() * sc.double()
        assert ((got - slope).abs() <= slope.abs() * 1e-5 + 1e-8).all()


@gpu
def test_unit_special_values(sg):  # noqa: F811
    """Large gates saturate without NaN, zeros stay zeros, a NaN or an infinity reaches its own blocks only."""
    g, u, dy = randn((256, 256), 131), randn((256, 256), 132), randn((256, 256), 133)
    g[0, :8] = torch.tensor([88.0, -88.0, 200.0, -200.0, 1e4, -1e4, 1e30, -1e30], device="cuda")
    g[40:42] = 0
    u[50:52] = 0
    o, d = sg.swiglu_fp8(g, u), sg.swiglu_backward_fp8(dy, g, u)
    assert torch.isfinite(o.scale).all() and torch.isfinite(o.q.float()).all()
    assert all(torch.isfinite(v.float()).all() for v in d)
    y, Ey, *_ = unit_bounds(g.double(), u.double())
    close_quantised(o.q, o.scale, y, Ey, 1, B)
    assert (o.q[40:42].float() == 0).all() and (o.q[50:52].float() == 0).all() and (o.scale[40:42] == 2.0 ** -126).all()
    for bad in (float("nan"), float("inf")):
        h = u.clone()
        h[3, 5] = bad
        p = sg.swiglu_fp8(g, h, checkpoint=E4M3)
        assert not torch.isfinite(p.scale[3, 0]) and not torch.isfinite(p.up8[1][3, 0])
        keep = torch.isfinite(p.scale)
        assert (~keep).sum() == 1 and torch.equal(p.scale[keep], o.scale[keep])
        e = sg.swiglu_backward_fp8(dy, g, h)
        assert not torch.isfinite(e.scale_rows[3, 0]) and not torch.isfinite(e.scale_cols[0, 5])
        assert not torch.isfinite(e.y_scale[0, 5])
        assert (~torch.isfinite(e.scale_rows)).sum() == (~torch.isfinite(e.scale_cols)).sum() == 1
        # a kept block that holds one stands for nothing finite, and reaches every column of its row's block
        k = sg.swiglu_backward_fp8(dy, p.gate8, p.up8)
        assert not torch.isfinite(k.scale_rows[3, 0]) and (~torch.isfinite(k.scale_rows)).sum() == 1
        assert not torch.isfinite(k.y_scale[0, :B]).any() and torch.isfinite(k.y_scale[0, B:]).all()


@gpu
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 8), (1, 1), (0, 5)])
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("cols", [141, 256])
def test_unit_strides(sg, pad, offset, dtype, cols):  # noqa: F811
    g, u, dy = (randn((130, cols), 141 + i, dtype) for i in range(3))
    odd = lambda v: strided(v, pad, offset)   # noqa: E731
    up = [strided(v, -cols % 16) for v in (g, u, dy)]
    want, got = sg.swiglu_fp8(up[0], up[1], checkpoint=E4M3), sg.swiglu_fp8(odd(g), odd(u), checkpoint=E4M3)
    for p, q in zip((got.q, got.scale, *got.gate8, *got.up8), (want.q, want.scale, *want.gate8, *want.up8)):
        assert same(p, q)
    for p, q in zip(sg.swiglu_backward_fp8(odd(dy), odd(g), odd(u)), sg.swiglu_backward_fp8(up[2], up[0], up[1])):
        assert same(p, q)
    kept = [tuple(odd(v) for v in k) for k in (want.gate8, want.up8)]
    for p, q in zip(sg.swiglu_backward_fp8(odd(dy), *kept), sg.swiglu_backward_fp8(up[2], want.gate8, want.up8)):
        assert same(p, q)
    # the halves of one product's output
    z = torch.cat([g, u], 1)
    for p, q in zip(sg.swiglu_fp8(z[:, :cols], z[:, cols:])[:2], want[:2]):
        assert same(p, q)


@gpu
def test_unit_writes_its_outputs_only(sg):  # noqa: F811
    rows, cols, kb = 131, 301, 3
    wide = 2 * kb * B
    g, u, dy = (randn((rows, cols), 151 + i) for i in range(3))
    stream = torch.cuda.current_stream().cuda_stream
    f = lambda r, n: torch.full((r, n + 3), -5.0, device="cuda")     # noqa: E731
    b = lambda n: torch.full((rows, n + 3), 0x55, dtype=torch.uint8, device="cuda")   # noqa: E731
    want = sg.swiglu_fp8(g, u, checkpoint=E4M3)
    q, qg, qu, s, s_g, su = b(cols), b(cols), b(cols), f(rows, kb), f(rows, kb), f(rows, kb)
    sg.sgemm_swiglu_fp8(rows, cols, g.data_ptr(), cols, u.data_ptr(), cols, 0, q.data_ptr(), 8, cols + 3, s.data_ptr(),
                        kb + 3, qg.data_ptr(), cols + 3, s_g.data_ptr(), kb + 3, qu.data_ptr(), cols + 3, su.data_ptr(),
                        kb + 3, 8, stream)
    for k in range(2):   # one of the checkpoints alone
        q1, s1 = b(cols), f(rows, kb)
        one = [(q1.data_ptr(), cols + 3, s1.data_ptr(), kb + 3), (None, 0, None, 0)]
        sg.sgemm_swiglu_fp8(rows, cols, g.data_ptr(), cols, u.data_ptr(), cols, 0, q.data_ptr(), 8, cols + 3, s.data_ptr(),
                            kb + 3, *one[k], *one[1 - k], 8, stream)
        ref8 = (want.gate8, want.up8)[k]
        assert torch.equal(q1[:, :cols], ref8[0].view(torch.uint8)) and torch.equal(s1[:, :kb], ref8[1])
    d = sg.swiglu_backward_fp8(dy, g, u, dtype=E5M2)
    qr, qc, qy, sr, sc, sy = b(wide), b(wide), b(cols), f(rows, 2 * kb), f(2, wide), f(2, cols)
    sg.sgemm_swiglu_backward_fp8(rows, cols, dy.data_ptr(), cols, 0, g.data_ptr(), 0, cols, None, 0, u.data_ptr(), 0, cols,
                                 None, 0, 9, qr.data_ptr(), wide + 3, sr.data_ptr(), 2 * kb + 3, qc.data_ptr(), wide + 3,
                                 sc.data_ptr(), wide + 3, 8, qy.data_ptr(), cols + 3, sy.data_ptr(), cols + 3, stream)
    for got, ref in ((q, want.q), (qg, want.gate8[0]), (qu, want.up8[0]), (s, want.scale), (s_g, want.gate8[1]),
                     (su, want.up8[1]), (qr, d.q_rows), (qc, d.q_cols), (qy, d.y_cols), (sr, d.scale_rows),
                     (sc, d.scale_cols), (sy, d.y_scale)):
        n = ref.shape[1]
        left = 0x55 if got.dtype == torch.uint8 else -5
        assert torch.equal(got[:, :n], ref.view(got.dtype)) and (got[:, n:] == left).all()


@gpu
@pytest.mark.parametrize("dtype,first", [(E4M3, 2.0 ** 0), (E5M2, 2.0 ** 0), (E4M3, 2.0 ** -118), (E5M2, 2.0 ** -111), (E4M3, 2.0 ** 127)])
def test_scales_are_the_quotients_for_every_significand(sg, dtype, first):  # noqa: F811
    """A block's scale is max|x| / F rounded to FP32, although it is not divided: all 2^23 significands of a binade, those
    next to the least scale and of the largest numbers among them."""
    x = (torch.arange(1 << 23, device="cuda", dtype=torch.int32) + torch.tensor(first).view(torch.int32).item()).view(torch.float32)
    o = sg.swiglu_fp8(x[:, None], torch.zeros_like(x)[:, None], dtype=dtype, checkpoint=dtype)
    want = (x.double() / FMAX[dtype]).float().clamp_min(2.0 ** -126)
    assert torch.equal(o.gate8[1][:, 0], want)
    q = sg.quantize_fp8(x[:, None], dtype=dtype)
    assert same(o.gate8[0], q[0]) and same(o.gate8[1], q[1])


# ---------------------------------------------------------------- kept rows as a weight gradient's operand
@gpu
@pytest.mark.parametrize("shape", UNIT_SHAPES)
@pytest.mark.parametrize("kind", [E4M3, E5M2])
@pytest.mark.parametrize("to", [None, E4M3, E5M2])
def test_requantise(sg, shape, kind, to):  # noqa: F811
    """Bit for bit what the quantiser makes of q * scale in FP32."""
    x = randn(shape, 161) * torch.exp(3 * randn((shape[0], 1), 162))
    q, s = sg.quantize_fp8(x, dtype=kind)
    value = q.float() * spread(s, 1, B, *shape).float()
    want = sg.quantize_fp8(value, (B, 1), to or kind)
    for got, w in zip(sg.requantize_fp8(q, s, dtype=to), want):
        assert same(got, w)
    for pad, offset in ((3, 0), (8, 8), (1, 1)):
        for got, w in zip(sg.requantize_fp8(strided(q, pad, offset), strided(s, pad), dtype=to), want):
            assert same(got, w)


@gpu
def test_requantise_special_values(sg):  # noqa: F811
    x = randn((256, 256), 163)
    x[:128, 128:] = 0
    x[130] = 0
    q, s = sg.quantize_fp8(x)
    want = sg.requantize_fp8(q, s)
    assert (want[0][:128, 128:].float() == 0).all() and (want[1][0, 128:] == 2.0 ** -126).all()
    for bad in (float("nan"), float("inf")):
        t = s.clone()
        t[200, 1] = bad
        got = sg.requantize_fp8(q, t)
        assert not torch.isfinite(got[1][1, 128:]).any()
        assert same(got[1][0], want[1][0]) and same(got[1][1, :128], want[1][1, :128])
        assert same(got[0][:, :128], want[0][:, :128]) and same(got[0][:128], want[0][:128])


# ---------------------------------------------------------------- offsets, streams, graphs
@gpu
def test_offsets_beyond_32_bits(sg):  # noqa: F811
    rows, cols, ld = 70000, 136, 32768
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)
    a, x, y = buf[:, :cols], buf[:, 1024:1024 + cols], buf[:, 2048:2048 + cols]
    for i, v in enumerate((a, x, y)):
        v.copy_(randn((rows, cols), 171 + i))
    near = [v.contiguous() for v in (a, x, y)]
    w = randn(cols, 175)
    for p, q in zip(sg.sandwich_norm_fp8(a, x, w, w, gate=y), sg.sandwich_norm_fp8(near[0], near[1], w, w, gate=near[2])):
        assert p is q is None or same(p, q)
    t = randn(rows, 176).abs()
    for p, q in zip(sg.sandwich_norm_backward(y, a, x, w, w, t, t), sg.sandwich_norm_backward(near[2], near[0], near[1], w, w, t, t)):
        assert p is q is None or same(p, q)
    for p, q in zip(sg.swiglu_fp8(a, x)[:2], sg.swiglu_fp8(near[0], near[1])[:2]):
        assert same(p, q)
    for p, q in zip(sg.swiglu_backward_fp8(y, a, x), sg.swiglu_backward_fp8(near[2], near[0], near[1])):
        assert same(p, q)
    far = torch.empty(rows * ld, dtype=torch.uint8, device="cuda").view(rows, ld)[:, :cols].view(E4M3)
    q, s = sg.quantize_fp8(near[0])
    far.view(torch.uint8).copy_(q.view(torch.uint8))
    for got, want in zip(sg.requantize_fp8(far, s), sg.requantize_fp8(q, s)):
        assert same(got, want)


class Block:
    """A gated block with sandwich norms, trained in 8 bits: down(silu(gate n) * (up n)), n the normalised stream."""

    def __init__(self, sg, width=256, inner=384):  # noqa: F811
        self.sg, self.inner = sg, inner
        self.w_in, self.wp, self.w = (1 + randn(width, 180 + i, scale=0.1) for i in range(3))
        self.gate = randn(width, 183, scale=0.3)
        self.W1, self.W2 = randn((2 * inner, width), 184, scale=width ** -0.5), randn((width, inner), 185, scale=inner ** -0.5)
        self.q1, self.q2 = (sg.quantize_fp8(W, (B, B)) for W in (self.W1, self.W2))

    def forward(self, x, **kw):
        sg = self.sg  # noqa: F811
        n = sg.rms_norm_fp8(x, self.w_in, training=True, **kw)
        z = sg.gemm_fp8(n.q, n.scale, *self.q1, transB=True, **kw)
        u = sg.swiglu_fp8(z[:, :self.inner], z[:, self.inner:], checkpoint=E4M3, **kw)
        a = sg.gemm_fp8(u.q, u.scale, *self.q2, transB=True, **kw)
        o = sg.sandwich_norm_fp8(a, x, self.wp, self.w, gate=self.gate, training=True, checkpoint=E4M3, **kw)
        return o, (n, u, x)

    def backward(self, dy, dh, o, kept, **kw):
        sg, (n, u, x) = self.sg, kept  # noqa: F811
        d = sg.sandwich_norm_backward(dy, o.a8, o.h8, self.wp, self.w, o.post_rstd, o.rstd, gate=self.gate, dh=dh, **kw)
        ar, as_, ac, acs = sg.quantize_fp8_both(d.da, **kw)
        du = sg.gemm_fp8(ar, as_, *self.q2, **kw)
        z = sg.swiglu_backward_fp8(du, u.gate8, u.up8, **kw)
        f32 = torch.float32
        dW2 = sg.gemm_fp8(ac, acs, z.y_cols, z.y_scale, transA=True, out_dtype=f32, **kw)
        dn = sg.gemm_fp8(z.q_rows, z.scale_rows, *self.q1, **kw)
        nq, ns = sg.requantize_fp8(n.q, n.scale, **kw)
        dW1 = sg.gemm_fp8(z.q_cols, z.scale_cols, nq, ns, transA=True, out_dtype=f32, **kw)
        dx, dw_in = sg.rms_norm_backward(dn, x, self.w_in, n.rstd, dh=d.dx, **kw)
        return dx, dw_in, dW1, dW2, d.dpost_weight, d.dweight, d.dgate

    def step(self, x, dy, dh, **kw):
        o, kept = self.forward(x, **kw)
        return (o.q, o.scale, o.h, *self.backward(dy, dh, o, kept, **kw))


def block_inputs(rows=300, width=256):
    return [randn((rows, width), 190 + i, torch.bfloat16) for i in range(3)]


@gpu
def test_a_block_trained_in_8_bits(sg, clean_status):  # noqa: F811
    """The whole block, forward and backward, against 64-bit autograd of the same block.  What differs is what is held in
    8 bits.  An E4M3 rounding is off by half a step, at most 2^-4 of the value and 2^-5.2 = 0.027 in the root mean square
    (the step over the value falls from 2^-3 to 2^-4 along a binade: 2^-3.6 / sqrt(12)); on the way to a gradient lie at
    most 13 such roundings one after the other (n, W1, y, W2, a, h, da, W2, gate, up, dz, W1, n), independent of each
    other: sqrt(13) 0.027 = 0.1, and twice that for factors above one on the way."""
    x, dy, dh = block_inputs()
    b = Block(sg)
    o, kept = b.forward(x)
    got = (o.h, *b.backward(dy, dh, o, kept))
    leaf = [v.double().requires_grad_() for v in (x, b.w_in, b.W1, b.W2, b.wp, b.w, b.gate)]
    X, w_in, W1, W2, wp, w, gate = leaf
    norm = lambda v: v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt()   # noqa: E731
    z = (norm(X) * w_in) @ W1.t()
    a = (torch.nn.functional.silu(z[:, :b.inner]) * z[:, b.inner:]) @ W2.t()
    h = X + gate * (norm(a) * wp)
    y = norm(h) * w
    ((y * dy.double()).sum() + (h * dh.double()).sum()).backward()
    for name, p, q in zip(("h", "dx", "dw_in", "dW1", "dW2", "dwp", "dw", "dgate"), got, (h.detach(), *(v.grad for v in leaf))):
        assert torch.isfinite(p).all() and (p.double() - q).norm() <= 0.2 * q.norm(), name


@gpu
def test_block_on_another_stream_and_in_graphs(sg):  # noqa: F811
    """The same bits on another stream, captured and replayed, and by two graphs in turn."""
    b = Block(sg)
    x, dy, dh = block_inputs()
    want = b.step(x, dy, dh)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(2):
        got = b.step(x, dy, dh, stream=s)
        s.synchronize()
        assert all(same(p, q) for p, q in zip(got, want))
    other = block_inputs(500)
    want2 = b.step(*other)
    with torch.cuda.stream(s):
        b.step(*other)
    s.synchronize()
    graphs = []
    for inputs in ((x, dy, dh), other):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = b.step(*inputs)
        graphs.append((graph, out))
    for _ in range(2):
        for (graph, out), ref in zip(graphs, (want, want2)):
            for v in out:
                v.view(torch.uint8).fill_(0) if v.dtype in FMAX else v.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(same(p, q) for p, q in zip(out, ref))


@gpu
@pytest.mark.parametrize("rows,cols", [(40, 3000), (700, 8192), (9, 16384), (3, 16400)])
def test_rows_over_clusters_in_graphs_and_side_by_side(sg, rows, cols):  # noqa: F811
    """The gradient of long rows: captured and replayed, on two streams at once, and again and again, the same bits."""
    a, x, dy, dh = (randn((rows, cols), 191 + i, torch.bfloat16) for i in range(4))
    wp, w, g = randn(cols, 195), randn(cols, 196), randn(cols, 197)
    o = sg.sandwich_norm_fp8(a, x, wp, w, gate=g, training=True, checkpoint=E4M3)

    def call(**kw):
        return sg.sandwich_norm_backward(dy, o.a8, o.h8, wp, w, o.post_rstd, o.rstd, gate=g, dh=dh, **kw)
    want = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [call(stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(same(p, q) for r in got for p, q in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [call() for _ in range(3)]
    for _ in range(2):
        for v in outs[-1]:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(p, q) for r in outs for p, q in zip(r, want))
    assert sg.sgemm_last_device_status() == 0


@gpu
def test_no_device_memory_of_the_librarys_own(sg):  # noqa: F811
    old, _ = sg.sgemm_get_scratch_limit()
    try:
        sg.sgemm_set_scratch_limit(0)
        Block(sg).step(*block_inputs())
        assert sg.sgemm_get_scratch_limit()[1] == 0
    finally:
        sg.sgemm_set_scratch_limit(old)


@gpu
@pytest.mark.parametrize("rows,cols", [(0, 7), (5, 0), (0, 0)])
def test_empty_matrices(sg, rows, cols):  # noqa: F811
    a, w, t = (torch.ones(s, device="cuda") for s in ((rows, cols), (cols,), (rows,)))
    o = sg.sandwich_norm_fp8(a, a, w, w, gate=w, training=True, checkpoint=E4M3)
    assert o.q.shape == o.h.shape == (rows, cols) and o.scale.shape == (rows, cdiv(cols, B)) and o.rstd.shape == (rows,)
    d = sg.sandwich_norm_backward(a, o.a8, o.h8, w, w, t, t, gate=w, dh=a)
    assert d.da.shape == (rows, cols) and all((v == 0).all() and v.shape == (cols,) for v in d[2:])
    d = sg.sandwich_norm_backward(a, a, a, w, w, t, t, gate=a)
    assert d.dgate.shape == (rows, cols)
    o = sg.swiglu_fp8(a, a, checkpoint=E4M3)
    d = sg.swiglu_backward_fp8(a, o.gate8, o.up8)
    assert d.q_rows.shape == (rows, 2 * B * cdiv(cols, B)) and d.y_scale.shape == (cdiv(rows, B), cols)
    q, s = sg.requantize_fp8(o.q, o.scale)
    assert q.shape == (rows, cols) and s.shape == (cdiv(rows, B), cols)


# ---------------------------------------------------------------- the extension module
def test_extension_leaves_the_unusual_to_python(lib):
    from dense_fp32_matrix_10_gb300 import fp8
    e, x = fp8._usual, torch.zeros(4, 8)
    w, t = x[0], x[:, 0]
    assert e.sandwich_norm(x, x, w, w, None, 1.0, 1e-6, 8, True, 8) is None                   # not on a GPU
    assert e.sandwich_norm_backward(x, (x, x), x, w, w, t, t, w, 1.0, None) is None
    assert e.swiglu(x, x, 8, -1) is None and e.swiglu_backward(x, x, x, 8, 8) is None and e.requantize(x, x, 8) is None
    assert e.sandwich_norm(None, None, w, w, 3, "1", 1e-6, 8, True, 8) is None                # not tensors
    assert e.swiglu(x, x) is None and e.swiglu_backward(x, (x,), x, 8, 8) is None              # arguments missing


@gpu
@pytest.mark.parametrize("cols", [1, 15, 333, 1024])
def test_rows_made_for_a_caller_are_aligned(sg, cols):  # noqa: F811
    """Any number of columns: the next call's vectors fit the rows that this one made."""
    a, x, dy = (randn((6, cols), 231 + i, torch.bfloat16) for i in range(3))
    w, g = randn(cols, 234), randn((3, cols), 235, torch.bfloat16)
    o = sg.sandwich_norm_fp8(a, x, w, w, gate=g, training=True, checkpoint=E4M3)
    d = sg.sandwich_norm_backward(dy, a, o.h, w, w, o.post_rstd, o.rstd, gate=g)
    for v in (o.h, d.da, d.dx, d.dgate, o.q, o.a8[0], o.h8[0]):
        assert v.stride() == (-(-cols // 16) * 16, 1) and v.data_ptr() % 32 == 0


@gpu
def test_kept_tensors_hold_no_others(sg):  # noqa: F811
    """Beyond a megabyte, what outlives the next product does not share its operand's memory."""
    a, x, dy = (randn((1024, 1030), 241 + i, torch.bfloat16) for i in range(3))
    w = randn(1030, 244)
    o = sg.sandwich_norm_fp8(a, x, w, w, training=True, checkpoint=E4M3)
    u = sg.swiglu_fp8(a, x, checkpoint=E4M3)
    d = sg.sandwich_norm_backward(dy, o.a8, o.h8, w, w, o.post_rstd, o.rstd)
    place = lambda t: t.untyped_storage().data_ptr()   # noqa: E731
    assert len({place(o.q), place(o.h), place(o.h8[0])}) == 3
    assert place(o.h8[0]) == place(o.a8[0]) == place(o.rstd)
    assert place(u.q) != place(u.gate8[0])
    assert len({place(d.da), place(d.dx), place(d.dweight)}) == 3
    assert d.dweight.untyped_storage().nbytes() <= 4 * 4 * 1280   # (no workspace)


@gpu
@pytest.mark.parametrize("shape", [(1, 128), (5, 0), (0, 7), (70, 333), (258, 1024)])
def test_both_ways_through_python(sg, monkeypatch, shape):  # noqa: F811
    """The extension module and the general code hand over the same calls."""
    from dense_fp32_matrix_10_gb300 import fp8
    rows, cols = shape
    a, x, dy, dh = (randn(shape, 201 + i, torch.bfloat16) for i in range(4))
    w, g, t = randn(cols, 205), randn((2, cols), 206, torch.bfloat16), randn(rows, 207).abs()
    g = g if rows % 2 == 0 and rows else g[0]

    def everything():
        o = sg.sandwich_norm_fp8(a, x, w, w, gate=g, residual_scale=0.5, training=True, checkpoint=E5M2)
        u = sg.swiglu_fp8(a, x, dtype=E5M2, checkpoint=E4M3)
        out = [o.q, o.scale, o.h, *o.a8, *o.h8, u.q, u.scale, *u.gate8, *u.up8]
        out += [o.post_rstd, o.rstd] if cols else []   # (rows of no elements have none)
        out += sg.sandwich_norm_fp8(a, x, w, w)[:3]
        out += sg.sandwich_norm_backward(dy, o.a8, o.h, w, w, t, t, gate=g, residual_scale=0.5, dh=dh)
        out += sg.sandwich_norm_backward(dy, a, o.h8, w, w, t, t)[:4]
        out += [*sg.swiglu_backward_fp8(dy, u.gate8, u.up8), *sg.swiglu_backward_fp8(dy, a, x, E5M2, E5M2)]
        out += [*sg.requantize_fp8(u.q, u.scale), *sg.requantize_fp8(u.q, u.scale, E4M3)]
        return out

    ours = everything()
    monkeypatch.setattr(fp8, "_usual", None)
    for p, q in zip(ours, everything()):
        assert p.stride() == q.stride() and same(p, q)


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib(sg):  # noqa: F811
    from dense_fp32_matrix_10_gb300 import build, fp8_block
    build.build()
    return fp8_block._library()


AT = [0x100000 * (i + 1) for i in range(20)]   # never dereferenced


def norms_status(lib, rows=8, cols=256, eps=1e-6, A=AT[0], lda=256, X=AT[1], ldx=256, tx=1, WP=AT[2], W=AT[3], tw=1,
                 GATE=None, ldg=256, tg=1, group=1, H=AT[5], ldh=256, Q=AT[6], tq=8, ldq=256, S=AT[7], lds=2, TP=None, T=None,
                 QA=None, ldqa=256, SA=None, ldsa=2, QH=None, ldqh=256, SH=None, ldsh=2, tk=8):
    return lib.sgemm_sandwich_norm_fp8(rows, cols, eps, 1.0, A, lda, X, ldx, tx, WP, W, tw, GATE, ldg, tg, group, H, ldh, Q,
                                       tq, ldq, S, lds, TP, T, QA, ldqa, SA, ldsa, QH, ldqh, SH, ldsh, tk, None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), 1), (dict(cols=1 << 31), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(tx=8), 1),
    (dict(tw=2), 1), (dict(tq=1), 1), (dict(A=None), 1), (dict(X=None), 1), (dict(WP=None), 1), (dict(W=None), 1),
    (dict(H=None), 1), (dict(Q=None), 1), (dict(S=None), 1), (dict(lda=255), 1), (dict(ldx=255), 1), (dict(ldh=255), 1),
    (dict(ldq=255), 1), (dict(lds=1), 1), (dict(GATE=AT[4], tg=2), 1), (dict(GATE=AT[4], group=0), 1),
    (dict(GATE=AT[4], ldg=255), 1), (dict(QA=AT[8]), 1), (dict(SA=AT[8]), 1), (dict(QH=AT[8]), 1), (dict(SH=AT[8]), 1),
    (dict(QA=AT[8], SA=AT[9], tk=1), 1), (dict(QA=AT[8], SA=AT[9], ldsa=1), 1), (dict(QH=AT[8], SH=AT[9], ldqh=255), 1),
    (dict(A=AT[0] + 1), 1), (dict(S=AT[7] + 2), 1), (dict(lda=1 << 41), 1), (dict(H=AT[0]), 2), (dict(H=AT[1] + 512), 2),
    (dict(Q=AT[5]), 2), (dict(S=AT[3]), 2), (dict(TP=AT[7]), 2), (dict(T=AT[0]), 2), (dict(TP=AT[8], T=AT[8]), 2),
    (dict(QA=AT[6], SA=AT[9]), 2), (dict(GATE=AT[5], group=4), 2), (dict(QH=AT[8], SH=AT[8]), 2)])
def test_norms_refuse(lib, change, status):
    assert norms_status(lib, **change) == status


def norms_gradient_status(lib, rows=8, cols=256, DY=AT[0], lddy=256, DH=None, lddh=256, tx=1, A=AT[1], ta=1, lda=256, SA=None,
                          ldsa=2, H=AT[2], th=1, ldh=256, SH=None, ldsh=2, WP=AT[3], W=AT[4], tw=1, GATE=None, ldg=256, tg=1,
                          group=1, TP=AT[5], T=AT[6], DA=AT[7], ldda=256, DX=AT[8], lddx=256, DWP=AT[9], DW=AT[10], DG=None,
                          lddg=256, ws=AT[11], size=None):
    need = lib.sgemm_sandwich_norm_backward_workspace(rows, cols)
    return lib.sgemm_sandwich_norm_backward(rows, cols, 1.0, DY, lddy, DH, lddh, tx, A, ta, lda, SA, ldsa, H, th, ldh, SH,
                                            ldsh, WP, W, tw, GATE, ldg, tg, group, TP, T, DA, ldda, DX, lddx, DWP, DW, DG,
                                            lddg, ws, need if size is None else size, None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), 1), (dict(tx=9), 1), (dict(ta=2), 1), (dict(ta=8), 1), (dict(SA=AT[12]), 1), (dict(th=8), 1),
    (dict(SH=AT[12], th=8, ldsh=1), 1), (dict(tw=2), 1), (dict(DY=None), 1), (dict(A=None), 1), (dict(H=None), 1),
    (dict(W=None), 1), (dict(WP=None), 1), (dict(TP=None), 1), (dict(T=None), 1), (dict(DA=None), 1), (dict(DX=None), 1),
    (dict(ws=None), 1), (dict(ws=AT[11] + 4), 1), (dict(size=100), 1), (dict(DH=AT[12], lddh=1), 1), (dict(lddy=255), 1),
    (dict(GATE=AT[12], group=0), 1), (dict(GATE=AT[12], tg=2), 1), (dict(DG=AT[12]), 1),
    (dict(GATE=AT[12], DG=AT[13], lddg=255), 1), (dict(DA=AT[0]), 2), (dict(DX=AT[7]), 2), (dict(DW=AT[9]), 2),
    (dict(DWP=AT[2]), 2), (dict(ws=AT[8]), 2), (dict(GATE=AT[12], DG=AT[12]), 2), (dict(DA=AT[12], SA=AT[12], ta=8), 2)])
def test_norms_gradient_refuses(lib, change, status):
    assert norms_gradient_status(lib, **change) == status


def unit_status(lib, rows=8, cols=256, G=AT[0], ldg=256, U_=AT[1], ldu=256, tx=1, Q=AT[2], tq=8, ldq=256, S=AT[3], lds=2,
                QG=None, ldqg=256, SG=None, ldsg=2, QU=None, ldqu=256, SU=None, ldsu=2, tk=8):
    return lib.sgemm_swiglu_fp8(rows, cols, G, ldg, U_, ldu, tx, Q, tq, ldq, S, lds, QG, ldqg, SG, ldsg, QU, ldqu, SU, ldsu,
                                tk, None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), 1), (dict(tx=8), 1), (dict(tq=2), 1), (dict(G=None), 1), (dict(U_=None), 1), (dict(Q=None), 1),
    (dict(S=None), 1), (dict(ldg=255), 1), (dict(ldu=255), 1), (dict(ldq=255), 1), (dict(lds=1), 1), (dict(QG=AT[4]), 1),
    (dict(SU=AT[4]), 1), (dict(QG=AT[4], SG=AT[5], tk=0), 1), (dict(QU=AT[4], SU=AT[5], ldsu=1), 1), (dict(G=AT[0] + 1), 1),
    (dict(Q=AT[0]), 2), (dict(S=AT[1]), 2), (dict(QG=AT[2], SG=AT[5]), 2), (dict(QU=AT[4], SU=AT[3]), 2)])
def test_unit_refuses(lib, change, status):
    assert unit_status(lib, **change) == status


def unit_gradient_status(lib, rows=8, cols=256, DY=AT[0], lddy=256, tx=1, G=AT[1], tg=1, ldg=256, SG=None, ldsg=2, U_=AT[2],
                         tu=1, ldu=256, SU=None, ldsu=2, tz=9, QR=AT[3], ldqr=512, SR=AT[4], ldsr=4, QC=AT[5], ldqc=512,
                         SC=AT[6], ldsc=512, ty=8, QY=AT[7], ldqy=256, SY=AT[8], ldsy=256):
    return lib.sgemm_swiglu_backward_fp8(rows, cols, DY, lddy, tx, G, tg, ldg, SG, ldsg, U_, tu, ldu, SU, ldsu, tz, QR, ldqr,
                                         SR, ldsr, QC, ldqc, SC, ldsc, ty, QY, ldqy, SY, ldsy, None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), 1), (dict(cols=(1 << 30) + 1), 1), (dict(tx=8), 1), (dict(tz=1), 1), (dict(ty=0), 1), (dict(tg=8), 1),
    (dict(SG=AT[9], tg=8), 1), (dict(SG=AT[9], SU=AT[10]), 1), (dict(SG=AT[9], SU=AT[10], tg=8, tu=8, ldsu=1), 1), (dict(SG=AT[9], SU=AT[10], tg=8, tu=9), 1),
    (dict(DY=None), 1), (dict(G=None), 1), (dict(U_=None), 1), (dict(QR=None), 1), (dict(SR=None), 1), (dict(QC=None), 1),
    (dict(SC=None), 1), (dict(QY=None), 1), (dict(SY=None), 1), (dict(ldqr=511), 1), (dict(ldsr=3), 1), (dict(ldqc=511), 1),
    (dict(ldsc=511), 1), (dict(ldqy=255), 1), (dict(ldsy=255), 1), (dict(QR=AT[0]), 2), (dict(QC=AT[3] + 4000), 2),
    (dict(QY=AT[1]), 2), (dict(SY=AT[6]), 2), (dict(SR=AT[2]), 2)])
def test_unit_gradient_refuses(lib, change, status):
    assert unit_gradient_status(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), 1), (dict(tx=1), 1), (dict(tq=2), 1), (dict(X=None), 1), (dict(SX=None), 1), (dict(Q=None), 1),
    (dict(S=None), 1), (dict(ldx=255), 1), (dict(ldsx=1), 1), (dict(ldq=255), 1), (dict(lds=255), 1), (dict(Q=AT[0]), 2),
    (dict(S=AT[1]), 2), (dict(S=AT[1] + 2), 1)])
def test_requantise_refuses(lib, change, status):
    a = dict(rows=8, cols=256, X=AT[0], tx=8, ldx=256, SX=AT[1], ldsx=2, Q=AT[2], tq=8, ldq=256, S=AT[3], lds=256) | change
    assert lib.sgemm_fp8_requantize(a["rows"], a["cols"], a["X"], a["tx"], a["ldx"], a["SX"], a["ldsx"], a["Q"], a["tq"],
                                    a["ldq"], a["S"], a["lds"], None) == status


def test_empty_calls_need_no_pointers(lib):
    nothing = {k: None for k in ("A", "X", "WP", "W", "H", "Q", "S")}
    assert norms_status(lib, rows=0, **nothing) == norms_status(lib, cols=0, **nothing) == 0
    nothing = {k: None for k in ("DY", "A", "H", "WP", "W", "TP", "T", "DA", "DX", "DWP", "DW", "ws")}
    assert norms_gradient_status(lib, rows=0, **nothing) == norms_gradient_status(lib, cols=0, **nothing) == 0
    nothing = {k: None for k in ("G", "U_", "Q", "S")}
    assert unit_status(lib, rows=0, **nothing) == unit_status(lib, cols=0, **nothing) == 0
    nothing = {k: None for k in ("DY", "G", "U_", "QR", "SR", "QC", "SC", "QY", "SY")}
    assert unit_gradient_status(lib, rows=0, **nothing) == unit_gradient_status(lib, cols=0, **nothing) == 0
    assert lib.sgemm_fp8_requantize(0, 5, None, 8, 5, None, 1, None, 8, 5, None, 5, None) == 0
    assert lib.sgemm_last_launch_count() == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_valid_calls_without_gpu_are_unsupported(lib):
    assert norms_status(lib) == norms_gradient_status(lib) == unit_status(lib) == unit_gradient_status(lib) == 3
    assert norms_status(lib, GATE=AT[4], group=1 << 40, QA=AT[8], SA=AT[9], TP=AT[10], T=AT[11]) == 3
    assert norms_gradient_status(lib, GATE=AT[12], group=3, DG=AT[13], SA=AT[14], ta=8, DH=AT[15]) == 3
    assert norms_gradient_status(lib, DWP=None, DW=None, ws=None) == 3
    assert unit_gradient_status(lib, SG=AT[9], SU=AT[10], tg=9, tu=9) == 3


def test_tensors_are_checked_before_any_call(sg):  # noqa: F811
    x, w = torch.zeros(8, 128), torch.ones(128)
    with pytest.raises(TypeError, match="CUDA"):
        sg.sandwich_norm_fp8(x, x, w, w)
    with pytest.raises(TypeError, match="CUDA"):
        sg.sandwich_norm_backward(x, x, x, w, w, x[:, 0], x[:, 0])
    with pytest.raises(TypeError, match="CUDA"):
        sg.swiglu_fp8(x, x)
    with pytest.raises(TypeError, match="2-D tensor"):
        sg.swiglu_backward_fp8(w, x, x)
    with pytest.raises(TypeError, match="2-D tensor"):
        sg.requantize_fp8(x, x)


@gpu
def test_tensors_that_do_not_fit_are_refused(sg):  # noqa: F811
    x, y, w, t = (torch.ones(s, device="cuda") for s in ((6, 256), (6, 255), (256,), (6,)))
    k, h = sg.quantize_fp8(x), x.bfloat16()
    f = sg.sandwich_norm_fp8
    for args, kw, error, match in [
            ((x, y, w, w), {}, ValueError, "x must be"), ((x, h, w, w), {}, TypeError, "x must be"),
            ((x, x, w[1:], w), {}, ValueError, "post_weight"), ((x, x, w, t), {}, ValueError, "weight"),
            ((h, h, w, w.bfloat16()), {}, TypeError, "one type"), ((x, x, w, w), dict(gate=t), ValueError, "gate"),
            ((x, x, w, w), dict(gate=x[:4]), ValueError, "gate"), ((x, x, w, w), dict(gate=y), ValueError, "gate"),
            ((x, x, w, w), dict(gate=h), TypeError, "gate"), ((x, x, w, w), dict(gate=3.0), TypeError, "gate"),
            ((x, x, w, w), dict(dtype=torch.uint8), TypeError, "dtype"),
            ((x, x, w, w), dict(checkpoint=torch.bfloat16), TypeError, "dtype"),
            ((x[:, ::2], x, w, w), {}, ValueError, "unit column stride"), ((x[:1].expand(6, 256), x, w, w), {}, ValueError, "overlapping")]:
        with pytest.raises(error, match=match):
            f(*args, **kw)
    f = sg.sandwich_norm_backward
    for args, kw, error, match in [
            ((x, y, x, w, w, t, t), {}, ValueError, "a must be"), ((x, x, h, w, w, t, t), {}, TypeError, "h must be"),
            ((x, (k[0], k[1][:5]), x, w, w, t, t), {}, ValueError, "a's scales"), ((x, (k[0],), x, w, w, t, t), {}, TypeError, "pair"),
            ((x, x, (k[0][:5], k[1]), w, w, t, t), {}, ValueError, "h must be"), ((x, x, x, w, w, t[1:], t), {}, ValueError, "post_rstd"),
            ((x, x, x, w, w, t, w), {}, ValueError, "rstd"), ((x, x, x, w, w, t, t), dict(dh=y), ValueError, "dh"),
            ((x, x, x, w, w, t, t), dict(gate=x[:4]), ValueError, "gate")]:
        with pytest.raises(error, match=match):
            f(*args, **kw)
    for args, error, match in [((x, y), ValueError, "up must be"), ((x, h), TypeError, "up must be")]:
        with pytest.raises(error, match=match):
            sg.swiglu_fp8(*args)
    for args, error, match in [((x, y, x), ValueError, "gate must be"), ((x, k, x), TypeError, "both"), ((x, k, sg.quantize_fp8(x, dtype=E5M2)), TypeError, "one type"), ((h, x, x), TypeError, "gate must be")]:
        with pytest.raises(error, match=match):
            sg.swiglu_backward_fp8(*args)
    with pytest.raises(ValueError, match="scale must be"):
        sg.requantize_fp8(k[0], k[1][:, :1])
    with pytest.raises(TypeError, match="dtype"):
        sg.requantize_fp8(*k, dtype=torch.float16)
