"""The 8-bit linear layer: quantiser, block-scaled product, RMS norm and its
gradient, each against its definition in 64 bits.

Tolerances, with u = 2^-24 (FP32 rounding) and ulp8(v) the spacing of the 8-bit
type at v:
  scale     equal to the FP32 quotient max|x| / F.
  q         x/s is formed with two roundings, then rounded to 8 bits:
            |q - x/s| <= ulp8/2 + 4 u |x/s|.
  product   8-bit products are exact; 128 of them are added in 32 bits (an
            addition loses at most 2 u of the sum of magnitudes), the block's
            sum meets two scale roundings and is added to the running sum, a
            rounding per block: |err| <= 2 u (128 + blocks + 4) * sum |a b|,
            plus the rounding of the output type.  Bit-exact where every value
            and partial sum is exact (small integers, power-of-two scales).
  norm      a row's sum of squares: at most 128 additions in a thread and 10
            after it, so t is within 2^-17 and y within 2^-16 relative.
  gradient  likewise 2^-16 of the sum of magnitudes of what is added.
These hold for the 32-bit value; rounding to the output type is monotone, so
the output lies between the bounds' own roundings (`within`).
"""
import numpy as np
import pytest
import torch

U = 2.0 ** -24
B = 128
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
FMAX = {E4M3: 448.0, E5M2: 57344.0}
FLOATS = [torch.float32, torch.bfloat16, torch.float16]
gpu = pytest.mark.gpu


def cdiv(a, b):
    return -(-a // b)


@pytest.fixture(scope="module")
def sg():
    import dense_fp32_matrix_10_gb300 as sg
    return sg


@pytest.fixture(scope="module")
def clean_status(sg):
    yield
    assert sg.sgemm_last_device_status() == 0


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def strided(t, pad, offset=0, fill=None):
    """A copy of t whose rows are `pad` elements longer, starting `offset` elements into its storage; the
    padding holds NaN."""
    r, c = t.shape
    big = torch.empty(r * (c + pad) + offset + 64, dtype=t.dtype, device=t.device)
    if t.dtype in FMAX:
        big.view(torch.uint8).fill_(0x7f)      # NaN in both types
    else:
        big.fill_(float("nan"))
    v = big[offset:offset + r * (c + pad)].view(r, c + pad)[:, :c]
    v.view(torch.uint8).copy_(t.view(torch.uint8)) if t.dtype in FMAX else v.copy_(t)
    return v


def spread(s, br, bc, rows, cols):
    return s.double().repeat_interleave(br, 0)[:rows].repeat_interleave(bc, 1)[:, :cols]


def within(got, want, lim):
    """Whether got is the rounding to its type of FP32 values no further than lim from want (64 bits)."""
    lo, hi = ((want + d).float().to(got.dtype) for d in (-lim, lim))
    return ((lo <= got) & (got <= hi)).all()


def ulp8(v, dtype):
    mant, least = (3, -6) if dtype == E4M3 else (2, -14)
    e = (torch.frexp(v.abs())[1] - 1).clamp_min(least) - mant
    return torch.ldexp(torch.ones_like(v), e)


def check_quantised(q, s, x, br, bc, rel=4 * U, exact_scale=True):
    """q, s against the definition for x (float64; any of its roundings up to `rel`)."""
    rows, cols = x.shape
    p = x.new_zeros(cdiv(rows, br) * br, cdiv(cols, bc) * bc)
    p[:rows, :cols] = x
    a = p.view(cdiv(rows, br), br, cdiv(cols, bc), bc).abs().amax((1, 3))
    want = (a / FMAX[q.dtype]).float().clamp_min(2.0 ** -126)   # 64 bits hold enough to round once to 32
    assert s.shape == want.shape and q.shape == x.shape
    if exact_scale:
        assert torch.equal(s, want)
    else:
        assert ((s.double() - want.double()).abs() <= rel * want.double()).all()
    v = x / spread(s, br, bc, rows, cols)
    err = (q.double() - v).abs()
    assert (err <= ulp8(v, q.dtype) / 2 + rel * v.abs()).all()


# ---------------------------------------------------------------- quantiser
SHAPES = [(1, 1), (1, 128), (7, 5), (128, 128), (129, 127), (1, 4096), (300, 1000), (257, 129)]
BLOCKS = [(1, B), (B, 1), (B, B)]


@gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("xtype", FLOATS)
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_quantise(sg, shape, block, xtype, dtype):
    x = torch.randn(shape, generator=rng(1), device="cuda")
    x *= torch.exp(3 * torch.randn(shape[0], 1, generator=rng(2), device="cuda"))
    x = x.to(xtype)
    q, s = sg.quantize_fp8(x, block, dtype)
    assert q.dtype == dtype and q.stride(0) % 16 == 0
    check_quantised(q, s, x.double(), *block)


@gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("xtype", FLOATS)
def test_quantise_both_is_the_two(sg, shape, xtype):
    x = torch.randn(shape, generator=rng(3), device="cuda").to(xtype)
    qr, sr, qc, sc = sg.quantize_fp8_both(x, E5M2)
    for (q, s), block in (((qr, sr), (1, B)), ((qc, sc), (B, 1))):
        want_q, want_s = sg.quantize_fp8(x, block, E5M2)
        assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s, want_s)


@gpu
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 8), (1, 1), (0, 5)])
@pytest.mark.parametrize("xtype", FLOATS)
@pytest.mark.parametrize("block", BLOCKS)
def test_quantise_strides(sg, pad, offset, xtype, block):
    """Any row stride and base; nothing outside the matrix is read (NaN there) or written."""
    x = torch.randn(130, 141, generator=rng(4), device="cuda").to(xtype)
    want_q, want_s = sg.quantize_fp8(x, block)
    q, s = sg.quantize_fp8(strided(x, pad, offset), block)
    assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s, want_s)
    # outputs with an odd row stride through the C entry
    big = torch.full((130 * 147,), 0x55, dtype=torch.uint8, device="cuda")
    out = torch.full((s.shape[0], s.shape[1] + 2), -5.0, device="cuda")
    sg.sgemm_fp8_quantize(130, 141, x.data_ptr(), {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[xtype], 141,
                          big.data_ptr(), 8, 147, out.data_ptr(), out.stride(0), *block,
                          torch.cuda.current_stream().cuda_stream)
    big = big.view(130, 147)
    assert torch.equal(big[:, :141], want_q.view(torch.uint8)) and (big[:, 141:] == 0x55).all()
    assert torch.equal(out[:, :-2], want_s) and (out[:, -2:] == -5).all()


@gpu
@pytest.mark.parametrize("block", BLOCKS)
def test_quantise_special_values(sg, block):
    x = torch.randn(256, 256, generator=rng(5), device="cuda")
    x[128:, 128:] = 0
    x[0, 200] = 1e-44            # a subnormal among larger ones
    q, s = sg.quantize_fp8(x, block)
    zero = s[-1, -1]
    assert zero == 2.0 ** -126 and (q[128:, 128:].float() == 0).all()
    tiny = torch.full((1, 128), 1e-44, device="cuda")
    q, s = sg.quantize_fp8(tiny)
    assert s.item() == 2.0 ** -126 and (q.float() == 0).all()   # 1e-44 / 2^-126 is below e4m3's least
    big = torch.full((1, 128), 3e38, device="cuda")
    q, s = sg.quantize_fp8(big)
    assert (q.float() == 448).all() and torch.isfinite(s).all()
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[3, 5] = bad
        q, s = sg.quantize_fp8(y, block)
        v = q.float() * spread(s, *block, 256, 256).float()
        i, j = (3, 0) if block == (1, B) else (0, 5) if block == (B, 1) else (0, 0)
        assert not torch.isfinite(s[i, j]) and not torch.isfinite(v[3, 5])
        keep = torch.isfinite(s)
        assert (~keep).sum() == 1
        want_q, want_s = sg.quantize_fp8(x, block)
        assert torch.equal(s[keep], want_s[keep])


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_quantise_finite_beside_an_infinity(sg, dtype):
    """x / inf is 0 for the block's finite elements, and NaN only where x is infinite."""
    x = torch.randn(256, 256, generator=rng(15), device="cuda").to(dtype)
    x[3, 5] = float("inf")
    qr, _, qc, _ = sg.quantize_fp8_both(x)
    t = sg.quantize_fp8(x, (B, B))
    for q, inside in ((qr, (slice(3, 4), slice(0, B))), (sg.quantize_fp8(x)[0], (slice(3, 4), slice(0, B))),
                      (qc, (slice(0, B), slice(5, 6))), (sg.quantize_fp8(x, (B, 1))[0], (slice(0, B), slice(5, 6))),
                      (t[0], (slice(0, B), slice(0, B)))):
        v = q.float()
        assert torch.isnan(v[3, 5])
        v[3, 5] = 0
        assert (v[inside] == 0).all()
        assert torch.isfinite(v).all() and (v != 0).any()


@gpu
def test_quantise_beyond_32_bit_offsets(sg):
    rows, cols, ld = 70000, 136, 32768
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(rows, ld)[:, :cols]
    x.copy_(torch.randn(rows, cols, generator=rng(6), device="cuda"))
    for block in BLOCKS:
        q, s = sg.quantize_fp8(x, block)
        check_quantised(q, s, x.double(), *block)


# ---------------------------------------------------------------- product
def operand(outer, k, block, dtype, inner_rows, seed, integers=False, pad=0, offset=0):
    """(q, s, exact outer x k matrix in 64 bits): random 8-bit values and scales in stored layout."""
    g = rng(seed)
    if integers:
        v = torch.randint(-3, 4, (outer, k), generator=g, device="cuda").float()
        s = torch.exp2(torch.randint(-2, 3, (cdiv(outer, block), cdiv(k, B)), generator=g, device="cuda").float())
    else:
        v = torch.randn(outer, k, generator=g, device="cuda") * 30
        s = torch.rand(cdiv(outer, block), cdiv(k, B), generator=g, device="cuda") * 0.02 + 1e-3
    q = v.to(dtype)
    exact = q.double() * spread(s, block, B, outer, k)
    if inner_rows:
        q, s = q.t().contiguous(), s.t().contiguous()
    if pad or offset:
        q = strided(q, pad, offset)
        s = strided(s, 3)
    else:
        q = strided(q, -q.shape[1] % 16)
    return q, s, exact


def check_product(sg, M, N, K, ta=0, tb=1, ba=1, bb=B, fa=E4M3, fb=E4M3, out=torch.float32, alpha=1.0, beta=0.0,
                  integers=False, pad=0, offset=0, seed=10):
    qa, sa, a = operand(M, K, ba, fa, ta == 1, seed, integers, pad, offset)
    qb, sb, b = operand(N, K, bb, fb, tb == 0, seed + 1, integers, pad, offset)
    c = None
    if beta != 0 or pad:
        c = torch.randint(-4, 5, (M, N), generator=rng(seed + 2), device="cuda").to(out)
        c = strided(c, pad)
    old = c.double() if c is not None else torch.zeros(M, N, dtype=torch.float64, device="cuda")
    got = sg.gemm_fp8(qa, sa, qb, sb, c, alpha, beta, bool(ta), bool(tb), out)
    assert got.shape == (M, N) and got.dtype == out
    want = alpha * (a @ b.t()) + beta * old
    if integers:
        assert torch.equal(got, want.to(out)), (M, N, K)
    else:
        size = abs(alpha) * (a.abs() @ b.abs().t())
        lim = 2 * U * (128 + cdiv(K, B) + 4) * size + 4 * U * (abs(beta) * old.abs() + want.abs())
        assert within(got, want, lim), (M, N, K)
        if out == torch.float32:
            # what is lost does not add up over the whole output either
            assert (got.double() - want).norm() <= 1e-6 * size.norm()
    return got


LAYOUTS = [(0, 1, 1, B), (0, 0, 1, B), (1, 0, 1, 1), (0, 1, 1, 1), (1, 1, B, B), (1, 0, B, 1), (0, 1, B, 1), (1, 1, 1, B)]
SIZES = [(1, 1, 1), (1, 128, 128), (3, 5, 7), (1, 300, 520), (16, 128, 256), (17, 130, 127), (31, 1000, 384),
         (64, 256, 1024), (65, 4097, 129), (128, 128, 128), (129, 257, 385), (200, 512, 2048), (256, 256, 512),
         (300, 777, 640), (513, 1025, 257), (1000, 1013, 997)]


@gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_product_integers_are_exact(sg, clean_status, size, layout):
    check_product(sg, *size, *layout, integers=True)


@gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("layout", LAYOUTS[:4])
@pytest.mark.parametrize("out", FLOATS)
def test_product_random(sg, clean_status, size, layout, out):
    check_product(sg, *size, *layout, out=out)


@gpu
@pytest.mark.parametrize("fa,fb", [(E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)])
@pytest.mark.parametrize("size", [(5, 200, 300), (150, 260, 400), (520, 1030, 640)])
@pytest.mark.parametrize("layout", [(0, 1, 1, B), (1, 0, 1, 1)])
def test_product_types(sg, clean_status, fa, fb, size, layout):
    check_product(sg, *size, *layout, fa=fa, fb=fb)
    check_product(sg, *size, *layout, fa=fa, fb=fb, integers=True)


@gpu
@pytest.mark.parametrize("alpha,beta", [(1.5, 0.0), (0.5, 2.0), (-1.0, 1.0), (0.0, 0.5), (0.0, 0.0)])
@pytest.mark.parametrize("size", [(1, 200, 300), (40, 129, 256), (300, 520, 640)])
@pytest.mark.parametrize("out", FLOATS)
def test_product_alpha_beta(sg, clean_status, alpha, beta, size, out):
    check_product(sg, *size, out=out, alpha=alpha, beta=beta, integers=out == torch.float32)
    check_product(sg, *size, 1, 0, 1, 1, out=out, alpha=alpha, beta=beta)


@gpu
@pytest.mark.parametrize("pad,offset", [(1, 0), (16, 16), (16, 1), (5, 7), (32, 0)])
@pytest.mark.parametrize("layout", [(0, 1, 1, B), (0, 0, 1, B), (1, 0, 1, 1)])
@pytest.mark.parametrize("size", [(3, 140, 300), (130, 270, 256), (600, 512, 384)])
def test_product_strides(sg, clean_status, pad, offset, layout, size):
    """Padded and misaligned operands, scales and outputs; NaN beyond every row's end."""
    check_product(sg, *size, *layout, pad=pad, offset=offset, integers=True)
    got = check_product(sg, *size, *layout, pad=pad, offset=offset)
    past = got.as_strided((size[0], pad), got.stride(), got.storage_offset() + size[1])
    assert torch.isnan(past).all()


@gpu
@pytest.mark.parametrize("M", [1, 5, 40, 200, 700])
def test_product_special_scales(sg, clean_status, M):
    """A NaN or infinite scale reaches its own rows only; zero rows stay zero; NaN in an unread C is overwritten."""
    K, N = 700, 400
    qa, sa, a = operand(M, K, 1, E4M3, False, 20)
    qb, sb, b = operand(N, K, B, E4M3, False, 21)
    clean = sg.gemm_fp8(qa, sa, qb, sb, transB=True, out_dtype=torch.float32)
    sa2 = sa.clone()
    sa2[M // 2, 3] = float("nan")
    got = sg.gemm_fp8(qa, sa2, qb, sb, torch.full((M, N), float("nan"), device="cuda"), transB=True)
    rest = torch.arange(M, device="cuda") != M // 2
    assert torch.isnan(got[M // 2]).all() and torch.equal(got[rest], clean[rest])
    qz = qa.clone()
    qz.view(torch.uint8)[M // 2].zero_()
    assert (sg.gemm_fp8(qz, sa, qb, sb, transB=True)[M // 2].float() == 0).all()
    sb2 = sb.clone()
    sb2[1, 0] = float("inf")
    got = sg.gemm_fp8(qa, sa, qb, sb2, transB=True, out_dtype=torch.float32)
    assert not torch.isfinite(got[:, 128:256]).any()
    assert torch.equal(got[:, :128], clean[:, :128]) and torch.equal(got[:, 256:], clean[:, 256:])


@gpu
@pytest.mark.parametrize("M,N,K", [(0, 5, 7), (5, 0, 7)])
def test_product_empty(sg, M, N, K):
    z = lambda r, c: (torch.zeros(r, c, device="cuda").to(E4M3), torch.zeros(r, cdiv(c, B), device="cuda"))
    assert sg.gemm_fp8(*z(M, K), *z(N, K), transB=True).shape == (M, N)


@gpu
def test_product_of_no_inner_dimension(sg):
    z = lambda r: (torch.zeros(r, 0, device="cuda").to(E4M3), torch.zeros(r, 0, device="cuda"))
    assert (sg.gemm_fp8(*z(5), *z(9), transB=True).float() == 0).all()
    c = torch.arange(45.0, device="cuda").view(5, 9)
    assert torch.equal(sg.gemm_fp8(*z(5), *z(9), c.clone(), beta=2.0, transB=True), 2 * c)


@gpu
@pytest.mark.parametrize("M,N,K", [(70000, 16, 32768), (24, 70000, 32768), (70000, 32768, 32)])
def test_product_beyond_32_bit_offsets(sg, clean_status, M, N, K):
    qa = (torch.randint(0, 2, (M, K), dtype=torch.uint8, device="cuda") * 0x38).view(E4M3)     # 0 or 1
    qb = (torch.randint(0, 2, (N, K), dtype=torch.uint8, device="cuda") * 0x38).view(E4M3)
    sa = torch.ones(M, cdiv(K, B), device="cuda")
    sb = torch.ones(cdiv(N, B), cdiv(K, B), device="cuda")
    got = sg.gemm_fp8(qa, sa, qb, sb, transB=True, out_dtype=torch.float32)
    i = torch.tensor(sorted({0, 1, M // 2, M - 2, M - 1}), device="cuda")
    j = torch.tensor(sorted({0, 1, N // 2, N - 2, N - 1}), device="cuda")
    want = qa.view(torch.uint8)[i].bool().double() @ qb.view(torch.uint8)[j].bool().double().t()
    assert torch.equal(got[i][:, j].double(), want)


@gpu
def test_product_repeats_bit_for_bit(sg):
    for M, N, K in ((1, 4096, 4096), (24, 1000, 4096), (300, 1000, 2000), (2048, 1024, 1024)):
        qa, sa, _ = operand(M, K, 1, E4M3, False, 30)
        qb, sb, _ = operand(N, K, B, E4M3, False, 31)
        first = sg.gemm_fp8(qa, sa, qb, sb, transB=True, out_dtype=torch.float32)
        for _ in range(3):
            assert torch.equal(sg.gemm_fp8(qa, sa, qb, sb, transB=True, out_dtype=torch.float32), first)


@gpu
def test_layer_gradients_are_the_adjoints(sg):
    """<dY, X W^T> is linear in X and in W: the input and weight gradients' products give its differences."""
    M, N, K = 200, 300, 400
    x, w, dy = (torch.randint(-3, 4, s, generator=rng(40 + i), device="cuda").float()
                for i, s in enumerate(((M, K), (N, K), (M, N))))
    one = lambda t, br, bc: (strided(t.to(E4M3), -t.shape[1] % 16),
                             torch.ones(cdiv(t.shape[0], br), cdiv(t.shape[1], bc), device="cuda"))
    f = lambda X, W: (dy.double() * sg.gemm_fp8(*one(X, 1, B), *one(W, B, B), transB=True,
                                                out_dtype=torch.float32).double()).sum()
    dx = sg.gemm_fp8(*one(dy, 1, B), *one(w, B, B), out_dtype=torch.float32)
    dw = sg.gemm_fp8(*one(dy, B, 1), *one(x, B, 1), transA=True, out_dtype=torch.float32)
    vx, vw = (torch.randint(-2, 3, t.shape, generator=rng(50), device="cuda").float() for t in (x, w))
    assert f(x + vx, w) - f(x - vx, w) == 2 * (dx.double() * vx.double()).sum()
    assert f(x, w + vw) - f(x, w - vw) == 2 * (dw.double() * vw.double()).sum()


# ---------------------------------------------------------------- norm
NORM_SHAPES = [(1, 1), (1, 128), (3, 7), (5, 130), (2, 1000), (1, 4096), (700, 256), (1300, 520), (1300, 1000),
               (33, 2056), (400, 5000), (3, 8192), (320, 8192), (2, 16385), (5, 40000)]


def norm_exact(x, r, w, eps):
    h = x.double() + (r.double() if r is not None else 0)
    t = 1 / torch.sqrt((h * h).mean(1) + eps)
    return h, t, h * t[:, None] * w.double()


@gpu
@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("xtype", FLOATS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(sg, shape, xtype, residual):
    rows, cols = shape
    x = torch.randn(shape, generator=rng(60), device="cuda").to(xtype)
    r = (3 * torch.randn(shape, generator=rng(61), device="cuda")).to(xtype) if residual else None
    if rows > 2:
        x[1] = 0
        if residual:
            r[1] = 0
    wtype = xtype if cols % 2 else torch.float32
    w = (1 + 0.2 * torch.randn(cols, generator=rng(62), device="cuda")).to(wtype)
    dtype = E5M2 if rows % 2 else E4M3
    o = sg.rms_norm_fp8(x, w, r, 1e-5, dtype, training=True)
    h, t, y = norm_exact(x, r, w, 1e-5)
    if residual:
        assert torch.equal(o.h, (x.float() + r.float()).to(xtype))
    else:
        assert o.h is None
    assert ((o.rstd.double() - t).abs() <= 2.0 ** -17 * t).all()
    assert within(o.y, y, 2.0 ** -16 * y.abs())
    check_quantised(o.q, o.scale, y, 1, B, rel=2.0 ** -15, exact_scale=False)
    bare = sg.rms_norm_fp8(x, w, r, 1e-5, dtype)
    assert torch.equal(bare.q.view(torch.uint8), o.q.view(torch.uint8)) and torch.equal(bare.scale, o.scale)
    assert bare.y is None and bare.rstd is None


@gpu
@pytest.mark.parametrize("shape", [(3, 141), (200, 1001), (3, 40001)])
@pytest.mark.parametrize("xtype", FLOATS)
def test_norm_strides(sg, shape, xtype):
    x, r = (torch.randn(shape, generator=rng(70 + i), device="cuda").to(xtype) for i in range(2))
    w = torch.randn(shape[1], generator=rng(72), device="cuda").to(xtype)
    want = sg.rms_norm_fp8(x, w, r, training=True)
    got = sg.rms_norm_fp8(strided(x, 3, 1), strided(w[None], 5, 1)[0], strided(r, 8, 8), training=True)
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@gpu
def test_norm_special_rows(sg):
    """A row that holds NaN or an infinity touches no other row; with eps = 0 a row of zeros is NaN, with eps zero."""
    x = torch.randn(6, 300, generator=rng(80), device="cuda")
    w = torch.ones(300, device="cuda")
    want = sg.rms_norm_fp8(x, w, training=True)
    x[1, 7], x[3, 299] = float("nan"), float("inf")
    x[4] = 0
    o = sg.rms_norm_fp8(x, w, training=True)
    for i in (0, 2, 5):
        assert torch.equal(o.y[i], want.y[i]) and torch.equal(o.q[i].float(), want.q[i].float())
    assert torch.isnan(o.y[1]).all() and torch.isnan(o.scale[1]).all()
    assert o.rstd[3] == 0 and torch.isnan(o.y[3, 299]) and (o.y[3, :299] == 0).all() and torch.isnan(o.scale[3, 2])
    assert (o.q[4].float() == 0).all() and (o.scale[4] == 2.0 ** -126).all()
    assert torch.isnan(sg.rms_norm_fp8(x, w, eps=0.0).scale[4]).all()


@gpu
@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("xtype", FLOATS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradient(sg, shape, xtype, residual):
    rows, cols = shape
    h, dy, dh = (torch.randn(shape, generator=rng(90 + i), device="cuda").to(xtype) for i in range(3))
    dh = dh if residual else None
    wtype = xtype if cols % 2 else torch.float32
    w = (1 + 0.2 * torch.randn(cols, generator=rng(93), device="cuda")).to(wtype)
    t = (1 / torch.sqrt(h.double().square().mean(1) + 1e-5)).float()
    dx, dw = sg.rms_norm_backward(dy, h, w, t, dh)
    assert dx.dtype == xtype and dw.dtype == wtype
    H, DY, T = h.double(), dy.double(), t.double()[:, None]
    g = DY * w.double()
    back = H * T ** 3
    want = T * g - back * (g * H).mean(1, keepdim=True) + (dh.double() if residual else 0)
    size = T * g.abs() + back.abs() * (g * H).abs().mean(1, keepdim=True) + (dh.double().abs() if residual else 0)
    assert within(dx, want, 2.0 ** -16 * size)
    want, size = (DY * H * T).sum(0), (DY * H * T).abs().sum(0)
    assert within(dw, want, 2.0 ** -16 * size)
    again = sg.rms_norm_backward(dy, h, w, t, dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@gpu
@pytest.mark.parametrize("shape", [(4, 100), (50, 3000)])
def test_norm_gradient_against_differences(sg, shape):
    """Along a direction v, the central difference of <dy, y> in 64 bits is <dx, v> (and <dw, v> for the weights)."""
    h, dy, v = (torch.randn(shape, generator=rng(100 + i), device="cuda") for i in range(3))
    w, vw = (torch.randn(shape[1], generator=rng(103 + i), device="cuda") for i in range(2))
    t = (1 / torch.sqrt(h.double().square().mean(1) + 1e-5)).float()
    dx, dw = sg.rms_norm_backward(dy, h, w, t)
    f = lambda H, W: (dy.double() * norm_exact(H, None, W, 1e-5)[2]).sum()
    e = 1e-4   # differences lose e^2 ~ 1e-8 of the third derivative and 1e-16 / e of the value
    for got, step in ((dx, (v, 0 * vw)), (dw, (0 * v, vw))):
        d = step[0] if got is dx else step[1]
        diff = (f(h.double() + e * step[0], w.double() + e * step[1]) -
                f(h.double() - e * step[0], w.double() - e * step[1])) / (2 * e)
        size = (got.double() * d.double()).abs().sum()
        assert abs((got.double() * d.double()).sum() - diff) <= (2.0 ** -15 + 1e-6) * size


@gpu
def test_norm_gradient_strides_and_no_rows(sg):
    shape = (70, 1001)
    h, dy, dh = (torch.randn(shape, generator=rng(110 + i), device="cuda").bfloat16() for i in range(3))
    w = torch.randn(shape[1], generator=rng(113), device="cuda").bfloat16()
    t = torch.rand(shape[0], generator=rng(114), device="cuda")
    want = sg.rms_norm_backward(dy, h, w, t, dh)
    got = sg.rms_norm_backward(strided(dy, 7, 1), strided(h, 0, 3), w, t, strided(dh, 1, 0))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dx, dw = sg.rms_norm_backward(dy[:0], h[:0], w, t[:0])
    assert dx.shape == (0, 1001) and (dw == 0).all()


@gpu
def test_norm_beyond_32_bit_offsets(sg):
    rows, cols, ld = 70000, 136, 32768
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(rows, ld)[:, :cols]
    x.copy_(torch.randn(rows, cols, generator=rng(120), device="cuda"))
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    got, want = (sg.rms_norm_fp8(v, w, v.clone(), training=True) for v in (x, x.contiguous()))
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    for a, b in zip(sg.rms_norm_backward(x, x, w, want.rstd), sg.rms_norm_backward(x.contiguous(), x.contiguous(), w, want.rstd)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- streams and graphs
def layer(sg, x, r, w, qw, sw, **kw):
    o = sg.rms_norm_fp8(x, w, residual=r, training=True, **kw)
    y = sg.gemm_fp8(o.q, o.scale, qw, sw, transB=True, **kw)
    g = sg.quantize_fp8_both(y, **kw)
    dn = sg.gemm_fp8(g[0], g[1], qw, sw, **kw)
    dx, dw = sg.rms_norm_backward(dn, o.h, w, o.rstd, dh=o.h, **kw)
    return y, dx, dw


def layer_inputs(sg, rows=300, cols=640, out=520):
    x, r = (torch.randn(rows, cols, generator=rng(130 + i), device="cuda").bfloat16() for i in range(2))
    w = torch.ones(cols, device="cuda").bfloat16()
    qw, sw = sg.quantize_fp8(torch.randn(out, cols, generator=rng(132), device="cuda"), (B, B))
    return x, r, w, qw, sw


@gpu
def test_on_another_stream(sg):
    args = layer_inputs(sg)
    want = layer(sg, *args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = layer(sg, *args, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_captured_into_a_graph(sg):
    args = layer_inputs(sg)
    want = layer(sg, *args)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer(sg, *args)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(sg, *args)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_no_device_memory_of_the_librarys_own(sg):
    old, _ = sg.sgemm_get_scratch_limit()
    try:
        sg.sgemm_set_scratch_limit(0)
        layer(sg, *layer_inputs(sg))
        assert sg.sgemm_get_scratch_limit()[1] == 0
    finally:
        sg.sgemm_set_scratch_limit(old)


# ---------------------------------------------------------------- the extension module
def test_extension_is_built_and_bound(lib):
    from dense_fp32_matrix_10_gb300 import fp8
    assert fp8._usual is not None and fp8._usual.__file__.startswith(fp8.__file__.rsplit("/", 1)[0])


def test_extension_leaves_the_unusual_to_python(lib):
    from dense_fp32_matrix_10_gb300 import fp8
    u, x = fp8._usual, torch.zeros(4, 8)
    assert u.quantize(x, 1, 128, 8) is None and u.quantize_both(x, 8) is None        # not on a GPU
    assert u.product(x, x, x, x, None, 1.0, 0.0, False, True, 1) is None
    assert u.product(None, None, None, None, None, "1", 0.0, False, True, 1) is None
    assert u.norm(x, x[0], None, 1e-6, 8, False) is None and u.norm_backward(x, x, x[0], x[0], None) is None
    assert u.norm(x, x[0], None, 1e-6) is None                                       # arguments missing


@gpu
@pytest.mark.parametrize("shape", [(1, 128), (5, 0), (0, 7), (70, 333), (257, 1024)])
def test_both_ways_through_python(sg, monkeypatch, shape):
    """The extension module and the general code hand over the same calls."""
    from dense_fp32_matrix_10_gb300 import fp8
    rows, cols = shape
    x, r = (torch.randn(shape, generator=rng(140 + i), device="cuda").bfloat16() for i in range(2))
    w = torch.randn(cols, generator=rng(142), device="cuda")
    qb, sb, _ = operand(96, cols, B, E4M3, False, 143)
    c = torch.randn(rows, 100, generator=rng(144), device="cuda")[:, :96]

    def everything():
        o = sg.rms_norm_fp8(x, w, residual=r, training=True)
        q, s = sg.quantize_fp8(x)
        out = [*o[:5 if cols else 4], q, s]   # (rows of no elements have no rstd)
        out += [*sg.quantize_fp8(x, (B, 1), E5M2), *sg.quantize_fp8_both(x)]
        out += [*sg.rms_norm_backward(x, o.h, w, o.rstd, dh=r), *sg.rms_norm_backward(x, o.h, w, o.rstd)]
        for kw in (dict(), dict(out_dtype=torch.float32, alpha=0.5), dict(C=c.clone(), beta=1.0)):
            out.append(sg.gemm_fp8(q, s, qb, sb, transB=True, **kw))
        return out

    ours = everything()
    monkeypatch.setattr(fp8, "_usual", None)
    for a, b in zip(ours, everything()):
        assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib(sg):
    from dense_fp32_matrix_10_gb300 import build
    build.build()
    from dense_fp32_matrix_10_gb300 import fp8
    return fp8._library()


A0, B0, C0, S0, S1 = 0x100000, 0x900000, 0x2000000, 0x4000000, 0x5000000   # never dereferenced


def product_status(lib, ta=0, tb=1, M=8, N=16, K=256, A=A0, fa=8, lda=256, SA=S0, ldsa=2, ba=1, B_=B0, fb=8, ldb=256,
                   SB=S1, ldsb=2, bb=128, C=C0, tc=1, ldc=16, alpha=1.0, beta=0.0):
    return lib.sgemm_fp8(ta, tb, M, N, K, alpha, A, fa, lda, SA, ldsa, ba, B_, fb, ldb, SB, ldsb, bb, beta, C, tc, ldc,
                         None)


@pytest.mark.parametrize("bad", [
    dict(ta=2), dict(tb=-1), dict(M=-1), dict(K=1 << 31), dict(fa=1), dict(fb=7), dict(tc=8), dict(ba=2), dict(bb=64),
    dict(lda=255), dict(ldb=255), dict(ldsa=1), dict(ldsb=1), dict(ldc=15), dict(A=None), dict(SA=None), dict(B_=None),
    dict(SB=None), dict(C=None), dict(SA=S0 + 2), dict(C=C0 + 1), dict(lda=1 << 41), dict(ta=1, lda=7),
    dict(ta=1, M=300, lda=300, ldsa=299), dict(tb=0, ldb=15)])
def test_product_refuses(lib, bad):
    assert product_status(lib, **bad) == 1


def test_product_refuses_overlaps(lib):
    for bad in (dict(C=A0), dict(C=B0 + 256), dict(C=S0), dict(C=S1 - 2)):
        assert product_status(lib, **bad) == 2


def test_empty_calls_need_no_pointers(lib):
    assert product_status(lib, M=0, A=None, SA=None, B_=None, SB=None, C=None) == 0
    assert product_status(lib, N=0, A=None, SA=None, B_=None, SB=None, C=None) == 0
    assert lib.sgemm_fp8_quantize(0, 5, None, 0, 5, None, 8, 5, None, 1, 1, 128, None) == 0
    assert lib.sgemm_rms_norm_fp8(4, 0, 1e-6, None, 1, None, 0, 1, None, 1, None, 0, None, 0, None, 8, 1, None, 1, None,
                                  None) == 0
    assert lib.sgemm_rms_norm_backward(0, 8, None, 8, None, 8, 1, None, 1, None, None, 0, None, 8, None, None, 0,
                                       None) == 0
    assert lib.sgemm_last_launch_count() == 0


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), 1), (dict(tx=8), 1), (dict(tq=1), 1), (dict(br=128, bc=64), 1), (dict(br=1, bc=1), 1),
    (dict(ldx=255), 1), (dict(ldq=255), 1), (dict(lds=1), 1), (dict(X=None), 1), (dict(Q=None), 1), (dict(S=None), 1),
    (dict(X=A0 + 2), 1), (dict(Q=A0 + 100), 2), (dict(S=B0 + 4), 2)])
def test_quantise_refuses(lib, change, status):
    a = dict(rows=8, cols=256, X=A0, tx=0, ldx=256, Q=B0, tq=8, ldq=256, S=S0, lds=2, br=1, bc=128) | change
    assert lib.sgemm_fp8_quantize(a["rows"], a["cols"], a["X"], a["tx"], a["ldx"], a["Q"], a["tq"], a["ldq"], a["S"],
                                  a["lds"], a["br"], a["bc"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(QR=None), 1), (dict(SR=None), 1), (dict(QC=None), 1), (dict(SC=None), 1), (dict(ldsc=255), 1),
    (dict(QC=B0), 2), (dict(SC=S0), 2)])
def test_quantise_both_refuses(lib, change, status):
    a = dict(QR=B0, SR=S0, QC=C0, SC=S1, ldsc=256) | change
    assert lib.sgemm_fp8_quantize_both(8, 256, A0, 1, 256, 8, a["QR"], 256, a["SR"], 2, a["QC"], 256, a["SC"],
                                       a["ldsc"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(tx=9), 1), (dict(tw=2), 1), (dict(tq=0), 1), (dict(X=None), 1),
    (dict(W=None), 1), (dict(Q=None), 1), (dict(S=None), 1), (dict(ldr=1), 1), (dict(H=A0), 2), (dict(Y=B0), 2),
    (dict(T=S0), 2), (dict(Q=C0, H=C0), 2)])
def test_norm_refuses(lib, change, status):
    a = dict(eps=1e-6, X=A0, R=B0, ldr=256, tx=1, W=S1, tw=1, H=None, Y=None, Q=C0, tq=8, S=S0, T=None) | change
    assert lib.sgemm_rms_norm_fp8(8, 256, a["eps"], a["X"], 256, a["R"], a["ldr"], a["tx"], a["W"], a["tw"], a["H"], 256,
                                  a["Y"], 256, a["Q"], a["tq"], 256, a["S"], 2, a["T"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(DY=None), 1), (dict(H=None), 1), (dict(W=None), 1), (dict(T=None), 1), (dict(DX=None), 1), (dict(ws=None), 1),
    (dict(bytes=8 * 256 * 4 - 1), 1), (dict(ws=S1 + 4), 1), (dict(tx=8), 1), (dict(tw=2), 1), (dict(DX=A0), 2),
    (dict(DW=B0), 2), (dict(ws=C0), 2)])
def test_norm_gradient_refuses(lib, change, status):
    a = dict(DY=A0, H=B0, tx=1, W=S0, tw=1, T=S0 + 4096, DX=C0, DW=S0 + 8192, ws=S1, bytes=8 * 256 * 4) | change
    assert lib.sgemm_rms_norm_backward_workspace(8, 256) == 8 * 256 * 4
    assert lib.sgemm_rms_norm_backward(8, 256, a["DY"], 256, a["H"], 256, a["tx"], a["W"], a["tw"], a["T"], None, 0,
                                       a["DX"], 256, a["DW"], a["ws"], a["bytes"], None) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_valid_calls_without_gpu_are_unsupported(lib):
    assert product_status(lib) == 3
    assert lib.sgemm_fp8_quantize(8, 256, A0, 0, 256, B0, 8, 256, S0, 2, 1, 128, None) == 3
    assert product_status(lib, K=0, lda=1, ldb=1, ldsa=1, ldsb=1) == 3


def test_tensors_are_checked_before_any_call(sg):
    f8 = torch.zeros(8, 128).to(E4M3)
    one = torch.ones(8, 1)
    with pytest.raises(TypeError, match="2-D tensor"):
        sg.gemm_fp8(torch.zeros(8, 128), one, f8, one, transB=True)
    with pytest.raises(TypeError, match="CUDA"):
        sg.gemm_fp8(f8, one, f8, one, transB=True)
    with pytest.raises(TypeError, match="2-D tensor"):
        sg.quantize_fp8(torch.zeros(8))
    with pytest.raises(TypeError, match="CUDA"):
        sg.rms_norm_fp8(torch.zeros(2, 8), torch.ones(8))


@gpu
def test_tensors_that_do_not_fit_are_refused(sg):
    q, s = sg.quantize_fp8(torch.randn(300, 256, device="cuda"))
    w, t = sg.quantize_fp8(torch.randn(200, 256, device="cuda"), (B, B))
    with pytest.raises(ValueError, match="inner dimensions"):
        sg.gemm_fp8(q, s, w, t)
    with pytest.raises(ValueError, match="A_scale"):
        sg.gemm_fp8(q, s[:299], w, t, transB=True)
    with pytest.raises(ValueError, match="B_scale"):
        sg.gemm_fp8(q, s, w, t[:1], transB=True)
    with pytest.raises(ValueError, match="beta"):
        sg.gemm_fp8(q, s, w, t, transB=True, beta=1.0)
    with pytest.raises(ValueError, match="C must be"):
        sg.gemm_fp8(q, s, w, t, torch.zeros(300, 201, device="cuda"), transB=True)
    with pytest.raises(TypeError, match="out_dtype"):
        sg.gemm_fp8(q, s, w, t, transB=True, out_dtype=torch.float64)
    with pytest.raises(TypeError):
        sg.quantize_fp8(torch.randn(4, 4, device="cuda"), dtype=torch.uint8)
    with pytest.raises(ValueError, match="block"):
        sg.quantize_fp8(torch.randn(4, 4, device="cuda"), block=(128, 64))
    with pytest.raises(ValueError, match="unit column stride"):
        sg.quantize_fp8(torch.randn(8, 8, device="cuda")[:, ::2])
    with pytest.raises(ValueError, match="overlapping"):
        sg.quantize_fp8(torch.randn(1, 8, device="cuda").expand(4, 8))
    with pytest.raises(ValueError, match="residual"):
        sg.rms_norm_fp8(torch.randn(4, 8, device="cuda"), torch.ones(8, device="cuda"), torch.randn(3, 8, device="cuda"))
    with pytest.raises(ValueError, match="weight"):
        sg.rms_norm_fp8(torch.randn(4, 8, device="cuda"), torch.ones(9, device="cuda"))
    with pytest.raises(sg.SgemmError, match="overlap"):
        x = torch.randn(128, 128, device="cuda")
        sg.sgemm_fp8_quantize(128, 128, x.data_ptr(), 0, 128, x.data_ptr(), 8, 128, s.data_ptr(), 1, 1, 128)


# ---------------------------------------------------------------- the example
@gpu
def test_example_learns_and_answers(clean_status):
    """40 steps bring the error to below a tenth (it falls until the weights' 8 bits limit it: their rounding error,
    up to 2^-4 of a value and 2^-5.8 in the mean square, is 2e-2 of the output's unit variance at most), and tokens
    one at a time give the rows that they give together up to BF16's last bit."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_layer.py")
    spec = importlib.util.spec_from_file_location("fp8_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer, _, errors = example.train(tokens=1024, inputs=256, outputs=384, steps=40)
    assert errors[-1] < errors[0] / 10
    one, together = example.decode(layer)
    assert ((one.float() - together.float()).abs() <= 2.0 ** -7 * together.float().abs() + 1e-6).all()
