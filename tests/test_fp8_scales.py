"""The 8-bit product with scales whose product nears the ends of FP32's normal
range, and below it, in every kind of form.

Within the range the usual tolerance holds (see test_fp8_forms.py), and each
addition to a subnormal sum may lose half of 2^-149.  Below it, the product of
the two scales is held to half of 2^-149, so a block's part is off by up to
2^-150 times the sum of its unscaled magnitudes besides.
"""
import pytest
import torch

from .test_fp8 import B, E4M3, E5M2, U, cdiv, clean_status, operand, sg, spread, within  # noqa: F401
from .test_fp8_forms import NN, NT, NT1, TN, TT, F32

pytestmark = pytest.mark.gpu

FORMS = [("few_16", NT, 5, 300, 1100, 0), ("few_64", NN, 50, 700, 900, 0), ("half", TN, 300, 520, 1400, 0),
         ("half", TT, 300, 520, 1400, 0), ("tile", NT, 500, 4100, 700, 0), ("tile", TN, 100, 5603, 1637, 0),
         ("loaded", NT, 130, 200, 700, 1), ("pair_bulk", NT, 2500, 2568, 700, 0), ("pair_bulk", TN, 2500, 2568, 700, 0),
         ("pair", NT1, 2500, 2571, 700, 0), ("pair_staged", NN, 2500, 2571, 700, 0)]


def product(sg, form, layout, M, N, K, pad, up_a, up_b, types=(E4M3, E4M3), values=None):
    """(what came, the same in 64 bits, sum of magnitudes, unscaled sum of magnitudes) with scales times 2^up;
    A's second block of 128 is zeros."""
    ta, tb, ba, bb = layout
    out = []
    for outer, block, dtype, inner_rows, up, seed in ((M, ba, types[0], ta == 1, up_a, 600),
                                                      (N, bb, types[1], tb == 0, up_b, 601)):
        q, s, _ = operand(outer, K, block, dtype, inner_rows, seed, pad=pad)
        if values is not None:
            q.copy_((torch.rand(q.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) * 3 - 1.5)
                    .round().mul(values).to(dtype))
        if seed == 600:
            (q[B:2 * B] if inner_rows else q[:, B:2 * B]).view(torch.uint8).zero_()
        s = s * 2.0 ** up
        assert torch.isfinite(s).all() and (s >= 2.0 ** -126).all()
        v, S = (q.t().double(), s.t()) if inner_rows else (q.double(), s)
        out.append((q, s, v, spread(S, block, B, outer, K)))
    (qa, sa, a, SA), (qb, sb, b, SB) = out
    ran = sg.sgemm_fp8_select_form(ta, tb, M, N, K, qa.data_ptr(), qa.stride(0), qb.data_ptr(), qb.stride(0), bb, 0.0,
                                   1 << 32, 0, N)
    assert ran[0] == form
    got = sg.gemm_fp8(qa, sa, qb, sb, transA=bool(ta), transB=bool(tb), out_dtype=F32)
    return got, (a * SA) @ (b * SB).t(), (a * SA).abs() @ (b * SB).abs().t(), a.abs() @ b.abs().t()


def limit(K, want, size):
    return 2 * U * (128 + cdiv(K, B) + 4) * size + 4 * U * want.abs() + (cdiv(K, B) + 2) * 2.0 ** -150


@pytest.mark.parametrize("form,layout,M,N,K,pad", FORMS)
@pytest.mark.parametrize("up", [(-106, 0), (0, -106), (-53, -53)])
def test_least_normal_products_of_scales(sg, clean_status, form, layout, M, N, K, pad, up):  # noqa: F811
    """Scales lie between 2^-10 and 2^-5.5, so their product is 2^-126 or more."""
    got, want, size, _ = product(sg, form, layout, M, N, K, pad, *up)
    assert within(got, want, limit(K, want, size)) and (got != 0).any()


@pytest.mark.parametrize("form,layout,M,N,K,pad", FORMS)
@pytest.mark.parametrize("up", [(120, 17), (17, 120), (69, 68)])
def test_greatest_normal_products_of_scales(sg, clean_status, form, layout, M, N, K, pad, up):  # noqa: F811
    """Scales of up to 2^126 between them, of values of 2^-9 (sums to 2^-11 a block); a block of zeros adds nothing."""
    got, want, size, _ = product(sg, form, layout, M, N, K, pad, *up, values=2.0 ** -9)
    assert torch.isfinite(got).all() and within(got, want, limit(K, want, size)) and (got.abs() > 2.0 ** 100).any()


@pytest.mark.parametrize("form,layout,M,N,K,pad", FORMS)
@pytest.mark.parametrize("types", [(E4M3, E4M3), (E5M2, E4M3), (E5M2, E5M2)])
def test_subnormal_products_of_scales(sg, clean_status, form, layout, M, N, K, pad, types):  # noqa: F811
    got, want, size, plain = product(sg, form, layout, M, N, K, pad, -60, -60, types)
    assert within(got, want, limit(K, want, size) + 2.0 ** -150 * plain) and (got != 0).any()
