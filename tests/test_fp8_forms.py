"""Every form of the 8-bit product's kernel, with every number of CTAs that
share a tile: whole outputs against the product in 64 bits, and bit for bit
where all values and sums are exact.  Each case names the form that it is there
for, and the library says whether that is what runs.

Tolerance (u = 2^-24): 8-bit products are exact; 128 of them are added in 32
bits, where an addition loses at most 2 u of the sum of magnitudes; a block's
sum meets its scale (two roundings) and is added to the running sum, one
rounding a block; the CTAs that share a tile add fewer sums than there are
blocks.  So |err| <= 2 u (128 + blocks + 4) sum |a b| + 4 u (|beta c| + |result|),
and the output is the rounding of a value within that.
"""
import pytest
import torch

from .test_fp8 import B, E4M3, E5M2, U, cdiv, clean_status, operand, rng, sg, strided, within  # noqa: F401

gpu = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
CODE = {F32: 0, BF16: 1, F16: 2}
# transA, transB, blocks of A along M, of B along N
NT, NN, TT = (0, 1, 1, B), (0, 0, 1, B), (1, 1, B, B)       # one scale for 128 columns
TN, NT1 = (1, 0, 1, 1), (0, 1, 1, 1)                        # one for each column

# form, CTAs sharing a tile, layout, M, N, K, more: C's type, beta, C's padding, operands' padding and offset
CASES = [
    # up to 64 rows: the columns of C are the tile's rows, so their scales make no difference to the form
    ("few_16", 1, NT, 9, 5003, 523), ("few_16", 1, NN, 16, 4100, 700), ("few_16", 1, NT1, 3, 4100, 400),
    ("few_16", 2, NT, 1, 5800, 1100), ("few_16", 2, NN, 11, 5803, 931), ("few_16", 2, NT1, 16, 5000, 1038),
    ("few_16", 4, NT, 1, 4096, 4096), ("few_16", 4, NN, 13, 301, 1029), ("few_16", 4, NT1, 16, 1000, 1300),
    ("few_16", 8, NT, 1, 520, 2100), ("few_16", 8, NN, 7, 1000, 4096), ("few_16", 8, NT1, 16, 261, 2500),
    ("few_32", 1, NT, 24, 4096, 700), ("few_32", 1, NN, 17, 5003, 523),
    ("few_32", 2, NT, 24, 8192, 4096), ("few_32", 2, NN, 21, 5353, 911), ("few_32", 2, NT1, 32, 5004, 924),
    ("few_32", 4, NT, 24, 1000, 1000), ("few_32", 4, NN, 19, 131, 1075),
    ("few_32", 8, NT, 24, 1000, 4096), ("few_32", 8, NN, 32, 257, 3900), ("few_32", 8, NT1, 26, 300, 4634),
    ("few_64", 1, NT, 50, 8192, 1000), ("few_64", 1, NN, 33, 4099, 700),
    ("few_64", 2, NT, 36, 700, 1454), ("few_64", 2, NN, 64, 1001, 1450), ("few_64", 2, NT1, 40, 260, 1434),
    ("few_64", 4, NT, 64, 520, 2100), ("few_64", 4, NN, 42, 1031, 2132),
    ("few_64", 8, NT, 37, 200, 8005), ("few_64", 8, NN, 64, 131, 7900), ("few_64", 8, NT1, 48, 300, 7735),
    # 128 x 64
    ("half", 1, NT, 300, 1001, 300), ("half", 1, NN, 200, 301, 350), ("half", 1, TN, 500, 1001, 329),
    ("half", 2, NT, 1000, 1013, 997), ("half", 2, NN, 1000, 1081, 900), ("half", 2, TN, 1000, 1013, 997),
    ("half", 4, NT, 300, 1000, 2000), ("half", 4, NN, 140, 141, 2100), ("half", 4, TN, 300, 1000, 2000),
    ("half", 4, TT, 260, 520, 1100), ("half", 4, NT1, 100, 1001, 1500),
    # 128 x 128
    ("tile", 1, NT, 700, 2000, 700), ("tile", 1, NN, 1200, 2603, 650), ("tile", 1, TN, 518, 7365, 332),
    ("tile", 2, NT, 512, 4096, 2000), ("tile", 2, NN, 159, 5611, 1229), ("tile", 2, TN, 161, 6305, 956),
    ("tile", 4, NT, 120, 6120, 1344), ("tile", 4, NN, 71, 6111, 1400), ("tile", 4, TN, 100, 5603, 1637),
    ("tile", 4, TT, 70, 6120, 1300),
    # the same of operands that TMA cannot read
    ("loaded", 1, NT, 1200, 2600, 500, dict(pad=1)), ("loaded", 1, NN, 400, 4001, 341, dict(pad=5, offset=3)),
    ("loaded", 1, TN, 1300, 2100, 330, dict(pad=3)),
    ("loaded", 2, NT, 1000, 1013, 997, dict(pad=1)), ("loaded", 2, NN, 1001, 1000, 900, dict(pad=7, offset=1)),
    ("loaded", 2, TN, 1000, 1013, 997, dict(pad=2, offset=1)),
    ("loaded", 4, NT, 300, 520, 1400, dict(pad=1)), ("loaded", 4, NN, 130, 261, 1100, dict(pad=16, offset=1)),
    ("loaded", 4, TN, 300, 520, 1400, dict(pad=1, offset=1)),
    # 256 x 256 on two SMs: several tiles a pair, odd and even numbers of blocks
    ("pair_bulk", 1, NT, 2500, 2568, 1400), ("pair_bulk", 1, NN, 2500, 2568, 1400), ("pair_bulk", 1, TT, 2500, 2568, 1400),
    ("pair_bulk", 1, NT, 4100, 4104, 650), ("pair_bulk", 1, NT, 2300, 2568, 129),
    ("pair_bulk", 1, TN, 2500, 2568, 1400), ("pair_bulk", 1, TN, 4100, 4104, 650), ("pair_bulk", 1, NT1, 2500, 2568, 1100),
    ("pair_bulk", 1, NT, 2500, 2568, 1100, dict(cpad=8)), ("pair_bulk", 1, TN, 2500, 2568, 1100, dict(cpad=8)),
    ("pair", 1, NT, 2500, 2568, 1400, dict(beta=0.5)), ("pair", 1, NN, 2500, 2568, 1100, dict(beta=0.5)),
    ("pair", 1, NT, 4100, 4104, 650, dict(beta=1.0)), ("pair", 1, NT, 2500, 2565, 1100, dict(cpad=3)),
    ("pair", 1, TN, 2500, 2568, 1400, dict(beta=0.5)), ("pair", 1, TN, 4100, 4104, 650, dict(beta=1.0)),
    ("pair", 1, TN, 2500, 2571, 1400), ("pair", 1, NT1, 2500, 2571, 1100, dict(beta=1.0)),
    ("pair_staged", 1, NT, 2500, 2571, 1400), ("pair_staged", 1, NN, 4100, 4103, 650),
    ("pair_staged", 1, TT, 2500, 2571, 1100, dict(beta=0.5)), ("pair_staged", 1, NT, 2500, 2571, 1100, dict(cpad=2)),
]
BASE = 1 << 32   # aligned addresses for the host's query, never dereferenced


def layout_rows(M, N, K, ta, tb):
    return (K if ta else M, M if ta else K), (N if tb else K, K if tb else N)


def settings(case):
    form, split, layout, M, N, K = case[:6]
    more = dict(beta=0.0, cpad=0, pad=0, offset=0) | (case[6] if len(case) > 6 else {})
    return form, split, layout, M, N, K, more


def ident(case):
    return "-".join(str(v) for v in case[:2]) + "-" + "".join(map(str, case[2])) + "-%dx%dx%d" % case[3:6] + \
        "".join(f"-{k}{v}" for k, v in (case[6] if len(case) > 6 else {}).items())


@pytest.mark.parametrize("case", CASES, ids=ident)
@pytest.mark.parametrize("out", [F32, BF16, F16])
def test_the_form_is_the_one_named(sg, case, out):
    form, split, (ta, tb, _, bb), M, N, K, more = settings(case)
    (_, ca), (_, cb) = layout_rows(M, N, K, ta, tb)
    ld = [c + more["pad"] if more["pad"] or more["offset"] else cdiv(c, 16) * 16 for c in (ca, cb)]
    got = sg.sgemm_fp8_select_form(ta, tb, M, N, K, BASE + more["offset"], ld[0], 2 * BASE + more["offset"], ld[1], bb,
                                   more["beta"], 3 * BASE, CODE[out], N + more["cpad"])
    assert got == (form, split)


def test_every_form_has_a_case():
    have = {(c[0], c[1], c[2][3] == 1) for c in CASES}
    want = {(f"few_{n}", s, False) for n in (16, 32, 64) for s in (1, 2, 4, 8)}
    want |= {(f, s, v) for f in ("half", "tile", "loaded") for s in (1, 2, 4) for v in (False, True)}
    want |= {("pair", 1, False), ("pair", 1, True), ("pair_bulk", 1, False), ("pair_bulk", 1, True),
             ("pair_staged", 1, False)}
    assert want <= have


def test_nothing_is_selected_for_what_is_refused(sg):
    good = dict(ta=0, tb=1, M=8, N=16, K=256, A=BASE, lda=256, B=2 * BASE, ldb=256, bb=128, beta=0.0, C=3 * BASE, tc=1, ldc=16)
    assert sg.sgemm_fp8_select_form(*good.values()) is not None
    for bad in (dict(ta=2), dict(M=0), dict(N=-1), dict(K=0), dict(K=1 << 31), dict(lda=255), dict(ldb=255), dict(bb=64),
                dict(tc=8), dict(ldc=15)):
        assert sg.sgemm_fp8_select_form(*(good | bad).values()) is None, bad


def run(sg, case, out, integers=False, alpha=1.0, fa=E4M3, fb=E4M3):
    form, split, (ta, tb, ba, bb), M, N, K, more = settings(case)
    qa, sa, a = operand(M, K, ba, fa, ta == 1, 500, integers, more["pad"], more["offset"])
    qb, sb, b = operand(N, K, bb, fb, tb == 0, 501, integers, more["pad"], more["offset"])
    c = torch.randint(-4, 5, (M, N), generator=rng(502), device="cuda").to(out)
    old = c.double()
    c = strided(c, more["cpad"])
    if more["beta"] == 0:
        c.fill_(float("nan"))   # not read
        old.zero_()
    ran = sg.sgemm_fp8_select_form(ta, tb, M, N, K, qa.data_ptr(), qa.stride(0), qb.data_ptr(), qb.stride(0), bb,
                                   more["beta"], c.data_ptr(), CODE[out], c.stride(0))
    assert ran == (form, split)
    assert sg.gemm_fp8(qa, sa, qb, sb, c, alpha, more["beta"], bool(ta), bool(tb), out) is c
    want = alpha * (a @ b.t()) + more["beta"] * old
    if integers:
        assert torch.equal(c, want.to(out))
    else:
        size = abs(alpha) * (a.abs() @ b.abs().t())
        lim = 2 * U * (128 + cdiv(K, B) + 4) * size + 4 * U * (more["beta"] * old.abs() + want.abs())
        assert within(c, want, lim)
    if more["cpad"]:
        assert torch.isnan(c.as_strided((M, more["cpad"]), c.stride(), c.storage_offset() + N)).all()


@gpu
@pytest.mark.parametrize("case", CASES, ids=ident)
def test_integers_are_exact(sg, clean_status, case):  # noqa: F811
    for out in (F32, BF16, F16):
        run(sg, case, out, integers=True)


@gpu
@pytest.mark.parametrize("case", CASES, ids=ident)
@pytest.mark.parametrize("out", [F32, BF16, F16])
def test_random(sg, clean_status, case, out):  # noqa: F811
    run(sg, case, out, alpha=-0.75)


@gpu
@pytest.mark.parametrize("case", CASES[::3], ids=ident)
def test_mixed_types(sg, clean_status, case):  # noqa: F811
    run(sg, case, F32, fa=E5M2)
    run(sg, case, F32, fb=E5M2, integers=True)


@gpu
@pytest.mark.parametrize("form,layout,M,N,K", [("pair_bulk", NT, 2500, 2568, 1400), ("pair_bulk", TN, 2500, 2568, 1400),
                                               ("pair_staged", NT, 2500, 2571, 1400), ("pair", TN, 2500, 2571, 1400),
                                               ("tile", NT, 120, 6120, 1344), ("half", TN, 300, 1000, 2000)])
def test_a_row_of_nan_stays_one(sg, clean_status, form, layout, M, N, K):  # noqa: F811
    """A NaN scale of one row's block is in that row only, whichever CTA and block it falls to."""
    ta, tb, ba, bb = layout
    qa, sa, _ = operand(M, K, ba, E4M3, ta == 1, 510)
    qb, sb, _ = operand(N, K, bb, E4M3, tb == 0, 511)
    got = [sg.sgemm_fp8_select_form(ta, tb, M, N, K, qa.data_ptr(), qa.stride(0), qb.data_ptr(), qb.stride(0), bb, 0.0,
                                    BASE, 0, N)]
    assert got[0][0] == form
    clean = sg.gemm_fp8(qa, sa, qb, sb, transA=bool(ta), transB=bool(tb), out_dtype=F32)
    row, block = M - 3, cdiv(K, B) - 2
    (sa.t() if ta else sa)[row, block] = float("nan")
    got = sg.gemm_fp8(qa, sa, qb, sb, transA=bool(ta), transB=bool(tb), out_dtype=F32)
    rest = torch.arange(M, device="cuda") != row
    assert torch.isnan(got[row]).all() and torch.equal(got[rest], clean[rest])
