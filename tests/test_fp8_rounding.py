"""Bits of the 8-bit quantisers' outputs that a comparison of values leaves open."""
import pytest
import torch

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
FLOATS = [torch.float32, torch.bfloat16, torch.float16]
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    import dense_fp32_matrix_10_gb300 as sg
    return sg


def quantised(sg, x, dtype):
    """Every form's q, by name."""
    qr, _, qc, _ = sg.quantize_fp8_both(x, dtype)
    forms = {"both, rows": qr, "both, columns": qc}
    for block in ((1, 128), (128, 1), (128, 128)):
        forms[block] = sg.quantize_fp8(x, block, dtype)[0]
    return forms


@gpu
@pytest.mark.parametrize("xtype", FLOATS)
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_quantisers_keep_signs(sg, xtype, dtype):
    """The sign of x / s is that of x: of -0, of what rounds to zero, and beside an infinity."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(260, 400, generator=g, device="cuda")
    x[3] = -0.0
    x[:, 5] = -0.0
    x[130:, 130:260] *= torch.exp2(torch.randint(-60, 1, (130, 130), generator=g, device="cuda").float())
    x[140:150, 7] = -0.0
    x[259, 399] = float("inf")
    x = x.to(xtype)
    for name, q in quantised(sg, x, dtype).items():
        keep = torch.isfinite(x)
        assert torch.equal((q.view(torch.uint8) >= 128)[keep], torch.signbit(x)[keep]), name


@gpu
@pytest.mark.parametrize("xtype", FLOATS)
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_quantisers_round_as_a_division(sg, xtype, dtype):
    """q is fp8 of the FP32 quotient x / s.  The quotient is formed to within 2^-46 of x / s before its one rounding to
    32 bits, so it is another number than the rounded x / s at one in 2^22 values, and another 8-bit value only if that
    is next to a midpoint of the 8-bit type as well.  (The product x * (1 / s) alone gives another 8-bit value at one in
    2000 of these in BF16.)"""
    x = torch.randn(640, 2048, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(xtype)
    for (br, bc), both in (((1, 128), (0, 1)), ((128, 1), (2, 3)), ((128, 128), None)):
        got = [sg.quantize_fp8(x, (br, bc), dtype)]
        if both:
            out = sg.quantize_fp8_both(x, dtype)
            got.append((out[both[0]], out[both[1]]))
        for q, s in got:
            full = s.double().repeat_interleave(br, 0).repeat_interleave(bc, 1)
            want = (x.double() / full).float().to(dtype)
            assert torch.equal(q.view(torch.uint8), want.view(torch.uint8)), (br, bc)
