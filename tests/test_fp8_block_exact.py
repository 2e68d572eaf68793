"""Around a gated block's 8-bit products: what has to hold exactly, or nearer than the bounds of test_fp8_block.py let see.
"""
import pytest
import torch

from .test_fp8 import B, E4M3, E5M2, FLOATS, rng, sg, strided  # noqa: F401
from .test_fp8_block import halves, randn, same

gpu = pytest.mark.gpu


# ---------------------------------------------------------------- behind a row's end
@gpu
@pytest.mark.parametrize("cols", [1, 15, 17, 141, 1013])
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("keep", [E4M3, E5M2])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_padding_is_zero_whatever_a_row_ends_on(sg, cols, dtype, keep, bad):  # noqa: F811
    """A last block whose scale is NaN or infinite reaches the row's own columns, not the zeros behind them."""
    rows = 200
    g, u, dy = (randn((rows, cols), 301 + i) for i in range(3))
    g[7, -1] = u[9, -1] = bad
    u[150, -1] = bad
    G, V = sg.quantize_fp8(g, dtype=keep), sg.quantize_fp8(u, dtype=keep)
    assert not torch.isfinite(G[1][7, -1]) and not torch.isfinite(V[1][9, -1])
    for odd in (False, True):
        kept = [tuple(strided(t, 3, 1) for t in k) if odd else k for k in (G, V)]
        o = sg.swiglu_backward_fp8(dy.to(dtype), *kept)
        halves(o, cols)
        wide = o.q_rows.shape[1] // 2
        assert (o.scale_cols.view(2, 2, wide)[:, :, cols:] == 2.0 ** -126).all()
        last = cols // B * B if cols % B else cols - B   # the last block's columns take in the bad rows, the others do not
        assert not torch.isfinite(o.scale_cols[0, last:cols]).any() and torch.isfinite(o.scale_cols[0, :last]).all()
        rows_bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
        rows_bad[[7, 9, 150]] = True
        for at in (0, wide):
            assert torch.isfinite(o.scale_rows[~rows_bad, at // B:(at + wide) // B]).all()


@gpu
@pytest.mark.parametrize("cols", [5, 141, 2101, 16401])
@pytest.mark.parametrize("dtype", FLOATS)
def test_an_infinite_scale_at_a_rows_end_in_the_norms_gradient(sg, cols, dtype):  # noqa: F811
    """h infinite in a row's last block: its mean of dy w h is infinite, and dx has the sign that the formula gives; zeros
    behind the row's end, which that scale would make NaN, are not of the mean."""
    rows = 4
    h = torch.where(torch.arange(cols, device="cuda") % 3 == 0, -1.0, 2.0).repeat(rows, 1)
    h[:, -1] = 1.0
    q, s = sg.quantize_fp8(h)
    first = (cols - 1) // B * B
    q[2, first:] = q[2, first:].float().abs().to(E4M3)
    s[2, -1] = float("inf")
    dy = torch.ones(rows, cols, dtype=dtype, device="cuda")
    w, t = torch.ones(cols, device="cuda"), torch.ones(rows, device="cuda")
    d = sg.sandwich_norm_backward(dy, dy, (q, s), w, w, t, t)
    sign = torch.where(torch.arange(cols, device="cuda") >= first, -1.0, -h[2].sign())
    assert torch.equal(d.dx[2].float(), sign * float("inf"))
    assert torch.isfinite(d.dx[[0, 1, 3]].float()).all()


# ---------------------------------------------------------------- h's checkpoint
@gpu
@pytest.mark.parametrize("keep", [E4M3, E5M2])
@pytest.mark.parametrize("kind", FLOATS)
@pytest.mark.parametrize("cols", [300, 1024, 5000, 8192, 16392])
@pytest.mark.parametrize("few", [False, True])
def test_the_streams_checkpoint_is_its_quantisation(sg, keep, kind, cols, few):  # noqa: F811
    """Bit for bit what the quantiser makes of h, wherever h is known: of an FP32 output, and of a 16-bit one where a is 0 and
    the residual is doubled (h then has the residual's bits, and many of its quotients lie between two 8-bit values; a
    rounded 1 / s is off by enough to leave them for the wrong one)."""
    rows = (8 << 20) // cols
    x = randn((rows, cols), 321, torch.bfloat16 if kind == torch.float32 else kind).to(kind)
    a = torch.zeros_like(x) if few or kind != torch.float32 else randn((rows, cols), 322)
    w = 1 + randn(cols, 323, scale=0.1)
    o = sg.sandwich_norm_fp8(a, x, w, w, residual_scale=2.0, training=True, checkpoint=keep)
    assert torch.equal(o.h, 2 * x) or not few
    for got, want in zip(o.h8, sg.quantize_fp8(o.h, dtype=keep)):
        assert same(got, want)


# ---------------------------------------------------------------- memory
@gpu
@pytest.mark.parametrize("rows", [1, 16, 100])
@pytest.mark.parametrize("gate", ["none", "one", "each"])
def test_a_weights_gradient_holds_no_more_than_the_weights(sg, rows, gate):  # noqa: F811
    """What an optimiser keeps of a small call does not keep da, dx and the workspace as well."""
    cols = 500
    a, x, dy = (randn((rows, cols), 341 + i, torch.bfloat16) for i in range(3))
    w, t = randn(cols, 344), randn(rows, 345).abs()
    g = {"none": None, "one": w, "each": a}[gate]
    d = sg.sandwich_norm_backward(dy, a, x, w, w, t, t, gate=g)
    kept = [d.dweight, d.dpost_weight] + ([d.dgate] if gate == "one" else [])
    for v in kept:
        assert v.untyped_storage().nbytes() <= len(kept) * 2048   # 500 floats, rounded up to the allocator's 512 bytes
        assert all(v.untyped_storage().data_ptr() != m.untyped_storage().data_ptr() for m in (d.da, d.dx))
