"""The norm and its gradient at sizes for every shape of a row (threads, chunks
a thread, rows a CTA), and with so many rows that a CTA of the gradient takes
its ring of copied rows several times round.  The checks and their tolerances
are those of test_fp8.py; the sums here are no longer: a CTA adds up to 24 rows
and then one thread up to 38 CTAs' sums.
"""
import pytest
import torch

from . import test_fp8 as base
from .test_fp8 import FLOATS, sg  # noqa: F401

pytestmark = pytest.mark.gpu

# forward: eight rows a CTA of one, two and four chunks a thread; one row of one, two and four; longer rows in segments
NORM = [(2000, 250), (700, 264), (700, 512), (613, 1024), (40, 2100), (305, 4097), (700, 8192), (3, 8200), (310, 16384),
        (320, 16392)]
# backward: one, two and four chunks a thread, longer rows; more rows than CTAs many times over
GRADIENT = [(7400, 250), (5000, 1032), (4000, 2048), (2500, 2056), (1500, 5000), (2500, 8192), (700, 8200), (613, 16384),
            (700, 16392)]


@pytest.mark.parametrize("shape", NORM)
@pytest.mark.parametrize("xtype", FLOATS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(sg, shape, xtype, residual):  # noqa: F811
    base.test_norm(sg, shape, xtype, residual)


@pytest.mark.parametrize("shape", GRADIENT)
@pytest.mark.parametrize("xtype", FLOATS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradient(sg, shape, xtype, residual):  # noqa: F811
    base.test_norm_gradient(sg, shape, xtype, residual)


@pytest.mark.parametrize("shape", [(2000, 1001), (900, 5001), (500, 16001), (700, 20001)])
@pytest.mark.parametrize("xtype", [torch.float32, torch.bfloat16])
def test_gradient_of_rows_off_16_bytes(sg, shape, xtype):  # noqa: F811
    """Rows that are copied by elements take the ring in the same order."""
    h, dy, dh = (torch.randn(shape, generator=base.rng(700 + i), device="cuda").to(xtype) for i in range(3))
    w = torch.randn(shape[1], generator=base.rng(703), device="cuda").to(xtype)
    t = torch.rand(shape[0], generator=base.rng(704), device="cuda")
    up = [base.strided(v, -shape[1] % 16) for v in (dy, h, dh)]
    want = sg.rms_norm_backward(up[0], up[1], w, t, up[2])
    got = sg.rms_norm_backward(base.strided(dy, 7, 1), base.strided(h, 0, 3), w, t, base.strided(dh, 1, 0))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
