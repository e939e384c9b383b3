"""Edges of the training operators: schedules of many short units, rows of huge values.

Bounds as in test_ops.py, whose plain fp64 forms are used.
"""
import pytest
import torch

import matrix_orthogonalising_optimizer_gb300 as pkg
from test_ops import U, check_loss, gen, loss_inputs, randn, within

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.mark.gpu
@pytest.mark.parametrize("n,d,v", [(700, 64, 60000), (1300, 40, 20011), (300, 8, 4096)])
def test_many_short_units(n, d, v):
    """Units of one K slab, up to nine per CTA pair: the slots through which the pair's CTAs
    learn their units are used again while loads of earlier units are still to come."""
    x, w, t, coef = loss_inputs(n, d, v, torch.bfloat16, 17)
    first = None
    for _ in range(5):
        out = pkg.vocab_loss_grad(x, w, t, coef=coef)
        if first is None:
            first = out
            check_loss(x, w, t, coef, out)
        assert all(torch.equal(a, b) for a, b in zip(out, first))
    assert pkg.ops_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows", [("fp32", 2000), ("bf16", 2000), ("fp32", 3)])
def test_norm_backward_of_huge_constant_rows(dtype, rows):
    """Rows of one value of 2^121: n is zero, dx finite.  With 64 columns a row does not
    fill its threads' vectors, and (0 - mean) rstd past its end is beyond fp32."""
    dt = DT[dtype]
    x = torch.full((rows, 64), 2.0 ** 121, device="cuda", dtype=dt)
    dy = randn(gen(3), rows, 64, dt=dt)
    y, mean, rstd = pkg.layer_norm(x)
    assert not y.any() and (mean == 2.0 ** 121).all()
    dx, dw, db = pkg.layer_norm_backward(dy, x, None, mean, rstd)
    want = rstd.double()[:, None] * (dy.double() - dy.double().mean(1, keepdim=True))
    within(dx, want, U[dt] * want.abs() + 2.0 ** -20 * rstd.double()[:, None] * dy.double().abs().amax(1, True), "dx")
    assert not dw.any()
