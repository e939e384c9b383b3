"""Edges of the training operators: schedules of many short units.

Bounds as in test_ops.py, whose plain fp64 forms are used.
"""
import pytest
import torch

import matrix_orthogonalising_optimizer_gb300 as pkg
from test_ops import check_loss, loss_inputs

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
