"""Edges of the training operators: schedules of many short units, rows of huge values,
masked logits, coefficients, status, refusals.

Bounds as in test_ops.py, whose plain fp64 forms are used.
"""
import math
from types import SimpleNamespace

import pytest
import torch

import matrix_orthogonalising_optimizer_gb300 as pkg
from matrix_orthogonalising_optimizer_gb300 import ops
from test_ops import FN, U, check_loss, gen, loss_inputs, randn, within

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


def masked_inputs(tokens, dt, seed):
    """A vocabulary of 640 whose columns 128 to 255 and 512 on (whole statistics blocks of
    every kernel) and 300 to 307 are masked through a feature that is 1 in every token."""
    x, w, t, coef = loss_inputs(tokens, 64, 640, dt, seed)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    mask = torch.zeros(640, dtype=torch.bool, device="cuda")
    mask[128:256] = mask[512:] = mask[300:308] = True
    kept = torch.cumsum(~mask, 0) - 1
    w[mask] = 0.0
    t = torch.where(t >= 0, t % 128, t)  # targets are not masked
    return x, w, t, coef, mask, kept


def check_masked(x, w, t, coef, mask, kept, grads=True):
    """The masked columns have no part in the loss and get no gradient."""
    t2 = torch.where(t >= 0, kept[t.clamp(min=0)], t)
    check_loss(x, w[~mask], t2, None, pkg.vocab_loss(x, w, t))
    loss, lse, dx, dw = pkg.vocab_loss_grad(x, w, t, coef=coef)
    assert not dw[mask].any()
    if grads:
        check_loss(x, w[~mask], t2, coef, (loss, lse, dx, dw[~mask]))
    else:  # dx of feature 0 is 0 times infinity
        check_loss(x, w[~mask], t2, None, (loss, lse))
        out = (loss, lse, dx[:, 1:].contiguous(), dw[~mask])
        assert torch.isfinite(out[2]).all() and torch.isfinite(out[3]).all()
    assert pkg.ops_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [-1e9, -1e10, -1e20, -1e30, "lowest"])
@pytest.mark.parametrize("tokens", [3, 12, 40, 300])
def test_vocab_loss_masked_blocks(tokens, value, dtype):
    """Finite logits far below the others, a whole block of columns of them."""
    x, w, t, coef, mask, kept = masked_inputs(tokens, DT[dtype], 40 + tokens)
    w[mask, 0] = torch.finfo(torch.bfloat16).min if value == "lowest" else value
    check_masked(x, w, t, coef, mask, kept)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,tokens", [("bf16", 3), ("bf16", 12), ("bf16", 40), ("bf16", 300), ("fp32", 3),
                                          ("fp32", 12), ("fp32", 40), ("fp32", 300)])
def test_vocab_loss_infinitely_masked_blocks(dtype, tokens):
    """Logits of -inf: weights of -inf, or for the fp32 products that take a weight apart
    (which such a weight turns into NaN) logits beyond the range."""
    x, w, t, coef, mask, kept = masked_inputs(tokens, DT[dtype], 50 + tokens)
    apart = dtype == "fp32" and tokens > 16
    if apart:
        x[:, 0] = 4.0
    w[mask, 0] = -3e38 if apart else -math.inf
    check_masked(x, w, t, coef, mask, kept, grads=apart)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [3, 12, 40, 300])
def test_vocab_loss_masked_by_the_lowest_fp32_value(tokens):
    x, w, t, coef, mask, kept = masked_inputs(tokens, torch.float32, 40 + tokens)
    w[mask, 0] = torch.finfo(torch.float32).min
    check_masked(x, w, t, coef, mask, kept)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens", [3, 12, 40])
def test_vocab_loss_of_a_row_of_minus_infinity(tokens, dtype):
    """A token without a finite logit has no softmax: NaN, and only in its row; none if it is ignored."""
    dt = DT[dtype]
    x, w, t, _ = loss_inputs(tokens, 64, 512, dt, 70 + tokens)
    t[t < 0] = 5
    x[:, 0] = 0.0
    x[1] = 0.0
    x[1, 0] = 16.0
    w[:, 0] = -3e38
    bad = torch.arange(tokens, device="cuda") == 1
    loss, lse, dx, dw = pkg.vocab_loss_grad(x, w, t)
    assert torch.equal(loss.isnan(), bad) and lse[1] == -math.inf and torch.isfinite(lse[~bad]).all()
    assert dx[1].isnan().all() and torch.isfinite(dx[~bad]).all()
    t[1] = -100
    loss, lse, dx, dw = pkg.vocab_loss_grad(x, w, t)
    assert loss[1] == 0 and not dx[1].any() and torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("tokens", [12, 40])
def test_products_of_the_largest_fp32_value(tokens, sign):
    """1 times the largest fp32 value is that value, whichever kernel multiplies."""
    big = sign * torch.finfo(torch.float32).max
    x = torch.zeros(tokens, 64, device="cuda")
    w = torch.zeros(300, 64, device="cuda")
    x[:, 0] = 1.0
    w[:, 0] = big
    _, lse = pkg.vocab_loss(x, w, torch.zeros(tokens, dtype=torch.int64, device="cuda"))
    assert (lse == big).all()
    # and where it shares its 16-byte group with other values, these stay exact to fp32
    w = torch.randn(300, 64, generator=gen(8), device="cuda")
    w[:, 0] = big
    x = torch.randn(tokens, 64, generator=gen(9), device="cuda")
    x[:, 0] = 0.0
    t = torch.randint(0, 300, (tokens,), generator=gen(10), device="cuda")
    check_loss(x, w * (torch.arange(64, device="cuda") > 0), t, None, pkg.vocab_loss(x, w, t))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [-1e10, -1e30, 1e4, 1e10, "lowest"])
@pytest.mark.parametrize("tokens", [3, 12, 40])
def test_vocab_loss_of_a_wholly_masked_row(tokens, value, dtype):
    """A token whose logits are all the same, far from zero: the loss is log(vocab) and the
    probabilities are 1 / vocab, although lse itself cannot hold log(vocab) beside them."""
    dt = DT[dtype]
    v = 512
    x, w, t, _ = loss_inputs(tokens, 64, v, dt, 60 + tokens)
    t[t < 0] = 5
    x[:, 0] = 0.0
    x[1] = 0.0
    x[1, 0] = 1.0
    w[:, 0] = torch.finfo(dt).min if value == "lowest" else value
    loss, lse, dx, dw = pkg.vocab_loss_grad(x, w, t)
    assert float((loss[1] - math.log(v)).abs()) <= FN * math.log(v)
    assert float((lse[1].double() - w[0, 0].double()).abs()) <= 2.0 ** -23 * float(w[0, 0].abs()) + math.log(v) + 1e-3
    # the gradient of feature 0 of the weights is this token's alone: x is 0 there in the others
    p = torch.full((v,), 1.0 / v, device="cuda", dtype=torch.double)
    p[t[1]] -= 1
    within(dw[:, 0], p, (2 * U[dt] + U[dt] ** 2 + FN + 2.0 ** -12 * (dt == torch.bfloat16)) * p.abs(), "dweight")
    # the other tokens
    rest = torch.arange(tokens, device="cuda") != 1
    check_loss(x[rest], w * (torch.arange(64, device="cuda") > 0), t[rest], None, (loss[rest], lse[rest]))


@pytest.mark.gpu
@pytest.mark.parametrize("coefs", ["1.005", "1/n", "mixed", "late"])
@pytest.mark.parametrize("tokens,budget", [(33, 0), (255, 0), (509, 0), (509, 1), (1021, 0), (9001, 0)])
def test_vocab_loss_grad_of_equal_coefficients(tokens, budget, coefs):
    """One coefficient for all tokens, halfway between two bf16 values: its rounding, the same
    in every token's gradient, would not average out.  The bound is that of a few tokens."""
    g = torch.Generator(device="cuda").manual_seed(32)
    x = torch.randn(tokens, 1024, generator=g, device="cuda").bfloat16()
    w = (torch.randn(1000, 1024, generator=g, device="cuda") * 0.001).bfloat16()
    targets = torch.arange(tokens, device="cuda") * 7 % 1000
    coef = torch.full((tokens,), 1.0 / tokens if coefs == "1/n" else 1.005, device="cuda")
    if coefs == "mixed":  # powers of two apart, some negative, some zero; a NaN where nothing counts
        coef *= 2.0 ** (torch.arange(tokens, device="cuda") % 5) * (1 - 2 * (torch.arange(tokens, device="cuda") % 2))
        coef[::9] = 0.0
        coef[4] = math.nan
        targets[4] = -100
    if coefs == "late":  # nothing counts at first
        coef[:tokens - tokens // 3] = 0.0
        targets[:tokens // 3] = -100
    _, _, dx, dw = pkg.vocab_loss_grad(x, w, targets, coef=coef, budget=budget)
    dz = torch.softmax(x.double() @ w.double().T, 1)
    dz.scatter_add_(1, targets.clamp(min=0)[:, None], -torch.ones(tokens, 1, device="cuda", dtype=torch.double))
    dz *= torch.where(targets >= 0, coef, torch.zeros_like(coef)).double()[:, None]
    for got, want in ((dx, dz @ w.double()), (dw, dz.T @ x.double())):
        assert float((got.double() - want).norm() / want.norm()) <= 1.05 * 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -12


@pytest.mark.gpu
def test_vocab_loss_grad_unusual_coefficients():
    x, w, t, _ = loss_inputs(60, 72, 500, torch.bfloat16, 33)
    zero = torch.zeros(60, device="cuda")
    _, _, dx, dw = pkg.vocab_loss_grad(x, w, t, coef=zero)
    assert not dx.any() and not dw.any()
    for c in (1e-38, 1e-20, 2.0 ** 100):  # dz keeps the range of the coefficients
        coef = torch.full((60,), c, device="cuda")
        check_loss(x, w, t, coef, pkg.vocab_loss_grad(x, w, t, coef=coef))
    # an infinite coefficient stays in its token's dx
    inf = torch.full((60,), 0.5, device="cuda")
    inf[2] = math.inf
    t[2] = 3
    _, _, dx, _ = pkg.vocab_loss_grad(x, w, t, coef=inf)
    ref = pkg.vocab_loss_grad(x, w, t, coef=torch.full((60,), 0.5, device="cuda"))[2]
    rest = torch.arange(60, device="cuda") != 2
    assert not torch.isfinite(dx[2]).any() and torch.equal(dx[rest], ref[rest])


@pytest.mark.gpu
def test_status_waits_for_every_stream():
    x = torch.randn(64, 256, device="cuda")
    side = torch.cuda.Stream()
    pkg.layer_norm(x)  # what a first call loads is loaded
    assert pkg.ops_status() == 0
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
    pkg.layer_norm(x, stream=side)
    assert not side.query()
    assert pkg.ops_status() == 0
    assert side.query()


def test_workspace_of_another_device_is_refused():
    ws = SimpleNamespace(is_cuda=True, device=torch.device("cuda:1"), is_contiguous=lambda: True,
                         data_ptr=lambda: 1 << 20, numel=lambda: 1 << 20, element_size=lambda: 1)
    with pytest.raises(ValueError, match="workspace"):
        ops._space(ws, lambda: 16, torch.device("cuda:0"))


@pytest.mark.gpu
def test_inputs_that_require_gradients_are_refused():
    x = torch.randn(4, 16, device="cuda", dtype=torch.bfloat16)
    w, d = torch.randn(32, 16, device="cuda").bfloat16(), torch.randn(16, 32, device="cuda").bfloat16()
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    p, q = torch.nn.Parameter(w), torch.ones(16, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    calls = [lambda: pkg.layer_norm(x, q), lambda: pkg.gated_ffn(x, p, w, d),
             lambda: pkg.gated_ffn(x, w, p, d, save=True), lambda: pkg.vocab_loss(x, p, t)]
    for call in calls:
        with pytest.raises(ValueError, match="autograd"):
            call()
        with torch.no_grad():
            call()
    # functions that return the gradients take them
    y, mean, rstd = pkg.layer_norm(x, q.detach())
    pkg.layer_norm_backward(x, x, q, mean, rstd)
    pkg.vocab_loss_grad(x, p, t)
