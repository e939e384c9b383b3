"""Layer norm, gated feed-forward block and vocabulary loss.

CPU: argument refusals, workspace queries.  GPU: every output against a plain
fp64 implementation, element by element, within bounds that follow from the
stated roundings:

- a stored bf16 value is off by at most U = 2^-8 of itself (fp32: 2^-24);
- a product that reads operands rounded to bf16 on the way (h, da, du, dz) is
  off by at most U per rounded operand of sum |a| |b|;
- fp32 accumulation of K terms adds at most (K + 64) 2^-23 of sum |a| |b|
  (2^-23, not 2^-24, per addition: the tensor cores may truncate), six times
  the terms where fp32 matrices run as bf16 parts, whose dropped products stay
  below 2^-22 of sum |a| |b|;
- exponentials, logarithms and activations are good to 2^-18 of themselves.
"""
import math

import pytest
import torch

import matrix_orthogonalising_optimizer_gb300 as pkg
from matrix_orthogonalising_optimizer_gb300 import _lib

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
FN = 2.0 ** -18
TINY = 1e-30


def acc(K, dt):
    """Relative accumulation bound of a K-deep product."""
    return (K + 64) * 2.0 ** -23 if dt == torch.bfloat16 else (6 * K + 64) * 2.0 ** -23 + 2.0 ** -22


def within(got, want, bound, what):
    assert got.shape == want.shape, what
    d = (got.double() - want).abs()
    bad = ~(d <= bound + TINY)
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first {i}: got "
                             f"{float(got.flatten()[i])}, want {float(want.flatten()[i])}, bound "
                             f"{float((bound + 0 * want).flatten()[i])}")


def randn(g, *shape, std=1.0, dt=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---------------------------------------------------------------- refusals (no GPU)

P16 = 1 << 20  # an aligned address that no refused call touches


def err(lib):
    return lib.dmuon_last_error().decode()


def test_layer_norm_refusals(lib):
    def fwd(x=P16, w=P16, y=P16, mean=P16, rows=4, cols=8, dtype=_lib.BF16, eps=1e-5):
        return lib.dmuon_layer_norm_forward(x, w, None, y, mean, mean, rows, cols, dtype, eps, None)

    assert fwd(rows=-1) == _lib.ERR_INVALID_ARG and "rows" in err(lib)
    assert fwd(cols=0) == _lib.ERR_INVALID_ARG
    assert fwd(cols=(1 << 20) + 1) == _lib.ERR_INVALID_ARG
    assert fwd(dtype=2) == _lib.ERR_UNSUPPORTED_DTYPE
    assert fwd(eps=-1.0) == _lib.ERR_INVALID_ARG and "eps" in err(lib)
    assert fwd(eps=float("nan")) == _lib.ERR_INVALID_ARG
    assert fwd(x=None) == _lib.ERR_INVALID_ARG and "x is NULL" in err(lib)
    assert fwd(y=P16 + 8) == _lib.ERR_ALIGN
    assert fwd(w=P16 + 2) == _lib.ERR_ALIGN
    assert fwd(mean=P16 + 2) == _lib.ERR_ALIGN
    assert fwd(rows=0, x=None) == _lib.OK

    need = lib.dmuon_layer_norm_workspace_bytes(4, 8, _lib.BF16)
    assert need >= 4 * 8 * 2

    def bwd(ws=P16, n=need, dx=P16, rstd=P16):
        return lib.dmuon_layer_norm_backward(P16, P16, None, P16, rstd, dx, P16, P16, 4, 8, _lib.BF16, ws, n, None)

    assert bwd(ws=None) == _lib.ERR_NO_WORKSPACE
    assert bwd(ws=P16 + 16) == _lib.ERR_ALIGN
    assert bwd(n=need - 1) == _lib.ERR_WORKSPACE_TOO_SMALL
    assert bwd(dx=None) == _lib.ERR_INVALID_ARG
    assert bwd(rstd=None) == _lib.ERR_INVALID_ARG
    assert lib.dmuon_layer_norm_workspace_bytes(-1, 8, _lib.BF16) == 0


def test_gated_ffn_refusals(lib):
    need = lib.dmuon_gated_ffn_workspace_bytes(4, 64, 128, _lib.BF16, 0)
    back = lib.dmuon_gated_ffn_workspace_bytes(4, 64, 128, _lib.BF16, 1)
    assert 0 < need < back
    # fp32 operands of more than a few rows are packed into bf16 parts
    many = [lib.dmuon_gated_ffn_workspace_bytes(400, 64, 128, t, 0) for t in (_lib.BF16, _lib.FP32)]
    assert many[1] > many[0] + 6 * 3 * 64 * 128

    def fwd(x=P16, y=P16, slope=P16, h=P16, saved=_lib.FP32, tokens=4, dim=64, hidden=128, dtype=_lib.BF16, act=0,
            ws=P16, n=need):
        return lib.dmuon_gated_ffn_forward(x, P16, P16, P16, y, P16, slope, h, saved, tokens, dim, hidden,
                                           dtype, act, ws, n, None)

    for bad in (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(dim=0), dict(hidden=0), dict(hidden=1 << 21)):
        assert fwd(**bad) == _lib.ERR_INVALID_ARG
    assert fwd(dtype=7) == _lib.ERR_UNSUPPORTED_DTYPE
    assert fwd(act=2) == _lib.ERR_INVALID_ARG and "activation" in err(lib)
    assert fwd(slope=None) == _lib.ERR_INVALID_ARG and "together" in err(lib)
    assert fwd(h=None) == _lib.ERR_INVALID_ARG
    assert fwd(saved=3) == _lib.ERR_UNSUPPORTED_DTYPE
    assert fwd(saved=_lib.BF16, dtype=_lib.FP32) == _lib.ERR_UNSUPPORTED_DTYPE
    assert fwd(x=None) == _lib.ERR_INVALID_ARG
    assert fwd(y=P16 + 4) == _lib.ERR_ALIGN
    assert fwd(ws=None) == _lib.ERR_NO_WORKSPACE
    assert fwd(ws=P16 + 128) == _lib.ERR_ALIGN
    assert fwd(n=need - 1) == _lib.ERR_WORKSPACE_TOO_SMALL
    assert fwd(tokens=0, ws=None) == _lib.OK

    def bwd(dy=P16, dwd=P16, ws=P16, n=back, saved=_lib.BF16):
        return lib.dmuon_gated_ffn_backward(dy, P16, P16, P16, P16, P16, P16, P16, saved, P16, P16, P16, dwd, 4, 64,
                                            128, _lib.BF16, ws, n, None)

    assert bwd(saved=-1) == _lib.ERR_UNSUPPORTED_DTYPE

    assert bwd(dy=None) == _lib.ERR_INVALID_ARG
    assert bwd(dwd=P16 + 2) == _lib.ERR_ALIGN
    assert bwd(n=need) == _lib.ERR_WORKSPACE_TOO_SMALL


def test_vocab_loss_refusals(lib):
    def need(tokens=300, dim=64, vocab=1000, dtype=_lib.BF16, grad=1, budget=0):
        return lib.dmuon_vocab_loss_workspace_bytes(tokens, dim, vocab, dtype, grad, budget)

    assert need(grad=0) < need()
    # a budget bounds the logits held at once; one piece of 256 tokens is the least
    assert need(tokens=100000, budget=1) < need(tokens=100000)
    assert need(tokens=200000, budget=1) == need(tokens=100000, budget=1)

    def call(x=P16, targets=P16, coef=None, loss=P16, dx=P16, dw=P16, tokens=300, dim=64, vocab=1000, dtype=_lib.BF16,
             ws=P16, n=None):
        return lib.dmuon_vocab_loss(x, P16, targets, coef, -100, loss, P16, dx, dw, tokens, dim, vocab, dtype, 0, ws,
                                    need() if n is None else n, None)

    for bad in (dict(tokens=-1), dict(dim=0), dict(vocab=0), dict(vocab=(1 << 22) + 1), dict(dw=None), dict(dx=None),
                dict(x=None), dict(targets=None), dict(loss=None)):
        assert call(**bad) == _lib.ERR_INVALID_ARG, bad
    assert call(dtype=-1) == _lib.ERR_UNSUPPORTED_DTYPE
    assert call(targets=P16 + 4) == _lib.ERR_ALIGN
    assert call(dw=P16 + 8) == _lib.ERR_ALIGN
    assert call(coef=P16 + 2) == _lib.ERR_ALIGN
    assert call(ws=None) == _lib.ERR_NO_WORKSPACE
    assert call(n=need() - 1) == _lib.ERR_WORKSPACE_TOO_SMALL


def test_bindings_refuse_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.layer_norm(x)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.gated_ffn(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.vocab_loss(x, x, torch.zeros(4, dtype=torch.int64))


@pytest.mark.gpu
def test_bindings_refuse_mismatches():
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(32, 16, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros(16, 32, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        pkg.layer_norm(x, torch.zeros(8, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        pkg.layer_norm(x.t())
    with pytest.raises(_lib_error(), match="dtype"):
        pkg.layer_norm(x.half())
    with pytest.raises(ValueError, match="torch.bfloat16"):
        pkg.gated_ffn(x, w.float(), w, d)
    with pytest.raises(ValueError, match="w_down"):
        pkg.gated_ffn(x, w, w, w)
    with pytest.raises(ValueError, match="activation"):
        pkg.gated_ffn(x, w, w, d, activation="relu")
    with pytest.raises(ValueError, match="int64"):
        pkg.vocab_loss(x, w, t.int())
    with pytest.raises(_lib_error(), match="needed"):
        pkg.vocab_loss(x, w, t, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def _lib_error():
    return _lib.DmuonError


# ---------------------------------------------------------------- layer norm

def norm_reference(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1)
    c = x - mean[..., None]
    rstd = ((c * c).mean(-1) + eps) ** -0.5
    n = c * rstd[..., None]
    y = n * (w.double() if w is not None else 1.0) + (b.double() if b is not None else 0.0)
    return y, mean, rstd, n


NORM_SHAPES = [(1, 1), (1, 768), (3, 7), (5, 64), (2, 1000), (37, 1001), (700, 96), (1300, 2048), (3, 4096),
               (640, 4100), (20, 8192), (9, 12000), (33, 16384), (5, 16400), (3, 40001), (1250, 4096),
               (2000, 96), (1217, 16384), (1500, 8192), (1300, 12288), (5000, 8), (3001, 520),
               (650, 768), (170, 4096), (400, 16384)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_layer_norm(rows, cols, dtype):
    dt = DT[dtype]
    g = gen(rows * 100003 + cols)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * 2 + 3 * torch.randn(rows, 1, generator=g, device="cuda"))
    x = x.to(dt)
    w, b = randn(g, cols, dt=dt), randn(g, cols, dt=dt)
    dy = randn(g, rows, cols, dt=dt)
    eps = 1e-5
    y, mean, rstd = pkg.layer_norm(x, w, b, eps=eps)
    ey, em, er, n = norm_reference(x, w, b, eps)
    # statistics in fp32: a sum of `cols` terms, tree-wise (at most cols/32 + 64 deep)
    k = (cols / 32 + 64) * 2.0 ** -24
    xabs = x.double().abs().mean(-1)
    within(mean, em, k * xabs + 2.0 ** -23 * em.abs(), "mean")
    # rstd: relative error of the sum of squares, and of the mean's error squared
    within(rstd, er, er * (k + 4 * 2.0 ** -23 + (k * xabs * er) ** 2), "rstd")
    wd = w.double().abs()
    within(y, ey, U[dt] * ey.abs() + 2 * (k + 2.0 ** -21) * (n.abs() + (xabs * er)[:, None]) * wd + 2.0 ** -22
           * b.double().abs(), "y")

    dx, dw, db = pkg.layer_norm_backward(dy, x, w, mean, rstd)
    # the backward pass's own formula from the fp32 statistics it is given
    n = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    gr = dy.double() * w.double()
    m1, m2 = gr.mean(1, keepdim=True), (gr * n).mean(1, keepdim=True)
    r = rstd.double()[:, None]
    edx = r * (gr - m1 - n * m2)
    nerr = (x.double().abs() + mean.double().abs()[:, None]) * r * 2.0 ** -23  # error of n from x - mean
    scale = r * (gr.abs() + gr.abs().mean(1, keepdim=True) + n.abs() * (gr * n).abs().mean(1, keepdim=True))
    within(dx, edx, U[dt] * edx.abs() + 2 * (k + 2.0 ** -21) * scale + 2 * r * nerr * (gr * n).abs().mean(1, True)
           + 2 * r * n.abs() * (gr.abs() * nerr).mean(1, True), "dx")
    kr = (rows + 64) * 2.0 ** -24
    edw, edb = (dy.double() * n).sum(0), dy.double().sum(0)
    within(dw, edw, U[dt] * edw.abs() + ((kr + 2.0 ** -21) * (dy.double() * n).abs()
                                         + dy.double().abs() * nerr).sum(0), "dweight")
    within(db, edb, U[dt] * edb.abs() + kr * dy.double().abs().sum(0), "dbias")


@pytest.mark.gpu
def test_layer_norm_without_weight_and_constant_rows():
    x = torch.full((3, 50), 7.25, device="cuda")
    x[1] = 0
    y, mean, rstd = pkg.layer_norm(x, eps=1e-5)
    assert (y == 0).all() and (mean == x[:, 0]).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    dy = torch.randn(3, 50, device="cuda")
    dx, dw, db = pkg.layer_norm_backward(dy, x, None, mean, rstd)
    want = rstd[:, None] * (dy - dy.mean(1, keepdim=True))
    assert torch.allclose(dx, want, atol=1e-3) and (dw == 0).all()
    # a large common offset leaves the variance exact to the rounding of x
    x = 4096.0 + torch.arange(64, device="cuda").float().repeat(2, 1)
    _, mean, rstd = pkg.layer_norm(x, eps=0.0)
    assert torch.allclose(rstd, torch.full_like(rstd, (64 * 64 - 1) / 12.0) ** -0.5, rtol=1e-6)
    # no rows: nothing forward, zero sums backward
    e = torch.empty(0, 24, device="cuda")
    y, mean, rstd = pkg.layer_norm(e)
    dx, dw, db = pkg.layer_norm_backward(e, e, None, mean, rstd)
    assert y.shape == (0, 24) and dx.shape == (0, 24) and not dw.any() and not db.any()
    # one column: the deviation is zero
    y, _, _ = pkg.layer_norm(torch.randn(4, 1, device="cuda"), torch.ones(1, device="cuda"),
                             torch.full((1,), 0.5, device="cuda"))
    assert (y == 0.5).all()


# ---------------------------------------------------------------- gated block

def act64(a, name):
    """act(a), act'(a) and a bound on the terms act' is made of."""
    if name == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s)), s * (1 + a.abs())
    p = torch.special.ndtr(a)
    pdf = torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    return a * p, p + a * pdf, p + a.abs() * pdf


def ffn_inputs(n, d, f, dt, seed):
    g = gen(seed)
    return (randn(g, n, d, dt=dt), randn(g, f, d, std=d ** -0.5, dt=dt), randn(g, f, d, std=d ** -0.5, dt=dt),
            randn(g, d, f, std=f ** -0.5, dt=dt), randn(g, n, d, dt=dt))


FFN_SHAPES = [(1, 64, 128), (1, 1, 1), (2, 72, 200), (17, 128, 96), (129, 64, 257), (257, 200, 384), (300, 101, 333),
              (512, 256, 768), (31, 2048, 512), (5, 64, 5000), (1000, 520, 264), (64, 4096, 64),
              (8, 2056, 104), (16, 40, 1032), (23, 1032, 2000), (32, 8, 8), (9, 520, 7),
              (1500, 64, 1280), (4000, 72, 640), (300, 1300, 1400),
              (7, 1028, 260), (12, 132, 2052), (26, 300, 100), (40, 16384, 72),
              (24, 2560, 1544), (29, 1544, 2560)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,d,f", FFN_SHAPES)
def test_gated_ffn(n, d, f, dtype):
    dt = DT[dtype]
    act = "gelu" if (n + d + f) % 2 else "silu"
    x, wg, wu, wd, dy = ffn_inputs(n, d, f, dt, n * 7 + d * 3 + f)
    save = "compact" if n % 3 == 0 else True
    y, (f_act, f_slope), h_out = pkg.gated_ffn(x, wg, wu, wd, activation=act, save=save)
    assert f_act.dtype == f_slope.dtype == (dt if save == "compact" else torch.float32)
    assert torch.equal(y, pkg.gated_ffn(x, wg, wu, wd, activation=act))
    X, G, UP, D, DY = (t.double() for t in (x, wg, wu, wd, dy))
    u = U[dt]
    ea, eu = X @ G.T, X @ UP.T
    da_, du_ = acc(d, dt) * (X.abs() @ G.abs().T), acc(d, dt) * (X.abs() @ UP.abs().T)
    p, dp, dpb = act64(ea, act)
    h = p * eu
    # |act'| <= 1.13 and |act''| <= 0.8
    perr = FN * p.abs() + 1.2 * da_
    us = U[f_act.dtype]
    within(f_act, p, us * p.abs() + (1 + us) * perr, "act")
    serr = FN * dpb + 0.8 * da_
    within(f_slope, dp * eu, us * (dp * eu).abs() + (1 + us) * (serr * (eu.abs() + du_) + dpb * du_), "slope")
    herr = FN * h.abs() + 1.2 * (da_ * eu.abs() + du_ * p.abs() + da_ * du_)
    within(h_out, h, u * h.abs() + (1 + u) * herr, "h")
    # the operand h is rounded once for bf16
    op = u if dt == torch.bfloat16 else 0.0
    herr = op * h.abs() + (1 + op) * herr
    ey = h @ D.T
    within(y, ey, u * ey.abs() + (1 + u) * (herr @ D.abs().T + acc(f, dt) * (h.abs() @ D.abs().T)), "y")

    dx, dwg, dwu, dwd = pkg.gated_ffn_backward(dy, x, wg, wu, wd, (f_act, f_slope), h_out, activation=act)
    # the backward pass's own formula from the tensors it is given
    h = h_out.double()
    dh = DY @ D
    eh = acc(d, dt) * (DY.abs() @ D.abs())
    da, du = dh * f_slope.double(), dh * f_act.double()
    hb = 0 * h
    dab = (1 + op) * eh * f_slope.double().abs() + (op + FN) * da.abs()
    dub = (1 + op) * eh * f_act.double().abs() + (op + FN) * du.abs()
    for name, got, want, bound in (
            ("dx", dx, da @ G + du @ UP, dab @ G.abs() + dub @ UP.abs()
             + acc(2 * f, dt) * (da.abs() @ G.abs() + du.abs() @ UP.abs())),
            ("dw_gate", dwg, da.T @ X, dab.T @ X.abs() + acc(n, dt) * (da.abs().T @ X.abs())),
            ("dw_up", dwu, du.T @ X, dub.T @ X.abs() + acc(n, dt) * (du.abs().T @ X.abs())),
            ("dw_down", dwd, DY.T @ h, DY.abs().T @ hb + acc(n, dt) * (DY.abs().T @ h.abs()))):
        within(got, want, u * want.abs() + (1 + u) * bound, name)
    assert pkg.ops_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,d,f", [(96, 1024, 1536), (48, 16384, 200), (20, 512, 8192)])
def test_gated_ffn_repeats_bitwise(n, d, f):
    # K deep enough that launches split tiles along it: the sums' order is fixed
    x, wg, wu, wd, dy = ffn_inputs(n, d, f, torch.bfloat16, 5)
    ws = torch.empty(pkg.gated_ffn_workspace(n, d, f, backward=True), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(5):
        ws.random_(0, 255)  # nothing is kept between calls
        y, saved, h = pkg.gated_ffn(x, wg, wu, wd, save=True, workspace=ws)
        out = (y, *saved, h, *pkg.gated_ffn_backward(dy, x, wg, wu, wd, saved, h, workspace=ws))
        if first is None:
            first = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(out, first))


@pytest.mark.gpu
def test_gated_ffn_leading_dimensions():
    x, wg, wu, wd, dy = ffn_inputs(96, 1024, 1536, torch.bfloat16, 5)
    y, _, _ = pkg.gated_ffn(x, wg, wu, wd, save=True)
    y3, _, h3 = pkg.gated_ffn(x.view(4, 24, 1024), wg, wu, wd, save=True)
    assert y3.shape == (4, 24, 1024) and h3.shape == (4, 24, 1536) and torch.equal(y3.view(96, 1024), y)


@pytest.mark.gpu
def test_long_sums_do_not_drift():
    # a weight gradient over 140000 rows: one chain of tensor-core additions that
    # long, each truncated, would drift by 8750 x 2^-24; equal signs make it visible
    n, d, f = 140000, 16, 24
    g = gen(4)
    x = torch.rand(n, d, generator=g, device="cuda").bfloat16()
    dy = torch.rand(n, d, generator=g, device="cuda").bfloat16()
    wg, wu, wd = (torch.rand(*s, generator=g, device="cuda").bfloat16() for s in ((f, d), (f, d), (d, f)))
    _, saved, h = pkg.gated_ffn(x, wg, wu, wd, save=True)
    dwd = pkg.gated_ffn_backward(dy, x, wg, wu, wd, saved, h)[3]
    want = dy.double().T @ h.double()
    # rounding of the result, and half of an eighth of it for the sum
    within(dwd, want, (U[torch.bfloat16] + 2.0 ** -12) * want, "dw_down")


@pytest.mark.gpu
def test_gated_ffn_saturated_and_empty():
    # gates far on both sides: sigmoid reaches 0 and 1 without NaN
    for act in ("silu", "gelu"):
        x = torch.tensor([[300.0, 0, 0, 0, 0, 0, 0, 0], [-300.0, 0, 0, 0, 0, 0, 0, 0]], device="cuda",
                         dtype=torch.bfloat16)
        w = torch.zeros(8, 8, device="cuda", dtype=torch.bfloat16)
        w[:, 0] = 1
        eye = torch.eye(8, device="cuda", dtype=torch.bfloat16)
        y, saved, h = pkg.gated_ffn(x, w, w, eye, activation=act, save=True)
        assert (y[0] == torch.tensor(90000.0, device="cuda").bfloat16()).all() and (y[1] == 0).all()
        dx, dwg, dwu, dwd = pkg.gated_ffn_backward(torch.ones_like(y), x, w, w, eye, saved, h, activation=act)
        assert torch.isfinite(dx).all() and torch.isfinite(dwg).all()
        assert (dx[0, 0] == 4800.0) and (dx[1] == 0).all()  # 8 (u act' + act) = 8 (300 + 300)
    e = torch.empty(0, 8, device="cuda", dtype=torch.bfloat16)
    y, saved, h = pkg.gated_ffn(e, w, w, eye, save=True)
    dx, dwg, dwu, dwd = pkg.gated_ffn_backward(e, e, w, w, eye, saved, h)
    assert y.shape == (0, 8) and not dwg.any() and not dwu.any() and not dwd.any()


# ---------------------------------------------------------------- vocabulary loss

def loss_inputs(n, d, v, dt, seed, ignore=-100, scale=1.0):
    g = gen(seed)
    w = randn(g, v, d, std=0.1, dt=dt)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    x = (torch.randn(n, d, generator=g, device="cuda") * scale
         + 8 * torch.rand(n, 1, generator=g, device="cuda") / (0.01 * d) * w[t].float()).to(dt)
    if n > 2:
        t[torch.rand(n, generator=g, device="cuda") < 0.2] = ignore
        t[0], t[1] = 0, v - 1  # first and last column
    coef = torch.rand(n, generator=g, device="cuda") / n
    return x, w, t, coef


def check_loss(x, w, t, coef, out, ignore=-100):
    """Losses and, when given, gradients of a call against the fp64 formula."""
    dt = x.dtype
    d = x.shape[1]
    loss, lse = out[:2]
    X, W = x.double(), w.double()
    z = X @ W.T
    ez = acc(d, dt) * (X.abs() @ W.abs().T).amax(1)
    want = torch.logsumexp(z, 1)
    keep = t != ignore
    idx = t.clamp(min=0)[:, None]
    zt = z.gather(1, idx)[:, 0]
    fl = FN * (1 + z.abs().amax(1))
    within(lse, want, ez + fl, "lse")
    within(loss, torch.where(keep, want - zt, torch.zeros_like(zt)), 2 * (ez + fl) * keep, "loss")
    if len(out) == 2:
        return
    dx, dw = out[2:]
    c = torch.where(keep, coef.double() if coef is not None else torch.ones_like(zt), torch.zeros_like(zt))[:, None]
    p = torch.softmax(z, 1)
    hot = torch.zeros_like(p).scatter_(1, idx, 1.0)
    dz = c * (p - hot)
    # bf16: exponentials keep 12 bits, those below 2^-31 of their block's largest are dropped,
    # and dz is rounded to bf16; the logits' errors shift p by twice as much
    op = U[dt] + 2.0 ** -12 if dt == torch.bfloat16 else 2.0 ** -22
    drop = 2.0 ** -31 if dt == torch.bfloat16 else 0.0
    dzb = (op + U[dt] ** 2 + FN) * dz.abs() + c * (p * (2 * (ez + fl)[:, None]) + drop)
    edx, edw = dz @ W, dz.T @ X
    u = U[dt]
    within(dx, edx, u * edx.abs() + (1 + u) * (dzb @ W.abs() + acc(w.shape[0], dt) * (dz.abs() @ W.abs())), "dx")
    within(dw, edw, u * edw.abs() + (1 + u) * (dzb.T @ X.abs() + acc(len(t), dt) * (dz.abs().T @ X.abs())), "dweight")


LOSS_SHAPES = [(1, 64, 1), (1, 64, 1000), (3, 1, 5), (2, 8, 129), (17, 100, 255), (130, 64, 1003), (257, 136, 640),
               (300, 512, 10007), (5, 2048, 700), (600, 72, 128), (8, 40, 33), (16, 1032, 4099), (32, 264, 1000),
               (9, 2052, 70), (27, 36, 3001), (40, 16384, 300)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,d,v", LOSS_SHAPES)
def test_vocab_loss(n, d, v, dtype):
    dt = DT[dtype]
    x, w, t, coef = loss_inputs(n, d, v, dt, n + d + v)
    check_loss(x, w, t, None, pkg.vocab_loss(x, w, t))
    check_loss(x, w, t, coef, pkg.vocab_loss_grad(x, w, t, coef=coef))
    assert pkg.ops_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_vocab_loss_in_pieces(dtype):
    # a budget of one 256-token piece: four pieces, dW summed in fp32 across them
    dt = DT[dtype]
    x, w, t, coef = loss_inputs(900, 96, 777, dt, 3)
    out = pkg.vocab_loss_grad(x, w, t, coef=coef, budget=1)
    check_loss(x, w, t, coef, out)
    # (not bitwise equal to one piece: how tiles split K depends on their number)
    check_loss(x, w, t, coef, pkg.vocab_loss_grad(x, w, t, coef=coef))
    check_loss(x, w, t, None, pkg.vocab_loss(x, w, t, budget=1))


@pytest.mark.gpu
def test_vocab_loss_targets():
    x, w, t, coef = loss_inputs(40, 64, 500, torch.bfloat16, 9)
    # nothing counted: no loss, no gradient
    none = torch.full_like(t, -100)
    loss, lse, dx, dw = pkg.vocab_loss_grad(x, w, none)
    assert not loss.any() and not dx.any() and not dw.any() and torch.isfinite(lse).all()
    # another ignore index, and a target it shadows
    t7 = torch.where(t == -100, torch.full_like(t, 7), t)
    check_loss(x, w, t7, coef, pkg.vocab_loss_grad(x, w, t7, coef=coef, ignore_index=7), ignore=7)
    # targets outside the vocabulary: NaN loss, no gradient, other rows untouched
    bad = t.clone()
    bad[3], bad[4] = 500, -1
    loss, lse, dx, dw = pkg.vocab_loss_grad(x, w, bad, coef=coef)
    assert loss[3:5].isnan().all() and not dx[3:5].any()
    good = t.clone()
    good[3:5] = -100
    rest = torch.arange(40, device="cuda")
    rest = rest[(rest != 3) & (rest != 4)]
    ref = pkg.vocab_loss_grad(x, w, good, coef=coef)
    assert torch.equal(loss[rest], ref[0][rest]) and torch.equal(dx, ref[2]) and torch.equal(dw, ref[3])
    # no tokens
    loss, lse, dx, dw = pkg.vocab_loss_grad(x[:0], w, t[:0])
    assert loss.shape == (0,) and dx.shape == (0, 64) and not dw.any()


@pytest.mark.gpu
def test_vocab_loss_large_logits():
    # logits of +-1e4: the blocks' maxima are far apart, probabilities are 0 or 1
    x = torch.zeros(3, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(1000, 64, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = 100.0
    w[700, 0] = 100.0
    w[13, 0] = -100.0
    t = torch.tensor([700, 13, 5], device="cuda")
    loss, lse, dx, dw = pkg.vocab_loss_grad(x, w, t)
    assert torch.equal(lse, torch.full((3,), 1e4, device="cuda"))
    assert torch.equal(loss, torch.tensor([0.0, 2e4, 1e4], device="cuda"))
    assert not dx[0].any() and dx[1, 0] == 200.0 and dx[2, 0] == 100.0
    assert dw[700, 0] == 200.0 and dw[13, 0] == -100.0 and dw[5, 0] == -100.0 and not dw[6].any()


@pytest.mark.gpu
@pytest.mark.parametrize("n,d,v", [(70, 1024, 2049), (70, 16384, 1000), (12, 256, 4000)])
def test_vocab_loss_repeats_bitwise(n, d, v):
    x, w, t, coef = loss_inputs(n, d, v, torch.bfloat16, 21)
    ws = torch.empty(pkg.vocab_loss_workspace(n, d, v, grad=True), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(4):
        ws.random_(0, 255)
        out = pkg.vocab_loss_grad(x, w, t, coef=coef, workspace=ws)
        if first is None:
            first = [o.clone() for o in out]
        assert all(torch.equal(a, b) for a, b in zip(out, first))


# ---------------------------------------------------------------- offsets past 2^31, alignment

@pytest.mark.gpu
def test_offsets_past_32_bits():
    # the last rows of tensors of more than 2^31 elements equal the same rows alone,
    # within the roundings of two different kernels
    free = torch.cuda.mem_get_info()[0]
    if free < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    g = gen(6)
    rows, cols = 140000, 16384
    x = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    x[-4:] = randn(g, 4, cols)
    x[:-4] = 1.0
    dy = torch.zeros_like(x)
    dy[-4:] = randn(g, 4, cols)
    y, mean, rstd = pkg.layer_norm(x)
    dx, dw, db = pkg.layer_norm_backward(dy, x, None, mean, rstd)
    ys, ms, rs = pkg.layer_norm(x[-4:].clone())
    dxs, dws, dbs = pkg.layer_norm_backward(dy[-4:].clone(), x[-4:].clone(), None, ms, rs)
    assert torch.allclose(y[-4:].float(), ys.float(), rtol=2.0 ** -7, atol=2.0 ** -8)
    assert torch.allclose(dx[-4:].float(), dxs.float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    assert torch.allclose(dw.float(), dws.float(), rtol=2.0 ** -7, atol=2.0 ** -6) and not y[:-4].any()
    del x, dy, y, dx
    n, d, f = 160000, 64, 14336
    x = torch.zeros(n, d, device="cuda", dtype=torch.bfloat16)
    dy = torch.zeros_like(x)
    x[-40:], dy[-40:] = randn(g, 40, d), randn(g, 40, d)
    wg, wu, wd = randn(g, f, d, std=0.1), randn(g, f, d, std=0.1), randn(g, d, f, std=0.01)
    y, saved, h = pkg.gated_ffn(x, wg, wu, wd, save="compact")
    out = pkg.gated_ffn_backward(dy, x, wg, wu, wd, saved, h)
    xs, dys = x[-40:].clone(), dy[-40:].clone()
    ysm, saveds, hs = pkg.gated_ffn(xs, wg, wu, wd, save="compact")
    outs = pkg.gated_ffn_backward(dys, xs, wg, wu, wd, saveds, hs)
    for a, b in ((y[-40:], ysm), (h[-40:], hs), (saved[1][-40:], saveds[1]), (out[0][-40:], outs[0]),
                 *zip(out[1:], outs[1:])):
        # two roundings of operands and one of the result, in norm
        assert float((a.double() - b.double()).norm()) <= 3 * 2.0 ** -8 * float(b.double().norm())
    assert not y[:-40].any() and not out[0][:-40].any()


@pytest.mark.gpu
def test_misaligned_views_are_refused():
    buf = torch.zeros(4 * 16 + 1, dtype=torch.bfloat16, device="cuda")
    x = buf[1:].view(4, 16)  # contiguous, but two bytes past a 16-byte boundary
    w = torch.zeros(32, 16, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros(16, 32, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: pkg.layer_norm(x), lambda: pkg.gated_ffn(x, w, w, d),
                 lambda: pkg.vocab_loss(x, w, torch.zeros(4, dtype=torch.int64, device="cuda"))):
        with pytest.raises(_lib.DmuonError) as e:
            call()
        assert e.value.status == _lib.ERR_ALIGN
    with pytest.raises(ValueError, match="contiguous"):
        pkg.gated_ffn(torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")[:, :16], w, w, d)


# ---------------------------------------------------------------- differences, streams, graphs

@pytest.mark.gpu
def test_gradients_against_differences():
    """fp32 chain norm -> block -> norm -> loss: the directional derivative along each
    gradient against central differences of the loss.  Step e along a unit
    direction: truncation O(e^2), rounding about 2^-22 |L| / e; e = 2^-6 keeps both
    below 2^-9 of a derivative of order one."""
    g = gen(77)
    n, d, f, v = 48, 40, 56, 90
    dt = torch.float32
    p = {"x": randn(g, n, d, dt=dt), "w1": 1 + randn(g, d, std=0.1, dt=dt), "b1": randn(g, d, std=0.1, dt=dt),
         "wg": randn(g, f, d, std=d ** -0.5, dt=dt), "wu": randn(g, f, d, std=d ** -0.5, dt=dt),
         "wd": randn(g, d, f, std=f ** -0.5, dt=dt), "w2": 1 + randn(g, d, std=0.1, dt=dt),
         "b2": randn(g, d, std=0.1, dt=dt), "wv": randn(g, v, d, std=0.3, dt=dt)}
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[5] = -100
    coef = torch.rand(n, generator=g, device="cuda")

    def forward(q, grads=False):
        y1, m1, r1 = pkg.layer_norm(q["x"], q["w1"], q["b1"])
        f1, saved, h = pkg.gated_ffn(y1, q["wg"], q["wu"], q["wd"], save=True)
        z = q["x"] + f1
        y2, m2, r2 = pkg.layer_norm(z, q["w2"], q["b2"])
        if not grads:
            return float((pkg.vocab_loss(y2, q["wv"], t)[0].double() * coef.double()).sum())
        _, _, dy2, dwv = pkg.vocab_loss_grad(y2, q["wv"], t, coef=coef)
        dz, dw2, db2 = pkg.layer_norm_backward(dy2, z, q["w2"], m2, r2)
        dy1, dwg, dwu, dwd = pkg.gated_ffn_backward(dz, y1, q["wg"], q["wu"], q["wd"], saved, h)
        dx, dw1, db1 = pkg.layer_norm_backward(dy1, q["x"], q["w1"], m1, r1)
        return {"x": dx + dz, "w1": dw1, "b1": db1, "wg": dwg, "wu": dwu, "wd": dwd, "w2": dw2, "b2": db2, "wv": dwv}

    grads = forward(p, grads=True)
    e = 2.0 ** -6
    for name, gr in grads.items():
        norm = gr.double().norm()
        direction = (gr.double() / norm).float()
        diff = [forward({**p, name: p[name] + s * e * direction}) for s in (1, -1)]
        slope = (diff[0] - diff[1]) / (2 * e)
        assert abs(slope - float(norm)) <= 2.0 ** -7 * max(float(norm), 1.0), name


@pytest.mark.gpu
def test_operators_on_another_stream_and_in_a_graph():
    x, wg, wu, wd, dy = ffn_inputs(130, 128, 256, torch.bfloat16, 2)
    t = torch.randint(0, 256, (130,), device="cuda")
    ws = torch.empty(max(pkg.gated_ffn_workspace(130, 128, 256, backward=True),
                         pkg.vocab_loss_workspace(130, 128, 256, grad=True)), dtype=torch.uint8, device="cuda")

    def work(stream=None):
        y, m, r = pkg.layer_norm(x, stream=stream)
        z, saved, h = pkg.gated_ffn(y, wg, wu, wd, save=True, workspace=ws, stream=stream)
        loss, _, dz, _ = pkg.vocab_loss_grad(z, wg, t, workspace=ws, stream=stream)
        dyy, *dws = pkg.gated_ffn_backward(dz, y, wg, wu, wd, saved, h, workspace=ws, stream=stream)
        return (loss, pkg.layer_norm_backward(dyy, x, None, m, r, stream=stream)[0], *dws)

    want = [o.clone() for o in work()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = work(stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for o in got:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_example_trains(dtype):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_residual_lm.py")
    spec = importlib.util.spec_from_file_location("train_residual_lm", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.train(steps=60, vocab=500, dim=128, hidden=384, tokens=2000, dtype=DT[dtype])
    # the first loss is near log(vocab); sixty steps at least halve it
    assert abs(losses[0] - math.log(500)) < 1.5 and losses[-1] < 0.5 * losses[0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens", [8, 40])
def test_nan_stays_in_its_row(tokens, dtype):
    """A NaN reaches every result that depends on it, and no other row."""
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(21)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").mul(0.5).to(dt)

    x, dy = rand(tokens, 64), rand(tokens, 64)
    wg, wu, wd, w = rand(96, 64), rand(96, 64), rand(64, 96), rand(200, 64)
    bad = torch.arange(tokens, device="cuda") == 3
    xn, dyn = x.clone(), dy.clone()
    xn[3, 5] = dyn[3, 7] = float("nan")

    def rows(t):
        assert torch.equal(t.isnan().all(1), bad) and torch.equal(t.isnan().any(1), bad)

    for act in ("silu", "gelu"):
        for save in (False, True):
            r = pkg.gated_ffn(xn, wg, wu, wd, activation=act, save=save)
            rows(r[0] if save else r)
        y, saved, h = pkg.gated_ffn(x, wg, wu, wd, activation=act, save=True)
        dx, dwg, dwu, dwd = pkg.gated_ffn_backward(dyn, x, wg, wu, wd, saved, h)
        rows(dx)
        assert dwg.isnan().all() and dwu.isnan().all() and dwd[7].isnan().all() and dwd.isnan().sum() == 96
    targets = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    loss, lse, dx, dw = pkg.vocab_loss_grad(xn, w, targets)
    assert torch.equal(loss.isnan(), bad) and torch.equal(lse.isnan(), bad)
    rows(dx)
    assert dw.isnan().all()


@pytest.mark.gpu
def test_largest_fp32_values():
    """fp32 values next to the largest are not rounded to infinity on their way to the tensor cores."""
    big = torch.finfo(torch.float32).max
    x = torch.zeros(40, 64, device="cuda")
    x[:, 0] = big
    w = torch.zeros(200, 64, device="cuda")
    w[:, 0] = torch.linspace(1, 1.99, 200, device="cuda") * 2.0 ** -126
    _, lse = pkg.vocab_loss(x, w, torch.zeros(40, dtype=torch.int64, device="cuda"))
    z = w[:, 0].double() * big
    # a part of w below the smallest normal number may count as zero: 2^-8 of a logit, all below 8
    assert torch.allclose(lse.double(), torch.logsumexp(z, 0).expand(40), rtol=0, atol=2.0 ** -5 + 2.0 ** -20)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 3, 12, 32])
def test_vocab_loss_grad_of_few_tokens(tokens):
    """A few tokens' gradients are as good as the rounding of the result."""
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(tokens, 1024, generator=g, device="cuda").bfloat16()
    w = (torch.randn(1000, 1024, generator=g, device="cuda") * 0.001).bfloat16()
    targets = torch.arange(tokens, device="cuda") * 7
    # coef (p - 1) halfway between two bf16 values, where a rounding of it costs most
    coef = torch.full((tokens,), 1.005, device="cuda")
    _, _, dx, dw = pkg.vocab_loss_grad(x, w, targets, coef=coef)
    dz = torch.softmax(x.double() @ w.double().T, 1)
    dz[torch.arange(tokens, device="cuda"), targets] -= 1
    dz *= coef.double()[:, None]
    # a rounding to bf16 is off by 2^-8 of the value at most, spread evenly: 2^-8 / sqrt(3) in norm (5 % for the
    # spread of a sample); the exponentials' codes by 2^-12
    for got, want in ((dx, dz @ w.double()), (dw, dz.T @ x.double())):
        assert float((got.double() - want).norm() / want.norm()) <= 1.05 * 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -12
