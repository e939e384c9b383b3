"""Attention: each sequence's outputs and gradients as a whole, in the 2-norm.

The element-wise bounds of the other tests add every rounding's worst case up, which for the
gradients is tens of percent of their size in long rows.  Here roundings count as what they
are, independent and at most half a step each: one of relative size up to U has a variance of
at most U^2 / 3 of the value's square, and the variances of a sum's terms add.  With R = 2^-8 /
sqrt(3) for bf16, per row i, key j and head (sums over the elements of a row in | |^2):

  o    R^2 (sum_j p^2 |v_j|^2 + |o|^2)                  p rounded as operand, o as result
  dv   R^2 (sum_i p^2 |do_i|^2 + |dv|^2)
  dq   R^2 (scale^2 sum_j ds^2 |k_j|^2 + |dq|^2) + scale^2 e_i^2 |sum_j p k_j|^2
  dk   R^2 (scale^2 sum_i ds^2 |q_i|^2 + |dk|^2) + scale^2 sum_i e_i^2 p^2 |q_i|^2
  e_i^2 = R^2 |do_i o_i|^2 (element by element): delta = do . o from o as it was rounded;
  0 where delta is the sum of p dp

fp32 arithmetic, of either type: the exponentials' arguments are below 2^6 here, three
roundings of them and the dot products' (sqrt(128) of 2^-24 of partial sums below 2^4 after
scaling) give less than 1e-5 of p; the sums' own roundings are smaller.  So 1e-5 takes the place of R, with
p^2 (dp^2 + delta^2) in the place of ds^2 (they are subtracted) and e_i = 1e-5 |do_i o_i|.

The sum S^2 of a sequence's variances is that of n x heads rows or more: its square root is exceeded
by a factor sqrt(1 + 6 sqrt(2 / (n heads))), six standard deviations of such a sum of squares, by
nothing but a mistake.  Rows that see one key only have dq = 0 and no part in dk.
"""
import math

import pytest
import torch

import matrix_orthogonalising_optimizer_gb300 as pkg
from test_attention import CASES, DT, check, inputs
from test_ops import gen, randn

ROUND = {torch.bfloat16: 2.0 ** -8 / math.sqrt(3), torch.float32: 0.0}
FP32 = 1e-5


def sequence(q, k, v, do, causal, scale, dt, delta_of_o=True):
    """One sequence's outputs and gradients in 64 bits, each with the variance of its error (summed over all)."""
    n, h, d = q.shape
    kv = k.shape[1]
    r2, f2 = ROUND[dt] ** 2, FP32 ** 2
    q, k, v, do = (x.double().transpose(0, 1) for x in (q, k, v, do))
    ks, vs = (x.repeat_interleave(h // kv, 0) for x in (k, v))

    def shared(x):
        return x.view(kv, h // kv, n, -1).sum(1)

    s = scale * q @ ks.transpose(1, 2)
    if causal:
        s = s.masked_fill(~torch.ones(n, n, dtype=torch.bool, device=q.device).tril(), float("-inf"))
    p = s.softmax(-1)
    o = p @ vs
    dp = do @ vs.transpose(1, 2)
    delta = (do * o).sum(-1, keepdim=True)
    one = torch.arange(n, device=q.device) == 0 if causal else torch.full((n,), n == 1, device=q.device)
    ds = (p * (dp - delta)).masked_fill(one[:, None], 0)
    p_ds = p.masked_fill(one[:, None], 0)  # what delta's error goes through
    size = (p_ds.square() * (dp.square() + delta.square()))
    dq, dk, dv = scale * ds @ ks, shared(scale * ds.transpose(1, 2) @ q), shared(p.transpose(1, 2) @ do)
    q2, k2, v2, do2 = (x.square().sum(-1, keepdim=True) for x in (q, ks, vs, do))
    e2 = (do * o).square().sum(-1, keepdim=True) * ((r2 if delta_of_o else 0.0) + f2)
    both = r2 + f2

    def total(x):
        return float(x.sum())

    var = {
        "o": both * (total(p.square() @ v2) + total(o.square())),
        "dv": both * (total(p.square().transpose(1, 2) @ do2) + total(dv.square())),
        "dq": scale ** 2 * (total((r2 * ds.square() + f2 * size) @ k2) + total(e2 * (p_ds @ ks).square()))
        + both * total(dq.square()),
        "dk": scale ** 2 * (total((r2 * ds.square() + f2 * size).transpose(1, 2) @ q2)
                            + total(p_ds.square().transpose(1, 2) @ (e2 * q2))) + both * total(dk.square()),
    }
    exact = {"o": o, "dq": dq, "dk": dk, "dv": dv}
    room = 1 + 6 * math.sqrt(2 / (n * h))
    return {name: (x.transpose(0, 1), math.sqrt(var[name] * room)) for name, x in exact.items()}


def compare(got, q, k, v, do, offsets, causal, scale, delta_of_o=True):
    """Every sequence; got: o, dq, dk, dv."""
    for a, b in zip(offsets, offsets[1:]):
        if a == b:
            continue
        want = sequence(*(x[a:b] for x in (q, k, v, do)), causal, scale, q.dtype, delta_of_o)
        for x, (name, (value, tol)) in zip(got, want.items()):
            off = float((x[a:b].double() - value).norm())
            assert off <= tol + 1e-14, (name, a, b, off / max(float(value.norm()), 1e-300),
                                        tol / max(float(value.norm()), 1e-300))


def kernels(q, k, v, do, offsets, causal, scale=None):
    off = torch.tensor(offsets, device="cuda")
    o, lse = pkg.attention(q, k, v, off, causal=causal, scale=scale)
    dq, dk, dv = pkg.attention_backward(do, q, k, v, o, lse, off, causal=causal, scale=scale)
    return o, dq, dk, dv


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[1]}x{c[2]}x{c[4]}-{len(c[0]) - 1}" for c in CASES])
def test_each_sequence(case, dtype, causal):
    offsets, n, h, kv, d = case
    q, k, v, do, _ = inputs(offsets, n, h, kv, d, dtype, True, n + d)
    compare(kernels(q, k, v, do, offsets, causal), q, k, v, do, offsets, causal, d ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("offsets,n,h,kv,d", [([0, 260, 700], 710, 4, 1, 64), ([0, 90, 130], 130, 2, 2, 128),
                                              ([0, 700], 700, 16, 2, 100), ([0, 3, 515], 520, 8, 2, 127)])
def test_each_sequence_off_16_bytes(offsets, n, h, kv, d, causal):
    x = inputs(offsets, n, h, kv, d, "bf16", False, n)[:4]
    wide = []
    for y in x:
        w = torch.full((n, y.shape[1], d + 5), float("nan"), dtype=y.dtype, device="cuda")
        w[..., 3:3 + d] = y
        wide.append(w[..., 3:3 + d])
    compare(kernels(*wide, offsets, causal), *wide, offsets, causal, d ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 50])
def test_rows_of_one_key_have_no_logit_gradient(d, dtype):
    # whichever kernel a batch takes: single tokens, and every causal sequence's first row
    for offsets in ([0, 1, 2, 90], [0, 1, 1601, 1602], [0, 2000], [3, 1203, 1204, 2600]):
        n, h, kv = offsets[-1] + 5, 4, 2
        q, k, v, do, _ = inputs(offsets, n, h, kv, d, dtype, False, n)
        for causal in (True, False):
            _, dq, dk, _ = kernels(q, k, v, do, offsets, causal)
            for a, b in zip(offsets, offsets[1:]):
                if b - a == 1:
                    assert not dq[a].any() and not dk[a].any(), (offsets, a, causal)
                elif causal:
                    assert not dq[a].any() and dq[b - 1].any(), (offsets, a)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 50])
def test_short_sequences_beside_a_long_one(d, dtype, causal):
    # an average of more than 512 tokens: bf16 runs all sequences in the kernel of the long ones
    offsets, n, h, kv = [0, 1, 3, 11, 4011, 4012, 4052], 4060, 4, 2
    q, k, v, do, _ = inputs(offsets, n, h, kv, d, dtype, False, d)
    compare(kernels(q, k, v, do, offsets, causal), q, k, v, do, offsets, causal, d ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128, 50])
def test_short_sequences_take_delta_unrounded(d, causal):
    # batches of short sequences: delta is the sum of p dp
    offsets, n, h, kv = [0, 2, 4, 7, 15, 31, 32, 100, 228], 228, 4, 2
    q, k, v, do, _ = inputs(offsets, n, h, kv, d, "bf16", False, d)
    compare(kernels(q, k, v, do, offsets, causal), q, k, v, do, offsets, causal, d ** -0.5, delta_of_o=False)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_along_themselves(dtype, causal):
    # The slope of sum(do o) along each gradient, by central differences in 64 bits from the definition of o
    # alone, is that gradient's norm; the kernels' gradient must give the same up to the tolerance above
    # (Cauchy-Schwarz: the error's norm).  Steps of 1e-4 per element: truncation about 1e-8 / 6
    # times third derivatives of some ten times the slope, rounding 1e-16 |sum(do o)| / 1e-4.
    offsets, n, h, kv, d = [0, 60, 205], 205, 4, 2, 64
    q, k, v, do, _ = inputs(offsets, n, h, kv, d, dtype, False, 9)
    grads = kernels(q, k, v, do, offsets, causal)[1:]

    def loss(x):
        total = 0.0
        for a, b in zip(offsets, offsets[1:]):
            for head in range(h):
                g = head // (h // kv)
                s = d ** -0.5 * x[0][a:b, head] @ x[1][a:b, g].T
                if causal:
                    s = s.masked_fill(~torch.ones_like(s, dtype=torch.bool).tril(), float("-inf"))
                total = total + (do[a:b, head].double() * (s.softmax(-1) @ x[2][a:b, g])).sum()
        return total

    want = [sequence(*(x[a:b] for x in (q, k, v, do)), causal, d ** -0.5, q.dtype) for a, b in zip(offsets, offsets[1:])]
    for i, name in enumerate(("dq", "dk", "dv")):
        exact = torch.cat([w[name][0] for w in want])
        tol = math.sqrt(sum(w[name][1] ** 2 for w in want))
        direction = exact / exact.norm() * math.sqrt(exact.numel())
        ends = []
        for sign in (1, -1):
            moved = [x.double() for x in (q, k, v)]
            moved[i] = moved[i] + sign * 1e-4 * direction
            ends.append(loss(moved))
        slope = float(ends[0] - ends[1]) / 2e-4
        assert abs(slope - float((exact * direction).sum())) <= 1e-5 * slope, name
        limit = tol * float(direction.norm()) + 1e-5 * slope
        assert limit <= 0.02 * slope, name
        assert abs(float((grads[i].double() * direction).sum()) - slope) <= limit, name


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_thousands_of_sequences(dtype, causal):
    # the search for a tile takes a third round from 962 sequences on, a fourth from 29792 on
    lengths = torch.randint(0, 5, (2500,), generator=torch.Generator().manual_seed(3)).tolist()
    offsets = [2]
    for x in lengths:
        offsets.append(offsets[-1] + x)
    q, k, v, do, out = inputs(offsets, offsets[-1] + 3, 1, 1, 32, dtype, False, 3)
    check(q, k, v, do, offsets, causal, out)
    # the same sequences by their offsets and as a batch of equal ones
    batch, n = 40000, 3
    q, k, v, do = (randn(gen(i), batch, n, 2, 16, dt=DT[dtype]) for i in range(4))
    o, lse = pkg.attention(q, k, v, causal=causal)
    want = (o, *pkg.attention_backward(do, q, k, v, o, lse, causal=causal))
    off = torch.arange(batch + 1, device="cuda") * n
    o, lse = pkg.attention(q, k, v, off, causal=causal)
    for a, b in zip((o, *pkg.attention_backward(do, q, k, v, o, lse, off, causal=causal)), want):
        assert torch.equal(a, b)
    assert pkg.ops_status() == 0
