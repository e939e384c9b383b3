"""Head norms with the position rotation, and attention over packed sequences.

CPU: argument refusals, workspace queries.  GPU: every output against a plain fp64
implementation, element by element, within bounds that follow from the roundings:

- a stored bf16 value is off by at most U = 2^-8 of itself (fp32: 2^-24), and so is
  an operand rounded to bf16 on the way (p and ds of bf16 attention; fp32 runs as
  fp32 FMAs, whose operands are not rounded);
- an fp32 sum of K terms is off by at most (K + 64) 2^-23 of the sum of their
  magnitudes (2^-23, not 2^-24, per addition: the tensor cores may truncate);
- an exponential or logarithm is good to 2^-18 of itself, and an error e of its
  argument is a relative error of at most 2 e of the exponential (e < 1/2); the
  argument s - lse is off by its two terms' own errors and three roundings, of s,
  of lse and of their scaled difference.
"""
import ctypes

import pytest
import torch

import matrix_orthogonalising_optimizer_gb300 as pkg
from matrix_orthogonalising_optimizer_gb300 import _lib
from test_ops import FN, P16, TINY, U, err, gen, randn, within

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
OPERAND = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
NEG = float("-inf")


def acc(K):
    return (K + 64) * 2.0 ** -23


# ---------------------------------------------------------------- refusals (no GPU)

def view(p=P16, token=64, head=64):
    return _lib.Heads(p, token, head)


def test_rotary_table_refusals(lib):
    def call(p=P16, positions=8, rotary=64, base=1e4):
        return lib.dmuon_rotary_table(p, positions, rotary, base, None)

    for bad in (dict(positions=-1), dict(positions=(1 << 24) + 1), dict(rotary=0), dict(rotary=63), dict(rotary=258),
                dict(base=0.0), dict(base=-2.0), dict(base=float("nan")), dict(base=float("inf")), dict(p=None)):
        assert call(**bad) == _lib.ERR_INVALID_ARG, bad
    assert call(p=P16 + 4) == _lib.ERR_ALIGN
    assert call(positions=0, p=None) == _lib.OK


def test_qk_norm_rotary_refusals(lib):
    def fwd(q=view(token=512), k=view(token=128), positions=P16, table=P16, rows=100, rotary=64, qw=P16, kw=P16, norm=1,
            eps=1e-6, qo=P16, ko=P16, tokens=4, heads=8, kv=2, dim=64, dtype=_lib.BF16):
        return lib.dmuon_qk_norm_rotary_forward(q, k, positions, table, rows, rotary, 0, qw, kw, norm, eps, qo, ko,
                                                tokens, heads, kv, dim, dtype, None)

    for bad in (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(heads=0), dict(heads=1025), dict(kv=0), dict(dim=0),
                dict(dim=257), dict(rotary=63), dict(rotary=66), dict(rotary=0), dict(rows=0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(norm=0), dict(q=None), dict(q=view(None)), dict(positions=None),
                dict(qo=None), dict(ko=None), dict(k=view(token=63)), dict(q=view(token=512, head=0)),
                dict(q=view(token=-512)), dict(q=view(token=(1 << 36) + 1))):
        assert fwd(**bad) == _lib.ERR_INVALID_ARG, bad
    assert fwd(dtype=2) == _lib.ERR_UNSUPPORTED_DTYPE
    for bad in (dict(q=view(P16 + 1, 512)), dict(qw=P16 + 2), dict(ko=P16 + 8), dict(table=P16 + 4),
                dict(positions=P16 + 4)):
        assert fwd(**bad) == _lib.ERR_ALIGN, bad
    assert fwd(tokens=0, q=None, k=None, positions=None) == _lib.OK

    need = lib.dmuon_qk_norm_rotary_workspace_bytes(4, 8, 2, 64, _lib.BF16)
    assert need >= 2 * 64 * 4
    assert lib.dmuon_qk_norm_rotary_workspace_bytes(4, 8, 2, 300, _lib.BF16) == 0

    def bwd(dq=P16, dqw=P16, norm=1, w=P16, ws=P16, n=need, g=view(token=512)):
        return lib.dmuon_qk_norm_rotary_backward(g, view(token=128), view(token=512), view(token=128), P16, P16, 100, 64,
                                                 0, w, w, norm, 1e-6, dq, P16, dqw, P16, 4, 8, 2, 64, _lib.BF16, ws, n,
                                                 None)

    assert bwd(dq=None) == _lib.ERR_INVALID_ARG
    assert bwd(g=view(token=1)) == _lib.ERR_INVALID_ARG
    assert bwd(norm=0, w=None) == _lib.ERR_INVALID_ARG and "without the norm" in err(lib)
    assert bwd(dqw=P16 + 2) == _lib.ERR_ALIGN
    assert bwd(ws=None) == _lib.ERR_NO_WORKSPACE
    assert bwd(ws=P16 + 64) == _lib.ERR_ALIGN
    assert bwd(n=need - 1) == _lib.ERR_WORKSPACE_TOO_SMALL


def test_attention_refusals(lib):
    def fwd(q=view(token=512), k=view(token=128), v=view(token=128), offsets=P16, sequences=2, o=P16, lse=P16, tokens=8,
            heads=8, kv=2, dim=64, dtype=_lib.BF16, scale=0.125):
        return lib.dmuon_attention_forward(q, k, v, offsets, sequences, o, lse, tokens, heads, kv, dim, dtype, 1, scale,
                                           P16, 1 << 30, None)

    for bad in (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(sequences=0), dict(sequences=(1 << 20) + 1),
                dict(heads=0), dict(heads=1026), dict(kv=3), dict(kv=0), dict(kv=16), dict(dim=0), dict(dim=129),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(offsets=None, sequences=3), dict(q=None), dict(k=view(None)), dict(v=view(token=32)),
                dict(q=view(token=512, head=32)), dict(o=None), dict(lse=None)):
        assert fwd(**bad) == _lib.ERR_INVALID_ARG, bad
    assert fwd(dtype=5) == _lib.ERR_UNSUPPORTED_DTYPE
    for bad in (dict(q=view(P16 + 1, 512)), dict(o=P16 + 2), dict(lse=P16 + 4), dict(offsets=P16 + 4),
                dict(k=view(P16 + 2, 128), dtype=_lib.FP32)):
        assert fwd(**bad) == _lib.ERR_ALIGN, bad
    assert fwd(tokens=0, q=None, o=None) == _lib.OK
    assert "multiple of sequences" in (fwd(offsets=None, sequences=3), err(lib))[1]
    # more blocks than a launch may have
    assert fwd(heads=1024, kv=1024, sequences=1 << 20, q=view(token=1 << 16), k=view(token=1 << 16),
               v=view(token=1 << 16)) == _lib.ERR_INVALID_ARG
    assert lib.dmuon_attention_workspace_bytes(1 << 20, 8, 1024, 1024, 64, _lib.BF16, 1) == 0
    assert lib.dmuon_attention_workspace_bytes(1, 1 << 24, 1024, 1024, 128, _lib.BF16, 1) > 0

    need = lib.dmuon_attention_workspace_bytes(2, 8, 8, 2, 64, _lib.BF16, 1)
    assert need >= 8 * 8 * 4
    # padded copies of rows that are no multiple of 16 bytes
    assert lib.dmuon_attention_workspace_bytes(1, 8, 8, 2, 33, _lib.BF16, 0) >= 8 * (8 + 2 + 2) * 40 * 2
    assert lib.dmuon_attention_workspace_bytes(1, 8, 8, 2, 33, _lib.FP32, 0) == 0
    assert lib.dmuon_attention_workspace_bytes(2, 8, 8, 3, 64, _lib.BF16, 1) == 0

    def bwd(g=view(token=512), o=P16, lse=P16, dk=P16, ws=P16, n=need):
        return lib.dmuon_attention_backward(g, view(token=512), view(token=128), view(token=128), o, lse, P16, 2, P16, dk,
                                            P16, 8, 8, 2, 64, _lib.BF16, 1, 0.125, ws, n, None)

    for bad in (dict(g=None), dict(g=view(token=8)), dict(o=None), dict(lse=None), dict(dk=None)):
        assert bwd(**bad) == _lib.ERR_INVALID_ARG, bad
    assert bwd(dk=P16 + 4) == _lib.ERR_ALIGN
    assert bwd(ws=None) == _lib.ERR_NO_WORKSPACE
    assert bwd(ws=P16 + 16) == _lib.ERR_ALIGN
    assert bwd(n=need - 1) == _lib.ERR_WORKSPACE_TOO_SMALL


def test_python_refuses_cpu_tensors():
    q = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.attention(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.qk_norm_rotary(q, q)
    with pytest.raises(ValueError, match="dimension"):
        pkg.attention(q[0, 0], q, q)


# ---------------------------------------------------------------- head norms and rotation

def turn(x, cos, sin, interleaved):
    half = cos.shape[1]
    y = x.clone()
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y[..., a] = x[..., a] * cos[:, None] - x[..., b] * sin[:, None]
    y[..., b] = x[..., a] * sin[:, None] + x[..., b] * cos[:, None]
    return y


def turn_size(x, cos, sin, interleaved):
    """The magnitudes of an element's two terms, added: |a cos| + |b sin| and |a sin| + |b cos|."""
    c, s = torch.zeros_like(cos), torch.zeros_like(sin)
    x, half = x.abs(), cos.shape[1]
    y = turn(x, cos.abs(), s, interleaved)  # a cos, b cos
    z = turn(x, c, sin.abs(), interleaved).abs()  # b sin, a sin
    e = torch.arange(x.shape[-1], device=x.device) < 2 * half
    return y + torch.where(e, z, 0.0)


ROTARY = [  # tokens, heads, kv_heads, dim, rotary (0: none), interleaved, norm, weights
    (1, 1, 1, 1, 0, False, True, True), (1, 12, 12, 64, 64, False, True, True), (5, 3, 1, 2, 2, True, True, True),
    (37, 8, 2, 128, 128, False, True, True), (130, 6, 3, 80, 34, True, True, True), (33, 4, 4, 96, 64, False, True, False),
    (65, 5, 1, 33, 32, False, True, True), (40, 2, 2, 256, 256, True, True, True), (29, 7, 7, 48, 16, False, True, True),
    (64, 8, 2, 64, 64, True, False, False), (300, 16, 4, 128, 64, False, False, False),
    (700, 32, 8, 128, 128, True, True, True), (17, 3, 3, 16, 16, False, True, True), (9, 2, 2, 250, 100, False, True, True),
]


def rotary_inputs(case, dtype, fused, seed):
    n, h, kv, d, rot, inter, norm, weights = case
    g, dt = gen(seed), DT[dtype]
    if fused:
        q, k, _ = randn(g, n, (h + 2 * kv) * d, dt=dt).split([h * d, kv * d, kv * d], 1)
        q, k = q.view(n, h, d), k.view(n, kv, d)
    else:
        q, k = randn(g, n, h, d, dt=dt), randn(g, n, kv, d, dt=dt)
    q[0, 0] *= 1e-3  # eps counts in this row
    table = pkg.rotary_table(5000, rot) if rot else None
    positions = torch.randint(0, 5000, (n,), generator=g, device="cuda") if rot else None
    qw, kw = ((1 + randn(g, d, std=0.2, dt=torch.float32)).to(dt) for _ in range(2)) if weights else (None, None)
    return g, q, k, positions, table, qw, kw


@pytest.mark.gpu
def test_rotary_table_angles():
    t = pkg.rotary_table(70001, 34, base=500.0).double()
    p = torch.arange(70001, device="cuda", dtype=torch.float64)
    a = p[:, None] * 500.0 ** (-2 * torch.arange(17, device="cuda", dtype=torch.float64) / 34)
    # one fp32 rounding of a value up to 1, and fp64 angles up to 7e4
    within(t, torch.cat([a.cos(), a.sin()], 1), 2.0 ** -25 + 1e-10, "table")


@pytest.mark.gpu
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", ROTARY)
def test_qk_norm_rotary(case, dtype, fused):
    n, h, kv, d, rot, inter, norm, weights = case
    g, q, k, pos, table, qw, kw = rotary_inputs(case, dtype, fused, n + d)
    u, eps, e = U[DT[dtype]], 1e-6, (d + 32) * 2.0 ** -23
    got = pkg.qk_norm_rotary(q, k, pos, table, qw, kw, norm=norm, eps=eps, interleaved=inter)
    dq, dk = randn(g, n, h, d, std=1e-2, dt=q.dtype), randn(g, n, kv, d, std=1e-2, dt=q.dtype)
    back = pkg.qk_norm_rotary_backward(dq, dk, q, k, pos, table, qw, kw, norm=norm, eps=eps, interleaved=inter)
    cs = table[pos].double().chunk(2, 1) if rot else None
    for i, (x, w, dy, name) in enumerate(((q, qw, dq, "q"), (k, kw, dk, "k"))):
        x, dy, w = x.double(), dy.double(), 1.0 if w is None else w.double()
        r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt() if norm else 1.0
        unit = x * r
        y = unit * w
        size = y.abs()
        if rot:
            size, y = turn_size(y, *cs, inter), turn(y, *cs, inter)
        within(got[i], y, u * y.abs() + e * size, f"{name} out")
        dn = turn(dy, cs[0], -cs[1], inter) if rot else dy
        dsize = turn_size(dy, *cs, inter) if rot else dy.abs()
        if norm:
            gr = dn * w
            dot = (gr * unit).mean(-1, keepdim=True)
            dx = r * (gr - unit * dot)
            mag = r * (dsize * abs(w) + unit.abs() * (dsize * abs(w) * unit.abs()).mean(-1, keepdim=True))
            within(back[i], dx, u * dx.abs() + 4 * e * mag, f"d{name}")
            if weights:
                dw = (dn * unit).sum((0, 1))
                size = (dsize * unit.abs()).sum((0, 1))
                within(back[2 + i], dw, u * dw.abs() + (e + acc(n * h)) * size, f"d{name}_weight")
        else:
            within(back[i], dn, u * dn.abs() + e * dsize, f"d{name}")
    if not weights:
        assert back[2] is None and back[3] is None


@pytest.mark.gpu
def test_qk_norm_rotary_positions_outside_and_no_tokens():
    q, k = randn(gen(1), 6, 2, 64), randn(gen(2), 6, 1, 64)
    table = pkg.rotary_table(10, 32)
    pos = torch.tensor([0, 9, 10, -1, 1 << 40, 3], device="cuda")
    for inter in (False, True):
        yq, yk = pkg.qk_norm_rotary(q, k, pos, table, interleaved=inter)
        bad = torch.tensor([False, False, True, True, True, False], device="cuda")
        for y in (yq, yk):
            assert torch.equal(y[..., :32].isnan().all(-1).all(-1), bad)
            assert not y[..., 32:].isnan().any() and not y[~bad].isnan().any()
    w = torch.ones(64, device="cuda", dtype=q.dtype)
    out = pkg.qk_norm_rotary_backward(q[:0], k[:0], q[:0], k[:0], pos[:0], table, w, w)
    assert out[0].shape == (0, 2, 64) and not out[2].any() and not out[3].any()
    assert pkg.qk_norm_rotary(q[:0], k[:0], pos[:0], table)[0].shape == (0, 2, 64)


# ---------------------------------------------------------------- attention

def plain(q, k, v, do, offsets, causal, scale, dt):
    """fp64 outputs and gradients, each with its error bound, of tensors tokens x heads x dim."""
    n, h, d = q.shape
    kv, op, u, dev = k.shape[1], OPERAND[dt], U[dt], q.device
    q, k, v, do = (x.double() for x in (q, k, v, do))

    def like(x):
        return torch.zeros_like(x), torch.zeros_like(x)

    (o, bo), (dq, bq), (dk, bk), (dv, bv) = like(q), like(q), like(k), like(v)
    lse = torch.full((h, n), NEG, dtype=torch.float64, device=dev)
    bl = torch.zeros_like(lse)
    for a, b in zip(offsets, offsets[1:]):
        if a == b:
            continue
        n_seq = b - a
        for head in range(h):
            g = head // (h // kv)
            Q, K, V, D = q[a:b, head], k[a:b, g], v[a:b, g], do[a:b, head]
            s, s_abs = scale * Q @ K.T, scale * Q.abs() @ K.abs().T
            seen = torch.ones(n_seq, n_seq, dtype=torch.bool, device=dev)
            if causal:
                seen = seen.tril()
            s = s.masked_fill(~seen, NEG)
            s_abs = s_abs.masked_fill(~seen, 0)
            L = torch.logsumexp(s, 1)
            p = (s - L[:, None]).exp()
            top = s_abs.amax(1)
            # of a logit: its sum, and the roundings of the argument of the exponential
            e_s = acc(d) * top + 2.0 ** -22 * (top + L.abs())
            e_l = 2 * e_s + FN + acc(n_seq) + 2.0 ** -22 * L.abs()
            lse[head, a:b], bl[head, a:b] = L, e_l
            e_p = (2 * (e_s + e_l) + FN)[:, None]
            O = p @ V
            o[a:b, head] = O
            bo[a:b, head] = (op + e_p + acc(n_seq)) * (p @ V.abs()) + (u + FN) * O.abs()
            dP, dP_abs = D @ V.T, D.abs() @ V.abs().T
            delta, delta_abs = (D * O).sum(1, keepdim=True), (D * O).abs().sum(1, keepdim=True)
            e_delta = (D.abs() * bo[a:b, head]).sum(1, keepdim=True) + acc(d) * delta_abs
            ds = p * (dP - delta)
            b_ds = p * (e_p * (dP_abs + delta_abs) + acc(d) * dP_abs + e_delta) + (op + 2.0 ** -22) * ds.abs()
            size = ds.abs() + b_ds
            dq[a:b, head] = scale * ds @ K
            bq[a:b, head] = scale * (b_ds + acc(n_seq) * size) @ K.abs() + u * dq[a:b, head].abs()
            dk[a:b, g] += scale * ds.T @ Q
            bk[a:b, g] += scale * (b_ds + acc(n_seq * h // kv) * size).T @ Q.abs()
            dv[a:b, g] += p.T @ D
            bv[a:b, g] += (p * (op + e_p + acc(n_seq * h // kv))).T @ D.abs()
    bk += u * dk.abs()
    bv += u * dv.abs()
    return {"o": (o, bo), "lse": (lse, bl), "dq": (dq, bq), "dk": (dk, bk), "dv": (dv, bv)}


def inputs(offsets, n, h, kv, d, dtype, fused, seed):
    """Queries, keys, values and the outputs' gradient; NaN in the rows of no sequence."""
    g, dt = gen(seed), DT[dtype]
    if fused:
        q, k, v = randn(g, n, (h + 2 * kv) * d, dt=dt).split([h * d, kv * d, kv * d], 1)
        q, k, v = q.view(n, h, d), k.view(n, kv, d), v.view(n, kv, d)
        do = randn(g, h, n, d, std=1e-2, dt=dt).transpose(0, 1)
    else:
        q, k, v = randn(g, n, h, d, dt=dt), randn(g, n, kv, d, dt=dt), randn(g, n, kv, d, dt=dt)
        do = randn(g, n, h, d, std=1e-2, dt=dt)
    q *= 1.5
    out = torch.ones(n, dtype=torch.bool, device="cuda")
    out[offsets[0]:offsets[-1]] = False
    for x in (q, k, v, do):
        x[out] = float("nan")
    return q, k, v, do, out


def check(q, k, v, do, offsets, causal, out, scale=None, given=None, what=""):
    """given: the offsets argument (default: the list as a tensor)."""
    off = torch.tensor(offsets, device="cuda") if given is None else given
    off = None if isinstance(off, str) else off
    o, lse = pkg.attention(q, k, v, off, causal=causal, scale=scale)
    dq, dk, dv = pkg.attention_backward(do, q, k, v, o, lse, off, causal=causal, scale=scale)
    d = q.shape[-1]
    want = plain(*(x.flatten(0, -3) for x in (q, k, v, do)), offsets, causal, d ** -0.5 if scale is None else scale, q.dtype)
    got = {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    assert (lse[:, out] == NEG).all()
    for name, (value, bound) in want.items():
        x = got[name] if name == "lse" else got[name].flatten(0, -3)
        if name == "lse":
            x, value, bound = x[:, ~out], value[:, ~out], bound[:, ~out]
        else:
            assert not x[out].any(), name
        within(x, value, bound, f"{what} {name}")
    return got


CASES = [  # offsets, tokens, heads, kv_heads, dim
    ([0, 1], 1, 1, 1, 64), ([0, 37], 37, 12, 12, 64), ([0, 1, 1, 131, 195, 198], 198, 6, 2, 128),
    ([0, 257, 257, 385, 514], 514, 4, 1, 64), ([5, 133, 400], 420, 4, 2, 128), ([0, 128, 256, 384], 384, 2, 2, 128),
    ([3, 3], 70, 3, 1, 64), ([0, 100, 520, 768], 777, 6, 2, 80), ([0, 300], 300, 3, 3, 96), ([0, 200], 211, 8, 1, 16),
    ([0, 150, 321], 321, 2, 1, 33), ([0, 5, 70], 70, 2, 2, 1), ([1, 90], 91, 4, 4, 7), ([0, 640], 640, 2, 1, 104),
    (list(range(0, 101)), 101, 2, 1, 64), (list(range(0, 1200, 3)), 1200, 1, 1, 32), ([0, 1100], 1100, 2, 1, 128),
    ([0, 255, 512, 767], 769, 2, 1, 72), ([0, 129], 129, 16, 16, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[1]}x{c[2]}x{c[4]}-{len(c[0]) - 1}" for c in CASES])
def test_attention(case, dtype, causal, fused):
    offsets, n, h, kv, d = case
    q, k, v, do, out = inputs(offsets, n, h, kv, d, dtype, fused, n + d)
    check(q, k, v, do, offsets, causal, out)
    assert pkg.ops_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("offsets,n,h,kv,d", [([0, 260, 700], 710, 4, 1, 64), ([0, 90, 130], 130, 2, 2, 128),
                                              ([0, 700], 700, 16, 2, 100), ([0, 3, 515], 520, 8, 2, 127),
                                              ([0, 400], 400, 2, 2, 65), ([0, 100, 200, 300], 310, 6, 3, 12)])
def test_attention_rows_off_16_bytes(offsets, n, h, kv, d, causal):
    # bf16 rows that begin at odd elements: of a length that is a multiple of 16 bytes, and of others
    q, k, v, do, out = inputs(offsets, n, h, kv, d, "bf16", False, n)
    x = []
    for y in (q, k, v, do):
        wide = torch.full((n, y.shape[1], d + 5), float("nan"), dtype=y.dtype, device="cuda")
        wide[..., 3:3 + d] = y
        x.append(wide[..., 3:3 + d])
    check(*x, offsets, causal, out)
    assert pkg.ops_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("batch,n", [(1, 130), (3, 64), (2, 257), (5, 1)])
def test_attention_batch_of_equal_sequences(batch, n, dtype):
    g, dt = gen(batch), DT[dtype]
    q, k, v, do = (randn(g, batch, n, x, 64, dt=dt) for x in (4, 2, 2, 4))
    out = torch.zeros(batch * n, dtype=torch.bool, device="cuda")
    offsets = list(range(0, batch * n + 1, n))
    got = check(q, k, v, do, offsets, True, out, scale=0.3, given="none")
    off = torch.tensor(offsets, device="cuda")
    o, lse = pkg.attention(*(x.flatten(0, 1) for x in (q, k, v)), off, scale=0.3)
    assert torch.equal(o, got["o"].flatten(0, 1)) and torch.equal(lse, got["lse"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 33, 128])
def test_attention_of_single_tokens(d, causal, dtype):
    # one key: o is v, dv is do, and dq and dk are exactly 0
    offsets = [0, 1, 1, 2, 3]
    q, k, v, do, out = inputs(offsets, 3, 4, 4, d, dtype, False, d)
    got = check(q, k, v, do, offsets, causal, out)
    assert torch.equal(got["o"], v) and not got["dq"].any() and not got["dk"].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_large_logits_and_growing_maxima(d, dtype):
    # logits up to several hundred whose row maxima grow from tile to tile
    g, dt, n = gen(d), DT[dtype], 700
    q, k, v, do = (randn(g, n, 2, d, dt=dt) for _ in range(4))
    k *= torch.linspace(0.1, 8, n, device="cuda")[:, None, None].to(dt)
    q *= 4
    out = torch.zeros(n, dtype=torch.bool, device="cuda")
    for causal in (True, False):
        check(q, k, v, do, [0, n], causal, out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_sequences_do_not_see_each_other(dtype):
    # one sequence's infinities and NaN leave the others' results as they are, bit for bit
    offsets, n = [0, 70, 200, 333], 340
    off = torch.tensor(offsets, device="cuda")
    for d in (64, 128):
        q, k, v, do, _ = inputs(offsets, n, 4, 2, d, dtype, False, d)
        for causal in (True, False):
            o, lse = pkg.attention(q, k, v, off, causal=causal)
            grads = pkg.attention_backward(do, q, k, v, o, lse, off, causal=causal)
            want = [x.clone() for x in (o, *grads)]
            bad = [x.clone() for x in (q, k, v, do)]
            for i, x in enumerate(bad):
                x[70:200] = (float("inf"), float("nan"), float("-inf"), float("nan"))[i]
            o2, lse2 = pkg.attention(*bad[:3], off, causal=causal)
            got = (o2, *pkg.attention_backward(bad[3], *bad[:3], o2, lse2, off, causal=causal))
            for a, b in zip(got, want):
                assert torch.equal(a[:70], b[:70]) and torch.equal(a[200:], b[200:])
            assert torch.equal(lse2[:, 200:], lse[:, 200:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_against_differences(dtype):
    # the directional derivative of sum(w o) in 64 bits by central differences (h = 1e-4: truncation and
    # rounding below 1e-6 of the terms' sizes) against the kernels' gradients, within their bounds
    offsets, n, h, kv, d = [0, 60, 205], 205, 4, 2, 64
    q, k, v, do, _ = inputs(offsets, n, h, kv, d, dtype, False, 9)
    off = torch.tensor(offsets, device="cuda")
    o, lse = pkg.attention(q, k, v, off)
    grads = pkg.attention_backward(do, q, k, v, o, lse, off)
    want = plain(q, k, v, do, offsets, True, d ** -0.5, q.dtype)
    g = gen(4)
    for i, name in enumerate(("dq", "dk", "dv")):
        x = (q, k, v)[i]
        direction = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            moved = [y.double() for y in (q, k, v)]
            moved[i] = moved[i] + sign * 1e-4 * direction
            ends.append((plain(*moved, do, offsets, True, d ** -0.5, q.dtype)["o"][0] * do.double()).sum())
        slope = (ends[0] - ends[1]) / 2e-4
        tol = (want[name][1] * direction.abs()).sum() + 1e-6 * (want[name][0] * direction).abs().sum()
        assert (grads[i].double() * direction).sum().sub(slope).abs() <= tol, name


@pytest.mark.gpu
def test_python_refusals_on_the_gpu():
    q, k = randn(gen(1), 8, 4, 64), randn(gen(2), 8, 2, 64)
    off = torch.tensor([0, 8], device="cuda")
    for bad in (lambda: pkg.attention(q, k.float(), k), lambda: pkg.attention(q, k, k[:7]),
                lambda: pkg.attention(q, k, k, off.int()), lambda: pkg.attention(q, k, k, off[:1]),
                lambda: pkg.attention(q, k, k, off.cpu()), lambda: pkg.attention(q, k[:, :, ::2], k[:, :, ::2]),
                lambda: pkg.attention(q[..., ::2], k, k), lambda: pkg.qk_norm_rotary(q, k, None, pkg.rotary_table(4, 8)),
                lambda: pkg.qk_norm_rotary(q, k, off, pkg.rotary_table(4, 8)),
                lambda: pkg.attention_backward(q, q, k, k, q, torch.zeros(4, 7, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pkg.DmuonError, match="dim in"):
        pkg.attention(q[..., :0].contiguous(), k[..., :0].contiguous(), k[..., :0].contiguous())
    with pytest.raises(pkg.DmuonError, match="strides"):
        pkg.attention(q, k[:1].expand(8, 2, 64), k)
    with pytest.raises(pkg.DmuonError, match="multiple of kv_heads"):
        pkg.attention(q[:, :3].contiguous(), k, k)
    grad = q.clone().requires_grad_()
    with pytest.raises(ValueError, match="no_grad"):
        pkg.attention(grad, k, k)
    with torch.no_grad():
        pkg.attention(grad, k, k)
