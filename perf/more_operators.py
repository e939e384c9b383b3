"""Attention and what goes directly before it, as measured cases.

The operators of a transformer block beside the feed-forward block: the norm of
each head's queries and keys with the position rotation in the same pass, and
attention over packed sequences with grouped heads, both with their gradients.
Each case is run in two forms on the same inputs: the plain form (elementary
torch operations in 32 bits, rounded once at the end) and, with ``own`` set, the
library's kernels through the package's public calls.  ``exact`` gives the
definition's values in 64 bits.

Formulas, per token t and head h (rows of `dim` elements):

norm and rotation  r = 1 / sqrt(mean(x^2) + eps), n = x r w; the first `rotary`
                   elements of n are taken in pairs (a, b) -- (i, i + rotary / 2),
                   or (2 i, 2 i + 1) interleaved -- and turned by the angle
                   position * base^(-2 i / rotary): a cos - b sin, a sin + b cos
                   dn = the gradient turned back, dw = sum dn x r, g = dn w,
                   dx = r (g - x r mean(g x r))
attention          s_ij = scale q_i k_j over the keys j that i sees (its own sequence;
                   causal: j <= i), lse_i = log sum_j exp s_ij, p = exp(s - lse),
                   o_i = sum_j p_ij v_j; heads / kv_heads heads share a key head
                   delta_i = do_i o_i, ds_ij = p_ij (do_i v_j - delta_i),
                   dq_i = scale sum_j ds_ij k_j, dk_j = scale sum_i ds_ij q_i,
                   dv_j = sum_i p_ij do_i, the last two summed over the heads that share
                   Tokens of no sequence see nothing: o = 0, lse = -inf, no gradients.
"""
import itertools
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 10000.0
_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _rot(name, mode, dtype, tokens, heads, kv_heads, dim, rotary, interleaved=False, norm=True):
    return {"name": name, "op": "qk_norm_rotary", "mode": mode, "dtype": dtype, "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "rotary": rotary, "interleaved": interleaved, "norm": norm}


def _attn(name, mode, dtype, tokens, sequences, heads, kv_heads, dim, causal=True, tail=0):
    """`tokens` rows, of which the last `tail` belong to no sequence (padding of a packed batch)."""
    return {"name": name, "op": "attention", "mode": mode, "dtype": dtype, "tokens": tokens, "sequences": sequences,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "causal": causal, "tail": tail}


def listed():
    return [
        # one token of the small-transformer width: all latency
        _rot("rotary_fwd_token", "forward", "bf16", 1, 12, 12, 64, 64),
        # a training batch of the Llama-3-8B-shaped block, forward and backward
        _rot("rotary_fwd_batch", "forward", "bf16", 16384, 32, 8, 128, 128),
        _rot("rotary_bwd_batch", "backward", "bf16", 16384, 32, 8, 128, 128),
        # fp32, odd everywhere: a part of each row is rotated, in neighbouring pairs
        _rot("rotary_bwd_odd_fp32", "backward", "fp32", 1023, 6, 3, 80, 34, interleaved=True),
        # a short prompt through a small-transformer block: latency
        _attn("attn_fwd_short", "forward", "bf16", 37, 1, 12, 12, 64),
        # scoring one long document with the Llama-3-8B-shaped heads
        _attn("attn_fwd_long", "forward", "bf16", 16384, 1, 32, 8, 128),
        # a batch of ragged texts, both directions visible, small-transformer heads
        _attn("attn_fwd_ragged", "forward", "bf16", 8191, 23, 12, 12, 64, causal=False),
        # a training micro-batch: documents packed into 8192 tokens, Llama-3-8B-shaped heads
        _attn("attn_train_packed", "train", "bf16", 8192, 5, 32, 8, 128, tail=100),
        # one full-length sequence of the same block
        _attn("attn_train_batch", "train", "bf16", 8192, 1, 32, 8, 128),
        # a micro-batch of the small transformer
        _attn("attn_train_small", "train", "bf16", 4096, 4, 12, 12, 64),
        # fp32 training of a small model, odd everywhere
        _attn("attn_train_odd_fp32", "train", "fp32", 777, 3, 6, 2, 80, tail=9),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _head_dim(rng):
    """A head's width: two times in three 64 or 128, else any multiple of 8, now and then any number."""
    u = rng.random()
    return rng.choice((64, 128)) if u < 0.67 else 8 * rng.randint(2, 16) if u < 0.92 else rng.randint(12, 128)


def draw(rng):
    dtype = "bf16" if rng.random() < 0.75 else "fp32"
    op = rng.choice(("qk_norm_rotary", "attention", "attention"))
    while True:
        dim, kv = _head_dim(rng), _log_int(rng, 1, 16)
        heads = kv * rng.choice((1, 1, 2, 3, 4, 8))
        if op == "qk_norm_rotary":
            rotary = dim // 2 * 2 if rng.random() < 0.7 else 2 * rng.randint(1, dim // 2)
            case = _rot(None, rng.choice(("forward", "backward")), dtype, _log_int(rng, 1, 16384), heads, kv, dim, rotary,
                        rng.random() < 0.3, rng.random() < 0.8)
            ok = case["tokens"] * (heads + kv) * dim <= 16384 * 40 * 128
        else:
            tokens = _log_int(rng, 1, 16384)
            sequences = _log_int(rng, 1, 64) if rng.random() < 0.7 else 1
            tail = _log_int(rng, 1, max(1, tokens // 8)) - 1 if rng.random() < 0.3 else 0
            case = _attn(None, rng.choice(("forward", "train")), dtype, tokens, sequences, heads, kv, dim,
                         rng.random() < 0.75, tail)
            longest = max(_lengths(case))
            # below the largest listed cases, also of the plain form, which pads every sequence to the longest
            padded = sequences * heads * longest * longest
            cap = 8192 * 8192 * 32 if case["mode"] == "train" else 16384 * 16384 * 32
            ok = padded <= (cap if dtype == "bf16" else cap // 16) and work(case)["flops"] <= 1.5e12
        if ok:
            del case["name"]
            return case


def _lengths(case):
    """The lengths of the sequences, of the same case always the same: ragged, some of them empty."""
    n, total = case["sequences"], case["tokens"] - case["tail"]
    rng = random.Random(1000003 * case["tokens"] + n)
    weights = [math.exp(rng.gauss(0.0, 0.6)) for _ in range(n)]
    whole = sum(weights)
    cuts = [0, *(min(total, round(total * at / whole)) for at in itertools.accumulate(weights[:-1])), total]
    return [b - a for a, b in zip(cuts, cuts[1:])]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    n, h, kv, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dt)

    s = {"case": case}
    # queries, keys and values as views of one projection's output
    fused = normal(n, (h + 2 * kv) * d)
    q, k, v = fused.split([h * d, kv * d, kv * d], dim=1)
    if case["op"] == "qk_norm_rotary":
        s["q"], s["k"] = q.view(n, h, d), k.view(n, kv, d)
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
            s["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        # packed documents: positions start anew, some of them far into a long context
        start = torch.randint(0, 32768 - n + 1, (1,), generator=g, device="cuda")
        at = torch.arange(n, device="cuda")
        s["positions"] = torch.where(at < n // 2, at, at + start)
        angle = (torch.arange(32768, device="cuda", dtype=torch.float64)[:, None]
                 * BASE ** (-2.0 * torch.arange(case["rotary"] // 2, device="cuda", dtype=torch.float64) / case["rotary"]))
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if case["mode"] == "backward":
            s["dq"], s["dk"] = normal(n, h, d, std=1e-3), normal(n, kv, d, std=1e-3)
    else:
        # normalised queries and keys; some heads look almost evenly, some at few keys
        warm = 1.0 + 2.0 * torch.rand(1, h, 1, generator=g, device="cuda")
        s["q"] = (torch.randn(n, h, d, generator=g, device="cuda") * warm).to(dt)
        s["k"] = normal(n, kv, d)
        s["v"] = v.view(n, kv, d)
        lengths = _lengths(case)
        offsets = [0]
        for x in lengths:
            offsets.append(offsets[-1] + x)
        s["offsets"] = torch.tensor(offsets, dtype=torch.int64, device="cuda")
        s["longest"] = max(lengths)
        if case["mode"] == "train":
            s["do"] = normal(n, h, d, std=1e-3)
    if own:
        import matrix_orthogonalising_optimizer_gb300 as pkg
        s["pkg"] = pkg
        if case["op"] == "qk_norm_rotary":
            nbytes = pkg.qk_norm_rotary_workspace(n, h, kv, d, case["dtype"]) if case["mode"] == "backward" else 0
        else:
            nbytes = pkg.attention_workspace(n, h, kv, d, case["dtype"], sequences=case["sequences"],
                                             backward=case["mode"] == "train")
        s["workspace"] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    form = _own if own else _plain
    return form[case["op"], case["mode"]](state)


def _own_rotary_forward(s):
    c = s["case"]
    q, k = s["pkg"].qk_norm_rotary(s["q"], s["k"], s["positions"], s["table"], s["q_weight"], s["k_weight"],
                                   norm=c["norm"], eps=EPS, interleaved=c["interleaved"])
    return {"q": q, "k": k}


def _own_rotary_backward(s):
    c = s["case"]
    dq, dk, dqw, dkw = s["pkg"].qk_norm_rotary_backward(
        s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["table"], s["q_weight"], s["k_weight"], norm=c["norm"],
        eps=EPS, interleaved=c["interleaved"], workspace=s["workspace"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw} if c["norm"] else {"dq": dq, "dk": dk}


def _own_attention_forward(s):
    o, lse = s["pkg"].attention(s["q"], s["k"], s["v"], s["offsets"], causal=s["case"]["causal"],
                                workspace=s["workspace"])
    return {"o": o, "lse": lse}


def _own_attention_train(s):
    pkg, causal = s["pkg"], s["case"]["causal"]
    o, lse = pkg.attention(s["q"], s["k"], s["v"], s["offsets"], causal=causal, workspace=s["workspace"])
    dq, dk, dv = pkg.attention_backward(s["do"], s["q"], s["k"], s["v"], o, lse, s["offsets"], causal=causal,
                                        workspace=s["workspace"])
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


_own = {("qk_norm_rotary", "forward"): _own_rotary_forward, ("qk_norm_rotary", "backward"): _own_rotary_backward,
        ("attention", "forward"): _own_attention_forward, ("attention", "train"): _own_attention_train}


def _turn(x, cos, sin, interleaved):
    """Rows (tokens x heads x dim) whose leading pairs are turned by angles (tokens x pairs)."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    first, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = first[..., 0::2], first[..., 1::2]
        first = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = first[..., :half], first[..., half:]
        first = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([first, rest], -1)


def _rotary_angles(s):
    return s["table"][s["positions"]].chunk(2, dim=1)


def _plain_rotary_forward(s):
    c = s["case"]
    cos, sin = _rotary_angles(s)

    def one(x, w):
        y = x.float()
        if c["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
        return _turn(y, cos, sin, c["interleaved"]).to(x.dtype)

    return {"q": one(s["q"], s["q_weight"]), "k": one(s["k"], s["k_weight"])}


def _plain_rotary_backward(s):
    c = s["case"]
    cos, sin = _rotary_angles(s)

    def one(dy, x, w):
        dn = _turn(dy.float(), cos, -sin, c["interleaved"])
        if not c["norm"]:
            return dn.to(x.dtype), None
        r = torch.rsqrt(x.float().square().mean(-1, keepdim=True) + EPS)
        unit = x.float() * r
        dw = (dn * unit).sum((0, 1))
        g = dn * w.float()
        return (r * (g - unit * (g * unit).mean(-1, keepdim=True))).to(x.dtype), dw.to(x.dtype)

    dq, dqw = one(s["dq"], s["q"], s["q_weight"])
    dk, dkw = one(s["dk"], s["k"], s["k_weight"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw} if c["norm"] else {"dq": dq, "dk": dk}


def _padded(s):
    """What the plain form pads by: row indices (sequences x longest), which of them are real, and where
    each token's row lies (its sequence, its place there, whether it is in one)."""
    offsets, n = s["offsets"], s["case"]["tokens"]
    at = torch.arange(s["longest"], device=offsets.device)
    real = at < (offsets[1:] - offsets[:-1])[:, None]
    rows = torch.where(real, offsets[:-1, None] + at, 0)
    token = torch.arange(n, device=offsets.device)
    seq = (torch.searchsorted(offsets, token, right=True) - 1).clamp(max=s["case"]["sequences"] - 1)
    place = token - offsets[seq]
    inside = place < offsets[seq + 1] - offsets[seq]
    return rows, real, seq, torch.where(inside, place, 0), inside


def _pad(x, heads, rows, real):
    """tokens x heads x dim -> sequences x key heads x (heads of a group, rows) x dim, padding zero."""
    y = torch.where(real[..., None, None], x[rows].float(), 0.0)
    n, length, h, d = y.shape
    return y.view(n, length, heads, h // heads, d).permute(0, 2, 3, 1, 4).reshape(n, heads, -1, d)


def _unpad(y, heads, seq, place, inside, length):
    """The reverse, for every token; tokens of no sequence zero."""
    n, kv, _, d = y.shape
    y = y.view(n, kv, heads // kv, length, d).permute(0, 3, 1, 2, 4).reshape(n, length, heads, d)
    return torch.where(inside[:, None, None], y[seq, place], 0.0)


def _plain_probabilities(s, pads):
    c = s["case"]
    rows, real = pads[:2]
    n, length, kv, group = c["sequences"], s["longest"], c["kv_heads"], c["heads"] // c["kv_heads"]
    qp, kp, vp = (_pad(s[x], kv, rows, real) for x in "qkv")
    p = torch.matmul(qp, kp.transpose(2, 3)).mul_(c["dim"] ** -0.5).view(n, kv, group, length, length)
    seen = real[:, None, :].expand(n, length, length)
    if c["causal"]:
        seen = seen & torch.ones(length, length, dtype=torch.bool, device=real.device).tril()
    p.masked_fill_(~seen[:, None, None], float("-inf"))
    top = p.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p.sub_(top).exp_()
    whole = p.sum(-1, keepdim=True)
    p.div_(whole)
    lse = (top + whole.log()).view(n, kv, group * length, 1)
    return qp, kp, vp, p.view(n, kv, group * length, length), lse


def _plain_attention_forward(s):
    c, pads = s["case"], _padded(s)
    _, _, vp, p, lse = _plain_probabilities(s, pads)
    back = (c["heads"], *pads[2:], s["longest"])
    o = _unpad(torch.matmul(p, vp), *back).to(s["q"].dtype)
    lse = torch.where(pads[4][:, None], _unpad(lse, *back)[..., 0], float("-inf"))
    return {"o": o, "lse": lse.t().contiguous()}


def _plain_attention_train(s):
    c, pads = s["case"], _padded(s)
    dt, scale = s["q"].dtype, c["dim"] ** -0.5
    qp, kp, vp, p, lse = _plain_probabilities(s, pads)
    back = (c["heads"], *pads[2:], s["longest"])
    shared = (c["kv_heads"], *pads[2:], s["longest"])
    op = torch.matmul(p, vp)
    do = _pad(s["do"], c["kv_heads"], *pads[:2])
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, vp.transpose(2, 3)).sub_((do * op).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, kp).mul_(scale)
    dk = torch.matmul(ds.transpose(2, 3), qp).mul_(scale)
    lse = torch.where(pads[4][:, None], _unpad(lse, *back)[..., 0], float("-inf"))
    return {"o": _unpad(op, *back).to(dt), "lse": lse.t().contiguous(), "dq": _unpad(dq, *back).to(dt),
            "dk": _unpad(dk, *shared).to(dt), "dv": _unpad(dv, *shared).to(dt)}


_plain = {("qk_norm_rotary", "forward"): _plain_rotary_forward, ("qk_norm_rotary", "backward"): _plain_rotary_backward,
          ("attention", "forward"): _plain_attention_forward, ("attention", "train"): _plain_attention_train}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk_norm_rotary":
        return _exact_rotary(s, case)
    return _exact_attention(s, case)


def _rotation(s, case):
    """Per token the dim x dim rotation matrix of its position, as pair indices and their cos and sin."""
    half, at = case["rotary"] // 2, torch.arange(case["rotary"] // 2, device="cuda")
    first, second = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
    # the angles' cos and sin are inputs, in 32 bits
    row = s["table"].index_select(0, s["positions"]).double()
    return first, second, row[:, None, :half], row[:, None, half:]


def _exact_rotary(s, case):
    first, second, cos, sin = _rotation(s, case)
    out = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "_weight"]
        rms = (x.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS).sqrt() if case["norm"] else None
        unit = x / rms if case["norm"] else x
        if case["mode"] == "forward":
            y = unit * w.double() if case["norm"] else unit.clone()
            a, b = y[..., first], y[..., second]
            y[..., first], y[..., second] = cos * a - sin * b, sin * a + cos * b
            out[name] = y
            continue
        dy = s["d" + name].double().clone()
        a, b = dy[..., first], dy[..., second]
        dy[..., first], dy[..., second] = cos * a + sin * b, cos * b - sin * a
        if case["norm"]:
            dweight = torch.einsum("thd,thd->d", dy, unit)
            dy *= w.double()
            dy = (dy - unit * (torch.einsum("thd,thd->th", dy, unit) / case["dim"])[..., None]) / rms
            out["d" + name + "_weight"] = dweight
        out["d" + name] = dy
    if case["mode"] == "forward":
        return {"q": out["q"], "k": out["k"]}
    if not case["norm"]:
        return {"dq": out["dq"], "dk": out["dk"]}
    return {key: out[key] for key in ("dq", "dk", "dq_weight", "dk_weight")}


def _exact_attention(s, case):
    if work(case)["flops"] > 6e12:
        return None
    train = case["mode"] == "train"
    n, h, kv, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    scale = 1.0 / math.sqrt(d)

    def zeros(heads):
        return torch.zeros(n, heads, d, dtype=torch.float64, device="cuda")

    o, lse = zeros(h), torch.full((h, n), float("-inf"), dtype=torch.float64, device="cuda")
    if train:
        dq, dk, dv = zeros(h), zeros(kv), zeros(kv)
    start = 0
    for length in _lengths(case):
        for head in range(h):
            shared = head // (h // kv)
            k, v = s["k"][start:start + length, shared].double(), s["v"][start:start + length, shared].double()
            for r0 in range(0, length, 2048):
                r1 = min(length, r0 + 2048)
                seen = r1 if case["causal"] else length
                here = slice(start + r0, start + r1)
                q = s["q"][here, head].double()
                logits = scale * (q @ k[:seen].T)
                if case["causal"]:
                    ahead = torch.arange(seen, device="cuda")[None] > torch.arange(r0, r1, device="cuda")[:, None]
                    logits[ahead] = float("-inf")
                total = torch.logsumexp(logits, 1)
                p = torch.exp(logits - total[:, None])
                o[here, head], lse[head, here] = p @ v[:seen], total
                if train:
                    do, there = s["do"][here, head].double(), slice(start, start + seen)
                    dv[there, shared] += p.T @ do
                    inner = torch.einsum("id,id->i", do, o[here, head])
                    ds = p * (do @ v[:seen].T - inner[:, None]) * scale
                    dq[here, head] = ds @ k[:seen]
                    dk[there, shared] += ds.T @ q
        start += length
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if train else {"o": o, "lse": lse}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    n, h, kv, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "qk_norm_rotary":
        rows = n * (h + kv) * d
        side = n * (8 + 4 * case["rotary"]) + (2 * d * size if case["norm"] else 0)
        if case["mode"] == "forward":
            return {"bytes": 2 * rows * size + side, "flops": 8 * rows}
        return {"bytes": 3 * rows * size + side + (2 * d * size if case["norm"] else 0), "flops": 16 * rows}
    pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in _lengths(case))
    side = 8 * (case["sequences"] + 1) + 4 * n * h
    if case["mode"] == "forward":
        return {"bytes": size * n * d * (2 * h + 2 * kv) + side, "flops": 4 * d * h * pairs}
    return {"bytes": size * n * d * (4 * h + 4 * kv) + side, "flops": 14 * d * h * pairs}
