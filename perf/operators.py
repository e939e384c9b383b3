"""The language-model operators beside the optimizer step, as measured cases.

Three operators that produce the gradients an optimizer step consumes: layer
norm, the gated feed-forward block and the vocabulary loss (softmax cross
entropy taken straight from the hidden states and the vocabulary matrix).
Each case is run in two forms on the same inputs: the plain form (elementary
torch operations in 32 bits, rounded once at the end) and, with ``own`` set,
the library's kernels through the package's public calls.  ``exact`` gives
the definition's values in 64 bits.

Formulas, for row-major tensors:

layer norm    mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), n = (x - mu) r
              y = n * w + b;  dw = sum_rows dy * n, db = sum_rows dy,
              dx = r (g - mean(g) - n mean(g n)),  g = dy * w
gated block   a = x Wg^T, u = x Wu^T, h = act(a) * u, y = h Wd^T
              dh = dy Wd, da = dh * u * act'(a), du = dh * act(a)
              dx = da Wg + du Wu, dWg = da^T x, dWu = du^T x, dWd = dy^T h
vocab loss    z = x W^T, lse = log sum_v exp z_v, loss = lse - z_target (0 if ignored)
              dz = c (softmax(z) - onehot(target)) (0 if ignored), dx = dz W, dW = dz^T x
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-5
_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _norm(name, mode, dtype, rows, cols):
    return {"name": name, "op": "layer_norm", "mode": mode, "dtype": dtype, "rows": rows, "cols": cols}


def _ffn(name, mode, dtype, tokens, dim, hidden, act):
    return {"name": name, "op": "gated_ffn", "mode": mode, "dtype": dtype, "tokens": tokens, "dim": dim,
            "hidden": hidden, "act": act}


def _loss(name, mode, dtype, tokens, dim, vocab):
    return {"name": name, "op": "vocab_loss", "mode": mode, "dtype": dtype, "tokens": tokens, "dim": dim,
            "vocab": vocab}


def listed():
    return [
        # one token of the small-transformer width: a generated token's norm, all latency
        _norm("norm_fwd_token", "forward", "bf16", 1, 768),
        # a training batch of the Llama-3-8B-shaped width, forward and backward
        _norm("norm_fwd_batch", "forward", "bf16", 16384, 4096),
        _norm("norm_bwd_batch", "backward", "bf16", 16384, 4096),
        # a ragged fp32 batch of a width that fills no vector
        _norm("norm_bwd_odd_fp32", "backward", "fp32", 1023, 1001),
        # serving one token: the weights are read once, nothing else counts
        _ffn("ffn_fwd_token", "forward", "bf16", 1, 4096, 14336, "silu"),
        # a short prompt through a small-transformer block
        _ffn("ffn_fwd_prompt", "forward", "bf16", 333, 768, 2048, "gelu"),
        # a training micro-batch of the Llama-3-8B-shaped block: every gradient Muon consumes
        _ffn("ffn_train_batch", "train", "bf16", 8192, 4096, 14336, "silu"),
        # fp32 training of a small block with an odd hidden width
        _ffn("ffn_train_odd_fp32", "train", "fp32", 777, 512, 1365, "silu"),
        # scoring sixteen positions against a large vocabulary: the vocabulary matrix is read once
        _loss("loss_few_tokens", "loss", "bf16", 16, 4096, 131072),
        # evaluation of a batch at the small-transformer width, odd vocabulary
        _loss("loss_eval_batch", "loss", "bf16", 2047, 768, 50257),
        # a training micro-batch against a large vocabulary: loss, dx and dW
        _loss("loss_grad_batch", "grad", "bf16", 4096, 4096, 131072),
        # fp32 training of a small model, odd everywhere
        _loss("loss_grad_odd_fp32", "grad", "fp32", 301, 512, 10007),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A model width: three times in four a multiple of 64, else any integer."""
    n = _log_int(rng, lo, hi)
    return max(lo, n // 64 * 64) if rng.random() < 0.75 else n


def draw(rng):
    dtype = "bf16" if rng.random() < 0.75 else "fp32"
    # costs stay below the largest listed cases (the plain form runs both types in 32 bits)
    cap = 8e12 if dtype == "bf16" else 1e12
    op = rng.choice(("layer_norm", "gated_ffn", "vocab_loss"))
    while True:
        if op == "layer_norm":
            case = _norm(None, rng.choice(("forward", "backward")), dtype, _log_int(rng, 1, 16384),
                         _width(rng, 64, 16384))
            ok = case["rows"] * case["cols"] <= 16384 * 4096
        elif op == "gated_ffn":
            case = _ffn(None, rng.choice(("forward", "train")), dtype, _log_int(rng, 1, 8192), _width(rng, 64, 8192),
                        _width(rng, 128, 28672), rng.choice(("silu", "gelu")))
            ok = work(case)["flops"] <= cap
        else:
            case = _loss(None, rng.choice(("loss", "grad")), dtype, _log_int(rng, 1, 8192), _width(rng, 64, 8192),
                         _log_int(rng, 1000, 131072))
            ok = work(case)["flops"] <= cap
        if ok:
            del case["name"]
            return case


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dt)

    s = {"case": case}
    if case["op"] == "layer_norm":
        rows, cols = case["rows"], case["cols"]
        # a residual stream: a mean of its own per row, a few large channels
        x = torch.randn(rows, cols, generator=g, device="cuda")
        x += 0.5 * torch.randn(rows, 1, generator=g, device="cuda")
        x *= 1.0 + 9.0 * (torch.rand(1, cols, generator=g, device="cuda") < 0.01)
        s["x"] = x.to(dt)
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)
        s["bias"] = normal(cols, std=0.1)
        if case["mode"] == "backward":
            s["dy"] = normal(rows, cols, std=1e-3)
            xf = s["x"].float()
            mean = xf.mean(1)
            s["mean"] = mean
            s["rstd"] = torch.rsqrt((xf - mean[:, None]).square().mean(1) + EPS)
    elif case["op"] == "gated_ffn":
        n, d, f = case["tokens"], case["dim"], case["hidden"]
        s["x"] = normal(n, d)
        # weights at the usual 1/sqrt(fan in): the projections keep the scale of x
        s["w_gate"] = normal(f, d, std=d ** -0.5)
        s["w_up"] = normal(f, d, std=d ** -0.5)
        s["w_down"] = normal(d, f, std=f ** -0.5)
        if case["mode"] == "train":
            s["dy"] = normal(n, d, std=1e-3)
    else:
        n, d, v = case["tokens"], case["dim"], case["vocab"]
        w = torch.randn(v, d, generator=g, device="cuda").mul_(0.02).to(dt)
        t = torch.randint(0, v, (n,), generator=g, device="cuda")
        # normalised hidden states that lean towards their target: its logit
        # rises by up to 12, so probabilities run from about 1/vocab to nearly 1
        lift = 12.0 / (0.0004 * d) * torch.rand(n, 1, generator=g, device="cuda")
        x = torch.randn(n, d, generator=g, device="cuda") + lift * w[t].float()
        drop = torch.rand(n, generator=g, device="cuda") < 0.05  # padding and prompt positions
        s["x"], s["weight"] = x.to(dt), w
        s["targets"] = torch.where(drop, torch.full_like(t, IGNORE), t)
        if case["mode"] == "grad":
            s["coef"] = torch.full((n,), 1.0 / n, device="cuda")
    if own:
        import matrix_orthogonalising_optimizer_gb300 as pkg
        s["pkg"] = pkg
        nbytes = 0
        if case["op"] == "layer_norm" and case["mode"] == "backward":
            nbytes = pkg.layer_norm_workspace(case["rows"], case["cols"], case["dtype"])
        elif case["op"] == "gated_ffn":
            nbytes = pkg.gated_ffn_workspace(case["tokens"], case["dim"], case["hidden"], case["dtype"],
                                             backward=case["mode"] == "train")
        elif case["op"] == "vocab_loss":
            nbytes = pkg.vocab_loss_workspace(case["tokens"], case["dim"], case["vocab"], case["dtype"],
                                              grad=case["mode"] == "grad")
        s["workspace"] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    form = _own if own else _plain
    return form[case["op"], case["mode"]](state)


def _own_norm_forward(s):
    y, mean, rstd = s["pkg"].layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
    return {"y": y, "mean": mean, "rstd": rstd}


def _own_norm_backward(s):
    dx, dw, db = s["pkg"].layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"],
                                              workspace=s["workspace"])
    return {"dx": dx, "dweight": dw, "dbias": db}


def _own_ffn_forward(s):
    return {"y": s["pkg"].gated_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"], activation=s["case"]["act"],
                                    workspace=s["workspace"])}


def _own_ffn_train(s):
    act = s["case"]["act"]
    y, gate, up = s["pkg"].gated_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"], activation=act, save=True,
                                     workspace=s["workspace"])
    dx, dwg, dwu, dwd = s["pkg"].gated_ffn_backward(s["dy"], s["x"], s["w_gate"], s["w_up"], s["w_down"], gate, up,
                                                    activation=act, workspace=s["workspace"])
    return {"y": y, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}


def _own_loss(s):
    loss, lse = s["pkg"].vocab_loss(s["x"], s["weight"], s["targets"], ignore_index=IGNORE, workspace=s["workspace"])
    return {"loss": loss, "lse": lse}


def _own_loss_grad(s):
    loss, lse, dx, dw = s["pkg"].vocab_loss_grad(s["x"], s["weight"], s["targets"], coef=s["coef"],
                                                 ignore_index=IGNORE, workspace=s["workspace"])
    return {"loss": loss, "lse": lse, "dx": dx, "dweight": dw}


def _plain_norm_forward(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    y = c * rstd * s["weight"].float() + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_backward(s):
    dt = s["x"].dtype
    dy = s["dy"].float()
    rstd = s["rstd"][:, None]
    n = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    return {"dx": dx.to(dt), "dweight": (dy * n).sum(0).to(dt), "dbias": dy.sum(0).to(dt)}


def _plain_act(a, act):
    """act(a) and its derivative."""
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-a))
        return a * sig, sig * (1.0 + a * (1.0 - sig))
    cdf = 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
    return a * cdf, cdf + a * torch.exp(-0.5 * a * a) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_ffn_forward(s):
    x = s["x"].float()
    a, u = x @ s["w_gate"].float().T, x @ s["w_up"].float().T
    h = _plain_act(a, s["case"]["act"])[0] * u
    return {"y": (h @ s["w_down"].float().T).to(s["x"].dtype)}


def _plain_ffn_train(s):
    dt = s["x"].dtype
    x, dy = s["x"].float(), s["dy"].float()
    wg, wu, wd = s["w_gate"].float(), s["w_up"].float(), s["w_down"].float()
    a, u = x @ wg.T, x @ wu.T
    p, dp = _plain_act(a, s["case"]["act"])
    h = p * u
    y = h @ wd.T
    dh = dy @ wd
    da, du = dh * u * dp, dh * p
    return {"y": y.to(dt), "dx": (da @ wg + du @ wu).to(dt), "dw_gate": (da.T @ x).to(dt),
            "dw_up": (du.T @ x).to(dt), "dw_down": (dy.T @ h).to(dt)}


def _plain_logits(s):
    """Logits, their log-sum-exp, the losses, and the target index with its mask."""
    z = s["x"].float() @ s["weight"].float().T
    m = z.amax(1, keepdim=True)
    lse = (m + torch.log(torch.exp(z - m).sum(1, keepdim=True)))[:, 0]
    keep = s["targets"] != IGNORE
    t = torch.where(keep, s["targets"], torch.zeros_like(s["targets"]))
    loss = torch.where(keep, lse - z.gather(1, t[:, None])[:, 0], torch.zeros_like(lse))
    return z, lse, loss, t, keep


def _plain_loss(s):
    _, lse, loss, _, _ = _plain_logits(s)
    return {"loss": loss, "lse": lse}


def _plain_loss_grad(s):
    z, lse, loss, t, keep = _plain_logits(s)
    dt = s["x"].dtype
    dz = z.sub_(lse[:, None]).exp_()
    rows = torch.arange(len(t), device=t.device)
    dz[rows, t] -= 1.0
    dz *= torch.where(keep, s["coef"], torch.zeros_like(s["coef"]))[:, None]
    return {"loss": loss, "lse": lse, "dx": (dz @ s["weight"].float()).to(dt),
            "dweight": (dz.T @ s["x"].float()).to(dt)}


_own = {("layer_norm", "forward"): _own_norm_forward, ("layer_norm", "backward"): _own_norm_backward,
        ("gated_ffn", "forward"): _own_ffn_forward, ("gated_ffn", "train"): _own_ffn_train,
        ("vocab_loss", "loss"): _own_loss, ("vocab_loss", "grad"): _own_loss_grad}
_plain = {("layer_norm", "forward"): _plain_norm_forward, ("layer_norm", "backward"): _plain_norm_backward,
          ("gated_ffn", "forward"): _plain_ffn_forward, ("gated_ffn", "train"): _plain_ffn_train,
          ("vocab_loss", "loss"): _plain_loss, ("vocab_loss", "grad"): _plain_loss_grad}


# ---------------------------------------------------------------- the definition in 64 bits

_EXACT_FLOPS = 1.4e13  # about 15 s of 64-bit products


def exact(case, seed):
    if work(case)["flops"] > _EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    f64 = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if case["op"] == "layer_norm":
        x, w = f64["x"], f64["weight"]
        if case["mode"] == "forward":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + EPS).pow(-0.5)
            y = torch.addcmul(f64["bias"], (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), w)
            return {"y": y, "mean": mean, "rstd": rstd}
        dy, r = f64["dy"], f64["rstd"].unsqueeze(1)
        xhat = (x - f64["mean"].unsqueeze(1)) * r
        cols = x.shape[1]
        dn = dy * w
        dx = (cols * dn - dn.sum(1, True) - xhat * (dn * xhat).sum(1, True)) * (r / cols)
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, xhat), "dbias": dy.sum(0)}
    if case["op"] == "gated_ffn":
        x, wg, wu, wd = f64["x"], f64["w_gate"], f64["w_up"], f64["w_down"]
        a, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        if case["act"] == "silu":
            gate = torch.sigmoid(a)
        else:
            gate = torch.special.ndtr(a)
        y = torch.mm(a * gate * u, wd.t())
        if case["mode"] == "forward":
            return {"y": y}
        dy = f64["dy"]
        # act(a) = a gate(a): act' = gate + a gate'
        if case["act"] == "silu":
            slope = gate * (1 - gate)
        else:
            slope = torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        dh = torch.mm(dy, wd)
        out = {"y": y, "dx": None, "dw_gate": None, "dw_up": None, "dw_down": torch.mm(dy.t(), a * gate * u)}
        da = dh * u * (gate + a * slope)
        du = dh * (a * gate)
        out["dw_gate"], out["dw_up"] = torch.mm(da.t(), x), torch.mm(du.t(), x)
        out["dx"] = torch.addmm(torch.mm(da, wg), du, wu)
        return out
    x, w, t = f64["x"], f64["weight"], s["targets"]
    logp = torch.mm(x, w.t())
    lse = torch.logsumexp(logp, 1)
    hit = t >= 0
    idx = t.clamp(min=0).unsqueeze(1)
    loss = (lse - logp.gather(1, idx).squeeze(1)) * hit
    if case["mode"] == "loss":
        return {"loss": loss, "lse": lse}
    dz = (logp - lse.unsqueeze(1)).exp_()
    dz.scatter_add_(1, idx, -torch.ones_like(idx, dtype=torch.float64))
    dz.mul_((f64["coef"] * hit).unsqueeze(1))
    return {"loss": loss, "lse": lse, "dx": torch.mm(dz, w), "dweight": torch.mm(dz.t(), x)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "layer_norm":
        n, c, r = case["rows"] * case["cols"], case["cols"], case["rows"]
        if case["mode"] == "forward":
            return {"bytes": es * (2 * n + 2 * c) + 8 * r, "flops": 8 * n}
        return {"bytes": es * (3 * n + 3 * c) + 8 * r, "flops": 14 * n}
    n, d = case["tokens"], case["dim"]
    if case["op"] == "gated_ffn":
        f = case["hidden"]
        if case["mode"] == "forward":
            return {"bytes": es * (3 * d * f + 2 * n * d), "flops": 6 * n * d * f}
        return {"bytes": es * (6 * d * f + 4 * n * d), "flops": 18 * n * d * f}
    v = case["vocab"]
    if case["mode"] == "loss":
        return {"bytes": es * (v * d + n * d) + 16 * n, "flops": 2 * n * v * d}
    return {"bytes": es * (2 * v * d + 2 * n * d) + 20 * n, "flops": 6 * n * v * d}
