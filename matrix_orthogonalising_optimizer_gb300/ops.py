"""Layer norm, gated feed-forward block and vocabulary loss: the operators whose
gradients the optimizer steps consume.

Thin bindings over the C ABI of ``include/dmuon.h`` (which states the formulas,
limits and status codes): they check shapes, allocate outputs and marshal
arguments.  Tensors are CUDA, contiguous, bf16 or fp32 -- one dtype per call for
activations, weights and gradients; row statistics and losses are fp32.  The
last dimension is the row; leading dimensions are flattened.

``stream`` (a torch stream or a raw handle) defaults to the current one; outputs
and a workspace that is not passed in are allocated on that stream, and the
caller orders it after the work that produced the inputs.  ``workspace`` is a
uint8 tensor of at least the bytes that the ``*_workspace`` function gives, to be
reused from call to call on one stream.

Autograd does not record these calls.  The forward functions refuse inputs that
require gradients unless they are called under ``torch.no_grad()``; the gradients
come from ``layer_norm_backward``, ``gated_ffn_backward`` and ``vocab_loss_grad``.
"""
from __future__ import annotations

import torch

from . import _lib

__all__ = ["layer_norm", "layer_norm_backward", "layer_norm_workspace", "gated_ffn", "gated_ffn_backward",
           "gated_ffn_workspace", "vocab_loss", "vocab_loss_grad", "vocab_loss_workspace", "ops_status"]

_DTYPES = {torch.bfloat16: _lib.BF16, torch.float32: _lib.FP32}
_NAMES = {"bf16": _lib.BF16, "fp32": _lib.FP32, **_DTYPES}
_ACTS = {"silu": _lib.ACT_SILU, "gelu": _lib.ACT_GELU}


def _dtype(d):
    return _NAMES.get(d, -1)


def _act(name):
    if name not in _ACTS:
        raise ValueError(f"activation must be one of {sorted(_ACTS)}, not {name!r}")
    return _ACTS[name]


def _refuse(where, name, t, dtype, shape, dev):
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{where}: {name} must be a CUDA tensor on the device of the first argument")
    if t.dtype is not dtype:
        raise ValueError(f"{where}: {name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{where}: {name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{where}: {name} must be contiguous")


def _check(where, dev, dt, *tensors):
    """Every (name, tensor, shape): on CUDA device dev, of dtype dt, of that shape, contiguous."""
    for name, t, shape in tensors:
        if t is not None and not (t.is_cuda and t.dtype is dt and t.shape == shape and t.is_contiguous()
                                  and t.device == dev):
            _refuse(where, name, t, dt, shape, dev)


def _no_graph(where, *tensors):
    """Autograd does not see these calls: results cut off from a graph that is being
    recorded would lose the inputs' gradients without a word."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError(f"{where}: an input requires gradients, but autograd does not record this call: make it "
                                 "under torch.no_grad() and take the gradients from the functions that return them")


def _elsewhere(stream, dev):
    """The call has to run under another device or stream than the current one."""
    return stream is not None or torch.cuda.current_device() != dev.index


def _run_elsewhere(stream, tensors, call):
    """call() with the tensors' device and the given stream current, so that outputs are
    allocated there; the inputs are kept alive for that stream."""
    dev = tensors[0].device
    with torch.cuda.device(dev):
        cur = torch.cuda.current_stream(dev)
        st = torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream or cur
        with torch.cuda.stream(st):
            out = call()
        if st.cuda_stream != cur.cuda_stream:
            for t in tensors:
                if t is not None:
                    t.record_stream(st)
        return out


_raw_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream without building an object


def _ptr(t):
    return None if t is None else t.data_ptr()


def _space(workspace, need, device):
    """(pointer, bytes, tensor) of the caller's workspace, or of a new one of need() bytes."""
    if workspace is None:
        workspace = torch.empty(need(), dtype=torch.uint8, device=device)
    elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the device of the first argument")
    return workspace.data_ptr() or None, workspace.numel() * workspace.element_size(), workspace


def ops_status() -> int:
    """Status of the operators' device-side waits on the current device (0 = fine), once all its
    streams have finished; clears it."""
    return int(_lib.load().dmuon_ops_status())


# ---------------------------------------------------------------- layer norm

def layer_norm(x, weight=None, bias=None, eps=1e-5, stream=None):
    """``(y, mean, rstd)`` of a layer norm over the last dimension (weight, bias optional)."""
    dt, dev, shape = x.dtype, x.device, x.shape
    cols = shape[-1]
    _check("layer_norm", dev, dt, ("x", x, shape), ("weight", weight, (cols,)), ("bias", bias, (cols,)))
    _no_graph("layer_norm", x, weight, bias)
    rows = x.numel() // cols if cols else 0

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (x, weight, bias),
                              lambda: layer_norm(x, weight, bias, eps))
    s = _raw_stream(dev.index)
    y = torch.empty_like(x)
    mean = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    rstd = torch.empty_like(mean)
    st = _lib.load().dmuon_layer_norm_forward(x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(),
                                              mean.data_ptr(), rstd.data_ptr(), rows, cols, _dtype(dt), eps, s)
    _lib.check(st, "dmuon_layer_norm_forward")
    return y, mean, rstd


def layer_norm_workspace(rows, cols, dtype="bf16") -> int:
    """Workspace bytes of ``layer_norm_backward``."""
    return int(_lib.load().dmuon_layer_norm_workspace_bytes(rows, cols, _dtype(dtype)))


def layer_norm_backward(dy, x, weight, mean, rstd, workspace=None, stream=None):
    """``(dx, dweight, dbias)`` from the forward pass's input and statistics."""
    dt, dev, shape = x.dtype, x.device, x.shape
    cols = shape[-1]
    _check("layer_norm_backward", dev, dt, ("x", x, shape), ("dy", dy, shape), ("weight", weight, (cols,)))
    _check("layer_norm_backward", dev, torch.float32, ("mean", mean, shape[:-1]), ("rstd", rstd, shape[:-1]))
    rows = x.numel() // cols if cols else 0

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (x, dy, weight, mean, rstd, workspace),
                              lambda: layer_norm_backward(dy, x, weight, mean, rstd, workspace))
    s = _raw_stream(dev.index)
    dx = torch.empty_like(x)
    dw = torch.empty(cols, dtype=dt, device=dev)
    db = torch.empty_like(dw)
    wp, wb, _keep = _space(workspace, lambda: layer_norm_workspace(rows, cols, dt), dev)
    st = _lib.load().dmuon_layer_norm_backward(dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(),
                                               rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(), db.data_ptr(), rows,
                                               cols, _dtype(dt), wp, wb, s)
    _lib.check(st, "dmuon_layer_norm_backward")
    return dx, dw, db


# ---------------------------------------------------------------- gated feed-forward block

def gated_ffn_workspace(tokens, dim, hidden, dtype="bf16", backward=False) -> int:
    """Workspace bytes of ``gated_ffn`` or, with ``backward``, of ``gated_ffn_backward``
    (which is also enough for the forward pass)."""
    return int(_lib.load().dmuon_gated_ffn_workspace_bytes(tokens, dim, hidden, _dtype(dtype), int(backward)))


def gated_ffn(x, w_gate, w_up, w_down, activation="silu", save=False, workspace=None, stream=None):
    """``y = h w_down^T`` with ``h = act(a) * u``, ``a = x w_gate^T``, ``u = x w_up^T``; with
    ``save`` ``(y, saved, h)``, what the backward pass reads: ``saved`` is the pair
    ``(act(a), u act'(a))``, in fp32, or with ``save="compact"`` in x's dtype."""
    dt, dev, shape = x.dtype, x.device, x.shape
    dim, hidden = shape[-1], w_gate.shape[0]
    tokens = x.numel() // dim if dim else 0
    _check("gated_ffn", dev, dt, ("x", x, shape), ("w_gate", w_gate, (hidden, dim)), ("w_up", w_up, (hidden, dim)),
           ("w_down", w_down, (dim, hidden)))
    _no_graph("gated_ffn", x, w_gate, w_up, w_down)
    act = _act(activation)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (x, w_gate, w_up, w_down, workspace),
                              lambda: gated_ffn(x, w_gate, w_up, w_down, activation, save, workspace))
    s = _raw_stream(dev.index)
    y = torch.empty_like(x)
    saved, h, kind = (None, None), None, dt
    if save:
        h = torch.empty(*shape[:-1], hidden, dtype=dt, device=dev)
        kind = dt if save == "compact" else torch.float32
        saved = (torch.empty_like(h, dtype=kind), torch.empty_like(h, dtype=kind))
    wp, wb, _keep = _space(workspace, lambda: gated_ffn_workspace(tokens, dim, hidden, dt), dev)
    st = _lib.load().dmuon_gated_ffn_forward(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                                             y.data_ptr(), _ptr(saved[0]), _ptr(saved[1]), _ptr(h), _dtype(kind),
                                             tokens, dim, hidden, _dtype(dt), act, wp, wb, s)
    _lib.check(st, "dmuon_gated_ffn_forward")
    return (y, saved, h) if save else y


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved, h, activation="silu", workspace=None, stream=None):
    """``(dx, dw_gate, dw_up, dw_down)``, the weights' gradients ready for the Muon step.

    ``saved`` already holds the activation and its slope; ``activation`` is only checked, so
    that both passes take the same keywords."""
    dt, dev, shape = x.dtype, x.device, x.shape
    dim, hidden = shape[-1], w_gate.shape[0]
    tokens = x.numel() // dim if dim else 0
    inner = (*shape[:-1], hidden)
    _check("gated_ffn_backward", dev, dt, ("x", x, shape), ("dy", dy, shape), ("w_gate", w_gate, (hidden, dim)),
           ("w_up", w_up, (hidden, dim)), ("w_down", w_down, (dim, hidden)), ("h", h, inner))
    kind = saved[0].dtype
    _check("gated_ffn_backward", dev, kind, ("saved[0]", saved[0], inner), ("saved[1]", saved[1], inner))
    _act(activation)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (x, dy, w_gate, w_up, w_down, *saved, h, workspace),
                              lambda: gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved, h, activation, workspace))
    s = _raw_stream(dev.index)
    dx = torch.empty_like(x)
    dwg, dwu, dwd = torch.empty_like(w_gate), torch.empty_like(w_up), torch.empty_like(w_down)
    wp, wb, _keep = _space(workspace, lambda: gated_ffn_workspace(tokens, dim, hidden, dt, backward=True), dev)
    st = _lib.load().dmuon_gated_ffn_backward(dy.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
                                              w_down.data_ptr(), saved[0].data_ptr(), saved[1].data_ptr(),
                                              h.data_ptr(), _dtype(kind), dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(),
                                              dwd.data_ptr(), tokens, dim, hidden, _dtype(dt), wp, wb, s)
    _lib.check(st, "dmuon_gated_ffn_backward")
    return dx, dwg, dwu, dwd


# ---------------------------------------------------------------- vocabulary loss

def vocab_loss_workspace(tokens, dim, vocab, dtype="bf16", grad=False, budget=0) -> int:
    """Workspace bytes of ``vocab_loss`` or, with ``grad``, of ``vocab_loss_grad``."""
    return int(_lib.load().dmuon_vocab_loss_workspace_bytes(tokens, dim, vocab, _dtype(dtype), int(grad), budget))


def _vocab_loss(where, x, weight, targets, coef, ignore_index, workspace, budget, stream, grad):
    dt, dev, rows = x.dtype, x.device, x.shape[:-1]
    dim, vocab = x.shape[-1], weight.shape[0]
    tokens = x.numel() // dim if dim else 0
    _check(where, dev, dt, ("x", x, x.shape), ("weight", weight, (vocab, dim)))
    _check(where, dev, torch.int64, ("targets", targets, rows))
    _check(where, dev, torch.float32, ("coef", coef, rows))
    if not grad:
        _no_graph(where, x, weight)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (x, weight, targets, coef, workspace),
                              lambda: _vocab_loss(where, x, weight, targets, coef, ignore_index, workspace, budget,
                                                  None, grad))
    s = _raw_stream(dev.index)
    loss = torch.empty(rows, dtype=torch.float32, device=dev)
    lse = torch.empty_like(loss)
    dx = torch.empty_like(x) if grad else None
    dw = torch.empty_like(weight) if grad else None
    wp, wb, _keep = _space(workspace, lambda: vocab_loss_workspace(tokens, dim, vocab, dt, grad, budget), dev)
    st = _lib.load().dmuon_vocab_loss(x.data_ptr(), weight.data_ptr(), targets.data_ptr(), _ptr(coef),
                                      ignore_index, loss.data_ptr(), lse.data_ptr(), _ptr(dx), _ptr(dw), tokens,
                                      dim, vocab, _dtype(dt), budget, wp, wb, s)
    _lib.check(st, "dmuon_vocab_loss")
    return loss, lse, dx, dw


def vocab_loss(x, weight, targets, ignore_index=-100, workspace=None, budget=0, stream=None):
    """``(loss, lse)`` per token of the softmax cross entropy of ``x weight^T``."""
    return _vocab_loss("vocab_loss", x, weight, targets, None, ignore_index, workspace, budget, stream, False)[:2]


def vocab_loss_grad(x, weight, targets, coef=None, ignore_index=-100, workspace=None, budget=0, stream=None):
    """``(loss, lse, dx, dweight)``: the losses and the gradients of ``sum(coef * loss)``
    (``coef``: fp32 per token, ones if None -- 1 / tokens for a mean)."""
    return _vocab_loss("vocab_loss_grad", x, weight, targets, coef, ignore_index, workspace, budget, stream, True)
