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
"""
from __future__ import annotations

import contextlib

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


def _check(where, like, **tensors):
    """Every given tensor: CUDA, contiguous, on like's device, of the given dtype and shape."""
    dev = like.device
    for name, (t, dtype, shape) in tensors.items():
        if t is None:
            continue
        if not t.is_cuda or t.device != dev:
            raise ValueError(f"{where}: {name} must be a CUDA tensor on the device of the first argument")
        if t.dtype != dtype:
            raise ValueError(f"{where}: {name} must be {dtype}, not {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{where}: {name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")


@contextlib.contextmanager
def _launch(stream, tensors):
    """The raw stream handle of a call, with its device and stream current (outputs are
    allocated there) and the inputs kept alive for it."""
    dev = tensors[0].device
    with torch.cuda.device(dev):
        cur = torch.cuda.current_stream()
        if stream is None:
            yield cur.cuda_stream
            return
        st = torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream
        with torch.cuda.stream(st):
            yield st.cuda_stream
        if st.cuda_stream != cur.cuda_stream:
            for t in tensors:
                if t is not None:
                    t.record_stream(st)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _space(workspace, nbytes, device):
    """(pointer, bytes, tensor) of the caller's workspace, or of a new one."""
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr() if nbytes else None, workspace.numel() * workspace.element_size(), workspace


def ops_status() -> int:
    """Status of the operators' device-side waits on the current device (0 = fine); clears it."""
    return int(_lib.load().dmuon_ops_status())


# ---------------------------------------------------------------- layer norm

def layer_norm(x, weight=None, bias=None, eps=1e-5, stream=None):
    """``(y, mean, rstd)`` of a layer norm over the last dimension (weight, bias optional)."""
    cols = x.shape[-1]
    _check("layer_norm", x, x=(x, x.dtype, x.shape), weight=(weight, x.dtype, (cols,)), bias=(bias, x.dtype, (cols,)))
    rows = x.numel() // cols if cols else 0
    with _launch(stream, (x, weight, bias)) as s:
        y = torch.empty_like(x)
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        _lib.check(_lib.load().dmuon_layer_norm_forward(x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(),
                                                        mean.data_ptr(), rstd.data_ptr(), rows, cols, _dtype(x.dtype),
                                                        eps, s), "dmuon_layer_norm_forward")
    return y, mean, rstd


def layer_norm_workspace(rows, cols, dtype="bf16") -> int:
    """Workspace bytes of ``layer_norm_backward``."""
    return int(_lib.load().dmuon_layer_norm_workspace_bytes(rows, cols, _dtype(dtype)))


def layer_norm_backward(dy, x, weight, mean, rstd, workspace=None, stream=None):
    """``(dx, dweight, dbias)`` from the forward pass's input and statistics."""
    cols = x.shape[-1]
    _check("layer_norm_backward", x, x=(x, x.dtype, x.shape), dy=(dy, x.dtype, x.shape),
           weight=(weight, x.dtype, (cols,)), mean=(mean, torch.float32, x.shape[:-1]),
           rstd=(rstd, torch.float32, x.shape[:-1]))
    rows = x.numel() // cols if cols else 0
    nbytes = layer_norm_workspace(rows, cols, x.dtype)
    with _launch(stream, (x, dy, weight, mean, rstd, workspace)) as s:
        dx = torch.empty_like(x)
        dw = torch.empty(cols, dtype=x.dtype, device=x.device)
        db = torch.empty_like(dw)
        wp, wb, _keep = _space(workspace, nbytes, x.device)
        _lib.check(_lib.load().dmuon_layer_norm_backward(dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(),
                                                         rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(), db.data_ptr(),
                                                         rows, cols, _dtype(x.dtype), wp, wb, s),
                   "dmuon_layer_norm_backward")
    return dx, dw, db


# ---------------------------------------------------------------- gated feed-forward block

def gated_ffn_workspace(tokens, dim, hidden, dtype="bf16", backward=False) -> int:
    """Workspace bytes of ``gated_ffn`` or, with ``backward``, of ``gated_ffn_backward``
    (which is also enough for the forward pass)."""
    return int(_lib.load().dmuon_gated_ffn_workspace_bytes(tokens, dim, hidden, _dtype(dtype), int(backward)))


def gated_ffn(x, w_gate, w_up, w_down, activation="silu", save=False, workspace=None, stream=None):
    """``y = (act(x w_gate^T) * (x w_up^T)) w_down^T``; with ``save`` ``(y, gate, up)``, the
    projections that the backward pass reads."""
    dim, hidden = x.shape[-1], w_gate.shape[0]
    tokens = x.numel() // dim if dim else 0
    _check("gated_ffn", x, x=(x, x.dtype, x.shape), w_gate=(w_gate, x.dtype, (hidden, dim)),
           w_up=(w_up, x.dtype, (hidden, dim)), w_down=(w_down, x.dtype, (dim, hidden)))
    act = _act(activation)
    nbytes = gated_ffn_workspace(tokens, dim, hidden, x.dtype)
    with _launch(stream, (x, w_gate, w_up, w_down, workspace)) as s:
        y = torch.empty_like(x)
        gate = up = None
        if save:
            gate = torch.empty(*x.shape[:-1], hidden, dtype=x.dtype, device=x.device)
            up = torch.empty_like(gate)
        wp, wb, _keep = _space(workspace, nbytes, x.device)
        _lib.check(_lib.load().dmuon_gated_ffn_forward(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
                                                       w_down.data_ptr(), y.data_ptr(), _ptr(gate), _ptr(up), tokens,
                                                       dim, hidden, _dtype(x.dtype), act, wp, wb, s),
                   "dmuon_gated_ffn_forward")
    return (y, gate, up) if save else y


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, gate, up, activation="silu", workspace=None, stream=None):
    """``(dx, dw_gate, dw_up, dw_down)``, the weights' gradients ready for the Muon step."""
    dim, hidden = x.shape[-1], w_gate.shape[0]
    tokens = x.numel() // dim if dim else 0
    inner = (*x.shape[:-1], hidden)
    _check("gated_ffn_backward", x, x=(x, x.dtype, x.shape), dy=(dy, x.dtype, x.shape),
           w_gate=(w_gate, x.dtype, (hidden, dim)), w_up=(w_up, x.dtype, (hidden, dim)),
           w_down=(w_down, x.dtype, (dim, hidden)), gate=(gate, x.dtype, inner), up=(up, x.dtype, inner))
    act = _act(activation)
    nbytes = gated_ffn_workspace(tokens, dim, hidden, x.dtype, backward=True)
    with _launch(stream, (x, dy, w_gate, w_up, w_down, gate, up, workspace)) as s:
        dx = torch.empty_like(x)
        dwg, dwu, dwd = torch.empty_like(w_gate), torch.empty_like(w_up), torch.empty_like(w_down)
        wp, wb, _keep = _space(workspace, nbytes, x.device)
        _lib.check(_lib.load().dmuon_gated_ffn_backward(dy.data_ptr(), x.data_ptr(), w_gate.data_ptr(),
                                                        w_up.data_ptr(), w_down.data_ptr(), gate.data_ptr(),
                                                        up.data_ptr(), dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(),
                                                        dwd.data_ptr(), tokens, dim, hidden, _dtype(x.dtype), act, wp,
                                                        wb, s), "dmuon_gated_ffn_backward")
    return dx, dwg, dwu, dwd


# ---------------------------------------------------------------- vocabulary loss

def vocab_loss_workspace(tokens, dim, vocab, dtype="bf16", grad=False, budget=0) -> int:
    """Workspace bytes of ``vocab_loss`` or, with ``grad``, of ``vocab_loss_grad``."""
    return int(_lib.load().dmuon_vocab_loss_workspace_bytes(tokens, dim, vocab, _dtype(dtype), int(grad), budget))


def _vocab_loss(where, x, weight, targets, coef, ignore_index, workspace, budget, stream, grad):
    dim, vocab = x.shape[-1], weight.shape[0]
    tokens = x.numel() // dim if dim else 0
    rows = x.shape[:-1]
    _check(where, x, x=(x, x.dtype, x.shape), weight=(weight, x.dtype, (vocab, dim)),
           targets=(targets, torch.int64, rows), coef=(coef, torch.float32, rows))
    nbytes = vocab_loss_workspace(tokens, dim, vocab, x.dtype, grad, budget)
    with _launch(stream, (x, weight, targets, coef, workspace)) as s:
        loss = torch.empty(rows, dtype=torch.float32, device=x.device)
        lse = torch.empty_like(loss)
        dx = torch.empty_like(x) if grad else None
        dw = torch.empty_like(weight) if grad else None
        wp, wb, _keep = _space(workspace, nbytes, x.device)
        _lib.check(_lib.load().dmuon_vocab_loss(x.data_ptr(), weight.data_ptr(), targets.data_ptr(), _ptr(coef),
                                                ignore_index, loss.data_ptr(), lse.data_ptr(), _ptr(dx), _ptr(dw),
                                                tokens, dim, vocab, _dtype(x.dtype), budget, wp, wb, s),
                   "dmuon_vocab_loss")
    return loss, lse, dx, dw


def vocab_loss(x, weight, targets, ignore_index=-100, workspace=None, budget=0, stream=None):
    """``(loss, lse)`` per token of the softmax cross entropy of ``x weight^T``."""
    return _vocab_loss("vocab_loss", x, weight, targets, None, ignore_index, workspace, budget, stream, False)[:2]


def vocab_loss_grad(x, weight, targets, coef=None, ignore_index=-100, workspace=None, budget=0, stream=None):
    """``(loss, lse, dx, dweight)``: the losses and the gradients of ``sum(coef * loss)``
    (``coef``: fp32 per token, ones if None -- 1 / tokens for a mean)."""
    return _vocab_loss("vocab_loss_grad", x, weight, targets, coef, ignore_index, workspace, budget, stream, True)
