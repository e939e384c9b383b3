"""Head norms with the position rotation, and attention over packed sequences: the
operators of a transformer block beside the feed-forward block.

Thin bindings over the C ABI of ``include/dmuon.h`` (which states the formulas, limits
and status codes), with the conventions of the other training operators: CUDA tensors,
bf16 or fp32, one dtype per call, ``stream`` and ``workspace`` as there, no autograd.
Queries, keys and values are (tokens, heads, dim), or with more leading dimensions that
can be flattened; the last dimension is contiguous, the others may be strided (views of
one projection's output are read in place).  Outputs are contiguous.
"""
from __future__ import annotations

import torch

from . import _lib
from .ops import _check, _dtype, _elsewhere, _no_graph, _ptr, _raw_stream, _refuse, _run_elsewhere, _space

__all__ = ["rotary_table", "qk_norm_rotary", "qk_norm_rotary_backward", "qk_norm_rotary_workspace", "attention",
           "attention_backward", "attention_workspace"]


def _heads(where, name, t, dtype, shape, dev):
    """The C ABI's view of a tensor of this shape (*lead, heads, dim); refuses what it cannot describe."""
    if not (t.dtype is dtype and t.shape == shape and t.is_cuda and t.device == dev):
        _refuse(where, name, t, dtype, shape, dev)
    strides = t.stride()
    if strides[-1] != 1 and shape[-1] > 1 and t.numel():
        raise ValueError(f"{where}: the last dimension of {name} must be contiguous")
    if len(shape) == 3:
        return _lib.Heads(t.data_ptr(), strides[0], strides[1])
    step, span = None, None
    for n, s in zip(reversed(shape[:-2]), reversed(strides[:-2])):
        if n == 1:
            continue
        if step is not None and s != span and t.numel():
            raise ValueError(f"{where}: the leading dimensions of {name} must have one stride")
        step = s if step is None else step
        span = s * n
    return _lib.Heads(t.data_ptr(), shape[-1] if step is None else step, strides[-2])


def _rows(lead):
    n = 1
    for x in lead:
        n *= x
    return n


def _shapes(where, q, k):
    """The shapes of q and, with q's leading dimensions and width, of k."""
    qs = q.shape
    if len(qs) < 2 or k.dim() < 2:
        raise ValueError(f"{where}: q and k must have a head and an element dimension")
    if len(qs) == 3:
        return qs, (qs[0], k.shape[-2], qs[2])
    return qs, (*qs[:-2], k.shape[-2], qs[-1])


def _like(t):
    """A contiguous tensor of t's shape."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


# ---------------------------------------------------------------- rotation

def rotary_table(positions, rotary, base=10000.0, device=None, stream=None):
    """fp32 table (positions, rotary) of the rotation's angles: cos(p base^(-2 i / rotary)), then the sines."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.type != "cuda":
        raise ValueError("rotary_table: device must be a CUDA device")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if positions < 0 or rotary < 0:
        raise ValueError("rotary_table: positions and rotary must not be negative")
    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (torch.empty(0, device=dev),),
                              lambda: rotary_table(positions, rotary, base, dev))
    table = torch.empty(positions, rotary, dtype=torch.float32, device=dev)
    st = _lib.load().dmuon_rotary_table(_ptr(table) or None, positions, rotary, base, _raw_stream(dev.index))
    _lib.check(st, "dmuon_rotary_table")
    return table


def _rotary_check(where, lead, dev, dt, dim, positions, table, q_weight, k_weight):
    """(table rows, rotary) of the checked arguments."""
    _check(where, dev, dt, ("q_weight", q_weight, (dim,)), ("k_weight", k_weight, (dim,)))
    if table is None:
        return 0, 0
    if positions is None:
        raise ValueError(f"{where}: a table needs positions")
    if table.dim() != 2:
        raise ValueError(f"{where}: table must have two dimensions")
    _check(where, dev, torch.int64, ("positions", positions, lead))
    _check(where, dev, torch.float32, ("table", table, table.shape))
    return table.shape


def qk_norm_rotary(q, k, positions=None, table=None, q_weight=None, k_weight=None, norm=True, eps=1e-6,
                   interleaved=False, stream=None):
    """``(q, k)``, each head's row normalised (``x / sqrt(mean(x^2) + eps) * weight``; not with
    ``norm=False``) and turned by its token's position: ``positions`` are rows of ``table``
    (``rotary_table``), whose width is the number of leading elements that are turned (no table:
    none)."""
    dt, dev = q.dtype, q.device
    qs, ks = _shapes("qk_norm_rotary", q, k)
    hq = _heads("qk_norm_rotary", "q", q, dt, qs, dev)
    hk = _heads("qk_norm_rotary", "k", k, dt, ks, dev)
    rows, rotary = _rotary_check("qk_norm_rotary", qs[:-2], dev, dt, qs[-1], positions, table, q_weight, k_weight)
    _no_graph("qk_norm_rotary", q, k, q_weight, k_weight)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (q, k, positions, table, q_weight, k_weight),
                              lambda: qk_norm_rotary(q, k, positions, table, q_weight, k_weight, norm, eps, interleaved))
    s = _raw_stream(dev.index)
    qo, ko = _like(q), _like(k)
    st = _lib.load().dmuon_qk_norm_rotary_forward(hq, hk, _ptr(positions), _ptr(table), rows, rotary, int(interleaved),
                                                  _ptr(q_weight), _ptr(k_weight), int(norm), eps, qo.data_ptr(),
                                                  ko.data_ptr(), _rows(qs[:-2]), qs[-2], ks[-2], qs[-1], _dtype(dt), s)
    _lib.check(st, "dmuon_qk_norm_rotary_forward")
    return qo, ko


def qk_norm_rotary_workspace(tokens, heads, kv_heads, dim, dtype="bf16") -> int:
    """Workspace bytes of ``qk_norm_rotary_backward``."""
    return int(_lib.load().dmuon_qk_norm_rotary_workspace_bytes(tokens, heads, kv_heads, dim, _dtype(dtype)))


def qk_norm_rotary_backward(dq, dk, q, k, positions=None, table=None, q_weight=None, k_weight=None, norm=True, eps=1e-6,
                            interleaved=False, workspace=None, stream=None):
    """``(dq, dk, dq_weight, dk_weight)`` from the gradients of ``qk_norm_rotary``'s outputs and its inputs;
    the gradient of a weight that was not given is None."""
    where = "qk_norm_rotary_backward"
    dt, dev = q.dtype, q.device
    qs, ks = _shapes(where, q, k)
    hq = _heads(where, "q", q, dt, qs, dev)
    hk = _heads(where, "k", k, dt, ks, dev)
    gq = _heads(where, "dq", dq, dt, qs, dev)
    gk = _heads(where, "dk", dk, dt, ks, dev)
    rows, rotary = _rotary_check(where, qs[:-2], dev, dt, qs[-1], positions, table, q_weight, k_weight)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (q, k, dq, dk, positions, table, q_weight, k_weight, workspace),
                              lambda: qk_norm_rotary_backward(dq, dk, q, k, positions, table, q_weight, k_weight, norm,
                                                              eps, interleaved, workspace))
    s = _raw_stream(dev.index)
    tokens, heads, kv, dim = _rows(qs[:-2]), qs[-2], ks[-2], qs[-1]
    dx, dy = _like(q), _like(k)
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    wp, wb, _keep = None, 0, None
    if dqw is not None or dkw is not None or workspace is not None:
        wp, wb, _keep = _space(workspace, lambda: qk_norm_rotary_workspace(tokens, heads, kv, dim, dt), dev)
    st = _lib.load().dmuon_qk_norm_rotary_backward(gq, gk, hq, hk, _ptr(positions), _ptr(table), rows, rotary,
                                                   int(interleaved), _ptr(q_weight), _ptr(k_weight), int(norm), eps,
                                                   dx.data_ptr(), dy.data_ptr(), _ptr(dqw), _ptr(dkw), tokens, heads,
                                                   kv, dim, _dtype(dt), wp, wb, s)
    _lib.check(st, "dmuon_qk_norm_rotary_backward")
    return dx, dy, dqw, dkw


# ---------------------------------------------------------------- attention

def attention_workspace(tokens, heads, kv_heads, dim, dtype="bf16", sequences=1, backward=False) -> int:
    """Workspace bytes of ``attention`` or, with ``backward``, of ``attention_backward`` (which is also
    enough for the forward pass)."""
    return int(_lib.load().dmuon_attention_workspace_bytes(sequences, tokens, heads, kv_heads, dim, _dtype(dtype),
                                                           int(backward)))


def _scale(scale, dim):
    return max(dim, 1) ** -0.5 if scale is None else scale


def _sequences(where, lead, offsets, dev):
    """Sequences of the batch: those of ``offsets``, or one per row of the dimensions before the last."""
    if offsets is None:
        return max(1, _rows(lead[:-1]))
    shape = offsets.shape
    if len(shape) != 1 or shape[0] < 2:
        raise ValueError(f"{where}: offsets must hold the sequences' starts and the last one's end")
    _check(where, dev, torch.int64, ("offsets", offsets, shape))
    return shape[0] - 1


def attention(q, k, v, offsets=None, causal=True, scale=None, workspace=None, stream=None):
    """``(o, lse)``: attention over whole sequences, ``scale`` 1 / sqrt(dim) if None.

    q is (tokens, heads, dim), k and v (tokens, kv_heads, dim), with heads / kv_heads query heads
    sharing a key head.  ``offsets`` (int64 on the device, sequences + 1) packs sequences of
    different lengths one behind the other: sequence s is tokens offsets[s] to offsets[s + 1], and
    tokens outside all of them get o = 0 and lse = -inf.  Without offsets the tokens are one
    sequence, or (batch, tokens, heads, dim) a batch of equal ones.  ``lse`` is (heads, all tokens)."""
    dt, dev = q.dtype, q.device
    qs, ks = _shapes("attention", q, k)
    hq = _heads("attention", "q", q, dt, qs, dev)
    hk = _heads("attention", "k", k, dt, ks, dev)
    hv = _heads("attention", "v", v, dt, ks, dev)
    sequences = _sequences("attention", qs[:-2], offsets, dev)
    tokens, heads, kv, dim = qs[0] if len(qs) == 3 else _rows(qs[:-2]), qs[-2], ks[-2], qs[-1]
    _no_graph("attention", q, k, v)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (q, k, v, offsets, workspace),
                              lambda: attention(q, k, v, offsets, causal, scale, workspace))
    s = _raw_stream(dev.index)
    o = _like(q)
    lse = torch.empty(heads, tokens, dtype=torch.float32, device=dev)
    wp, wb, _keep = _space(workspace, lambda: attention_workspace(tokens, heads, kv, dim, dt, sequences), dev)
    st = _lib.load().dmuon_attention_forward(hq, hk, hv, _ptr(offsets), sequences, o.data_ptr(), lse.data_ptr(), tokens,
                                             heads, kv, dim, _dtype(dt), int(causal),
                                             _scale(scale, dim), wp, wb, s)
    _lib.check(st, "dmuon_attention_forward")
    return o, lse


def attention_backward(do, q, k, v, o, lse, offsets=None, causal=True, scale=None, workspace=None, stream=None):
    """``(dq, dk, dv)`` from the gradient of ``o`` and the inputs and outputs of ``attention``; dk and dv
    are summed over the query heads that share a key head."""
    where = "attention_backward"
    dt, dev = q.dtype, q.device
    qs, ks = _shapes(where, q, k)
    hq = _heads(where, "q", q, dt, qs, dev)
    hk = _heads(where, "k", k, dt, ks, dev)
    hv = _heads(where, "v", v, dt, ks, dev)
    ho = _heads(where, "do", do, dt, qs, dev)
    tokens, heads, kv, dim = _rows(qs[:-2]), qs[-2], ks[-2], qs[-1]
    _check(where, dev, dt, ("o", o, qs))
    _check(where, dev, torch.float32, ("lse", lse, (heads, tokens)))
    sequences = _sequences(where, qs[:-2], offsets, dev)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (q, k, v, do, o, lse, offsets, workspace),
                              lambda: attention_backward(do, q, k, v, o, lse, offsets, causal, scale, workspace))
    s = _raw_stream(dev.index)
    dq, dk, dv = _like(q), _like(k), _like(v)
    wp, wb, _keep = _space(workspace, lambda: attention_workspace(tokens, heads, kv, dim, dt, sequences, True), dev)
    st = _lib.load().dmuon_attention_backward(ho, hq, hk, hv, o.data_ptr(), lse.data_ptr(), _ptr(offsets), sequences,
                                              dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), tokens, heads, kv, dim,
                                              _dtype(dt), int(causal), _scale(scale, dim), wp, wb,
                                              s)
    _lib.check(st, "dmuon_attention_backward")
    return dq, dk, dv
