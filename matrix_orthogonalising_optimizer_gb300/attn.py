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


def _heads(where, name, t, dtype, lead, heads, dim, dev):
    """The C ABI's view of (*lead, heads, dim); refuses what it cannot describe."""
    shape = (*lead, heads, dim)
    if not (t.is_cuda and t.dtype is dtype and t.shape == shape and t.device == dev):
        _refuse(where, name, t, dtype, shape, dev)
    strides, step, span = t.stride(), None, None
    if t.numel() and dim > 1 and strides[-1] != 1:
        raise ValueError(f"{where}: the last dimension of {name} must be contiguous")
    for n, s in zip(reversed(lead), reversed(strides[:-2])):
        if n == 1:
            continue
        if step is not None and s != span and t.numel():
            raise ValueError(f"{where}: the leading dimensions of {name} must have one stride")
        step = s if step is None else step
        span = s * n
    return _lib.Heads(t.data_ptr(), dim if step is None else step, strides[-2])


def _rows(lead):
    n = 1
    for x in lead:
        n *= x
    return n


def _sizes(where, q, k):
    """(dtype, device, leading dimensions, heads, key heads, dim) of a call."""
    if q.dim() < 2 or k.dim() < 2:
        raise ValueError(f"{where}: q and k must have a head and an element dimension")
    return q.dtype, q.device, q.shape[:-2], q.shape[-2], k.shape[-2], q.shape[-1]


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
    dt, dev, lead, heads, kv, dim = _sizes("qk_norm_rotary", q, k)
    hq = _heads("qk_norm_rotary", "q", q, dt, lead, heads, dim, dev)
    hk = _heads("qk_norm_rotary", "k", k, dt, lead, kv, dim, dev)
    rows, rotary = _rotary_check("qk_norm_rotary", lead, dev, dt, dim, positions, table, q_weight, k_weight)
    _no_graph("qk_norm_rotary", q, k, q_weight, k_weight)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (q, k, positions, table, q_weight, k_weight),
                              lambda: qk_norm_rotary(q, k, positions, table, q_weight, k_weight, norm, eps, interleaved))
    s = _raw_stream(dev.index)
    qo = torch.empty(q.shape, dtype=dt, device=dev)
    ko = torch.empty(k.shape, dtype=dt, device=dev)
    st = _lib.load().dmuon_qk_norm_rotary_forward(hq, hk, _ptr(positions), _ptr(table), rows, rotary, int(interleaved),
                                                  _ptr(q_weight), _ptr(k_weight), int(norm), eps, qo.data_ptr(),
                                                  ko.data_ptr(), _rows(lead), heads, kv, dim, _dtype(dt), s)
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
    dt, dev, lead, heads, kv, dim = _sizes(where, q, k)
    hq = _heads(where, "q", q, dt, lead, heads, dim, dev)
    hk = _heads(where, "k", k, dt, lead, kv, dim, dev)
    gq = _heads(where, "dq", dq, dt, lead, heads, dim, dev)
    gk = _heads(where, "dk", dk, dt, lead, kv, dim, dev)
    rows, rotary = _rotary_check(where, lead, dev, dt, dim, positions, table, q_weight, k_weight)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (q, k, dq, dk, positions, table, q_weight, k_weight, workspace),
                              lambda: qk_norm_rotary_backward(dq, dk, q, k, positions, table, q_weight, k_weight, norm,
                                                              eps, interleaved, workspace))
    s = _raw_stream(dev.index)
    tokens = _rows(lead)
    dx = torch.empty(q.shape, dtype=dt, device=dev)
    dy = torch.empty(k.shape, dtype=dt, device=dev)
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


def _sequences(where, lead, offsets, dev):
    """Sequences of the batch: those of ``offsets``, or one per row of the dimensions before the last."""
    if offsets is None:
        return max(1, _rows(lead[:-1]))
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"{where}: offsets must hold the sequences' starts and the last one's end")
    _check(where, dev, torch.int64, ("offsets", offsets, offsets.shape))
    return offsets.shape[0] - 1


def attention(q, k, v, offsets=None, causal=True, scale=None, workspace=None, stream=None):
    """``(o, lse)``: attention over whole sequences, ``scale`` 1 / sqrt(dim) if None.

    q is (tokens, heads, dim), k and v (tokens, kv_heads, dim), with heads / kv_heads query heads
    sharing a key head.  ``offsets`` (int64 on the device, sequences + 1) packs sequences of
    different lengths one behind the other: sequence s is tokens offsets[s] to offsets[s + 1], and
    tokens outside all of them get o = 0 and lse = -inf.  Without offsets the tokens are one
    sequence, or (batch, tokens, heads, dim) a batch of equal ones.  ``lse`` is (heads, all tokens)."""
    dt, dev, lead, heads, kv, dim = _sizes("attention", q, k)
    tokens = _rows(lead)
    hq = _heads("attention", "q", q, dt, lead, heads, dim, dev)
    hk = _heads("attention", "k", k, dt, lead, kv, dim, dev)
    hv = _heads("attention", "v", v, dt, lead, kv, dim, dev)
    sequences = _sequences("attention", lead, offsets, dev)
    _no_graph("attention", q, k, v)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (q, k, v, offsets, workspace),
                              lambda: attention(q, k, v, offsets, causal, scale, workspace))
    s = _raw_stream(dev.index)
    o = torch.empty(q.shape, dtype=dt, device=dev)
    lse = torch.empty(heads, tokens, dtype=torch.float32, device=dev)
    wp, wb, _keep = _space(workspace, lambda: attention_workspace(tokens, heads, kv, dim, dt, sequences), dev)
    st = _lib.load().dmuon_attention_forward(hq, hk, hv, _ptr(offsets), sequences, o.data_ptr(), lse.data_ptr(), tokens,
                                             heads, kv, dim, _dtype(dt), int(causal),
                                             dim ** -0.5 if scale is None else scale, wp, wb, s)
    _lib.check(st, "dmuon_attention_forward")
    return o, lse


def attention_backward(do, q, k, v, o, lse, offsets=None, causal=True, scale=None, workspace=None, stream=None):
    """``(dq, dk, dv)`` from the gradient of ``o`` and the inputs and outputs of ``attention``; dk and dv
    are summed over the query heads that share a key head."""
    where = "attention_backward"
    dt, dev, lead, heads, kv, dim = _sizes(where, q, k)
    tokens = _rows(lead)
    hq = _heads(where, "q", q, dt, lead, heads, dim, dev)
    hk = _heads(where, "k", k, dt, lead, kv, dim, dev)
    hv = _heads(where, "v", v, dt, lead, kv, dim, dev)
    ho = _heads(where, "do", do, dt, lead, heads, dim, dev)
    _check(where, dev, dt, ("o", o, q.shape))
    _check(where, dev, torch.float32, ("lse", lse, (heads, tokens)))
    sequences = _sequences(where, lead, offsets, dev)

    if _elsewhere(stream, dev):
        return _run_elsewhere(stream, (q, k, v, do, o, lse, offsets, workspace),
                              lambda: attention_backward(do, q, k, v, o, lse, offsets, causal, scale, workspace))
    s = _raw_stream(dev.index)
    dq = torch.empty(q.shape, dtype=dt, device=dev)
    dk = torch.empty(k.shape, dtype=dt, device=dev)
    dv = torch.empty(k.shape, dtype=dt, device=dev)
    wp, wb, _keep = _space(workspace, lambda: attention_workspace(tokens, heads, kv, dim, dt, sequences, True), dev)
    st = _lib.load().dmuon_attention_backward(ho, hq, hk, hv, o.data_ptr(), lse.data_ptr(), _ptr(offsets), sequences,
                                              dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), tokens, heads, kv, dim,
                                              _dtype(dt), int(causal), dim ** -0.5 if scale is None else scale, wp, wb,
                                              s)
    _lib.check(st, "dmuon_attention_backward")
    return dq, dk, dv
