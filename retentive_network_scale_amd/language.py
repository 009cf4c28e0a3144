"""Binding of the operators around the layers of a language model (include/language.h):
argument marshalling only, as the package's other functions, on the helpers of
recurrent.py, whose rules of streams, devices and memory hold here too.

Leading axes are rows: ids of any shape, x of [..., K].  Rows of a wider tensor are read
in place where a function says so; they need unit stride inside and one stride between all.
"""
import ctypes
from collections import namedtuple

import torch

from . import _dtc, lib
from .recurrent import _bad, _Call, _dense, _rows

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32

GroupNormGateGrads = namedtuple("GroupNormGateGrads", "dx dgate dweight dbias")
LinearGrads = namedtuple("LinearGrads", "dx dw dbias")
BeamSelection = namedtuple("BeamSelection", "tokens parents scores")

_ACTIVATIONS = {None: 0, "gelu": 1, "silu": 2}


def _act(name):
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation must be None, 'gelu' or 'silu', got {name!r}")
    return _ACTIVATIONS[name]


def _addr(t):
    return None if t is None else t.data_ptr()


def embedding(ids, table, scale=1.0, out_dtype=None, out=None, stream=None):
    """out = scale table[ids]: ids int32 of any shape, table [V, D]; an id outside 0..V-1
    (padding: -1) gives zeros.  Returns out [*ids.shape, D]."""
    call = _Call(ids, "ids", stream)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must have 2 axes")
    v, d = table.shape
    out = call.out(out, "out", (*ids.shape, d), table.dtype if out_dtype is None and out is None else out_dtype)
    call.run(lib().embedding, _dense(ids, "ids", None, _I32, call.index), _dense(table, "table", None, None, call.index),
             out.data_ptr(), ids.numel(), v, d, float(scale), _dtc(table.dtype), _dtc(out.dtype))
    return out


def embedding_bwd_workspace_bytes(n, V, D):
    return int(lib().embedding_bwd_workspace_bytes(n, V, D))


def embedding_bwd(ids, d_o, V, scale=1.0, out_dtype=None, out=None, workspace=None, stream=None):
    """The table's gradient for d_o [*ids.shape, D] (rows of a wider tensor may be read in place):
    [V, D] of out_dtype (default: d_o's), every row written, each the sum of its tokens in their
    order."""
    call = _Call(ids, "ids", stream)
    d, n, lead = d_o.shape[-1], ids.numel(), ids.dim()
    op, old = _rows(d_o, "d_o", lead, (*ids.shape, d), d_o.dtype, call.index, d)
    out = call.out(out, "out", (V, d), d_o.dtype if out_dtype is None and out is None else out_dtype)
    ws, wp, wb = call.workspace(workspace, embedding_bwd_workspace_bytes(n, V, d))
    call.run(lib().embedding_bwd, _dense(ids, "ids", None, _I32, call.index), op, out.data_ptr(), n, V, d, old,
             float(scale), _dtc(d_o.dtype), _dtc(out.dtype), wp, wb)
    return out


def _norm_inputs(x, gate, weight, bias, lengths, call):
    """Addresses, strides and sizes that the norm's calls share."""
    if x.dim() != 4:
        raise ValueError("x must be [B, H, L, W]")
    b, h, L, w = x.shape
    ix, sb, sh, sl = call.index, *x.stride()[:3]
    if w > 1 and x.stride(3) != 1:
        raise ValueError(f"x needs channels next to each other, got strides {x.stride()}")
    if x.is_contiguous():  # axes of one element may have any stride
        sb, sh, sl = h * L * w, L * w, w
    else:
        sb, sh, sl = (s if n > 1 else w for s, n in ((sb, b), (sh, h), (sl, L)))
    gp, gld = _rows(gate, "gate", 2, (b, L, h * w), x.dtype, ix, h * w)
    return ((x.data_ptr(), gp, _dense(weight, "weight", (h * w,), _F32, ix), _dense(bias, "bias", (h * w,), _F32, ix)),
            _dense(lengths, "lengths", (b,), _I32, ix), (b, h, L, w), (sb, sh, sl, gld))


def group_norm_gate(x, gate=None, weight=None, bias=None, silu=True, eps=1e-5, lengths=None, out_dtype=None, out=None,
                    stream=None):
    """GroupNorm of each token and head times act(gate): x [B, H, L, W] (a retention's output, or
    any strides over its first three axes), gate [B, L, H W], weight and bias [H W] fp32, lengths
    int32 [B]; act is silu or, with silu=False, the identity, and without a gate it is applied to
    the norm itself.  Returns out [B, L, H W]."""
    call = _Call(x, "x", stream)
    ins, ln, (b, h, L, w), strides = _norm_inputs(x, gate, weight, bias, lengths, call)
    out = call.out(out, "out", (b, L, h * w), x.dtype if out_dtype is None and out is None else out_dtype)
    call.run(lib().group_norm_gate, *ins, out.data_ptr(), ln, b, h, L, w, *strides, int(bool(silu)), float(eps),
             _dtc(x.dtype), _dtc(out.dtype))
    return out


def group_norm_gate_bwd_workspace_bytes(B, H, L, W):
    return int(lib().group_norm_gate_bwd_workspace_bytes(B, H, L, W))


def group_norm_gate_bwd(x, d_o, gate=None, weight=None, bias=None, silu=True, eps=1e-5, lengths=None, out_dtype=None,
                        workspace=None, stream=None):
    """Gradients of group_norm_gate for d_o [B, L, H W]: a GroupNormGateGrads, dx [B, H, L, W] (dense,
    as retention_chunkwise_bwd takes it) and dgate of out_dtype (default: x's), dweight and dbias
    fp32; None where the input is None."""
    call = _Call(x, "x", stream)
    ins, ln, (b, h, L, w), strides = _norm_inputs(x, gate, weight, bias, lengths, call)
    od = x.dtype if out_dtype is None else out_dtype
    odc = _dtc(od)
    dx = call.empty((b, h, L, w), od)
    dg = None if gate is None else call.empty((b, L, h * w), od)
    dw = None if weight is None else call.empty((h * w,), _F32)
    db = None if bias is None else call.empty((h * w,), _F32)
    need = 0 if dw is None and db is None else group_norm_gate_bwd_workspace_bytes(b, h, L, w)
    ws, wp, wb = call.workspace(workspace, need) if need else (None, None, 0)
    call.run(lib().group_norm_gate_bwd, *ins, _dense(d_o, "d_o", (b, L, h * w), x.dtype, call.index), ln, dx.data_ptr(),
             _addr(dg), _addr(dw), _addr(db), b, h, L, w, *strides, int(bool(silu)), float(eps), _dtc(x.dtype), odc, wp,
             wb)
    return GroupNormGateGrads(dx, dg, dw, db)


def linear_workspace_bytes(M, N, K):
    return int(lib().linear_workspace_bytes(M, N, K))


def linear(x, w, bias=None, activation=None, residual=None, out_dtype=None, out=None, pre_out=None, workspace=None,
           stream=None):
    """out = act(x w^T + bias) + residual: x [..., K] bf16 (rows of a wider tensor are read in
    place), w [N, K] and bias [N] bf16, activation None, "gelu" or "silu", residual [..., N] bf16 or
    fp32 (out may be residual).  Returns out [..., N], bf16 or fp32 (out_dtype); with pre_out=True
    or a bf16 tensor (out, pre), pre being x w^T + bias for linear_bwd."""
    call = _Call(x, "x", stream)
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must have 2 axes")
    lead, (n, k), ix = x.shape[:-1], w.shape, call.index
    xp, xld = _rows(x, "x", x.dim() - 1, (*lead, k), _BF16, ix, k)
    out = call.out(out, "out", (*lead, n), x.dtype if out_dtype is None and out is None else out_dtype)
    if pre_out is True:
        pre_out = call.empty((*lead, n), _BF16)
    elif pre_out is False:
        pre_out = None
    m = x.numel() // max(k, 1)
    need = linear_workspace_bytes(m, n, k)
    ws, wp, wb = call.workspace(workspace, need) if need else (None, None, 0)
    call.run(lib().linear, xp, _dense(w, "w", None, _BF16, ix), _dense(bias, "bias", (n,), _BF16, ix),
             _dense(residual, "residual", (*lead, n), None, ix), out.data_ptr(),
             _dense(pre_out, "pre_out", (*lead, n), _BF16, ix), m, n, k, xld, _act(activation),
             1 if residual is None else _dtc(residual.dtype), _dtc(out.dtype), wp, wb)
    return out if pre_out is None else (out, pre_out)


def linear_bwd_workspace_bytes(M, N, K):
    return int(lib().linear_bwd_workspace_bytes(M, N, K))


def linear_bwd(x, w, d_o, pre=None, activation=None, dx=True, dw=True, dbias=False, out_dtype=None, workspace=None,
               stream=None):
    """Gradients of linear for d_o [..., N] bf16 and, with an activation, the forward call's pre: a
    LinearGrads, dx [..., K] and dw [N, K] of out_dtype (default bf16), dbias [N] fp32; None where
    not wanted.  The residual's gradient is d_o."""
    call = _Call(x, "x", stream)
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must have 2 axes")
    if activation is not None and pre is None:
        raise ValueError("pre is needed with an activation")
    lead, (n, k), ix = x.shape[:-1], w.shape, call.index
    xp, xld = _rows(x, "x", x.dim() - 1, (*lead, k), _BF16, ix, k)
    od = x.dtype if out_dtype is None else out_dtype
    odc, act, m = _dtc(od), _act(activation), x.numel() // max(k, 1)
    gx = call.empty((*lead, k), od) if dx else None
    gw = call.empty((n, k), od) if dw else None
    gb = call.empty((n,), _F32) if dbias else None
    ws, wp, wb = call.workspace(workspace, linear_bwd_workspace_bytes(m, n, k))
    call.run(lib().linear_bwd, xp, _dense(w, "w", None, _BF16, ix), _dense(d_o, "d_o", (*lead, n), _BF16, ix),
             _dense(pre, "pre", (*lead, n), _BF16, ix), _addr(gx), _addr(gw), _addr(gb), m, n, k, xld, act, odc, wp, wb)
    return LinearGrads(gx, gw, gb)


def beam_select_workspace_bytes(B, W, V, K):
    return int(lib().beam_select_workspace_bytes(B, W, V, K))


def beam_select(logits, scores, K, ended=None, eos=0, workspace=None, stream=None):
    """The K best continuations of every request by scores[b, w] + log_softmax(logits[b, w]):
    logits [B, W, V] bf16 or fp32 (rows of a wider tensor are read in place), scores [B, W] fp32,
    ended [B, W] bool or None (a beam that has ended offers eos at its own score).  Returns a
    BeamSelection: tokens and parents int32 [B, K], scores fp32 [B, K], best first, ties to the
    lowest beam, in it by logit and then to the lowest token."""
    call = _Call(logits, "logits", stream)
    if logits.dim() != 3:
        raise ValueError("logits must be [B, W, V]")
    b, w, v = logits.shape
    ix = call.index
    lp, ld = _rows(logits, "logits", 2, (b, w, v), logits.dtype, ix, v)
    if ended is not None and (not isinstance(ended, torch.Tensor) or ended.dtype not in (torch.bool, torch.uint8)):
        raise TypeError("ended must be a bool tensor")
    out = BeamSelection(call.empty((b, K), _I32), call.empty((b, K), _I32), call.empty((b, K), _F32))
    need = beam_select_workspace_bytes(b, w, v, K)
    ws, wp, wb = call.workspace(workspace, need) if need else (None, None, 0)
    call.run(lib().beam_select, lp, _dense(scores, "scores", (b, w), _F32, ix), _dense(ended, "ended", (b, w), None, ix),
             *(t.data_ptr() for t in out), b, w, v, K, ld, int(eos), _dtc(logits.dtype), wp, wb)
    return out


def beam_reorder(states, parents, stream=None):
    """states[i][b, w] <- states[i][b, parents[b, w]] in place, for one tensor or a sequence of them
    (up to 64; dense, any type, [B, W, ...] or [B W, ...] of whole beams), parents int32 [B, W]; a
    beam whose parent is outside 0..W-1 keeps its own.  Returns states."""
    call = _Call(parents, "parents", stream)
    if parents.dim() != 2:
        raise ValueError("parents must be [B, W]")
    b, w = parents.shape
    one = isinstance(states, torch.Tensor)
    every = [states] if one else list(states)
    n = len(every)
    at, size = (ctypes.c_void_p * max(n, 1))(), (ctypes.c_longlong * max(n, 1))()
    for i, t in enumerate(every):
        if not isinstance(t, torch.Tensor) or t.get_device() != call.index or not t.is_contiguous():
            _bad(t, f"states[{i}]", None, None, call.index)
        if t.dim() == 0 or not (t.shape[:2] == (b, w) or t.shape[0] == b * w):
            raise ValueError(f"states[{i}] must be [{b}, {w}, ...] or [{b * w}, ...], got {tuple(t.shape)}")
        at[i], size[i] = t.data_ptr(), t.numel() * t.element_size() // max(b * w, 1)
    call.run(lib().beam_reorder, at, size, n, _dense(parents, "parents", (b, w), _I32, call.index), b, w)
    return states
