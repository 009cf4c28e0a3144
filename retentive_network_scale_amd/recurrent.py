"""Binding of the recurrent-layer operators (include/recurrent.h) and of the decode
step with 4-bit weights: argument marshalling only, as the package's other functions.

Activations are token-major.  A slice of a wider projection's rows (x and z of one
[B, L, 2 D] tensor, B and C of another) is read in place: rows need unit stride inside
and one stride between all tokens.  Calls run on `stream` (default: the current stream
of the tensors' device) with that device current; what they allocate belongs to that
stream.
"""
from collections import namedtuple

import torch

from . import _check, _dtc, _host_f32, lib

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32

SelectiveScanGrads = namedtuple("SelectiveScanGrads", "du ddelta dA dB dC dD dz ddelta_bias d_state_in")
CausalConvGrads = namedtuple("CausalConvGrads", "dx dw dbias d_state_in")


# The calls here are short (a decode step's kernels take a few microseconds), so what
# every call does on the host is kept to a few comparisons per tensor.  Stream and device
# come from torch._C at the call: a torch built without a GPU runtime has no such names.


def _bad(t, name, shape, dtype, index):
    """Raises what is wrong with a tensor that failed a check."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{index}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _dense(t, name, shape, dtype, index):
    """Address of a contiguous tensor, or None."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.get_device() == index >= 0 and (dtype is None or t.dtype == dtype)
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        _bad(t, name, shape, dtype, index)
    return t.data_ptr()


def _rows(t, name, lead, shape, dtype, index, width):
    """(address, elements between one row and the next) of a tensor whose first `lead`
    axes are rows and whose others, `width` elements, are dense."""
    if t is None:
        return None, 0
    if not (isinstance(t, torch.Tensor) and t.get_device() == index >= 0 and t.dtype == dtype and t.shape == shape):
        _bad(t, name, shape, dtype, index)
    if t.is_contiguous():
        return t.data_ptr(), width
    strides = t.stride()
    ld = strides[lead - 1]
    if (shape[lead - 1] > 1 and ld >= width and (lead == 1 or strides[0] == shape[1] * ld) and strides[-1] == 1
            and (len(shape) == lead + 1 or strides[-2] == shape[-1])):
        return t.data_ptr(), ld
    want, bad = 1, False  # axes of one element may have any stride
    for n, s in zip(reversed(shape[lead:]), reversed(strides[lead:])):
        bad |= n > 1 and s != want
        want *= n
    ld, rows = None, 1
    for n, s in zip(reversed(shape[:lead]), reversed(strides[:lead])):
        if n > 1:
            ld = s if ld is None else ld
            bad |= s != rows * ld
        rows *= n
    ld = width if ld is None else ld
    if bad or ld < width:
        raise ValueError(f"{name} needs dense rows at one stride, got strides {strides}")
    return t.data_ptr(), ld


class _Call:
    """The device and stream of one call, from its first tensor."""
    __slots__ = ("index", "device", "stream", "raw")

    def __init__(self, t, name, stream):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a GPU tensor")
        self.index, self.device, self.stream = t.get_device(), t.device, stream
        if stream is None:
            self.raw = torch._C._cuda_getCurrentRawStream(self.index)
        else:
            if stream.device != self.device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {self.device}")
            self.raw = stream.cuda_stream

    def empty(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):  # the memory belongs to the call's stream
            return torch.empty(shape, dtype=dtype, device=self.device)

    def out(self, t, name, shape, dtype):
        """A caller's output, checked, or a new one."""
        if t is None:
            return self.empty(shape, dtype)
        _dense(t, name, shape, dtype, self.index)
        return t

    def workspace(self, t, need):
        """The caller's workspace or a new one (to be kept until the call), its address and bytes."""
        if t is None:
            t = self.empty(max(need, 16), torch.uint8)
        return t, _dense(t, "workspace", None, None, self.index), t.numel() * t.element_size()

    def run(self, fn, *args):
        if torch._C._cuda_getDevice() == self.index:
            status = fn(*args, self.raw)
        else:
            with torch.cuda.device(self.index):
                status = fn(*args, self.raw)
        if status:
            _check(status)


def selective_scan_workspace_bytes(B, L, D, N, G=1):
    return int(lib().selective_scan_workspace_bytes(B, L, D, N, G))


def selective_scan_bwd_workspace_bytes(B, L, D, N, G=1):
    return int(lib().selective_scan_bwd_workspace_bytes(B, L, D, N, G))


def _scan_inputs(u, delta, A, B, C, D, z, delta_bias, rows, call):
    """Addresses, row strides and sizes that the scan's calls share; rows: the leading axes."""
    dt, n, ix, d = u.dtype, len(rows), call.index, u.shape[-1]
    if not isinstance(B, torch.Tensor) or B.dim() != n + 2:
        raise ValueError(f"B must have {n + 2} axes")
    g, ns = B.shape[n:]
    wide, bc = (*rows, d), (*rows, g, ns)
    up, uld = _rows(u, "u", n, wide, dt, ix, d)
    dp, dld = _rows(delta, "delta", n, wide, dt, ix, d)
    zp, zld = _rows(z, "z", n, wide, dt, ix, d)
    bp, bld = _rows(B, "B", n, bc, dt, ix, g * ns)
    cp, cld = _rows(C, "C", n, bc, dt, ix, g * ns)
    return ((up, dp, _dense(A, "A", (d, ns), _F32, ix), bp, cp, _dense(D, "D", (d,), _F32, ix), zp,
             _dense(delta_bias, "delta_bias", (d,), _F32, ix)), (uld, dld, zld, bld, cld), (d, ns, g))


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=False, lengths=None,
                   state_in=None, state_out=None, out_dtype=None, out=None, workspace=None, stream=None):
    """h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t, out_t = (C_t . h_t + D u_t) silu(z_t) over L
    tokens; u, delta, z [Bt, L, Dm], A [Dm, N] fp32, B, C [Bt, L, G, N], D, delta_bias [Dm]
    fp32, lengths int32 [Bt].  Returns (out, state_out); pass state_out=True to have the
    [Bt, Dm, N] fp32 final state allocated, or a tensor (may be state_in)."""
    call = _Call(u, "u", stream)
    bt, L, _ = u.shape
    ins, lds, (d, n, g) = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, (bt, L), call)
    out = call.out(out, "out", (bt, L, d), u.dtype if out_dtype is None and out is None else out_dtype)
    f = _F32
    if state_out is True:
        state_out = call.empty((bt, d, n), f)
    elif state_out is False:
        state_out = None
    need = selective_scan_workspace_bytes(bt, L, d, n, g)
    ws, wp, wb = call.workspace(workspace, need) if need else (None, None, 0)
    call.run(lib().selective_scan, *ins, out.data_ptr(), _dense(lengths, "lengths", (bt,), _I32, call.index),
             _dense(state_in, "state_in", (bt, d, n), f, call.index),
             _dense(state_out, "state_out", (bt, d, n), f, call.index), bt, L, d, n, g, *lds, int(bool(delta_softplus)),
             _dtc(u.dtype), _dtc(out.dtype), wp, wb)
    return out, state_out


def selective_scan_bwd(u, delta, A, B, C, d_o, D=None, z=None, delta_bias=None, delta_softplus=False, lengths=None,
                       state_in=None, d_state_out=None, out_dtype=None, workspace=None, stream=None):
    """Gradients of selective_scan for the output gradient d_o [Bt, L, Dm] and, where given,
    the final state's gradient d_state_out: a SelectiveScanGrads, None where the input is
    None.  du, ddelta, dz, dB and dC are of out_dtype (default: u's), the others fp32."""
    call = _Call(u, "u", stream)
    bt, L, _ = u.shape
    ins, lds, (d, n, g) = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, (bt, L), call)
    od, f, dev = u.dtype if out_dtype is None else out_dtype, _F32, call.index
    odc = _dtc(od)
    du, ddelta = call.empty((bt, L, d), od), call.empty((bt, L, d), od)
    dA, dB, dC = call.empty((d, n), f), call.empty((bt, L, g, n), od), call.empty((bt, L, g, n), od)
    dD = None if D is None else call.empty((d,), f)
    dz = None if z is None else call.empty((bt, L, d), od)
    db = None if delta_bias is None else call.empty((d,), f)
    dh = None if state_in is None else call.empty((bt, d, n), f)
    ws, wp, wb = call.workspace(workspace, selective_scan_bwd_workspace_bytes(bt, L, d, n, g))
    outs = [None if t is None else t.data_ptr() for t in (du, ddelta, dA, dB, dC, dD, dz, db, dh)]
    call.run(lib().selective_scan_bwd, *ins, _dense(d_o, "d_o", (bt, L, d), u.dtype, dev),
             _dense(lengths, "lengths", (bt,), _I32, dev), _dense(state_in, "state_in", (bt, d, n), f, dev),
             _dense(d_state_out, "d_state_out", (bt, d, n), f, dev), *outs, bt, L, d, n, g, *lds,
             int(bool(delta_softplus)), _dtc(u.dtype), odc, wp, wb)
    return SelectiveScanGrads(du, ddelta, dA, dB, dC, dD, dz, db, dh)


def selective_scan_step(u, delta, A, B, C, state, D=None, z=None, delta_bias=None, delta_softplus=False,
                        out_dtype=None, out=None, stream=None):
    """One token of the scan: u, delta, z [Bt, Dm], B, C [Bt, G, N]; updates `state`
    [Bt, Dm, N] fp32 in place and returns out [Bt, Dm]."""
    call = _Call(u, "u", stream)
    bt, _ = u.shape
    ins, lds, (d, n, g) = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, (bt,), call)
    out = call.out(out, "out", (bt, d), u.dtype if out_dtype is None and out is None else out_dtype)
    call.run(lib().selective_scan_step, *ins, out.data_ptr(),
             _dense(state, "state", (bt, d, n), _F32, call.index), bt, d, n, g, *lds,
             int(bool(delta_softplus)), _dtc(u.dtype), _dtc(out.dtype))
    return out


def causal_conv1d(x, w, bias=None, silu=True, lengths=None, state_in=None, state_out=None, out=None, stream=None):
    """c_t = silu(bias + sum_j w_j x_{t-K+1+j}) per channel: x [Bt, L, Dm], w [Dm, K], bias [Dm]
    (one dtype), lengths int32 [Bt].  Returns (out, state_out): the states are the K - 1
    inputs before and at the end, [Bt, K-1, Dm], oldest first; state_out=True allocates it."""
    call = _Call(x, "x", stream)
    bt, L, d = x.shape
    k, dt, dev = w.shape[-1], x.dtype, call.index
    xp, xld = _rows(x, "x", 2, (bt, L, d), dt, dev, d)
    out = call.out(out, "out", (bt, L, d), dt)
    if state_out is True:
        state_out = call.empty((bt, k - 1, d), dt)
    elif state_out is False:
        state_out = None
    call.run(lib().causal_conv1d, xp, _dense(w, "w", (d, k), dt, dev), _dense(bias, "bias", (d,), dt, dev),
             out.data_ptr(), _dense(lengths, "lengths", (bt,), _I32, dev),
             _dense(state_in, "state_in", (bt, k - 1, d), dt, dev),
             _dense(state_out, "state_out", (bt, k - 1, d), dt, dev), bt, L, d, k, xld, int(bool(silu)), _dtc(x.dtype))
    return out, state_out


def causal_conv1d_bwd_workspace_bytes(B, L, D, K):
    return int(lib().causal_conv1d_bwd_workspace_bytes(B, L, D, K))


def causal_conv1d_bwd(x, w, d_o, bias=None, silu=True, lengths=None, state_in=None, d_state_out=None, workspace=None,
                      stream=None):
    """Gradients of causal_conv1d: a CausalConvGrads, dx and d_state_in of x's dtype, dw and
    dbias fp32; None where the input is None."""
    call = _Call(x, "x", stream)
    bt, L, d = x.shape
    k, dt, dev, f = w.shape[-1], x.dtype, call.index, _F32
    xp, xld = _rows(x, "x", 2, (bt, L, d), dt, dev, d)
    dx, dw = call.empty((bt, L, d), dt), call.empty((d, k), f)
    db = None if bias is None else call.empty((d,), f)
    dh = None if state_in is None else call.empty((bt, k - 1, d), dt)
    ws, wp, wb = call.workspace(workspace, causal_conv1d_bwd_workspace_bytes(bt, L, d, k))
    call.run(lib().causal_conv1d_bwd, xp, _dense(w, "w", (d, k), dt, dev), _dense(bias, "bias", (d,), dt, dev),
             _dense(d_o, "d_o", (bt, L, d), dt, dev), _dense(lengths, "lengths", (bt,), _I32, dev),
             _dense(state_in, "state_in", (bt, k - 1, d), dt, dev),
             _dense(d_state_out, "d_state_out", (bt, k - 1, d), dt, dev), dx.data_ptr(), dw.data_ptr(),
             None if db is None else db.data_ptr(), None if dh is None else dh.data_ptr(), bt, L, d, k, xld,
             int(bool(silu)), _dtc(x.dtype), wp, wb)
    return CausalConvGrads(dx, dw, db, dh)


def causal_conv1d_step(x, state, w, bias=None, silu=True, out=None, stream=None):
    """One token of the convolution: x [Bt, Dm]; shifts `state` [Bt, K-1, Dm] in place and
    returns out [Bt, Dm]."""
    call = _Call(x, "x", stream)
    bt, d = x.shape
    k, dt, dev = w.shape[-1], x.dtype, call.index
    xp, xld = _rows(x, "x", 1, (bt, d), dt, dev, d)
    out = call.out(out, "out", (bt, d), dt)
    call.run(lib().causal_conv1d_step, xp, _dense(w, "w", (d, k), dt, dev), _dense(bias, "bias", (d,), dt, dev),
             out.data_ptr(), _dense(state, "state", (bt, k - 1, d), dt, dev), bt, d, k, xld, int(bool(silu)), _dtc(x.dtype))
    return out


def pack_w4(q):
    """Whole numbers 0..15 [N, K] as linear_w4's bytes [N, K / 2]: element 2 i in the low half of byte i."""
    q = q.to(torch.uint8)
    return (q[:, 0::2] | q[:, 1::2] << 4).contiguous()


def _w4(q, scales, zeros, n, k, index, name):
    """Addresses and group size of a 4-bit matrix [n, k]."""
    if scales is None:
        raise TypeError(f"{name}scales must be a GPU tensor")
    sp, groups = _dense(scales, name + "scales", None, _BF16, index), scales.shape
    if len(groups) != 2 or groups[0] != n or groups[1] == 0 or k % groups[1]:
        raise ValueError(f"{name}scales must be [{n}, groups of {k}], got {tuple(groups)}")
    return (_dense(q, name + "qweight", (n, k // 2), torch.uint8, index), sp,
            _dense(zeros, name + "zeros", groups, torch.uint8, index), k // groups[1])


def linear_w4(x, qweight, scales, zeros=None, out_dtype=None, out=None, stream=None):
    """out = x W^T with W[n, k] = (q[n, k] - zero[n, k // group]) scale[n, k // group]: x [M, K]
    bf16, qweight [N, K/2] uint8 (pack_w4), scales [N, K/group] bf16, zeros [N, K/group] uint8
    (None: 8).  Returns out [M, N], bf16 or fp32 (out_dtype)."""
    call = _Call(x, "x", stream)
    m, k = x.shape
    xp, xld = _rows(x, "x", 1, (m, k), _BF16, call.index, k)
    n = qweight.shape[0]
    qp, sp, zp, group = _w4(qweight, scales, zeros, n, k, call.index, "")
    out = call.out(out, "out", (m, n), x.dtype if out_dtype is None and out is None else out_dtype)
    call.run(lib().linear_w4, xp, qp, sp, zp, out.data_ptr(), m, n, k, group, xld, _dtc(out.dtype))
    return out


def msr_layer_step_w4_workspace_bytes(B, d_model, H, dk, dv):
    return int(lib().msr_layer_step_w4_workspace_bytes(B, d_model, H, dk, dv))


def msr_layer_step_w4(x, w_in, w_o, state, pos, H, dk, dv, gamma, theta=None, gn_eps=1e-5, advance_pos=True, out=None,
                      workspace=None, stream=None):
    """msr_layer_step with 4-bit weights: w_in and w_o are (qweight, scales, zeros or None) as
    linear_w4's; w_in's rows are those of W_Q, W_K, W_V and W_G."""
    call = _Call(x, "x", stream)
    b, dm = x.shape
    dev = call.index
    iq, isc, iz, ig = _w4(*w_in, 2 * H * dk + 2 * H * dv, dm, dev, "w_in ")
    oq, osc, oz, og = _w4(*w_o, dm, H * dv, dev, "w_o ")
    out = call.out(out, "out", (b, dm), _BF16)
    g, gp = _host_f32(gamma, H, "gamma")
    th, thp = _host_f32(theta, dk // 2, "theta")
    ws, wp, wb = call.workspace(workspace, msr_layer_step_w4_workspace_bytes(b, dm, H, dk, dv))
    call.run(lib().msr_layer_step_w4, _dense(x, "x", (b, dm), _BF16, dev), iq, isc, iz, ig, oq, osc, oz, og,
             out.data_ptr(), _dense(state, "state", (b, H, dk, dv), _F32, dev),
             _dense(pos, "pos", (b,), _I32, dev), int(bool(advance_pos)), b, dm, H, dk, dv, gp, thp,
             float(gn_eps), wp, wb)
    return out
