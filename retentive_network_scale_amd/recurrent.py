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

from . import RET_BF16, RET_F32, RetentionError, _check, _dt, _dtc, _eps, _host_f32, _torch_dt, lib  # noqa: F401

SelectiveScanGrads = namedtuple("SelectiveScanGrads", "du ddelta dA dB dC dD dz ddelta_bias d_state_in")
CausalConvGrads = namedtuple("CausalConvGrads", "dx dw dbias d_state_in")


def _gpu(t, name, shape, dtype, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _dense(t, name, shape, dtype, device):
    """Address of a contiguous tensor, or None."""
    if t is None:
        return None
    if not _gpu(t, name, shape, dtype, device).is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, lead, shape, dtype, device):
    """(address, elements between one row and the next) of a tensor whose first `lead`
    axes are rows and whose others are dense."""
    if t is None:
        return None, 0
    _gpu(t, name, shape, dtype, device)
    width, bad = 1, False
    for n, s in zip(reversed(t.shape[lead:]), reversed(t.stride()[lead:])):
        bad |= n > 1 and s != width
        width *= n
    ld, rows = None, 1
    for n, s in zip(reversed(t.shape[:lead]), reversed(t.stride()[:lead])):
        if n > 1:
            ld = s if ld is None else ld
            bad |= s != rows * ld
        rows *= n
    ld = width if ld is None else ld
    if t.numel() and (bad or ld < width):
        raise ValueError(f"{name} needs dense rows at one stride, got strides {t.stride()}")
    return t.data_ptr(), max(ld, width)


class _Call:
    """The device and stream of one call."""

    def __init__(self, device, stream):
        self.device = device
        self.stream = torch.cuda.current_stream(device) if stream is None else stream
        if self.stream.device != device:
            raise ValueError(f"the stream is on {self.stream.device}, the tensors on {device}")

    def empty(self, shape, dtype):
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def out(self, t, name, shape, dtype):
        """A caller's output, checked, or a new one."""
        if t is None:
            return self.empty(shape, dtype)
        _dense(t, name, shape, dtype, self.device)
        return t

    def workspace(self, t, need):
        """(address, bytes) of the caller's workspace or a new one, and what keeps it alive."""
        if t is None:
            t = self.empty(max(need, 16), torch.uint8)
        return t, _dense(t, "workspace", None, None, self.device), t.numel() * t.element_size()

    def run(self, fn, *args):
        with torch.cuda.device(self.device):
            _check(fn(*args, self.stream.cuda_stream))


def _device_of(t, name):
    return _gpu(t, name, None, None, None).device


def selective_scan_workspace_bytes(B, L, D, N, G=1):
    return int(lib().selective_scan_workspace_bytes(B, L, D, N, G))


def selective_scan_bwd_workspace_bytes(B, L, D, N, G=1):
    return int(lib().selective_scan_bwd_workspace_bytes(B, L, D, N, G))


def _scan_inputs(u, delta, A, B, C, D, z, delta_bias, rows, call):
    """Addresses and row strides that the scan's calls share; rows: the leading axes."""
    dt, n, dev, d = u.dtype, len(rows), call.device, u.shape[-1]
    _dt(u)
    if B.dim() != n + 2:
        raise ValueError(f"B must have {n + 2} axes, got {tuple(B.shape)}")
    g, ns = B.shape[-2:]
    up, uld = _rows(u, "u", n, (*rows, d), dt, dev)
    dp, dld = _rows(delta, "delta", n, (*rows, d), dt, dev)
    zp, zld = _rows(z, "z", n, (*rows, d), dt, dev)
    bp, bld = _rows(B, "B", n, (*rows, g, ns), dt, dev)
    cp, cld = _rows(C, "C", n, (*rows, g, ns), dt, dev)
    f = torch.float32
    return ((up, dp, _dense(A, "A", (d, ns), f, dev), bp, cp, _dense(D, "D", (d,), f, dev), zp,
             _dense(delta_bias, "delta_bias", (d,), f, dev)), (uld, dld, zld, bld, cld), (d, ns, g))


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=False, lengths=None,
                   state_in=None, state_out=None, out_dtype=None, out=None, workspace=None, stream=None):
    """h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t, out_t = (C_t . h_t + D u_t) silu(z_t) over L
    tokens; u, delta, z [Bt, L, Dm], A [Dm, N] fp32, B, C [Bt, L, G, N], D, delta_bias [Dm]
    fp32, lengths int32 [Bt].  Returns (out, state_out); pass state_out=True to have the
    [Bt, Dm, N] fp32 final state allocated, or a tensor (may be state_in)."""
    call = _Call(_device_of(u, "u"), stream)
    bt, L, _ = u.shape
    ins, lds, (d, n, g) = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, (bt, L), call)
    out = call.out(out, "out", (bt, L, d), u.dtype if out_dtype is None and out is None else out_dtype)
    f = torch.float32
    if state_out is True:
        state_out = call.empty((bt, d, n), f)
    elif state_out is False:
        state_out = None
    need = selective_scan_workspace_bytes(bt, L, d, n, g)
    ws, wp, wb = call.workspace(workspace, need) if need else (None, None, 0)
    call.run(lib().selective_scan, *ins, out.data_ptr(), _dense(lengths, "lengths", (bt,), torch.int32, call.device),
             _dense(state_in, "state_in", (bt, d, n), f, call.device),
             _dense(state_out, "state_out", (bt, d, n), f, call.device), bt, L, d, n, g, *lds, int(bool(delta_softplus)),
             _dt(u), _dt(out), wp, wb)
    return out, state_out


def selective_scan_bwd(u, delta, A, B, C, d_o, D=None, z=None, delta_bias=None, delta_softplus=False, lengths=None,
                       state_in=None, d_state_out=None, out_dtype=None, workspace=None, stream=None):
    """Gradients of selective_scan for the output gradient d_o [Bt, L, Dm] and, where given,
    the final state's gradient d_state_out: a SelectiveScanGrads, None where the input is
    None.  du, ddelta, dz, dB and dC are of out_dtype (default: u's), the others fp32."""
    call = _Call(_device_of(u, "u"), stream)
    bt, L, _ = u.shape
    ins, lds, (d, n, g) = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, (bt, L), call)
    od, f, dev = u.dtype if out_dtype is None else out_dtype, torch.float32, call.device
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
             _dense(lengths, "lengths", (bt,), torch.int32, dev), _dense(state_in, "state_in", (bt, d, n), f, dev),
             _dense(d_state_out, "d_state_out", (bt, d, n), f, dev), *outs, bt, L, d, n, g, *lds,
             int(bool(delta_softplus)), _dt(u), odc, wp, wb)
    return SelectiveScanGrads(du, ddelta, dA, dB, dC, dD, dz, db, dh)


def selective_scan_step(u, delta, A, B, C, state, D=None, z=None, delta_bias=None, delta_softplus=False,
                        out_dtype=None, out=None, stream=None):
    """One token of the scan: u, delta, z [Bt, Dm], B, C [Bt, G, N]; updates `state`
    [Bt, Dm, N] fp32 in place and returns out [Bt, Dm]."""
    call = _Call(_device_of(u, "u"), stream)
    bt, _ = u.shape
    ins, lds, (d, n, g) = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, (bt,), call)
    out = call.out(out, "out", (bt, d), u.dtype if out_dtype is None and out is None else out_dtype)
    call.run(lib().selective_scan_step, *ins, out.data_ptr(),
             _dense(state, "state", (bt, d, n), torch.float32, call.device), bt, d, n, g, *lds,
             int(bool(delta_softplus)), _dt(u), _dt(out))
    return out


def causal_conv1d(x, w, bias=None, silu=True, lengths=None, state_in=None, state_out=None, out=None, stream=None):
    """c_t = silu(bias + sum_j w_j x_{t-K+1+j}) per channel: x [Bt, L, Dm], w [Dm, K], bias [Dm]
    (one dtype), lengths int32 [Bt].  Returns (out, state_out): the states are the K - 1
    inputs before and at the end, [Bt, K-1, Dm], oldest first; state_out=True allocates it."""
    call = _Call(_device_of(x, "x"), stream)
    bt, L, d = x.shape
    k, dt, dev = w.shape[-1], x.dtype, call.device
    xp, xld = _rows(x, "x", 2, (bt, L, d), dt, dev)
    out = call.out(out, "out", (bt, L, d), dt)
    if state_out is True:
        state_out = call.empty((bt, k - 1, d), dt)
    elif state_out is False:
        state_out = None
    call.run(lib().causal_conv1d, xp, _dense(w, "w", (d, k), dt, dev), _dense(bias, "bias", (d,), dt, dev),
             out.data_ptr(), _dense(lengths, "lengths", (bt,), torch.int32, dev),
             _dense(state_in, "state_in", (bt, k - 1, d), dt, dev),
             _dense(state_out, "state_out", (bt, k - 1, d), dt, dev), bt, L, d, k, xld, int(bool(silu)), _dt(x))
    return out, state_out


def causal_conv1d_bwd_workspace_bytes(B, L, D, K):
    return int(lib().causal_conv1d_bwd_workspace_bytes(B, L, D, K))


def causal_conv1d_bwd(x, w, d_o, bias=None, silu=True, lengths=None, state_in=None, d_state_out=None, workspace=None,
                      stream=None):
    """Gradients of causal_conv1d: a CausalConvGrads, dx and d_state_in of x's dtype, dw and
    dbias fp32; None where the input is None."""
    call = _Call(_device_of(x, "x"), stream)
    bt, L, d = x.shape
    k, dt, dev, f = w.shape[-1], x.dtype, call.device, torch.float32
    xp, xld = _rows(x, "x", 2, (bt, L, d), dt, dev)
    dx, dw = call.empty((bt, L, d), dt), call.empty((d, k), f)
    db = None if bias is None else call.empty((d,), f)
    dh = None if state_in is None else call.empty((bt, k - 1, d), dt)
    ws, wp, wb = call.workspace(workspace, causal_conv1d_bwd_workspace_bytes(bt, L, d, k))
    call.run(lib().causal_conv1d_bwd, xp, _dense(w, "w", (d, k), dt, dev), _dense(bias, "bias", (d,), dt, dev),
             _dense(d_o, "d_o", (bt, L, d), dt, dev), _dense(lengths, "lengths", (bt,), torch.int32, dev),
             _dense(state_in, "state_in", (bt, k - 1, d), dt, dev),
             _dense(d_state_out, "d_state_out", (bt, k - 1, d), dt, dev), dx.data_ptr(), dw.data_ptr(),
             None if db is None else db.data_ptr(), None if dh is None else dh.data_ptr(), bt, L, d, k, xld,
             int(bool(silu)), _dt(x), wp, wb)
    return CausalConvGrads(dx, dw, db, dh)


def causal_conv1d_step(x, state, w, bias=None, silu=True, out=None, stream=None):
    """One token of the convolution: x [Bt, Dm]; shifts `state` [Bt, K-1, Dm] in place and
    returns out [Bt, Dm]."""
    call = _Call(_device_of(x, "x"), stream)
    bt, d = x.shape
    k, dt, dev = w.shape[-1], x.dtype, call.device
    xp, xld = _rows(x, "x", 1, (bt, d), dt, dev)
    out = call.out(out, "out", (bt, d), dt)
    call.run(lib().causal_conv1d_step, xp, _dense(w, "w", (d, k), dt, dev), _dense(bias, "bias", (d,), dt, dev),
             out.data_ptr(), _dense(state, "state", (bt, k - 1, d), dt, dev), bt, d, k, xld, int(bool(silu)), _dt(x))
    return out


def pack_w4(q):
    """Whole numbers 0..15 [N, K] as linear_w4's bytes [N, K / 2]: element 2 i in the low half of byte i."""
    q = q.to(torch.uint8)
    return (q[:, 0::2] | q[:, 1::2] << 4).contiguous()


def _w4(q, scales, zeros, n, k, device, name):
    """Addresses and group size of a 4-bit matrix [n, k]."""
    _gpu(scales, f"{name}scales", None, torch.bfloat16, device)
    if scales.dim() != 2 or scales.shape[0] != n or scales.shape[1] == 0 or k % scales.shape[1]:
        raise ValueError(f"{name}scales must be [{n}, groups of {k}], got {tuple(scales.shape)}")
    return (_dense(q, f"{name}qweight", (n, k // 2), torch.uint8, device),
            _dense(scales, f"{name}scales", None, None, device),
            _dense(zeros, f"{name}zeros", tuple(scales.shape), torch.uint8, device), k // scales.shape[1])


def linear_w4(x, qweight, scales, zeros=None, out_dtype=None, out=None, stream=None):
    """out = x W^T with W[n, k] = (q[n, k] - zero[n, k // group]) scale[n, k // group]: x [M, K]
    bf16, qweight [N, K/2] uint8 (pack_w4), scales [N, K/group] bf16, zeros [N, K/group] uint8
    (None: 8).  Returns out [M, N], bf16 or fp32 (out_dtype)."""
    call = _Call(_device_of(x, "x"), stream)
    m, k = x.shape
    xp, xld = _rows(x, "x", 1, (m, k), torch.bfloat16, call.device)
    n = qweight.shape[0]
    qp, sp, zp, group = _w4(qweight, scales, zeros, n, k, call.device, "")
    out = call.out(out, "out", (m, n), x.dtype if out_dtype is None and out is None else out_dtype)
    call.run(lib().linear_w4, xp, qp, sp, zp, out.data_ptr(), m, n, k, group, xld, _dt(out))
    return out


def msr_layer_step_w4_workspace_bytes(B, d_model, H, dk, dv):
    return int(lib().msr_layer_step_w4_workspace_bytes(B, d_model, H, dk, dv))


def msr_layer_step_w4(x, w_in, w_o, state, pos, H, dk, dv, gamma, theta=None, gn_eps=1e-5, advance_pos=True, out=None,
                      workspace=None, stream=None):
    """msr_layer_step with 4-bit weights: w_in and w_o are (qweight, scales, zeros or None) as
    linear_w4's; w_in's rows are those of W_Q, W_K, W_V and W_G."""
    call = _Call(_device_of(x, "x"), stream)
    b, dm = x.shape
    dev = call.device
    iq, isc, iz, ig = _w4(*w_in, 2 * H * dk + 2 * H * dv, dm, dev, "w_in ")
    oq, osc, oz, og = _w4(*w_o, dm, H * dv, dev, "w_o ")
    out = call.out(out, "out", (b, dm), torch.bfloat16)
    g, gp = _host_f32(gamma, H, "gamma")
    th, thp = _host_f32(theta, dk // 2, "theta")
    ws, wp, wb = call.workspace(workspace, msr_layer_step_w4_workspace_bytes(b, dm, H, dk, dv))
    call.run(lib().msr_layer_step_w4, _dense(x, "x", (b, dm), torch.bfloat16, dev), iq, isc, iz, ig, oq, osc, oz, og,
             out.data_ptr(), _dense(state, "state", (b, H, dk, dv), torch.float32, dev),
             _dense(pos, "pos", (b,), torch.int32, dev), int(bool(advance_pos)), b, dm, H, dk, dv, gp, thp,
             float(gn_eps), wp, wb)
    return out
