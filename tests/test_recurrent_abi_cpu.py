"""C-ABI checks of the recurrent-layer operators that need no GPU: exports, and the refusal
of bad arguments on the host before any launch (no call here reaches a kernel)."""
import ctypes
import os
import re

import pytest
import torch

import retentive_network_scale_amd as rn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
F32, BF16 = 0, 1


def P(i, off=0):
    """A stand-in address, never dereferenced; 16 MiB apart."""
    return ctypes.c_void_p((i << 24) + off)


def test_every_declared_symbol_is_exported_and_bound():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "recurrent.h")).read(), flags=re.S)
    names = set(re.findall(r"\b((?:selective|causal|linear)_\w+)\s*\(", src))
    assert names == set(rn.RECURRENT_SYMBOLS)
    for n in names:
        assert hasattr(rn.lib(), n), n


def _scan(fn="selective_scan", **kw):
    v = dict(u=P(1), delta=P(2), A=P(3), B=P(4), C=P(5), D=P(6), z=P(7), bias=P(8), out=P(9), lengths=None, h0=P(10),
             hT=P(11), bt=2, L=600, d=64, n=16, g=2, uld=64, dld=64, zld=64, bld=32, cld=32, sp=1, ind=BF16, outd=BF16,
             ws=P(12), wb=1 << 23)
    v.update(kw)
    return rn.lib().selective_scan(*(v[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "bias", "out", "lengths", "h0",
                                                    "hT", "bt", "L", "d", "n", "g", "uld", "dld", "zld", "bld", "cld",
                                                    "sp", "ind", "outd", "ws", "wb")), None)


@pytest.mark.parametrize("kw,code", [
    (dict(bt=0), INVALID), (dict(L=-1), INVALID), (dict(d=0), INVALID), (dict(n=0), INVALID), (dict(g=0), INVALID),
    (dict(g=3), INVALID), (dict(n=65, bld=130, cld=130), UNSUPPORTED), (dict(ind=7), INVALID), (dict(outd=-1), INVALID),
    (dict(u=None), INVALID), (dict(delta=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(C=None), INVALID), (dict(out=None), INVALID), (dict(uld=63), INVALID), (dict(bld=31), INVALID),
    (dict(zld=10), INVALID), (dict(uld=1 << 40), UNSUPPORTED), (dict(u=P(1, 1)), INVALID), (dict(A=P(3, 2)), INVALID),
    (dict(out=P(9, 1)), INVALID), (dict(lengths=P(13, 2)), INVALID), (dict(hT=P(11, 1)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wb=100), WORKSPACE), (dict(ws=P(12, 8)), INVALID), (dict(out=P(1)), INVALID),
    (dict(out=P(1, 100)), INVALID), (dict(hT=P(2)), INVALID), (dict(hT=P(10, 64)), INVALID), (dict(out=P(10)), INVALID),
    (dict(ws=P(4)), INVALID), (dict(ws=P(9)), INVALID), (dict(ws=P(10)), INVALID), (dict(lengths=P(9)), INVALID),
    (dict(bt=1 << 20, L=1 << 10), UNSUPPORTED), (dict(bt=1 << 20, L=1, d=1 << 20, g=1, uld=1 << 20, dld=1 << 20), UNSUPPORTED),
    # grids of 2^32 threads and more: too many channels, states, or groups of few channels
    (dict(bt=1, L=1, d=1 << 21, g=1, uld=1 << 21, dld=1 << 21, zld=1 << 21), UNSUPPORTED),
    (dict(bt=1 << 16, L=1, d=1 << 12, g=1, uld=1 << 12, dld=1 << 12, zld=1 << 12), UNSUPPORTED),
    (dict(bt=1 << 18, L=1, d=64, n=1, g=64, bld=64, cld=64), UNSUPPORTED),
])
def test_scan_refuses(kw, code):
    assert _scan(**kw) == code
    assert rn.lib().retention_last_error() != b""


def test_scan_workspace_queries():
    L = rn.lib()
    assert L.selective_scan_workspace_bytes(2, 600, 64, 16, 2) > 0
    assert L.selective_scan_workspace_bytes(1, 16, 64, 16, 1) == 0  # one segment
    for bad in ((0, 600, 64, 16, 2), (2, 0, 64, 16, 2), (2, 600, 64, 65, 2), (2, 600, 64, 16, 3), (1 << 20, 1 << 12, 64, 16, 1)):
        assert L.selective_scan_workspace_bytes(*bad) == 0 == L.selective_scan_bwd_workspace_bytes(*bad), bad


def _bwd(**kw):
    v = dict(u=P(1), delta=P(2), A=P(3), B=P(4), C=P(5), D=P(6), z=P(7), bias=P(8), d_o=P(9), lengths=None, h0=P(10),
             dhT=P(11), du=P(12), dd=P(13), dA=P(14), dB=P(15), dC=P(16), dD=P(17), dz=P(18), db=P(19), dh0=P(20),
             bt=2, L=60, d=64, n=16, g=2, uld=64, dld=64, zld=64, bld=32, cld=32, sp=1, ind=BF16, outd=BF16, ws=P(21),
             wb=1 << 24)
    v.update(kw)
    return rn.lib().selective_scan_bwd(*(v[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "bias", "d_o", "lengths", "h0",
                                                        "dhT", "du", "dd", "dA", "dB", "dC", "dD", "dz", "db", "dh0", "bt",
                                                        "L", "d", "n", "g", "uld", "dld", "zld", "bld", "cld", "sp", "ind",
                                                        "outd", "ws", "wb")), None)


@pytest.mark.parametrize("kw,code", [
    (dict(d_o=None), INVALID), (dict(du=None), INVALID), (dict(dd=None), INVALID), (dict(dA=None), INVALID),
    (dict(dB=None), INVALID), (dict(dC=None), INVALID), (dict(dz=None), INVALID), (dict(z=None), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wb=1000), WORKSPACE), (dict(ws=P(21, 4)), INVALID), (dict(du=P(1)), INVALID),
    (dict(dd=P(12, 64)), INVALID), (dict(dh0=P(11)), INVALID), (dict(dA=P(3)), INVALID), (dict(dC=P(15)), INVALID),
    (dict(ws=P(9)), INVALID), (dict(dD=P(17, 2)), INVALID), (dict(dB=P(15, 1)), INVALID), (dict(g=5), INVALID),
    (dict(n=80), UNSUPPORTED), (dict(cld=16), INVALID), (dict(ind=3), INVALID), (dict(L=0, dA=None), INVALID),
    (dict(bt=1 << 18, L=1, d=64, n=1, g=64, bld=64, cld=64), UNSUPPORTED),
])
def test_scan_bwd_refuses(kw, code):
    assert _bwd(**kw) == code
    assert rn.lib().retention_last_error() != b""


def _step(**kw):
    v = dict(u=P(1), delta=P(2), A=P(3), B=P(4), C=P(5), D=P(6), z=P(7), bias=P(8), out=P(9), h=P(10), bt=2, d=64, n=16,
             g=1, uld=64, dld=64, zld=64, bld=16, cld=16, sp=1, ind=F32, outd=F32)
    v.update(kw)
    return rn.lib().selective_scan_step(*v.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(h=None), INVALID), (dict(out=None), INVALID), (dict(h=P(1)), INVALID), (dict(out=P(10)), INVALID),
    (dict(h=P(10, 2)), INVALID), (dict(n=100), UNSUPPORTED), (dict(bt=-1), INVALID), (dict(zld=5), INVALID),
    (dict(bt=1 << 18, n=1, g=64, bld=64, cld=64), UNSUPPORTED),
])
def test_scan_step_refuses(kw, code):
    assert _step(**kw) == code


def _conv(**kw):
    v = dict(x=P(1), w=P(2), bias=P(3), out=P(4), lengths=None, s0=P(5), sT=P(6), bt=2, L=50, d=64, k=4, xld=64, silu=1,
             dt=BF16)
    v.update(kw)
    return rn.lib().causal_conv1d(*v.values(), None)


def _conv_bwd(**kw):
    v = dict(x=P(1), w=P(2), bias=P(3), d_o=P(4), lengths=None, s0=P(5), dsT=P(6), dx=P(7), dw=P(8), db=P(9), ds0=P(10),
             bt=2, L=50, d=64, k=4, xld=64, silu=1, dt=BF16, ws=P(11), wb=1 << 20)
    v.update(kw)
    return rn.lib().causal_conv1d_bwd(*v.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(bt=0), INVALID), (dict(L=-1), INVALID), (dict(d=0), INVALID), (dict(k=0), INVALID), (dict(k=1), UNSUPPORTED),
    (dict(k=9), UNSUPPORTED), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(xld=60), INVALID),
    (dict(dt=2), INVALID), (dict(x=P(1, 1)), INVALID), (dict(xld=1 << 33), UNSUPPORTED),
    (dict(d=1 << 21, xld=1 << 21), UNSUPPORTED), (dict(bt=1 << 20, L=1, d=1 << 10, xld=1 << 10), UNSUPPORTED),
])
def test_conv_refuses(kw, code):
    assert _conv(**kw) == code
    assert _conv_bwd(**kw) == code


def test_conv_refuses_overlaps_and_workspaces():
    for kw in (dict(out=P(1)), dict(sT=P(5)), dict(sT=P(4)), dict(out=P(5)), dict(out=None), dict(lengths=P(12, 1))):
        assert _conv(**kw) == INVALID, kw
    for kw in (dict(dx=P(4)), dict(dw=P(2)), dict(ds0=P(6)), dict(dw=None), dict(dx=None), dict(ws=P(4)), dict(dw=P(8, 2))):
        assert _conv_bwd(**kw) == INVALID, kw
    assert _conv_bwd(ws=None) == WORKSPACE == _conv_bwd(wb=64)
    # 2^24 workgroups of 256 threads
    assert _conv_bwd(bt=1 << 24, L=1, d=1, xld=1, x=P(1, 0), ws=P(200), wb=1 << 33, dx=P(100), d_o=P(120), s0=None, dsT=None,
                     ds0=None) == UNSUPPORTED
    lib = rn.lib()
    assert lib.causal_conv1d_bwd_workspace_bytes(2, 50, 64, 4) > 0
    assert lib.causal_conv1d_bwd_workspace_bytes(2, 0, 64, 4) == 0 == lib.causal_conv1d_bwd_workspace_bytes(2, 50, 64, 9)
    r = lib.causal_conv1d_step(P(1), P(2), P(3), P(4), P(4), 2, 64, 4, 64, 1, BF16, None)
    assert r == INVALID and lib.causal_conv1d_step(P(1), P(2), P(3), P(4), None, 2, 64, 4, 64, 1, BF16, None) == INVALID


def _w4(**kw):
    v = dict(x=P(1), q=P(2), s=P(3), z=P(4), out=P(5), m=3, n=48, k=256, g=128, xld=256, od=BF16)
    v.update(kw)
    return rn.lib().linear_w4(*v.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(m=-1), INVALID),
    (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(g=0), INVALID), (dict(g=16), UNSUPPORTED), (dict(g=96), UNSUPPORTED),
    (dict(k=192, xld=192), UNSUPPORTED), (dict(q=P(2, 4)), INVALID), (dict(s=P(3, 1)), INVALID), (dict(xld=255), INVALID),
    (dict(out=P(1)), INVALID), (dict(out=P(2)), INVALID), (dict(out=P(4)), INVALID), (dict(od=5), INVALID),
    (dict(m=1 << 30), UNSUPPORTED), (dict(n=(1 << 26) + 1), UNSUPPORTED), (dict(k=1 << 27, xld=1 << 27), UNSUPPORTED),
])
def test_w4_refuses(kw, code):
    assert _w4(**kw) == code
    assert rn.lib().retention_last_error() != b""


def test_w4_without_rows_is_a_noop():
    assert _w4(m=0, x=None, out=None) == 0


def test_msr_step_w4_refuses():
    lib = rn.lib()
    gamma = (ctypes.c_float * 2)(0.9, 0.9)
    need = lib.msr_layer_step_w4_workspace_bytes(4, 256, 2, 64, 128)
    assert need >= 4 * (2 * 2 * 64 + 2 * 2 * 128) * 4 + 4 * 2 * 128 * 2
    assert lib.msr_layer_step_w4_workspace_bytes(0, 256, 2, 64, 128) == 0

    def call(x=P(1), iq=P(2), ig=64, oq=P(3), y=P(4), state=P(5), pos=P(6), dm=256, ws=P(7), wb=need, eps=1e-5, osc=P(9)):
        return lib.msr_layer_step_w4(x, iq, P(8), None, ig, oq, osc, None, 64, y, state, pos, 1, 4, dm, 2, 64, 128, gamma,
                                     None, eps, ws, wb, None)
    for kw in (dict(x=None), dict(iq=None), dict(oq=None), dict(osc=None), dict(y=None), dict(state=None), dict(pos=None),
               dict(eps=-1.0), dict(y=P(1)), dict(state=P(7)), dict(y=P(3)), dict(ws=P(2)), dict(pos=P(6, 2)), dict(pos=P(5))):
        assert call(**kw) == INVALID, kw
    assert call(ig=48) == UNSUPPORTED == call(dm=200)
    assert call(wb=need - 1) == WORKSPACE == call(ws=None)


def test_binding_refuses_what_is_not_on_a_gpu():
    t = torch.zeros(1, 4, 8)
    for fn in (lambda: rn.selective_scan(t, t, t, t, t), lambda: rn.causal_conv1d(t, t[0]),
               lambda: rn.selective_scan_step(t, t, t, t, t, t), lambda: rn.linear_w4(t[0], t, t)):
        with pytest.raises(TypeError):
            fn()


def test_pack_w4():
    q = torch.tensor([[1, 2, 15, 0], [3, 4, 5, 6]])
    assert rn.pack_w4(q).tolist() == [[0x21, 0x0F], [0x43, 0x65]]
