"""GPU parity of the recurrent-layer operators at the sizes whose kernels small calls do not reach: passes of two
channels a lane, single tokens four sequences at a time, long runs of the convolution, 4-bit products over several
chunks of K in every tile; and the widths of states between them.  Channels do not mix (in the gradients: where the others' output gradient is zero), so the
64-bit forms compute a few of them, spread over the tiles; tolerances are test_gpu_recurrent's."""
import pytest
import torch

import retentive_network_scale_amd as rn
from tests.test_gpu_recurrent import (BF, DEV, F32, _bwd, _check_bwd, _check_conv, _check_conv_bwd, _check_scan, _check_w4,
                                      _dev, _scan_gpu, _scan_inputs, _w4_inputs)

pytestmark = pytest.mark.gpu
SIMDS = 1024


def _cdiv(a, b):
    return -(-a // b)


def _waves(bt, d, G, channels):
    return bt * G * _cdiv(d // G, channels)


def _picked(d, G, per_group, gen):
    """Channels spread over every group, the first and the last of each among them, in order."""
    dg = d // G
    inner = torch.randperm(dg - 2, generator=gen)[:per_group - 2] + 1
    one = torch.sort(torch.cat([torch.tensor([0, dg - 1]), inner]))[0]
    return torch.cat([g * dg + one for g in range(G)])


def _scan_big(bt, L, d, n, G, dt, seed, lengths=None):
    """Device tensors of a scan (u and z, B and C side by side in one row, as projections leave them); rows behind an
    end hold NaN."""
    g = torch.Generator(DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    xz, bc, delta = r(bt, L, 2 * d).to(dt), r(bt, L, 2 * G * n).to(dt), (0.5 * r(bt, L, d)).to(dt)
    for b, end in enumerate(lengths or []):
        for t in (xz, bc, delta):
            t[b, end:] = float("nan")
    return dict(u=xz[..., :d], z=xz[..., d:], delta=delta, A=-2 * torch.rand(d, n, generator=g, device=DEV),
                B=bc[..., :G * n].unflatten(-1, (G, n)), C=bc[..., G * n:].unflatten(-1, (G, n)), D=r(d), bias=0.3 * r(d),
                h0=r(bt, d, n))


def _of(v, ch):
    """The picked channels, on the CPU."""
    at = ch.to(DEV)
    last = {k: v[k][..., at].cpu() for k in ("u", "z", "delta", "D", "bias")}
    return last | {"A": v["A"][at].cpu(), "B": v["B"].cpu(), "C": v["C"].cpu(), "h0": v["h0"][:, at].cpu()}


def _args(v):
    return (v["u"], v["delta"], v["A"], v["B"], v["C"]), dict(D=v["D"], z=v["z"], delta_bias=v["bias"], delta_softplus=True)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d,n,G", [(12288, 4, 1), (12296, 8, 2), (12288, 12, 1), (12300, 16, 1), (12304, 20, 4), (12288, 32, 1)])
def test_scan_two_channels_a_lane(d, n, G, dt):
    """Uncut: three waves of 32 channels per SIMD and more."""
    bt, L = 8, 35
    assert _waves(bt, d, G, 32) >= 3 * SIMDS and d // G % 4 == 0
    lengths = [35, 17, 32, 0, 1, 35, 33, 16]
    v = _scan_big(bt, L, d, n, G, dt, 200, lengths)
    args, kw = _args(v)
    out, st = rn.selective_scan(*args, state_in=v["h0"], state_out=True, out=torch.zeros(bt, L, d, dtype=dt, device=DEV),
                                lengths=torch.tensor(lengths, dtype=torch.int32, device=DEV), **kw)
    ch = _picked(d, G, 24 // G, torch.Generator().manual_seed(201))
    at = ch.to(DEV)
    _check_scan(_of(v, ch), True, lengths, out[..., at], st[:, at], f"{d} {n} {G}")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d,n,G", [(4100, 4, 1), (4104, 8, 2), (4100, 16, 1), (4104, 24, 2), (4100, 32, 1)])
def test_scan_two_channels_a_lane_in_segments(d, n, G, dt):
    """Cut: less than a wave of 16 channels per SIMD, three of 32 with the segments; ends inside a segment."""
    bt, L = 2, 725
    assert _waves(bt, d, G, 16) < SIMDS and _waves(bt, d, G, 32) * _cdiv(L, 64) >= 3 * SIMDS
    lengths = [L, 451]
    v = _scan_big(bt, L, d, n, G, dt, 202, lengths)
    args, kw = _args(v)
    out, st = rn.selective_scan(*args, state_in=v["h0"], state_out=True, out=torch.zeros(bt, L, d, dtype=dt, device=DEV),
                                lengths=torch.tensor(lengths, dtype=torch.int32, device=DEV), **kw)
    ch = _picked(d, G, 24 // G, torch.Generator().manual_seed(203))
    at = ch.to(DEV)
    _check_scan(_of(v, ch), True, lengths, out[..., at], st[:, at], f"{d} {n} {G}")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d,n,G", [(4100, 4, 1), (4104, 8, 2), (4100, 16, 1), (4104, 24, 2), (4100, 32, 1)])
def test_scan_bwd_two_channels_a_lane(d, n, G, dt):
    """Checkpoints of 32 channels a wave, spans of several segments; ends inside a segment."""
    bt, L = 2, 400
    assert _waves(bt, d, G, 32) * _cdiv(L, 32) >= 3 * SIMDS
    four = 4 * 16 * (1 if n > 16 else 2)  # channels of the main pass's workgroups
    span = 16 * _cdiv(_cdiv(L, min(_cdiv(2048, 4 * _waves(bt, d, G, four)), _cdiv(L, 32))), 16)
    assert span > 32 and 4096 // (_waves(bt, d, G, 32) * _cdiv(L, span)) >= 2
    lengths = [L, 211]
    v = _scan_big(bt, L, d, n, G, dt, 204, lengths)
    args, kw = _args(v)
    ch = _picked(d, G, 40 // G, torch.Generator().manual_seed(205))
    at = ch.to(DEV)
    g = torch.Generator(DEV).manual_seed(206)
    d_o, dhT = torch.zeros(bt, L, d, dtype=dt, device=DEV), torch.zeros(bt, d, n, device=DEV)
    d_o[..., at] = torch.randn(bt, L, len(ch), generator=g, device=DEV).to(dt)
    dhT[:, at] = torch.randn(bt, len(ch), n, generator=g, device=DEV)
    got = rn.selective_scan_bwd(*args, d_o, state_in=v["h0"], d_state_out=dhT,
                                lengths=torch.tensor(lengths, dtype=torch.int32, device=DEV), **kw)
    rest = torch.ones(d, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert not any(bool(t.any()) for t in (got.du[..., rest], got.ddelta[..., rest], got.dz[..., rest], got.dA[rest],
                                           got.dD[rest], got.ddelta_bias[rest], got.d_state_in[:, rest]))
    few = got._replace(**{k: getattr(got, k)[..., at] for k in ("du", "ddelta", "dz", "dD", "ddelta_bias")}, dA=got.dA[at],
                       d_state_in=got.d_state_in[:, at])
    _check_bwd(_of(v, ch), d_o[..., at].cpu(), dhT[:, at].cpu(), True, lengths, few, f"{d} {n} {G}")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d,n,G", [(4100, 4, 1), (4104, 8, 2), (4100, 12, 1), (4096, 16, 1), (4100, 24, 1), (4104, 40, 2),
                                   (4096, 64, 1)])
def test_scan_step_of_many_sequences(d, n, G, dt):
    """Four sequences a workgroup, the last one of three."""
    bt = 67
    assert _waves(bt, d, G, 64) >= 4096
    v = _scan_big(bt, 1, d, n, G, dt, 207)
    args, kw = _args({k: t[:, 0] if k in ("u", "z", "delta", "B", "C") else t for k, t in v.items()})
    h = v["h0"].clone()
    out = rn.selective_scan_step(*args, h, **kw)
    ch = _picked(d, G, 24 // G, torch.Generator().manual_seed(208))
    at = ch.to(DEV)
    _check_scan(_of(v, ch), True, None, out[:, None, at], h[:, at], f"{d} {n} {G}")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", [(1, 300, 64, 4, 1), (1, 290, 64, 8, 1), (1, 300, 36, 32, 1), (1, 300, 65, 8, 1),
                                   (1, 290, 65, 16, 1), (1, 290, 33, 64, 1)])
def test_scan_segments_by_width(shape, dt):
    """States by fours and not, in segments of a wave of 16 channels."""
    v = _scan_inputs(*shape, dt, 212, state=True)
    out, state = _scan_gpu(v, state_out=True)
    _check_scan(v, True, None, out, state, f"{shape}")
    g = torch.Generator().manual_seed(213)
    d_o, dhT = torch.randn(*shape[:3], generator=g).to(dt), torch.randn(shape[0], shape[2], shape[3], generator=g)
    _check_bwd(v, d_o, dhT, True, None, _bwd(v, d_o, dhT), f"{shape}")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bt,d,n", [(3, 64, 4), (3, 68, 8), (2, 64, 32), (3, 66, 16), (2, 66, 32)])
def test_scan_step_by_width(bt, d, n, dt):
    v = _scan_inputs(bt, 1, d, n, 1, dt, 214, state=True)
    dev = {k: _dev(t) for k, t in v.items()}
    h = dev["h0"].clone()
    o = rn.selective_scan_step(*(dev[k][:, 0] if k != "A" else dev[k] for k in ("u", "delta", "A", "B", "C")), h,
                               D=dev["D"], z=dev["z"][:, 0], delta_bias=dev["bias"], delta_softplus=True)
    _check_scan(v, True, None, o[:, None], h, "step")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d,wide,L,run", [(16384, 4, 250, 16), (16384, 4, 500, 32), (16384, 4, 1000, 64), (4099, 1, 1000, 64)])
def test_conv_long_runs(d, wide, L, run, dt):
    """A thread's run of 16, 32 and 64 tokens, of four channels and of one; ends inside a run and between two."""
    bt, k = 4, 4
    per = bt * (d // wide)
    assert per * _cdiv(L, run) >= SIMDS * 256 and (run == 64 or per * _cdiv(L, 2 * run) < SIMDS * 256)
    lengths = [L, L - 123, 128, 0]
    g = torch.Generator(DEV).manual_seed(209)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dt)  # noqa: E731
    v = dict(x=r(bt, L, d), w=r(d, k), bias=r(d), s0=r(bt, k - 1, d), d_o=r(bt, L, d), dsT=r(bt, k - 1, d))
    for b, end in enumerate(lengths):
        v["x"][b, end:] = v["d_o"][b, end:] = float("nan")
    ln = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    out, st = rn.causal_conv1d(v["x"], v["w"], v["bias"], lengths=ln, state_in=v["s0"], state_out=True,
                               out=torch.zeros(bt, L, d, dtype=dt, device=DEV))
    got = rn.causal_conv1d_bwd(v["x"], v["w"], v["d_o"], v["bias"], lengths=ln, state_in=v["s0"], d_state_out=v["dsT"])
    ch = _picked(d, 1, 24, torch.Generator().manual_seed(210))
    at = ch.to(DEV)
    few = {n: (t[at] if n in ("w", "bias") else t[..., at]).cpu() for n, t in v.items()}
    for b, end in enumerate(lengths):
        few["x"][b, end:] = few["d_o"][b, end:] = 0
    _check_conv(few, True, lengths, out[..., at], st[..., at], f"{d} {L}")
    sub = got._replace(dx=got.dx[..., at], dw=got.dw[at], dbias=got.dbias[at], d_state_in=got.d_state_in[..., at])
    _check_conv_bwd(few, True, lengths, sub, f"{d} {L}")


W4_CHUNKS = [  # M, N, K, group: several chunks of K, the last one not full
    (3, 70, 4160, 64), (2, 33, 6176, 32), (4, 50, 2304, 128),                          # up to four tokens
    (16, 40, 4224, 128), (16, 33, 2080, 32), (9, 50, 4160, 64), (5, 100, 2304, 384),    # chunks of 2048
    (64, 1100, 1184, 32), (64, 1100, 2112, 64), (48, 1500, 2304, 256),                  # 16 rows of W, chunks of 1024
    (16, 8200, 1152, 64), (16, 8200, 2080, 32), (16, 6200, 2176, 128),                  # 32 rows
    (33, 6200, 2080, 32), (64, 6150, 2304, 128), (64, 6150, 1152, 64),                  # 64 rows by 32 tokens
]


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("shape", W4_CHUNKS)
def test_w4_chunks(shape, pad):
    """pad: rows of x that are not aligned for loads of 16 bytes; zero points go with them."""
    M, N, K, g = shape
    x, q, scale, zero = _w4_inputs(M, N, K, g, pad > 0, 211)
    full = torch.zeros(M, K + pad, dtype=BF, device=DEV)
    full[:, pad:] = x.to(DEV)
    out = rn.linear_w4(full[:, pad:], q.to(DEV), scale.to(DEV), None if zero is None else zero.to(DEV), out_dtype=F32)
    _check_w4(x, q, scale, zero, out, f"{shape} {pad}")
