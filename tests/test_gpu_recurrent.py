"""GPU parity of the recurrent-layer operators (include/recurrent.h) with their plain
64-bit forms, at the sizes, types, strides, lengths and masks where a kernel's edges are.

Roundings counted, per element, relative to the sum of the absolute terms:
  scan: a step rounds A log2 e, its product with dt, the exponential (two half steps) and
  the update: 4 per token of age and 2 |dt A| more for the argument, which the state's own
  decay e^-|dt A| takes back; dt itself comes with some 20 (sum, exp, log) times |dt A|.
  The sum over states N, the skip, the gate (exp, reciprocal, two products) and the final
  rounding add up to less than 2 N + 128.
  gradients: the states above, the same recurrence against time, and one more product and
  sum each: 12 L + 4 N + 512, with a sum over the group's channels for dB and dC, and over
  tokens for dA, dD and the bias: + D / G + L.
"""
import pytest
import torch

import retentive_network_scale_amd as rn
from tests import _recurrent_ref as ref
from tests._recurrent_ref import assert_near

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _scan_inputs(bt, L, d, n, G, dt, seed, z=True, skip=True, bias=True, state=False, wide=0):
    """CPU tensors; wide > 0: u and z, B and C are slices of rows with that many more elements."""
    g = _gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    xz, bc = r(bt, L, 2 * d + wide).to(dt), r(bt, L, 2 * G * n + wide).to(dt)
    v = dict(u=xz[..., wide:wide + d], z=xz[..., wide + d:] if z else None, delta=(0.5 * r(bt, L, d)).to(dt),
             A=-2 * torch.rand(d, n, generator=g), B=bc[..., :G * n].unflatten(-1, (G, n)),
             C=bc[..., G * n:2 * G * n].unflatten(-1, (G, n)), D=r(d) if skip else None,
             bias=0.3 * r(d) if bias else None, h0=r(bt, d, n) if state else None)
    if not wide:
        v = {k: None if t is None else t.contiguous() for k, t in v.items()}
    return v


def _dev(t):
    """On the GPU with the same strides."""
    if t is None:
        return None
    if t.is_contiguous():
        return t.to(DEV)
    base = t._base.to(DEV)
    return base.as_strided(t.shape, t.stride(), t.storage_offset())


def _scan_gpu(v, softplus=True, lengths=None, **kw):
    d = {k: _dev(t) for k, t in v.items()}
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    return rn.selective_scan(d["u"], d["delta"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"], delta_bias=d["bias"],
                             delta_softplus=softplus, lengths=ln, state_in=d["h0"], **kw)


def _check_scan(v, softplus, lengths, out, state, what):
    args = (v["u"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["z"], v["bias"], softplus, lengths, v["h0"])
    o, last, *_ = ref.scan(*args)
    om, lm, *_ = ref.scan(*args, absolute=True)
    L, n = v["u"].shape[1], v["A"].shape[1]
    k = 4 * L + 2 * n + 128
    assert_near(out, o, om, k, f"{what}: out")
    if state is not None:
        assert_near(state, last, lm, k, f"{what}: state")


SCAN_SHAPES = [  # Bt, L, D, N, G
    (1, 1, 1, 1, 1), (2, 1, 64, 16, 1), (1, 15, 67, 3, 1), (3, 16, 64, 4, 2), (1, 17, 130, 5, 2), (2, 33, 96, 8, 3),
    (1, 65, 256, 16, 1), (2, 50, 66, 17, 2), (1, 40, 64, 32, 1), (1, 37, 20, 33, 4), (2, 21, 130, 64, 1),
    (1, 300, 64, 16, 1), (1, 257, 70, 24, 1), (2, 500, 12, 2, 3), (1, 290, 20, 64, 1),
]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", SCAN_SHAPES)
def test_scan_shapes(shape, dt):
    v = _scan_inputs(*shape, dt, 10, state=True)
    out, state = _scan_gpu(v, state_out=True)
    _check_scan(v, True, None, out, state, f"{shape}")


@pytest.mark.parametrize("z,skip,bias,softplus,state", [(False, True, True, True, False), (True, False, False, True, True),
                                                        (False, False, False, False, False), (True, True, True, False, True)])
def test_scan_options(z, skip, bias, softplus, state):
    v = _scan_inputs(2, 45, 72, 16, 1, F32, 11, z, skip, bias, state)
    if not softplus:
        v["delta"] = 0.2 * v["delta"]  # time steps of both signs: states that grow as well
        v["bias"] = None if v["bias"] is None else 0.2 * v["bias"]
    out, st = _scan_gpu(v, softplus, state_out=True)
    _check_scan(v, softplus, None, out, st, "options")


@pytest.mark.parametrize("dt,out_dtype", [(BF, F32), (F32, BF)])
def test_scan_out_dtype(dt, out_dtype):
    v = _scan_inputs(1, 30, 64, 16, 1, dt, 12)
    out, st = _scan_gpu(v, out_dtype=out_dtype)
    assert out.dtype == out_dtype and st is None
    _check_scan(v, True, None, out, None, "out dtype")


@pytest.mark.parametrize("wide", [1, 3, 4, 8])
@pytest.mark.parametrize("dt", [BF, F32])
def test_scan_strided_rows(wide, dt):
    v = _scan_inputs(2, 35, 68, 16, 2, dt, 13, wide=wide)
    v["z"] = v["z"][..., :68]
    out, st = _scan_gpu(v, state_out=True)
    _check_scan(v, True, None, out, st, f"wide {wide}")


@pytest.mark.parametrize("shape,lengths", [((5, 40, 64, 16, 1), [0, 40, 17, 55, -3]), ((2, 400, 64, 16, 1), [130, 64]),
                                           ((3, 1, 33, 5, 1), [1, 0, 1])])
def test_scan_lengths(shape, lengths):
    """Rows behind an end hold NaN in every input; the output there keeps its bits."""
    v = _scan_inputs(*shape, BF, 14, state=True)
    clean = {k: None if t is None else t.clone() for k, t in v.items()}
    for b, n in enumerate(lengths):
        for k in ("u", "z", "delta", "B", "C"):
            v[k][b, max(n, 0):] = float("nan")
            clean[k][b, max(n, 0):] = 0
    mark = torch.full(shape[:3], -7.0, dtype=BF, device=DEV)
    out, st = _scan_gpu(v, True, lengths, state_out=True, out=mark)
    live = torch.arange(shape[1])[None] < torch.tensor(lengths)[:, None]
    assert (out.cpu()[~live] == -7.0).all()
    out = torch.where(live[..., None].to(DEV), out, 0)
    _check_scan(clean, True, lengths, out, st, "lengths")


def test_scan_final_state_may_be_the_initial_one():
    for L in (20, 700):  # one segment, several
        v = _scan_inputs(1, L, 64, 16, 1, F32, 15, state=True)
        want_o, want_s = _scan_gpu(v, state_out=True)
        h = v["h0"].to(DEV)
        d = {k: _dev(t) for k, t in v.items()}
        o, s = rn.selective_scan(d["u"], d["delta"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"], delta_bias=d["bias"],
                                 delta_softplus=True, state_in=h, state_out=h)
        assert s is h and torch.equal(h, want_s) and torch.equal(o, want_o)


def test_scan_in_pieces_is_the_scan():
    """A prompt taken in pieces through the state, then token by token, against the 64-bit form of the whole."""
    bt, L, d, n = 2, 90, 128, 16
    v = _scan_inputs(bt, L, d, n, 1, F32, 16)
    dev = {k: _dev(t) for k, t in v.items()}
    outs, h = [], None
    for lo, hi in ((0, 1), (1, 33), (33, 70)):
        o, h = rn.selective_scan(*(dev[k][:, lo:hi].contiguous() if k != "A" else dev[k] for k in ("u", "delta", "A", "B", "C")),
                                 D=dev["D"], z=dev["z"][:, lo:hi].contiguous(), delta_bias=dev["bias"],
                                 delta_softplus=True, state_in=h, state_out=True)
        outs.append(o)
    for t in range(70, L):
        outs.append(rn.selective_scan_step(dev["u"][:, t].contiguous(), dev["delta"][:, t].contiguous(), dev["A"],
                                           dev["B"][:, t].contiguous(), dev["C"][:, t].contiguous(), h, D=dev["D"],
                                           z=dev["z"][:, t].contiguous(), delta_bias=dev["bias"],
                                           delta_softplus=True)[:, None])
    _check_scan(v, True, None, torch.cat(outs, 1), h, "pieces")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bt,d,n,G", [(1, 1, 1, 1), (3, 67, 5, 1), (2, 96, 16, 3), (1, 256, 64, 1), (5, 64, 33, 2)])
def test_scan_step(bt, d, n, G, dt):
    v = _scan_inputs(bt, 1, d, n, G, dt, 17, state=True, wide=4)
    v["z"] = v["z"][..., :d]
    h = v["h0"].to(DEV)
    dev = {k: _dev(t) for k, t in v.items()}
    o = rn.selective_scan_step(*(dev[k][:, 0] if k != "A" else dev[k] for k in ("u", "delta", "A", "B", "C")), h,
                               D=dev["D"], z=dev["z"][:, 0], delta_bias=dev["bias"], delta_softplus=True)
    _check_scan(v, True, None, o[:, None], h, "step")


def test_scan_large_time_steps_and_rates():
    """softplus far out on both sides, decays that underflow, states that do not decay."""
    v = _scan_inputs(1, 40, 64, 8, 1, F32, 18)
    v["delta"][:, :, :16] -= 30
    v["delta"][:, :, 16:32] += 25
    v["delta"][:, ::3, 32:48] += 60
    v["A"][:, 1] = 0
    v["A"][:, 2] = -40
    out, st = _scan_gpu(v, state_out=True)
    _check_scan(v, True, None, out, st, "large steps")


@pytest.mark.parametrize("L", [40, 300])
def test_scan_rates_of_the_lowest_value(L):
    """Such a state forgets at every token that has a time step, and no other: tokens of no time step leave it."""
    v = _scan_inputs(2, L, 64, 8, 1, F32, 61, bias=False, state=True)
    v["A"][:, 1] = torch.finfo(F32).min
    v["A"][:, 2] = -3e38
    lengths = [L, L - 23]
    d_o = torch.randn(2, L, 64, generator=_gen(62))
    _check_bwd(v, d_o, None, True, lengths, _bwd(v, d_o, None, lengths=lengths), "lowest")
    v["delta"][0, 5:9] = v["delta"][1, 3:40:2] = float("-inf")
    out, st = _scan_gpu(v, lengths=lengths, state_out=True, out=torch.zeros(2, L, 64, device=DEV))
    _check_scan(v, True, lengths, out, st, "lowest, masked")
    state = _dev(v["h0"]).clone()
    rn.selective_scan_step(*(_dev(t[:, 5]) for t in (v["u"], v["delta"])), _dev(v["A"]), *(_dev(v[k][:, 5]) for k in "BC"),
                           state, delta_softplus=True)
    assert torch.equal(state[0], _dev(v["h0"])[0]) and torch.equal(state[1], _dev(v["h0"])[1])
    v = _scan_inputs(2, L, 64, 8, 1, F32, 63, state=True)
    v["A"][:, 1] = float("-inf")
    out, st = _scan_gpu(v, lengths=lengths, state_out=True, out=torch.zeros(2, L, 64, device=DEV))
    _check_scan(v, True, lengths, out, st, "-inf")


@pytest.mark.parametrize("dt", [BF, F32])
def test_scan_tokens_masked_by_their_time_step(dt):
    """delta of -inf or the type's lowest value makes a token do nothing, forward and backward; +inf
    and NaN reach only their own channel from their token on."""
    v = _scan_inputs(2, 40, 68, 16, 1, dt, 19, bias=False, state=True)
    v["delta"][0, 3:20] = float("-inf")
    v["delta"][1, 5:9, ::2] = torch.finfo(dt).min
    out, st = _scan_gpu(v, state_out=True)
    _check_scan(v, True, None, out, st, "masked")
    d_o = torch.randn(2, 40, 68, generator=_gen(190)).to(dt)
    _check_bwd(v, d_o, None, True, None, _bwd(v, d_o, None), "masked")
    bad = {k: None if t is None else t.clone() for k, t in v.items()}
    bad["delta"][0, 25, 7] = float("nan")
    bad["u"][1, 30, 66] = float("inf")
    o2, s2 = _scan_gpu(bad, state_out=True)
    clean = torch.ones(2, 40, 68, dtype=torch.bool)
    clean[0, 25:, 7] = clean[1, 30:, 66] = False
    assert torch.equal(o2.cpu()[clean], out.cpu()[clean])
    assert not torch.isfinite(o2.cpu()[~clean]).any() and torch.isnan(s2[0, 7]).all()


def _bwd(v, d_o, dhT, softplus=True, lengths=None, **kw):
    d = {k: _dev(t) for k, t in v.items()}
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    return rn.selective_scan_bwd(d["u"], d["delta"], d["A"], d["B"], d["C"], d_o.to(DEV), D=d["D"], z=d["z"],
                                 delta_bias=d["bias"], delta_softplus=softplus, lengths=ln, state_in=d["h0"],
                                 d_state_out=None if dhT is None else dhT.to(DEV), **kw)


def _check_bwd(v, d_o, dhT, softplus, lengths, got, what):
    args = (v["u"], v["delta"], v["A"], v["B"], v["C"], d_o, v["D"], v["z"], v["bias"], softplus, lengths, v["h0"], dhT)
    want, mag = ref.scan_bwd(*args), ref.scan_bwd(*args, absolute=True)
    bt, L, d = v["u"].shape
    n, G = v["A"].shape[1], v["B"].shape[2]
    k = 12 * L + 4 * n + 512
    for name, r, roundings in (("du", "du", k), ("ddelta", "ddelta", k), ("dA", "dA", k + L), ("dB", "dB", k + d // G),
                               ("dC", "dC", k + d // G), ("dD", "dD", k + L), ("dz", "dz", k),
                               ("ddelta_bias", "dbias", k + L), ("d_state_in", "dh0", k)):
        t = getattr(got, name)
        if t is not None:
            assert_near(t, want[r], mag[r], roundings, f"{what}: {name}")
    absent = dict(dD="D", dz="z", ddelta_bias="bias", d_state_in="h0")
    for name, given in absent.items():
        assert (getattr(got, name) is None) == (v[given] is None), name


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", SCAN_SHAPES)
def test_scan_bwd_shapes(shape, dt):
    v = _scan_inputs(*shape, dt, 20, state=True)
    g = _gen(21)
    d_o, dhT = torch.randn(*shape[:3], generator=g).to(dt), torch.randn(shape[0], shape[2], shape[3], generator=g)
    _check_bwd(v, d_o, dhT, True, None, _bwd(v, d_o, dhT), f"{shape}")


@pytest.mark.parametrize("z,skip,bias,softplus,state", [(False, True, True, True, False), (True, False, False, True, True),
                                                        (False, False, False, False, False), (True, True, True, False, True)])
def test_scan_bwd_options(z, skip, bias, softplus, state):
    v = _scan_inputs(2, 45, 72, 16, 1, F32, 22, z, skip, bias, state)
    if not softplus:
        v["delta"] = 0.2 * v["delta"]
        v["bias"] = None if v["bias"] is None else 0.2 * v["bias"]
    d_o = torch.randn(2, 45, 72, generator=_gen(23))
    got = _bwd(v, d_o, None, softplus, out_dtype=BF)
    assert got.du.dtype == got.dB.dtype == BF and got.dA.dtype == F32
    _check_bwd(v, d_o, None, softplus, None, got, "options")


def test_scan_bwd_strided_rows():
    for wide in (3, 4):
        v = _scan_inputs(2, 35, 68, 16, 2, BF, 24, wide=wide)
        v["z"] = v["z"][..., :68]
        d_o = torch.randn(2, 35, 68, generator=_gen(25)).to(BF)
        _check_bwd(v, d_o, None, True, None, _bwd(v, d_o, None), f"wide {wide}")


@pytest.mark.parametrize("shape,lengths", [((5, 40, 64, 16, 1), [0, 40, 17, 55, -3]), ((2, 400, 64, 16, 1), [130, 64])])
def test_scan_bwd_lengths(shape, lengths):
    v = _scan_inputs(*shape, F32, 26, state=True)
    g = _gen(27)
    d_o, dhT = torch.randn(*shape[:3], generator=g), torch.randn(shape[0], shape[2], shape[3], generator=g)
    clean = {k: None if t is None else t.clone() for k, t in v.items()}
    dirty = d_o.clone()
    for b, n in enumerate(lengths):
        for k in ("u", "z", "delta", "B", "C"):
            v[k][b, max(n, 0):] = float("nan")
            clean[k][b, max(n, 0):] = 0
        dirty[b, max(n, 0):] = float("inf")
    got = _bwd(v, dirty, dhT, True, lengths)
    _check_bwd(clean, d_o, dhT, True, lengths, got, "lengths")


def test_scan_bwd_more_tokens_than_workgroups():
    # 2^22 tokens and some, N 64: the last sums walk more values than their grid has threads, as do the rows behind
    # the end.  The last tokens' du, dz and dB follow from the tokens behind them alone, so a short piece has them too.
    L, n, d, piece = (1 << 22) + 999, 64, 4, 200
    end = L - 400
    g = torch.Generator(DEV).manual_seed(60)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    u, delta, d_o, B, C = r(1, L, d), 0.5 * r(1, L, d), r(1, L, d), r(1, L, 1, n), r(1, L, 1, n)
    A = -1 - torch.rand(d, n, generator=g, device=DEV)
    for shape in ((1, L, d), (1, L, d), (1, L, 1, n), (1, L, 1, n)):
        torch.full(shape, float("nan"), device=DEV)  # what the outputs' memory may hold
    got = rn.selective_scan_bwd(u, delta, A, B, C, d_o, delta_softplus=True,
                                lengths=torch.tensor([end], dtype=torch.int32, device=DEV))
    for t in (got.du, got.ddelta, got.dB, got.dC):
        assert bool((t[:, end:] == 0).all()) and bool(torch.isfinite(t).all())
    v = {k: t[:, end - piece:end].cpu() for k, t in dict(u=u, delta=delta, B=B, C=C, d_o=d_o).items()}
    args = (v["u"], v["delta"], A.cpu(), v["B"], v["C"], v["d_o"])
    want, mags = ref.scan_bwd(*args, softplus_on=True), ref.scan_bwd(*args, softplus_on=True, absolute=True)
    for name in ("du", "dB"):
        assert_near(getattr(got, name)[:, end - piece:end], want[name], mags[name], 12 * piece + 4 * n + 512 + d, name)


def test_scan_repeats_to_the_bit():
    v = _scan_inputs(2, 300, 192, 16, 1, BF, 28, state=True)
    d_o = torch.randn(2, 300, 192, generator=_gen(29)).to(BF)
    a, b = _bwd(v, d_o, None), _bwd(v, d_o, None)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------------------ convolution
# Roundings: a product and a sum per tap, silu and its slope (exp, reciprocal, products): 2 K + 40;
# a slope's error enters g, and sums over tokens add one per token.
CONV_SHAPES = [  # Bt, L, D, K
    (1, 1, 1, 2), (2, 1, 64, 4), (1, 2, 8, 4), (3, 7, 24, 3), (1, 9, 40, 8), (2, 64, 136, 4), (1, 65, 33, 5),
    (2, 130, 16, 2), (1, 300, 72, 6), (2, 17, 12, 7),
]


def _conv_inputs(bt, L, d, k, dt, seed, bias=True, state=True):
    g = _gen(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    return dict(x=r(bt, L, d), w=r(d, k), bias=r(d) if bias else None, s0=r(bt, k - 1, d) if state else None,
                d_o=r(bt, L, d), dsT=r(bt, k - 1, d))


def _check_conv(v, silu, lengths, out, state, what):
    args = (v["x"], v["w"], v["bias"], silu, lengths, v["s0"])
    o, s, *_ = ref.conv(*args)
    mag = ref.conv(*args[:3], False, lengths, v["s0"], absolute=True)[0]
    # silu's slope is at most 1.1, so an error of the sum reaches the output as at most 1.1 of it
    assert_near(out, o, 1.1 * mag, 2 * v["w"].shape[1] + 40, f"{what}: out")
    if state is not None:
        assert torch.equal(state.cpu().double(), s), f"{what}: state"


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", CONV_SHAPES)
def test_conv_shapes(shape, dt):
    v = _conv_inputs(*shape, dt, 30)
    d = {k: t.to(DEV) for k, t in v.items()}
    out, st = rn.causal_conv1d(d["x"], d["w"], d["bias"], state_in=d["s0"], state_out=True)
    _check_conv(v, True, None, out, st, f"{shape}")


@pytest.mark.parametrize("silu,bias,state", [(False, True, False), (True, False, False), (False, False, True)])
def test_conv_options(silu, bias, state):
    v = _conv_inputs(2, 20, 24, 4, F32, 31, bias, state)
    d = {k: None if t is None else t.to(DEV) for k, t in v.items()}
    out, st = rn.causal_conv1d(d["x"], d["w"], d["bias"], silu=silu, state_in=d["s0"], state_out=True)
    _check_conv(v, silu, None, out, st, "options")
    g = rn.causal_conv1d_bwd(d["x"], d["w"], d["d_o"], d["bias"], silu=silu, state_in=d["s0"])
    _check_conv_bwd({**v, "dsT": None}, silu, None, g, "options")


def _check_conv_bwd(v, silu, lengths, got, what):
    args = (v["x"], v["w"], v["d_o"], v["bias"], silu, lengths, v["s0"], v["dsT"])
    want, mag = ref.conv_bwd(*args), ref.conv_bwd(*args, absolute=True)
    # the slope of silu depends on the sum in front of it: |silu''| <= 1/2 times that sum's own error,
    # relative to the slope's terms at most the sum of the absolute products
    L, k = v["x"].shape[1], v["w"].shape[1]
    pre = ref.conv(*args[:2], v["bias"], False, lengths, v["s0"], absolute=True)[0].max().item() if L else 0
    rounds = 2 * k + 60 + (2 * k + 40) * pre * 4
    assert_near(got.dx, want["dx"], mag["dx"], rounds, f"{what}: dx")
    n = v["x"].shape[0] * L
    assert_near(got.dw, want["dw"], mag["dw"], rounds + n, f"{what}: dw")
    if v["bias"] is not None:
        assert_near(got.dbias, want["dbias"], mag["dbias"], rounds + n, f"{what}: dbias")
    assert (got.dbias is None) == (v["bias"] is None) and (got.d_state_in is None) == (v["s0"] is None)
    if v["s0"] is not None:
        assert_near(got.d_state_in, want["ds0"], mag["ds0"], rounds, f"{what}: d_state_in")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", CONV_SHAPES)
def test_conv_bwd_shapes(shape, dt):
    v = _conv_inputs(*shape, dt, 32)
    d = {k: t.to(DEV) for k, t in v.items()}
    g = rn.causal_conv1d_bwd(d["x"], d["w"], d["d_o"], d["bias"], state_in=d["s0"], d_state_out=d["dsT"])
    _check_conv_bwd(v, True, None, g, f"{shape}")


@pytest.mark.parametrize("shape,lengths", [((5, 30, 24, 4), [0, 30, 2, 41, -1]), ((2, 200, 16, 3), [129, 64])])
def test_conv_lengths(shape, lengths):
    v = _conv_inputs(*shape, BF, 33)
    clean = {k: t.clone() for k, t in v.items()}
    for b, n in enumerate(lengths):
        for k in ("x", "d_o"):
            v[k][b, max(n, 0):] = float("nan")
            clean[k][b, max(n, 0):] = 0
    d = {k: t.to(DEV) for k, t in v.items()}
    ln = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    mark = torch.full(shape[:3], -7.0, dtype=BF, device=DEV)
    out, st = rn.causal_conv1d(d["x"], d["w"], d["bias"], lengths=ln, state_in=d["s0"], state_out=True, out=mark)
    live = (torch.arange(shape[1])[None] < torch.tensor(lengths)[:, None])[..., None]
    assert (out.cpu()[~live.expand(shape[:3])] == -7.0).all()
    _check_conv(clean, True, lengths, torch.where(live.to(DEV), out, 0), st, "lengths")
    g = rn.causal_conv1d_bwd(d["x"], d["w"], d["d_o"], d["bias"], lengths=ln, state_in=d["s0"], d_state_out=d["dsT"])
    _check_conv_bwd(clean, True, lengths, g, "lengths")


def test_conv_strided_rows_and_steps():
    """A slice of wider rows, in pieces through the state, then token by token, equals the whole to the bit."""
    for dt, pad in ((BF, 8), (BF, 3), (F32, 4), (F32, 1)):
        g = _gen(34)
        bt, L, d, k = 2, 40, 48, 4
        full = torch.randn(bt, L, d + pad, generator=g).to(dt).to(DEV)
        w, bias = torch.randn(d, k, generator=g).to(dt).to(DEV), torch.randn(d, generator=g).to(dt).to(DEV)
        x = full[..., pad:]
        whole, end = rn.causal_conv1d(x, w, bias, state_out=True)
        dense, _ = rn.causal_conv1d(x.contiguous(), w, bias)
        assert torch.equal(whole, dense)
        a, s = rn.causal_conv1d(x[:, :2].contiguous(), w, bias, state_out=True)
        b, s = rn.causal_conv1d(x[:, 2:25].contiguous(), w, bias, state_in=s, state_out=True)
        steps = [rn.causal_conv1d_step(x[:, t], s, w, bias)[:, None] for t in range(25, L)]
        assert torch.equal(torch.cat([a, b, *steps], 1), whole) and torch.equal(s, end)


# ------------------------------------------------------------------------------ 4-bit weights
# Products are exact; a matrix step adds 33 of them to the accumulator, the offset's step takes at
# most (31 + 31) / 1 of the largest |q - zero| = 1 back: magnitudes of sum |x| (|16 + q| + |16 + zero|)
# <= 62 sum |x| in K / 4 + 64 roundings, then a scale per group and the sum over groups and waves.
W4_SHAPES = [  # M, N, K, group
    (1, 1, 32, 32), (1, 16, 64, 64), (2, 17, 128, 128), (16, 40, 256, 128), (17, 16, 96, 32), (33, 100, 192, 64),
    (64, 64, 384, 128), (65, 33, 512, 256), (5, 24, 1024, 512), (130, 8, 160, 32), (3, 500, 2048, 128), (1, 7, 384, 384),
    (9, 8200, 96, 32), (16, 8200, 192, 64), (20, 4100, 256, 128), (33, 6150, 160, 32), (40, 6100, 384, 384), (64, 6150, 1152, 64),
    (4, 40, 4224, 128),
]


def _w4_inputs(M, N, K, g, zeros, seed):
    gen = _gen(seed)
    q = torch.randint(0, 16, (N, K), generator=gen, dtype=torch.uint8)
    scale = (0.02 * torch.randn(N, K // g, generator=gen)).to(BF)
    zero = torch.randint(0, 16, (N, K // g), generator=gen, dtype=torch.uint8) if zeros else None
    return torch.randn(M, K, generator=gen).to(BF), rn.pack_w4(q), scale, zero


def _check_w4(x, q, scale, zero, out, what):
    w = ref.w4_dense(q, scale, zero)
    xd, K = x.double(), x.shape[1]
    mag = xd.abs() @ (62 * scale.double().abs().repeat_interleave(K // scale.shape[1], 1)).T
    assert_near(out, xd @ w.T, mag, 8 + K // 32 * 2, what)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("shape", W4_SHAPES)
def test_w4_shapes(shape, zeros):
    x, q, scale, zero = _w4_inputs(*shape, zeros, 40)
    for od in (F32, BF):
        out = rn.linear_w4(x.to(DEV), q.to(DEV), scale.to(DEV), None if zero is None else zero.to(DEV), out_dtype=od)
        assert out.dtype == od
        _check_w4(x, q, scale, zero, out, f"{shape} {od}")


@pytest.mark.parametrize("pad", [1, 8])
def test_w4_strided_rows(pad):
    x, q, scale, zero = _w4_inputs(19, 48, 256, 64, True, 41)
    full = torch.zeros(19, 256 + pad, dtype=BF, device=DEV)
    full[:, pad:] = x.to(DEV)
    out = rn.linear_w4(full[:, pad:], q.to(DEV), scale.to(DEV), zero.to(DEV), out_dtype=F32)
    _check_w4(x, q, scale, zero, out, f"pad {pad}")


def test_w4_is_exact_where_it_can_be():
    """Whole numbers below 2^24: no rounding anywhere, so every weight, zero point and place shows."""
    M, N, K, g = 16, 48, 256, 64
    gen = _gen(42)
    q = torch.randint(0, 16, (N, K), generator=gen, dtype=torch.uint8)
    zero = torch.randint(0, 16, (N, K // g), generator=gen, dtype=torch.uint8)
    scale = torch.randint(1, 5, (N, K // g), generator=gen).to(BF)
    x = torch.randint(-8, 9, (M, K), generator=gen).to(BF)
    out = rn.linear_w4(x.to(DEV), rn.pack_w4(q).to(DEV), scale.to(DEV), zero.to(DEV), out_dtype=F32)
    w = (q.double() - zero.double().repeat_interleave(g, 1)) * scale.double().repeat_interleave(g, 1)
    assert torch.equal(out.cpu().double(), x.double() @ w.T)


def test_w4_rows_do_not_depend_on_their_number():
    """A token's output has the same bits alone and in a batch of the same kernel's tiles."""
    x, q, scale, zero = (None if t is None else t.to(DEV) for t in _w4_inputs(64, 80, 512, 128, True, 43))
    whole = rn.linear_w4(x, q, scale, zero, out_dtype=F32)
    for lo, hi in ((0, 33), (10, 60)):
        assert torch.equal(rn.linear_w4(x[lo:hi], q, scale, zero, out_dtype=F32), whole[lo:hi])


@pytest.mark.parametrize("B,dm,H,dk,dv,g,zeros,rot", [(1, 256, 2, 64, 128, 128, False, True), (3, 128, 4, 32, 64, 32, True, True),
                                                      (20, 384, 2, 128, 256, 64, True, False)])
def test_msr_step_w4(B, dm, H, dk, dv, g, zeros, rot):
    """Steps against the bf16 step on the weights' own values where those are exact in bf16
    (scales of powers of two), so the two differ by the order of fp32 sums and the roundings
    of the gated heads and of y alone: two bf16 half steps through W_O and one of y."""
    gen = _gen(44)
    NP = 2 * H * dk + 2 * H * dv

    def mat(n, k):
        q = torch.randint(0, 16, (n, k), generator=gen, dtype=torch.uint8)
        s = torch.exp2(-torch.randint(7, 10, (n, k // g), generator=gen).float()).to(BF)
        z = torch.randint(5, 12, (n, k // g), generator=gen, dtype=torch.uint8) if zeros else None
        p = rn.pack_w4(q)
        return tuple(None if t is None else t.to(DEV) for t in (p, s, z)), ref.w4_dense(p, s, z).to(BF).to(DEV)

    w_in, dense_in = mat(NP, dm)
    w_o, dense_o = mat(dm, H * dv)
    gamma = torch.tensor([1 - 2.0 ** (-5 - h) for h in range(H)])
    theta = torch.tensor([10000.0 ** (-2 * i / dk) for i in range(dk // 2)]) if rot else None
    s1 = torch.randn(B, H, dk, dv, generator=gen).to(DEV)
    s2 = s1.clone()
    p1 = torch.randint(0, 5000, (B,), generator=gen, dtype=torch.int32).to(DEV)
    p2 = p1.clone()
    split = [t.contiguous() for t in dense_in.split([H * dk, H * dk, H * dv, H * dv])]
    for _ in range(3):
        x = torch.randn(B, dm, generator=gen).to(BF).to(DEV)
        y1 = rn.msr_layer_step_w4(x, w_in, w_o, s1, p1, H, dk, dv, gamma, theta)
        y2 = rn.msr_layer_step(x, *split, dense_o, s2, p2, H, dk, dv, gamma, theta)
        assert torch.equal(p1, p2)
        torch.testing.assert_close(s1, s2, rtol=1e-4, atol=1e-4)
        off = (y1.double() - y2.double()).norm() / y2.double().norm()
        assert off <= 3 * 2.0 ** -8, off


def test_msr_step_w4_positions_in_a_graph():
    """The positions advance within the step (40 sequences: several tiles of tokens), or stay; a captured
    step replays as the eager steps, bit for bit."""
    B, dm, H, dk, dv = 40, 256, 2, 64, 128
    gen = _gen(47)

    def mat(n, k):
        return (rn.pack_w4(torch.randint(0, 16, (n, k), generator=gen)).to(DEV),
                (0.01 * torch.rand(n, k // 64, generator=gen)).to(BF).to(DEV), None)

    w_in, w_o = mat(2 * H * dk + 2 * H * dv, dm), mat(dm, H * dv)
    gamma, theta = torch.tensor([0.97, 0.99]), torch.rand(dk // 2, generator=gen)
    start = torch.randint(0, 5000, (B,), generator=gen, dtype=torch.int32).to(DEV)
    s1 = torch.zeros(B, H, dk, dv, device=DEV)
    s2, p1, p2 = s1.clone(), start.clone(), start.clone()
    x = torch.randn(B, dm, generator=gen).to(BF).to(DEV)
    step = lambda s, p, **kw: rn.msr_layer_step_w4(x, w_in, w_o, s, p, H, dk, dv, gamma, theta, **kw)  # noqa: E731
    step(s1.clone(), p1, advance_pos=False)
    assert torch.equal(p1, start)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s1.clone(), p1.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1 = step(s1, p1)
    for i in range(4):
        x.copy_(torch.randn(B, dm, generator=_gen(48 + i)).to(BF))
        graph.replay()
        y2 = step(s2, p2)
        torch.cuda.synchronize()
        assert torch.equal(y1, y2) and torch.equal(s1, s2) and torch.equal(p1, p2)
        assert torch.equal(p1, start + i + 1)


# ------------------------------------------------------------------------------ long sequences
def test_offsets_beyond_32_bits():
    """2^31 elements and more in one tensor: the last tokens, and their gradients, equal those of a call
    on these tokens alone that starts from the state in front of them (computed by a call on the rest)."""
    L, cut, d, n = (1 << 19) + 40, 1 << 19, 4096, 4
    gen = torch.Generator(device=DEV).manual_seed(90)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=BF)  # noqa: E731
    u, delta, bc = r(1, L, d), r(1, L, d), r(1, L, 2, 1, n)
    A = -2 * torch.rand(d, n, generator=gen, device=DEV)
    w, bias = r(d, 4), r(d)
    c, cs = rn.causal_conv1d(u, w, bias, state_out=True)
    tail, ts = rn.causal_conv1d(u[:, cut:].contiguous(), w, bias, state_in=u[:, cut - 3:cut].contiguous(), state_out=True)
    assert torch.equal(c[:, cut:], tail) and torch.equal(cs, ts)
    del c
    Bm, Cm = bc[:, :, 0], bc[:, :, 1]
    whole, end = rn.selective_scan(u, delta, A, Bm, Cm, delta_softplus=True, state_out=True)
    _, h = rn.selective_scan(u[:, :cut], delta[:, :cut], A, Bm[:, :cut], Cm[:, :cut], delta_softplus=True, state_out=True)
    part, e2 = rn.selective_scan(u[:, cut:], delta[:, cut:], A, Bm[:, cut:], Cm[:, cut:], delta_softplus=True,
                                 state_in=h, state_out=True)
    # other segments, other orders: fp32 roundings of some 40 tokens, then bf16's
    torch.testing.assert_close(end, e2, rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(whole[:, cut:].float(), part.float(), rtol=2 ** -7, atol=1e-3)
    del whole
    d_o = r(1, L, d)
    g = rn.selective_scan_bwd(u, delta, A, Bm, Cm, d_o, delta_softplus=True)
    t = rn.selective_scan_bwd(u[:, cut:], delta[:, cut:], A, Bm[:, cut:], Cm[:, cut:], d_o[:, cut:].contiguous(),
                              delta_softplus=True, state_in=h)
    for a, b in ((g.du, t.du), (g.ddelta, t.ddelta), (g.dB, t.dB), (g.dC, t.dC)):
        off = (a[:, cut:].float() - b.float()).norm() / b.float().norm()
        assert off <= 2 ** -8, off


# ------------------------------------------------------------------------------ graphs, streams
def _layer(dev, w_in, w_o, st, x):
    """One token of a recurrent layer: projection, convolution, scan, projection."""
    p = rn.linear_w4(x, *w_in)
    d = st["h"].shape[1]
    u = rn.causal_conv1d_step(p[:, :d], st["c"], dev["cw"], dev["cb"])
    bc = p[:, 3 * d:].unflatten(-1, (2, 1, 16))
    y = rn.selective_scan_step(u, p[:, 2 * d:3 * d], dev["A"], bc[:, 0], bc[:, 1], st["h"], D=dev["D"], z=p[:, d:2 * d],
                               delta_bias=dev["bias"], delta_softplus=True)
    return rn.linear_w4(y, *w_o)


def _layer_weights(d, dm, seed):
    gen = _gen(seed)
    dev = dict(cw=torch.randn(d, 4, generator=gen).to(BF), cb=torch.randn(d, generator=gen).to(BF),
               A=-2 * torch.rand(d, 16, generator=gen), D=torch.randn(d, generator=gen), bias=0.3 * torch.randn(d, generator=gen))
    dev = {k: t.to(DEV) for k, t in dev.items()}

    def mat(n, k):
        q = torch.randint(0, 16, (n, k), generator=gen, dtype=torch.uint8)
        return rn.pack_w4(q).to(DEV), (0.01 * torch.rand(n, k // 64, generator=gen)).to(BF).to(DEV), None
    return dev, mat(3 * d + 32, dm), mat(dm, d)


def test_layer_step_in_two_captured_graphs():
    """Two layers' decode steps captured into two graphs, replayed in turn with eager work between
    the replays: every replay's output and states equal the eager calls', bit for bit."""
    B, d, dm = 3, 192, 128
    gen = _gen(50)
    layers = []
    for i in range(2):
        dev, w_in, w_o = _layer_weights(d, dm, 51 + i)
        mk = lambda: {"h": torch.zeros(B, d, 16, device=DEV), "c": torch.zeros(B, 3, d, dtype=BF, device=DEV)}  # noqa: E731
        layers.append([dev, w_in, w_o, mk(), mk()])
    xs = torch.randn(5, B, dm, generator=gen).to(BF).to(DEV)
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for dev, w_in, w_o, st, _ in layers:
            _layer(dev, w_in, w_o, {k: t.clone() for k, t in st.items()}, x)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for dev, w_in, w_o, st, _ in layers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_layer(dev, w_in, w_o, st, x))
        graphs.append(g)
    for i in range(5):
        x.copy_(xs[i])
        for g, out, (dev, w_in, w_o, st, st2) in zip(graphs, outs, layers):
            g.replay()
            want = _layer(dev, w_in, w_o, st2, xs[i])
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            assert all(torch.equal(st[k], st2[k]) for k in st)


def test_scan_training_step_in_a_graph():
    """Convolution, scan and both gradients captured, replayed on new inputs, equal to the eager calls."""
    bt, L, d, n = 2, 200, 128, 16
    v = {k: _dev(t) for k, t in _scan_inputs(bt, L, d, n, 1, BF, 60).items()}
    c = {k: t.to(DEV) for k, t in _conv_inputs(bt, L, d, 4, BF, 61, state=False).items() if t is not None}

    def step():
        u, _ = rn.causal_conv1d(c["x"], c["w"], c["bias"])
        o, _ = rn.selective_scan(u, v["delta"], v["A"], v["B"], v["C"], D=v["D"], z=v["z"], delta_bias=v["bias"],
                                 delta_softplus=True)
        g = rn.selective_scan_bwd(u, v["delta"], v["A"], v["B"], v["C"], c["d_o"], D=v["D"], z=v["z"],
                                  delta_bias=v["bias"], delta_softplus=True)
        h = rn.causal_conv1d_bwd(c["x"], c["w"], g.du, c["bias"])
        return [o, *(t for t in g if t is not None), *(t for t in h if t is not None)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        c["x"].copy_(torch.randn(bt, L, d, generator=_gen(62 + i)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        _ = (c["x"].float() * 2).sum()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)


def test_calls_on_another_stream():
    """A call on a stream that is not the current one: workspace and outputs belong to it."""
    v = {k: _dev(t) for k, t in _scan_inputs(1, 800, 64, 16, 1, BF, 70).items()}
    args = (v["u"], v["delta"], v["A"], v["B"], v["C"])
    kw = dict(D=v["D"], z=v["z"], delta_bias=v["bias"], delta_softplus=True)
    want, _ = rn.selective_scan(*args, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [rn.selective_scan(*args, **kw, stream=side)[0] for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_two_calls_at_once():
    """Calls of one kind on two streams, each with its own workspace, while both run."""
    v = {k: _dev(t) for k, t in _scan_inputs(1, 3000, 192, 16, 1, BF, 71).items()}
    d_o = torch.randn(1, 3000, 192, generator=_gen(72)).to(BF).to(DEV)
    q, s = rn.pack_w4(torch.randint(0, 16, (256, 192), generator=_gen(73))).to(DEV), torch.ones(256, 3, dtype=BF, device=DEV)

    def both(u, stream):
        kw = dict(D=v["D"], z=v["z"], delta_bias=v["bias"], delta_softplus=True, stream=stream)
        o, st = rn.selective_scan(u, v["delta"], v["A"], v["B"], v["C"], state_out=True, **kw)
        g = rn.selective_scan_bwd(u, v["delta"], v["A"], v["B"], v["C"], d_o, **kw)
        h = rn.causal_conv1d_bwd(v["u"], v["w"], d_o, stream=stream)
        return [o, st, rn.linear_w4(u[0], q, s, stream=stream), *(t for t in (*g, *h) if t is not None)]

    v["w"] = torch.randn(192, 4, generator=_gen(74)).to(BF).to(DEV)
    us = [v["u"], (2 * v["u"]).contiguous()]
    want = [both(u, None) for u in us]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[both(u, stream) for u, stream in zip(us, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


@pytest.mark.parametrize("dt", [BF, F32])
def test_calls_without_tokens(dt):
    """L = 0: the state passes through, sums over no tokens are zero."""
    v = {k: _dev(t) for k, t in _scan_inputs(2, 1, 68, 5, 2, dt, 75, state=True).items()}
    none = lambda t: t[:, :0]  # noqa: E731
    args = [none(v["u"]), none(v["delta"]), v["A"], none(v["B"]), none(v["C"])]
    out, st = rn.selective_scan(*args, z=none(v["z"]), state_in=v["h0"], state_out=True)
    assert out.shape == (2, 0, 68) and torch.equal(st, v["h0"])
    assert (rn.selective_scan(*args, state_out=True)[1] == 0).all()
    dh = torch.randn(2, 68, 5, device=DEV)
    g = rn.selective_scan_bwd(*args, none(v["u"]), D=v["D"], delta_bias=v["bias"], state_in=v["h0"], d_state_out=dh)
    assert torch.equal(g.d_state_in, dh) and not any(bool(t.any()) for t in (g.dA, g.dD, g.ddelta_bias))
    g = rn.selective_scan_bwd(*args, none(v["u"]), state_in=v["h0"])
    assert not g.d_state_in.any()
    w, s0 = torch.randn(68, 4, device=DEV).to(dt), torch.randn(2, 3, 68, device=DEV).to(dt)
    out, st = rn.causal_conv1d(none(v["u"]), w, state_in=s0, state_out=True)
    assert out.shape == (2, 0, 68) and torch.equal(st, s0)
    assert not rn.causal_conv1d(none(v["u"]), w, state_out=True)[1].any()
    g = rn.causal_conv1d_bwd(none(v["u"]), w, none(v["u"]), bias=w[:, 0].contiguous(), state_in=s0, d_state_out=s0)
    assert torch.equal(g.d_state_in, s0) and not g.dw.any() and not g.dbias.any()


def test_layer_prompt_then_tokens():
    """A recurrent layer's prompt in one call each and then its tokens, against the whole sequence in
    64 bits: the same states carry both, at bf16 hand-offs between the operators."""
    bt, L, d, n, cut = 2, 70, 128, 16, 61
    v = _scan_inputs(bt, L, d, n, 1, BF, 80)
    c = _conv_inputs(bt, L, d, 4, BF, 81, state=False)
    dev = {k: _dev(t) for k, t in v.items()}
    cd = {k: None if t is None else t.to(DEV) for k, t in c.items()}
    kw = dict(D=dev["D"], delta_bias=dev["bias"], delta_softplus=True)
    cut_ = lambda t: t[:, :cut].contiguous()  # noqa: E731
    u, cs = rn.causal_conv1d(cut_(cd["x"]), cd["w"], cd["bias"], state_out=True)
    o, h = rn.selective_scan(u, *(cut_(dev[k]) if k != "A" else dev[k] for k in ("delta", "A", "B", "C")),
                             z=cut_(dev["z"]), state_out=True, **kw)
    us, os_ = [u], [o]
    for t in range(cut, L):
        u = rn.causal_conv1d_step(cd["x"][:, t], cs, cd["w"], cd["bias"])
        os_.append(rn.selective_scan_step(u, dev["delta"][:, t], dev["A"], dev["B"][:, t], dev["C"][:, t], h,
                                          z=dev["z"][:, t], **kw)[:, None])
        us.append(u[:, None])
    us, os_ = torch.cat(us, 1), torch.cat(os_, 1)
    _check_conv(c, True, None, us, None, "layer")
    _check_scan({**v, "u": us.cpu()}, True, None, os_, h, "layer")
