"""GPU parity of the operators around the layers (include/language.h) with their plain 64-bit forms
(tests/_language_ref.py), at the sizes, types, strides, lengths and masks where a kernel's edges are.

Roundings counted, in units of half a step of fp32 of the sum of the absolute terms:
  embedding: one product.  Its gradient: a sum of c tokens, at most c, in pieces, and a product: c + 4.
  norm: the mean of W values, the variance, its root, a division and three products: W + 32, with
  some 16 more for the gate's exponential and reciprocal; gradients W + 96; sums over T tokens T more.
  linear: K products, exact in fp32, and K sums, which the matrix cores may cut off rather than
  round: 2 K; bias, activation (gelu's tail is good to 5.7e-6 = 96 U), residual: 160 more.
  gradients of linear: 2 N or 2 M; the slope of an activation some 16 for its terms (gelu's tail
  3.2e-8, its density an exponential and two products); dbias: M + 64.
  scores: a sum of exponentials of three roundings each, in partial sums of at most 32 and their
  tree of 8, and the logarithm's share: 64 at most, absolute, beside the result's own rounding.
"""
import math

import pytest
import torch

import retentive_network_scale_amd as rn
from tests import _language_ref as ref
from tests._recurrent_ref import assert_near

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _r(seed, *shape, dt=F32):
    return torch.randn(*shape, generator=_gen(seed)).to(dt)


def _wide(seed, rows, width, extra, dt):
    """CPU rows that are slices of rows `extra` elements wider, starting `extra` in."""
    return _r(seed, *rows, width + extra, dt=dt)[..., extra:]


def _dev(t):
    """On the GPU with the same strides and offset."""
    if t is None:
        return None
    if t.is_contiguous():
        return t.to(DEV)
    return t._base.to(DEV).as_strided(t.shape, t.stride(), t.storage_offset())


# --------------------------------------------------------------------------------- embedding
@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (3, 10, 7), (64, 50, 64), (5, 1000, 8), (130, 33, 100), (2, 7, 2050), (1, 3, 5000)])
@pytest.mark.parametrize("dt,od", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_embedding(n, V, D, dt, od):
    ids = torch.randint(-1, V + 1, (n,), generator=_gen(1), dtype=I32)  # both kinds outside among them
    table = _r(2, V, D, dt=dt)
    out = rn.embedding(ids.to(DEV), table.to(DEV), scale=3.0, out_dtype=od)
    want = ref.embedding(ids, table, 3.0)
    assert out.dtype == od
    assert_near(out, want, want.abs(), 1, "out")
    # rows behind the end of out stay as they were
    big = torch.full((n + 1, D), -7.0, dtype=od, device=DEV)
    rn.embedding(ids.to(DEV), table.to(DEV), scale=3.0, out=big[:n])
    assert torch.equal(big[:n], out) and (big[n] == -7.0).all()


def _ids(kind, n, V, seed):
    if kind == "one":
        return torch.full((n,), V // 2, dtype=I32)
    if kind == "outside":
        return torch.randint(0, 2, (n,), generator=_gen(seed), dtype=I32) * (V + 5) - 1
    u = torch.rand(n, generator=_gen(seed), dtype=torch.float64)
    ids = (torch.exp(u * math.log(V + 1)) - 1).floor().clamp(0, V - 1).to(I32)  # the frequencies of words
    if kind == "holes":
        ids[torch.rand(n, generator=_gen(seed + 1)) < 0.3] = -1
    return ids


@pytest.mark.parametrize("kind,n,V,D", [
    ("words", 1, 1, 1), ("words", 1, 600, 3), ("words", 63, 7, 8), ("words", 64, 300, 40), ("words", 65, 3, 100),
    ("one", 33, 5, 16), ("one", 1000, 2, 24), ("holes", 500, 40, 33), ("outside", 70, 20, 16), ("words", 1025, 4, 2050),
    ("words", 3000, 1000, 20), ("holes", 4100, 513, 9), ("one", 2049, 700, 65), ("words", 2500, 9, 700), ("one", 1500, 3, 1030),
    ("words", 1200, 2000, 4100)])
@pytest.mark.parametrize("dt,od", [(BF, F32), (F32, F32), (BF, BF)])
def test_embedding_gradient(kind, n, V, D, dt, od):
    ids, d_o = _ids(kind, n, V, 3), _r(4, n, D, dt=dt)
    got = rn.embedding_bwd(ids.to(DEV), d_o.to(DEV), V, scale=0.5, out_dtype=od)
    want, mag, most = ref.embedding_bwd(ids, d_o, V, 0.5)
    assert got.shape == (V, D) and got.dtype == od
    assert_near(got, want, mag, most + 4, f"{kind} {n} {V} {D}")


def test_embedding_gradient_of_strided_rows_and_batches():
    ids = _ids("holes", 60, 11, 5).reshape(4, 15)
    for dt, extra in ((BF, 3), (F32, 8)):
        d_o = _wide(6, (4, 15), 20, extra, dt)
        want, mag, most = ref.embedding_bwd(ids, d_o, 11, 1.0)
        assert_near(rn.embedding_bwd(ids.to(DEV), _dev(d_o), 11), want, mag, most + 4, "strided")


def test_embedding_without_tokens():
    ids = torch.empty(0, dtype=I32, device=DEV)
    table = torch.ones(5, 3, device=DEV)
    assert rn.embedding(ids, table).shape == (0, 3)
    out = torch.full((5, 3), 9.0, device=DEV)
    rn.embedding_bwd(ids, torch.empty(0, 3, device=DEV), 5, out=out)
    assert not out.any()


# -------------------------------------------------------------------------------------- norm
WIDTHS = [1, 2, 7, 8, 63, 64, 65, 100, 128, 129, 256, 257, 512, 513, 1000, 1023, 1024]


def _norm_case(B, H, L, W, dt, seed, gate=True, weight=True, bias=True):
    x = _r(seed, B, H, L, W, dt=dt) + (0.3 * _r(seed + 1, H, 1, W)).to(dt)
    return dict(x=x, gate=_r(seed + 2, B, L, H * W, dt=dt) if gate else None, w=1 + 0.2 * _r(seed + 3, H * W) if weight else None,
                b=0.3 * _r(seed + 4, H * W) if bias else None, d_o=_r(seed + 5, B, L, H * W, dt=dt))


def _check_norm(v, silu, eps, lengths, out, what):
    want = ref.norm(v["x"], v["gate"], v["w"], v["b"], silu, eps, lengths)
    B, H, L, W = v["x"].shape
    o, mag = (torch.where(want["live"], want[k], 0.0).reshape(B, L, H * W) for k in ("out", "mag"))
    assert_near(out, o, mag, W + 48, f"{what}: out")


def _check_grads(v, silu, eps, lengths, g, what):
    want = ref.norm_bwd(v["x"], v["d_o"], v["gate"], v["w"], v["b"], silu, eps, lengths)
    B, H, L, W = v["x"].shape
    for name, k in (("dx", W + 96), ("dgate", W + 96), ("dweight", W + 96 + B * L), ("dbias", W + 96 + B * L)):
        got = getattr(g, name)
        if got is None:
            assert (name == "dgate" and v["gate"] is None) or (name == "dweight" and v["w"] is None) or \
                (name == "dbias" and v["b"] is None)
        else:
            assert_near(got, *want[name], k, f"{what}: {name}")


def _run_norm(v, silu=True, eps=1e-5, lengths=None, **kw):
    d = {k: _dev(t) for k, t in v.items()}
    ln = None if lengths is None else torch.tensor(lengths, dtype=I32, device=DEV)
    out = rn.group_norm_gate(d["x"], d["gate"], d["w"], d["b"], silu=silu, eps=eps, lengths=ln, **kw)
    return out, rn.group_norm_gate_bwd(d["x"], d["d_o"], d["gate"], d["w"], d["b"], silu=silu, eps=eps, lengths=ln)


@pytest.mark.parametrize("W", WIDTHS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_norm_widths(W, dt):
    v = _norm_case(2, 3, 5, W, dt, 10)
    out, g = _run_norm(v, eps=1e-3)
    _check_norm(v, True, 1e-3, None, out, f"W {W}")
    _check_grads(v, True, 1e-3, None, g, f"W {W}")


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("weight,bias", [(True, True), (True, False), (False, True), (False, False)])
def test_norm_options(gate, silu, weight, bias):
    v = _norm_case(1, 2, 9, 40, F32, 20, gate, weight, bias)
    out, g = _run_norm(v, silu)
    _check_norm(v, silu, 1e-5, None, out, "options")
    _check_grads(v, silu, 1e-5, None, g, "options")


@pytest.mark.parametrize("B,H,L,W", [(1, 1, 1, 512), (64, 8, 1, 64), (1, 1, 3000, 16), (3, 16, 100, 33), (2, 2, 700, 256)])
def test_norm_shapes(B, H, L, W):
    v = _norm_case(B, H, L, W, BF, 30)
    out, g = _run_norm(v)
    _check_norm(v, True, 1e-5, None, out, "shapes")
    _check_grads(v, True, 1e-5, None, g, "shapes")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("lengths", [[0, 6, 3], [9, -2, 1], [6, 6, 6], [0, 0, 0]])
def test_norm_lengths(dt, lengths):
    """Rows behind an end hold NaN in every input; the output there keeps its bits, the gradients are zero."""
    v = _norm_case(3, 2, 6, 50, dt, 40)
    clean = {k: None if t is None else t.clone() for k, t in v.items()}
    for b, n in enumerate(lengths):
        v["x"][b, :, max(n, 0):] = float("nan")
        v["gate"][b, max(n, 0):] = float("nan")
        v["d_o"][b, max(n, 0):] = float("nan")
    mark = torch.full((3, 6, 100), -7.0, dtype=dt, device=DEV)
    out, g = _run_norm(v, lengths=lengths, out=mark)
    live = torch.arange(6)[None] < torch.tensor(lengths)[:, None]
    assert (out.cpu()[~live] == -7.0).all()
    out = torch.where(live[..., None].to(DEV), out, 0)
    _check_norm(clean, True, 1e-5, lengths, out, "lengths")
    _check_grads(clean, True, 1e-5, lengths, g, "lengths")
    assert not g.dx.transpose(1, 2).cpu()[~live].any() and not g.dgate.cpu()[~live].any()


def test_norm_strides():
    """x as heads of token-major rows, as a slice of wider rows, a gate that is a slice; one token's heads."""
    v = _norm_case(2, 3, 7, 20, BF, 50)
    v["x"] = _r(51, 2, 7, 3 * 20 + 5, dt=BF)[..., 5:].unflatten(-1, (3, 20)).transpose(1, 2)
    v["gate"] = _wide(52, (2, 7), 60, 3, BF)
    out, g = _run_norm(v)
    _check_norm(v, True, 1e-5, None, out, "strides")
    _check_grads(v, True, 1e-5, None, g, "strides")
    one = _r(53, 4, 3, 20, dt=BF)
    v = dict(v, x=one.unsqueeze(2), gate=_r(54, 4, 1, 60, dt=BF))
    d = {k: _dev(v[k]) for k in ("x", "gate", "w", "b")}
    _check_norm(v, True, 1e-5, None, rn.group_norm_gate(one.to(DEV).unsqueeze(2), d["gate"], d["w"], d["b"]), "one token")


@pytest.mark.parametrize("dt,od", [(BF, F32), (F32, BF)])
def test_norm_out_dtype(dt, od):
    v = _norm_case(2, 2, 5, 70, dt, 60)
    out, _ = _run_norm(v, out_dtype=od)
    d = {k: _dev(t) for k, t in v.items()}
    g = rn.group_norm_gate_bwd(d["x"], d["d_o"], d["gate"], d["w"], d["b"], out_dtype=od)
    assert out.dtype == g.dx.dtype == g.dgate.dtype == od and g.dweight.dtype == F32
    _check_norm(v, True, 1e-5, None, out, "out dtype")
    _check_grads(v, True, 1e-5, None, g, "out dtype")


def test_norm_rows_of_one_value():
    """A variance of zero: the norm is 0 (times the weight, plus the bias), its gradient that of x / sqrt(eps)."""
    v = _norm_case(1, 2, 3, 64, F32, 70)
    v["x"] = torch.full_like(v["x"], 0.5)
    out, g = _run_norm(v)
    _check_norm(v, True, 1e-5, None, out, "constant")
    _check_grads(v, True, 1e-5, None, g, "constant")


def test_norm_spoils_no_other_row():
    """An infinity or NaN stays in its own token and head."""
    v = _norm_case(1, 2, 4, 72, F32, 75)
    d = {k: _dev(t) for k, t in v.items()}
    want = rn.group_norm_gate(d["x"], d["gate"], d["w"], d["b"])
    d["x"][0, 1, 2, 5] = float("inf")
    d["x"][0, 0, 1, 0] = float("nan")
    got = rn.group_norm_gate(d["x"], d["gate"], d["w"], d["b"]).reshape(4, 2, 72)
    bad = torch.zeros(4, 2, dtype=torch.bool, device=DEV)
    bad[2, 1] = bad[1, 0] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want.reshape(4, 2, 72)[~bad])


def test_norm_without_tokens():
    x, gate, w = torch.empty(2, 3, 0, 8, device=DEV), torch.empty(2, 0, 24, device=DEV), torch.ones(24, device=DEV)
    assert rn.group_norm_gate(x, gate, w, w).shape == (2, 0, 24)
    g = rn.group_norm_gate_bwd(x, gate, gate, w, w)
    assert g.dx.shape == x.shape and not g.dweight.any() and not g.dbias.any()


# ------------------------------------------------------------------------------------ linear
def _linear_case(M, N, K, seed, bias=True, residual=False, rdt=BF, extra=0):
    return dict(x=_wide(seed, (M,), K, extra, BF) if extra else _r(seed, M, K, dt=BF), w=(_r(seed + 1, N, K) * K ** -0.5).to(BF),
                b=_r(seed + 2, N, dt=BF) if bias else None, r=_r(seed + 3, M, N, dt=rdt) if residual else None,
                d_o=_r(seed + 4, M, N, dt=BF))


def _check_linear(v, activation=None, **kw):
    d = {k: _dev(t) for k, t in v.items()}
    out, pre = rn.linear(d["x"], d["w"], d["b"], activation=activation, residual=d["r"], pre_out=True, **kw)
    o, om, z, zm = ref.linear(v["x"], v["w"], v["b"], activation, v["r"])
    K = v["w"].shape[1]
    assert_near(out, o, om, 2 * K + 160, "out")
    assert_near(pre, z, zm, 2 * K + 2, "pre")
    return d, pre


def _check_linear_bwd(v, d, pre, activation, **kw):
    M, N, K = v["x"].shape[0], *v["w"].shape
    g = rn.linear_bwd(d["x"], d["w"], d["d_o"], pre=pre if activation else None, activation=activation, dbias=True, **kw)
    want = ref.linear_bwd(v["x"], v["w"], v["d_o"], pre, activation, 16 if activation else 0)
    for name, k in (("dx", 2 * N + 8), ("dw", 2 * M + 8), ("dbias", M + 64)):
        value, mag, turn = want[name]
        # what a turned rounding of dz may add joins the magnitude
        assert_near(getattr(g, name), value, mag + turn / (k * ref.U), k, name)


SIZES = [(1, 1, 1), (1, 64, 64), (2, 3, 5), (3, 4096, 512), (5, 37, 1000), (8, 130, 513), (9, 1, 8), (9, 64, 64), (16, 100, 72),
         (33, 65, 40), (63, 64, 64), (64, 192, 128), (65, 63, 65), (100, 2, 300), (127, 129, 64), (128, 128, 64), (200, 256, 1024),
         (257, 255, 96), (17, 8, 5000), (300, 520, 33)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("activation", [None, "gelu", "silu"])
def test_linear_sizes(M, N, K, activation):
    v = _linear_case(M, N, K, 100)
    d, pre = _check_linear(v, activation)
    _check_linear_bwd(v, d, pre, activation)


@pytest.mark.parametrize("M,N,K", [(4, 50, 24), (70, 130, 200), (300, 300, 64)])
@pytest.mark.parametrize("rdt,od", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("bias", [True, False])
def test_linear_residuals_and_types(M, N, K, rdt, od, bias):
    v = _linear_case(M, N, K, 110, bias, True, rdt)
    d, pre = _check_linear(v, "gelu", out_dtype=od)
    _check_linear_bwd(v, d, pre, "gelu", out_dtype=od)


@pytest.mark.parametrize("M", [3, 40, 130])
@pytest.mark.parametrize("extra", [1, 2, 8])
def test_linear_strided_rows(M, extra):
    v = _linear_case(M, 72, 96, 120, extra=extra)
    d, pre = _check_linear(v, "silu")
    _check_linear_bwd(v, d, pre, "silu")


@pytest.mark.parametrize("M,N,K", [(2, 30, 70), (90, 61, 64)])
def test_linear_misaligned_weights(M, N, K):
    """A weight and d_o that start two bytes behind a 16-byte border."""
    v = _linear_case(M, N, K, 125)
    d, pre = _check_linear(v)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].reshape(t.shape)  # noqa: E731
    assert torch.equal(rn.linear(off(d["x"]), off(d["w"]), d["b"]), rn.linear(d["x"], d["w"], d["b"]))
    a, b = (rn.linear_bwd(f(d["x"]), f(d["w"]), f(d["d_o"])) for f in (off, lambda t: t))
    assert torch.equal(a.dx, b.dx) and torch.equal(a.dw, b.dw)


def test_linear_large_tiles():
    """Sizes at which the larger tiles and, with few tiles and a long k, its parts are taken."""
    for M, N, K in ((4096, 4160, 72), (2304, 2050, 128), (130, 70, 6000)):
        v = _linear_case(M, N, K, 130)
        d, pre = _check_linear(v, "gelu")
        _check_linear_bwd(v, d, pre, "gelu")


@pytest.mark.parametrize("M,N,K", [(777, 1302, 200), (520, 700, 1000), (1100, 2100, 72), (2304, 2050, 64), (300, 4000, 71),
                                   (2200, 2050, 77), (4096, 4100, 9), (1000, 33, 3001)])
def test_linear_between_the_tiles(M, N, K):
    """Sizes at which one kind of tile gives way to the next, aligned and not."""
    v = _linear_case(M, N, K, 135, True, True)
    d, pre = _check_linear(v, "silu")
    _check_linear_bwd(v, d, pre, "silu")


def test_linear_in_place_and_leading_axes():
    v = _linear_case(6, 24, 16, 140, True, True)
    d = {k: _dev(t) for k, t in v.items()}
    want = rn.linear(d["x"], d["w"], d["b"], "gelu", d["r"])
    x3, r3 = d["x"].reshape(2, 3, 16), d["r"].clone().reshape(2, 3, 24)
    got = rn.linear(x3, d["w"], d["b"], "gelu", r3, out=r3)
    assert got is r3 and torch.equal(got.reshape(6, 24), want)
    for m in (20, 300):  # tiles, and parts of k that are joined
        big = _linear_case(m, 40, 2048, 141, True, True)
        b = {k: _dev(t) for k, t in big.items()}
        want = rn.linear(b["x"], b["w"], b["b"], "silu", b["r"])
        assert torch.equal(rn.linear(b["x"], b["w"], b["b"], "silu", b["r"], out=b["r"]), want)


def test_linear_wanted_gradients_only():
    v = _linear_case(30, 24, 16, 145)
    d = {k: _dev(t) for k, t in v.items()}
    z = _r(146, 30, 24, dt=BF).to(DEV)
    every = rn.linear_bwd(d["x"], d["w"], d["d_o"], z, "gelu", dbias=True)
    for i, name in enumerate(("dx", "dw", "dbias")):
        one = rn.linear_bwd(d["x"], d["w"], d["d_o"], z, "gelu", **{n: n == name for n in ("dx", "dw", "dbias")})
        assert all((t is None) == (j != i) for j, t in enumerate(one)) and torch.equal(one[i], every[i])


def test_linear_infinities_and_nan_stay_in_their_rows():
    """A token's NaN or infinity reaches its own row of the output only; of w, its own column."""
    for M in (4, 70):
        v = _linear_case(M, 80, 65, 150)
        d = {k: _dev(t) for k, t in v.items()}
        want = rn.linear(d["x"], d["w"])
        d["x"][2, 64], d["x"][M - 1, 0] = float("nan"), float("inf")
        d["w"][79, 3] = float("nan")
        got = rn.linear(d["x"], d["w"])
        assert torch.isnan(got[2]).all() and not torch.isfinite(got[M - 1]).any() and torch.isnan(got[:, 79]).all()
        ok = torch.ones(M, 80, dtype=torch.bool, device=DEV)
        ok[2] = ok[M - 1] = False
        ok[:, 79] = False
        assert torch.equal(got[ok], want[ok])


@pytest.mark.parametrize("M", [9, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("N,K", [(1, 1), (15, 63), (17, 64), (300, 65), (48, 700), (130, 2047), (2100, 1000)])
def test_linear_a_batch_of_tokens(M, N, K):
    """Up to 64 tokens: rows of w and of x behind the last, chunks of k that not every wave has, and a part of one."""
    v = _linear_case(M, N, K, 160, True, True, F32 if M % 2 else BF, extra=M % 3)
    d, _ = _check_linear(v, "gelu" if M % 2 else "silu", out_dtype=F32 if M % 2 else BF)
    x = torch.cat([d["x"].new_zeros(1), d["x"].reshape(-1)])[1:].reshape(M, K) if M % 3 == 0 else d["x"]
    want = rn.linear(d["x"], d["w"], d["b"], residual=d["r"], out_dtype=d["r"].dtype)
    assert torch.equal(rn.linear(x, d["w"], d["b"], residual=d["r"], out=d["r"]), want)


@pytest.mark.parametrize("M,N,K", [(9, 2100, 4200), (12, 2300, 4160), (20, 8200, 500), (60, 4200, 130)])
def test_linear_a_batch_of_tokens_in_turns(M, N, K):
    """More chunks of k than a wave has under way at a time, and more workgroups than there are CUs."""
    _check_linear(_linear_case(M, N, K, 165, True, True), "silu")


@pytest.mark.parametrize("M", [12, 40])
def test_linear_a_batch_keeps_nan_in_its_row(M):
    v = _linear_case(M, 80, 200, 170)
    d = {k: _dev(t) for k, t in v.items()}
    want = rn.linear(d["x"], d["w"])
    d["x"][M - 1, 199], d["w"][79, 3] = float("nan"), float("inf")
    got = rn.linear(d["x"], d["w"])
    assert torch.isnan(got[M - 1]).all() and not torch.isfinite(got[:, 79]).any()
    assert torch.equal(got[:M - 1, :79], want[:M - 1, :79])


def test_rows_of_three_leading_axes():
    """Three axes of rows at one stride are taken, in another order refused, also where a part of the strides fits."""
    x, w, ids = _r(180, 3, 2, 2, 16, dt=BF).to(DEV), _r(181, 8, 16, dt=BF).to(DEV), torch.zeros(3, 2, 2, dtype=torch.int32, device=DEV)
    wide = torch.cat([x, x], -1)[..., :16]
    assert torch.equal(rn.linear(wide, w), rn.linear(x, w)) and torch.equal(rn.embedding_bwd(ids, wide, 4), rn.embedding_bwd(ids, x, 4))
    for axes in ((1, 0), (0, 2), (1, 2)):
        t, i = x.transpose(*axes), ids.transpose(*axes).contiguous()
        with pytest.raises(ValueError, match="one stride"):
            rn.linear(t, w)
        with pytest.raises(ValueError, match="one stride"):
            rn.linear_bwd(t, w, rn.linear(t.contiguous(), w))
        with pytest.raises(ValueError, match="one stride"):
            rn.embedding_bwd(i, t, 4)
    assert torch.equal(rn.linear(x[0, 0, 0], w), rn.linear(x, w)[0, 0, 0])
    with pytest.raises(ValueError, match="one stride"):
        rn.linear(x[0, 0, 0, ::8], w[:, :2].contiguous())
    with pytest.raises(rn.RetentionError, match="sizes must be positive"):
        rn.linear(x[..., :0].contiguous(), w[:, :0].contiguous())


def test_activations_far_out():
    """gelu and silu of pre-activations from -40 to 40 and at infinity, through a product with the identity."""
    z = torch.cat([torch.linspace(-40, 40, 801), torch.tensor([float("inf"), 1e-30, -1e-30, 0.0])]).to(BF)
    x, w = z[:, None].contiguous().to(DEV), torch.ones(1, 1, dtype=BF, device=DEV)
    for name in ("gelu", "silu"):
        out = rn.linear(x, w, activation=name, out_dtype=F32)[:, 0].cpu()
        assert out[801] == float("inf")
        out[801] = z[801] = 0.0
        want = ref.act(z.double(), name)
        # gelu's tail to 5.7e-6 of it, and 1e-9 of z behind -6; silu's exponential grows with |z|
        tail = 5.8e-6 * (want.abs()) if name == "gelu" else (8 + 2 * z.double().abs()) * ref.U * want.abs()
        assert ((out.double() - want).abs() <= tail + 4 * ref.U * want.abs() + 6e-9 + 1e-37).all(), name
        one = torch.ones_like(z)[:, None].to(DEV)
        g = rn.linear_bwd(x, w, one, pre=z[:, None].to(DEV), activation=name, dw=False, out_dtype=F32).dx[:, 0].cpu()
        assert ((g.double() - ref.act_slope(z.double(), name)).abs() <= 2.0 ** -8 * ref.act_slope(z.double(), name).abs() + 1e-7).all()


def test_linear_without_tokens():
    w, b = torch.ones(5, 3, dtype=BF, device=DEV), torch.ones(5, dtype=BF, device=DEV)
    x, d_o = torch.empty(0, 3, dtype=BF, device=DEV), torch.empty(0, 5, dtype=BF, device=DEV)
    assert rn.linear(x, w, b).shape == (0, 5)
    g = rn.linear_bwd(x, w, d_o, pre=d_o, activation="gelu", dbias=True)
    assert g.dx.shape == (0, 3) and not g.dw.any() and not g.dbias.any()


# ------------------------------------------------------------------------------------- beams
def _check_select(z, cum, K, ended=None, eos=0):
    e = None if ended is None else ended.to(DEV)
    got = rn.beam_select(_dev(z), cum.to(DEV), K, ended=e, eos=eos)
    tokens, parents, best, gap = ref.beam_select(z, cum, K, ended, eos)
    assert gap > 1e-5, "the oracle's own scores are too near each other to tell"
    assert torch.equal(got.tokens.cpu().long(), tokens) and torch.equal(got.parents.cpu().long(), parents)
    s, fine = got.scores.cpu().double(), torch.isfinite(best)
    assert torch.equal(s[~fine], best[~fine])
    assert ((s - best)[fine].abs() <= (64 + best[fine].abs()) * ref.U).all()
    return got


SELECT = [(2, 16, 4096, 32), (3, 17, 2049, 9), (2, 1, 65536, 32), (2, 2, 40000, 33), (1, 1, 1, 1), (1, 1, 5, 5), (3, 2, 3, 6), (2, 4, 100, 8), (1, 1, 2048, 64), (2, 3, 2049, 7), (1, 2, 8193, 16),
          (4, 5, 1000, 10), (5, 64, 40, 64), (1, 1, 20000, 4), (70, 4, 300, 4), (300, 2, 64, 3), (1, 3, 33, 64)]


@pytest.mark.parametrize("B,W,V,K", SELECT)
@pytest.mark.parametrize("dt", [BF, F32])
def test_select_shapes(B, W, V, K, dt):
    """Values of 16 bits meet their like in a row, so ties are everywhere with bf16."""
    _check_select((2.5 * _r(200, B, W, V)).to(dt), -5 * torch.rand(B, W, generator=_gen(201)), K)


def test_select_all_tied():
    """Equal logits, equal beams: the lowest indices, whatever the slices are."""
    for V, K in ((10, 7), (5000, 64), (30000, 20), (2000, 32), (30000, 64)):
        z, cum = torch.zeros(2, 3, V), torch.full((2, 3), -1.5)
        got = rn.beam_select(z.to(DEV), cum.to(DEV), K)
        assert torch.equal(got.tokens.cpu(), (torch.arange(K) % V).to(I32).expand(2, K))
        assert torch.equal(got.parents.cpu(), (torch.arange(K) // V).to(I32).expand(2, K))
    # minus zero and zero are one value
    z = torch.zeros(1, 1, 100)
    z[..., ::2] = -0.0
    assert torch.equal(rn.beam_select(z.to(DEV), torch.zeros(1, 1, device=DEV), 9).tokens.cpu()[0], torch.arange(9, dtype=I32))


def test_select_first_step():
    """Beams that are not open yet, at -inf, offer nothing while there is anything else."""
    z = (2.0 * _r(210, 1, 1, 500)).expand(2, 4, 500).contiguous()
    cum = torch.full((2, 4), -math.inf)
    cum[:, 0] = 0.0
    got = _check_select(z, cum, 4)
    assert not got.parents.any()
    got = _check_select(z[..., :3].contiguous(), cum, 8)  # more wanted than there is: by index
    assert torch.equal(got.parents.cpu()[0], torch.tensor([0, 0, 0, 1, 1, 1, 2, 2], dtype=I32))


@pytest.mark.parametrize("eos", [0, 3, 49])
def test_select_ended_beams(eos):
    z, cum = _r(220, 4, 3, 50), -3 * torch.rand(4, 3, generator=_gen(221))
    ended = torch.tensor([[1, 0, 0], [0, 1, 1], [1, 1, 1], [0, 0, 0]], dtype=torch.bool)
    z[2, 1], z[0, 0, 7] = float("nan"), float("inf")  # an ended beam's logits are not looked at
    _check_select(z, cum, 5, ended, eos)
    _check_select(z[:, :, :eos + 1].contiguous(), cum, 3 if eos else 2, ended, eos)


@pytest.mark.parametrize("dt", [BF, F32])
def test_select_masks(dt):
    """Forbidden tokens at -inf or the type's lowest value, a row of nothing else, NaN and +inf."""
    z = _r(230, 3, 4, 3000).to(dt)
    z[0, 0, 5:] = -math.inf
    z[0, 1] = -math.inf
    z[0, 2, 17] = math.nan
    z[0, 3, 2999] = math.inf
    z[1, :, 1:] = torch.finfo(dt).min
    z[2, 1] = torch.finfo(dt).min
    cum = -torch.rand(3, 4, generator=_gen(231))
    cum[1, 3], cum[2, 3] = math.nan, math.inf
    _check_select(z, cum, 8)


def test_select_strided_rows():
    z = _wide(240, (3, 4), 70, 5, BF)
    _check_select(z, -torch.rand(3, 4, generator=_gen(241)), 6)


def test_select_large_vocabulary():
    """2^20 tokens, two beams: some 500 slices a beam."""
    V = 1 << 20
    z = _r(250, 1, 2, V)
    cum = torch.tensor([[0.0, -0.1]])
    got = rn.beam_select(z.to(DEV), cum.to(DEV), 64)
    s = (cum[..., None].double() + torch.log_softmax(z.double(), -1)).reshape(-1)
    best, at = s.sort(descending=True, stable=True)
    assert (best[:64] - best[1:65]).min() > 1e-6
    assert torch.equal(got.parents.cpu()[0].long() * V + got.tokens.cpu()[0].long(), at[:64])


REORDER = [(1, 2, 16), (3, 4, 4096 * 5), (2, 5, 12), (2, 8, 100), (4, 3, 7), (1, 16, 64), (2, 17, 48), (1, 33, 36), (1, 64, 20),
           (2, 64, 8192)]


@pytest.mark.parametrize("B,W,size", REORDER)
def test_reorder(B, W, size):
    parents = torch.randint(-1, W + 1, (B, W), generator=_gen(300), dtype=I32)  # both kinds outside among them
    every = [torch.randint(0, 256, (B, W, size), generator=_gen(301), dtype=torch.uint8), _r(302, B, W, 3, 5, dt=BF),
             torch.arange(B * W, dtype=I32).reshape(B, W), _r(303, B * W, 6).reshape(B * W, 6)]
    p = torch.where((parents >= 0) & (parents < W), parents, torch.arange(W, dtype=I32)).long()
    want = [t.reshape(B, W, -1)[torch.arange(B)[:, None], p].reshape(t.shape) for t in every]
    states = [t.to(DEV) for t in every]
    assert rn.beam_reorder(states, parents.to(DEV)) is states
    for got, w in zip(states, want):
        assert torch.equal(got.cpu(), w)
    # a size and an address that nothing but bytes divides
    odd = torch.randint(0, 256, (B * W * size + 1,), generator=_gen(304), dtype=torch.uint8)
    t = odd.to(DEV)[1:].reshape(B, W, size)
    rn.beam_reorder(t, parents.to(DEV))
    assert torch.equal(t.cpu(), odd[1:].reshape(B, W, size)[torch.arange(B)[:, None], p])


def test_reorder_exchanges_and_rotations():
    parents = torch.tensor([[1, 0, 3, 2], [3, 0, 1, 2], [0, 1, 2, 3], [2, 2, 2, 2]], dtype=I32)
    t = _r(310, 4, 4, 1000)
    got = rn.beam_reorder(t.to(DEV), parents.to(DEV)).cpu()
    assert torch.equal(got, t[torch.arange(4)[:, None], parents.long()])


def test_reorder_many_tensors():
    parents = torch.randint(0, 3, (2, 3), generator=_gen(320), dtype=I32)
    every = [_r(321 + i, 2, 3, 1 + 37 * i) for i in range(64)]
    states = [t.to(DEV) for t in every]
    rn.beam_reorder(states, parents.to(DEV))
    for got, t in zip(states, every):
        assert torch.equal(got.cpu(), t[torch.arange(2)[:, None], parents.long()])


# --------------------------------------------------------------------- refusals of the binding
def test_binding_refuses():
    x, w, ids = torch.zeros(4, 8, dtype=BF, device=DEV), torch.zeros(6, 8, dtype=BF, device=DEV), torch.zeros(4, dtype=I32, device=DEV)
    t = torch.zeros(1, 2, 4, 8, device=DEV)
    p = torch.zeros(1, 2, dtype=I32, device=DEV)
    cases = [(TypeError, lambda: rn.embedding(ids.long(), w)), (ValueError, lambda: rn.embedding(ids, w[0])),
             (TypeError, lambda: rn.embedding(ids, w.half())), (ValueError, lambda: rn.embedding(ids, w.T)),
             (ValueError, lambda: rn.embedding_bwd(ids, x[:3], 9)),
             (ValueError, lambda: rn.group_norm_gate(t[0])), (ValueError, lambda: rn.group_norm_gate(t.transpose(2, 3))),
             (ValueError, lambda: rn.group_norm_gate(t, torch.zeros(1, 4, 8, device=DEV))),
             (rn.RetentionError, lambda: rn.group_norm_gate(t, eps=0.0)),
             (TypeError, lambda: rn.linear(x.float(), w)), (ValueError, lambda: rn.linear(x, w[:, :4])),
             (ValueError, lambda: rn.linear(x, w, activation="relu")), (TypeError, lambda: rn.linear(x, w, residual=torch.zeros(4, 6, device=DEV).half())),
             (ValueError, lambda: rn.linear(x, w, bias=torch.zeros(5, dtype=BF, device=DEV))),
             (ValueError, lambda: rn.linear_bwd(x, w, torch.zeros(4, 6, dtype=BF, device=DEV), activation="gelu")),
             (TypeError, lambda: rn.beam_select(t[0], torch.zeros(2, 4, device=DEV), 2, ended=p.expand(2, 2))),
             (ValueError, lambda: rn.beam_select(t, torch.zeros(2, 4, device=DEV), 2)),
             (rn.RetentionError, lambda: rn.beam_select(t[0], torch.zeros(2, 4, device=DEV), 65)),
             (ValueError, lambda: rn.beam_reorder(torch.zeros(3, 2, device=DEV), p)),
             (ValueError, lambda: rn.beam_reorder(torch.zeros(1, 2, 4, device=DEV)[..., ::2], p)),
             (TypeError, lambda: rn.beam_reorder(t, p.long())), (rn.RetentionError, lambda: rn.beam_reorder([t] * 2, p))]
    for kind, call in cases:
        with pytest.raises(kind):
            call()
