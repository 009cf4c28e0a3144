"""GPU tests of the operators around the layers (include/language.h) at the edges of what their calls take, and at the
sizes that small calls do not reach: row strides beyond 32 bits within a tile, beams whose scores are so far out
that their tokens' scores meet, rows that hold almost everything in one token, parameters that are not finite
beside rows that do not count, activations far out, workgroups that take several tokens, full batches of a
selection, a search whose beams end."""
import math

import pytest
import torch

import retentive_network_scale_amd as rn
from tests import _language_ref as ref
from tests._recurrent_ref import assert_near
from tests.test_gpu_language import _check_grads, _check_norm, _norm_case, _run_norm
from tests.test_gpu_language_model import Search

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _r(seed, *shape, dt=F32):
    return torch.randn(*shape, generator=_gen(seed)).to(dt)


# -------------------------------------------------------------------------------------- norm
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_norm_rows_behind_an_end_have_no_gradient(gate, value):
    """Whatever weight and bias hold; sums over no token at all are zero."""
    B, H, L, W = 3, 2, 7, 40
    x, d_o = _r(30, B, H, L, W).to(DEV), _r(31, B, L, H * W).to(DEV)
    g = _r(32, B, L, H * W).to(DEV) if gate else None
    w, b = torch.ones(H * W, device=DEV), torch.zeros(H * W, device=DEV)
    w[50], b[3] = value, value
    for lengths in ([2, 0, 7], [0, 0, 0]):
        got = rn.group_norm_gate_bwd(x, d_o, g, w, b, lengths=torch.tensor(lengths, dtype=I32, device=DEV))
        dead = torch.arange(L)[None] >= torch.tensor(lengths)[:, None]
        assert (got.dx.transpose(1, 2).cpu()[dead] == 0).all()
        assert not gate or (got.dgate.cpu()[dead] == 0).all()
    assert (got.dweight == 0).all() and (got.dbias == 0).all()


@pytest.mark.parametrize("B,H,L,W", [(3, 64, 3500, 20), (2, 32, 2000, 100), (3, 64, 220, 512), (5, 128, 31, 700)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_norm_many_tokens_a_workgroup(B, H, L, W, dt):
    """Workgroups that take several tokens, one after the other: with lengths, so that tokens that count follow
    ones that do not, and sums over tokens that stay in registers."""
    v = _norm_case(B, H, L, W, dt, 35)
    for lengths in (None, [L] + [(i * 7 + 3) * L // 29 if i % 2 else 0 for i in range(1, B)]):
        out, g = _run_norm(v, lengths=lengths, out=torch.zeros(B, L, H * W, dtype=dt, device=DEV))
        _check_norm(v, True, 1e-5, lengths, out, "many")
        _check_grads(v, True, 1e-5, lengths, g, "many")


# ------------------------------------------------------------------------------------ linear
@pytest.mark.parametrize("ld", [(1 << 26) + (1 << 22) + 8, (1 << 26) + (1 << 22) + 7])
@pytest.mark.parametrize("M,N,K", [(70, 320, 136), (128, 32000, 72), (128, 2100, 65), (9, 40, 72), (3, 40, 72)])
def test_linear_rows_far_apart(M, N, K, ld):
    """The last token of each of many long prompts: rows of x so far apart that a tile's offsets pass 2^32
    elements.  The result is that of the same rows one behind the other, and so is dw: each is the same
    sum in the same order."""
    rows = _r(1, M, K, dt=BF).to(DEV)
    far = torch.empty(M * ld, dtype=BF, device=DEV).as_strided((M, K), (ld, 1))  # what lies between has no values
    far.copy_(rows)
    w, b, d_o = (_r(2, N, K) * K ** -0.5).to(BF).to(DEV), _r(3, N, dt=BF).to(DEV), _r(4, M, N, dt=BF).to(DEV)
    assert torch.equal(rn.linear(far, w, b), rn.linear(rows, w, b))
    far_g, g = (rn.linear_bwd(x, w, d_o, dbias=True) for x in (far, rows))
    assert all(torch.equal(s, t) for s, t in zip(far_g, g))


@pytest.mark.parametrize("M,N,K", [(9, 300, 1401), (16, 300, 2047), (33, 200, 999), (40, 200, 999), (64, 130, 699), (12, 100, 4095)])
def test_linear_rows_of_odd_length(M, N, K):
    """Few tokens on both sides of where rows of odd length go to the tiles."""
    x, w, b = _r(5, M, K, dt=BF), (_r(6, N, K) * K ** -0.5).to(BF), _r(7, N, dt=BF)
    out, pre = rn.linear(x.to(DEV), w.to(DEV), b.to(DEV), "silu", out_dtype=F32, pre_out=True)
    o, om, z, zm = ref.linear(x, w, b, "silu", None)
    assert_near(out, o, om, 2 * K + 160, "out")
    assert_near(pre, z, zm, 2 * K + 2, "pre")


def _gelu(z):
    """z Phi(z) in 64 bits, with Phi's relative accuracy for far negative z."""
    return z * torch.exp(torch.special.log_ndtr(z))


@pytest.mark.parametrize("M", [3, 40, 200])
@pytest.mark.parametrize("od", [BF, F32])
def test_linear_gelu_of_far_values(M, od):
    """Through a product with the identity, by each of the kernels: in fp32 to (10 + 2 z^2) half steps of the value
    (and its rounding's one) where that is a normal number; in bf16 to half a step and 5.7e-6, behind -6 to 1e-13;
    far out 0."""
    z = torch.cat([torch.linspace(-13, 13, 997), torch.linspace(-40, 40, 401), torch.logspace(-30, 0, 301), -torch.logspace(-30, 0, 301)]).to(BF)
    z = z[:z.numel() // M * M].reshape(M, -1)
    N = z.shape[1]
    got = rn.linear(z.to(DEV), torch.eye(N, dtype=BF, device=DEV), activation="gelu", out_dtype=od).cpu().double()
    want = _gelu(z.double())
    tol = 2.0 ** -24 * (11 + 2 * z.double() ** 2).clamp(max=400) * want.abs() if od == F32 else (2.0 ** -8 + 5.8e-6) * want.abs() + (z < -6) * 1e-13
    assert ((got - want).abs() <= tol + 1.2e-38).all()
    assert not got[z < -14].any()


def test_linear_gelu_slope_of_far_values():
    """The slope, by way of the bias's gradient, to 3.2e-8 and the roundings of z phi(z); far out 0 and 1."""
    z = torch.linspace(-40, 40, 1601).to(BF)[None]
    one = torch.ones(1, z.shape[1], dtype=BF, device=DEV)
    w = torch.zeros(z.shape[1], 8, dtype=BF, device=DEV)
    got = rn.linear_bwd(one[:, :8], w, one, pre=z.to(DEV), activation="gelu", dx=False, dw=False, dbias=True).dbias.cpu().double()
    z = z[0].double()
    phi = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    want = torch.exp(torch.special.log_ndtr(z)) + z * phi
    assert ((got - want).abs() <= 3.3e-8 + 2.0 ** -24 * ((4 + z * z) * z.abs() * phi + 2 * want.abs())).all()
    assert not got[z < -20].any() and (got[z > 20] == 1).all()


# ------------------------------------------------------------------------------------- beams
def _select_ref(z, cum, K):
    """(tokens, parents), every continuation sorted by score, then beam, then logit, then token."""
    B, W, V = z.shape
    got = []
    for b in range(B):
        every = []
        for w in range(W):
            top = z[b, w].double().max().item()
            lse = top + math.log(torch.exp(z[b, w].double() - top).sum().item())
            every += [(-(cum[b, w].item() + (x - lse)), w, -x, v) for v, x in enumerate(z[b, w].tolist())]
        got.append([(v, w) for _, w, _, v in sorted(every)[:K]])
    got = torch.tensor(got, dtype=I32)
    return got[..., 0], got[..., 1]


@pytest.mark.parametrize("score", [torch.finfo(F32).min, -1e30, -1e15])
@pytest.mark.parametrize("W,V,K", [(1, 100, 4), (3, 5, 12), (2, 9000, 20), (1, 70000, 9), (4, 30000, 40), (2, 300, 64)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_select_closed_beams(W, V, K, dt, score):
    """Beams that are closed by a score far out, where the scores of all their tokens are one: a beam's tokens
    come by logit, equal beams by index; and behind an open beam's tokens."""
    z, cum = (2.5 * _r(10, 2, W, V)).to(dt), torch.full((2, W), score)
    cum[1, 0] = -1.0
    got = rn.beam_select(z.to(DEV), cum.to(DEV), K)
    tokens, parents = _select_ref(z, cum, K)
    assert torch.equal(got.tokens.cpu(), tokens) and torch.equal(got.parents.cpu(), parents)
    want = cum.gather(1, parents.long())
    assert ((got.scores.cpu() - want).abs() <= 30 + 2.0 ** -24 * want.abs()).all()


def test_select_logits_closer_than_scores():
    """Logits that differ by less than a score can tell are still in their own order."""
    z = torch.full((1, 1, 4000), -10.0)
    z[0, 0, 7], z[0, 0, 3], z[0, 0, 3999] = 1e-20, 0.0, 2e-20
    got = rn.beam_select(z.to(DEV), torch.zeros(1, 1, device=DEV), 3)
    assert got.tokens.cpu().tolist() == [[3999, 7, 3]]


@pytest.mark.parametrize("V,B", [(50, 1), (9000, 1), (70000, 1), (9000, 100), (40000, 60)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("top", [0.0, 19.5])
def test_select_confident_beams(V, B, dt, top):
    """Beams of one score whose rows hold almost everything in one token: they differ by what is left, far below
    2^-24.  Of the remainder's terms, e^-d, each is off by at most (16 + 3 d) 2^-24, and so is the score."""
    W, K = 8, 8
    left = 17.0 + torch.randperm(W, generator=_gen(20)).double() / 4  # -log of what is left, in steps that both types hold
    z = torch.full((B, W, V), -math.inf)
    at = torch.randint(0, V - 1, (B, W, 1), generator=_gen(21))
    z.scatter_(2, at, top)
    z.scatter_(2, at + 1, (top - left.float())[None, :, None].expand(B, W, 1).clone())
    z = z.to(dt)
    got = rn.beam_select(z.to(DEV), torch.zeros(B, W, device=DEV), K)
    gap = (top - z.gather(2, at + 1).double())[..., 0]
    order = gap.argsort(-1, descending=True)
    want = -torch.log1p(torch.exp(-gap)).gather(1, order)
    assert len(set(gap[0].tolist())) == W
    assert torch.equal(got.parents.cpu().long(), order) and torch.equal(got.tokens.cpu().long(), at[..., 0].gather(1, order))
    assert ((got.scores.cpu().double() - want).abs() <= (17 + 3 * gap.gather(1, order)) * 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("V", [1, 8, 3000, 70000])
def test_select_log_sum_of_equal_logits(V):
    """A row of one value is counted: its log-sum is log V, whatever the slices are, and the score is rounded once."""
    got = rn.beam_select(torch.full((1, 2, V), 3.25, device=DEV), torch.zeros(1, 2, device=DEV), 1)
    assert abs(got.scores.item() + math.log(V)) <= 2.0 ** -24 * math.log(V) + 1e-15


def _check_sorted(z, cum, K, ended=None, eos=0):
    """Against a stable sort of all continuations in 64 bits, on the GPU."""
    got = rn.beam_select(z, cum, K, ended=ended, eos=eos)
    B, W, V = z.shape
    p = z.double() - z.double().amax(-1, keepdim=True)
    p = p - torch.log(torch.exp(p).sum(-1, keepdim=True))
    if ended is not None:
        only = torch.where(torch.arange(V, device=DEV) == eos, 0.0, -math.inf).double()
        p = torch.where(ended[..., None], only, p)
    p = (cum.double()[..., None] + p).reshape(B, -1)
    best, at = p.sort(dim=-1, descending=True, stable=True)
    flat = got.parents.long() * V + got.tokens.long()
    # a score is off by the log-sum's exponentials, at most (16 + 3 d) 2^-24, here with d below 25: 5.5e-6.  Neighbours
    # of different beams that are nearer than twice that may change places; every other row has one answer
    near = 1.1e-5
    gap = best[:, :K] - best[:, 1:K + 1]
    told = ((gap < 1e-9) | (gap > near) | gap.isnan()).all(-1)
    assert told.sum() >= 0.8 * B and torch.equal(flat[told], at[told, :K])
    assert (p.gather(1, flat)[~told] - best[~told, :K]).abs().max() <= near if not told.all() else True
    assert all(len(set(row)) == K for row in flat.tolist())
    off = (got.scores.double() - best[:, :K]).abs()
    assert ((got.scores == best[:, :K]) | (off <= (91 + best[:, :K].abs()) * ref.U) | (~told[:, None] & (off <= 2 * near))).all()


@pytest.mark.parametrize("B,W,V,K", [(16, 8, 8200, 8), (16, 8, 8192, 5), (11, 16, 16385, 12), (70, 2, 40001, 4), (8, 16, 24576, 33),
                                     (20, 8, 8207, 40)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_select_full_batches(B, W, V, K, dt):
    """Rows enough for 32 elements a thread: whole slices, ragged last ones, of odd lengths and strides, ended beams."""
    z = (2.5 * _r(40, B, W, V + 1)).to(dt)[..., 1:] if V % 2 else (2.5 * _r(40, B, W, V)).to(dt)
    z = z._base.to(DEV).as_strided(z.shape, z.stride(), z.storage_offset()) if V % 2 else z.to(DEV)
    cum = -5 * torch.rand(B, W, generator=_gen(41)).to(DEV)
    ended = (torch.rand(B, W, generator=_gen(42)) < 0.2).to(DEV)
    _check_sorted(z, cum, K)
    _check_sorted(z, cum, K, ended, V - 1)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V,K", [(16385, 12), (20000, 50)])
def test_select_full_batches_of_equal_logits(V, K, dt):
    """More elements at the bound than there is room for, in whole slices and in the last: the lowest indices."""
    B, W = 16, 16
    z = torch.zeros(B, W, V, dtype=dt, device=DEV)
    cum = torch.full((B, W), -1.5, device=DEV)
    cum[3, 2], cum[4] = -1.0, -torch.rand(W, generator=_gen(43)).to(DEV)
    z[5, 0, V - 3:], z[6, 0, :V - 3] = 1.0, -math.inf  # the best in the last slice; little but -inf
    z[7, 0, ::2] = -0.0
    got = rn.beam_select(z, cum, K)
    for b in range(B):
        first = {3: 2, 4: cum[4].argmax().item()}.get(b, 0)
        row = [(first, v) for v in range(K)]
        if b in (5, 6):
            row = [(0, V - 3), (0, V - 2), (0, V - 1)] + [(1, v) for v in range(K - 3)]
        assert list(zip(got.parents[b].tolist(), got.tokens[b].tolist())) == row, b


# --------------------------------------------------------------------------------- generation
def test_beam_search_with_ends():
    """A search whose beams end while others go on: its end token is one that a beam takes at its third step."""
    first = Search(31, 3, 4)
    first.eos = 0  # never the best of these rows' tokens by accident: checked below
    first.w_out[0] = 0
    for _ in range(3):
        first.step()
    eos = first.history[1, 2, 2].item()
    assert not first.ended.any()
    own, plain = Search(31, 3, 4), Search(31, 3, 4)
    own.eos = plain.eos = eos
    own.w_out[0] = plain.w_out[0] = 0
    plain.layer = own.layer
    some = 0
    for step in range(10):
        own.step()
        plain.plain_step()
        assert torch.equal(own.history, plain.history), step
        same = [torch.equal(getattr(own, k), getattr(plain, k)) for k in ("state", "pos", "ended")]
        assert all(same), (step, same)
        torch.testing.assert_close(own.scores, plain.scores, rtol=2e-6, atol=2e-5)
        plain.scores.copy_(own.scores)
        some += bool(own.ended[1].any()) and not bool(own.ended.all())
    assert some > 0
