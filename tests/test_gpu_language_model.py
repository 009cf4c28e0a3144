"""The operators of include/language.h together with the framework's own, as a program uses them: a training
step of a small retention language model against autograd in 64 bits, a beam search over the gated
layer's decode step, and all of them captured into graphs, on other streams, two at once, and at offsets
beyond 32 bits."""
import math

import pytest
import torch

import retentive_network_scale_amd as rn
from workloads import multiscale_gamma, rotation_theta

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------------------- training
V, DM, H, DK, DV, FF, CHUNK = 61, 96, 2, 32, 64, 160, 32
B, L = 2, 70


def _weights(seed):
    g = _gen(seed)
    r = lambda n, k: (torch.randn(n, k, generator=g) * k ** -0.5).to(BF)  # noqa: E731
    return dict(table=(torch.randn(V, DM, generator=g) * DM ** -0.5).to(BF), w_q=r(H * DK, DM), w_k=r(H * DK, DM), w_v=r(H * DV, DM),
                w_g=r(H * DV, DM), gn_w=1 + 0.1 * torch.randn(H * DV, generator=g), gn_b=0.1 * torch.randn(H * DV, generator=g),
                w_o=r(DM, H * DV), w_1=r(FF, DM), b_1=(0.1 * torch.randn(FF, generator=g)).to(BF), w_2=r(DM, FF),
                b_2=(0.1 * torch.randn(DM, generator=g)).to(BF), w_out=r(V, DM))


def _heads(t, d):
    """[B, L, H d] -> [B, H, L, d]"""
    return t.unflatten(-1, (H, d)).transpose(1, 2).contiguous()


def _rows(t):
    return t.transpose(1, 2).flatten(2).contiguous()


def _train_own(w, ids, d_logits):
    """Logits and the gradients of every weight: x + MSR(x), then y + FFN(y), logits in fp32."""
    gamma, theta = multiscale_gamma(H), rotation_theta(DK)
    x = rn.embedding(ids, w["table"], scale=DM ** 0.5)
    q, k = (_heads(rn.linear(x, w[n]), DK) for n in ("w_q", "w_k"))
    v, gate = _heads(rn.linear(x, w["w_v"]), DV), rn.linear(x, w["w_g"])
    o, _ = rn.retention_chunkwise(q, k, v, gamma, CHUNK, theta)
    n = rn.group_norm_gate(o, gate, w["gn_w"], w["gn_b"])
    y = rn.linear(n, w["w_o"], residual=x)
    f, pre = rn.linear(y, w["w_1"], w["b_1"], activation="gelu", pre_out=True)
    z = rn.linear(f, w["w_2"], w["b_2"], residual=y)
    logits = rn.linear(z, w["w_out"], out_dtype=F32)
    g = {}
    d = rn.linear_bwd(z, w["w_out"], d_logits)
    g["w_out"], dz = d.dw, d.dx
    d = rn.linear_bwd(f, w["w_2"], dz, dbias=True)
    g["w_2"], g["b_2"] = d.dw, d.dbias
    d = rn.linear_bwd(y, w["w_1"], d.dx, pre, "gelu", dbias=True)
    g["w_1"], g["b_1"], dy = d.dw, d.dbias, dz + d.dx
    d = rn.linear_bwd(n, w["w_o"], dy)
    g["w_o"] = d.dw
    d = rn.group_norm_gate_bwd(o, d.dx, gate, w["gn_w"], w["gn_b"])
    g["gn_w"], g["gn_b"] = d.dweight, d.dbias
    dq, dk, dv = rn.retention_chunkwise_bwd(q, k, v, d.dx, gamma, CHUNK, theta)
    dx = dy
    for name, t in (("w_q", _rows(dq)), ("w_k", _rows(dk)), ("w_v", _rows(dv)), ("w_g", d.dgate)):
        e = rn.linear_bwd(x, w[name], t)
        g[name] = e.dw
        dx = dx + e.dx
    g["table"] = rn.embedding_bwd(ids, dx, V, scale=DM ** 0.5)
    return logits, g


def _train_plain(w, ids, d_logits):
    w = {k: t.double().requires_grad_() for k, t in w.items()}
    gamma, theta = (torch.as_tensor(t).double() for t in (multiscale_gamma(H), rotation_theta(DK)))
    inside = (ids >= 0)[..., None]
    x = torch.where(inside, w["table"][ids.clamp(min=0).long()] * DM ** 0.5, 0.0)
    p = torch.arange(L).double()
    turn = torch.polar(torch.ones(L, DK // 2, dtype=torch.float64), p[:, None] * theta)
    rot = lambda t: torch.view_as_real(torch.view_as_complex(t.unflatten(-1, (DK // 2, 2)).contiguous()) * turn).flatten(-2)  # noqa: E731
    q, k = (rot((x @ w[n].T).unflatten(-1, (H, DK)).transpose(1, 2)) for n in ("w_q", "w_k"))
    v = (x @ w["w_v"].T).unflatten(-1, (H, DV)).transpose(1, 2)
    far = p[:, None] - p
    decay = torch.where(far >= 0, gamma[:, None, None] ** far.clamp(min=0), 0.0)
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2).contiguous()) * decay, v)
    n = torch.nn.functional.layer_norm(o, (DV,), eps=1e-5).transpose(1, 2).flatten(2) * w["gn_w"] + w["gn_b"]
    y = (n * torch.nn.functional.silu(x @ w["w_g"].T)) @ w["w_o"].T + x
    z = torch.nn.functional.gelu(y @ w["w_1"].T + w["b_1"]) @ w["w_2"].T + w["b_2"] + y
    logits = z @ w["w_out"].T
    names = list(w)
    return logits.detach(), dict(zip(names, torch.autograd.grad((logits * d_logits.double()).sum(), [w[k] for k in names])))


def test_training_step_of_a_model():
    """bf16 hand-offs between the operators: some 16 on a gradient's longest way, each within a quarter of
    a percent of the whole (2^-8 of an element at most, 2^-9.8 in the mean), doubled where a norm's
    differences lose a bit: 16 * 2 * 2^-9.8 = 3.6 %."""
    w = _weights(1)
    ids = torch.randint(0, V, (B, L), generator=_gen(2), dtype=I32)
    ids[0, 60:], ids[1, 3] = -1, 5
    d_logits = torch.randn(B, L, V, generator=_gen(3)).to(BF)
    logits, g = _train_own({k: t.to(DEV) for k, t in w.items()}, ids.to(DEV), d_logits.to(DEV))
    want, gw = _train_plain(w, ids, d_logits)
    assert set(g) == set(gw)
    for name, got, ref in [("logits", logits, want), *((k, g[k], gw[k]) for k in gw)]:
        off = ((got.cpu().double() - ref).norm() / ref.norm()).item()
        print(f"{name}: {off:.2e}")
        assert off <= 3.6e-2, name


def test_training_step_in_a_graph():
    """Forward and gradients captured while eager results of the same weights live, replayed on new
    inputs with eager work between: every replay has the eager calls' bits."""
    w = {k: t.to(DEV) for k, t in _weights(4).items()}
    ids = torch.randint(0, V, (B, L), generator=_gen(5), dtype=I32).to(DEV)
    d_logits = torch.randn(B, L, V, generator=_gen(6)).to(BF).to(DEV)
    kept = _train_own(w, ids, d_logits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _train_own(w, ids, d_logits)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits, grads = _train_own(w, ids, d_logits)
    for i in range(4):
        ids.copy_(torch.randint(-1, V, (B, L), generator=_gen(7 + i), dtype=I32))
        d_logits.copy_(torch.randn(B, L, V, generator=_gen(17 + i)))
        graph.replay()
        torch.cuda.synchronize()
        _ = (kept[0].float() * 2).sum()
        want, gw = _train_own(w, ids, d_logits)
        torch.cuda.synchronize()
        same = {"logits": torch.equal(logits, want), **{k: torch.equal(grads[k], gw[k]) for k in gw}}
        assert all(same.values()), same


# -------------------------------------------------------------------------------- generation
class Search:
    """A beam search of R requests, W beams, over one gated layer and an FFN, all state on the GPU."""

    def __init__(self, seed, R, W, dm=128, heads=2, dk=64, dv=128, ff=192, vocab=300):
        g = _gen(seed)
        r = lambda n, k: (torch.randn(n, k, generator=g) * k ** -0.5).to(BF).to(DEV)  # noqa: E731
        self.R, self.W, self.dims, self.eos, self.scale = R, W, (heads, dk, dv), 2, dm ** 0.5
        self.table = (torch.randn(vocab, dm, generator=g) * dm ** -0.5).to(BF).to(DEV)
        self.layer = [r(n, dm) for n in (heads * dk, heads * dk, heads * dv, heads * dv)] + [r(dm, heads * dv)]
        self.w_1, self.w_2 = r(ff, dm), r(dm, ff)
        self.b_1 = (0.1 * torch.randn(ff, generator=g)).to(BF).to(DEV)
        self.w_out = 4 * r(vocab, dm)
        self.gamma, self.theta = multiscale_gamma(heads), rotation_theta(dk)
        self.state = torch.zeros(R * W, heads, dk, dv, device=DEV)
        self.pos = torch.zeros(R * W, dtype=I32, device=DEV)
        self.tokens = torch.randint(3, vocab, (R, 1), generator=g, dtype=I32).expand(R, W).contiguous().to(DEV)
        self.scores = torch.full((R, W), -math.inf, device=DEV)
        self.scores[:, 0] = 0.0
        self.ended = torch.zeros(R, W, dtype=torch.bool, device=DEV)
        self.history = torch.zeros(R, W, 12, dtype=I32, device=DEV)
        self.at = torch.zeros(1, dtype=torch.long, device=DEV)

    def everything(self):
        return [self.state, self.pos, self.tokens, self.scores, self.ended, self.history, self.at]

    def logits(self):
        x = rn.embedding(self.tokens.reshape(-1), self.table, scale=self.scale)
        y = x + rn.msr_layer_step(x, *self.layer, self.state, self.pos, *self.dims, self.gamma, self.theta)
        z = rn.linear(rn.linear(y, self.w_1, self.b_1, activation="gelu"), self.w_2, residual=y)
        return rn.linear(z, self.w_out, out_dtype=F32).reshape(self.R, self.W, -1)

    def step(self):
        pick = rn.beam_select(self.logits(), self.scores, self.W, ended=self.ended, eos=self.eos)
        rn.beam_reorder([self.state, self.pos, self.history, self.ended], pick.parents)
        self._after(pick.tokens, pick.scores)

    def _after(self, tokens, scores):
        self.tokens.copy_(tokens)
        self.scores.copy_(scores)
        self.ended.logical_or_(tokens == self.eos)
        self.history.scatter_(2, self.at.expand(self.R, self.W, 1), tokens[..., None])
        self.at += 1

    def plain_step(self):
        """The same with torch's own selection and indexing."""
        z = self.logits().double()
        V = z.shape[-1]
        z = torch.log_softmax(z, -1)
        only = torch.where(torch.arange(V, device=DEV) == self.eos, 0.0, -math.inf).double()
        z = torch.where(self.ended[..., None], only, z) + self.scores.double()[..., None]
        v, i = z.reshape(self.R, -1).sort(dim=-1, descending=True, stable=True)
        v, i = v[:, :self.W], i[:, :self.W]
        row = (torch.arange(self.R, device=DEV)[:, None] * self.W + i // V).reshape(-1)
        for t in (self.state, self.pos, self.history, self.ended):
            t.copy_(t.reshape(self.R * self.W, -1)[row].reshape(t.shape))
        self._after((i % V).to(I32), v.float())


def test_beam_search():
    """Tokens, parents (by way of the states) and positions are those of a search with torch's sort and
    indexing over the same layers, and the scores to fp32's roundings."""
    own, plain = Search(30, 3, 4), Search(30, 3, 4)
    plain.layer = own.layer  # the layer's products depend on whether its weights lie one behind the other
    for step in range(10):
        own.step()
        plain.plain_step()
        assert torch.equal(own.history, plain.history), step
        same = [torch.equal(getattr(own, k), getattr(plain, k)) for k in ("state", "pos", "ended")]
        assert all(same), (step, same)
        torch.testing.assert_close(own.scores, plain.scores, rtol=2e-6, atol=2e-5)
        plain.scores.copy_(own.scores)
    assert own.ended.any() or own.at.item() == 10


def test_beam_searches_in_two_captured_graphs():
    """Two searches' steps, each in its own graph, replayed in turn with eager work between."""
    runs = [(Search(40 + i, 2, 3), Search(40 + i, 2, 3)) for i in range(2)]
    for a, b in runs:
        b.layer = a.layer
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Search(50, 2, 3).step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for a, _ in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.step()
        graphs.append(g)
    for _ in range(6):
        for g, (a, b) in zip(graphs, runs):
            g.replay()
            b.step()
            torch.cuda.synchronize()
            same = [torch.equal(x, y) for x, y in zip(a.everything(), b.everything())]
            assert all(same), same


# ------------------------------------------------------------------------------ streams, offsets
def _calls(seed, stream=None):
    """One call of each operator on inputs made from the seed."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, to=BF: torch.randn(*s, generator=g, device=DEV).to(to)  # noqa: E731
    ids = torch.randint(-1, 50, (900,), generator=g, device=DEV, dtype=I32)
    table, rows = r(50, 200), r(900, 200)
    x, gate, d_o, w, b = r(2, 3, 150, 72), r(2, 150, 216), r(2, 150, 216), r(216, to=F32), r(216, to=F32)
    lx, lw, lb, ld = r(300, 1024), r(88, 1024), r(88), r(300, 88)
    z, cum = r(4, 3, 5000), r(4, 3, to=F32)
    states, parents = [r(4, 3, 1000), r(4, 3, 17)], torch.randint(0, 3, (4, 3), generator=g, device=DEV, dtype=I32)
    torch.cuda.synchronize()
    kw = dict(stream=stream)

    def run():
        n = rn.group_norm_gate_bwd(x, d_o, gate, w, b, **kw)
        p, pre = rn.linear(lx, lw, lb, "gelu", pre_out=True, **kw)
        q = rn.linear_bwd(lx, lw, ld, pre, "gelu", dbias=True, **kw)
        return [rn.embedding(ids, table, 2.0, **kw), rn.embedding_bwd(ids, rows, 50, **kw), rn.group_norm_gate(x, gate, w, b, **kw), *n,
                p, pre, *q, rn.linear(lx[:3], lw, lb, "silu", **kw), *rn.beam_select(z, cum, 6, **kw),
                *rn.beam_reorder([t.clone() for t in states] if stream is None else states, parents, **kw)]
    return run


def test_calls_on_another_stream():
    want = _calls(60)()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = _calls(60, side)()
    side.synchronize()
    same = [torch.equal(a, b) for a, b in zip(got, want)]
    assert len(got) == len(want) and all(same), same


def test_two_calls_at_once():
    want = [_calls(70 + i)() for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = [_calls(70 + i, s) for i, s in enumerate(streams)]
    got = [run() for run in runs]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        same = [torch.equal(a, b) for a, b in zip(g, w)]
        assert all(same), same


def test_the_same_bits_again():
    a, b = _calls(80)(), _calls(80)()
    same = [torch.equal(x, y) for x, y in zip(a, b)]
    assert all(same), same


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in a tensor: the last rows equal those of a call on them alone."""
    g = torch.Generator(device=DEV).manual_seed(90)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=BF)  # noqa: E731
    n, d, cut = (1 << 20) + 37, 2056, 1 << 20
    x = r(n, d)
    # norm: token-major heads of 257 channels
    heads = x.reshape(1, n, 8, 257).transpose(1, 2)
    out = rn.group_norm_gate(heads, x.reshape(1, n, d))
    assert torch.equal(out[:, cut:], rn.group_norm_gate(heads[:, :, cut:], x.reshape(1, n, d)[:, cut:]))
    a = rn.group_norm_gate_bwd(heads, out, x.reshape(1, n, d))
    b = rn.group_norm_gate_bwd(heads[:, :, cut:], out[:, cut:], x.reshape(1, n, d)[:, cut:])
    assert torch.equal(a.dx[:, :, cut:], b.dx) and torch.equal(a.dgate[:, cut:], b.dgate)
    del a, b
    # linear: the rows of x and of out; the bits do not depend on the tile for one k tile
    w = r(2056, 64)
    y = rn.linear(x[:, :64], w)
    assert torch.equal(y[cut:], rn.linear(x[cut:, :64], w))
    e = rn.linear_bwd(x[:, :64], w, out[0], dw=False)
    torch.testing.assert_close(e.dx[cut:].float(), rn.linear_bwd(x[cut:, :64], w, out[0, cut:], dw=False).dx.float(), rtol=2 ** -7,
                               atol=2 ** -7 * 0.1)
    del y, e, out
    # embedding: a table and an output of that size
    ids = torch.cat([torch.arange(n - 300, n, device=DEV), torch.randint(0, n, (n - 300,), generator=g, device=DEV)]).to(I32)
    out = rn.embedding(ids, x, 0.5)
    assert torch.equal(out[:300], x[n - 300:] * 0.5) and torch.equal(out[cut:], x[ids[cut:].long()] * 0.5)
    dt = rn.embedding_bwd(ids, out, n)
    at = torch.nonzero(ids == n - 1)[:, 0]
    want = out[at].double().sum(0)
    assert ((dt[n - 1].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all()
    del dt, out
    # reorder: beams of 1.4 GB
    s = x[:n // 3 * 3].reshape(1, 3, -1)
    last = s[0, :, -1000:].clone()
    rn.beam_reorder(s, torch.tensor([[2, 0, 1]], dtype=I32, device=DEV))
    assert torch.equal(s[0, :, -1000:], last[[2, 0, 1]])
