"""The plain 64-bit forms that the GPU tests of include/language.h compare with, checked here:
gradients against autograd and against differences, the selection against torch's sort."""
import math

import pytest
import torch

from tests import _language_ref as ref


def _r(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)


def _differences(f, leaves, grads, r):
    for t, g in zip(leaves, grads):
        way = r(*t.shape)
        with torch.no_grad():
            at = [f(*(v + s * 1e-5 * way if v is t else v for v in leaves)) for s in (1, -1)]
        diff = ((at[0] - at[1]) / 2e-5).item()
        assert abs(diff - (g * way).sum().item()) <= 1e-6 * (1 + abs(diff))


@pytest.mark.parametrize("gated,use_silu,lengths", [(True, True, None), (True, False, [3, 0]), (False, True, [5, 2]),
                                                    (False, False, None)])
def test_norm_gradients(gated, use_silu, lengths):
    r = _r(1)
    B, H, L, W = 2, 3, 5, 6
    x, g, w, b, d_o = r(B, H, L, W), r(B, L, H * W), 1 + 0.2 * r(H * W), r(H * W), r(B, L, H * W)

    def loss(x, g, w, b):
        n = torch.nn.functional.layer_norm(x, (W,), eps=1e-3).permute(0, 2, 1, 3).reshape(B, L, H * W) * w + b
        a = torch.nn.functional.silu if use_silu else lambda t: t
        y = n * a(g) if gated else a(n)
        live = ref._live(B, L, lengths)[..., 0]
        return (torch.where(live, y, 0.0) * d_o).sum()

    leaves = [t.requires_grad_() for t in (x, g, w, b)]
    want = torch.autograd.grad(loss(*leaves), leaves, allow_unused=True)
    got = ref.norm_bwd(x, d_o, g if gated else None, w, b, use_silu, 1e-3, lengths)
    for name, a in zip(("dx", "dgate", "dweight", "dbias"), want):
        if a is not None and name in got:
            torch.testing.assert_close(got[name][0], a, rtol=1e-10, atol=1e-10)
            assert (got[name][1] >= a.abs() - 1e-9).all()
    _differences(loss, leaves, [got[n][0] if n in got else torch.zeros(B, L, H * W) for n in
                                ("dx", "dgate", "dweight", "dbias")], r)


@pytest.mark.parametrize("activation", [None, "gelu", "silu"])
def test_linear_gradients(activation):
    r = _r(2)
    M, N, K = 5, 4, 6
    x, w, b, res, d_o = r(M, K), r(N, K), r(N), r(M, N), r(M, N)
    d_o = d_o.bfloat16().double()
    fn = {"gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu, None: lambda t: t}[activation]

    def loss(x, w, b):
        return ((fn(x @ w.T + b) + res) * d_o).sum()

    leaves = [t.requires_grad_() for t in (x, w, b)]
    want = torch.autograd.grad(loss(*leaves), leaves)
    out, _, pre, _ = ref.linear(x, w, b, activation, res)
    torch.testing.assert_close((out * d_o).sum(), loss(x, w, b).detach(), rtol=1e-10, atol=1e-10)
    got = ref.linear_bwd(x, w, d_o, pre, activation, 0)
    torch.testing.assert_close(got["dbias"][0], want[2], rtol=1e-10, atol=1e-10)
    _differences(loss, leaves, want, r)
    # the rounding of dz, at most half a step of bf16 for each term
    for name, a, other in (("dx", want[0], w.abs()), ("dw", want[1], None)):
        most = got["dx"][1] if name == "dx" else got["dw"][1]
        assert ((got[name][0] - a).abs() <= 2.0 ** -7 * most + 1e-12).all()


def test_embedding_gradient():
    r = _r(3)
    table = r(5, 3).requires_grad_()
    ids = torch.tensor([[1, 4, -1], [1, 9, 0]])
    d_o = r(2, 3, 3)
    inside = (ids >= 0) & (ids < 5)
    y = torch.where(inside[..., None], table[ids.clamp(0, 4)] * 1.5, 0.0)
    torch.testing.assert_close(ref.embedding(ids, table, 1.5), y.detach())
    want, = torch.autograd.grad((y * d_o).sum(), table)
    got, _, most = ref.embedding_bwd(ids, d_o, 5, 1.5)
    torch.testing.assert_close(got, want)
    assert most == 2


def test_selection_is_the_sort():
    r = _r(4)
    B, W, V, K = 3, 4, 7, 6
    z, cum = r(B, W, V), r(B, W)
    ended = torch.zeros(B, W, dtype=torch.bool)
    ended[1, 2] = True
    s = cum[..., None] + torch.log_softmax(z, -1)
    s[1, 2] = -math.inf
    s[1, 2, 5] = cum[1, 2]
    v, i = s.reshape(B, -1).sort(dim=-1, descending=True, stable=True)
    tokens, parents, best, _ = ref.beam_select(z, cum, K, ended, 5)
    assert torch.equal(tokens, i[:, :K] % V) and torch.equal(parents, i[:, :K] // V)
    torch.testing.assert_close(best, v[:, :K])
