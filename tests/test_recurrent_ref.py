"""The plain 64-bit forms that the recurrent-layer GPU tests compare with, checked here:
gradients against autograd and against differences, the scan against its closed form."""
import pytest
import torch

from tests import _recurrent_ref as ref


def _inputs(bt, L, d, n, G, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(u=r(bt, L, d), delta=0.5 * r(bt, L, d), A=-torch.rand(d, n, generator=g, dtype=torch.float64) * 2,
                B=r(bt, L, G, n), C=r(bt, L, G, n), D=r(d), z=r(bt, L, d), bias=0.3 * r(d), h0=r(bt, d, n))


def test_scan_closed_form():
    """h_t = sum_s exp(A sum_{s<r<=t} dt_r) dt_s u_s B_s for constant dt, written out."""
    bt, L, d, n = 1, 9, 3, 4
    v = _inputs(bt, L, d, n, 1, 1)
    dt = torch.full((bt, L, d), 0.3, dtype=torch.float64)
    out, last, y, hs, _ = ref.scan(v["u"], dt, v["A"], v["B"], v["C"])
    for t in range(L):
        h = sum(torch.exp(v["A"] * 0.3 * (t - s)) * (0.3 * v["u"][0, s])[:, None] * v["B"][0, s] for s in range(t + 1))
        torch.testing.assert_close(hs[0, t], h, rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(last[0], hs[0, -1])
    torch.testing.assert_close(out, y)


def _loss_scan(v, w_out, w_state, softplus_on, lengths, gated):
    """The scan again, differentiable."""
    bt, L, d = v["u"].shape
    rep = d // v["B"].shape[2]
    dt = v["delta"] + v["bias"]
    dt = torch.nn.functional.softplus(dt) if softplus_on else dt
    loss = 0.0
    for b in range(bt):
        h = v["h0"][b]
        for t in range(L if lengths is None else lengths[b]):
            Bt, Ct = (v[k][b, t].repeat_interleave(rep, 0) for k in "BC")
            h = torch.exp(dt[b, t][:, None] * v["A"]) * h + (dt[b, t] * v["u"][b, t])[:, None] * Bt
            y = (h * Ct).sum(1) + v["D"] * v["u"][b, t]
            if gated:
                y = y * torch.nn.functional.silu(v["z"][b, t])
            loss = loss + (y * w_out[b, t]).sum()
        loss = loss + (h * w_state[b]).sum()
    return loss


@pytest.mark.parametrize("softplus_on,lengths,gated,G", [(True, None, True, 1), (False, [3, 0], False, 2),
                                                         (True, [5, 7], True, 3)])
def test_scan_gradients_are_autograds_and_differences(softplus_on, lengths, gated, G):
    bt, L, d, n = 2, 7, 6, 3
    v = _inputs(bt, L, d, n, G, 2)
    g = torch.Generator().manual_seed(3)
    w_out = torch.randn(bt, L, d, generator=g, dtype=torch.float64)
    w_state = torch.randn(bt, d, n, generator=g, dtype=torch.float64)
    got = ref.scan_bwd(v["u"], v["delta"], v["A"], v["B"], v["C"], w_out, v["D"], v["z"] if gated else None, v["bias"],
                       softplus_on, lengths, v["h0"], w_state)
    names = dict(u="du", delta="ddelta", A="dA", B="dB", C="dC", D="dD", z="dz", bias="dbias", h0="dh0")
    for t in v.values():
        t.requires_grad_()
    loss = _loss_scan(v, w_out, w_state, softplus_on, lengths, gated)
    want = torch.autograd.grad(loss, list(v.values()), allow_unused=True)
    for (k, t), a in zip(v.items(), want):
        if a is not None:
            torch.testing.assert_close(got[names[k]], a, rtol=1e-10, atol=1e-10, msg=lambda m: f"{k}: {m}")
    with torch.no_grad():  # a central difference along a random direction of every input
        for k, t in v.items():
            if k == "z" and not gated:
                continue
            way = torch.randn(t.shape, generator=g, dtype=torch.float64)
            f = [_loss_scan({**v, k: t + s * 1e-5 * way}, w_out, w_state, softplus_on, lengths, gated) for s in (1, -1)]
            diff = (f[0] - f[1]).item() / 2e-5
            assert abs(diff - (got[names[k]] * way).sum().item()) <= 1e-6 * (1 + abs(diff)), k


@pytest.mark.parametrize("silu,lengths,k", [(True, None, 4), (False, [0, 5], 2), (True, [2, 1], 4)])
def test_conv_gradients_are_autograds(silu, lengths, k):
    bt, L, d = 2, 6, 5
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, bias, s0, d_o, dsT = r(bt, L, d), r(d, k), r(d), r(bt, k - 1, d), r(bt, L, d), r(bt, k - 1, d)
    got = ref.conv_bwd(x, w, d_o, bias, silu, lengths, s0, dsT)
    leaves = [t.requires_grad_() for t in (x, w, bias, s0)]
    p = torch.cat([s0, x], 1)
    pre = torch.nn.functional.conv1d(p.transpose(1, 2), w[:, None], bias, groups=d).transpose(1, 2)
    out = torch.nn.functional.silu(pre) if silu else pre
    loss = 0.0
    for b in range(bt):
        n = L if lengths is None else lengths[b]
        loss = loss + (out[b, :n] * d_o[b, :n]).sum() + (p[b, n:n + k - 1] * dsT[b]).sum()
    for name, a in zip(("dx", "dw", "dbias", "ds0"), torch.autograd.grad(loss, leaves)):
        torch.testing.assert_close(got[name], a, rtol=1e-10, atol=1e-10, msg=lambda m: f"{name}: {m}")
    fwd = ref.conv(x, w, bias, silu, lengths, s0)[0]
    for b in range(bt):
        n = L if lengths is None else lengths[b]
        torch.testing.assert_close(fwd[b, :n], out[b, :n].detach(), rtol=1e-12, atol=1e-12)
