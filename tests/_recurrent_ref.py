"""Plain 64-bit forms of the recurrent-layer operators, token by token, on the CPU, and
the tolerances that the GPU results are held to.

Every form takes absolute=True: the same sums over the absolute values of their terms.
A result of fp32 arithmetic is off by at most (roundings on the longest path) * 2^-24
times that sum, and by half a step of its own type at the end; the counts stand at the
tests.
"""
import torch


def f64(t):
    return None if t is None else t.detach().cpu().double()


def _len(lengths, b, L):
    return L if lengths is None else min(max(int(lengths[b]), 0), L)


def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def scan(u, delta, A, B, C, D=None, z=None, bias=None, softplus_on=False, lengths=None, h0=None, absolute=False):
    """(out, final state, y before the gate, states [Bt, L, Dm, N], dt); rows behind an end are zero."""
    u, delta, A, B, C, D, z, bias, h0 = (f64(t) for t in (u, delta, A, B, C, D, z, bias, h0))
    bt, L, d = u.shape
    rep = d // B.shape[2]
    dt = delta + (0 if bias is None else bias)
    dt = softplus(dt) if softplus_on else dt
    gate = torch.ones_like(u) if z is None else z * torch.sigmoid(z)
    mag = torch.abs if absolute else (lambda t: t)
    y, out, hs = torch.zeros_like(u), torch.zeros_like(u), torch.zeros(bt, L, d, A.shape[1], dtype=torch.float64)
    last = torch.zeros(bt, d, A.shape[1], dtype=torch.float64)
    for b in range(bt):
        h = torch.zeros(d, A.shape[1], dtype=torch.float64) if h0 is None else mag(h0[b])
        for t in range(_len(lengths, b, L)):
            Bt, Ct = (mag(m[b, t]).repeat_interleave(rep, 0) for m in (B, C))
            h = torch.exp(dt[b, t][:, None] * A) * h + mag(dt[b, t] * u[b, t])[:, None] * Bt
            hs[b, t] = h
            y[b, t] = (h * Ct).sum(1) + (0 if D is None else mag(D * u[b, t]))
            out[b, t] = y[b, t] * mag(gate[b, t])
        last[b] = h
    return out, last, y, hs, dt


def scan_bwd(u, delta, A, B, C, d_o, D=None, z=None, bias=None, softplus_on=False, lengths=None, h0=None, dhT=None,
             absolute=False):
    """Gradients by the formulas of include/recurrent.h, as a dict."""
    _, _, y, hs, dt = scan(u, delta, A, B, C, D, z, bias, softplus_on, lengths, h0, absolute)
    pre = f64(delta) + (0 if bias is None else f64(bias))
    u, A, B, C, D, z, d_o, h0, dhT = (f64(t) for t in (u, A, B, C, D, z, d_o, h0, dhT))
    bt, L, d = u.shape
    n, G = A.shape[1], B.shape[2]
    rep = d // G
    mag = torch.abs if absolute else (lambda t: t)
    sg = None if z is None else torch.sigmoid(z)
    g_ = {k: torch.zeros(bt, L, d, dtype=torch.float64) for k in ("du", "ddelta", "dz")}
    g_ |= {k: torch.zeros(bt, L, G, n, dtype=torch.float64) for k in ("dB", "dC")}
    g_ |= {"dA": torch.zeros(d, n, dtype=torch.float64), "dD": torch.zeros(d, dtype=torch.float64),
           "dbias": torch.zeros(d, dtype=torch.float64), "dh0": torch.zeros(bt, d, n, dtype=torch.float64)}
    for b in range(bt):
        carry = torch.zeros(d, n, dtype=torch.float64) if dhT is None else mag(dhT[b])
        for t in reversed(range(_len(lengths, b, L))):
            dy = d_o[b, t] if z is None else d_o[b, t] * z[b, t] * sg[b, t]
            dy = mag(dy)
            if z is not None:
                # silu' = s + z s (1 - s), whose terms are rounded apart
                slope = sg[b, t] + mag(z[b, t]) * sg[b, t] * (1 - sg[b, t])
                g_["dz"][b, t] = mag(d_o[b, t]) * y[b, t] * slope
            Bt, Ct = (mag(m[b, t]).repeat_interleave(rep, 0) for m in (B, C))
            ut = mag(u[b, t])
            step = mag(dt[b, t])
            a = torch.exp(dt[b, t][:, None] * A)
            before = hs[b, t - 1] if t else (torch.zeros(d, n, dtype=torch.float64) if h0 is None else mag(h0[b]))
            g = Ct * dy[:, None] + carry
            carry = a * g
            w = carry * before
            gB = (g * Bt).sum(1)
            g_["du"][b, t] = step * gB + (0 if D is None else mag(D) * dy)
            slope = torch.sigmoid(pre[b, t]) if softplus_on else torch.ones(d, dtype=torch.float64)
            g_["ddelta"][b, t] = ((mag(A) * w).sum(1) + ut * gB) * slope
            g_["dA"] += step[:, None] * w
            g_["dB"][b, t] = (g * (step * ut)[:, None]).reshape(G, rep, n).sum(1)
            g_["dC"][b, t] = (hs[b, t] * dy[:, None]).reshape(G, rep, n).sum(1)
            g_["dD"] += dy * ut
            g_["dbias"] += g_["ddelta"][b, t]
        g_["dh0"][b] = carry
    return g_


def conv(x, w, bias=None, silu=True, lengths=None, s0=None, absolute=False):
    """(out, final state, sums before the activation, the padded inputs)."""
    x, w, bias, s0 = (f64(t) for t in (x, w, bias, s0))
    bt, L, d = x.shape
    k = w.shape[1]
    mag = torch.abs if absolute else (lambda t: t)
    front = torch.zeros(bt, k - 1, d, dtype=torch.float64) if s0 is None else s0
    p = torch.cat([front, x], 1)
    out, pre = torch.zeros_like(x), torch.zeros_like(x)
    state = torch.zeros(bt, k - 1, d, dtype=torch.float64)
    for b in range(bt):
        n = _len(lengths, b, L)
        for t in range(n):
            pre[b, t] = sum((mag(w[:, j] * p[b, t + j]) for j in range(k)), torch.zeros(d, dtype=torch.float64))
            pre[b, t] += 0 if bias is None else mag(bias)
            out[b, t] = pre[b, t] * torch.sigmoid(pre[b, t]) if silu else pre[b, t]
        state[b] = p[b, n:n + k - 1]
    return out, state, pre, p


def conv_bwd(x, w, d_o, bias=None, silu=True, lengths=None, s0=None, dsT=None, absolute=False):
    _, _, pre, p = conv(x, w, bias, silu, lengths, s0)
    w, d_o, dsT = (f64(t) for t in (w, d_o, dsT))
    bt, L, d = d_o.shape
    k = w.shape[1]
    mag = torch.abs if absolute else (lambda t: t)
    sg = torch.sigmoid(pre)
    g = mag(d_o) * (sg + mag(pre) * sg * (1 - sg) if absolute else sg + pre * sg * (1 - sg)) if silu else mag(d_o)
    dp, dw, db = torch.zeros_like(p), torch.zeros_like(w), torch.zeros(d, dtype=torch.float64)
    for b in range(bt):
        n = _len(lengths, b, L)
        if dsT is not None:
            dp[b, n:n + k - 1] += mag(dsT[b])
        for t in range(n):
            db += g[b, t]
            for j in range(k):
                dp[b, t + j] += mag(w[:, j]) * g[b, t]
                dw[:, j] += mag(p[b, t + j]) * g[b, t]
        dp[b, n + k - 1:] = 0
    return {"dx": dp[:, k - 1:], "dw": dw, "dbias": db, "ds0": dp[:, :k - 1]}


def w4_dense(q, scale, zero=None):
    """[N, K] of the packed weights, element by element."""
    q, scale = q.cpu(), f64(scale)
    n, k = q.shape[0], 2 * q.shape[1]
    g = k // scale.shape[1]
    w = torch.zeros(n, k, dtype=torch.float64)
    for i in range(k):
        nib = (q[:, i // 2].int() >> (4 * (i % 2))) & 15
        off = 8.0 if zero is None else zero.cpu()[:, i // g].double()
        w[:, i] = (nib.double() - off) * scale[:, i // g]
    return w


def assert_near(got, ref, mag, roundings, what):
    """|got - ref| <= half a step of got's type + roundings * 2^-24 * mag, everywhere."""
    assert got.dtype in (torch.float32, torch.bfloat16), got.dtype
    assert tuple(got.shape) == tuple(ref.shape), (what, got.shape, ref.shape)
    x = got.detach().cpu().double()
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny
    assert torch.isfinite(x).all(), f"{what}: not finite"
    off, most = (x - ref).abs(), half * ref.abs() + (1 + half) * roundings * 2.0 ** -24 * mag + tiny
    worst = (off / most).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times its tolerance ({(off > most).sum().item()} of {off.numel()} values)"
    return worst
