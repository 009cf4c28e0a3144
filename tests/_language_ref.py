"""Plain 64-bit forms of the operators of include/language.h, on the CPU, and with each result the
sum of the absolute terms that its tolerance is counted in (tests/_recurrent_ref.assert_near)."""
import math

import torch

U = 2.0 ** -24  # half a step of fp32


def f64(t):
    return None if t is None else t.detach().cpu().double()


# --------------------------------------------------------------------------------- embedding
def embedding(ids, table, scale):
    ids, table = ids.cpu().long(), f64(table)
    inside = (ids >= 0) & (ids < table.shape[0])
    rows = table[ids.clamp(0, table.shape[0] - 1)] * scale
    return torch.where(inside[..., None], rows, 0.0)


def embedding_bwd(ids, d_o, V, scale):
    """(dtable, the same sum of absolute values, the most tokens of one id)."""
    d = f64(d_o).reshape(-1, d_o.shape[-1])
    out, mag, count = torch.zeros(V, d.shape[1], dtype=torch.float64), torch.zeros(V, d.shape[1], dtype=torch.float64), [0] * V
    for t, i in enumerate(ids.cpu().reshape(-1).tolist()):
        if 0 <= i < V:
            out[i] += scale * d[t]
            mag[i] += abs(scale) * d[t].abs()
            count[i] += 1
    return out, mag, max(count)


# -------------------------------------------------------------------------------------- norm
def silu(x):
    return x / (1 + torch.exp(-x))


def silu_slope(x):
    s = 1 / (1 + torch.exp(-x))
    return s * (1 + x * (1 - s))


def _live(B, L, lengths):
    ends = torch.full((B,), L) if lengths is None else torch.tensor(lengths).clamp(0, L)
    return (torch.arange(L) < ends[:, None])[..., None, None]  # [B, L, 1, 1]


def norm(x, gate, weight, bias, use_silu, eps, lengths=None):
    """Rows [B, L, H, W] of everything: dict of out and the terms that the gradients need.  `e`: xh is off
    by at most (W + 8) U e, from the mean (W U max|x|), the variance and its root."""
    B, H, L, W = x.shape
    live = _live(B, L, lengths)
    x = torch.where(live, f64(x).transpose(1, 2), 0.0)
    w = torch.ones(H, W, dtype=torch.float64) if weight is None else f64(weight).reshape(H, W)
    b = torch.zeros(H, W, dtype=torch.float64) if bias is None else f64(bias).reshape(H, W)
    d = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    xh = d * r
    big = r * x.abs().amax(-1, keepdim=True)
    e = big * (1 + xh.abs()) + xh.abs()
    n = w * xh + b
    v = dict(live=live, xh=xh, r=r, e=e, n=n, w=w, big=big, n_mag=w.abs() * e + b.abs() + n.abs())
    if gate is not None:
        g = torch.where(live, f64(gate).reshape(B, L, H, W), 0.0)
        a, s = (silu(g), silu_slope(g)) if use_silu else (g, torch.ones_like(g))
        v |= dict(a=a, s=s, s_mag=(1 + g.abs()) if use_silu else s, out=n * a, mag=v["n_mag"] * a.abs())
    elif use_silu:
        v |= dict(out=silu(n), mag=1.1 * v["n_mag"])
    else:
        v |= dict(out=n, mag=v["n_mag"])
    return v


def norm_bwd(x, d_o, gate, weight, bias, use_silu, eps, lengths=None):
    """name -> (gradient, magnitude): dx [B, H, L, W], dgate [B, L, H W], dweight, dbias [H W]."""
    v = norm(x, gate, weight, bias, use_silu, eps, lengths)
    B, H, L, W = x.shape
    d = torch.where(v["live"], f64(d_o).reshape(B, L, H, W), 0.0)
    got = {}
    if gate is not None:
        dn, dn_mag = d * v["a"], d.abs() * v["a"].abs()
        got["dgate"] = (d * v["n"] * v["s"], d.abs() * v["n_mag"] * v["s_mag"])
    elif use_silu:
        dn = d * silu_slope(v["n"])
        dn_mag = d.abs() * (1 + v["n"].abs() + 0.5 * v["n_mag"])
    else:
        dn, dn_mag = d, d.abs()
    xh, r, e, w = v["xh"], v["r"], v["e"], v["w"]
    p, p_mag = w * dn, w.abs() * dn_mag
    m1, m2 = p.mean(-1, keepdim=True), (p * xh).mean(-1, keepdim=True)
    m1_mag, m2_mag = p_mag.mean(-1, keepdim=True), (p_mag * (xh.abs() + e)).mean(-1, keepdim=True)
    dx = r * (p - m1 - xh * m2)
    dx_mag = r * (p_mag + m1_mag + xh.abs() * m2_mag + e * m2.abs()) + dx.abs() * (v["big"] + 1)
    got["dx"] = (dx.transpose(1, 2), dx_mag.transpose(1, 2))
    got["dweight"] = ((dn * xh).sum((0, 1)), (dn_mag * (xh.abs() + e)).sum((0, 1)))
    got["dbias"] = (dn.sum((0, 1)), dn_mag.sum((0, 1)))
    shape = dict(dgate=(B, L, H * W), dx=(B, H, L, W), dweight=(H * W,), dbias=(H * W,))
    return {k: tuple(t.reshape(shape[k]) for t in pair) for k, pair in got.items()}


# ------------------------------------------------------------------------------------ linear
def act(z, name):
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return silu(z) if name == "silu" else z


def act_slope(z, name):
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return silu_slope(z) if name == "silu" else torch.ones_like(z)


def linear(x, w, bias, activation, residual):
    """(out, its magnitude, pre, its magnitude); x [M, K]."""
    x, w, bias, residual = f64(x), f64(w), f64(bias), f64(residual)
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + bias, mag + bias.abs()
    out, out_mag = act(z, activation), 1.2 * mag
    if residual is not None:
        out, out_mag = out + residual, out_mag + residual.abs()
    return out, out_mag, z, mag


def linear_bwd(x, w, d_o, pre, activation, slope_roundings):
    """name -> (gradient, magnitude, a tolerance beside the roundings).  dz is rounded to bf16 here as the
    operator does; where its error (slope_roundings U of its terms) could turn the rounding, the
    difference between the two neighbours is that last tolerance's."""
    x, w, d = f64(x), f64(w), f64(d_o)
    if activation is None:
        dz, terms = d, d.abs()
    else:
        z = f64(pre)
        dz = d * act_slope(z, activation)
        terms = d.abs() * (1 + z.abs() * (torch.exp(-0.5 * z * z) if activation == "gelu" else 1))
    to = lambda t: t.float().to(torch.bfloat16).double()  # noqa: E731
    off = slope_roundings * U * terms
    r, turn = to(dz), to(dz + off) - to(dz - off)
    return dict(dx=(r @ w, r.abs() @ w.abs(), turn @ w.abs()), dw=(r.T @ x, r.abs().T @ x.abs(), turn.T @ x.abs()),
                dbias=(dz.sum(0), terms.sum(0), 0.0))


# ------------------------------------------------------------------------------------- beams
def beam_select(logits, scores, K, ended=None, eos=0):
    """(tokens, parents, scores) and the smallest difference between scores, not equal, of the K + 1 best."""
    z, cum = f64(logits), f64(scores)
    B, W, V = z.shape
    tokens, parents, best, gap = [], [], [], math.inf
    for b in range(B):
        every = []
        for w in range(W):
            c = cum[b, w].item()
            row = [-math.inf] * V
            if math.isfinite(c):
                if ended is not None and bool(ended[b, w]):
                    row[eos] = c
                else:
                    top = z[b, w].max().item()
                    if math.isfinite(top) and not bool(torch.isnan(z[b, w]).any()):
                        lse = top + math.log(torch.exp(z[b, w] - top).sum().item())
                        row = [c + (v - lse) for v in z[b, w].tolist()]
            every += [(-s, w * V + v) for v, s in enumerate(row)]
        every.sort()
        tokens.append([i % V for _, i in every[:K]])
        parents.append([i // V for _, i in every[:K]])
        best.append([-s for s, _ in every[:K]])
        for (s, _), (t, _) in zip(every[:K], every[1:K + 1]):
            if s != t and math.isfinite(t):
                gap = min(gap, t - s)
    return torch.tensor(tokens), torch.tensor(parents), torch.tensor(best, dtype=torch.float64), gap
