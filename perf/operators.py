"""Cases that measure the recurrent-layer operators next to retention: the selective state space
scan (prompts, training, single tokens), its short causal convolution, and the products with 4-bit
weights that feed and leave such a layer, also inside the decode step of the gated retention layer.

Notation: u, delta [B, L, D]; A [D, N]; Bm, Cm [B, L, G, N] (channel d reads group d // (D / G)).
  dt = softplus(delta + bias);  h_t = exp(dt_t A) h_{t-1} + dt_t u_t Bm_t;  y_t = Cm_t . h_t + D u_t
  out = y silu(z)
  conv:  c_t = silu(bias + sum_j w_j x_{t-K+1+j})
  w4:    out = x W^T, W[n, k] = (q[n, k] - zero[n, k // g]) scale[n, k // g]
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the last tokens of a prompt, where the call's latency counts
        _scan("scan tail", 1, 17, 2048, 16, 1, "bf16"),
        # a batch of prompts of different lengths, two groups of B and C, fp32
        _scan("scan padded prompts", 8, 777, 1000, 8, 2, "f32", ragged=True),
        # one long document
        _scan("scan long prompt", 1, 32768, 2048, 16, 1, "bf16"),
        # gradients of a small fp32 run, truncated in time: it starts from a state and hands one on
        _scan("scan gradients fp32", 2, 500, 512, 16, 1, "f32", train=True, carried=True),
        # gradients of one layer at the training length
        _scan("scan gradients", 2, 4096, 4096, 16, 1, "bf16", train=True),
        # the next piece of a batch of prompts of different lengths, continued from a state
        _conv("conv padded prompts", 8, 333, 1000, 4, "f32", ragged=True),
        # forward and gradients of one layer at the training length
        _conv("conv training", 4, 4096, 4096, 4, "bf16", train=True),
        # one token of one sequence: convolution, then scan
        _step("step one sequence", 1, 2048, 16, 1, 4, "bf16"),
        # one token of a full batch
        _step("step batch", 128, 4096, 16, 1, 4, "bf16"),
        # the input projection of one token, and the output projection of a batch
        _w4("w4 one token", 1, 2048, 12288, 128, False, "f32"),
        _w4("w4 batch", 64, 4096, 2048, 64, True, "bf16"),
        # a decode step of the gated retention layer with 4-bit weights
        {"name": "retention step w4", "kind": "msr", "B": 16, "d_model": 2048, "H": 8, "dk": 256, "dv": 512, "g": 128,
         "zeros": True},
    ]


def _scan(name, B, L, D, N, G, dtype, ragged=False, train=False, carried=False):
    return {"name": name, "kind": "scan", "B": B, "L": L, "D": D, "N": N, "G": G, "dtype": dtype, "ragged": ragged,
            "train": train, "carried": carried}


def _conv(name, B, L, D, K, dtype, ragged=False, train=False):
    return {"name": name, "kind": "conv", "B": B, "L": L, "D": D, "K": K, "dtype": dtype, "ragged": ragged,
            "train": train}


def _step(name, B, D, N, G, K, dtype):
    return {"name": name, "kind": "step", "B": B, "D": D, "N": N, "G": G, "K": K, "dtype": dtype}


def _w4(name, M, K, N, g, zeros, out):
    return {"name": name, "kind": "w4", "M": M, "K": K, "N": N, "g": g, "zeros": zeros, "out": out}


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["scan", "scan", "grad", "grad", "conv", "conv", "step", "w4", "w4", "msr"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    G = rng.choice([1, 1, 2, 4])
    if kind in ("scan", "grad"):
        N = rng.choice([4, 8, 16, 16, 16, 24, 32, 64])
        B, D = log(1, 16), G * log(64 // G, 4096 // G)
        L = log(1, min(32768 if kind == "scan" else 4096, (1 << 29) // (B * D * N)))
        c = _scan("", B, L, D, N, G, dtype, rng.random() < 0.4, kind == "grad", rng.random() < 0.4)
    elif kind == "conv":
        B, D = log(1, 16), log(64, 4096)
        L = log(1, min(32768, (1 << 26) // (B * D)))
        c = _conv("", B, L, D, rng.choice([2, 3, 4, 4, 4]), dtype, rng.random() < 0.4, rng.random() < 0.6)
    elif kind == "step":
        c = _step("", log(1, 128), G * log(64 // G, 4096 // G), rng.choice([8, 16, 16, 32, 64]), G,
                  rng.choice([2, 3, 4, 4]), dtype)
    elif kind == "w4":
        g = rng.choice([32, 64, 128])
        c = _w4("", log(1, 96), g * log(2, 8192 // g), 8 * log(8, 2048), g, rng.random() < 0.5,
                rng.choice(["bf16", "f32"]))
    else:
        dk = rng.choice([64, 128, 256])
        H = rng.choice([2, 4, 8])
        c = {"kind": "msr", "B": log(1, 64), "d_model": 128 * rng.randint(2, 16), "H": H, "dk": dk, "dv": 2 * dk,
             "g": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5}
    c.pop("name", None)
    return c


# --------------------------------------------------------------------------------------- inputs
class _State:
    pass


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    s = _State()
    s.c = case
    s.graph = None
    if case["kind"] in ("scan", "step"):
        B, D, N, G, t = case["B"], case["D"], case["N"], case["G"], _DT[case["dtype"]]
        rows = (B, case["L"]) if case["kind"] == "scan" else (B,)
        # x and z leave one projection side by side, delta another, B and C a third: rows with a stride
        xz = randn(*rows, 2 * D).to(t)
        bc = randn(*rows, 2 * G * N).to(t)
        s.u, s.z = xz[..., :D], xz[..., D:]
        s.Bm, s.Cm = (bc[..., i * G * N:(i + 1) * G * N].unflatten(-1, (G, N)) for i in (0, 1))
        s.delta = (0.5 * randn(*rows, D)).to(t)
        # time steps of 1e-3 to 1e-1, spread over their logarithm, through the inverse of softplus
        dt = torch.exp(rand(D) * math.log(100.0) + math.log(1e-3))
        s.bias = dt + torch.log(-torch.expm1(-dt))
        s.A = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(0.1 * randn(D, N))
        s.D = 1.0 + 0.1 * randn(D)
        s.h = randn(B, D, N) if case["kind"] == "step" or case["carried"] else None
    if case["kind"] in ("scan", "conv"):
        B, L, D, t = case["B"], case["L"], case["D"], _DT[case["dtype"]]
        s.lengths, s.out = None, None
        if case["ragged"]:
            s.lengths = torch.randint(0, L + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
            s.lengths[B // 2] = L
            s.out = torch.zeros(B, L, D, device=dev, dtype=t)  # rows behind a sequence's end stay as they are
        s.d_o = randn(B, L, D).to(t) if case["train"] else None
        if case["kind"] == "scan":
            s.d_h = randn(B, D, N) if case["train"] and case["carried"] else None
    if case["kind"] in ("conv", "step"):
        B, D, K, t = case["B"], case["D"], case["K"], _DT[case["dtype"]]
        s.x = randn(B, case["L"], D).to(t) if case["kind"] == "conv" else randn(B, D).to(t)
        s.w, s.cbias = (randn(D, K) / math.sqrt(K)).to(t), (0.1 * randn(D)).to(t)
        s.cs = randn(B, K - 1, D).to(t)
    if case["kind"] == "w4":
        s.x = randn(case["M"], case["K"]).to(torch.bfloat16)
        s.w = _packed(gen, dev, case["N"], case["K"], case["g"], case["zeros"])
    if case["kind"] == "msr":
        B, dm, H, dk, dv = (case[k] for k in ("B", "d_model", "H", "dk", "dv"))
        s.x = randn(B, dm).to(torch.bfloat16)
        s.w_in = _packed(gen, dev, 2 * H * dk + 2 * H * dv, dm, case["g"], case["zeros"])
        s.w_o = _packed(gen, dev, dm, H * dv, case["g"], case["zeros"])
        s.h = randn(B, H, dk, dv)
        s.pos = torch.randint(0, 4096, (B,), generator=gen, device=dev, dtype=torch.int32)
        s.gamma = torch.tensor([1.0 - 2.0 ** (-5 - h) for h in range(H)])
        s.theta = torch.tensor([10000.0 ** (-2.0 * i / dk) for i in range(dk // 2)])
    return s


def _packed(gen, dev, N, K, g, zeros):
    """(bytes [N, K/2], scales [N, K/g] bf16, zero points [N, K/g] or None): weights of about 0.02."""
    q = torch.randint(0, 256, (N, K // 2), generator=gen, device=dev, dtype=torch.uint8)
    scale = (0.004 * (0.5 + torch.rand(N, K // g, generator=gen, device=dev))).to(torch.bfloat16)
    zero = torch.randint(6, 11, (N, K // g), generator=gen, device=dev, dtype=torch.uint8) if zeros else None
    return q, scale, zero


# ------------------------------------------------------------------------------------------ run
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import retentive_network_scale_amd as rn

    c = s.c
    if c["kind"] == "scan" and not c["train"]:
        out, h = rn.selective_scan(s.u, s.delta, s.A, s.Bm, s.Cm, D=s.D, z=s.z, delta_bias=s.bias, delta_softplus=True,
                                   lengths=s.lengths, state_in=s.h, state_out=True, out=s.out)
        return {"out": out, "state": h}
    if c["kind"] == "scan":
        g = rn.selective_scan_bwd(s.u, s.delta, s.A, s.Bm, s.Cm, s.d_o, D=s.D, z=s.z, delta_bias=s.bias,
                                  delta_softplus=True, lengths=s.lengths, state_in=s.h, d_state_out=s.d_h)
        return {"du": g.du, "ddelta": g.ddelta, "dA": g.dA, "dB": g.dB, "dC": g.dC, "dD": g.dD, "dz": g.dz,
                "dbias": g.ddelta_bias, "dstate": g.d_state_in}
    if c["kind"] == "conv":
        out, cs = rn.causal_conv1d(s.x, s.w, s.cbias, lengths=s.lengths, state_in=s.cs, state_out=True, out=s.out)
        if not c["train"]:
            return {"out": out, "state": cs}
        g = rn.causal_conv1d_bwd(s.x, s.w, s.d_o, s.cbias, lengths=s.lengths, state_in=s.cs)
        return {"out": out, "state": cs, "dx": g.dx, "dw": g.dw, "dbias": g.dbias, "dstate": g.d_state_in}
    if c["kind"] == "step":
        u = rn.causal_conv1d_step(s.x, s.cs, s.w, s.cbias)
        out = rn.selective_scan_step(u, s.delta, s.A, s.Bm, s.Cm, s.h, D=s.D, z=s.z, delta_bias=s.bias,
                                     delta_softplus=True)
        return {"conv": u, "out": out, "conv_state": s.cs, "state": s.h}
    if c["kind"] == "w4":
        return {"out": rn.linear_w4(s.x, *s.w, out_dtype=_DT[c["out"]])}
    y = rn.msr_layer_step_w4(s.x, s.w_in, s.w_o, s.h, s.pos, c["H"], c["dk"], c["dv"], s.gamma, s.theta)
    return {"out": y, "state": s.h, "pos": s.pos}


# ---------------------------------------------------------------------------- the plain forms
def _run_plain(s):
    k = s.c["kind"]
    return {"scan": _plain_scan, "conv": _plain_conv, "step": _plain_step, "w4": _plain_w4, "msr": _plain_msr}[k](s)


def _linear_recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0, along dim 1, by doubling."""
    n, L = 1, a.shape[1]
    while n < L:
        b = torch.cat([b[:, :n], torch.addcmul(b[:, n:], a[:, n:], b[:, :-n])], 1)
        if 2 * n < L:
            a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _valid(s):
    """[B, L, 1]: rows before their sequence's end."""
    L = s.c["L"]
    return None if s.lengths is None else (torch.arange(L, device=s.lengths.device) < s.lengths[:, None])[..., None]


def _plain_scan(s):
    D, G, t = s.c["D"], s.c["G"], _DT[s.c["dtype"]]
    u, z, Bm, Cm = (v.float() for v in (s.u, s.z, s.Bm, s.Cm))
    Bm, Cm = (v.repeat_interleave(D // G, 2) if G > 1 else v for v in (Bm, Cm))
    pre = s.delta.float() + s.bias
    dt, valid = _softplus(pre), _valid(s)
    if valid is not None:
        dt = torch.where(valid, dt, 0)
    a = torch.exp(dt[..., None] * s.A)
    b = (dt * u)[..., None] * Bm
    if s.h is not None:
        b[:, 0] += a[:, 0] * s.h
    h = _linear_recurrence(a, b)
    y = (h * Cm).sum(-1) + s.D * u
    if not s.c["train"]:
        out = (y * _silu(z)).to(t)
        return {"out": out if valid is None else torch.where(valid, out, s.out), "state": h[:, -1]}
    sig = torch.sigmoid(z)
    d_o = s.d_o.float() if valid is None else torch.where(valid, s.d_o.float(), 0)
    dy, dz = d_o * z * sig, d_o * y * sig * (1 + z * (1 - sig))
    # the adjoint runs against time: g_t = Cm_t dy_t + a_{t+1} g_{t+1}
    g = dy[..., None] * Cm
    if s.d_h is not None:
        g[:, -1] += s.d_h
    back = torch.cat([torch.ones_like(a[:, :1]), a[:, 1:].flip(1)], 1)
    g = _linear_recurrence(back, g.flip(1)).flip(1)
    first = torch.zeros_like(h[:, :1]) if s.h is None else s.h[:, None]
    ga = g * a * torch.cat([first, h[:, :-1]], 1)  # the gradient of dt A
    gB = (g * Bm).sum(-1)
    du = gB * dt + dy * s.D
    ddelta = ((ga * s.A).sum(-1) + gB * u) * torch.sigmoid(pre)
    if valid is not None:
        ddelta, du = torch.where(valid, ddelta, 0), torch.where(valid, du, 0)
    per = (s.c["B"], s.c["L"], G, D // G, s.c["N"])
    dB, dC = ((v.unsqueeze(-1) * w).reshape(per).sum(3) for v, w in ((dt * u, g), (dy, h)))
    return {"du": du.to(t), "ddelta": ddelta.to(t), "dA": (ga * dt[..., None]).sum((0, 1)), "dB": dB.to(t),
            "dC": dC.to(t), "dD": (dy * u).sum((0, 1)), "dz": dz.to(t), "dbias": ddelta.sum((0, 1)),
            "dstate": None if s.h is None else a[:, 0] * g[:, 0]}


def _plain_conv(s):
    B, L, K, t = s.c["B"], s.c["L"], s.c["K"], _DT[s.c["dtype"]]
    x, w = torch.cat([s.cs, s.x], 1).float(), s.w.float()
    taps = x.unfold(1, K, 1)  # [B, L, D, K]
    pre = (taps * w).sum(-1) + s.cbias.float()
    out, valid = _silu(pre).to(t), _valid(s)
    end = torch.full((B,), L, device=x.device) if valid is None else s.lengths.long()
    at = end[:, None] + torch.arange(K - 1, device=x.device)
    state = torch.gather(x, 1, at[..., None].expand(-1, -1, x.shape[2])).to(t)
    out = out if valid is None else torch.where(valid, out, s.out)
    if not s.c["train"]:
        return {"out": out, "state": state}
    sig = torch.sigmoid(pre)
    g = s.d_o.float() * sig * (1 + pre * (1 - sig))
    if valid is not None:
        g = torch.where(valid, g, 0)
    late = torch.nn.functional.pad(g, (0, 0, K - 1, K - 1)).unfold(1, K, 1)  # g_{t-K+1..t} of each padded input
    dx = (late * w.flip(1)).sum(-1)
    return {"out": out, "state": state, "dx": dx[:, K - 1:].to(t), "dw": (g[..., None] * taps).sum((0, 1)),
            "dbias": g.sum((0, 1)), "dstate": dx[:, :K - 1].to(t)}


def _plain_step(s):
    D, G, t = s.c["D"], s.c["G"], _DT[s.c["dtype"]]
    x = torch.cat([s.cs, s.x[:, None]], 1)
    u = _silu((x.float() * s.w.float().T).sum(1) + s.cbias.float()).to(t)
    s.cs.copy_(x[:, 1:])
    Bm, Cm = (v.float().repeat_interleave(D // G, 1) for v in (s.Bm, s.Cm))
    dt, z, uf = _softplus(s.delta.float() + s.bias), s.z.float(), u.float()
    s.h.copy_(torch.exp(dt[..., None] * s.A) * s.h + (dt * uf)[..., None] * Bm)
    out = ((s.h * Cm).sum(-1) + s.D * uf) * _silu(z)
    return {"conv": u, "out": out.to(t), "conv_state": s.cs, "state": s.h}


def _weights(w, to):
    q, scale, zero = w
    n = torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], scale.shape[1], -1).to(to)
    return ((n - (8 if zero is None else zero.to(to)[..., None])) * scale.to(to)[..., None]).flatten(1)


def _plain_w4(s):
    return {"out": (s.x.float() @ _weights(s.w, torch.float32).T).to(_DT[s.c["out"]])}


def _msr(s, to):
    """The decode step of the gated retention layer in `to`: (y, the new state)."""
    B, H, dk, dv = (s.c[k] for k in ("B", "H", "dk", "dv"))
    p = s.x.to(to) @ _weights(s.w_in, to).T
    q, k, v, gate = p.split([H * dk, H * dk, H * dv, H * dv], 1)
    angle = s.pos.double()[:, None] * s.theta.to(s.pos.device).double()
    cos, sin = (f(angle).to(to)[:, None] for f in (torch.cos, torch.sin))
    q, k = (r.reshape(B, H, dk // 2, 2) for r in (q, k))
    q, k = (torch.stack([r[..., 0] * cos - r[..., 1] * sin, r[..., 0] * sin + r[..., 1] * cos], -1).flatten(2)
            for r in (q, k))
    gamma = s.gamma.to(s.pos.device).to(to)[:, None, None]
    h = gamma * s.h.to(to) + k[..., None] * v.reshape(B, H, 1, dv)
    o = (q[..., None] * h).sum(2)
    o = o - o.mean(-1, keepdim=True)
    o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-5)
    return (o.flatten(1) * _silu(gate)) @ _weights(s.w_o, to).T, h


def _plain_msr(s):
    y, h = _msr(s, torch.float32)
    s.h.copy_(h)
    s.pos += 1
    return {"out": y.to(torch.bfloat16), "state": s.h, "pos": s.pos}


# ------------------------------------------------------------------------------ 64-bit results
def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "conv": _exact_conv, "step": _exact_step, "w4": _exact_w4, "msr": _exact_msr}[
        case["kind"]](s)


def _f64(*ts):
    return tuple(None if t is None else t.double().clone() for t in ts)


def _token(h, u, delta, Bm, Cm, A, D, bias, z):
    """One token of the scan: (new state, gated output); the definition."""
    rep = u.shape[-1] // Bm.shape[-2]
    Bm, Cm = (v.repeat_interleave(rep, -2) for v in (Bm, Cm))
    dt = torch.nn.functional.softplus(delta + bias, threshold=50)
    h = torch.exp(dt.unsqueeze(-1) * A) * h + (dt * u).unsqueeze(-1) * Bm
    y = torch.linalg.vecdot(h, Cm) + D * u
    return h, y * z * torch.sigmoid(z)


def _exact_scan(s):
    B, L, D, N = (s.c[k] for k in ("B", "L", "D", "N"))
    train = s.c["train"]
    names = ("u", "delta", "A", "Bm", "Cm", "D", "z", "bias")
    v = dict(zip(names, _f64(*(getattr(s, n) for n in names))))
    h0 = torch.zeros(B, D, N, dtype=torch.float64, device=s.u.device) if s.h is None else s.h.double().clone()
    if train:
        for t in (*v.values(), h0):
            t.requires_grad_()
    with torch.set_grad_enabled(train):
        h, outs = h0, []
        rows = {n: v[n].unbind(1) for n in ("u", "delta", "Bm", "Cm", "z")}  # one node for all rows
        for t in range(L):
            new, o = _token(h, rows["u"][t], rows["delta"][t], rows["Bm"][t], rows["Cm"][t], v["A"], v["D"], v["bias"],
                            rows["z"][t])
            h = new if s.lengths is None else torch.where((t < s.lengths)[:, None, None], new, h)
            outs.append(o)
        out = torch.stack(outs, 1)
        live = None if s.lengths is None else (torch.arange(L, device=h.device) < s.lengths[:, None])[..., None]
        if not train:
            return {"out": out if live is None else torch.where(live, out, 0.0), "state": h}
        weight = s.d_o.double() if live is None else torch.where(live, s.d_o.double(), 0.0)
        loss = (out * weight).sum()
        if s.d_h is not None:
            loss = loss + (h * s.d_h.double()).sum()
        g = torch.autograd.grad(loss, [*v.values(), h0])
    g = dict(zip((*names, "h0"), g))
    return {"du": g["u"], "ddelta": g["delta"], "dA": g["A"], "dB": g["Bm"], "dC": g["Cm"], "dD": g["D"], "dz": g["z"],
            "dbias": g["bias"], "dstate": None if s.h is None else g["h0"]}


def _exact_conv(s):
    B, L, D, K = (s.c[k] for k in ("B", "L", "D", "K"))
    x, w, bias, cs = _f64(s.x, s.w, s.cbias, s.cs)
    leaves = [x, w, bias, cs]
    train = s.c["train"]
    for t in leaves:
        t.requires_grad_(train)
    with torch.set_grad_enabled(train):
        padded = torch.cat([cs, x], 1)
        pre = bias + sum(w[:, j] * padded[:, j:j + L] for j in range(K))
        out = pre * torch.sigmoid(pre)
    ends = [L] * B if s.lengths is None else s.lengths.tolist()
    state = torch.stack([padded[b, e:e + K - 1] for b, e in enumerate(ends)]).detach()
    live = torch.ones(B, L, 1, dtype=torch.bool, device=x.device)
    for b, e in enumerate(ends):
        live[b, e:] = False
    got = {"out": torch.where(live, out.detach(), 0.0), "state": state}
    if train:
        g = torch.autograd.grad((out * torch.where(live, s.d_o.double(), 0.0)).sum(), leaves)
        got |= {"dx": g[0], "dw": g[1], "dbias": g[2], "dstate": g[3]}
    return got


def _exact_step(s):
    x, w, bias, cs = _f64(s.x, s.w, s.cbias, s.cs)
    pre = bias + torch.einsum("bkd,dk->bd", cs, w[:, :-1]) + x * w[:, -1]
    c = pre * torch.sigmoid(pre)
    # the scan reads the convolution's output as it is handed on, in the inputs' type
    u = c.to(_DT[s.c["dtype"]]).double()
    h, o = _token(*_f64(s.h), u, *_f64(s.delta, s.Bm, s.Cm, s.A, s.D, s.bias, s.z))
    return {"conv": c, "out": o, "conv_state": torch.cat([cs[:, 1:], x[:, None]], 1), "state": h}


def _dense(w):
    q, scale, zero = w
    N, K = q.shape[0], 2 * q.shape[1]
    full = torch.empty(N, K, dtype=torch.float64, device=q.device)
    full[:, 0::2] = (q % 16).double()
    full[:, 1::2] = torch.div(q, 16, rounding_mode="floor").double()
    g = K // scale.shape[1]
    full -= 8.0 if zero is None else zero.double().repeat_interleave(g, 1)
    return full.mul_(scale.double().repeat_interleave(g, 1))


def _exact_w4(s):
    return {"out": torch.mm(s.x.double(), _dense(s.w).t())}


def _exact_msr(s):
    B, H, dk, dv = (s.c[k] for k in ("B", "H", "dk", "dv"))
    p = torch.mm(s.x.double(), _dense(s.w_in).t())
    q, k = (torch.view_as_complex(p[:, i * H * dk:(i + 1) * H * dk].reshape(B, H, dk // 2, 2).contiguous())
            for i in (0, 1))
    turn = torch.polar(torch.ones(B, 1, dk // 2, dtype=torch.float64, device=p.device),
                       (s.pos.double()[:, None] * s.theta.double().to(p.device))[:, None])
    q, k = (torch.view_as_real(r * turn).reshape(B, H, dk) for r in (q, k))
    v, gate = p[:, 2 * H * dk:].reshape(B, 2, H, dv).unbind(1)
    h = s.h.double() * s.gamma.double().to(p.device)[:, None, None]
    for b in range(B):
        h[b] += k[b][:, :, None] * v[b][:, None, :]
    o = torch.stack([(q[b][:, :, None] * h[b]).sum(1) for b in range(B)])
    o = torch.nn.functional.layer_norm(o, (dv,), eps=1e-5)
    return {"out": torch.mm((o * gate * torch.sigmoid(gate)).reshape(B, H * dv), _dense(s.w_o).t()), "state": h,
            "pos": s.pos + 1}


# ----------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["kind"] == "w4":
        b, f = _w4_work(c["M"], c["N"], c["K"], c["g"], c["zeros"])
        return {"bytes": b + 2 * c["M"] * c["K"] + c["M"] * c["N"] * (4 if c["out"] == "f32" else 2), "flops": f}
    if c["kind"] == "msr":
        B, dm, H, dk, dv = (c[k] for k in ("B", "d_model", "H", "dk", "dv"))
        b1, f1 = _w4_work(B, 2 * H * dk + 2 * H * dv, dm, c["g"], c["zeros"])
        b2, f2 = _w4_work(B, dm, H * dv, c["g"], c["zeros"])
        return {"bytes": b1 + b2 + 4 * B * dm + 8 * B * H * dk * dv + 8 * B, "flops": f1 + f2 + 5 * B * H * dk * dv}
    e, B, D, L = (2 if c["dtype"] == "bf16" else 4), c["B"], c["D"], c.get("L", 1)
    rows = B * L * D
    if c["kind"] == "conv":
        K = c["K"]
        b = e * (2 * rows + 2 * B * (K - 1) * D + D * (K + 1))
        f = rows * (2 * K + 5)
        if c["train"]:
            b += e * (3 * rows + 2 * B * (K - 1) * D) + 4 * D * (K + 1)
            f += rows * (6 * K + 12)
        return {"bytes": b, "flops": f}
    N, G = c["N"], c["G"]
    if c["kind"] == "step":
        K = c["K"]
        return {"bytes": e * (5 * rows + 2 * B * G * N + 2 * B * (K - 1) * D + D * (K + 1)) + 8 * B * D * N
                + 4 * D * (N + 2), "flops": B * D * (7 * N + 2 * K + 25)}
    states = 4 * B * D * N
    b = e * (4 * rows + 2 * B * L * G * N) + 4 * D * (N + 2) + states * (1 + c["carried"])
    f = rows * (7 * N + 20)
    if c["train"]:
        b += e * (3 * rows + 2 * B * L * G * N) + 4 * D * (N + 2) + states * (2 * c["carried"] - 1)
        f = rows * (20 * N + 45)
    return {"bytes": b, "flops": f}


def _w4_work(M, N, K, g, zeros):
    """Bytes of the weights and operations of x W^T."""
    return N * K // 2 + N * (K // g) * (3 if zeros else 2), 2 * M * N * K
