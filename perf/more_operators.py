"""Cases that measure the operators around the layers of a retention language model: the scaled embedding
and its gradient, the GroupNorm with its swish gate, the products with bias, activation and residual, the
selection of beams, and the reordering of the beams' recurrent states.

  embedding   out_t = scale table[id_t], zero for an id outside the table;  dtable_v = scale sum_{t: id_t = v} d_o_t
  norm        xh = (x - mean) / sqrt(var + eps) over a head's channels, n = w xh + b, out = n silu(gate)
  linear      z = x W^T + b, out = act(z) + residual;  dz = d_o act'(z), dx = dz W, dW = dz^T x, db = sum dz
  select      the K best of scores[b, w] + log_softmax(logits[b, w])[v] over w and v, ties to the lowest (w, v)
  reorder     state[b, w] <- state[b, parents[b, w]], in place
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the tokens of one decode step of 16 requests with 4 beams
        _embed("embedding decode step", 64, 32000, 2048, "bf16"),
        # lookup and gradient of a training batch, 4 x 4096 tokens
        _embed("embedding training", 16384, 32000, 2048, "bf16", train=True),
        # the retention heads' norm and gate for a padded batch of prompts, fp32, a width of no power of two
        _norm("norm padded prompts", 3, 5, 333, 100, "f32", ragged=True),
        # forward and gradients of one layer at the training length
        _norm("norm training", 4, 8, 4096, 512, "bf16", affine=True, train=True),
        # the FFN's first product for one token
        _linear("linear one token", 1, 2048, 4096, "gelu", True, False, "bf16"),
        # sizes that no tile divides: an output projection onto a residual stream kept in fp32
        _linear("linear ragged", 777, 1000, 2302, None, True, True, "f32"),
        # the FFN's first product for a training batch, 4 x 4096 tokens
        _linear("linear training batch", 16384, 2048, 4096, "gelu", True, False, "bf16"),
        # its gradients
        _linear("linear gradients", 16384, 2048, 4096, "gelu", True, False, "bf16", train=True),
        # the first step of a search: one beam, its four best tokens
        _select("select first step", 1, 1, 32000, 4, "f32"),
        # a step of a full batch, some beams at their end
        _select("select batch", 64, 8, 32000, 8, "bf16", ended=True),
        # the states of one request with four beams, two layers
        _reorder("reorder one request", 1, 4, 2, 4, 64, 128),
        # the states of a batch, two layers of 1 MiB a beam
        _reorder("reorder batch", 32, 4, 2, 8, 128, 256),
    ]


def _embed(name, n, V, D, dtype, train=False, masked=False):
    return {"name": name, "kind": "embed", "n": n, "V": V, "D": D, "dtype": dtype, "train": train, "masked": masked}


def _norm(name, B, H, L, W, dtype, affine=False, ragged=False, train=False):
    return {"name": name, "kind": "norm", "B": B, "H": H, "L": L, "W": W, "dtype": dtype, "affine": affine,
            "ragged": ragged, "train": train}


def _linear(name, M, K, N, act, bias, residual, out, train=False):
    return {"name": name, "kind": "linear", "M": M, "K": K, "N": N, "act": act, "bias": bias, "residual": residual,
            "out": out, "train": train}


def _select(name, B, W, V, K, dtype, ended=False):
    return {"name": name, "kind": "select", "B": B, "W": W, "V": V, "K": K, "dtype": dtype, "ended": ended}


def _reorder(name, B, W, layers, H, dk, dv):
    return {"name": name, "kind": "reorder", "B": B, "W": W, "layers": layers, "H": H, "dk": dk, "dv": dv}


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["embed", "embed", "norm", "norm", "linear", "linear", "linear", "select", "select", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "embed":
        train = rng.random() < 0.6
        V, D = log(100, 32000), log(32, 2048)
        c = _embed("", log(1, 16384), V, D, dtype, train, rng.random() < 0.4)
    elif kind == "norm":
        H, W = rng.choice([1, 2, 3, 4, 8, 16]), log(16, 512)
        B = log(1, 16)
        L = log(1, min(4096, (1 << 26) // (B * H * W)))
        c = _norm("", B, H, L, W, dtype, rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.5)
    elif kind == "linear":
        train = rng.random() < 0.4
        K, N = log(32, 4096), log(32, 8192)
        if rng.random() < 0.5:
            K, N = 64 * max(1, K // 64), 64 * max(1, N // 64)
        M = log(1, min(16384, (1 << 37) // (K * N)))
        c = _linear("", M, K, N, rng.choice([None, "gelu", "silu"]), rng.random() < 0.6,
                    not train and rng.random() < 0.4, rng.choice(["bf16", "bf16", "f32"]) if not train else "bf16", train)
    elif kind == "select":
        W = rng.choice([1, 2, 3, 4, 5, 8, 16])
        V = log(64, 65536)
        K = rng.randint(1, min(32, 2 * W))
        B = log(1, min(64, max(1, (1 << 24) // (W * V))))
        c = _select("", B, W, V, K, dtype, rng.random() < 0.4)
    else:
        H, dk = rng.choice([1, 2, 4, 8]), rng.choice([32, 64, 100, 128, 256])
        dv = rng.choice([dk, 2 * dk])
        W = rng.choice([2, 3, 4, 5, 8, 16])
        layers = rng.randint(1, 4)
        B = log(1, min(64, (1 << 26) // (H * dk * dv * W * layers)))
        c = _reorder("", B, W, layers, H, dk, dv)
    c.pop("name")
    return c


# --------------------------------------------------------------------------------------- inputs
class _State:
    pass


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, to=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(to)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    s, c = _State(), case
    s.c = case
    t = _DT[case.get("dtype", "bf16")]
    if c["kind"] == "embed":
        # ids with the frequencies of words, 1 / rank; masked: padding, id -1
        s.ids = torch.exp(rand(c["n"]) * math.log(c["V"] + 1)).sub(1).floor().clamp(0, c["V"] - 1).to(torch.int32)
        if c["masked"]:
            s.ids[rand(c["n"]) < 0.2] = -1
        s.table = randn(c["V"], c["D"], to=t)
        s.table *= c["D"] ** -0.5
        s.scale = c["D"] ** 0.5
        s.d_o = randn(c["n"], c["D"], to=t) if c["train"] else None
    if c["kind"] == "norm":
        B, H, L, W = (c[k] for k in ("B", "H", "L", "W"))
        # a retention's output, head-major, with heads of different sizes; the gate leaves a projection, token-major
        s.x = (randn(B, H, L, W) * (0.1 + rand(H, 1, 1)) + 0.1 * randn(H, 1, W)).to(t)
        s.gate = randn(B, L, H * W, to=t)
        s.w, s.b = (1 + 0.1 * randn(H * W), 0.1 * randn(H * W)) if c["affine"] else (None, None)
        s.d_o = randn(B, L, H * W, to=t) if c["train"] else None
        s.lengths, s.out = None, None
        if c["ragged"]:
            s.lengths = torch.randint(0, L + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
            s.lengths[B // 2] = L
            s.out = torch.zeros(B, L, H * W, device=dev, dtype=t)  # rows behind a sequence's end stay as they are
    if c["kind"] == "linear":
        M, K, N = (c[k] for k in ("M", "K", "N"))
        s.x = randn(M, K, to=t)
        s.w = (randn(N, K) * K ** -0.5).to(t)
        s.b = (0.1 * randn(N)).to(t) if c["bias"] else None
        s.r = randn(M, N, to=t) if c["residual"] else None
        s.pre, s.d_o = None, None
        if c["train"]:
            s.pre = randn(M, N, to=t) if c["act"] else None  # as the forward call left it
            s.d_o = randn(M, N, to=t)
    if c["kind"] == "select":
        B, W, V = (c[k] for k in ("B", "W", "V"))
        s.logits = (2.5 * randn(B, W, V)).to(t)
        s.scores = -20 * rand(B, W)
        s.ended = rand(B, W) < 0.2 if c["ended"] else None
        s.eos = 2
    if c["kind"] == "reorder":
        B, W = c["B"], c["W"]
        s.states = [randn(B, W, c["H"], c["dk"], c["dv"]) for _ in range(c["layers"])]
        s.parents = torch.randint(0, W, (B, W), generator=gen, device=dev, dtype=torch.int32)
    return s


# ------------------------------------------------------------------------------------------ run
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import retentive_network_scale_amd as rn

    c = s.c
    if c["kind"] == "embed":
        out = {"out": rn.embedding(s.ids, s.table, scale=s.scale)}
        if c["train"]:
            out["dtable"] = rn.embedding_bwd(s.ids, s.d_o, c["V"], scale=s.scale)
        return out
    if c["kind"] == "norm":
        out = {"out": rn.group_norm_gate(s.x, s.gate, s.w, s.b, lengths=s.lengths, out=s.out)}
        if c["train"]:
            g = rn.group_norm_gate_bwd(s.x, s.d_o, s.gate, s.w, s.b, lengths=s.lengths)
            out |= {"dx": g.dx, "dgate": g.dgate, "dweight": g.dweight, "dbias": g.dbias}
        return out
    if c["kind"] == "linear":
        if not c["train"]:
            return {"out": rn.linear(s.x, s.w, s.b, activation=c["act"], residual=s.r, out_dtype=_DT[c["out"]])}
        g = rn.linear_bwd(s.x, s.w, s.d_o, pre=s.pre, activation=c["act"], dbias=c["bias"])
        return {"dx": g.dx, "dw": g.dw, "dbias": g.dbias}
    if c["kind"] == "select":
        g = rn.beam_select(s.logits, s.scores, c["K"], ended=s.ended, eos=s.eos)
        return {"tokens": g.tokens, "parents": g.parents, "scores": g.scores}
    rn.beam_reorder(s.states, s.parents)
    return {"states": s.states}


# ---------------------------------------------------------------------------- the plain forms
def _run_plain(s):
    return {"embed": _plain_embed, "norm": _plain_norm, "linear": _plain_linear, "select": _plain_select,
            "reorder": _plain_reorder}[s.c["kind"]](s)


def _plain_embed(s):
    ids, valid = s.ids.long(), (s.ids >= 0)[:, None]
    rows = s.table[ids.clamp(min=0)].float() * s.scale
    out = {"out": torch.where(valid, rows, 0).to(s.table.dtype)}
    if s.c["train"]:
        g = torch.where(valid, s.d_o.float() * s.scale, 0)
        dt = torch.zeros(s.c["V"], s.c["D"], device=g.device).index_add_(0, ids.clamp(min=0), g)
        out["dtable"] = dt.to(s.d_o.dtype)
    return out


def _valid(s):
    L = s.c["L"]
    return None if s.lengths is None else (torch.arange(L, device=s.x.device) < s.lengths[:, None])[:, :, None, None]


def _plain_norm(s):
    B, H, L, W = (s.c[k] for k in ("B", "H", "L", "W"))
    t, valid = s.x.dtype, _valid(s)
    x = s.x.float().transpose(1, 2)  # [B, L, H, W], as all that follows
    g = s.gate.float().reshape(B, L, H, W)
    x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    xh = x * r
    n = xh if s.w is None else xh * s.w.reshape(H, W) + s.b.reshape(H, W)
    sig = 1 / (1 + torch.exp(-g))
    y = (n * g * sig).to(t)
    if valid is not None:
        y = torch.where(valid, y, s.out.reshape(B, L, H, W))
    out = {"out": y.reshape(B, L, H * W)}
    if not s.c["train"]:
        return out
    d_o = s.d_o.float().reshape(B, L, H, W)
    if valid is not None:
        d_o = torch.where(valid, d_o, 0)
    dn = d_o * g * sig
    dxh = dn if s.w is None else dn * s.w.reshape(H, W)
    dx = r * (dxh - dxh.mean(-1, keepdim=True) - xh * (dxh * xh).mean(-1, keepdim=True))
    dg = d_o * n * sig * (1 + g * (1 - sig))
    out |= {"dx": dx.transpose(1, 2).to(t), "dgate": dg.reshape(B, L, H * W).to(t), "dweight": None, "dbias": None}
    if s.w is not None:
        out |= {"dweight": (dn * xh).sum((0, 1)).reshape(-1), "dbias": dn.sum((0, 1)).reshape(-1)}
    return out


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _plain_linear(s):
    act, x, w = s.c["act"], s.x.float(), s.w.float()
    if not s.c["train"]:
        z = x @ w.T
        z = _act(z if s.b is None else z + s.b.float(), act)
        return {"out": (z if s.r is None else z + s.r.float()).to(_DT[s.c["out"]])}
    dz = s.d_o.float()
    if act == "gelu":
        z = s.pre.float()
        dz = dz * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    elif act == "silu":
        z = s.pre.float()
        sig = 1 / (1 + torch.exp(-z))
        dz = dz * sig * (1 + z * (1 - sig))
    return {"dx": (dz @ w).to(s.x.dtype), "dw": (dz.T @ x).to(s.w.dtype), "dbias": dz.sum(0) if s.c["bias"] else None}


def _plain_select(s):
    B, W, V = s.logits.shape
    K = s.c["K"]
    # scores next to each other decide which token is taken: in 64 bits
    z = s.logits.double()
    z = z - z.amax(-1, keepdim=True)
    z = z - torch.log(torch.exp(z).sum(-1, keepdim=True))
    if s.ended is not None:
        only = torch.where(torch.arange(V, device=z.device) == s.eos, 0.0, -math.inf).double()
        z = torch.where(s.ended[..., None], only, z)
    z = (s.scores.double()[..., None] + z).reshape(B, W * V)
    # of the values tied with the K-th best the lowest indices, then in descending order
    kth = z.topk(K, -1).values[:, -1:]
    above, tied = z > kth, z == kth
    tied = tied & (torch.cumsum(tied, -1) <= K - above.sum(-1, keepdim=True))
    flat = torch.where(above | tied, torch.arange(W * V, device=z.device), W * V).topk(K, -1, largest=False).values
    flat = flat.sort(-1).values
    best, order = z.gather(-1, flat).sort(dim=-1, descending=True, stable=True)
    flat = flat.gather(-1, order)
    return {"tokens": (flat % V).to(torch.int32), "parents": (flat // V).to(torch.int32), "scores": best.float()}


def _plain_reorder(s):
    b = torch.arange(s.c["B"], device=s.parents.device)[:, None]
    p = s.parents.long()
    for x in s.states:
        x.copy_(x[b, p])
    return {"states": s.states}


# ------------------------------------------------------------------------------ 64-bit results
def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "norm": _exact_norm, "linear": _exact_linear, "select": _exact_select,
            "reorder": _exact_reorder}[case["kind"]](s)


def _exact_embed(s):
    seen = s.ids >= 0
    out = torch.zeros(s.c["n"], s.c["D"], dtype=torch.float64, device=s.ids.device)
    out[seen] = torch.index_select(s.table, 0, s.ids[seen]).double() * s.scale
    if not s.c["train"]:
        return {"out": out}
    # tokens in the table's order, running sums, and their differences at the borders
    order = torch.argsort(s.ids, stable=True)
    sums = torch.cumsum(s.d_o[order].double() * s.scale, 0)
    sums = torch.cat([torch.zeros_like(sums[:1]), sums])
    ends = torch.searchsorted(s.ids[order].contiguous(), torch.arange(-1, s.c["V"], device=out.device), right=True)
    return {"out": out, "dtable": torch.diff(sums[ends], dim=0)}


def _exact_norm(s):
    B, H, L, W = (s.c[k] for k in ("B", "H", "L", "W"))
    train = s.c["train"]
    leaves = [s.x.double(), s.gate.double()]
    if s.w is not None:
        leaves += [s.w.double(), s.b.double()]
    for v in leaves:
        v.requires_grad_(train)
    live = torch.ones(B, L, dtype=torch.bool, device=s.x.device)
    if s.lengths is not None:
        for b, e in enumerate(s.lengths.tolist()):
            live[b, e:] = False
    with torch.set_grad_enabled(train):
        n = torch.nn.functional.layer_norm(leaves[0], (W,), eps=1e-5)
        n = n.permute(0, 2, 1, 3).reshape(B, L, H * W)
        if s.w is not None:
            n = n * leaves[2] + leaves[3]
        y = torch.where(live[..., None], n * leaves[1] * torch.sigmoid(leaves[1]), 0.0)
    out = {"out": y.detach()}
    if train:
        g = torch.autograd.grad((y * s.d_o.double()).sum(), leaves)
        out |= dict(zip(("dx", "dgate", "dweight", "dbias"), (*g, None, None)))
    return out


def _exact_linear(s):
    act = {"gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu, None: lambda z: z}[s.c["act"]]
    if not s.c["train"]:
        z = torch.nn.functional.linear(s.x.double(), s.w.double(), None if s.b is None else s.b.double())
        z = act(z)
        return {"out": z if s.r is None else z.add_(s.r.double())}
    dz = s.d_o.double()
    if s.pre is not None:
        z = s.pre.double().requires_grad_()
        dz, = torch.autograd.grad(act(z), z, dz)
    return {"dx": torch.mm(dz, s.w.double()), "dw": torch.mm(dz.t(), s.x.double()),
            "dbias": dz.sum(0) if s.c["bias"] else None}


def _exact_select(s):
    B, W, V = s.logits.shape
    K, got = s.c["K"], []
    for b in range(B):
        z = torch.log_softmax(s.logits[b].double(), -1)
        if s.ended is not None:
            z[s.ended[b]] = -math.inf
            z[s.ended[b], s.eos] = 0.0
        got.append((z + s.scores[b].double()[:, None]).flatten().sort(descending=True, stable=True))
    at = torch.stack([i[:K] for _, i in got])
    return {"tokens": (at % V).to(torch.int32), "parents": torch.div(at, V, rounding_mode="floor").to(torch.int32),
            "scores": torch.stack([v[:K] for v, _ in got])}


def _exact_reorder(s):
    pick = s.parents.tolist()
    return {"states": [torch.stack([x[b][row] for b, row in enumerate(pick)]).double() for x in s.states]}


# ----------------------------------------------------------------------------------------- work
def work(case):
    c = case
    e = 2 if c.get("dtype", "bf16") == "bf16" else 4
    if c["kind"] == "embed":
        n, V, D = c["n"], c["V"], c["D"]
        b, f = 4 * n + e * D * (min(n, V) + n), n * D
        return {"bytes": b + (e * D * (n + V) if c["train"] else 0), "flops": f * (3 if c["train"] else 1)}
    if c["kind"] == "norm":
        rows = c["B"] * c["H"] * c["L"] * c["W"]
        par = 8 * c["H"] * c["W"] if c["affine"] else 0
        return {"bytes": e * rows * (6 if c["train"] else 3) + par * (2 if c["train"] else 1),
                "flops": rows * (36 if c["train"] else 14)}
    if c["kind"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        if c["train"]:
            return {"bytes": 2 * (2 * M * K + 2 * N * K + M * N * (2 if c["act"] else 1)) + (4 * N if c["bias"] else 0),
                    "flops": 4 * M * N * K + (20 * M * N if c["act"] else 0)}
        b = 2 * (M * K + N * K) + M * N * ((2 if c["out"] == "bf16" else 4) + 2 * c["residual"]) + 2 * N * c["bias"]
        return {"bytes": b, "flops": 2 * M * N * K + (15 * M * N if c["act"] else 0)}
    if c["kind"] == "select":
        B, W, V, K = (c[k] for k in ("B", "W", "V", "K"))
        return {"bytes": e * B * W * V + 4 * B * W + 12 * B * K, "flops": 4 * B * W * V}
    # of uniformly drawn parents: beams that are not their own parent, and the different parents that those have
    B, W, size = c["B"], c["W"], 4 * c["H"] * c["dk"] * c["dv"]
    moved, others = W - 1, W * (1 - (1 - 1 / W) ** (W - 1))
    return {"bytes": int(B * c["layers"] * size * (moved + others)) + 4 * B * W, "flops": 0}
