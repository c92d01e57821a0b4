"""Workloads of the operators that serve and train a dense gated feed-forward block beside a mixture-of-experts layer.

Three kinds of case, each a plain dict:

  ffn        a gated feed-forward block (a shared expert, a dense layer): out = base + (silu(x Wg^T) * (x Wu^T)) Wd^T
  ffn_bwd    its gradients from x and dout alone: dx (added to dx_base), d[Wg; Wu] and dWd
  muon       one step over weight matrices whose update is orthogonalised: momentum, five Newton-Schulz steps, the
             parameters in 32 bits and their bf16 copies

`run` computes a case in plain torch (32-bit arithmetic, rounded once at the end) or, with `own`, through the package's
entry points.  `exact` restates each in 64 bits.  Sizes follow the package's own layer shapes (hidden 7168 with 2048
features, hidden 2048 with 1024) and its adapters' pools, and odd ones between.
"""
import math

import torch

own = False

NS = (3.4445, -4.7750, 2.0315)   # the Newton-Schulz polynomial s -> a s + b s^3 + c s^5
LR, MOMENTUM, DECAY, EPS, RMS = 1e-3, 0.95, 0.1, 1e-7, 0.2


def listed():
    return [
        # one user's next token: a shared expert added to the routed experts' output
        {"name": "ffn_one_token", "kind": "ffn", "tokens": 1, "hidden": 7168, "inter": 2048, "base": True},
        # a decode batch
        {"name": "ffn_decode_24", "kind": "ffn", "tokens": 24, "hidden": 7168, "inter": 2048, "base": True},
        # a large decode batch, an odd number of users
        {"name": "ffn_batch_131", "kind": "ffn", "tokens": 131, "hidden": 7168, "inter": 2048, "base": True},
        # a short prompt through a small layer, no base
        {"name": "ffn_prompt_1021", "kind": "ffn", "tokens": 1021, "hidden": 2048, "inter": 1024, "base": False},
        # a prompt batch
        {"name": "ffn_prompt_8192", "kind": "ffn", "tokens": 8192, "hidden": 7168, "inter": 2048, "base": True},
        # a short fine-tuning batch, a width that is no multiple of a tile
        {"name": "ffn_bwd_77", "kind": "ffn_bwd", "tokens": 77, "hidden": 2048, "inter": 1000, "base": False},
        # a training batch, an odd number of tokens
        {"name": "ffn_bwd_4099", "kind": "ffn_bwd", "tokens": 4099, "hidden": 7168, "inter": 2048, "base": True},
        # pools of low-rank adapters: many flat matrices, many tall ones
        {"name": "muon_adapters", "kind": "muon", "count": 48, "rows": 16, "cols": 7168, "tall": 48, "tall_rows": 4096,
         "tall_cols": 16, "bf16_grads": False},
        # a router's matrix
        {"name": "muon_router", "kind": "muon", "count": 1, "rows": 256, "cols": 7168, "tall": 0, "tall_rows": 1, "tall_cols": 1,
         "bf16_grads": False},
        # odd sizes of both orientations
        {"name": "muon_odd", "kind": "muon", "count": 3, "rows": 333, "cols": 1001, "tall": 2, "tall_rows": 777, "tall_cols": 129,
         "bf16_grads": True},
        # a shared expert's gate, up and down projections, bf16 gradients
        {"name": "muon_shared_expert", "kind": "muon", "count": 2, "rows": 2048, "cols": 7168, "tall": 1, "tall_rows": 7168,
         "tall_cols": 2048, "bf16_grads": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["ffn", "ffn", "ffn_bwd", "muon"])
    if kind == "muon":
        rows, tall_cols = _log(rng, 1, 1024), _log(rng, 1, 1024)
        cols, tall_rows = _log(rng, 16, 7168), _log(rng, 16, 7168)
        room = 2 ** 26   # elements, and fewer of large matrices
        count = _log(rng, 1, max(1, min(64, room // (rows * cols), 2 ** 33 // (rows * rows * cols))))
        tall = rng.choice([0, _log(rng, 1, max(1, min(64, room // (tall_rows * tall_cols),
                                                      2 ** 33 // (tall_rows * tall_cols * tall_cols))))])
        return {"kind": kind, "count": count, "rows": rows, "cols": cols, "tall": tall, "tall_rows": tall_rows,
                "tall_cols": tall_cols, "bf16_grads": rng.random() < 0.5}
    hidden = rng.choice([2048, 7168, 8 * _log(rng, 32, 896)])
    inter = rng.choice([1024, 2048, 8 * _log(rng, 16, 256)])
    tokens = _log(rng, 1, 8192) if kind == "ffn" else _log(rng, 1, 4099)
    return {"kind": kind, "tokens": tokens, "hidden": hidden, "inter": inter, "base": rng.random() < 0.6}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _prepare_ffn(case, seed):
    g = _gen(seed)
    T, H, I = (case[k] for k in ("tokens", "hidden", "inter"))
    s = {"case": case}
    s["x"] = _randn(g, T, H).to(torch.bfloat16)
    s["w_gate_up"] = (_randn(g, 2 * I, H) / math.sqrt(H)).to(torch.bfloat16)
    s["w_down"] = (_randn(g, H, I) / math.sqrt(I)).to(torch.bfloat16)
    if case["kind"] == "ffn":
        s["base"] = _randn(g, T, H).to(torch.bfloat16) if case["base"] else None
    else:
        s["dout"] = (_randn(g, T, H) * 1e-2).to(torch.bfloat16)
        s["dx_base"] = (_randn(g, T, H) * 1e-2).to(torch.bfloat16) if case["base"] else None
    if own:
        import precision_moe_grouped_gb300 as P
        s["op"] = P.GatedFFN(s["w_gate_up"], s["w_down"])
    return s


def _gradient(g, count, rows, cols):
    """A few strong directions over a floor of noise, as gradients of weight matrices have."""
    r = min(rows, cols, 32)
    strength = torch.arange(1, r + 1, device="cuda", dtype=torch.float32) ** -0.5
    strong = (_randn(g, count, rows, r) * strength) @ _randn(g, count, r, cols)
    return (strong + _randn(g, count, rows, cols)) * 1e-3


def _prepare_muon(case, seed):
    g = _gen(seed)
    kind = torch.bfloat16 if case["bf16_grads"] else torch.float32
    s = {"case": case}
    shapes = [(case["count"], case["rows"], case["cols"]), (case["tall"], case["tall_rows"], case["tall_cols"])]
    shapes = [n for n in shapes if n[0]]
    s["grads"] = [_gradient(g, *n).to(kind) for n in shapes]
    s["momentum"] = [t.float() * 0.5 + _randn(g, *t.shape) * 5e-4 for t in s["grads"]]
    s["params"] = [_randn(g, *n) * 0.02 for n in shapes]
    s["copies"] = [p.to(torch.bfloat16) for p in s["params"]]
    if own:
        import precision_moe_grouped_gb300 as P
        s["op"] = P.Muon(s["params"], s["grads"], copies=s["copies"], state=s["momentum"], lr=LR, momentum=MOMENTUM,
                         nesterov=True, weight_decay=DECAY, eps=EPS, ns_steps=5, ns_coefficients=NS, update_scale="rms")
    return s


def prepare(case, seed):
    return _prepare_muon(case, seed) if case["kind"] == "muon" else _prepare_ffn(case, seed)


# -------------------------------------------------------------- plain forms

def _plain_ffn(s):
    w, x = s["w_gate_up"].float(), s["x"].float()
    gate, up = (x @ w.T).chunk(2, dim=1)
    out = (gate / (1 + torch.exp(-gate)) * up) @ s["w_down"].float().T
    return (out if s["base"] is None else out + s["base"].float()).to(torch.bfloat16)


def _plain_ffn_bwd(s):
    w, wd, x, dout = s["w_gate_up"].float(), s["w_down"].float(), s["x"].float(), s["dout"].float()
    gate, up = (x @ w.T).chunk(2, dim=1)
    sig = 1 / (1 + torch.exp(-gate))
    act = gate * sig
    dh = dout @ wd
    d = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * act], dim=1)
    dx = d @ w
    dx = dx if s["dx_base"] is None else dx + s["dx_base"].float()
    return dx.to(torch.bfloat16), (d.T @ x).to(torch.bfloat16), (dout.T @ (act * up)).to(torch.bfloat16)


def _plain_ns(x):
    a = x @ x.transpose(1, 2)
    return NS[0] * x + (NS[1] * a + NS[2] * (a @ a)) @ x


def _plain_orthogonal(u):
    """Newton-Schulz steps on the side with fewer rows."""
    x = u.transpose(1, 2) if u.shape[1] > u.shape[2] else u
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    x = _plain_ns(_plain_ns(_plain_ns(_plain_ns(_plain_ns(x)))))
    return x.transpose(1, 2) if u.shape[1] > u.shape[2] else x


def _plain_muon_tensor(p, grad, m, copy):
    g = grad.float()
    m.copy_(m * MOMENTUM + g * (1 - MOMENTUM))
    o = _plain_orthogonal(m * MOMENTUM + g * (1 - MOMENTUM))
    p.copy_(p * (1 - LR * DECAY) - o * (LR * RMS * math.sqrt(max(p.shape[1:]))))
    copy.copy_(p)


def _plain_muon(s):
    [_plain_muon_tensor(*t) for t in zip(s["params"], s["grads"], s["momentum"], s["copies"])]
    return s["params"], s["momentum"], s["copies"]


def run(s):
    kind = s["case"]["kind"]
    if not own:
        return {"ffn": _plain_ffn, "ffn_bwd": _plain_ffn_bwd, "muon": _plain_muon}[kind](s)
    if kind == "ffn":
        return s["op"].forward(s["x"], base=s["base"])
    if kind == "ffn_bwd":
        return s["op"].backward(s["dout"], s["x"], dx_base=s["dx_base"])
    s["op"].step()
    return s["params"], s["momentum"], s["copies"]


def _muon_flops(m, n):
    """Least of the ways to run five steps on an m x n matrix, m <= n: products with the long side once before and once
    after the steps, m x m products between, symmetric results half computed."""
    return 3 * m * m * n + 17 * m * m * m


def work(case):
    if case["kind"] == "muon":
        per = (2 if case["bf16_grads"] else 4) + 16 + 2
        bytes_, flops = 0, 0
        for count, rows, cols in ((case["count"], case["rows"], case["cols"]), (case["tall"], case["tall_rows"], case["tall_cols"])):
            bytes_ += count * rows * cols * per
            flops += count * _muon_flops(min(rows, cols), max(rows, cols))
        return {"bytes": bytes_, "flops": flops}
    T, H, I = (case[k] for k in ("tokens", "hidden", "inter"))
    weights, rows = 6 * H * I, 2 * T * H
    if case["kind"] == "ffn":
        return {"bytes": weights + rows * (3 if case["base"] else 2), "flops": 6 * T * H * I}
    return {"bytes": 2 * weights + rows * (4 if case["base"] else 3), "flops": 16 * T * H * I}


# ------------------------------------------------------------ in 64 bits

def _features(s):
    """Gate, up and their derivatives' parts, in 64 bits: silu(z) = z (1 + tanh(z / 2)) / 2."""
    I = s["case"]["inter"]
    x, w = s["x"].double(), s["w_gate_up"].double()
    gate = torch.einsum("th,ih->ti", x, w[:I])
    up = torch.einsum("th,ih->ti", x, w[I:])
    half = 0.5 * (1 + torch.tanh(0.5 * gate))
    return x, w, gate, up, half


def _exact_ffn(s):
    _, _, gate, up, half = _features(s)
    out = torch.einsum("ti,hi->th", gate * half * up, s["w_down"].double())
    return out if s["base"] is None else s["base"].double() + out


def _exact_ffn_bwd(s):
    x, w, gate, up, half = _features(s)
    I = s["case"]["inter"]
    dout = s["dout"].double()
    dh = torch.einsum("th,hi->ti", dout, s["w_down"].double())
    dup = dh * gate * half
    dgate = dh * up * (half + gate * half * (1 - half))
    dx = torch.einsum("ti,ih->th", dgate, w[:I]) + torch.einsum("ti,ih->th", dup, w[I:])
    if s["dx_base"] is not None:
        dx = s["dx_base"].double() + dx
    dw = torch.cat([torch.einsum("ti,th->ih", dgate, x), torch.einsum("ti,th->ih", dup, x)])
    return dx, dw, torch.einsum("th,ti->hi", dout, gate * half * up)


def _exact_matrix(p, g, m):
    """One matrix of a step, in 64 bits."""
    a, b, c = NS
    p, g, m = p.double(), g.double(), m.double()
    m = MOMENTUM * m + (1 - MOMENTUM) * g
    u = MOMENTUM * m + (1 - MOMENTUM) * g
    x = u / (torch.linalg.vector_norm(u) + EPS)
    flip = x.shape[0] > x.shape[1]
    for _ in range(5):
        gram = x.T @ x if flip else x @ x.T
        poly = b * gram + c * torch.linalg.matrix_power(gram, 2)
        x = a * x + (x @ poly if flip else poly @ x)
    return p - LR * (DECAY * p + RMS * math.sqrt(max(p.shape)) * x), m


def _exact_muon(s):
    done = [[_exact_matrix(p, g, m) for p, g, m in zip(*t)] for t in zip(s["params"], s["grads"], s["momentum"])]
    params = [torch.stack([p for p, _ in t]) for t in done]
    return params, [torch.stack([m for _, m in t]) for t in done], params


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        return {"ffn": _exact_ffn, "ffn_bwd": _exact_ffn_bwd, "muon": _exact_muon}[case["kind"]](s)
