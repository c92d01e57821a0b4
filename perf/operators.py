"""Workloads of the operators that adapt and train beside a frozen mixture-of-experts layer.

Four kinds of case, each a plain dict:

  adapters   low-rank adapters of many requests beside a shared projection: out = base + scale_a B_a A_a x
  adapters_bwd   their gradients: dx (added to the shared projection's), dA and dB
  balance    the router's load-balance loss, per-expert counts, and the gradient of the router logits
  adamw      one AdamW step over many tensors, states in 32 or in 8 bits

`run` computes a case in plain torch (32-bit arithmetic, rounded once at the end) or, with `own`, through the
package's entry points.  `exact` restates each in 64 bits.  Sizes follow the package's own layer shapes
(hidden 7168 and 2048, 8 / 64 / 256 / 384 experts, 2 * 2048 gate and up features).
"""
import itertools
import math
import random

import numpy as np
import torch

own = False

BLOCK = 256          # elements that share one scale in an 8-bit optimiser state
E4M3_MAX = 448.0
TINY = 2.0 ** -100   # an 8-bit state block below this is stored as zero


def listed():
    return [
        # one user's next token, one adapter, beside the layer's output
        {"name": "adapters_one_token", "kind": "adapters", "tokens": 1, "requests": 1, "adapters": 16, "rank": 16,
         "hidden": 7168, "out": 7168, "bf16": True},
        # a decode batch: every request its own token, popular adapters shared by a few of them
        {"name": "adapters_decode_64", "kind": "adapters", "tokens": 64, "requests": 64, "adapters": 48, "rank": 32,
         "hidden": 7168, "out": 4096, "bf16": True},
        # a prompt batch of ragged requests
        {"name": "adapters_prompt_8192", "kind": "adapters", "tokens": 8192, "requests": 24, "adapters": 16, "rank": 16,
         "hidden": 7168, "out": 7168, "bf16": True},
        # the router's float32 logits of 256 experts, ragged requests, an odd token count
        {"name": "adapters_router_1021", "kind": "adapters", "tokens": 1021, "requests": 13, "adapters": 8, "rank": 8,
         "hidden": 7168, "out": 256, "bf16": False},
        # training the router's adapters: float32 gradients of the logits
        {"name": "adapters_bwd_router", "kind": "adapters_bwd", "tokens": 4096, "requests": 16, "adapters": 8, "rank": 16,
         "hidden": 7168, "out": 256, "bf16": False},
        # training adapters beside a bf16 projection, ragged requests
        {"name": "adapters_bwd_2048", "kind": "adapters_bwd", "tokens": 5003, "requests": 20, "adapters": 6, "rank": 64,
         "hidden": 2048, "out": 2048, "bf16": True},
        # a small router, a short batch
        {"name": "balance_e8", "kind": "balance", "tokens": 201, "experts": 8, "top_k": 2, "sequences": 1, "masked": False,
         "gates": False},
        # a training batch of ragged sequences, padding masked out, gate gradients joined
        {"name": "balance_e256_long", "kind": "balance", "tokens": 65536, "experts": 256, "top_k": 8, "sequences": 24,
         "masked": True, "gates": True},
        # the widest router, one odd batch
        {"name": "balance_e384", "kind": "balance", "tokens": 8191, "experts": 384, "top_k": 6, "sequences": 1,
         "masked": True, "gates": False},
        # the adapters of a layer: many small and odd tensors
        {"name": "adamw_adapters", "kind": "adamw", "tensors": 96, "elements": 3000001, "bits": 32, "bf16_grads": False},
        # a large model's trainable part, bf16 gradients, states in 32 bits
        {"name": "adamw_large_32", "kind": "adamw", "tensors": 40, "elements": 200000000, "bits": 32, "bf16_grads": True},
        # the same with states in 8 bits
        {"name": "adamw_large_8", "kind": "adamw", "tensors": 200, "elements": 200000000, "bits": 8, "bf16_grads": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["adapters", "adapters", "adapters_bwd", "balance", "adamw"])
    if kind == "adapters":
        tokens = min(8192, _log(rng, 1, 8192))
        requests = min(tokens, rng.choice([tokens, _log(rng, 1, 96)])) if tokens <= 128 else _log(rng, 1, 48)
        return {"kind": kind, "tokens": tokens, "requests": requests, "adapters": _log(rng, 1, 64),
                "rank": rng.choice([8, 16, 24, 32, 64]), "hidden": rng.choice([2048, 7168, 8 * _log(rng, 32, 896)]),
                "out": rng.choice([64, 256, 384, 4096, 7168, 8 * _log(rng, 32, 896)]), "bf16": rng.random() < 0.6}
    if kind == "adapters_bwd":
        tokens = _log(rng, 64, 5003)
        return {"kind": kind, "tokens": tokens, "requests": min(tokens, _log(rng, 1, 32)), "adapters": _log(rng, 1, 8),
                "rank": rng.choice([8, 16, 32, 40, 64]), "hidden": rng.choice([2048, 8 * _log(rng, 32, 256)]),
                "out": rng.choice([256, 384, 2048, 8 * _log(rng, 32, 256)]), "bf16": rng.random() < 0.5}
    if kind == "balance":
        experts = rng.choice([8, 64, 256, 384, _log(rng, 8, 512)])
        tokens = _log(rng, 16, 32768)
        return {"kind": kind, "tokens": tokens, "experts": experts, "top_k": rng.choice([1, 2, 4, 6, 8]),
                "sequences": rng.choice([1, min(tokens, _log(rng, 2, 48))]), "masked": rng.random() < 0.5,
                "gates": rng.random() < 0.5}
    return {"kind": kind, "tensors": _log(rng, 1, 256), "elements": _log(rng, 100000, 100000000),
            "bits": rng.choice([8, 32]), "bf16_grads": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _cuts(g, total, parts):
    """parts + 1 offsets into `total` items, every part non-empty."""
    inner = torch.randperm(total - 1, generator=g, device="cuda")[: parts - 1] + 1
    edge = torch.tensor([0, total], device="cuda")
    return torch.cat([edge[:1], inner.sort().values, edge[1:]])


def _adapted(case):
    """Requests that use an adapter: with more than eight, every eighth uses none."""
    n = case["requests"]
    return n - n // 8


def _adapter_ids(case, g):
    """Each token's adapter.  Requests hold consecutive tokens; adapters go round in a shuffled order, so the number
    of adapters in use does not depend on the seed."""
    T, R, NA = case["tokens"], case["requests"], case["adapters"]
    offs = _cuts(g, T, R)
    perm = torch.randperm(NA, generator=g, device="cuda")
    n = _adapted(case)
    of_request = torch.full((R,), -1, dtype=torch.int64, device="cuda")
    place = torch.randperm(R, generator=g, device="cuda")[:n]
    of_request[place] = perm[torch.arange(n, device="cuda") % NA]
    token = torch.arange(T, device="cuda")
    return of_request[torch.searchsorted(offs[1:], token, right=True)].to(torch.int32)


def _prepare_adapters(case, seed):
    g = _gen(seed)
    T, NA, r, H, N = (case[k] for k in ("tokens", "adapters", "rank", "hidden", "out"))
    kind = torch.bfloat16 if case["bf16"] else torch.float32
    s = {"case": case}
    s["ids"] = _adapter_ids(case, g)
    s["x"] = _randn(g, T, H).to(torch.bfloat16)
    s["a"] = (_randn(g, NA, r, H) / math.sqrt(H)).to(torch.bfloat16)
    s["b"] = (_randn(g, NA, N, r) * 0.1).to(torch.bfloat16)
    s["scale"] = torch.rand((NA,), generator=g, device="cuda") + 0.5
    if case["kind"] == "adapters":
        s["base"] = _randn(g, T, N).to(kind)
    else:
        s["dout"] = (_randn(g, T, N) * 1e-2).to(kind)
        s["dx_base"] = (_randn(g, T, H) * 1e-2).to(torch.bfloat16)
    if own:
        import precision_moe_grouped_gb300 as P
        s["op"] = P.LowRankAdapters(s["a"], s["b"], s["scale"])
    return s


def _prepare_balance(case, seed):
    g = _gen(seed)
    T, E, k, S = (case[n] for n in ("tokens", "experts", "top_k", "sequences"))
    s = {"case": case, "coef": 0.01}
    rank = torch.randperm(E, generator=g, device="cuda").float() + 1.0
    s["logits"] = _randn(g, T, E) - 0.5 * torch.log(rank)          # popular and rare experts
    top = torch.topk(s["logits"], k, dim=1)
    s["ids"] = top.indices.to(torch.int32).contiguous()
    s["mask"] = (torch.rand((T,), generator=g, device="cuda") < 0.9).to(torch.uint8) if case["masked"] else None
    s["seq"] = _cuts(g, T, S).to(torch.int32) if S > 1 else None
    s["weights"] = torch.softmax(top.values, dim=1) if case["gates"] else None
    s["dweights"] = _randn(g, T, k) * 1e-3 if case["gates"] else None
    if own:
        import precision_moe_grouped_gb300 as P
        s["op"] = P.BalanceLoss(E, k, coef=s["coef"])
    return s


def _tensor_sizes(case):
    """Sizes of the step's tensors: ragged, odd ones among them, `elements` in all."""
    r = random.Random(1000003 * case["tensors"] + case["elements"])
    share = [math.exp(r.gauss(0.0, 1.0)) for _ in range(case["tensors"])]
    sizes = [max(1, int(case["elements"] * w / sum(share))) for w in share]
    sizes[0] += max(0, case["elements"] - sum(sizes))
    return sizes


ADAMW = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01, "step": 100}


def _prepare_adamw(case, seed):
    """Tensors lie one after another in flat buffers, each begun on a multiple of BLOCK elements (what is between
    them stays zero), so that the plain form takes all of them in one go."""
    g = _gen(seed)
    sizes = _tensor_sizes(case)
    ends = list(itertools.accumulate(-(-n // BLOCK) * BLOCK for n in sizes))
    starts, at = [0] + ends[:-1], ends[-1]
    kind = torch.bfloat16 if case["bf16_grads"] else torch.float32
    s = {"case": case}
    place = torch.arange(at, device="cuda")
    tensor = torch.searchsorted(torch.tensor(ends, device="cuda"), place, right=True)
    stop = torch.tensor([o + n for o, n in zip(starts, sizes)], device="cuda")
    inside = (place < stop[tensor]).float()
    p = torch.randn(at, generator=g, device="cuda") * 0.02 * inside
    grad = torch.randn(at, generator=g, device="cuda") * 1e-3 * inside
    m = torch.randn(at, generator=g, device="cuda") * 3e-4 * inside
    v = (torch.rand(at, generator=g, device="cuda") + 0.2) * 1e-6 * inside
    s["p"], s["grad"], s["copy"] = p, grad.to(kind), p.to(torch.bfloat16)
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["m"], s["m_scale"] = _encode(m, False)
        s["v"], s["v_scale"] = _encode(v.sqrt(), True)
    if own:
        import precision_moe_grouped_gb300 as P

        def views(t, per=1):
            return [t[o // per:o // per + -(-n // per)] for n, o in zip(sizes, starts)]

        state = {"m": views(s["m"]), "v": views(s["v"])}
        if case["bits"] == 8:
            state |= {"m_scale": views(s["m_scale"], BLOCK), "v_scale": views(s["v_scale"], BLOCK)}
        s["op"] = P.AdamW(views(s["p"]), views(s["grad"]), copies=views(s["copy"]), state_bits=case["bits"], state=state,
                          lr=ADAMW["lr"], betas=(ADAMW["beta1"], ADAMW["beta2"]), eps=ADAMW["eps"],
                          weight_decay=ADAMW["weight_decay"])
    return s


def prepare(case, seed):
    kind = case["kind"]
    if kind == "balance":
        return _prepare_balance(case, seed)
    return _prepare_adamw(case, seed) if kind == "adamw" else _prepare_adapters(case, seed)


# -------------------------------------------------------------- plain forms

def _lanes(s):
    """[T, NA]: 1 where the token uses the adapter."""
    return s["ids"][:, None] == torch.arange(s["a"].shape[0], device=s["ids"].device)


def _plain_adapters(s):
    a, b = s["a"].float(), s["b"].float()
    NA, r, H = a.shape
    x = s["x"].float()
    use = (_lanes(s) * s["scale"])[:, :, None]
    v = (x @ a.reshape(NA * r, H).T).reshape(-1, NA, r) * use
    delta = v.reshape(-1, NA * r) @ b.transpose(1, 2).reshape(NA * r, -1)
    return (s["base"].float() + delta).to(s["base"].dtype)


def _plain_adapters_bwd(s):
    a, b, x, dout = s["a"].float(), s["b"].float(), s["x"].float(), s["dout"].float()
    NA, r, H = a.shape
    N = b.shape[1]
    flat_a, flat_b = a.reshape(NA * r, H), b.transpose(1, 2).reshape(NA * r, N)
    use = (_lanes(s) * s["scale"])[:, :, None]
    u = ((dout @ flat_b.T).reshape(-1, NA, r) * use).reshape(-1, NA * r)
    v = ((x @ flat_a.T).reshape(-1, NA, r) * use).reshape(-1, NA * r)
    dx = (s["dx_base"].float() + u @ flat_a).to(torch.bfloat16)
    da = (u.T @ x).reshape(NA, r, H)
    db = (v.T @ dout).reshape(NA, r, N).transpose(1, 2).contiguous()
    return dx, da, db


def _plain_balance(s):
    z, ids, k = s["logits"], s["ids"].long(), s["case"]["top_k"]
    T, E = z.shape
    S = s["case"]["sequences"]
    token = torch.arange(T, device=z.device)
    seq = torch.zeros_like(token) if s["seq"] is None else torch.searchsorted(s["seq"][1:].long(), token, right=True)
    valid = torch.ones(T, device=z.device) if s["mask"] is None else s["mask"].float()
    top = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - top)
    p = e / e.sum(dim=1, keepdim=True)
    n = torch.zeros(S, device=z.device).index_add_(0, seq, valid)
    counts = torch.zeros(S * E, device=z.device)
    counts.index_add_(0, (seq[:, None] * E + ids).reshape(-1), valid[:, None].expand(T, k).reshape(-1))
    counts = counts.reshape(S, E)
    total = torch.zeros(S, E, device=z.device).index_add_(0, seq, p * valid[:, None])
    some = n.clamp(min=1.0)
    f = counts * E / (k * some)[:, None]
    live = (n > 0).float().sum().clamp(min=1.0)
    loss = s["coef"] / live * (f * total / some[:, None]).sum()
    ft = f[seq]
    c = s["coef"] / live * valid / some[seq]
    dz = c[:, None] * p * (ft - (ft * p).sum(dim=1, keepdim=True))
    if s["weights"] is not None:
        w, dw = s["weights"], s["dweights"]
        dz = dz.scatter_add(1, ids, w * (dw - (w * dw).sum(dim=1, keepdim=True)))
    return loss.reshape(1), counts.to(torch.int32), dz


def _encode(t, positive):
    """E4M3 codes of t by blocks of BLOCK with a 32-bit scale, amax / 448; with `positive` what is above zero stays
    above zero."""
    t = t.reshape(-1, BLOCK)
    amax = t.abs().amax(dim=1)
    some = ~(amax < TINY)
    full = torch.full_like(amax, E4M3_MAX)
    inv = torch.where(some, full / amax, torch.zeros_like(amax))
    scale = torch.where(some, amax / full, torch.ones_like(amax))
    q = (t * inv[:, None]).to(torch.float8_e4m3fn)
    if positive:
        least = torch.full_like(t, 2.0 ** -9)
        q = torch.where((q.float() == 0) & (t > 0) & some[:, None], least, q.float()).to(torch.float8_e4m3fn)
    return q.reshape(-1), scale


def _decode(q, scale):
    return (q.float().reshape(-1, BLOCK) * scale[:, None]).reshape(-1)


def _plain_adamw(s):
    b1, b2, t = ADAMW["beta1"], ADAMW["beta2"], ADAMW["step"]
    small = s["case"]["bits"] == 8
    g = s["grad"].float()
    m = _decode(s["m"], s["m_scale"]) if small else s["m"]
    if small:
        r = _decode(s["v"], s["v_scale"])
        v = r * r
    else:
        v = s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    r = v.sqrt()
    step = ADAMW["lr"] / (1 - b1 ** t)
    p = s["p"] * (1 - ADAMW["lr"] * ADAMW["weight_decay"]) - m * step / (r * (1 / math.sqrt(1 - b2 ** t)) + ADAMW["eps"])
    s["p"].copy_(p)
    s["copy"].copy_(p)
    if not small:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return s["p"], s["copy"], s["m"], s["v"]
    q, scale = _encode(m, False)
    s["m"].copy_(q)
    s["m_scale"].copy_(scale)
    q, scale = _encode(r, True)
    s["v"].copy_(q)
    s["v_scale"].copy_(scale)
    return s["p"], s["copy"], s["m"], s["m_scale"], s["v"], s["v_scale"]


def run(s):
    kind = s["case"]["kind"]
    if not own:
        return {"adapters": _plain_adapters, "adapters_bwd": _plain_adapters_bwd, "balance": _plain_balance,
                "adamw": _plain_adamw}[kind](s)
    op = s["op"]
    if kind == "adapters":
        return op.forward(s["x"], s["ids"], s["base"])
    if kind == "adapters_bwd":
        return op.backward(s["dout"], s["x"], s["ids"], s["dx_base"])
    if kind == "balance":
        return op(s["logits"], s["ids"], mask=s["mask"], seq_offsets=s["seq"], weights=s["weights"], dweights=s["dweights"])
    op.step(step=ADAMW["step"])
    if s["case"]["bits"] == 32:
        return s["p"], s["copy"], s["m"], s["v"]
    return s["p"], s["copy"], s["m"], s["m_scale"], s["v"], s["v_scale"]


def work(case):
    kind = case["kind"]
    if kind == "balance":
        T, E, k, S = (case[n] for n in ("tokens", "experts", "top_k", "sequences"))
        per = 8 * E + 4 * k + (8 * k if case["gates"] else 0) + (1 if case["masked"] else 0)
        return {"bytes": T * per + 4 * S * E, "flops": 10 * T * E}
    if kind == "adamw":
        per = 8 + (2 if case["bf16_grads"] else 4) + 2 + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
        return {"bytes": per * case["elements"], "flops": 16 * case["elements"]}
    T, NA, r, H, N = (case[k] for k in ("tokens", "adapters", "rank", "hidden", "out"))
    es = 2 if case["bf16"] else 4
    touched = min(NA, _adapted(case))
    pools = 2 * touched * r * (H + N) + 4 * touched
    if kind == "adapters":
        return {"bytes": T * (2 * H + 2 * es * N + 4) + pools, "flops": 2 * T * r * (H + N)}
    return {"bytes": T * (2 * H + es * N + 4 * H + 4) + pools + 4 * NA * r * (H + N), "flops": 2 * T * r * (3 * H + 2 * N)}


# ------------------------------------------------------------ in 64 bits

def _exact_adapters(s):
    """Adapter by adapter, its own tokens only."""
    out = s["base"].double().clone()
    for i in range(s["a"].shape[0]):
        rows = torch.nonzero(s["ids"] == i).reshape(-1)
        low = torch.einsum("th,rh->tr", s["x"][rows].double(), s["a"][i].double())
        out[rows] += torch.einsum("tr,nr->tn", low, s["b"][i].double()) * s["scale"][i].double()
    return out


def _exact_adapters_bwd(s):
    dx = s["dx_base"].double().clone()
    da = torch.zeros(s["a"].shape, dtype=torch.float64, device=dx.device)
    db = torch.zeros(s["b"].shape, dtype=torch.float64, device=dx.device)
    for i in range(s["a"].shape[0]):
        rows = torch.nonzero(s["ids"] == i).reshape(-1)
        x, d = s["x"][rows].double(), s["dout"][rows].double() * s["scale"][i].double()
        a, b = s["a"][i].double(), s["b"][i].double()
        up = torch.einsum("tn,nr->tr", d, b)
        dx[rows] += torch.einsum("tr,rh->th", up, a)
        da[i] = torch.einsum("tr,th->rh", up, x)
        db[i] = torch.einsum("tn,tr->nr", d, torch.einsum("th,rh->tr", x, a))
    return dx, da, db


def _exact_balance(s):
    """Sequence by sequence on the host."""
    z = s["logits"].double().cpu().numpy()
    ids = s["ids"].cpu().numpy()
    T, E = z.shape
    k = ids.shape[1]
    ok = np.ones(T, bool) if s["mask"] is None else s["mask"].cpu().numpy() != 0
    offs = np.array([0, T]) if s["seq"] is None else s["seq"].cpu().numpy()
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    parts = [(a, b) for a, b in zip(offs[:-1], offs[1:])]
    live = max(1, sum(bool(ok[a:b].any()) for a, b in parts))
    loss, dz, counts = 0.0, np.zeros((T, E)), np.zeros((len(parts), E), np.int64)
    for i, (a, b) in enumerate(parts):
        rows = np.arange(a, b)[ok[a:b]]
        if len(rows):
            counts[i] = np.bincount(ids[rows].reshape(-1), minlength=E)
            f = counts[i] * (E / (k * len(rows)))
            loss += s["coef"] / live * float(f @ p[rows].mean(0))
            dz[rows] = s["coef"] / (live * len(rows)) * p[rows] * (f[None] - (p[rows] @ f)[:, None])
    if s["weights"] is not None:
        w, dw = s["weights"].double().cpu().numpy(), s["dweights"].double().cpu().numpy()
        np.add.at(dz, (np.arange(T)[:, None], ids), w * (dw - (w * dw).sum(1, keepdims=True)))
    return np.array([loss]), torch.from_numpy(counts.astype(np.int32)), dz


def _exact_codes(t, positive):
    """Nearest E4M3 value (ties to even) of each block's elements over amax / 448, and that scale."""
    t = t.reshape(-1, BLOCK)
    amax = t.abs().amax(dim=1)
    scale = torch.where(amax < TINY, torch.ones_like(amax), amax / E4M3_MAX)
    q = t / scale[:, None] * (amax >= TINY)[:, None]
    _, e = torch.frexp(q)
    ulp = torch.ldexp(torch.ones_like(q), (e - 4).clamp(min=-9))
    y = torch.round(q / ulp) * ulp
    if positive:
        y = torch.where((y == 0) & (q > 0), torch.full_like(y, 2.0 ** -9), y)
    return y.reshape(-1), scale


def _exact_adamw(s):
    b1, b2, t = ADAMW["beta1"], ADAMW["beta2"], ADAMW["step"]
    g = s["grad"].double()
    if s["case"]["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        m = s["m"].double() * s["m_scale"].double().repeat_interleave(BLOCK)
        v = torch.square(s["v"].double() * s["v_scale"].double().repeat_interleave(BLOCK))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * torch.square(g)
    hat_m, hat_v = m / (1 - b1 ** t), v / (1 - b2 ** t)
    p = s["p"].double()
    p = p - ADAMW["lr"] * (hat_m / (hat_v.sqrt() + ADAMW["eps"]) + ADAMW["weight_decay"] * p)
    if s["case"]["bits"] == 32:
        return p, p, m, v
    qm, sm = _exact_codes(m, False)
    qv, sv = _exact_codes(v.sqrt(), True)
    return p, p, qm, sm, qv, sv


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        return {"adapters": _exact_adapters, "adapters_bwd": _exact_adapters_bwd, "balance": _exact_balance,
                "adamw": _exact_adamw}[case["kind"]](s)
