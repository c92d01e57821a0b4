"""Adapting the router of a frozen mixture-of-experts layer, tenant by tenant.

The layer's expert weights stay as they are (MXFP4); each tenant gets a low-rank
adapter beside the router's projection.  A training step runs

    logits = x Wr^T + adapters          LowRankAdapters.forward
    out, routing = the layer            FusedMoE
    loss, counts, dlogits               BalanceLoss
    dA, dB                              LowRankAdapters.backward
    AdamW on float masters              AdamW (bf16 pools written by the step)

so that the experts' load evens out, and the trained pools then serve
batches of single tokens.  One GPU; synthetic data.

    python examples/adapt_router.py --steps 40 --state-bits 8
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import moe_inputs as MI  # noqa: E402
import precision_moe_grouped_gb300 as P  # noqa: E402


def run(steps: int = 40, tokens: int = 600, tenants: int = 3, rank: int = 8, state_bits: int = 32,
        seed: int = 0, sync: bool = False, experts: int = 16, top_k: int = 2, hidden: int = 512,
        inter: int = 256) -> dict:
    """sync: wait for the GPU after every call (the results are the same)."""
    wait = torch.cuda.synchronize if sync else (lambda: None)
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    cfg = MI.custom_config(experts, top_k, hidden, inter)
    case = MI.make_case(cfg, 1, device=str(dev), seed=seed)
    moe = P.FusedMoE(case.w1, case.w1_sf, case.w2, case.w2_sf, top_k)
    # a router that prefers some experts
    router = torch.randn((experts, hidden), generator=g, device=dev) / hidden ** 0.5
    bias = torch.linspace(0.8, -0.8, experts, device=dev)

    a = torch.randn((tenants, rank, hidden), generator=g, device=dev) / hidden ** 0.5
    b = torch.zeros((tenants, experts, rank), device=dev)
    pools = [a.bfloat16(), b.bfloat16()]
    adapters = P.LowRankAdapters(*pools)
    grads = [torch.empty_like(a), torch.empty_like(b)]
    adamw = P.AdamW([a, b], grads, copies=pools, state_bits=state_bits, lr=2e-2, weight_decay=0.0)
    balance = P.BalanceLoss(experts, top_k)

    def layer(x, tenant):
        # a constant feature lets an adapter learn a bias
        logits = torch.addmm(bias, x.float(), router.t())
        wait()
        adapters.forward(x, tenant, logits, out=logits)
        wait()
        out = moe(x, logits)
        wait()
        return logits, out

    def batch(n):
        x = torch.randn((n, hidden), generator=g, device=dev)
        x[:, 0] = 4.0
        return x.bfloat16()

    history, loads = [], []
    tenant = (torch.arange(tokens, device=dev) * tenants // tokens).to(torch.int32)
    edges = torch.arange(tenants + 1, device=dev) * tokens
    seqs = ((edges + tenants - 1) // tenants).to(torch.int32)
    for _ in range(steps):
        x = batch(tokens)
        logits, _ = layer(x, tenant)
        ids, _ = moe.routing(tokens)
        loss, counts, dlogits = balance(logits, ids, seq_offsets=seqs)
        wait()
        adapters.backward(dlogits, x, tenant, da=grads[0], db=grads[1], need_dx=False)
        wait()
        adamw.step()
        wait()
        history.append(loss)
        loads.append(counts.float().max(dim=1).values.mean())
    # serving: one token a request, a tenant each
    x = batch(8)
    served = (torch.arange(8, device=dev) % tenants).to(torch.int32)
    logits, out = layer(x, served)
    torch.cuda.synchronize()
    ideal = tokens / tenants * top_k / experts
    return {"loss": torch.cat(history).tolist(), "load": [float(v) / ideal for v in loads],
            "pools": pools, "logits": logits, "out": out}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=600)
    ap.add_argument("--tenants", type=int, default=3)
    ap.add_argument("--rank", type=int, default=8)
    ap.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    a = ap.parse_args()
    r = run(a.steps, a.tokens, a.tenants, a.rank, a.state_bits)
    print(f"balance loss {r['loss'][0]:.4f} -> {r['loss'][-1]:.4f} (1 is even), "
          f"fullest expert {r['load'][0]:.2f}x -> {r['load'][-1]:.2f}x its share")


if __name__ == "__main__":
    main()
