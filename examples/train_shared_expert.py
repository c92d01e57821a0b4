"""Training the shared expert of a mixture-of-experts layer beside its frozen
routed experts.

The routed experts stay as they are (MXFP4); the shared expert, a dense gated
feed-forward block in bf16, is trained to what another block would have added.
A training step runs

    routed = the layer                      FusedMoE
    out = routed + the shared expert        GatedFFN.forward (the sum in its last product)
    dout                                    mean squared error, in torch
    dWgu, dWd                               GatedFFN.backward (activations computed again)
    the weights                             Muon on float masters (bf16 weights written by the step)

and the trained block then serves single tokens.  One GPU; synthetic data.

    python examples/train_shared_expert.py --steps 60
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


def block(g, hidden: int, inter: int):
    """Float weights [2, I, H] (gate, up) and [H, I] of a block with outputs of about the inputs' size."""
    dev = g.device
    gate_up = torch.randn((2, inter, hidden), generator=g, device=dev) / hidden ** 0.5
    down = torch.randn((hidden, inter), generator=g, device=dev) / inter ** 0.5
    return gate_up, down


def run(steps: int = 60, tokens: int = 600, seed: int = 0, sync: bool = False, experts: int = 16, top_k: int = 2,
        hidden: int = 512, inter: int = 256, lr: float = 4e-3) -> dict:
    """sync: wait for the GPU after every call (the results are the same)."""
    wait = torch.cuda.synchronize if sync else (lambda: None)
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    case = MI.make_case(MI.custom_config(experts, top_k, hidden, inter), 1, device=str(dev), seed=seed)
    moe = P.FusedMoE(case.w1, case.w1_sf, case.w2, case.w2_sf, top_k)
    router = torch.randn((hidden, experts), generator=g, device=dev) / hidden ** 0.5

    teacher = P.GatedFFN(*(w.bfloat16().reshape(-1, w.shape[-1]) for w in block(g, hidden, inter)))
    masters = list(block(g, hidden, inter))
    weights = [w.bfloat16() for w in masters]
    shared = P.GatedFFN(weights[0].view(2 * inter, hidden), weights[1])
    grads = [torch.empty_like(w) for w in weights]
    muon = P.Muon(masters, grads, copies=weights, lr=lr, weight_decay=0.0)

    def batch(n):
        x = torch.randn((n, hidden), generator=g, device=dev).bfloat16()
        routed = moe(x, x.float() @ router)
        wait()
        return x, routed

    history, first = [], None
    for _ in range(steps):
        x, routed = batch(tokens)
        target = teacher(x, base=routed)
        out = shared(x, base=routed)
        wait()
        off = out.float() - target.float()
        history.append(off.square().mean())
        dout = (off * (2.0 / off.numel())).bfloat16()
        shared.backward(dout, x, dw_gate_up=grads[0].view(2 * inter, hidden), dw_down=grads[1], need_dx=False)
        wait()
        if first is None:
            first = {"x": x, "dout": dout, "weights": [w.clone() for w in weights], "grads": [t.clone() for t in grads]}
        muon.step()
        wait()
    # serving: one token
    x, routed = batch(1)
    out = shared(x, base=routed)
    torch.cuda.synchronize()
    assert shared.device_status() == 0 and muon.device_status() == 0
    return {"loss": torch.stack(history).tolist(), "masters": masters, "weights": weights, "first": first, "x": x,
            "routed": routed, "out": out}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=600)
    a = ap.parse_args()
    r = run(a.steps, a.tokens)
    print(f"mean squared error {r['loss'][0]:.4f} -> {r['loss'][-1]:.4f}")


if __name__ == "__main__":
    main()
