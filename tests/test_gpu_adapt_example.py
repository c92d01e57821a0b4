"""The adapters, the layer, the balance loss and the optimiser together, as
examples/adapt_router.py runs them."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "adapt_router", os.path.join(ROOT, "examples", "adapt_router.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,bits", [(600, 32), (600, 8), (100, 32)])
def test_training_evens_the_load_and_needs_no_waits(cuda_ok, tokens, bits):
    """The load evens out; and every call's results are complete when the next
    one reads them (the layer's forward reads its logits ahead of its grid
    wait): waiting for the GPU after each call changes no bit."""
    ex = example()
    r = ex.run(steps=25, tokens=tokens, state_bits=bits)
    assert r["loss"][-1] < r["loss"][0] - 0.25 * (r["loss"][0] - 1)
    assert r["load"][-1] < r["load"][0]
    assert torch.isfinite(r["out"].float()).all()
    waited = ex.run(steps=25, tokens=tokens, state_bits=bits, sync=True)
    assert r["loss"] == waited["loss"]
    for p, q in zip(r["pools"] + [r["logits"], r["out"]],
                    waited["pools"] + [waited["logits"], waited["out"]]):
        assert torch.equal(p, q)


@pytest.mark.gpu
def test_routing_views_match_the_router(cuda_ok):
    """FusedMoE.routing: the ids and weights of the last forward."""
    import moe_inputs as MI
    import precision_moe_grouped_gb300 as P
    for T in (5, 100, 700):
        case = MI.make_case(MI.custom_config(16, 4, 256, 128), T, device="cuda", seed=T)
        moe = P.FusedMoE(case.w1, case.w1_sf, case.w2, case.w2_sf, 4)
        moe(case.x, case.logits)
        ids, w = moe.routing(T)
        top = case.logits.topk(4, dim=1)
        assert torch.equal(ids.long(), top.indices)
        assert torch.allclose(w, top.values.softmax(1), atol=1e-6)
