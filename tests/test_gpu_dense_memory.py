"""Tensors of the gated feed-forward block that lie between one another's rows in one
buffer: apart, so accepted, with the bits of tensors that lie alone; and refusals of
those that are not apart, through the binding."""
import pytest
import torch

import precision_moe_grouped_gb300 as P
import test_gpu_ffn as F

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
H, I = 264, 136


def block(T):
    s = F.make(T, H, I, seed=3)
    return s, P.GatedFFN(s["wgu"], s["wd"])


@pytest.mark.parametrize("T", [1, 20, 100, 300, 900])
def test_between_rows(cuda_ok, T):
    s, op = block(T)
    names = ("x", "base", "dout", "dx_base")
    wide = torch.full((T, 6 * H), 7.0, device="cuda", dtype=BF16)
    at = {k: wide[:, i * H:(i + 1) * H] for i, k in enumerate(names)}
    for k in names:
        at[k].copy_(s[k])
    out, dx = wide[:, 4 * H:5 * H], wide[:, 5 * H:]
    want = op(s["x"], base=s["base"])
    assert torch.equal(op(at["x"], base=at["base"], out=out), want) and out.data_ptr() == wide.data_ptr() + 8 * H
    grads = op.backward(s["dout"], s["x"], dx_base=s["dx_base"])
    got = op.backward(at["dout"], at["x"], dx_base=at["dx_base"], dx=dx)
    for a, b in zip(got, grads):
        assert torch.equal(a, b)
    for k in names:
        assert torch.equal(at[k], s[k])
    # both weights' gradients in one buffer, end to end, and dx in place
    flat = torch.empty(3 * H * I, device="cuda", dtype=BF16)
    got = op.backward(at["dout"], at["x"], dx_base=at["dx_base"], dx=at["dx_base"],
                      dw_gate_up=flat[:2 * H * I].view(2 * I, H), dw_down=flat[2 * H * I:].view(H, I))
    for a, b in zip(got, grads):
        assert torch.equal(a, b)


def test_shared_rows_are_refused(cuda_ok):
    s, op = block(100)
    more = torch.zeros((300, H), device="cuda", dtype=BF16)
    for out, base in ((more[1:101], more[:100]), (more[:200:2], more[:100]), (more[:100], more[:300:3])):
        with pytest.raises(P.MoeError, match="overlaps"):
            op(s["x"], base=base, out=out)
        with pytest.raises(P.MoeError, match="overlaps"):
            op(base, out=out)
        with pytest.raises(P.MoeError, match="overlaps"):
            op.backward(s["dout"], s["x"], dx=out, dx_base=base)
    w = more.view(-1)[:2 * I * H].view(2 * I, H)
    for bad in (dict(dx_base=more[:100]), dict(dx=more[150:250])):
        with pytest.raises(P.MoeError, match="overlaps"):
            op.backward(s["dout"], s["x"], dw_gate_up=w, **bad)
    assert not more.any()
