"""Adapters, balance loss and AdamW at their edges: attributes that change
between calls, views that outlive what they show, the longest batches,
infinities, and inputs that the kernel before has only just written."""
import pytest
import torch

import precision_moe_grouped_gb300 as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.set_device(0)


@pytest.mark.parametrize("T", [50, 3000])   # one kernel, and two
def test_balance_coefficient_changes(T):
    """A changed coefficient takes effect with the next call of the same size:
    with one a power of two of the other, exactly."""
    g = torch.Generator(device=DEV).manual_seed(T)
    z = torch.randn(T, 16, generator=g, device=DEV)
    ids = z.topk(2, dim=1).indices.to(torch.int32).contiguous()
    op = P.BalanceLoss(16, 2, coef=1.0)
    one = op(z, ids)
    op.coef = 0.25
    quarter = op(z, ids)
    fresh = P.BalanceLoss(16, 2, coef=0.25)(z, ids)
    assert all(torch.equal(p, q) for p, q in zip(quarter, fresh))
    assert torch.equal(quarter[0], one[0] * 0.25) and torch.equal(quarter[2], one[2] * 0.25)


def test_captured_step_repeats_its_number():
    """Replays of a captured step are eager steps of its number, whatever the
    gradients; a step whose number is only counted is refused under a capture."""
    g = torch.Generator(device=DEV).manual_seed(1)
    p = torch.randn(5000, generator=g, device=DEV)
    q, grad = p.clone(), torch.randn(5000, generator=g, device=DEV)
    a, b = P.AdamW([p], [grad], lr=1e-2), P.AdamW([q], [grad], lr=1e-2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(P.MoeError, match="captured step"):
            b.step()
        b.step(step=3)
    b.lr = 1.0                       # no part of the graph any more
    assert b.steps_done == 0
    for _ in range(4):
        grad.copy_(torch.randn(5000, generator=g, device=DEV))
        graph.replay()
        a.step(step=3)
    torch.cuda.synchronize()
    assert torch.equal(p, q) and torch.equal(a.state["v"][0], b.state["v"][0])


def test_balance_of_the_most_tokens():
    """2^31 - 1 tokens, the most that the entry point takes: token indices that
    step past 2^31 and byte offsets beyond 2^33.  With one expert p = 1, so loss
    = coef * counted / valid and the gradient is 0.  A thread of the row kernel
    adds some 2^31 / (608 * 128) terms in float, each sum off by 2^-24."""
    T = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    z, ids = torch.zeros(T, 1, device=DEV), torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    mask[-3000::2] = 0               # 1500 of the last ones: padding
    ids[-2999:-999:2] = -1           # 1000 valid ones: no expert
    loss, counts, dz = P.BalanceLoss(1, 1, coef=2.0)(z, ids, mask=mask)
    valid = T - 1500
    assert counts.tolist() == [[valid - 1000]]
    assert not bool(dz.any())
    assert abs(float(loss) - 2 * (valid - 1000) / valid) <= 2 * (T / (608 * 128) + 100) * 2.0 ** -24
