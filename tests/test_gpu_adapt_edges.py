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
