"""The layer, the adapters and the balance loss right behind the kernels that
write their inputs, without waiting: the same bits as with everything
complete beforehand."""
import pytest
import torch

import moe_inputs as MI
import precision_moe_grouped_gb300 as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.set_device(0)


@pytest.mark.parametrize("T", [1, 8, 32, 33, 200, 700])   # every front end
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_layer_behind_its_producers(T, kind):
    """Logits from a library's GEMM (float, or bf16 and converted), x from a copy,
    both into buffers that still hold the step before."""
    E, H, steps = 64, 512, 12
    case = MI.make_case(MI.custom_config(E, 4, H, 256), 1, device=DEV, seed=T)
    moe = P.FusedMoE(case.w1, case.w1_sf, case.w2, case.w2_sf, 4)
    g = torch.Generator(device=DEV).manual_seed(T)
    router = (torch.randn(H, E, generator=g, device=DEV) / H ** 0.5).to(kind)
    xs = [torch.randn(T, H, generator=g, device=DEV).bfloat16() for _ in range(steps)]
    x, logits = torch.zeros_like(xs[0]), torch.zeros(T, E, device=DEV)

    def run(wait):
        got = []
        for step in xs:
            x.copy_(step)
            wait()
            if kind is torch.float32:
                torch.mm(x.float(), router, out=logits)
            else:
                logits.copy_(x @ router)
            wait()
            out = moe(x, logits)
            ids, w = moe.routing(T)
            got.append((out, ids.clone(), w.clone()))
        torch.cuda.synchronize()
        return got

    run(lambda: None)                # warm: allocations, library handles
    free, waited = run(lambda: None), run(torch.cuda.synchronize)
    for a, b in zip(free, waited):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("T", [40, 2000])   # one kernel, and several
def test_operators_behind_their_producers(T):
    E, H, k, steps = 64, 512, 4, 12
    g = torch.Generator(device=DEV).manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)        # noqa: E731
    ad = P.LowRankAdapters((rnd(3, 16, H) / H ** 0.5).bfloat16(), rnd(3, E, 16).bfloat16())
    balance, router = P.BalanceLoss(E, k), (rnd(H, E) / H ** 0.5).bfloat16()
    tenant = (torch.arange(T, device=DEV) % 4 - 1).to(torch.int32)
    xs = [rnd(T, H).bfloat16() for _ in range(steps)]
    x, base = torch.zeros_like(xs[0]), torch.zeros(T, E, device=DEV)

    def run(wait):
        got = []
        for step in xs:
            x.copy_(step)
            base.copy_(x @ router)
            wait()
            logits = ad(x, tenant, base)
            wait()
            ids = logits.topk(k, dim=1).indices.to(torch.int32)
            wait()
            loss, counts, dz = balance(logits, ids)
            wait()
            got.append((logits, loss, counts, dz) + ad.backward(dz, x, tenant))
        torch.cuda.synchronize()
        return got

    run(lambda: None)
    for a, b in zip(run(lambda: None), run(torch.cuda.synchronize)):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
