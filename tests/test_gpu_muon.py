"""The orthogonalised step against the formula in 64 bits.

With p = 0, lr = 1 and no decay a step leaves p = -s X, so that X itself is seen.
Its error is held against the plain form's in 32 bits, e32, on the same input:
- numbers between the products have 22 bits instead of 24, and the products
  leave out lo lo terms of 2^-22: 4 times the roundings of the plain form, and
  there are up to twice as many of them: 8 e32;
- an MMA adds 16 terms at a time and truncates its sum to 24 bits: a diagonal
  element of X X^T, a sum of n squares, shrinks by up to n / 16 2^-24 of itself
  (the mean partial sum is half the whole), and X follows with |s f'(s) / f(s)|,
  below 4 for the five steps' polynomial f where f is not near 0, at two Gram
  matrices of half that effect each: 4 n / 16 2^-24;
- 2^-18 for one that e32 happens to leave out."""
import math

import pytest
import torch

import precision_moe_grouped_gb300 as P

pytestmark = pytest.mark.gpu
NS = (3.4445, -4.7750, 2.0315)


def orthogonal(u, steps, eps, coef=NS):
    """The formula in u's precision, on the shorter side."""
    a, b, c = coef
    x = u.transpose(-1, -2) if u.shape[-2] > u.shape[-1] else u
    x = x / (x.square().sum(dim=(-1, -2), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        g = x @ x.transpose(-1, -2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.transpose(-1, -2) if u.shape[-2] > u.shape[-1] else x


def factor(kind, rows, cols):
    return 0.2 * math.sqrt(max(rows, cols)) if kind == "rms" else math.sqrt(max(1.0, rows / cols))


def inputs(kind, shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    r, c = shape[-2:]
    if kind == "noise":
        return randn(*shape) * 1e-3
    if kind == "strong":   # few directions over a floor
        k = min(r, c, 32)
        w = torch.arange(1, k + 1, device="cuda").float() ** -0.5
        return ((randn(*shape[:-1], k) * w) @ randn(*shape[:-2], k, c) + randn(*shape)) * 1e-3
    k = max(1, min(r, c) // 8)   # "low": most singular values are zero
    return randn(*shape[:-1], k) @ randn(*shape[:-2], k, c)


def relative(x, ref):
    return float(((x.double() - ref).norm() / ref.norm()).cpu())


SHAPES = [(1, 1), (1, 7), (5, 3), (2, 16, 7168), (16, 33), (3, 64, 64), (4, 65, 200), (333, 1001), (2, 777, 129),
          (256, 7168), (3, 300, 256), (640, 640), (2, 129, 1024), (1000, 520), (16, 30001), (60, 7168), (2, 9000, 40)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["noise", "strong", "low"])
def test_update_is_orthogonalised(cuda_ok, shape, kind):
    grad = inputs(kind, shape, 5)
    p = torch.zeros(shape, device="cuda")
    op = P.Muon([p], [grad], lr=1.0, weight_decay=0.0, momentum=0.0, nesterov=False, update_scale="spectral")
    op.step()
    assert op.device_status() == 0
    x = -p / factor("spectral", *shape[-2:])
    ref = orthogonal(grad.double(), 5, 1e-7)
    e32 = relative(orthogonal(grad, 5, 1e-7), ref)
    bound = 8 * e32 + max(shape[-2:]) / 4 * 2.0 ** -24 + 2.0 ** -18
    e = relative(x, ref)
    print(shape, kind, "error %.2g, 32 bits %.2g, bound %.2g" % (e, e32, bound))
    assert e <= bound


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("kind", ["rms", "spectral"])
def test_step(cuda_ok, bf16, nesterov, kind):
    """Several tensors of several shapes, momenta, decay, copies, a gradient scale; two steps."""
    shapes = [(3, 48, 100), (100, 48), (77, 200), (2, 130, 70), (48, 100), (0, 5, 5)]
    g = torch.Generator(device="cuda").manual_seed(3)
    params = [torch.randn(s, generator=g, device="cuda") * 0.02 for s in shapes]
    state = [torch.randn(s, generator=g, device="cuda") * 1e-3 for s in shapes]
    copies = [torch.zeros(s, device="cuda", dtype=torch.bfloat16) for s in shapes]
    scale = torch.tensor(0.5, device="cuda")
    want = [(p.double(), m.double()) for p, m in zip(params, state)]
    lr, wd, mu = 0.02, 0.1, 0.9
    op = None
    for step in range(2):
        grads = [inputs("strong", s, 10 * step + i).to(torch.bfloat16 if bf16 else torch.float32) if 0 not in s
                 else torch.zeros(s, device="cuda", dtype=torch.bfloat16 if bf16 else torch.float32)
                 for i, s in enumerate(shapes)]
        if op is None:
            op = P.Muon(params, grads, copies=copies, state=state, lr=lr, weight_decay=wd, momentum=mu,
                        nesterov=nesterov, update_scale=kind)
            op.step(grad_scale=scale)
        else:
            op.step(grads, grad_scale=scale)
        new = []
        for (p, m), gr in zip(want, grads):
            if not p.numel():
                new.append((p, m))
                continue
            gr = gr.double() * 0.5
            m = mu * m + (1 - mu) * gr
            u = mu * m + (1 - mu) * gr if nesterov else m
            o = orthogonal(u, 5, 1e-7)
            new.append((p * (1 - lr * wd) - lr * factor(kind, *p.shape[-2:]) * o, m))
        want = new
    assert op.device_status() == 0
    for p, m, c, (wp, wm) in zip(params, state, copies, want):
        if not p.numel():
            continue
        # m: two roundings a step; p: the update is at most 0.25 of p, its error 1e-4 of it
        assert relative(m, wm) <= 2.0 ** -22
        assert relative(p, wp) <= 4e-5
        assert torch.equal(c, p.to(torch.bfloat16))
