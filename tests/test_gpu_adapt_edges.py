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


def formula(x, ids, a, b, scale, dout):
    """out (without a base), dx, da, db in 64 bits."""
    x, a, b, dout = x.double(), a.double(), b.double(), dout.double()
    out, dx = torch.zeros_like(dout), torch.zeros_like(x)
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for i in range(a.shape[0]):
        rows = torch.nonzero(ids == i).reshape(-1)
        s = scale[i].double()
        v, u = x[rows] @ a[i].T, s * (dout[rows] @ b[i])
        out[rows], dx[rows] = s * (v @ b[i].T), u @ a[i]
        da[i], db[i] = u.T @ x[rows], s * dout[rows].T @ v
    return out, dx, da, db


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,r", [(20, 8), (20, 24), (20, 16), (60, 72), (1100, 8), (1100, 40), (80, 72), (1100, 128)])
def test_infinities(T, r, kind):
    """An infinite x or dout: out and dx are infinite, with the formula's sign, or
    NaN where the formula's are (ranks that a kernel pads with zeros must not
    make NaN of them), da and db not finite where the formula's are not, and all
    else is what it was."""
    H, N, NA = 72, 64, 3
    g = torch.Generator(device=DEV).manual_seed(T + r)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)        # noqa: E731
    x, dout, ids = rnd(T, H).bfloat16(), rnd(T, N).to(kind), (torch.arange(T, device=DEV) % NA).to(torch.int32)
    a, b, scale = rnd(NA, r, H).bfloat16(), rnd(NA, N, r).bfloat16(), torch.rand(NA, generator=g, device=DEV) + 0.5
    # one sign throughout for some outputs, so that the formula gives infinities beside NaN
    a[:, :, 5], b[:, 1::2] = a[:, :, 5].abs(), b[:, 1::2].abs()
    b[:, 7], a[:, :, 2::3] = b[:, 7].abs(), a[:, :, 2::3].abs()
    op = P.LowRankAdapters(a, b, scale)
    clean = (op.forward(x, ids, out_dtype=kind),) + op.backward(dout, x, ids)
    for sign in (1, -1):
        xi, di = x.clone(), dout.clone()
        xi[4, 5], di[7, 7] = sign * float("inf"), sign * float("inf")
        out, dx, da, db = (op.forward(xi, ids, out_dtype=kind),) + op.backward(di, xi, ids)
        ref = formula(xi, ids, a, b, scale, di)
        assert bool(ref[0].isinf().any()) and bool(ref[1].isinf().any())
        for name, got, want, old in zip(("out", "dx"), (out, dx), ref, clean):
            assert torch.equal(got.isnan(), want.isnan()), name
            assert torch.equal(got.double()[want.isinf()], want[want.isinf()]), name
            assert torch.equal(got[want.isfinite()], old[want.isfinite()]), name
        for name, got, want, old in zip(("da", "db"), (da, db), ref[2:], clean[2:]):
            assert torch.equal(got.isfinite(), want.isfinite()), name
            assert torch.equal(got[want.isfinite()], old[want.isfinite()]), name


@pytest.mark.parametrize("E,T", [(64, 40), (256, 3000)])
def test_rare_experts(E, T):
    """Logits up to 80 below their row's largest: an exponential is within 2 +
    1.2 |z - max| units (2^-23) of it, its argument is rounded once (|z - max|
    2^-24), and 70 roundings of 2^-24 hold the sums over the experts and the
    products after them."""
    g = torch.Generator(device=DEV).manual_seed(E)
    z = -80 * torch.rand(T, E, generator=g, device=DEV)
    z[:, 0] = 0
    ids = torch.randint(0, E, (T, 2), generator=g, device=DEV).to(torch.int32)
    _, counts, dz = P.BalanceLoss(E, 2, coef=1.0)(z, ids)
    p = z.double().softmax(1)
    f = counts[0].double() * (E / (2 * T))
    dot = p @ f
    ref = p / T * (f - dot[:, None])
    tol = p / T * (f + dot[:, None]) * ((2 - 1.2 * z.double()) * 2.0 ** -23 + (70 - z.double()) * 2.0 ** -24)
    bad = (dz.double() - ref).abs() > tol + 1e-37
    assert not bool(bad.any()), int(bad.sum())
