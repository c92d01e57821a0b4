"""The AdamW step (moe_adamw_step) against its definition.

32-bit moments, in 64 bits: every result is a few float operations on float
scalars, each off by 2^-24 of its operands; 8 of them bound a moment, 32 the
step, each against the absolute values that went in.  8-bit moments: the step
is defined operation by operation in float, so that numpy's IEEE float32
reproduces codes and scales bit for bit."""
import numpy as np
import pytest
import torch

import precision_moe_grouped_gb300 as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HP = dict(lr=3e-3, betas=(0.9, 0.995), eps=1e-8, weight_decay=0.05)


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.set_device(0)


def tensors(sizes, kind, seed=0):
    g = torch.Generator().manual_seed(seed + len(sizes))
    p = [torch.randn(n, generator=g).to(DEV) for n in sizes]
    gr = [(torch.randn(n, generator=g) * 0.1 * torch.randn(n, generator=g).exp()).to(kind).to(DEV)
          for n in sizes]
    return p, gr


def ref32(p, g, m, v, t, gs=1.0):
    (b1, b2), lr = HP["betas"], HP["lr"]
    p, g, m, v = (x.double().cpu().numpy() for x in (p, g, m, v))
    g = g * gs
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    den = np.sqrt(v2 / (1 - b2 ** t)) + HP["eps"]
    p2 = p - lr * HP["weight_decay"] * p - lr / (1 - b1 ** t) * m2 / den
    u = 2.0 ** -24
    tm, tv = 8 * u * (np.abs(m) + np.abs(g)), 8 * u * (v + g * g)
    tp = 32 * u * (np.abs(p) + lr / (1 - b1 ** t) * (np.abs(m) + np.abs(g)) / den)
    return (p2, tp), (m2, tm), (v2, tv)


SIZES = [[1], [3, 4, 5], [255, 256, 257], [2047, 2048, 2049, 0, 1], [100003, 7, 64, 4096],
         [n % 37 + 1 for n in range(450)], [1 << 20, 12345]]


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_float_moments(sizes, kind):
    p, g = tensors(sizes, kind)
    copies = [torch.zeros(n, dtype=torch.bfloat16, device=DEV) for n in sizes]
    opt = P.AdamW(p, g, copies=copies, **HP)
    for t in (1, 2, 3):
        before = [[x.clone() for x in xs] for xs in (p, opt.state["m"], opt.state["v"])]
        opt.step()
        for i in range(len(sizes)):
            ref = ref32(before[0][i], g[i], before[1][i], before[2][i], t)
            for got, (r, tol) in zip((p[i], opt.state["m"][i], opt.state["v"][i]), ref):
                assert (np.abs(got.double().cpu().numpy() - r) <= tol).all(), (i, t)
            assert torch.equal(copies[i], p[i].bfloat16())


def np_codes(x, positive):
    """(codes, scales) of float32 x in blocks of 256, as include/moe.h says."""
    n = len(x)
    blocks = -(-n // 256)
    pad = np.zeros(blocks * 256, np.float32)
    pad[:n] = x
    b = pad.reshape(blocks, 256)
    amax = np.abs(b).max(1)
    some = ~(amax < np.float32(2.0 ** -100))
    with np.errstate(divide="ignore"):
        inv = np.where(some, np.float32(448) / amax, np.float32(0)).astype(np.float32)
    scale = np.where(some, amax / np.float32(448), np.float32(1)).astype(np.float32)
    q = (b * inv[:, None]).astype(np.float32)
    codes = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    if positive:
        codes = np.where((codes == 0) & (b > 0) & some[:, None], 1, codes).astype(np.uint8)
    return codes.reshape(-1)[:n], scale


def np_decode(codes, scale):
    val = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    return val * np.repeat(scale, 256)[:len(codes)]


def ref8(p, g, mc, ms, vc, vs, t):
    f = np.float32
    (b1, b2), lr = HP["betas"], HP["lr"]
    m, r = np_decode(mc, ms), np_decode(vc, vs)
    m = m * f(b1) + g * f(1 - b1)
    v = (r * r) * f(b2) + (g * g) * f(1 - b2)
    r = np.sqrt(v)
    den = r * f(1 / np.sqrt(1 - b2 ** t)) + f(HP["eps"])
    p = p * f(1 - lr * HP["weight_decay"]) - (m * f(lr / (1 - b1 ** t))) / den
    return p, np_codes(m, False), np_codes(r, True)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_eight_bit_moments(sizes, kind):
    p, g = tensors(sizes, kind)
    opt = P.AdamW(p, g, state_bits=8, **HP)
    cpu = lambda t: t.view(torch.uint8).cpu().numpy() if t.element_size() == 1 else t.float().cpu().numpy()  # noqa: E731
    for t in (1, 2, 3):
        before = [[cpu(opt.state[k][i]).copy() for k in ("m", "m_scale", "v", "v_scale")] + [cpu(p[i]).copy()]
                  for i in range(len(sizes))]
        opt.step()
        for i in range(len(sizes)):
            mc, ms, vc, vs, pp = before[i]
            rp, (rmc, rms), (rvc, rvs) = ref8(pp, cpu(g[i]), mc, ms, vc, vs, t)
            np.testing.assert_array_equal(cpu(opt.state["m"][i]), rmc)
            np.testing.assert_array_equal(cpu(opt.state["v"][i]), rvc)
            np.testing.assert_array_equal(cpu(opt.state["m_scale"][i]), rms)
            np.testing.assert_array_equal(cpu(opt.state["v_scale"][i]), rvs)
            np.testing.assert_array_equal(cpu(p[i]), rp)


def test_eight_bits_follow_thirty_two():
    """50 steps on noisy gradients end near the float moments' parameters: the
    update's error is the moments' 3 bits of mantissa, at most 1/8 a step."""
    n = 5000
    g = torch.Generator(device=DEV).manual_seed(1)
    mean = torch.randn(n, generator=g, device=DEV) * 0.1
    p32 = torch.zeros(n, device=DEV)
    p8, gr = p32.clone(), torch.empty(n, device=DEV)
    a = P.AdamW([p32], [gr], weight_decay=0.0, lr=1e-2)
    b = P.AdamW([p8], [gr], weight_decay=0.0, lr=1e-2, state_bits=8)
    for _ in range(50):
        gr.copy_(mean + 0.05 * torch.randn(n, generator=g, device=DEV))
        a.step()
        b.step()
    assert float((p8 - p32).norm() / p32.norm()) < 0.125


def test_small_roots_do_not_vanish():
    """A block with one large gradient: the others' second moments are far
    below it, and their parameters still move by no more than the step."""
    g = torch.full((256,), 1e-9, device=DEV)
    g[0] = 1.0
    p = torch.zeros(256, device=DEV)
    opt = P.AdamW([p], [g], state_bits=8, lr=1e-3, weight_decay=0.0)
    for _ in range(20):
        opt.step()
    assert bool((opt.state["v"][0].view(torch.uint8) != 0).all())
    assert float(p.abs().max()) <= 20 * 1.01e-3


def test_zero_and_nonfinite_gradients():
    for bits in (32, 8):
        p, g = [torch.ones(600, device=DEV)], [torch.zeros(600, device=DEV)]
        opt = P.AdamW(p, g, state_bits=bits, lr=0.1, weight_decay=0.0)
        opt.step()
        assert bool((p[0] == 1).all())
        g[0][300] = float("nan")
        opt.step()
        bad = p[0].isnan()
        assert bool(bad[300]) and int(bad.sum()) == 1
        opt.step()
        bad = p[0].isnan()
        assert bool(bad[300]) and not bool(bad[:256].any()) and not bool(bad[512:].any())
        assert int(bad.sum()) == (1 if bits == 32 else 256)      # its block


def test_grad_scale_and_resume():
    p, g = tensors([1000, 33], torch.float32)
    q = [t.clone() for t in p]
    s = torch.tensor([0.25], device=DEV)
    a = P.AdamW(p, g, **HP)
    b = P.AdamW(q, [t * 0.25 for t in g], **HP)
    a.step(grad_scale=s)
    b.step()
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    c = P.AdamW(q, b.grads, state=b.state, steps_done=b.steps_done, **HP)
    a.step(grad_scale=s)
    c.step()
    assert all(torch.equal(x, y) for x, y in zip(p, q)) and c.steps_done == 2


def test_unaligned_tensors():
    """Views that begin anywhere give what aligned ones give."""
    sizes = [1000, 515]
    for bits in (32, 8):
        for kind in (torch.float32, torch.bfloat16):
            p, g = tensors(sizes, kind)
            q = [torch.empty(n + 3, device=DEV)[3:] for n in sizes]
            h = [torch.empty(n + 1, dtype=kind, device=DEV)[1:] for n in sizes]
            for x, y in zip(q + h, p + g):
                x.copy_(y)
            a = P.AdamW(p, g, state_bits=bits, **HP)
            b = P.AdamW(q, h, state_bits=bits, **HP)
            for _ in range(2):
                a.step()
                b.step()
            assert all(torch.equal(x, y) for x, y in zip(p, q))


def test_stream_graph_and_new_gradients():
    p, g = tensors([4000, 77], torch.float32)
    q = [t.clone() for t in p]
    a, b = P.AdamW(p, g, **HP), P.AdamW(q, [torch.zeros_like(t) for t in g], **HP)
    a.step()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b.step(grads=g)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(step=2)
    graph.replay()
    a.step(step=2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(p, q))


def test_refusals():
    p, g = tensors([100, 20], torch.float32)
    good = dict(HP)
    bad = [
        lambda: P.AdamW([t.bfloat16() for t in p], g),
        lambda: P.AdamW(p, g[:1]),
        lambda: P.AdamW(p, [g[0], g[1].bfloat16()]),
        lambda: P.AdamW(p, [g[0], g[1][:5]]),
        lambda: P.AdamW(p, [t.half() for t in g]),
        lambda: P.AdamW([t.cpu() for t in p], g),
        lambda: P.AdamW(p, g, state_bits=16),
        lambda: P.AdamW([p[0], p[0]], [g[0], g[0]]),
        lambda: P.AdamW(p, g, copies=[t.clone() for t in p]),
        lambda: P.AdamW(p, g, state={"m": p, "v": p[:1]}),
        lambda: P.AdamW(p, g, state_bits=8, state={"m": g, "v": g}),
        lambda: P.AdamW([torch.zeros(4, 4, device=DEV).t()[:2]], [torch.zeros(2, 4, device=DEV)]),
        lambda: P.AdamW(p, g, **good).step(step=0),
        lambda: P.AdamW(p, g, betas=(1.0, 0.9)).step(),
        lambda: P.AdamW(p, g, lr=float("nan")).step(),
        lambda: P.AdamW(p, g, eps=-1.0).step(),
        lambda: P.AdamW(p, g).step(grad_scale=torch.ones(2, device=DEV)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(P.MoeError):
            call()
            pytest.fail(f"refusal {i} did not come")
