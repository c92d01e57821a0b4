"""The gated feed-forward block and the orthogonalised step where they can go
wrong: strides, memory in place, empty and non-finite inputs, streams, graphs,
long offsets, odd alignments, many tensors.  Tolerances: test_gpu_ffn.py's and
test_gpu_muon.py's, whose helpers are used."""
import importlib.util
import math
import os

import pytest
import torch

import precision_moe_grouped_gb300 as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load(name, folder="tests"):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, folder, name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


F, M = load("test_gpu_ffn"), load("test_gpu_muon")
pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
TOKENS = [1, 24, 33, 200, 256, 257, 700]       # every path: streamed weights, shares of K, tiles


def block(T, H=4104, I=264, seed=1):
    s = F.make(T, H, I, seed=seed)
    return s, P.GatedFFN(s["wgu"], s["wd"])


# ------------------------------------------------------- feed-forward block
@pytest.mark.parametrize("T", TOKENS)
def test_strides_and_neighbours(cuda_ok, T):
    """Strided inputs and outputs give the same bits, and what lies between and
    behind the rows stays as it was."""
    s, op = block(T)
    H = 4104
    wide = {k: torch.full((T + 5, H + 40), 7.0, device="cuda", dtype=BF16) for k in ("x", "base", "dout", "dx_base")}
    for k, t in wide.items():
        t[:T, 16:16 + H] = s[k]
    at = {k: t[:T, 16:16 + H] for k, t in wide.items()}
    want = op(s["x"], base=s["base"])
    out = torch.full((T + 5, H + 24), -3.0, device="cuda", dtype=BF16)
    op(at["x"], base=at["base"], out=out[:T, 8:8 + H])
    assert torch.equal(out[:T, 8:8 + H], want)
    assert (out[T:] == -3).all() and (out[:, :8] == -3).all() and (out[:, 8 + H:] == -3).all()
    want = op.backward(s["dout"], s["x"], dx_base=s["dx_base"])
    dx = torch.full((T + 5, H + 24), -3.0, device="cuda", dtype=BF16)
    flat = [torch.full((n + 64,), -3.0, device="cuda", dtype=BF16) for n in (2 * 264 * H, H * 264)]
    got = op.backward(at["dout"], at["x"], dx_base=at["dx_base"], dx=dx[:T, 8:8 + H],
                      dw_gate_up=flat[0][:2 * 264 * H].view(2 * 264, H), dw_down=flat[1][:H * 264].view(H, 264))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (dx[T:] == -3).all() and (dx[:, :8] == -3).all() and (dx[:, 8 + H:] == -3).all()
    assert all((t[-64:] == -3).all() for t in flat)
    for k, t in wide.items():                                            # inputs untouched
        assert (t[T:] == 7).all() and (t[:, :16] == 7).all() and torch.equal(at[k], s[k])


@pytest.mark.parametrize("T", TOKENS)
def test_in_place_and_parts(cuda_ok, T):
    s, op = block(T)
    want = op(s["x"], base=s["base"])
    base = s["base"].clone()
    assert op(s["x"], base=base, out=base) is base and torch.equal(base, want)
    x = s["x"].clone()
    assert torch.equal(op(x, base=s["base"], out=x), want)
    full = op.backward(s["dout"], s["x"], dx_base=s["dx_base"])
    dx = s["dx_base"].clone()
    got = op.backward(s["dout"], s["x"], dx_base=dx, dx=dx)
    assert got[0] is dx and torch.equal(dx, full[0])
    a = op.backward(s["dout"], s["x"], need_dx=False)
    assert a[0] is None and torch.equal(a[1], full[1]) and torch.equal(a[2], full[2])
    b = op.backward(s["dout"], s["x"], dx_base=s["dx_base"], need_weights=False)
    assert b[1] is None and b[2] is None and torch.equal(b[0], full[0])


def test_without_tokens(cuda_ok):
    _, op = block(1)
    x = torch.empty((0, 4104), device="cuda", dtype=BF16)
    assert op(x).shape == (0, 4104)
    dw = [torch.ones((2 * 264, 4104), device="cuda", dtype=BF16), torch.ones((4104, 264), device="cuda", dtype=BF16)]
    dx, a, b = op.backward(x, x, dw_gate_up=dw[0], dw_down=dw[1])
    assert dx.shape == (0, 4104) and not a.any() and not b.any()


@pytest.mark.parametrize("T", TOKENS[1:])
def test_non_finite_tokens_keep_to_themselves(cuda_ok, T):
    """A NaN or an infinity in one token's x (or dout) reaches that token's out and
    dx, and no other's."""
    s, op = block(T)
    out, dx = op(s["x"], base=s["base"]), op.backward(s["dout"], s["x"], need_weights=False)[0]
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    for t in {0, T // 2, T - 1}:
        for bad in (float("nan"), float("inf")):
            x, dout = s["x"].clone(), s["dout"].clone()
            x[t, 3] = bad
            others.fill_(True)
            others[t] = False
            got = op(x, base=s["base"])
            assert torch.equal(got[others], out[others]) and not torch.isfinite(got[t].float()).all()
            assert torch.equal(op.backward(s["dout"], x, need_weights=False)[0][others], dx[others])
            dout[t, 3] = bad
            got = op.backward(dout, s["x"], need_weights=False)[0]
            assert torch.equal(got[others], dx[others]) and not torch.isfinite(got[t].float()).all()


@pytest.mark.parametrize("T", [5, 100, 300])
def test_saturated_gates(cuda_ok, T):
    """Gates of some hundreds: silu is 0 or the gate itself, its derivative 0 or 1."""
    s, op = block(T)
    s["x"] = (s["x"].float() * 300).to(BF16)
    want = F.reference(s)
    F.close(op(s["x"], base=s["base"]), want[0], "out")
    for a, b, name in zip(op.backward(s["dout"], s["x"], dx_base=s["dx_base"]), want[1:], ("dx", "dwgu", "dwd")):
        F.close(a, b, name)


@pytest.mark.parametrize("T", [7, 150, 400])
def test_gradients_against_differences(cuda_ok, T):
    """Along a random direction of x and of each weight, the gradient's slope is that of
    the formula in 64 bits, (f(p + e v) - f(p - e v)) / 2 e of f = sum of dout * out.
    The slope's error is at most |v| |error of the gradient|, held to u |v| |gradient|
    (u = 2^-8, as the gradients' own test), and e^2 of the third derivative."""
    s, op = block(T, 136, 72)
    s["base"] = s["dx_base"] = None
    got = dict(zip(("x", "wgu", "wd"), op.backward(s["dout"], s["x"])))
    g = torch.Generator(device="cuda").manual_seed(9)

    def f(**moved):
        t = {k: s[k].double() for k in ("x", "wgu", "wd")} | moved
        gate, up = (t["x"] @ t["wgu"].T).chunk(2, dim=1)
        return (s["dout"].double() * ((gate * torch.sigmoid(gate) * up) @ t["wd"].T)).sum()

    for k, grad in got.items():
        v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-4
        slope = (f(**{k: s[k].double() + e * v}) - f(**{k: s[k].double() - e * v})) / (2 * e)
        off = (slope - (grad.double() * v).sum()).abs()
        assert off <= 2.0 ** -8 * v.norm() * grad.double().norm() + 1e-6 * slope.abs(), k


@pytest.mark.parametrize("T", TOKENS)
def test_streams(cuda_ok, T):
    """Calls on two streams at once, inputs made on them just before: each on its own workspace."""
    H, I = 2048, 1024
    ops = [block(T, H, I, seed=i) for i in range(2)]
    want = [(op(s["x"], base=s["base"]), *op.backward(s["dout"], s["x"])) for s, op in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, (s, op) in enumerate(ops):
            with torch.cuda.stream(streams[i]):
                x, dout = s["x"] * 1, s["dout"] * 1
                got[i] = (op(x, base=s["base"]), *op.backward(dout, x))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("T", TOKENS)
def test_graph(cuda_ok, T):
    """Forward and backward captured (the first call of this size, so nothing is set up
    outside) and replayed with new inputs and weights, beside another graph."""
    a, b = F.make(T, 4104, 264, seed=1), F.make(T, 4104, 264, seed=2)
    op = P.GatedFFN(a["wgu"].clone(), a["wd"].clone())
    held = {k: a[k].clone() for k in ("x", "base", "dout")}
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((op(held["x"], base=held["base"]), *op.backward(held["dout"], held["x"])))
        graphs.append(g)
    for s in (a, b, a):
        for k, t in held.items():
            t.copy_(s[k])
        op.w_gate_up.copy_(s["wgu"])
        op.w_down.copy_(s["wd"])
        for g in graphs:
            g.replay()
        eager = P.GatedFFN(s["wgu"], s["wd"])
        want = (eager(s["x"], base=s["base"]), *eager.backward(s["dout"], s["x"]))
        for got in outs:
            for x, y in zip(got, want):
                assert torch.equal(x, y)


@pytest.mark.parametrize("T", [20, 200, 300])
def test_chain_without_waits(cuda_ok, T):
    """Each call reads what the one before writes: waiting between them changes nothing.
    (Brought back to 1 in between: the block is quadratic in large x, and would overflow bf16.)"""
    s, op = block(T, 1024, 512)

    def run(wait):
        x = s["x"]
        for _ in range(6):
            x = op(x, base=x)
            wait()
            x = x / x.abs().max()
            dx, dwgu, dwd = op.backward(x, x)
            wait()
            dx = dx / dx.abs().max()
            x = op(dx, base=s["base"], out=dx)
            wait()
        assert torch.isfinite(x.float()).all()
        return x, dwgu, dwd

    for a, b in zip(run(lambda: None), run(torch.cuda.synchronize)):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(cuda_ok):
    """x, out, dout and dx of more than 2^31 elements."""
    H, I, T = 16384, 64, 135000
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty((T, H), device="cuda", dtype=BF16)
    part = torch.randn((1000, H), generator=g, device="cuda").to(BF16)
    for i in range(0, T, 1000):
        x[i:i + 1000] = part
    assert x.numel() > 1 << 31
    wgu = (torch.randn((2 * I, H), generator=g, device="cuda") / math.sqrt(H)).to(BF16)
    wd = (torch.randn((H, I), generator=g, device="cuda") / math.sqrt(I)).to(BF16)
    op = P.GatedFFN(wgu, wd)
    want = op(part, base=part)
    out = op(x, base=x)
    for i in range(0, T, 1000):                       # the same rows everywhere, to the last
        assert torch.equal(out[i:i + 1000], want), i
    del out
    want = op.backward(part, part, dx_base=part, need_weights=False)[0]
    dx = op.backward(x, x, dx_base=x, need_weights=False)[0]
    for i in range(0, T, 1000):
        assert torch.equal(dx[i:i + 1000], want), i
    assert op.device_status() == 0


# ------------------------------------------------------ orthogonalised step
def one(p, grad, **kw):
    op = P.Muon([p], [grad], **kw)
    op.step()
    assert op.device_status() == 0
    return op


@pytest.mark.parametrize("shape", [(4, 16, 48), (3, 100, 90), (2, 60, 7168)], ids=str)
def test_nothing_to_learn(cuda_ok, shape):
    """Zero gradients and momenta: the parameters decay, nothing else."""
    p = torch.randn(shape, device="cuda")
    want = p * torch.tensor(1 - 0.5 * 0.25, device="cuda")
    op = one(p, torch.zeros(shape, device="cuda"), lr=0.5, weight_decay=0.25)
    assert torch.equal(p, want) and not op.state[0].any()


@pytest.mark.parametrize("shape", [(4, 16, 48), (5, 100, 90), (4, 60, 7168), (6, 70, 260)], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_matrices_keep_to_themselves(cuda_ok, shape, bad):
    grad = M.inputs("strong", shape, 3)
    p, q = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    one(p, grad)
    broken = grad.clone()
    broken[2, 5, 7] = bad
    one(q, broken)
    assert torch.isnan(q[2]).all()
    for z in range(shape[0]):
        assert z == 2 or torch.equal(p[z], q[z])


@pytest.mark.parametrize("shape", [(16, 48), (3, 33, 100), (100, 90), (3, 65, 333), (333, 65)], ids=str)
@pytest.mark.parametrize("bf16", [False, True])
def test_alignment_and_neighbours(cuda_ok, shape, bf16):
    """Tensors that begin anywhere in a buffer: the same step, and the buffer around them stays as it was."""
    n = math.prod(shape)
    kind = torch.float32

    def odd(t, dtype):
        flat = torch.full((n + 20,), -3.0, device="cuda", dtype=dtype)
        flat[9:9 + n] = t.reshape(-1)
        return flat, flat[9:9 + n].view(shape)

    grad = M.inputs("strong", shape, 1).to(BF16 if bf16 else kind)
    m0, p0 = torch.randn(shape, device="cuda") * 1e-3, torch.randn(shape, device="cuda") * 0.02
    p, m, c = p0.clone(), m0.clone(), torch.empty(shape, device="cuda", dtype=BF16)
    P.Muon([p], [grad], copies=[c], state=[m], lr=0.02).step()
    buffers = [odd(p0, kind), odd(m0, kind), odd(torch.zeros(shape, device="cuda"), BF16), odd(grad, grad.dtype)]
    (_, pv), (_, mv), (_, cv), (_, gv) = buffers
    P.Muon([pv], [gv], copies=[cv], state=[mv], lr=0.02).step()
    assert torch.equal(mv, m) and torch.equal(cv, pv.to(BF16)) and torch.equal(gv, grad)
    # sums of u^2 in another order: the update moves by a few units of 2^-24, times what the steps make of it
    assert ((pv - p).norm() <= 1e-4 * (p - p0 * (1 - 0.02 * 0.1)).norm() + 2.0 ** -22 * p.norm())
    for flat, _ in buffers:
        assert (flat[:9] == -3).all() and (flat[9 + n:] == -3).all()


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7])
@pytest.mark.parametrize("coef", [M.NS, (2.0, -1.5, 0.5)])
def test_step_counts_and_coefficients(cuda_ok, steps, coef):
    for shape in ((24, 200), (2, 48, 20000), (70, 300), (2, 300, 129)):
        grad = M.inputs("strong", shape, 8)
        p = torch.zeros(shape, device="cuda")
        one(p, grad, lr=1.0, weight_decay=0.0, momentum=0.0, nesterov=False, update_scale="spectral", ns_steps=steps,
            ns_coefficients=coef)
        x = -p / M.factor("spectral", *shape[-2:])
        ref = M.orthogonal(grad.double(), steps, 1e-7, coef)
        e32 = M.relative(M.orthogonal(grad, steps, 1e-7, coef), ref)
        assert M.relative(x, ref) <= 8 * e32 + max(shape[-2:]) / 4 * 2.0 ** -24 + 2.0 ** -18, (shape, steps)


def test_many_tensors(cuda_ok):
    """More tensors of a shape than a launch holds, more shapes than share their launches,
    more small tensors than a table holds, matrices beyond a grid's 65535 and beyond what L2 keeps."""
    shapes = [(70 + i % 7, 90) for i in range(23)] + [(90, 70)] * 3 + [(3 + i % 30, 40 + i) for i in range(97)]
    shapes += [(70000, 2, 3), (4000, 65, 66), (17, 40, 33)]
    grads = [M.inputs("noise", s, i) for i, s in enumerate(shapes)]
    params = [torch.zeros(s, device="cuda") for s in shapes]
    op = P.Muon(params, grads, lr=1.0, weight_decay=0.0, momentum=0.5, nesterov=True, update_scale="rms")
    op.step()
    assert op.device_status() == 0
    for p, g, s in zip(params, grads, shapes):
        if len(s) == 3 and s[0] > 100:
            pick = torch.tensor([0, 1, s[0] // 2, s[0] - 2, s[0] - 1], device="cuda")
            p, g = p[pick], g[pick]
        u = (0.5 * 0.5 + 0.5) * g
        ref = M.orthogonal(u.double(), 5, 1e-7)
        e32 = M.relative(M.orthogonal(u, 5, 1e-7), ref)
        assert M.relative(-p / M.factor("rms", *s[-2:]), ref) <= 8 * e32 + max(s[-2:]) / 4 * 2.0 ** -24 + 2.0 ** -18, s


@pytest.mark.parametrize("shape", [(8, 1 << 20), (1 << 18, 70)], ids=str)
def test_long_sides(cuda_ok, shape):
    grad = M.inputs("noise", shape, 2)
    p = torch.zeros(shape, device="cuda")
    one(p, grad, lr=1.0, weight_decay=0.0, momentum=0.0, nesterov=False, update_scale="spectral")
    ref = M.orthogonal(grad.double(), 5, 1e-7)
    e32 = M.relative(M.orthogonal(grad, 5, 1e-7), ref)
    assert M.relative(-p / M.factor("spectral", *shape), ref) <= 8 * e32 + max(shape) / 4 * 2.0 ** -24 + 2.0 ** -18


SETS = [[(3, 16, 100), (40, 16)], [(2, 100, 300), (300, 100), (129, 65)], [(2, 60, 7168)]]


@pytest.mark.parametrize("shapes", SETS, ids=str)
def test_muon_repeats_streams_and_graphs(cuda_ok, shapes):
    """The same bits from run to run, on two streams at once, and from a captured step (of a first call) replayed."""
    grads = [M.inputs("strong", s, i) for i, s in enumerate(shapes)]

    def fresh():
        return P.Muon([torch.full(s, 0.01, device="cuda") for s in shapes], [g.clone() for g in grads],
                      copies=[torch.zeros(s, device="cuda", dtype=BF16) for s in shapes], lr=0.02)

    def tensors(op):
        return [t.clone() for group in (op.params, op.state, op.copies) for t in group]

    captured = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    one_, two = fresh(), fresh()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for op, st in zip((one_, two), streams):
            with torch.cuda.stream(st):
                op.step()
        graph.replay()
        torch.cuda.synchronize()
    for x, y, z in zip(tensors(one_), tensors(two), tensors(captured)):
        assert torch.equal(x, y) and torch.equal(x, z)
    # other gradients in the same memory
    for op in (one_, captured):
        for g in op.grads:
            g.mul_(-0.5)
            g[..., 0, :] += 1e-3
    one_.step()
    graph.replay()
    for x, z in zip(tensors(one_), tensors(captured)):
        assert torch.equal(x, z)


# ------------------------------------------------------------ all together
def test_shared_expert_example(cuda_ok):
    """The layer, the block and the optimiser in one loop (examples/train_shared_expert.py): its gradients are the
    formula's, it serves a token, and waiting after each call changes no bit."""
    ex = load("train_shared_expert", "examples")
    r = ex.run(steps=6, tokens=600)
    first = r["first"]
    s = {"x": first["x"], "dout": first["dout"], "wgu": first["weights"][0].reshape(512, 512),
         "wd": first["weights"][1], "base": None, "dx_base": None}
    want = F.reference(s)
    F.close(first["grads"][0].reshape(512, 512), want[2], "dw_gate_up")
    F.close(first["grads"][1], want[3], "dw_down")
    s = {"x": r["x"], "dout": r["x"], "wgu": r["weights"][0].reshape(512, 512), "wd": r["weights"][1],
         "base": r["routed"], "dx_base": None}
    F.close(r["out"], F.reference(s)[0], "served", few=True)
    waited = ex.run(steps=6, tokens=600, sync=True)
    assert r["loss"] == waited["loss"]
    for a, b in zip(r["masters"] + r["weights"] + [r["out"]], waited["masters"] + waited["weights"] + [waited["out"]]):
        assert torch.equal(a, b)


def test_steps_follow_the_formula_in_a_loop(cuda_ok):
    """Forward, backward and step three times over; each step's masters are the formula's for the gradients that the
    backward left, momentum included."""
    T, H, I = 300, 264, 136
    s = F.make(T, H, I, seed=4)
    masters = [torch.randn((2, I, H), device="cuda") / math.sqrt(H), torch.randn((H, I), device="cuda") / math.sqrt(I)]
    weights = [m.to(BF16) for m in masters]
    op = P.GatedFFN(weights[0].view(2 * I, H), weights[1])
    grads = [torch.empty_like(w) for w in weights]
    muon = P.Muon(masters, grads, copies=weights, lr=0.02, weight_decay=0.1, momentum=0.9)
    want = [(m.double(), torch.zeros_like(m, dtype=torch.float64)) for m in masters]
    for _ in range(3):
        out = op(s["x"], base=s["base"])
        F.close(out, F.reference(s | {"wgu": op.w_gate_up, "wd": op.w_down})[0], "out")
        op.backward(out, s["x"], dw_gate_up=grads[0].view(2 * I, H), dw_down=grads[1], need_dx=False)
        muon.step()
        new = []
        for (p, m), g in zip(want, grads):
            m = 0.9 * m + 0.1 * g.double()
            o = M.orthogonal(0.9 * m + 0.1 * g.double(), 5, 1e-7)
            new.append((p * (1 - 0.02 * 0.1) - 0.02 * M.factor("rms", *p.shape[-2:]) * o, m))
        want = new
        for p, w, (wp, _) in zip(masters, weights, want):
            # an update is at most 0.3 of p; its error 1e-4 of it (test_gpu_muon.py)
            assert M.relative(p, wp) <= 4e-5 and torch.equal(w, p.to(BF16))
