"""Orthogonalised steps of matrices with a short side of up to 64, in packs of four
elements where the memory allows it and element by element elsewhere: the same
arithmetic in the same order, so the same bits."""
import pytest
import torch

import precision_moe_grouped_gb300 as P
import test_gpu_muon as M

pytestmark = pytest.mark.gpu


def off_by(t, n):
    """The same values n elements behind a 256-byte boundary."""
    room = torch.zeros(t.numel() + n, dtype=t.dtype, device="cuda")
    room[n:].copy_(t.flatten())
    return room[n:].view(t.shape)


def steps(shape, bf16, nesterov, offset):
    kind = torch.bfloat16 if bf16 else torch.float32
    grad = off_by(M.inputs("strong", shape, 3).to(kind), offset)
    param = off_by(M.inputs("noise", shape, 4), offset)
    copy = off_by(torch.zeros(shape, device="cuda", dtype=torch.bfloat16), offset)
    state = off_by(M.inputs("noise", shape, 6) * 1e-2, offset)
    op = P.Muon([param], [grad], copies=[copy], state=[state], lr=0.02, nesterov=nesterov)
    for _ in range(2):
        op.step()
    assert op.device_status() == 0
    return param, state, copy


# wide and tall, the last pack of a tile's and of the matrix's, one pack in all, rows that fill their class or not;
# (8, 70000) and (64, 20000) do not fit into a cluster's shared memory
SHAPES = [(1, 4), (16, 4), (5, 8), (3, 16, 260), (2, 260, 16), (2, 300, 12), (3, 20, 516), (2, 1001, 32), (1001, 28), (40, 132), (4, 64, 200),
          (3, 333, 64), (257, 60), (8, 70000), (70001, 8), (64, 20000), (9999, 36)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("nesterov", [False, True])
def test_packs_and_single_elements(cuda_ok, shape, bf16, nesterov):
    packs = steps(shape, bf16, nesterov, 0)
    for offset in (1, 2, 4):   # (two and four elements: aligned for some of the types)
        for x, y in zip(packs, steps(shape, bf16, nesterov, offset)):
            assert torch.equal(x, y), offset


def test_tensors_of_both_kinds(cuda_ok):
    """A launch holds several tensors; one that is met element by element takes the others with it."""
    shapes = [(3, 16, 400), (16, 333), (4, 900, 12), (7, 30)]
    grads = [M.inputs("strong", s, 5) for s in shapes]

    def run(which):
        params = [torch.zeros(shapes[i], device="cuda") for i in which]
        op = P.Muon(params, [grads[i] for i in which], lr=1.0, weight_decay=0.0)
        op.step()
        assert op.device_status() == 0
        return params

    together = run(range(len(shapes)))
    for i, p in enumerate(together):
        assert torch.equal(p, run([i])[0]), shapes[i]


def test_long_matrix_among_many(cuda_ok):
    """Beside many others it is shared out as it is alone: together they take no longer than apart, by a wide margin
    (one block for 2^20 columns took 30 times as long), and come out by the formula."""
    shapes = [(400, 64, 7168), (64, 1 << 20)]
    grads = [M.inputs("strong", s, 9) for s in shapes]

    def run(which):
        params = [torch.zeros(shapes[i], device="cuda") for i in which]
        op = P.Muon(params, [grads[i] for i in which], lr=1.0, weight_decay=0.0, momentum=0.0, nesterov=False,
                    update_scale="spectral")
        op.step()
        first = [-p.clone() for p in params]
        times = []
        for _ in range(3):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            op.step()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        assert op.device_status() == 0
        return min(times), first

    together, x = run([0, 1])
    assert together <= 4 * (run([0])[0] + run([1])[0])
    for got, grad, s in zip(x, grads, shapes):
        got, grad = (t[::57] if len(s) == 3 else t for t in (got, grad))
        ref = M.orthogonal(grad.double(), 5, 1e-7)
        e32 = M.relative(M.orthogonal(grad, 5, 1e-7), ref)
        assert M.relative(got / M.factor("spectral", *s[-2:]), ref) <= 8 * e32 + s[-1] / 4 * 2.0 ** -24 + 2.0 ** -18


@pytest.mark.parametrize("shapes", [[(150, 16, 400), (8, 70000), (5, 1000, 12), (16, 200)],
                                    [(400, 32, 200), (2, 20, 40000), (150, 100, 20)]], ids=str)
def test_many_short_beside_long(cuda_ok, shapes):
    """Many matrices that stay in a cluster's shared memory, and one that is too long for it: neither changes a bit of
    the other's step."""
    grads = [M.inputs("strong", s, 5 + i) for i, s in enumerate(shapes)]

    def run(which):
        params = [M.inputs("noise", shapes[i], 3) for i in which]
        op = P.Muon(params, [grads[i] for i in which], lr=0.02)
        for _ in range(2):
            op.step()
        assert op.device_status() == 0
        return {(i, k): t for k, group in enumerate((params, op.state)) for i, t in zip(which, group)}

    every = range(len(shapes))
    together = run(every)
    for which in ([i for i in every if i != 1], [1]):
        for at, got in run(which).items():
            assert torch.equal(together[at], got), at


@pytest.mark.parametrize("mp,long", [(16, (8, 70000)), (32, (2, 24, 20000)), (64, (64, 20000))])
def test_few_short_beside_long(cuda_ok, mp, long):
    """Few of them go with the long one: by the formula."""
    shapes = [(3, mp, 400), long, (5, 1000, mp - 4), (mp, 200)]
    grads = [M.inputs("strong", s, 5 + i) for i, s in enumerate(shapes)]
    params = [torch.zeros(s, device="cuda") for s in shapes]
    op = P.Muon(params, grads, lr=1.0, weight_decay=0.0, momentum=0.0, nesterov=False, update_scale="spectral")
    op.step()
    assert op.device_status() == 0
    for p, grad, s in zip(params, grads, shapes):
        ref = M.orthogonal(grad.double(), 5, 1e-7)
        e32 = M.relative(M.orthogonal(grad, 5, 1e-7), ref)
        bound = 8 * e32 + max(s[-2:]) / 4 * 2.0 ** -24 + 2.0 ** -18
        assert M.relative(-p / M.factor("spectral", *s[-2:]), ref) <= bound, s


def test_an_odd_tensor_beside_many(cuda_ok):
    """One that cannot be met in packs: the others' step is the same to the bit, and takes no longer for it but for one
    more launch (a quarter, when all went by single elements)."""
    shapes = [(600, 16, 4096), (16, 333)]
    grads = [M.inputs("strong", s, 5 + i) for i, s in enumerate(shapes)]

    def run(which):
        params = [M.inputs("noise", shapes[i], 3) for i in which]
        op = P.Muon(params, [grads[i] for i in which], lr=0.02)
        op.step()
        first = [p.clone() for p in params]
        times = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                op.step()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        assert op.device_status() == 0
        return min(times), first

    together, x = run([0, 1])
    alone, pool = run([0])
    assert torch.equal(x[0], pool[0]) and torch.equal(x[1], run([1])[1][0])
    assert together <= 1.12 * alone, (together, alone)
