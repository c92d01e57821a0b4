"""Orthogonalised steps over more matrices of a shape than a slice of the workspace
holds (4 GiB): the same bits as in calls whose matrices fit into one."""
import pytest
import torch

import precision_moe_grouped_gb300 as P
import test_gpu_muon as M

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
MB = 1 << 20


def make(shapes, kind):
    grads = [M.inputs("strong", s, 20 + i).to(kind) for i, s in enumerate(shapes)]
    params = [M.inputs("noise", s, 30 + i) for i, s in enumerate(shapes)]
    state = [M.inputs("noise", s, 40 + i) * 1e-2 for i, s in enumerate(shapes)]
    return params, grads, state, [torch.zeros(s, device="cuda", dtype=BF16) for s in shapes]


def run(params, grads, state, copies):
    op = P.Muon(params, grads, copies=copies, state=state, lr=0.02)
    for _ in range(2):
        op.step()
    assert op.device_status() == 0
    return op


# a matrix of 100 x 310 takes 0.75 MB of workspace (planes of 128 x 320 twice, five of 128 x 128, 128 x 256, four bytes
# each), of 200 x 310 2.1, of 1100 x 1300 38: slices begin and end inside tensors, of both orientations
SETS = [[(2800, 100, 310), (3600, 310, 100), (1400, 100, 310)], [(2000, 310, 200), (1400, 200, 310)],
        [(68, 1100, 1300), (52, 1300, 1100)], [(2800, 100, 310), (50, 500, 80), (3600, 310, 100), (70, 300)]]


@pytest.mark.parametrize("shapes", SETS, ids=str)
def test_slices_change_no_bit(cuda_ok, shapes):
    inputs = make(shapes, BF16 if len(shapes) == 3 else torch.float32)
    whole = [[t.clone() for t in group] for group in inputs]
    op = run(*whole)
    assert 2000 * MB < op._need < 4120 * MB
    # each tensor by itself, which is one slice
    for i, s in enumerate(shapes):
        part = [[group[i].clone()] for group in inputs]
        alone = run(*part)
        assert alone._need < 4000 * MB
        for got, want in zip(whole, part):
            assert torch.equal(got[i], want[0]), s


def test_many_slices_follow_the_formula(cuda_ok):
    """12000 matrices of three slices, among them the first and last of each: the update's error as test_gpu_muon.py's."""
    shape = (12000, 100, 310)
    grad = M.inputs("strong", shape, 3)
    p = torch.zeros(shape, device="cuda")
    op = P.Muon([p], [grad], lr=1.0, weight_decay=0.0, momentum=0.0, nesterov=False, update_scale="spectral")
    op.step()
    assert op.device_status() == 0
    pick = torch.tensor([0, 3999, 4000, 4001, 7999, 8000, 8001, 11999], device="cuda")
    x, g = -p[pick] / M.factor("spectral", 100, 310), grad[pick]
    ref = M.orthogonal(g.double(), 5, 1e-7)
    e32 = M.relative(M.orthogonal(g, 5, 1e-7), ref)
    assert M.relative(x, ref) <= 8 * e32 + 310 / 4 * 2.0 ** -24 + 2.0 ** -18
    # every matrix was met once: a step of size lr s X, whose norm is that of its neighbours
    norms = p.norm(dim=(1, 2))
    assert float(norms.min()) > 0.5 * float(norms.max())


def test_a_captured_step_of_several_slices(cuda_ok):
    shapes = [(2800, 100, 310), (3600, 310, 100)]
    eager, held = make(shapes, torch.float32), make(shapes, torch.float32)
    op = P.Muon(eager[0], eager[1], copies=eager[3], state=eager[2], lr=0.02)
    captured = P.Muon(held[0], held[1], copies=held[3], state=held[2], lr=0.02)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    for _ in range(2):
        op.step()
        graph.replay()
    for a, b in zip(eager, held):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
