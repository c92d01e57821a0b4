"""Orthogonalised steps whose m x m products share one launch (few matrices with a
short side of 65 to 384), beside those that take a launch each.  Tolerances:
test_gpu_muon.py's."""
import pytest
import torch

import precision_moe_grouped_gb300 as P
import test_gpu_muon as M

pytestmark = pytest.mark.gpu


def step(grads, steps=5):
    """X of every gradient, from one step."""
    params = [torch.zeros_like(g) for g in grads]
    op = P.Muon(params, grads, lr=1.0, weight_decay=0.0, momentum=0.0, nesterov=False, ns_steps=steps,
                update_scale="spectral")
    op.step()
    assert op.device_status() == 0
    return [-p / M.factor("spectral", *p.shape[-2:]) for p in params]


def check(x, grad, steps=5):
    ref = M.orthogonal(grad.double(), steps, 1e-7)
    e32 = M.relative(M.orthogonal(grad, steps, 1e-7), ref)
    assert M.relative(x, ref) <= 8 * e32 + max(grad.shape[-2:]) / 4 * 2.0 ** -24 + 2.0 ** -18


# one shape to four; the last tile's columns 64 to 256; the first size beyond; matrices of every cluster and too many
SETS = [[(65, 66)], [(128, 600)], [(3, 192, 200)], [(257, 300)], [(320, 321)], [(384, 2000)], [(385, 400)],
        [(100, 300), (300, 257), (384, 500), (130, 129)], [(100, 300), (600, 65), (250, 251), (200, 90), (70, 71)],
        [(2, 65, 384), (2, 384, 65), (384, 384)], [(7, 200, 256)], [(9, 300, 310)], [(20, 128, 130)], [(40, 70, 80)]]


@pytest.mark.parametrize("shapes", SETS, ids=str)
def test_sets_of_shapes(cuda_ok, shapes):
    grads = [M.inputs("strong", s, 7 + i) for i, s in enumerate(shapes)]
    got = step(grads)
    for x, g in zip(got, grads):
        check(x, g)
    for x, y in zip(got, step(grads)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 7])
@pytest.mark.parametrize("side", [100, 300])
def test_one_launch_or_many(cuda_ok, side, steps):
    """A matrix's result does not depend on how many others there are: 60 are more than the GPU holds clusters of.
    (The long side is too short for its sum to be shared out, so that both ways add in the same order.)"""
    grads = M.inputs("strong", (60, side, 310), 11)
    many = step([grads], steps)[0]
    for z in (0, 31, 59):
        one = step([grads[z]], steps)[0]
        assert torch.equal(one, many[z]), z
        check(one, grads[z], steps)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_matrices_keep_to_themselves(cuda_ok, bad):
    grads = M.inputs("noise", (4, 300, 320), 5)
    clean = step([grads])[0]
    grads[1, 7, 9] = bad
    got = step([grads])[0]
    assert torch.isnan(got[1]).all()
    for z in (0, 2, 3):
        assert torch.equal(got[z], clean[z])


def test_two_streams(cuda_ok):
    """Clusters of both sizes from two streams at once, and among other work."""
    sets = [[(3, 333, 400)], [(5, 100, 700), (256, 900)]]
    grads = [[M.inputs("strong", s, 3) for s in shapes] for shapes in sets]
    want = [step(g) for g in grads]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for g, st in zip(grads, streams):
            with torch.cuda.stream(st):
                got.append(step(g))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
