"""The router's balance loss (moe_balance_loss) against its definition in 64
bits.  Tolerances: the exponentials carry a few units in the last place and
the rounding of their argument, |z - max| 2^-24, below 2^-19 for the logits
here; the sums over experts and tokens run in float, at most 64 additions
deep.  2^-17 of the terms' absolute sum holds all of it, 2^-20 the gate part's
three roundings and its sum of at most 32 products."""
import numpy as np
import pytest
import torch

import precision_moe_grouped_gb300 as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.set_device(0)


def make(T, E, k, seed=0, masked=False, seqs=None, gates=False, drop=False):
    g = torch.Generator().manual_seed(seed + T + 3 * E + k)
    z = torch.randn(T, E, generator=g) * 2
    top = z.topk(k, dim=1)
    c = dict(logits=z, ids=top.indices.to(torch.int32), mask=None, seq_offsets=None, weights=None,
             dweights=None)
    if drop:
        c["ids"][::5, -1] = -1
        c["ids"][1::7, 0] = E + 3
        c["ids"][2::9, 0] = -2 ** 31
    if masked:
        c["mask"] = torch.rand(T, generator=g) < 0.7
    if seqs is not None:
        c["seq_offsets"] = torch.tensor(seqs, dtype=torch.int32)
    if gates:
        c["weights"] = top.values.softmax(1).contiguous()
        c["dweights"] = torch.randn(T, k, generator=g)
    return c


def reference(c, coef, z=None):
    z = (c["logits"] if z is None else z).double().numpy()
    ids = c["ids"].numpy()
    (T, E), k = z.shape, ids.shape[1]
    ok = np.ones(T, bool) if c["mask"] is None else c["mask"].numpy().astype(bool)
    offs = [0, T] if c["seq_offsets"] is None else c["seq_offsets"].tolist()
    S = len(offs) - 1
    rows = [np.arange(offs[s], offs[s + 1])[ok[offs[s]:offs[s + 1]]] for s in range(S)]
    live = max(1, sum(len(r) > 0 for r in rows))
    counts, loss = np.zeros((S, E), np.int64), 0.0
    dz, size = np.zeros((T, E)), np.zeros((T, E))
    for s, r in enumerate(rows):
        if not len(r):
            continue
        i = ids[r].reshape(-1)
        counts[s] = np.bincount(i[(i >= 0) & (i < E)], minlength=E)
        top = z[r].max(1, keepdims=True)
        e = np.exp(z[r] - np.where(np.isneginf(top), 0, top))
        tot = e.sum(1, keepdims=True)
        p = e / np.where(tot == 0, 1, tot)
        f = counts[s] * (E / (k * len(r)))
        loss += coef / live * float((f * p.mean(0)).sum())
        dot = (p @ f)[:, None]
        dz[r] = coef / (live * len(r)) * p * (f - dot)
        size[r] = abs(coef) / (live * len(r)) * p * (f + dot)
    gate = np.zeros((T, E))
    if c["weights"] is not None:
        w, dw = c["weights"].double().numpy(), c["dweights"].double().numpy()
        good = (ids >= 0) & (ids < E)
        w = np.where(good, w, 0)
        add = w * (dw - (w * dw).sum(1, keepdims=True))
        sz = w * (np.abs(dw) + (w * np.abs(dw)).sum(1, keepdims=True))
        t = np.broadcast_to(np.arange(T)[:, None], ids.shape)
        np.add.at(dz, (t[good], ids[good]), add[good])
        np.add.at(gate, (t[good], ids[good]), sz[good])
    return loss, counts, dz, size * 2.0 ** -17 + gate * 2.0 ** -20


def call(op, c, **kw):
    to = lambda t: None if t is None else t.to(DEV)               # noqa: E731
    return op(to(c["logits"]), to(c["ids"]), mask=to(c["mask"]), seq_offsets=to(c["seq_offsets"]),
              weights=to(c["weights"]), dweights=to(c["dweights"]), **kw)


def check(c, coef=0.01):
    op = P.BalanceLoss(c["logits"].shape[1], c["ids"].shape[1], coef)
    loss, counts, dz = call(op, c)
    ref_loss, ref_counts, ref_dz, tol = reference(c, coef)
    np.testing.assert_array_equal(counts.cpu().numpy(), ref_counts)
    assert abs(float(loss) - ref_loss) <= 2.0 ** -17 * abs(ref_loss)
    err = np.abs(dz.double().cpu().numpy() - ref_dz)
    assert (err <= tol + 1e-37).all(), float((err / np.maximum(tol, 1e-37)).max())
    again = call(op, c)
    assert all(torch.equal(p, q) for p, q in zip((loss, counts, dz), again))
    only = call(op, c, need_grad=False)
    assert only[2] is None and torch.equal(only[0], loss) and torch.equal(only[1], counts)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (5, 3), (8, 2), (16, 4), (31, 8), (33, 32), (64, 4),
                                 (127, 8), (256, 8), (258, 8), (384, 6), (512, 1), (1000, 8),
                                 (1024, 32)])
@pytest.mark.parametrize("T", [1, 2, 33, 700])
def test_sizes(T, E, k):
    check(make(T, E, k))
    check(make(T, E, k, masked=True, gates=True, drop=k > 1))


@pytest.mark.parametrize("seqs", [[0, 100], [0, 0, 40, 40, 41, 100, 100], [0, 33, 66, 100],
                                  [10, 20, 90], list(range(101))])
def test_sequences(seqs):
    """Ragged and empty ones; tokens of no sequence have no part in the loss."""
    check(make(100, 64, 4, seqs=seqs))
    check(make(100, 12, 2, seqs=seqs, masked=True, gates=True))


@pytest.mark.parametrize("E,k", [(8, 2), (16, 2), (30, 4), (64, 8), (200, 8), (256, 8), (384, 6), (1024, 4)])
def test_either_side_of_the_small_batches(E, k):
    """The largest batch that one kernel takes and the next one, masked and not,
    and one sequence that is a part of the batch."""
    lib = P.load()
    small = lambda T: lib.moe_balance_workspace_size(P._lib.BalanceShape(T, E, k, 1, 1.0)) == 256  # noqa: E731
    T = max(t for t in range(1, 4000) if small(t))
    for n in (T, T + 1):
        check(make(n, E, k))
        check(make(n, E, k, masked=True, gates=True, drop=True))
        check(make(n, E, k, seqs=[3, n - 20], gates=True))


def test_long_batches():
    check(make(20011, 256, 8, masked=True, seqs=[0, 7, 9000, 9000, 15000, 20011], gates=True))
    check(make(30000, 8, 2))


@pytest.mark.parametrize("T,E,k", [(4096, 40, 4), (8195, 384, 6), (20011, 7, 3), (70001, 64, 8)])
def test_one_long_sequence(T, E, k):
    """One sequence counted by several clusters: whole, masked, a part of the
    batch, and none of it."""
    check(make(T, E, k))
    check(make(T, E, k, masked=True, gates=True, drop=True, seqs=[11, T - 100]))
    check(make(T, E, k, gates=True, seqs=[5, 5]))


def test_masked_infinite_and_nan():
    c = make(50, 64, 4, masked=True)
    c["mask"][:10] = False
    c["logits"][:10] = float("nan")          # padding: not read
    c["logits"][20, :30] = float("-inf")     # experts that cannot be chosen
    c["logits"][21] = float("-inf")          # nothing can: p = 0
    c["logits"][22] = torch.finfo(torch.float32).min
    c["mask"][20:23] = True
    check(c)
    c["logits"][30, 3], c["mask"][30] = float("nan"), True
    loss, _, dz = call(P.BalanceLoss(64, 4), c)
    assert bool(loss.isnan()) and bool(dz[30].isnan().all())
    assert not bool(dz[[i for i in range(50) if i != 30]].isnan().any())


def test_nothing_valid_and_no_tokens():
    c = make(40, 16, 2, gates=True)
    c["mask"] = torch.zeros(40, dtype=torch.uint8)
    check(c)
    loss, counts, dz = call(P.BalanceLoss(16, 2), make(0, 16, 2))
    assert float(loss) == 0 and counts.shape == (1, 16) and not counts.any() and dz.shape == (0, 16)


def test_balanced_router_costs_coef():
    """Equal logits and equal counts: the loss is its coefficient."""
    T, E, k = 64, 16, 2
    ids = torch.arange(T * k, dtype=torch.int32).view(T, k) % E
    loss, counts, dz = P.BalanceLoss(E, k, 0.25)(torch.zeros(T, E, device=DEV), ids.to(DEV))
    assert abs(float(loss) - 0.25) < 1e-6 and bool((counts == T * k // E).all())
    assert float(dz.abs().max()) < 1e-9


def test_gradient_against_differences():
    """Central differences of the 64-bit loss (its error: h^2 of the loss)."""
    c = make(12, 8, 2, masked=True, seqs=[0, 5, 12])
    _, _, dz = call(P.BalanceLoss(8, 2, 1.0), c)
    h = 1e-4
    for t in range(12):
        for e in range(8):
            up, down = c["logits"].double().clone(), c["logits"].double().clone()
            up[t, e] += h
            down[t, e] -= h
            d = (reference(c, 1.0, up)[0] - reference(c, 1.0, down)[0]) / (2 * h)
            assert abs(float(dz[t, e]) - d) < 1e-6


def test_gate_gradient_against_autograd():
    """sum_j dweights_j * weights_j through softmax over the selected logits."""
    c = make(30, 24, 4, gates=True)
    z = c["logits"].double().requires_grad_()
    w = torch.gather(z, 1, c["ids"].long()).softmax(1)
    (w * c["dweights"].double()).sum().backward()
    _, _, dz = call(P.BalanceLoss(24, 4, 0.0), c)
    assert float((dz.cpu().double() - z.grad).abs().max()) < 1e-6


def test_stream_and_graph():
    c, d = make(300, 64, 4, masked=True), make(300, 64, 4, seed=9, masked=True)
    op = P.BalanceLoss(64, 4, 0.5)
    z, ids, m = (c[k].to(DEV) for k in ("logits", "ids", "mask"))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = op(z, ids, mask=m)
    torch.cuda.current_stream().wait_stream(st)
    assert abs(float(got[0]) - reference(c, 0.5)[0]) < 1e-5
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, counts, dz = op(z, ids, mask=m)
    for t, k in ((z, "logits"), (ids, "ids"), (m, "mask")):
        t.copy_(d[k])
    graph.replay()
    ref = reference(d, 0.5)
    assert abs(float(loss) - ref[0]) <= 2.0 ** -17 * ref[0]
    assert (np.abs(dz.double().cpu().numpy() - ref[2]) <= ref[3] + 1e-37).all()


def test_unaligned_rows():
    """Logits that begin on a 4-byte boundary take the scalar accesses."""
    c = make(40, 64, 4)
    flat = torch.empty(40 * 64 + 1, device=DEV)
    z = flat[1:].view(40, 64)
    z.copy_(c["logits"])
    op = P.BalanceLoss(64, 4)
    for p, q in zip(op(z, c["ids"].to(DEV)), call(op, c)):
        assert torch.equal(p, q)


def test_refusals():
    c = make(20, 16, 2, gates=True)
    op = P.BalanceLoss(16, 2)
    z, ids, w = c["logits"].to(DEV), c["ids"].to(DEV), c["weights"].to(DEV)
    bad = [
        lambda: op(z.bfloat16(), ids),
        lambda: op(z[:, :8], ids),
        lambda: op(z, ids.long()),
        lambda: op(z, ids[:, :1]),
        lambda: op(z.cpu(), ids),
        lambda: op(z, ids, mask=torch.ones(19, dtype=torch.bool, device=DEV)),
        lambda: op(z, ids, mask=torch.ones(20, device=DEV)),
        lambda: op(z, ids, seq_offsets=torch.tensor([0], dtype=torch.int32, device=DEV)),
        lambda: op(z, ids, seq_offsets=torch.tensor([0, 20], device=DEV)),
        lambda: op(z, ids, weights=w),
        lambda: P.BalanceLoss(16, 17),
        lambda: P.BalanceLoss(2000, 2),
        lambda: P.BalanceLoss(16, 2, float("nan")),
    ]
    for i, call_ in enumerate(bad):
        with pytest.raises(P.MoeError):
            call_()
            pytest.fail(f"refusal {i} did not come")
