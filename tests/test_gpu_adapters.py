"""Low-rank adapters (moe_adapter_forward / moe_adapter_backward) against the
formulas in 64 bits.

Tolerances, elementwise, with S the same expression over absolute values (the
most its terms can add up to):
  * a float intermediate (A x, B^T dout) enters the second product as two
    bf16 terms: 2^-17 of it at most, and so of S; a float dout once more
  * an MMA rounds (or truncates) each partial sum: at most 2^-23 S for each
    of the steps of 16 it runs, K / 16 of them, and for each of the at most
    128 partial sums joined after it
  * a bf16 result is rounded once: 2^-8 of it bounds half a unit in the last
    place with room for the error before it
"""
import pytest
import torch

import precision_moe_grouped_gb300 as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.set_device(0)


def make(T, NA, r, H, N, kind, ids="mixed", seed=0, scale=True):
    g = torch.Generator().manual_seed(seed + T + 7 * NA + 13 * r + H + N)
    rnd = lambda *s: torch.randn(s, generator=g)                  # noqa: E731
    x = rnd(T, H).bfloat16()
    a = (rnd(NA, r, H) / H ** 0.5).bfloat16()
    b = rnd(NA, N, r).bfloat16()
    sc = torch.rand(NA, generator=g) + 0.5 if scale else None
    base = rnd(T, N).to(kind)
    if ids == "mixed":       # none, some out of range, the rest at random
        i = torch.randint(-1, NA, (T,), generator=g)
        i[::11] = NA
        i[5::17] = -2 ** 31
        i[7::19] = 2 ** 31 - 1
    elif ids == "one":
        i = torch.full((T,), NA - 1)
    elif ids == "none":
        i = torch.full((T,), -1)
    else:                    # runs of a request's tokens
        i = (torch.arange(T) // 37) % NA
    dout = (rnd(T, N) * 0.1).to(kind)
    dx_base = rnd(T, H).bfloat16()
    to = lambda t: None if t is None else t.to(DEV)               # noqa: E731
    return dict(x=to(x), a=to(a), b=to(b), scale=to(sc), base=to(base), ids=to(i.to(torch.int32)),
                dout=to(dout), dx_base=to(dx_base))


def rows_of(c, i):
    return torch.nonzero(c["ids"].long() == i).reshape(-1)


def reference(c):
    """out, dx, da, db in 64 bits, and the same over absolute values."""
    def go(f):
        x, a, b = f(c["x"].double()), f(c["a"].double()), f(c["b"].double())
        base, dout, dxb = f(c["base"].double()), f(c["dout"].double()), f(c["dx_base"].double())
        out, dx = base.clone(), dxb.clone()
        da, db = torch.zeros_like(a), torch.zeros_like(b)
        for i in range(a.shape[0]):
            rows = rows_of(c, i)
            if len(rows) == 0:
                continue
            s = 1.0 if c["scale"] is None else c["scale"][i].double()
            v, u = x[rows] @ a[i].T, s * (dout[rows] @ b[i])
            out[rows] += s * (v @ b[i].T)
            dx[rows] += u @ a[i]
            da[i] = u.T @ x[rows]
            db[i] = s * dout[rows].T @ v
        return dict(out=out, dx=dx, da=da, db=db)
    return go(lambda t: t), go(torch.abs)


def assert_close(name, got, ref, size, splits, steps, bf16):
    tol = size * (splits * 2.0 ** -17 + (steps + 128) * 2.0 ** -23)
    if bf16:
        tol = tol + 2.0 ** -8 * ref.abs()
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), (name, int(bad.sum()), float(((got.double() - ref).abs() / tol.clamp(min=1e-300)).max()))


def check_forward(c, got, kind):
    ref, size = reference(c)
    H, r = c["x"].shape[1], c["a"].shape[1]
    assert got.dtype == kind
    assert_close("out", got, ref["out"], size["out"], 1, (H + r) / 16, kind == torch.bfloat16)


def check_backward(c, dx, da, db, kind):
    ref, size = reference(c)
    (T, H), N, r = c["x"].shape, c["b"].shape[1], c["a"].shape[1]
    f = 2 if kind == torch.float32 else 1    # u carries dout's split too
    if dx is not None:
        assert_close("dx", dx, ref["dx"], size["dx"], f, (N + r) / 16, True)
    if da is not None:
        assert_close("da", da, ref["da"], size["da"], f, (N + T) / 16, False)
        # both factors split, their residuals' product dropped
        assert_close("db", db, ref["db"], size["db"], 3 if f == 2 else 1, (H + T) / 16, False)


SHAPES = [
    # T, NA, r, H, N, ids
    (1, 1, 8, 8, 8, "one"),
    (1, 5, 16, 7168, 256, "one"),
    (3, 2, 24, 40, 24, "mixed"),
    (17, 4, 16, 264, 1000, "mixed"),
    (64, 1, 32, 256, 256, "one"),
    (65, 3, 64, 136, 72, "mixed"),
    (130, 1024, 8, 64, 64, "mixed"),
    (200, 6, 40, 2048, 40, "runs"),
    (257, 3, 128, 200, 520, "mixed"),
    (300, 7, 72, 96, 264, "runs"),
    (333, 2, 104, 248, 104, "runs"),
    (1100, 5, 16, 2048, 384, "runs"),
    (4099, 1, 64, 256, 520, "one"),
    (100, 4, 16, 128, 128, "none"),
    # either side of the batches that one kernel takes
    (1024, 1024, 16, 72, 136, "mixed"),
    (1024, 3, 64, 264, 520, "runs"),
    (1025, 1024, 16, 72, 136, "mixed"),
    (1025, 2, 32, 1000, 264, "one"),
    (64, 9, 128, 520, 264, "mixed"),
    (65, 9, 128, 520, 264, "mixed"),
]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,NA,r,H,N,ids", SHAPES)
def test_forward(T, NA, r, H, N, ids, kind):
    c = make(T, NA, r, H, N, kind, ids)
    op = P.LowRankAdapters(c["a"], c["b"], c["scale"])
    out = op.forward(c["x"], c["ids"], c["base"])
    check_forward(c, out, kind)
    plain = (c["ids"] < 0) | (c["ids"] >= NA)
    assert torch.equal(out[plain], c["base"][plain])        # no adapter: base, bit for bit
    assert torch.equal(out, op.forward(c["x"], c["ids"], c["base"]))
    here = c["base"].clone()                                # in place
    assert op.forward(c["x"], c["ids"], here, out=here) is here and torch.equal(here, out)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,NA,r,H,N,ids", SHAPES)
def test_backward(T, NA, r, H, N, ids, kind):
    c = make(T, NA, r, H, N, kind, ids)
    op = P.LowRankAdapters(c["a"], c["b"], c["scale"])
    dx, da, db = op.backward(c["dout"], c["x"], c["ids"], c["dx_base"])
    check_backward(c, dx, da, db, kind)
    for i in range(NA):
        if len(rows_of(c, i)) == 0:
            assert not da[i].any() and not db[i].any()
    again = op.backward(c["dout"], c["x"], c["ids"], c["dx_base"])
    assert all(torch.equal(p, q) for p, q in zip((dx, da, db), again))
    # each part alone gives the same
    here = c["dx_base"].clone()
    only = op.backward(c["dout"], c["x"], c["ids"], here, dx=here, need_weights=False)
    assert only[0] is here and torch.equal(here, dx) and only[1] is None and only[2] is None
    none, da2, db2 = op.backward(c["dout"], c["x"], c["ids"], need_dx=False)
    assert none is None and torch.equal(da, da2) and torch.equal(db, db2)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_without_base_or_scale(kind):
    c = make(70, 3, 16, 128, 136, kind, scale=False)
    op = P.LowRankAdapters(c["a"], c["b"])
    out = op.forward(c["x"], c["ids"], out_dtype=kind)
    c["base"] = torch.zeros_like(c["base"])
    check_forward(c, out, kind)
    dx, da, db = op.backward(c["dout"], c["x"], c["ids"])
    c["dx_base"] = torch.zeros_like(c["dx_base"])
    check_backward(c, dx, da, db, kind)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_strided_rows(kind):
    """Rows that are slices of wider ones; what lies between them stays."""
    c = make(150, 4, 24, 96, 80, kind)
    wide = lambda t, off, cols: torch.full((t.shape[0], cols), 7.0, dtype=t.dtype, device=DEV)  # noqa: E731
    def inside(t, off, cols):
        w = wide(t, off, cols)
        w[:, off:off + t.shape[1]] = t
        return w, w[:, off:off + t.shape[1]]
    _, c["x"] = inside(c["x"], 16, 136)
    _, c["base"] = inside(c["base"], 8, 104)
    ow, out = inside(torch.zeros_like(c["base"]), 24, 112)
    op = P.LowRankAdapters(c["a"], c["b"], c["scale"])
    op.forward(c["x"], c["ids"], c["base"], out=out)
    check_forward(c, out, kind)
    assert bool((ow[:, :24] == 7).all()) and bool((ow[:, 104:] == 7).all())
    _, c["dout"] = inside(c["dout"], 8, 96)
    _, c["dx_base"] = inside(c["dx_base"], 8, 112)
    xw, dx = inside(torch.zeros_like(c["dx_base"]), 16, 128)
    _, da, db = op.backward(c["dout"], c["x"], c["ids"], c["dx_base"], dx=dx)
    check_backward(c, dx, da, db, kind)
    assert bool((xw[:, :16] == 7).all()) and bool((xw[:, 112:] == 7).all())


def test_other_tokens_nan_stays_theirs():
    """A NaN or an infinity in the row of a token without an adapter reaches
    nothing; in an adapted token's row it reaches that row and its adapter's
    gradients only."""
    c = make(90, 4, 16, 128, 64, torch.float32, "runs")
    c["ids"][3], c["ids"][50] = -1, 9
    op = P.LowRankAdapters(c["a"], c["b"], c["scale"])
    clean = op.forward(c["x"], c["ids"], c["base"])
    grads = op.backward(c["dout"], c["x"], c["ids"], c["dx_base"])
    c["x"][3], c["x"][50] = float("nan"), float("inf")
    c["dout"][3], c["dout"][50] = float("inf"), float("nan")
    assert torch.equal(clean, op.forward(c["x"], c["ids"], c["base"]))
    assert all(torch.equal(p, q) for p, q in
               zip(grads, op.backward(c["dout"], c["x"], c["ids"], c["dx_base"])))
    t = 20                                   # adapter 0, as tokens 0 .. 36 but 3
    c["x"][t, 5] = float("nan")
    out = op.forward(c["x"], c["ids"], c["base"])
    _, da, db = op.backward(c["dout"], c["x"], c["ids"])
    keep = torch.arange(90, device=DEV) != t
    assert torch.equal(out[keep], clean[keep]) and bool(out[t].isnan().all())
    assert torch.equal(da[1:], grads[1][1:]) and torch.equal(db[1:], grads[2][1:])
    assert bool(da[0].isnan().any()) and bool(db[0].isnan().all())


def test_gradients_against_differences():
    """The output is linear in a, in b and in x, so that the difference of
    sum(dout * out) between two of them is the gradient's product with their
    difference, whatever the step; held to the forward's own float error."""
    c = make(140, 3, 24, 256, 72, torch.float32, "runs")
    d = make(140, 3, 24, 256, 72, torch.float32, "runs", seed=5)
    def loss(a, b, x):
        out = P.LowRankAdapters(a, b, c["scale"]).forward(x, c["ids"], c["base"])
        return float((out.double() * c["dout"].double()).sum())
    dx, da, db = P.LowRankAdapters(c["a"], c["b"], c["scale"]).backward(c["dout"], c["x"], c["ids"])
    at = loss(c["a"], c["b"], c["x"])
    _, size = reference(c)
    _, size2 = reference(d)
    bound = float((c["dout"].double().abs() * (size["out"] + size2["out"])).sum()) * 2.0 ** -15
    for got, diff, moved in ((da, d["a"].double() - c["a"].double(), loss(d["a"], c["b"], c["x"])),
                             (db, d["b"].double() - c["b"].double(), loss(c["a"], d["b"], c["x"]))):
        assert abs(float((got.double() * diff).sum()) - (moved - at)) <= bound
    # dx is rounded to bf16
    diff = d["x"].double() - c["x"].double()
    slack = bound + float((dx.double().abs() * diff.abs()).sum()) * 2.0 ** -8
    assert abs(float((dx.double() * diff).sum()) - (loss(c["a"], c["b"], d["x"]) - at)) <= slack


def test_no_tokens():
    c = make(1, 3, 16, 64, 64, torch.bfloat16)
    op = P.LowRankAdapters(c["a"], c["b"], c["scale"])
    x, ids = c["x"][:0], c["ids"][:0]
    assert op.forward(x, ids, c["base"][:0]).shape == (0, 64)
    dx, da, db = op.backward(c["dout"][:0], x, ids)
    assert dx.shape == (0, 64) and not da.any() and not db.any()


def test_stream_and_graph():
    """On a side stream, and captured into a graph that is replayed with new
    inputs and new pools."""
    c, d = make(64, 6, 16, 512, 256, torch.bfloat16), make(64, 6, 16, 512, 256, torch.bfloat16, seed=3)
    op = P.LowRankAdapters(c["a"].clone(), c["b"].clone(), c["scale"].clone())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out = op.forward(c["x"], c["ids"], c["base"])
    torch.cuda.current_stream().wait_stream(st)
    check_forward(c, out, torch.bfloat16)
    x, ids, base, dout = (c[k].clone() for k in ("x", "ids", "base", "dout"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = op.forward(x, ids, base)
        dx, da, db = op.backward(dout, x, ids)
    for t, k in ((x, "x"), (ids, "ids"), (base, "base"), (dout, "dout"), (op.a, "a"), (op.b, "b"),
                 (op.scale, "scale")):
        t.copy_(d[k])
    graph.replay()
    torch.cuda.synchronize()
    check_forward(d, out, torch.bfloat16)
    d["dx_base"] = torch.zeros_like(d["dx_base"])
    check_backward(d, dx, da, db, torch.bfloat16)


def test_offsets_beyond_32_bits():
    """Rows whose element offsets pass 2^31 and 2^32."""
    T, H, N, ld = 3, 64, 64, (1 << 31) - 8
    c = make(T, 2, 8, H, N, torch.bfloat16, "one")
    wide = torch.empty(2 * ld + H, dtype=torch.bfloat16, device=DEV)       # 8.6 GB
    x = torch.as_strided(wide, (T, H), (ld, 1))
    x.copy_(c["x"])
    op = P.LowRankAdapters(c["a"], c["b"], c["scale"])
    assert torch.equal(op.forward(x, c["ids"], c["base"]), op.forward(c["x"], c["ids"], c["base"]))
    ref = op.backward(c["dout"], c["x"], c["ids"])
    assert all(torch.equal(p, q) for p, q in zip(ref, op.backward(c["dout"], x, c["ids"])))


@pytest.mark.parametrize("T,NA,ids", [(4096, 2, "runs"), (4097, 1024, "mixed"), (20011, 200, "mixed"),
                                      (70001, 3, "runs")])
def test_long_batches(T, NA, ids):
    """Token lists that each of the grouping's warps walks in several rounds."""
    c = make(T, NA, 8, 64, 64, torch.float32, ids)
    op = P.LowRankAdapters(c["a"], c["b"], c["scale"])
    check_forward(c, op.forward(c["x"], c["ids"], c["base"]), torch.float32)
    check_backward(c, *op.backward(c["dout"], c["x"], c["ids"], c["dx_base"]), torch.float32)


@pytest.mark.parametrize("T", [3, 200, 1500])
def test_forward_over_its_input(T):
    """x += the adapters' products of x: a tile's rows are read before any of
    them is written."""
    c = make(T, 4, 16, 512, 512, torch.bfloat16)
    op = P.LowRankAdapters(c["a"], c["b"], c["scale"])
    want = op.forward(c["x"], c["ids"], c["x"])
    x = c["x"].clone()
    assert op.forward(x, c["ids"], x, out=x) is x and torch.equal(x, want)


def test_refusals():
    c = make(20, 3, 16, 64, 64, torch.bfloat16)
    op = P.LowRankAdapters(c["a"], c["b"], c["scale"])
    x, ids, base = c["x"], c["ids"], c["base"]
    bad = [
        lambda: op.forward(x.float(), ids, base),
        lambda: op.forward(x[:, :32], ids, base),
        lambda: op.forward(x.cpu(), ids, base),
        lambda: op.forward(x, ids.long(), base),
        lambda: op.forward(x, ids[:5], base),
        lambda: op.forward(x, ids, base.half()),
        lambda: op.forward(x, ids, base, out=base.float()),
        lambda: op.forward(x.t().contiguous().t(), ids, base),
        lambda: op.backward(c["dout"], x, ids, dx=x),
        lambda: op.backward(c["dout"][:4], x, ids),
        lambda: op.backward(c["dout"], x, ids, da=torch.empty(3, 16, 64, device=DEV).half()),
        lambda: P.LowRankAdapters(c["a"][:, :12].contiguous(), c["b"][:, :, :12].contiguous()),
        lambda: P.LowRankAdapters(c["a"], c["b"][:2]),
        lambda: P.LowRankAdapters(c["a"].float(), c["b"]),
        lambda: P.LowRankAdapters(c["a"], c["b"], c["scale"][:2]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(P.MoeError):
            call()
            pytest.fail(f"refusal {i} did not come")
    odd = torch.empty(20 * 72 + 1, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(P.MoeError, match="aligned"):
        op.forward(odd[1:1 + 20 * 64].view(20, 64), ids, base)
    with pytest.raises(P.MoeError, match="multiple of 8"):
        op.forward(torch.as_strided(odd, (20, 64), (68, 1)), ids, base)
