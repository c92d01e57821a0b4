"""The float precision of the adapters' float results: what the low-rank rows
keep between the two products, and what the long sums lose.

The terms of a product with ones are exact, so that a row of 24 significant
bits has to come through bit for bit; kept as two bf16 terms it would not (the
tests check that of their own inputs).  A long sum of positive terms shows a
bias: an MMA truncates its accumulator, by 2^-24 of it on average at most.
The sums run in pieces of at most 8 such steps (12 in da and db) that are
added with rounding, so the mean error is at most 8 * 2^-24 (12 * 2^-24) of
the sum; a rounded addition adds no bias and at most 2^-24 to a single error."""
import pytest
import torch

import precision_moe_grouped_gb300 as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.set_device(0)


def whole(n, seed):
    """[n, 3] of bf16 values whose sums have all of their 24 bits, and the sums."""
    g = torch.Generator().manual_seed(seed)
    m = [torch.randint(0, 128, (n,), generator=g), torch.randint(0, 128, (n,), generator=g),
         2 * torch.randint(0, 64, (n,), generator=g)]
    parts = torch.stack([(1 + q.double() / 128) * 2.0 ** -s for q, s in zip(m, (0, 9, 17))], 1)
    sums = parts.sum(1)
    assert torch.equal(parts.bfloat16().double(), parts) and torch.equal(sums.float().double(), sums)
    hi = sums.float().bfloat16()
    mid = (sums - hi.double()).float().bfloat16()
    lo = (sums - hi.double() - mid.double()).float().bfloat16()
    two = hi.double() + mid.double()
    assert torch.equal(two + lo.double(), sums) and int((two != sums).sum()) > 0.9 * n
    return parts.float().to(DEV), sums.float().to(DEV)


def zeros(*shape, kind=BF16):
    return torch.zeros(*shape, dtype=kind, device=DEV)


@pytest.mark.parametrize("T,r", [(5, 8), (64, 128), (1000, 16), (300, 128), (1200, 8), (1200, 32), (1200, 64)])
def test_low_rank_rows_are_whole_in_a_float_output(T, r):
    parts, sums = whole(T, T + r)
    H, N = 40, 136
    x, a, b = zeros(T, H), zeros(2, r, H), zeros(2, N, r)
    x[:, 11:14] = parts.bfloat16()
    a[1, r - 1, 11:14] = 1
    b[1, :, r - 1] = 1
    ids = torch.ones(T, dtype=torch.int32, device=DEV)
    out = P.LowRankAdapters(a, b).forward(x, ids, out_dtype=F32)
    assert torch.equal(out, sums[:, None].expand(T, N))


@pytest.mark.parametrize("r", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("kind", [F32, BF16])
def test_low_rank_rows_are_whole_in_the_gradients(r, kind):
    """A token an adapter: da and db are products of one row."""
    T, H, N = 40, 136, 72
    parts, sums = whole(T, r)
    ids = torch.arange(T, dtype=torch.int32, device=DEV)
    ones = lambda *s: torch.ones(*s, dtype=BF16, device=DEV)         # noqa: E731
    a, b = zeros(T, r, H), zeros(T, N, r)
    b[:, 3:6, 1] = 1
    dout = zeros(T, N, kind=kind)
    dout[:, 3:6] = parts.to(kind)                      # u = its sum
    _, da, _ = P.LowRankAdapters(a, b).backward(dout, ones(T, H), ids)
    assert torch.equal(da[:, 1], sums[:, None].expand(T, H)) and not da[:, 2:].any() and not da[:, 0].any()
    x = zeros(T, H)
    x[:, 7:10] = parts.bfloat16()                      # w = its sum
    a[:, 1, 7:10] = 1
    _, _, db = P.LowRankAdapters(a, b).backward(ones(T, N).to(kind), x, ids)
    assert torch.equal(db[:, :, 1], sums[:, None].expand(T, N)) and not db[:, :, 2:].any()
    if kind is F32:                                    # dout of 24 bits
        x.zero_()
        x[:, 7] = 1                                    # w = 1
        d = sums[:, None] * 2.0 ** torch.arange(-8, N - 8, device=DEV).clamp(max=8)
        _, _, db = P.LowRankAdapters(a, b).backward(d.contiguous(), x, ids)
        assert torch.equal(db[:, :, 1], d)


def mean_and_most(got, ref):
    e = (got.double() - ref) / ref
    return float(e.mean().abs()), float(e.abs().max())


@pytest.mark.parametrize("T,r", [(256, 8), (1000, 32), (2000, 8), (2000, 64), (300, 128)])
def test_long_contractions_have_no_drift(T, r):
    """w over 7168 positive terms; b passes it on as it is."""
    H = 7168
    g = torch.Generator(device=DEV).manual_seed(T + r)
    x = (torch.rand(T, H, generator=g, device=DEV) + 0.5).bfloat16()
    a = (torch.rand(1, r, H, generator=g, device=DEV) + 0.5).bfloat16()
    b = torch.eye(r, dtype=BF16, device=DEV)[None].contiguous()
    out = P.LowRankAdapters(a, b).forward(x, zeros(T, kind=torch.int32), out_dtype=F32)
    mean, most = mean_and_most(out, x.double() @ a[0].double().T)
    assert mean <= 8 * 2.0 ** -24, mean
    # 16 for the steps of a piece, an addition for each piece, warp and CTA
    assert most <= (16 + H / 128 + 32) * 2.0 ** -24, most


@pytest.mark.parametrize("T", [500, 20000])
@pytest.mark.parametrize("r", [8, 32, 64, 128])
@pytest.mark.parametrize("kind", [F32, BF16])
def test_long_sums_over_tokens_have_no_drift(T, r, kind):
    """da and db over one adapter's tokens, positive terms; a and b pass x and
    dout on as they are."""
    n = 128
    g = torch.Generator(device=DEV).manual_seed(T + r)
    x = (torch.rand(T, n, generator=g, device=DEV) + 0.5).bfloat16()
    dout = (torch.rand(T, n, generator=g, device=DEV) + 0.5).to(kind)
    a, b = zeros(1, r, n), zeros(1, n, r)
    at = torch.arange(r, device=DEV)
    a[0, at, at] = b[0, at, at] = 1
    _, da, db = P.LowRankAdapters(a, b).backward(dout, x, zeros(T, kind=torch.int32))
    for name, got, ref in (("da", da[0], dout[:, :r].double().T @ x.double()),
                           ("db", db[0], dout.double().T @ x[:, :r].double())):
        mean, most = mean_and_most(got, ref)
        assert mean <= 12 * 2.0 ** -24, (name, mean)
        # 24 for the steps of a piece, an addition for each piece of 32 tokens and CTA; the
        # dropped products of a float dout's planes are below 2^-24
        assert most <= (24 + T / 32 + 16) * 2.0 ** -24, (name, most)
