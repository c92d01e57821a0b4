"""The gated feed-forward block against the formula in 64 bits.

Tolerances.  A rounding to bf16 is off by at most u = 2^-8 of the value, and
by u / sqrt(3) in the mean square when it is uniform within that.  An output has
its own rounding, and those of the rounded intermediates that enter it (h, or dg
and du): relative to the output's norm at most as large again, as their errors
are independent of the terms that they multiply.  The error's norm is then at
most sqrt(2 / 3) u of the output's, held to u; with few values (T I < 4096) to
the sum of both largest errors, 2 u.

One element, sum of a_k b_k with every b_k off by at most u |b_k|, then rounded:
|err| <= u |ref| + (1 + u) u S, S = sum of |a_k b_k|.  Sums in float and the fast
exponential add less than 0.05 u S: float sums of up to n = 2^14 terms, in
pieces of 16, n / 16 2^-23 S = 2^-13 S = 0.03 u S; a relative 2e-6 = 0.0005 u of
each b_k for the exponential; and g, u and dh, sums of K = 7168 terms themselves,
off by 2^-14 of their own S, whose effect on h, dg and du is of the order of the
terms' spread: held to 1.1 u S + 2^-12 rms."""
import math

import pytest
import torch

import precision_moe_grouped_gb300 as P

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -8


def make(T, H, I, seed=0, base=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    bf = torch.bfloat16
    return {"x": randn(T, H).to(bf), "wgu": (randn(2 * I, H) / math.sqrt(H)).to(bf),
            "wd": (randn(H, I) / math.sqrt(I)).to(bf), "dout": (randn(T, H) * 1e-2).to(bf),
            "base": randn(T, H).to(bf) if base else None,
            "dx_base": (randn(T, H) * 1e-2).to(bf) if base else None}


def reference(s):
    """(out, dx, dw_gate_up, dw_down) in 64 bits, and for each the sum S of its terms' sizes."""
    x, w, wd, dout = (s[k].double() for k in ("x", "wgu", "wd", "dout"))
    gate, up = (x @ w.T).chunk(2, dim=1)
    sig = torch.sigmoid(gate)
    h = gate * sig * up
    dh = dout @ wd
    d = torch.cat([dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig], dim=1)
    base = 0 if s["base"] is None else s["base"].double()
    dx_base = 0 if s["dx_base"] is None else s["dx_base"].double()
    refs = h @ wd.T + base, d @ w + dx_base, d.T @ x, dout.T @ h
    return list(zip(refs, (h.abs() @ wd.abs().T, d.abs() @ w.abs(), d.abs().T @ x.abs(), dout.abs().T @ h.abs())))


def close(got, want, name, few=False):
    got, (ref, size) = got.double(), want
    assert got.shape == ref.shape and torch.isfinite(got).all(), name
    rms = ref.square().mean().sqrt()
    err = (got - ref).abs()
    off = float(err.square().mean().sqrt() / rms)
    assert off <= (2 if few else 1) * EPS, (name, off)
    worst = float((err / (EPS * ref.abs() + 1.1 * EPS * size + 2.0 ** -12 * rms)).max())
    assert worst <= 1, (name, worst)


SIZES = [(1, 256, 128), (1, 8, 8), (3, 2048, 1000), (8, 7168, 2048), (9, 520, 264), (17, 1024, 512),
         (32, 2048, 1024), (33, 2048, 1024), (64, 256, 128), (77, 2048, 1000), (131, 7168, 2048),
         (64, 2048, 2048), (100, 4096, 136), (255, 512, 256), (255, 4096, 1024), (256, 512, 256), (256, 7168, 256),
         (257, 520, 264), (513, 2048, 1024), (768, 264, 520), (769, 264, 520), (1021, 904, 8),
         (1021, 8, 360), (2500, 2048, 1024)]


@pytest.mark.parametrize("T,H,I", SIZES)
def test_forward(cuda_ok, T, H, I):
    for base in (True, False):
        s = make(T, H, I, seed=T + H, base=base)
        op = P.GatedFFN(s["wgu"], s["wd"])
        out = op(s["x"], base=s["base"])
        close(out, reference(s)[0], "out", T * I < 4096)
        assert torch.equal(out, op(s["x"], base=s["base"]))
        assert op.device_status() == 0


@pytest.mark.parametrize("T", [1, 9, 20, 32])
@pytest.mark.parametrize("H,I", [(64, 3000), (64, 4000), (64, 9000), (5000, 40), (8200, 72), (9608, 64), (20008, 64)])
def test_long_sides_of_small_batches(cuda_ok, T, H, I):
    """One to many tiles of weight rows a block, whole and in part, in either product."""
    s = make(T, H, I, seed=T + H + I)
    out = P.GatedFFN(s["wgu"], s["wd"])(s["x"], base=s["base"])
    close(out, reference(s)[0], "out")


@pytest.mark.parametrize("T,H,I", SIZES)
def test_backward(cuda_ok, T, H, I):
    for base in (True, False):
        s = make(T, H, I, seed=T + H, base=base)
        op = P.GatedFFN(s["wgu"], s["wd"])
        got = op.backward(s["dout"], s["x"], dx_base=s["dx_base"])
        for a, b, name in zip(got, reference(s)[1:], ("dx", "dw_gate_up", "dw_down")):
            close(a, b, name, T * I < 4096)
        for a, b in zip(got, op.backward(s["dout"], s["x"], dx_base=s["dx_base"])):
            assert torch.equal(a, b)
        assert op.device_status() == 0


def test_long_sums_over_tokens(cuda_ok):
    """The weights' gradients of as many tokens as a call takes, all terms of one sign.  The tensor cores cut their
    sums off, which is held to 2^-11 of the sum (2^18 terms came out 2^-9.3 short and are refused).  The roundings of h and of the result are
    as often up as down; over all elements (64 x 64 at least) their mean is below 2^-8 / sqrt(3 * 4096) = 2^-14.8."""
    T, H, I = 1 << 16, 64, 64
    s = make(T, H, I, seed=5)
    s = {k: v.abs() if k in ("x", "wgu", "wd", "dout") else None for k, v in s.items()}
    op = P.GatedFFN(s["wgu"], s["wd"])
    got = op.backward(s["dout"], s["x"])
    for a, (ref, size), name in zip(got[1:], reference(s)[2:], ("dw_gate_up", "dw_down")):
        err = a.double() - ref
        assert float((err.abs() / (EPS * ref.abs() + 1.1 * EPS * size + 2.0 ** -11 * size)).max()) <= 1, name
        assert float(ref.min()) > 0 and abs(float((err / ref).mean())) <= 2.0 ** -11 + 2.0 ** -13, name
    assert op.device_status() == 0
