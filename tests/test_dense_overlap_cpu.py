"""Weights' gradients in memory that the same call reads or writes are refused, before any CUDA call."""
import random

import pytest
import torch

from precision_moe_grouped_gb300 import _lib as L

X, DOUT, WGU, WD, DX, DWGU, DWD = ((i + 1) << 20 for i in range(7))


@pytest.mark.parametrize("T", [0, 3, 100, 1000])
@pytest.mark.parametrize("dwgu,dwd", [(WGU, DWD), (DWGU, WD), (WD, DWD), (DWGU, WGU), (X, DWD), (DWGU, X), (DOUT, DWD),
                                      (DWGU, DOUT), (DX, DWD), (DWGU, DX), (DWGU, DWGU)])
def test_gradients_are_memory_of_their_own(T, dwgu, dwd):
    lib = L.load()
    assert lib.moe_ffn_backward(L.FfnShape(T, 64, 32), DOUT, 64, X, 64, WGU, WD, None, 64, DX, 64, dwgu, dwd, 1 << 24,
                                1 << 40, 1 << 25, None) == L.MOE_ERR_INVALID_ARG
    assert b"memory of their own" in lib.moe_last_error()


# ------------------------------------------------ parts of one another, and strides
H, I = 64, 32
WS, STATUS = 1 << 24, 1 << 25
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are no memory: where nothing can be launched")


def forward(T, x=X, ld_x=H, base=None, ld_base=H, out=DX, ld_out=H, wgu=WGU, wd=WD, ws=WS, status=STATUS, hidden=H):
    lib = L.load()
    return lib.moe_ffn_forward(L.FfnShape(T, hidden, I), x, ld_x, wgu, wd, base, ld_base, out, ld_out, ws, 1 << 40,
                               status, None)


def backward(T, dout=DOUT, ld_dout=H, x=X, ld_x=H, base=None, ld_base=H, dx=DX, ld_dx=H, dwgu=DWGU, dwd=DWD, wgu=WGU,
             wd=WD, ws=WS, status=STATUS):
    lib = L.load()
    return lib.moe_ffn_backward(L.FfnShape(T, H, I), dout, ld_dout, x, ld_x, wgu, wd, base, ld_base, dx, ld_dx, dwgu,
                                dwd, ws, 1 << 40, status, None)


def refused(rc):
    return rc == L.MOE_ERR_INVALID_ARG and b"overlap" in L.load().moe_last_error()


def passed(rc):
    """The arguments' checks: what comes next asks for a device."""
    return rc == L.MOE_ERR_CUDA or rc == L.MOE_ERR_UNSUPPORTED and b"overlap" not in L.load().moe_last_error()


ROW, W = 2 * H, 4 * H * I          # bytes of a row; of w_gate_up (w_down has half)
BASE = 9 << 20


@pytest.mark.parametrize("T", [3, 100, 1000])
@pytest.mark.parametrize("bad", [
    dict(out=X + ROW), dict(out=X - ROW), dict(out=X, ld_out=2 * H), dict(x=DX, ld_x=2 * H),
    dict(base=DX + ROW), dict(base=DX, ld_base=2 * H), dict(base=DX - 16),
    dict(out=WGU), dict(out=WGU + W - 16), dict(out=WD - ROW), dict(out=WD + W // 2 - 16),
    dict(ws=X), dict(x=WS + 128), dict(base=WS), dict(out=WS), dict(ws=WGU), dict(ws=WD), dict(status=DX + 4),
    dict(status=WS + 4)], ids=str)
def test_forward_writes_to_memory_of_its_own(T, bad):
    assert refused(forward(T, **bad))


@pytest.mark.parametrize("T", [3, 100, 1000])
@pytest.mark.parametrize("bad", [
    dict(base=DWGU), dict(base=DWD), dict(base=DWGU + W - 16), dict(dwgu=BASE - 16, base=BASE),
    dict(dwgu=X + 16), dict(dwd=X - 16), dict(dwgu=DOUT + 16), dict(dwd=DOUT + 16), dict(dwgu=WGU + 16),
    dict(dwgu=WD - 16), dict(dwd=WGU + W - 16), dict(dwd=WD + 16), dict(dwgu=DX + 16), dict(dx=DWD + 16),
    dict(dwd=DWGU + W - 16), dict(dwgu=DWD - W + 16), dict(dx=X + ROW), dict(dx=DOUT + ROW), dict(dx=WGU),
    dict(dx=WD + 16), dict(base=DX, ld_base=2 * H), dict(base=DX + ROW), dict(base=DX - 16), dict(ws=X), dict(ws=DX),
    dict(base=WS), dict(ws=DWGU), dict(ws=DWD), dict(dout=WS + 256), dict(status=DX), dict(status=DWGU + 8),
    dict(status=DWD), dict(status=WS + 4)], ids=str)
def test_gradients_go_to_memory_of_their_own(T, bad):
    assert refused(backward(T, **bad))


def test_gradients_without_tokens():
    """They are set to zero: not a part of the weights, nor of one another."""
    for bad in (dict(dwgu=WGU + 16), dict(dwgu=WD - 16), dict(dwd=WGU - 16), dict(dwd=WD + 16), dict(dwd=DWGU + 16)):
        assert refused(backward(0, **bad)), bad


@no_gpu
@pytest.mark.parametrize("T", [3, 100, 1000])
def test_what_may_share_memory(T):
    row = 2 * H    # elements between rows: two matrices side by side
    for good in (dict(), dict(out=X), dict(base=DX), dict(out=X, base=X), dict(out=X, ld_x=row, ld_out=row),
                 dict(x=X, ld_x=row, out=X + ROW, ld_out=row), dict(base=DX + ROW, ld_base=row, ld_out=row),
                 dict(base=BASE, x=BASE + 16), dict(out=WGU + W), dict(out=WD + W // 2), dict(status=STATUS + 4)):
        assert passed(forward(T, **good)), good
    for good in (dict(), dict(base=DX), dict(base=DX, ld_base=row, ld_dx=row), dict(base=X), dict(base=DOUT), dict(x=DOUT),
                 dict(dx=X + ROW, ld_dx=row, ld_x=row), dict(dwd=DWGU + W), dict(dwgu=WGU + W),
                 dict(dx=None, base=DWGU), dict(dwgu=None, dwd=None, base=DWGU)):
        assert passed(backward(T, **good)), good
    # a single row's stride says nothing
    assert passed(forward(1, out=X, ld_x=H, ld_out=2 * H)) and passed(backward(1, base=DX, ld_base=2 * H))
    assert passed(backward(0)) or torch.cuda.is_available()


@no_gpu
def test_rows_between_rows():
    """Against the set of bytes: two matrices of 16-byte pieces with any strides and distances."""
    rng = random.Random(0)
    said = [0, 0]
    for _ in range(1000):
        T, width = rng.randint(1, 7), rng.randint(1, 4)
        ld_x, ld_out = (width + rng.choice([0, 0, 1, 2, 3, 5, 9]) for _ in range(2))
        if rng.random() < 0.5:
            ld_out = ld_x
        d = rng.randint(-60, 60)
        pieces = lambda at, ld: {at + i * ld + k for i in range(T) for k in range(width)}   # noqa: E731
        same = d == 0 and (ld_x == ld_out or T == 1)
        meet = bool(pieces(0, ld_x) & pieces(d, ld_out)) and not same
        rc = forward(T, x=X, ld_x=8 * ld_x, out=X + 16 * d, ld_out=8 * ld_out, hidden=8 * width)
        assert (refused(rc) if meet else passed(rc)), (T, width, ld_x, ld_out, d)
        said[meet] += 1
    assert min(said) > 150
