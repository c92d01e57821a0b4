"""Weights' gradients in memory that the same call reads or writes are refused, before any CUDA call."""
import pytest

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
