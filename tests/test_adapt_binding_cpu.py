"""What the adapters', balance loss's and optimiser's binding hands to the
library, without a GPU: host tensors that say they are on device 0, and a
library whose launches are recorded instead of made."""
import os

import pytest
import torch

import precision_moe_grouped_gb300 as P
from precision_moe_grouped_gb300 import _adapt
from precision_moe_grouped_gb300 import _lib as L


class OnDevice(torch.Tensor):
    """A host tensor that passes for one of device 0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def on(t):
    return t.as_subclass(OnDevice)


class Recorder:
    """The built library, but that every call which would launch is noted in
    `calls` (its name and arguments) and returns success."""

    def __init__(self, lib):
        self._lib, self.calls = lib, []

    def __getattr__(self, name):
        if name in ("moe_adapter_forward", "moe_adapter_backward", "moe_balance_loss", "moe_adamw_step"):
            return lambda *args: self.calls.append((name, args)) or L.MOE_OK
        return getattr(self._lib, name)


@pytest.fixture
def lib(monkeypatch):
    if not os.path.exists(L.LIB_PATH):
        from precision_moe_grouped_gb300 import build
        try:
            build.build()
        except (RuntimeError, FileNotFoundError) as e:  # no nvcc on this machine
            pytest.skip(f"cannot build libmoe.so here: {e}")
    _adapt._bind_torch()
    r = Recorder(P.load())
    monkeypatch.setattr(_adapt, "load", lambda: r)
    monkeypatch.setattr(_adapt, "_device", lambda: 0)
    monkeypatch.setattr(_adapt, "_raw_stream", lambda device: 0)
    return r


def test_balance_coefficient_is_read_at_every_call(lib):
    """A coefficient that changes between two calls of the same size."""
    op = P.BalanceLoss(8, 2, coef=0.5)
    z, ids = on(torch.zeros(6, 8)), on(torch.zeros(6, 2, dtype=torch.int32))
    for coef in (0.5, 0.25, 0.5, torch.tensor(0.125)):
        op.coef = coef
        op(z, ids)
        assert lib.calls[-1][1][0].coef == float(coef)
    op.coef = float("nan")
    with pytest.raises(P.MoeError, match="coef"):
        op(z, ids)
