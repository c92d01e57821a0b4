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


def test_routing_is_of_the_last_call(monkeypatch, lib):
    """Views of a workspace that no call of so many tokens has filled are
    refused, a replaced workspace's among them."""
    monkeypatch.setattr(P, "prepare_weights", lambda *a, **k: None)
    monkeypatch.setattr(P, "forward", lambda *a, **k: None)
    E, H, I = 8, 256, 128
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)                # noqa: E731
    moe = P.FusedMoE(u8(E, 2 * I, H // 2), u8(E, 2 * I, H // 32), u8(E, H, I // 2), u8(E, H, I // 32), 2)
    x, z = torch.zeros(2000, H, dtype=torch.bfloat16), torch.zeros(2000, E)

    def refused(T):
        with pytest.raises(P.MoeError, match="no routing"):
            moe.routing(T)

    refused(5)                       # nothing forwarded yet
    moe(x[:100], z[:100])
    ids, w = moe.routing(100)
    assert ids.shape == w.shape == (100, 2)
    for T in (5, 101, 2000):         # smaller, and larger than the workspace
        refused(T)
    assert moe.routing(100)[0].data_ptr() == ids.data_ptr()    # the refusals left it as it was
    moe(x[:5], z[:5])
    moe.routing(5)
    refused(100)                     # overwritten since
    moe.workspace(2000)              # grows: a new one
    refused(5)
    moe(x, z)
    assert moe.routing(2000)[0].shape == (2000, 2)

    def fails(*a, **k):
        raise P.MoeError(L.MOE_ERR_INVALID_ARG, "x")
    monkeypatch.setattr(P, "forward", fails)
    with pytest.raises(P.MoeError):
        moe(x[:7], z[:7])
    refused(7)


def adapters(NA=3, r=8, H=64, N=32):
    a = on(torch.zeros(NA, r, H, dtype=torch.bfloat16))
    b = on(torch.zeros(NA, N, r, dtype=torch.bfloat16))
    return P.LowRankAdapters(a, b, on(torch.ones(NA)))


def test_pools_are_checked_at_every_call(lib):
    """A pool whose memory, type, size, layout or place changed after the
    construction: the library sees the new one or the call is refused."""
    x, ids = on(torch.zeros(4, 64, dtype=torch.bfloat16)), on(torch.zeros(4, dtype=torch.int32))
    dout = on(torch.zeros(4, 32))
    bf16 = torch.bfloat16

    class Host(OnDevice):
        is_cuda = property(lambda self: False)

    changes = {
        "a": [torch.zeros(3, 8, 32, dtype=bf16), torch.zeros(2, 8, 64, dtype=bf16), torch.zeros(3, 8, 64),
              torch.zeros(3, 64, 8, dtype=bf16).transpose(1, 2), None],
        "b": [torch.zeros(3, 32, 16, dtype=bf16), torch.zeros(3, 16, 8, dtype=bf16), torch.zeros(3, 32, 8), None],
        "scale": [torch.zeros(2), torch.zeros(3, dtype=torch.float64), torch.zeros(6)[::2]],
    }
    for name, bad in changes.items():
        bad.append(  # as its module moved to the host
            getattr(adapters(), name).as_subclass(Host))
        for t in bad:
            op = adapters()
            setattr(op, name, on(t) if t is not None and not isinstance(t, Host) else t)
            for call in (lambda: op.forward(x, ids), lambda: op.backward(dout, x, ids)):
                with pytest.raises(P.MoeError):
                    call()
                    pytest.fail(f"{name}: {t if t is None else (t.shape, t.dtype)}")
    assert not lib.calls
    # .data of the caller's own tensor
    op = adapters()
    op.forward(x, ids)
    op.a.data = torch.zeros(1, dtype=bf16)
    with pytest.raises(P.MoeError):
        op.forward(x, ids)
    assert len(lib.calls) == 1 and len(op._held) == 3      # the first call's memory is held
    lib.calls.clear()
    # good ones are followed, and the sizes of the construction stay
    op = adapters()
    op.a, op.b, op.scale = adapters().a, adapters().b, None
    op.rank = op.in_features = 8
    op.forward(x, ids)
    op.backward(dout, x, ids)
    (_, f), (_, b) = lib.calls
    assert f[4:7] == (op.a.data_ptr(), op.b.data_ptr(), None) and b[6:9] == f[4:7]
    assert f[0].rank == b[0].rank == 8 and f[0].in_features == b[0].in_features == 64


def adamw(n=2, **kw):
    zeros = lambda: [on(torch.zeros(8 + i)) for i in range(n)]        # noqa: E731
    return P.AdamW(zeros(), zeros(), state={"m": zeros(), "v": zeros()}, **kw)


def test_gradients_of_another_device_are_refused(lib, monkeypatch):
    """Bound while their device is current, they would reach a step on the
    parameters' device."""
    class OnOther(OnDevice):
        def get_device(self):
            return 1

    opt = adamw(1)
    monkeypatch.setattr(_adapt, "_device", lambda: 1)
    for call in (lambda: opt.bind_grads([torch.zeros(8).as_subclass(OnOther)]),
                 lambda: opt.step(grads=[torch.zeros(8).as_subclass(OnOther)]), opt.step):
        with pytest.raises(P.MoeError, match="current device is cuda:1"):
            call()
    monkeypatch.setattr(_adapt, "_device", lambda: 0)
    opt.step()
    (_, (table, count, options, stream)), = lib.calls
    assert count == 1 and table[0].grad == opt.grads[0].data_ptr() and opt.steps_done == 1


def test_bound_tensors_stay_alive_and_counted(lib):
    """What a caller does to the lists and tensors it gave or reads back changes
    neither the table's memory nor its length."""
    import gc
    zeros = lambda: [on(torch.zeros(8 + i)) for i in range(2)]        # noqa: E731
    params, grads, moments = zeros(), zeros(), {"m": zeros(), "v": zeros()}
    opt = P.AdamW(params, grads, state=moments)
    opt.step()
    table = lib.calls[-1][1][0]
    addresses = [[getattr(e, f) for e in table] for f in ("param", "grad", "m", "v")]
    for name in ("params", "grads", "copies", "state"):
        with pytest.raises(AttributeError):
            setattr(opt, name, None)
    for read in (opt.params, opt.grads, opt.state["m"]):
        with pytest.raises((TypeError, AttributeError)):
            read[0] = on(torch.zeros(8))
        with pytest.raises(AttributeError):
            read.append(on(torch.zeros(8)))
    opt.state["m"] = zeros()                       # of a copy
    for held in (params, grads, moments["m"], moments["v"]):
        held[0].data = torch.zeros(8)
        held.pop()
    moments.clear()
    gc.collect()
    opt.step()
    table, count = lib.calls[-1][1][:2]
    assert count == 2 and [[getattr(e, f) for e in table] for f in ("param", "grad", "m", "v")] == addresses
    held = opt.params + opt.grads + opt.state["m"] + opt.state["v"]
    assert [t.data_ptr() for t in held] == sum(addresses, [])
    again = P.AdamW(opt.params, opt.grads, state=opt.state, steps_done=opt.steps_done)
    assert again.params[1].data_ptr() == addresses[0][1] and again.copies is None


def test_captured_step_wants_its_number(lib, monkeypatch):
    """A graph repeats the step number it was captured with, so that one counted
    here would be wrong from the second replay on."""
    opt = adamw()
    opt.step()
    monkeypatch.setattr(_adapt, "_capturing", lambda: True, raising=False)
    with pytest.raises(P.MoeError, match="captured step"):
        opt.step()
    assert len(lib.calls) == 1 and opt.steps_done == 1
    opt.step(step=7)
    assert lib.calls[-1][1][2].step == 7 and opt.steps_done == 1     # nothing has run
    monkeypatch.setattr(_adapt, "_capturing", lambda: False)
    opt.step()
    assert lib.calls[-1][1][2].step == 2 and opt.steps_done == 2


def test_sizes_past_32_bits_are_refused(lib):
    """Not taken modulo 2^32 (of views that repeat a row, which cost no memory)."""
    n = 2 ** 32 + 4

    class Dense(OnDevice):
        def is_contiguous(self):
            return True

        def stride(self):
            return 64, 1

    def long(*shape, dtype):
        return torch.zeros(1, dtype=dtype).expand(n, *shape).as_subclass(Dense)

    op = adapters()
    x, ids = long(64, dtype=torch.bfloat16), long(dtype=torch.int32)
    out = long(32, dtype=torch.bfloat16)
    calls = [lambda: op.forward(x, ids, out=out),
             lambda: op.backward(long(32, dtype=torch.float32), x, ids, need_dx=False),
             lambda: P.BalanceLoss(1, 1)(long(1, dtype=torch.float32), long(1, dtype=torch.int32), need_grad=False),
             lambda: P.BalanceLoss(2 ** 32 + 8, 2), lambda: P.BalanceLoss(8, 2 ** 32 + 2),
             lambda: adamw().step(step=2 ** 32 + 1)]
    for i, call in enumerate(calls):
        with pytest.raises(P.MoeError, match="2\\^31"):
            call()
            pytest.fail(f"refusal {i} did not come")
    assert not lib.calls
