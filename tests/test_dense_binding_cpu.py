"""What the binding of the gated feed-forward block and of the orthogonalised
step hands to the library, without a GPU: host tensors that say they are on
device 0, and a library whose launches are recorded instead of made."""
import ctypes
import gc
import os

import pytest
import torch

import precision_moe_grouped_gb300 as P
from precision_moe_grouped_gb300 import _adapt, _dense
from precision_moe_grouped_gb300 import _lib as L

BF16 = torch.bfloat16


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
        if name in ("moe_ffn_forward", "moe_ffn_backward", "moe_muon_step"):
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
    _dense._bind_torch()
    r = Recorder(P.load())
    monkeypatch.setattr(_adapt, "load", lambda: r)
    monkeypatch.setattr(_adapt, "_device", lambda: 0)
    monkeypatch.setattr(_adapt, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(_dense._Status, "_new_status",
                        lambda self, device: setattr(self, "_status", on(torch.zeros(1, dtype=torch.int32))) or
                        setattr(self, "_at_status", self._status.data_ptr()))
    return r


def zeros(*shape, dtype=BF16):
    return on(torch.zeros(*shape, dtype=dtype))


def ffn(H=64, I=32):
    return P.GatedFFN(zeros(2 * I, H), zeros(H, I))


def test_ffn_arguments(lib):
    op = ffn()
    x = zeros(5, 96)[:, 16:80]           # rows 96 apart
    base, out = zeros(5, 64), zeros(10, 64)[::2]
    assert op(x, base=base, out=out) is out
    name, (s, xp, ld_x, wgu, wd, bp, ld_base, op_, ld_out, ws, n, status, stream) = lib.calls.pop()
    assert name == "moe_ffn_forward" and (s.num_tokens, s.hidden, s.inter) == (5, 64, 32)
    assert (xp, ld_x, bp, ld_base, op_, ld_out) == (x.data_ptr(), 96, base.data_ptr(), 64, out.data_ptr(), 128)
    assert (wgu, wd, status) == (op.w_gate_up.data_ptr(), op.w_down.data_ptr(), op._status.data_ptr())
    assert n == lib.moe_ffn_workspace_size(s, 0) and ws
    dout, dx = zeros(5, 64), zeros(5, 72)[:, :64]
    got = op.backward(dout, x, dx_base=base, dx=dx)
    _, a = lib.calls.pop()
    assert got[0] is dx and got[1].shape == (64, 64) and got[2].shape == (64, 32)
    assert all(t.dtype is BF16 for t in got)
    assert a[1:5] == (dout.data_ptr(), 64, x.data_ptr(), 96) and a[7:11] == (base.data_ptr(), 64, dx.data_ptr(), 72)
    assert a[11:13] == (got[1].data_ptr(), got[2].data_ptr())
    got = op.backward(dout, x, need_dx=False, dx=dx, dx_base=base)
    _, a = lib.calls.pop()
    assert got[0] is None and a[7:11] == (None, 0, None, 0)
    got = op.backward(dout, x, need_weights=False)
    _, a = lib.calls.pop()
    assert got[1] is None and got[2] is None and a[11:13] == (None, None)
    # a single row's stride says nothing
    op(zeros(1, 3, 64)[:, 1])
    assert lib.calls.pop()[1][2] == 64


def test_ffn_refuses(lib):
    op, x = ffn(), zeros(5, 64)
    bad = [None, torch.zeros(5, 64, dtype=BF16), zeros(5, 64, dtype=torch.float16), zeros(5, 56), zeros(4, 64)[:, :32],
           zeros(64, 5).T, zeros(5, 128)[:, ::2], zeros(5)]
    for t in bad:
        with pytest.raises(P.MoeError):
            op(t)
        with pytest.raises(P.MoeError):
            op.backward(t, x)
        for k in ("base", "out"):
            if t is not None:
                with pytest.raises(P.MoeError):
                    op(x, **{k: t})
        for k in ("dx", "dx_base", "dw_gate_up", "dw_down"):
            if t is not None:
                with pytest.raises(P.MoeError):
                    op.backward(x, x, **{k: t})
    for t in (zeros(64, 64, dtype=torch.float32), zeros(64, 128)[:, ::2], zeros(32, 64)):
        with pytest.raises(P.MoeError):
            op.backward(x, x, dw_gate_up=t)
    for w, d in ((zeros(63, 64), zeros(64, 32)), (zeros(64, 64), zeros(32, 64)), (zeros(64, 64), None),
                 (None, zeros(64, 32)), (zeros(64, 64, dtype=torch.float32), zeros(64, 32)), (zeros(64, 60), zeros(60, 32)),
                 (zeros(24, 64), zeros(64, 12)), (zeros(2, 64, 64), zeros(64, 32)),
                 (torch.zeros(64, 64, dtype=BF16), zeros(64, 32))):
        with pytest.raises(P.MoeError):
            P.GatedFFN(w, d)
    assert not lib.calls


def test_ffn_weights_are_checked_at_every_call(lib):
    """Weights whose memory, type or size changed after the construction."""
    x = zeros(4, 64)
    for name, bad in (("w_gate_up", [zeros(64, 32), zeros(64, 64, dtype=torch.float32), zeros(64, 128)[:, ::2],
                                     torch.zeros(64, 64, dtype=BF16), None]),
                      ("w_down", [zeros(32, 64), zeros(64, 32, dtype=torch.float16), None])):
        for t in bad:
            op = ffn()
            setattr(op, name, t)
            for call in (lambda: op(x), lambda: op.backward(x, x)):
                with pytest.raises((P.MoeError, AttributeError)) as e:
                    call()
                assert t is None or e.type is P.MoeError
    assert not lib.calls
    op = ffn()
    new = zeros(64, 64)
    op.w_gate_up = new
    op(x)
    op.backward(x, x)
    assert lib.calls[0][1][3] == lib.calls[1][1][5] == new.data_ptr()
    op.w_down.data = torch.zeros(1, dtype=BF16)
    with pytest.raises(P.MoeError):
        op(x)
    assert len(op._held) == 2


def test_ffn_weights_in_the_same_memory(lib):
    """Another tensor at the old address, by assignment or to .data: one of another layout, type or size is refused,
    as it is at an address of its own."""
    x = zeros(4, 64)
    for name, others in (("w_down", [lambda t: t.t(), lambda t: t.view(torch.float16), lambda t: t.view(32, 128),
                                     lambda t: t[:, :32], lambda t: t.view(-1), lambda t: t[:32]]),
                         ("w_gate_up", [lambda t: t.view(torch.int16), lambda t: t[:64], lambda t: t.view(64, 128)])):
        for other in others:
            for assign in (True, False):
                op = ffn(64, 64)
                old = getattr(op, name)
                new = other(old)
                assert new.data_ptr() == old.data_ptr()
                if assign:
                    setattr(op, name, new)
                elif new.dtype is BF16:
                    old.data = other(old.data)
                else:
                    continue
                for call in (lambda: op(x), lambda: op.backward(x, x)):
                    with pytest.raises(P.MoeError, match=name):
                        call()
                setattr(op, name, zeros(64, 64) if name == "w_down" else zeros(128, 64))
                op(x)
    assert all(name == "moe_ffn_forward" for name, _ in lib.calls)
    # the same rows again are no other tensor
    op, calls = ffn(), len(lib.calls)
    op.w_down = op.w_down[:]
    op(x)
    assert len(lib.calls) == calls + 1


def muon(shapes=((3, 20, 30), (40, 16)), grads=torch.float32, copies=True, **kw):
    z = lambda kind: [zeros(*s, dtype=kind) for s in shapes]                       # noqa: E731
    return P.Muon(z(torch.float32), z(grads), copies=z(BF16) if copies else None, state=z(torch.float32), **kw)


def test_muon_gradients_are_memory_of_their_own(lib):
    """Gradients are read again after the first momentum is written."""
    op = muon(grads=BF16)
    for held, kind in ((op.params, torch.float32), (op.state, torch.float32), (op.copies, BF16)):
        grads = [zeros(3, 20, 30, dtype=kind), held[1]]
        with pytest.raises(P.MoeError):
            op.bind_grads(grads)
        with pytest.raises(P.MoeError):
            op.step(grads=grads)
    assert op.grads[0].dtype is BF16 and not any(name == "moe_muon_step" for name, *_ in lib.calls)
    op.step()


def test_muon_tensors_share_no_memory(lib):
    """Slices of one buffer: end to end they are accepted; what is written may not begin or end inside another tensor,
    nor lie in one."""
    f32 = torch.float32
    room, half = zeros(400, dtype=f32), zeros(400)
    part = lambda at, of=room: of[at:at + 48].view(8, 6)                          # noqa: E731
    good = dict(params=[part(0), part(48)], grads=[part(192), part(192)], state=[part(96), part(144)],
                copies=[part(0, half), part(48, half)])
    op = P.Muon(**good)
    op.step()
    assert len(lib.calls) == 1
    for bad in (dict(params=[part(0), part(47)]), dict(state=[part(49), part(144)]), dict(state=[part(96), part(97)]),
                dict(copies=[part(0, half), part(47, half)]), dict(copies=[part(0, half), room[50:74].view(BF16).view(8, 6)]),
                dict(params=[part(0), room[20:26].view(1, 6)], state=[part(96), part(144)[:1]], grads=[part(192), part(192)[:1]],
                     copies=None)):
        with pytest.raises(P.MoeError, match="distinct"):
            P.Muon(**{**good, **bad})
    for grads in ([part(192), part(1)], [part(145), part(300)], [part(191), part(300)], [part(192), part(47)]):
        for call in (lambda: P.Muon(**{**good, "grads": grads}), lambda: op.bind_grads(grads), lambda: op.step(grads)):
            with pytest.raises(P.MoeError, match="grads must not"):
                call()
    for at in (0, 191):
        with pytest.raises(P.MoeError, match="grad_scale must not"):
            op.step(grad_scale=room[at])
    assert len(lib.calls) == 1
    op.step(grad_scale=room[192])
    # a tensor without elements has no bytes
    P.Muon([part(0), room[20:20].view(0, 6)], [part(192), room[0:0].view(0, 6)], state=[part(96), room[100:100].view(0, 6)]).step()


def test_muon_arguments(lib):
    op = muon(lr=0.5, momentum=0.25, weight_decay=0.125, eps=1e-3, ns_steps=3, nesterov=False,
              ns_coefficients=(2.0, -1.5, 0.5), update_scale="spectral")
    op.step()
    name, (table, count, o, ws, n, status, stream) = lib.calls.pop()
    assert name == "moe_muon_step" and count == 2 and status == op._status.data_ptr() and n and ws
    assert [(e.count, e.rows, e.cols) for e in table] == [(3, 20, 30), (1, 40, 16)]
    for e, p, g, m, c in zip(table, op.params, op.grads, op.state, op.copies):
        assert (e.param, e.grad, e.momentum, e.param_bf16) == tuple(t.data_ptr() for t in (p, g, m, c))
    assert (o.lr, o.momentum, o.weight_decay, o.eps, o.ns_steps, o.nesterov) == (0.5, 0.25, 0.125, 1e-3, 3, 0)
    assert tuple(o.coefficients) == (2.0, -1.5, 0.5) and o.update_scale == L.MOE_MUON_SPECTRAL
    assert o.grad_dtype == L.MOE_DTYPE_F32 and o.grad_scale is None
    # read at every step
    op.lr, op.momentum, op.weight_decay, op.nesterov, op.update_scale = 1.0, 0.5, 0.0, True, "rms"
    op.ns_steps, op.ns_coefficients = 7, (3.0, -3.0, 1.0)
    scale = zeros(1, dtype=torch.float32)
    grads = [zeros(*p.shape) for p in op.params]
    op.step(grads, grad_scale=scale)
    o, table = lib.calls[-1][1][2], lib.calls[-1][1][0]
    assert (o.lr, o.momentum, o.weight_decay, o.nesterov, o.update_scale) == (1.0, 0.5, 0.0, 1, L.MOE_MUON_RMS)
    assert (o.ns_steps, tuple(o.coefficients)) == (7, (3.0, -3.0, 1.0)) and o.grad_scale == scale.data_ptr()
    assert o.grad_dtype == L.MOE_DTYPE_BF16 and [e.grad for e in table] == [g.data_ptr() for g in grads]
    op.step()
    assert lib.calls[-1][1][2].grad_scale is None
    for name, value in (("ns_steps", 0), ("ns_steps", 13), ("ns_steps", 1 << 40), ("ns_coefficients", (1.0, 2.0)),
                        ("ns_coefficients", (1.5, -0.5, 0.0)), ("update_scale", "other"), ("eps", 0.0), ("momentum", 1.0),
                        ("lr", float("nan"))):
        old, calls = getattr(op, name), len(lib.calls)
        setattr(op, name, value)
        with pytest.raises(P.MoeError):
            op.step()
        setattr(op, name, old)
        op.step()
        assert len(lib.calls) == calls + 1


def test_muon_refuses(lib):
    f32 = torch.float32
    good = dict(params=[zeros(8, 6, dtype=f32)], grads=[zeros(8, 6, dtype=f32)])
    bad = {"params": [None, [None], [zeros(8, 6)], [zeros(48, dtype=f32)], [zeros(1, 1, 8, 6, dtype=f32)],
                      [zeros(8, 12, dtype=f32)[:, ::2]], [torch.zeros(8, 6)]],
           "grads": [None, [], [None], [zeros(6, 8, dtype=f32)], [zeros(8, 6, dtype=torch.float16)],
                     [zeros(6, 8, dtype=f32).T]],
           "copies": [[], [zeros(8, 6, dtype=f32)], [zeros(6, 8)]],
           "state": [[], [zeros(8, 6)], [zeros(6, 8, dtype=f32)], {"m": [zeros(8, 6, dtype=f32)]}]}
    for name, values in bad.items():
        for v in values:
            with pytest.raises(P.MoeError):
                P.Muon(**{**good, **{name: v}})
    p = good["params"][0]
    for again in (dict(params=[p, p], grads=[p, p]), dict(state=[p])):       # written twice in a step
        with pytest.raises(P.MoeError, match="distinct"):
            P.Muon(**{**good, **again})
    with pytest.raises(P.MoeError):
        P.Muon([zeros(3, 4, dtype=f32), zeros(3, 4, dtype=f32)], [zeros(3, 4, dtype=f32), zeros(3, 4)])
    op = muon()
    with pytest.raises(P.MoeError):
        op.step(grad_scale=zeros(2, dtype=f32))
    with pytest.raises(P.MoeError):
        op.step([zeros(3, 20, 30, dtype=f32)])
    assert not lib.calls
    P.Muon([], []).step()                                                   # nothing to do


def test_muon_holds_what_it_bound(lib):
    params, grads = [zeros(8, 6, dtype=torch.float32)], [zeros(8, 6, dtype=torch.float32)]
    op = P.Muon(params, grads, state=[zeros(8, 6, dtype=torch.float32)])
    addresses = [(e.param, e.grad, e.momentum) for e in op._table]
    for name in ("params", "grads", "copies", "state"):
        with pytest.raises(AttributeError):
            setattr(op, name, None)
    params[0].data = torch.zeros(1)
    params[0], grads[0] = None, None
    gc.collect()
    keep = [torch.zeros(8, 6) for _ in range(50)]                           # would take freed memory
    op.step()
    assert [(e.param, e.grad, e.momentum) for e in lib.calls[-1][1][0]] == addresses
    assert not {t.data_ptr() for t in keep} & set(addresses[0])
    view = (ctypes.c_float * 48).from_address(addresses[0][0])
    view[0] = 1.0
    assert float(op.params[0][0, 0]) == 1.0


def test_another_current_device_is_refused(lib, monkeypatch):
    op, block, x = muon(), ffn(), zeros(4, 64)
    monkeypatch.setattr(_adapt, "_device", lambda: 1)
    for call in (op.step, lambda: op.bind_grads(op.grads), lambda: block(x), lambda: block.backward(x, x)):
        with pytest.raises(P.MoeError, match="current device is cuda:1"):
            call()
    assert not lib.calls


def test_host_tensors_are_refused():
    with pytest.raises(P.MoeError, match="CUDA"):
        P.GatedFFN(torch.zeros(64, 64, dtype=BF16), torch.zeros(64, 32, dtype=BF16))
    with pytest.raises(P.MoeError, match="CUDA"):
        P.Muon([torch.zeros(4, 4)], [torch.zeros(4, 4)])
