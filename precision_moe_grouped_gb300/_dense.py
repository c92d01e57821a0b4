"""A dense gated feed-forward block beside the routed experts (a shared expert,
a dense layer), over the C ABI (include/moe.h).

As in _adapt, every tensor is checked before the library sees its address, a
bad one raises MoeError, calls run on the current stream of the current
device, and a call's workspace comes from torch's allocator for that stream.
"""
from __future__ import annotations

import bisect

from . import _adapt as A
from . import _lib
from ._adapt import _check_flat, _check_rows, _int32, _ptr, _rows, _same_device, _same_layout, _scratch
from ._lib import FfnShape, _bad, check

torch = None   # bound when the first object is made: the build imports this package without it


def _bind_torch() -> None:
    global torch
    if torch is None:
        A._bind_torch()
        torch = A.torch


def _bytes(t) -> tuple:
    """(first, behind the last) of a contiguous tensor's bytes."""
    at = t.data_ptr()
    return at, at + t.numel() * t.element_size()


class _Status:
    """A device word where kernels record a bounded wait that ran out."""

    def _new_status(self, device) -> None:
        self._status = torch.zeros(1, dtype=torch.int32, device=device)
        self._at_status = self._status.data_ptr()

    def device_status(self) -> int:
        """MOE_OK, or the first device-side error of this object's calls
        (MOE_ERR_DEVICE_TIMEOUT: results since then are undefined).  Waits for
        the device."""
        return int(self._status.item())


class GatedFFN(_Status):
    """out = base + (silu(x Wg^T) * (x Wu^T)) Wd^T, in bf16 with float sums.

    w_gate_up bf16 [2 I, H] (rows 0 .. I-1 the gate projection, I .. 2I-1 the
    up projection), w_down bf16 [H, I]; H and I multiples of 8.  The weights
    are read at every call, so that an update in place takes effect with the
    next one.  So does another tensor in their place, by assignment here or to
    a tensor's .data: a call that finds other memory, another shape, type or
    layout checks it, and refuses what is not as at the start.

    Nothing here is recorded for autograd: outputs require no gradient whatever
    the inputs do, and backward() is called by hand."""

    def __init__(self, w_gate_up, w_down):
        _bind_torch()
        dev = A._device()
        if w_gate_up is None or w_gate_up.dim() != 2 or w_gate_up.shape[0] % 2:
            _bad("w_gate_up must be [2 * features, hidden]")
        I, H = self.inter, self.hidden = w_gate_up.shape[0] // 2, w_gate_up.shape[1]
        self._shapes = torch.Size((2 * I, H)), torch.Size((H, I))
        self.w_gate_up, self.w_down, self.device, self._dev = w_gate_up, w_down, w_gate_up.device, dev
        self._check_weights(_ptr(w_gate_up), _ptr(w_down))
        self._lib, self._sizes = A.load(), {}
        self._call(0, 0)   # rejects unsupported sizes here
        self._new_status(self.device)

    def _check_weights(self, *at) -> None:
        """Checks the weights, which are not as in the last call.  That one's
        memory is held (detached): while it was the last call's, no other tensor
        but its views could get its addresses."""
        for t, name, shape in zip((self.w_gate_up, self.w_down), ("w_gate_up", "w_down"), self._shapes):
            _check_flat(t, name, torch.bfloat16, shape, self._dev)
        self._held = [self.w_gate_up.detach(), self.w_down.detach()]
        self._at = at

    def _call(self, T: int, backward: int):
        """(shape, workspace bytes) of a call with T tokens."""
        got = self._sizes.get((T, backward))
        if got is None:
            _int32("tokens and features", T, self.hidden, self.inter)
            s = FfnShape(T, self.hidden, self.inter)
            n = self._lib.moe_ffn_workspace_size(s, backward)
            if n == 0:
                raise _lib.MoeError(_lib.MOE_ERR_INVALID_ARG, self._lib.moe_last_error().decode())
            if len(self._sizes) > 4096:
                self._sizes.clear()
            got = self._sizes[(T, backward)] = (s, n)
        return got

    def _start(self):
        """(device, addresses of the weights), checked."""
        dev = A._device()
        if dev != self._dev:
            _same_device(dev, self._dev)
        w, d, (w_shape, d_shape) = self.w_gate_up, self.w_down, self._shapes
        at = _ptr(w), _ptr(d)
        if (at != self._at or not _same_layout(w, torch.bfloat16, w_shape)
                or not _same_layout(d, torch.bfloat16, d_shape)):
            self._check_weights(*at)
        return dev, at

    def forward(self, x, base=None, out=None):
        """base + the block's output: bf16 [T, H].  x and base bf16 [T, H], rows
        may be strided; `out` may be `base` itself, or x, and shares no memory with
        the call's tensors otherwise (a call where it does is refused)."""
        dev, (wgu, wd) = self._start()
        T, H = _rows(x, "x"), self.hidden
        shape, bf16 = (T, H), torch.bfloat16
        ld_x = _check_rows(x, "x", bf16, shape, dev)
        ld_base = 0 if base is None else _check_rows(base, "base", bf16, shape, dev)
        if out is None:
            out, ld_out = torch.empty(shape, dtype=bf16, device=self.device), H
        else:
            ld_out = _check_rows(out, "out", bf16, shape, dev)
        s, n = self._call(T, 0)
        ws = _scratch(n, x)
        rc = self._lib.moe_ffn_forward(s, x.data_ptr(), ld_x, wgu, wd, _ptr(base), ld_base,
                                       out.data_ptr(), ld_out, ws.data_ptr(), n, self._at_status,
                                       A._raw_stream(dev))
        if rc:
            check(rc)
        return out

    __call__ = forward

    def backward(self, dout, x, dx_base=None, dx=None, dw_gate_up=None, dw_down=None,
                 need_dx: bool = True, need_weights: bool = True):
        """(dx, dw_gate_up, dw_down), all bf16, for dout bf16 [T, H]: dx [T, H]
        with dx_base added, the weights' gradients in the weights' shapes (zero
        without tokens; of at most 65536 tokens a call).  The activations are
        computed again from x.  What is not needed comes back as None.  `dx` may
        be `dx_base`; what is written shares no memory with the call's tensors
        otherwise (a call where it does is refused)."""
        dev, (wgu, wd) = self._start()
        T, H = _rows(x, "x"), self.hidden
        shape, bf16 = (T, H), torch.bfloat16
        ld_dout = _check_rows(dout, "dout", bf16, shape, dev)
        ld_x = _check_rows(x, "x", bf16, shape, dev)
        ld_dx = ld_base = 0
        if not need_dx:
            dx = dx_base = None
        elif dx is None:
            dx, ld_dx = torch.empty(shape, dtype=bf16, device=self.device), H
        else:
            ld_dx = _check_rows(dx, "dx", bf16, shape, dev)
        if dx_base is not None:
            ld_base = _check_rows(dx_base, "dx_base", bf16, shape, dev)
        if not need_weights:
            dw_gate_up = dw_down = None
        else:
            if dw_gate_up is None:
                dw_gate_up = torch.empty(self._shapes[0], dtype=bf16, device=self.device)
            else:
                _check_flat(dw_gate_up, "dw_gate_up", bf16, self._shapes[0], dev)
            if dw_down is None:
                dw_down = torch.empty(self._shapes[1], dtype=bf16, device=self.device)
            else:
                _check_flat(dw_down, "dw_down", bf16, self._shapes[1], dev)
        s, n = self._call(T, 1)
        ws = _scratch(n, x)
        rc = self._lib.moe_ffn_backward(s, dout.data_ptr(), ld_dout, x.data_ptr(), ld_x, wgu, wd,
                                        _ptr(dx_base), ld_base, _ptr(dx), ld_dx, _ptr(dw_gate_up),
                                        _ptr(dw_down), ws.data_ptr(), n, self._at_status,
                                        A._raw_stream(dev))
        if rc:
            check(rc)
        return dx, dw_gate_up, dw_down


class Muon(_Status):
    """Steps over weight matrices whose update is made (nearly) orthogonal by
    Newton-Schulz steps on the momentum (the formulas: moe_muon_step in
    include/moe.h).

    params: contiguous float32 CUDA tensors [rows, cols], or [n, rows, cols] for
    n matrices (a pool of adapters; a gate and an up projection as two), updated
    in place; grads: tensors of the same shapes, all float32 or all bfloat16;
    copies: bfloat16 tensors of the same shapes that receive the rounded
    parameters, or None.  `state`: the momenta, float32 of the same shapes, to
    resume from; by default they start at zero.  What is written (params, state,
    copies) shares no memory with another tensor: calls where it does are refused.
    update_scale "rms" makes an
    update's root mean square about 0.2 whatever the shape, "spectral" its
    largest singular value about sqrt(max(1, rows / cols)).  The tensors are
    bound and held here (params, grads, copies and state name them and cannot be
    assigned): after replacing a parameter's or a gradient's memory, build a new
    Muon (state=old.state) or pass the new gradients to step().

    lr, momentum, weight_decay, eps, nesterov, ns_steps, ns_coefficients and
    update_scale are read at every step.  They are the host's: a step captured
    into a CUDA graph repeats the capture's at every replay."""

    def __init__(self, params, grads, copies=None, state=None, lr: float = 1e-3,
                 momentum: float = 0.95, nesterov: bool = True, weight_decay: float = 0.1,
                 eps: float = 1e-7, ns_steps: int = 5, ns_coefficients=(3.4445, -4.7750, 2.0315),
                 update_scale: str = "rms"):
        _bind_torch()
        dev = self._dev = A._device()
        # detached: keeps the bound memory alive whatever becomes of the originals
        bound = self._params = tuple(A._detached(params, "params"))
        self.lr, self.momentum, self.nesterov, self.weight_decay = lr, momentum, nesterov, weight_decay
        self.eps, self.ns_steps, self.ns_coefficients = eps, ns_steps, ns_coefficients
        self.update_scale = update_scale
        for i, p in enumerate(bound):
            if p.dim() not in (2, 3):
                _bad(f"params[{i}] must be [rows, cols] or [n, rows, cols], got {tuple(p.shape)}")
            _int32(f"params[{i}]'s sizes", *p.shape)
            _check_flat(p, f"params[{i}]", torch.float32, p.shape, dev)
        if state is None:
            state = [torch.zeros_like(p) for p in bound]
        self._state = self._bound(state, "state", torch.float32)
        self._copies = None if copies is None else self._bound(copies, "copies", torch.bfloat16)
        written = sorted(_bytes(t) for t in (*bound, *self._state, *(self._copies or ())) if t.numel())
        if any(a[1] > b[0] for a, b in zip(written, written[1:])):
            _bad("params, state and copies must be distinct memory")   # all written, side by side
        self._written = [a for a, _ in written], [b for _, b in written]
        self._table = (_lib.MuonTensor * max(1, len(bound)))()
        for i, (e, p, m) in enumerate(zip(self._table, bound, self._state)):
            e.param, e.momentum = p.data_ptr(), m.data_ptr()
            e.count = p.shape[0] if p.dim() == 3 else 1
            e.rows, e.cols = p.shape[-2:]
            e.param_bf16 = None if self._copies is None else self._copies[i].data_ptr()
        self._options = _lib.MuonOptions()
        self._lib = A.load()
        self.bind_grads(grads)
        self._sized = None
        self._workspace_size()   # rejects unsupported sizes here
        self._new_status(torch.device("cuda", dev) if dev is not None else None)

    def _bound(self, tensors, name: str, dtype) -> tuple:
        held = tuple(A._detached(tensors, name))
        if len(held) != len(self._params):
            _bad(f"{name} must hold {len(self._params)} tensors")
        for i, (t, p) in enumerate(zip(held, self._params)):
            _check_flat(t, f"{name}[{i}]", dtype, p.shape, self._dev)
        return held

    def _is_written(self, t) -> bool:
        """Whether a step writes any byte of t."""
        begin, end = _bytes(t)
        i = bisect.bisect_left(self._written[0], end)
        return begin < end and i > 0 and self._written[1][i - 1] > begin

    @property
    def params(self) -> tuple:
        return self._params

    @property
    def grads(self) -> tuple:
        return self._grads

    @property
    def copies(self) -> tuple | None:
        return self._copies

    @property
    def state(self) -> tuple:
        return self._state

    def bind_grads(self, grads) -> None:
        """Take the next steps' gradients from these tensors."""
        grads = tuple(A._detached(grads, "grads"))
        _same_device(A._device(), self._dev)
        kind = grads[0].dtype if grads else torch.float32
        if kind not in (torch.float32, torch.bfloat16):
            _bad(f"grads must be float32 or bfloat16, got {kind}")
        grads = self._bound(grads, "grads", kind)
        if any(map(self._is_written, grads)):   # read again after a momentum is written
            _bad("grads must not share memory with params, state or copies")
        self._grads = grads
        for e, t in zip(self._table, self._grads):
            e.grad = t.data_ptr()
        self._options.grad_dtype = _lib.MOE_DTYPE_F32 if kind == torch.float32 else _lib.MOE_DTYPE_BF16

    def _workspace_size(self) -> int:
        o = self._options
        if self.update_scale not in ("rms", "spectral"):
            _bad(f"update_scale must be 'rms' or 'spectral', got {self.update_scale!r}")
        if len(self.ns_coefficients) != 3:
            _bad("ns_coefficients must be three numbers")
        _int32("ns_steps", self.ns_steps)
        o.lr, o.momentum, o.weight_decay, o.eps = self.lr, self.momentum, self.weight_decay, self.eps
        o.coefficients[:] = self.ns_coefficients
        o.ns_steps, o.nesterov = self.ns_steps, bool(self.nesterov)
        o.update_scale = _lib.MOE_MUON_RMS if self.update_scale == "rms" else _lib.MOE_MUON_SPECTRAL
        # the sizes are bound: only what the schedule of the steps depends on can change the need
        key = o.ns_steps, tuple(o.coefficients), o.lr, o.momentum, o.weight_decay, o.eps
        if key != self._sized:
            n = self._lib.moe_muon_workspace_size(self._table, len(self._params), o)
            if n == 0:
                raise _lib.MoeError(_lib.MOE_ERR_INVALID_ARG, self._lib.moe_last_error().decode())
            self._sized, self._need = key, n
        return self._need

    def step(self, grads=None, grad_scale=None) -> None:
        """One step, in place.  grad_scale: float32 CUDA scalar every gradient is
        multiplied by."""
        if grads is not None:
            self.bind_grads(grads)
        dev, o = A._device(), self._options
        _same_device(dev, self._dev)
        o.grad_scale = None if grad_scale is None else A._check_numel(
            grad_scale, "grad_scale", 0, torch.float32, 1, dev)
        if grad_scale is not None and self._is_written(grad_scale):
            _bad("grad_scale must not share memory with params, state or copies")
        n = self._workspace_size()
        ws = _scratch(n, self._status)
        check(self._lib.moe_muon_step(self._table, len(self._params), o, ws.data_ptr(), n,
                                      self._at_status, A._raw_stream(dev)))
