"""A dense gated feed-forward block beside the routed experts (a shared expert,
a dense layer), over the C ABI (include/moe.h).

As in _adapt, every tensor is checked before the library sees its address, a
bad one raises MoeError, calls run on the current stream of the current
device, and a call's workspace comes from torch's allocator for that stream.
"""
from __future__ import annotations

from . import _adapt as A
from . import _lib
from ._adapt import _check_flat, _check_rows, _int32, _ptr, _rows, _same_device, _scratch
from ._lib import FfnShape, _bad, check

torch = None   # bound when the first object is made: the build imports this package without it


def _bind_torch() -> None:
    global torch
    if torch is None:
        A._bind_torch()
        torch = A.torch


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
    a tensor's .data: a call that finds other memory checks it.

    Nothing here is recorded for autograd: outputs require no gradient whatever
    the inputs do, and backward() is called by hand."""

    def __init__(self, w_gate_up, w_down):
        _bind_torch()
        dev = A._device()
        if w_gate_up is None or w_gate_up.dim() != 2 or w_gate_up.shape[0] % 2:
            _bad("w_gate_up must be [2 * features, hidden]")
        I, H = self.inter, self.hidden = w_gate_up.shape[0] // 2, w_gate_up.shape[1]
        self._shapes = (2 * I, H), (H, I)
        self.w_gate_up, self.w_down, self.device, self._dev = w_gate_up, w_down, w_gate_up.device, dev
        self._check_weights(_ptr(w_gate_up), _ptr(w_down))
        self._lib, self._sizes = A.load(), {}
        self._call(0, 0)   # rejects unsupported sizes here
        self._new_status(self.device)

    def _check_weights(self, *at) -> None:
        """Checks the weights, whose addresses are not the last call's.  That one's
        memory is held (detached): while it was the last call's, no other tensor
        could get its addresses."""
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
        at = _ptr(self.w_gate_up), _ptr(self.w_down)
        if at != self._at:
            self._check_weights(*at)
        return dev, at

    def forward(self, x, base=None, out=None):
        """base + the block's output: bf16 [T, H].  x and base bf16 [T, H], rows
        may be strided; `out` may be `base` itself, or x."""
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
        without tokens).  The activations are computed again from x.  What is
        not needed comes back as None.  `dx` may be `dx_base`, not x or dout."""
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
