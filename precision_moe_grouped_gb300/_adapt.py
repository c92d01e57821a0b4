"""Adapting a frozen layer: low-rank adapters, the router's balance loss and
the AdamW step, over the C ABI (include/moe.h).

As in _lib, every tensor is checked (placement, device, dtype, shape, layout)
before the library sees its address, and a bad one raises MoeError.  Calls
run on the current stream of the current device; a call's workspace comes
from torch's allocator for that stream, so calls on different streams and
calls captured into a CUDA graph do not share one.
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import (MOE_ADAMW_BLOCK, MOE_DTYPE_BF16, MOE_DTYPE_F32,
                   AdamwOptions, AdamwTensor, AdapterShape, BalanceShape, _bad, _check_tensor,
                   check, load)

torch = None   # bound when the first object is made: the build imports this package without it
_raw_stream = None


def _bind_torch() -> None:
    global torch, _raw_stream
    if torch is None:
        import torch as module
        # the handle alone: building torch's stream object takes 3 us
        _raw_stream = getattr(module._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: module.cuda.current_stream(device).cuda_stream)
        torch = module


def _device() -> int | None:
    """The current CUDA device's index; None where there is none (every tensor
    then fails its check)."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() else _lib._current_device()


def _capturing() -> bool:
    """Whether the current stream is captured into a CUDA graph."""
    return torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()


def _int32(name: str, *values: int) -> None:
    """The structures' integers have 32 bits, and ctypes drops the rest."""
    for n in values:
        if not -1 << 31 <= n < 1 << 31:
            _bad(f"{name} must be below 2^31, got {n}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(t, name: str) -> int:
    try:
        return t.shape[0]
    except (AttributeError, IndexError):
        _bad(f"{name} must be a tensor of rows, got {t if t is None else type(t)}")


def _detached(ts, name: str) -> list:
    try:
        return [t.detach() for t in ts]
    except (AttributeError, TypeError):
        _bad(f"{name} must be a list of tensors")


def _check_rows(t, name: str, dtype, shape: tuple, device) -> int:
    """A [rows, cols] CUDA tensor with unit column stride; rows may be apart.
    Returns the elements between rows (a single row's stride says nothing)."""
    if t is None:
        _bad(f"{name} is None")
    if not t.is_cuda or t.get_device() != device:
        _bad(f"{name} is on {t.device}, the current device is cuda:{device}")
    if t.dtype is not dtype:
        _bad(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        _bad(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    row, col = t.stride()
    if col != 1 and shape[0] and shape[1] > 1:
        _bad(f"{name} must have unit stride along its rows")
    return row if shape[0] > 1 else shape[1]


def _check_flat(t, name: str, dtype, shape: tuple, device) -> None:
    """A contiguous CUDA tensor (_check_tensor at a fraction of its time)."""
    if not (t is not None and t.is_cuda and t.get_device() == device and t.dtype is dtype
            and t.shape == shape and t.is_contiguous()):
        _check_tensor(t, name, cuda=True, dtype=dtype, shape=shape, device=device)


def _same_layout(t, dtype, shape) -> bool:
    """What tells a tensor at a known address from a view of the same memory.
    (shape: torch.Size, which size() is compared with the quickest.)"""
    return t.dtype is dtype and t.size() == shape and t.is_contiguous()


def _same_device(device, made_on) -> None:
    if device != made_on:
        _bad(f"the current device is cuda:{device}, this object's tensors are on cuda:{made_on}")


def _check_numel(t, name: str, key, dtype, n: int, device) -> int:
    """A contiguous CUDA tensor of n elements (dtype None: of one byte each);
    returns its address."""
    if not (t is not None and t.is_cuda and t.get_device() == device and t.numel() == n
            and t.is_contiguous() and (t.dtype is dtype if dtype else t.element_size() == 1)):
        _check_tensor(t, f"{name}[{key}]", cuda=True, dtype=dtype, numel=n, device=device,
                      itemsize=None if dtype else 1)
    return t.data_ptr()


def _scratch(n: int, like):
    """The call's workspace, from torch's allocator for the current stream."""
    return torch.empty(n, dtype=torch.uint8, device=like.device)


class LowRankAdapters:
    """Pools of low-rank adapters beside a shared projection: token t of a
    call uses adapter a = ids[t] and gets scale[a] * b[a] @ (a[a] @ x[t])
    beside the projection's own result.

    a bf16 [NA, r, H], b bf16 [NA, N, r], scale float32 [NA] or None for 1;
    r, H and N multiples of 8, r <= 128, NA <= 1024.  The pools are read at
    every call, so that an update in place takes effect with the next one.  So
    does another tensor in their place, by assignment here or to a tensor's
    .data: a call that finds other memory, another shape, type or layout checks
    it, and refuses what is not as at the start (a module moved to the host or to
    another type).

    Nothing here is recorded for autograd: outputs require no gradient whatever
    the inputs do, and backward() is called by hand."""

    def __init__(self, a, b, scale=None):
        _bind_torch()
        dev = _device()
        if a is None or a.dim() != 3:
            _bad("a must be [adapters, rank, in_features]")
        NA, r, H = self.num_adapters, self.rank, self.in_features = tuple(a.shape)
        if b is None or b.dim() != 3:
            _bad("b must be [adapters, out_features, rank]")
        N = self.out_features = b.shape[1]
        self._dims, self._H, self._N = (NA, r, H, N), H, N
        self._shapes = torch.Size((NA, r, H)), torch.Size((NA, N, r)), torch.Size((NA,))
        self.a, self.b, self.scale, self.device, self._dev = a, b, scale, a.device, dev
        self._check_pools(a.data_ptr(), b.data_ptr(), _ptr(scale))
        self._lib = load()
        self._sizes = {}
        for kind in (MOE_DTYPE_BF16, MOE_DTYPE_F32):   # rejects unsupported sizes here
            self._call(0, kind, 0)

    def _check_pools(self, *at) -> None:
        """Checks a, b and scale, which are not as in the last call.  That one's
        memory is held (detached): while it was the last call's, no other tensor
        but its views could get its addresses."""
        shapes = self._shapes
        _check_flat(self.a, "a", torch.bfloat16, shapes[0], self._dev)
        _check_flat(self.b, "b", torch.bfloat16, shapes[1], self._dev)
        if self.scale is not None:
            _check_flat(self.scale, "scale", torch.float32, shapes[2], self._dev)
        self._held = [t.detach() for t in (self.a, self.b, self.scale) if t is not None]
        self._at_a, self._at_b, self._at_scale = at

    def _addresses(self):
        """(a, b, scale) of the pools, checked."""
        pa, pb, ps, shapes = self.a, self.b, self.scale, self._shapes
        a, b, scale = _ptr(pa), _ptr(pb), _ptr(ps)
        if (a != self._at_a or b != self._at_b or scale != self._at_scale
                or not _same_layout(pa, torch.bfloat16, shapes[0])
                or not _same_layout(pb, torch.bfloat16, shapes[1])
                or ps is not None and not _same_layout(ps, torch.float32, shapes[2])):
            self._check_pools(a, b, scale)
        return a, b, scale

    def _call(self, T: int, kind: int, backward: int):
        """(shape, workspace bytes) of a call with T tokens."""
        got = self._sizes.get((T, kind, backward))
        if got is None:
            _int32("tokens, adapters and features", T, *self._dims)
            s = AdapterShape(T, *self._dims, kind)
            n = self._lib.moe_adapter_workspace_size(s, backward)
            if n == 0:
                raise _lib.MoeError(_lib.MOE_ERR_INVALID_ARG, self._lib.moe_last_error().decode())
            if len(self._sizes) > 4096:
                self._sizes.clear()
            got = self._sizes[(T, kind, backward)] = (s, n)
        return got

    @staticmethod
    def _kind(dtype, name: str) -> int:
        if dtype is torch.bfloat16:
            return MOE_DTYPE_BF16
        if dtype is not torch.float32:
            _bad(f"{name} must be bfloat16 or float32, got {dtype}")
        return MOE_DTYPE_F32

    def forward(self, x, ids, base=None, out=None, out_dtype=None):
        """base + the adapters' products: [T, N] of base's dtype (without a
        base: of `out`'s, of out_dtype's, or bfloat16).

        x bf16 [T, H], ids int32 [T] (outside [0, NA): no adapter), base
        [T, N] bf16 or float32; rows may be strided.  `out` may be `base`
        itself, or x."""
        dev = _device()
        if dev != self._dev:
            _same_device(dev, self._dev)
        a, b, scale = self._addresses()
        T, H, N = _rows(x, "x"), self._H, self._N
        ld_x = _check_rows(x, "x", torch.bfloat16, (T, H), dev)
        _check_flat(ids, "ids", torch.int32, (T,), dev)
        dtype = base.dtype if base is not None else out.dtype if out is not None else (
            out_dtype or torch.bfloat16)
        kind, shape = self._kind(dtype, "base"), (T, N)
        ld_base = 0 if base is None else _check_rows(base, "base", dtype, shape, dev)
        if out is None:
            ld_out = N
            out = (torch.empty_like(base) if ld_base == ld_out else   # (quicker)
                   torch.empty(shape, dtype=dtype, device=self.device))
        else:
            ld_out = _check_rows(out, "out", dtype, shape, dev)
        s, n = self._call(T, kind, 0)
        ws = None if n <= 256 else _scratch(n, x)   # small batches use none
        rc = self._lib.moe_adapter_forward(
            s, x.data_ptr(), ld_x, ids.data_ptr(), a, b, scale, _ptr(base), ld_base, out.data_ptr(),
            ld_out, _ptr(ws), n, _raw_stream(dev))
        if rc:
            check(rc)
        return out

    __call__ = forward

    def backward(self, dout, x, ids, dx_base=None, dx=None, da=None, db=None,
                 need_dx: bool = True, need_weights: bool = True):
        """(dx, da, db) for dout [T, N] (bf16 or float32): dx bf16 [T, H] with
        dx_base (the shared projection's) added, da float32 [NA, r, H], db
        float32 [NA, N, r], zero for adapters without tokens.  What is not
        needed comes back as None.  `dx` may be `dx_base`, not x or dout."""
        dev = _device()
        if dev != self._dev:
            _same_device(dev, self._dev)
        a, b, scale = self._addresses()
        T, H, N = _rows(x, "x"), self._H, self._N
        if dout is None:
            _bad("dout is None")
        kind, wide = self._kind(dout.dtype, "dout"), (T, H)
        ld_dout = _check_rows(dout, "dout", dout.dtype, (T, N), dev)
        ld_x = _check_rows(x, "x", torch.bfloat16, wide, dev)
        _check_flat(ids, "ids", torch.int32, (T,), dev)
        ld_dx = ld_base = 0
        if not need_dx:
            dx = dx_base = None
        elif dx is None:
            dx, ld_dx = torch.empty(wide, dtype=torch.bfloat16, device=self.device), wide[1]
        else:
            ld_dx = _check_rows(dx, "dx", torch.bfloat16, wide, dev)
        if dx_base is not None:
            ld_base = _check_rows(dx_base, "dx_base", torch.bfloat16, wide, dev)
        if not need_weights:
            da = db = None
        else:
            da_shape, db_shape, _ = self._shapes
            if da is None:
                da = torch.empty(da_shape, dtype=torch.float32, device=self.device)
            else:
                _check_flat(da, "da", torch.float32, da_shape, dev)
            if db is None:
                db = torch.empty(db_shape, dtype=torch.float32, device=self.device)
            else:
                _check_flat(db, "db", torch.float32, db_shape, dev)
        s, n = self._call(T, kind, 1)
        ws = _scratch(n, x)
        rc = self._lib.moe_adapter_backward(
            s, dout.data_ptr(), ld_dout, x.data_ptr(), ld_x, ids.data_ptr(), a, b, scale,
            _ptr(dx_base), ld_base, _ptr(dx), ld_dx, _ptr(da), _ptr(db), ws.data_ptr(), n,
            _raw_stream(dev))
        if rc:
            check(rc)
        return dx, da, db


class BalanceLoss:
    """The router's load-balance loss over `num_experts` experts and top-k
    routing, per-expert counts and the gradient of the logits (the formulas:
    moe_balance_loss in include/moe.h).  The attributes are read at every call, so
    that coef may follow a schedule."""

    def __init__(self, num_experts: int, top_k: int, coef: float = 1.0):
        _bind_torch()
        self.num_experts, self.top_k, self.coef = num_experts, top_k, coef
        self._lib, self._calls = load(), {}
        _int32("num_experts and top_k", num_experts, top_k)
        self._size(BalanceShape(0, num_experts, top_k, 1, coef))   # rejects bad sizes here

    def _size(self, s: BalanceShape) -> int:
        n = self._lib.moe_balance_workspace_size(s)
        if n == 0:
            raise _lib.MoeError(_lib.MOE_ERR_INVALID_ARG, self._lib.moe_last_error().decode())
        return n

    def __call__(self, logits, ids, mask=None, seq_offsets=None, weights=None, dweights=None,
                 need_grad: bool = True):
        """(loss float32 [1], counts int32 [S, E], dlogits float32 [T, E] or
        None).

        logits float32 [T, E], ids int32 [T, k], mask bool or uint8 [T] (zero:
        padding), seq_offsets int32 [S + 1] (None: the whole batch as one
        sequence), weights and dweights float32 [T, k] (both or neither: adds
        the gradient of the routing weights; dweights, dL/dw of the layer's
        combine, is the caller's to bring: FusedMoE has no backward).  Nothing is
        recorded for autograd: the gradient is dlogits."""
        dev, E, k, coef = _device(), self.num_experts, self.top_k, float(self.coef)
        T = _rows(logits, "logits")
        _check_flat(logits, "logits", torch.float32, (T, E), dev)
        _check_flat(ids, "ids", torch.int32, (T, k), dev)
        if mask is not None:
            if mask.dtype not in (torch.bool, torch.uint8):
                _bad(f"mask must be bool or uint8, got {mask.dtype}")
            _check_flat(mask, "mask", mask.dtype, (T,), dev)
        S = 1
        if seq_offsets is not None:
            if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2:
                _bad("seq_offsets must be [sequences + 1]")
            S = seq_offsets.shape[0] - 1
            _check_flat(seq_offsets, "seq_offsets", torch.int32, (S + 1,), dev)
        if (weights is None) != (dweights is None):
            _bad("weights and dweights go together")
        if weights is not None:
            _check_flat(weights, "weights", torch.float32, (T, k), dev)
            _check_flat(dweights, "dweights", torch.float32, (T, k), dev)
        key = (T, E, k, S, coef)   # all that the shape holds
        got = self._calls.get(key)
        if got is None:
            _int32("tokens, experts, top_k and sequences", *key[:4])
            s = BalanceShape(*key)
            if len(self._calls) > 4096:
                self._calls.clear()
            got = self._calls[key] = (s, self._size(s))
        s, n = got
        ws = None if n <= 256 else _scratch(n, logits)   # small batches use none
        loss = torch.empty(1, dtype=torch.float32, device=logits.device)
        counts = torch.empty((S, E), dtype=torch.int32, device=logits.device)
        dlogits = torch.empty_like(logits) if need_grad else None
        rc = self._lib.moe_balance_loss(s, logits.data_ptr(), ids.data_ptr(), _ptr(mask),
                                        _ptr(seq_offsets), _ptr(weights), _ptr(dweights),
                                        loss.data_ptr(), counts.data_ptr(), _ptr(dlogits),
                                        _ptr(ws), n, _raw_stream(dev))
        if rc:
            check(rc)
        return loss, counts, dlogits


class AdamW:
    """AdamW over a list of tensors, one launch a step (400 tensors a launch).

    params: contiguous float32 CUDA tensors, updated in place; grads: tensors
    of the same sizes, all float32 or all bfloat16; copies: bfloat16 tensors
    that receive the rounded parameters, or None.  state_bits 32 keeps float32
    moments; 8 keeps E4M3 codes in blocks of 256 with a float32 scale each
    (v holds the codes of the second moment's root).  `state`: {"m": [...],
    "v": [...]} and, with 8 bits, "m_scale" and "v_scale", to resume from; by
    default it starts at zero.  The tensors are bound and held here (params,
    grads, copies and state name them and cannot be assigned): after replacing
    a parameter's or a gradient's memory, build a new AdamW (state=old.state)
    or pass the new gradients to step().

    The step number and lr, betas, eps and weight_decay are the host's: they go
    into the launch.  A step captured into a CUDA graph keeps the capture's at
    every replay, so that the graph is good for that step number only (a
    training loop captures forward and backward and calls step() after the
    replay).  Under a capture step() therefore wants its number named, and
    steps_done is left as it is: nothing has run yet."""

    def __init__(self, params, grads, copies=None, state_bits: int = 32, state=None,
                 lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, steps_done: int = 0):
        _bind_torch()
        if state_bits not in (8, 32):
            _bad(f"state_bits must be 8 or 32, got {state_bits}")
        dev = self._dev = _device()
        # detached: keeps the bound memory alive whatever becomes of the originals
        bound = self._params = tuple(_detached(params, "params"))
        self.state_bits, self.lr, self.betas, self.eps = state_bits, lr, betas, eps
        self.weight_decay, self.steps_done = weight_decay, steps_done
        sizes = [p.numel() for p in bound]
        blocks = [-(-n // MOE_ADAMW_BLOCK) for n in sizes]
        if state is None:
            kind = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
            state = {k: [torch.zeros(n, dtype=torch.uint8 if state_bits == 8 else kind,
                                     device=p.device).view(kind)
                         for n, p in zip(sizes, bound)] for k in ("m", "v")}
            if state_bits == 8:
                state |= {k: [torch.ones(n, device=p.device) for n, p in zip(blocks, bound)]
                          for k in ("m_scale", "v_scale")}
        keys = ("m", "v") if state_bits == 32 else ("m", "v", "m_scale", "v_scale")
        self._state = {}
        self._table = (AdamwTensor * max(1, len(sizes)))()
        f32 = torch.float32
        for e, p, n, i in zip(self._table, bound, sizes, range(len(sizes))):
            e.param, e.n = _check_numel(p, "params", i, f32, n, dev), n
        if len({p.data_ptr() for p in bound if p.numel()}) < sum(n > 0 for n in sizes):
            _bad("params must be distinct")   # updated in place, side by side
        for key in keys:
            held = self._state[key] = tuple(_detached(state.get(key) or (), f"state[{key!r}]"))
            if len(held) != len(sizes):
                _bad(f"state[{key!r}] must hold {len(sizes)} tensors")
            scales = key.endswith("scale")
            kind = f32 if scales or state_bits == 32 else None   # None: one byte each
            for e, t, n, i in zip(self._table, held, blocks if scales else sizes, range(len(held))):
                setattr(e, key, _check_numel(t, f"state[{key!r}]", i, kind, n, dev))
        self._copies = None if copies is None else tuple(_detached(copies, "copies"))
        if self._copies is not None:
            if len(self._copies) != len(sizes):
                _bad(f"copies must hold {len(sizes)} tensors")
            for e, t, n, i in zip(self._table, self._copies, sizes, range(len(sizes))):
                e.param_bf16 = _check_numel(t, "copies", i, torch.bfloat16, n, dev)
        self._options = AdamwOptions(state_bits=state_bits)
        self.bind_grads(grads)

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
    def state(self) -> dict:
        return dict(self._state)

    def bind_grads(self, grads) -> None:
        """Take the next steps' gradients from these tensors."""
        grads = tuple(_detached(grads, "grads"))
        if len(grads) != len(self._params):
            _bad(f"grads must hold {len(self._params)} tensors")
        kind = grads[0].dtype if grads else torch.float32
        if kind not in (torch.float32, torch.bfloat16):
            _bad(f"grads must be float32 or bfloat16, got {kind}")
        dev = _device()
        _same_device(dev, self._dev)
        at = [_check_numel(t, "grads", i, kind, p.numel(), dev)
              for i, (t, p) in enumerate(zip(grads, self._params))]
        self._grads = grads
        for e, address in zip(self._table, at):
            e.grad = address
        self._options.grad_dtype = MOE_DTYPE_F32 if kind == torch.float32 else MOE_DTYPE_BF16

    def step(self, grads=None, step: int | None = None, grad_scale=None) -> None:
        """One step, in place.  `step` (from 1) overrides the count kept here;
        grad_scale: float32 CUDA scalar every gradient is multiplied by.
        (Tensors given here are checked one by one: 1.5 us of host time each.
        A backward that writes into the bound gradients costs none of it.)"""
        captured = _capturing()
        if captured and step is None:
            _bad("a captured step keeps its number at every replay: name it (step=...), or "
                 "call step() outside the graph")
        if grads is not None:
            self.bind_grads(grads)
        t = self.steps_done + 1 if step is None else step
        _int32("step", t)
        dev, o = _device(), self._options
        _same_device(dev, self._dev)
        if grad_scale is not None:
            _check_tensor(grad_scale, "grad_scale", cuda=True, dtype=torch.float32, numel=1,
                          device=dev)
        o.grad_scale = None if grad_scale is None else grad_scale.data_ptr()
        o.lr, (o.beta1, o.beta2), o.eps = self.lr, self.betas, self.eps
        o.weight_decay, o.step = self.weight_decay, t
        check(load().moe_adamw_step(self._table, len(self._params), o, _raw_stream(dev)))
        if not captured:
            self.steps_done = t
