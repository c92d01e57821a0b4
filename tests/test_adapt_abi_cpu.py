"""The adapters', balance loss's and optimiser's entry points without a GPU:
sizes, limits and refusals of the C ABI, which come before any CUDA call, and
the Python binding's checks."""
import ctypes
import os

import pytest
import torch

import precision_moe_grouped_gb300 as P
from precision_moe_grouped_gb300 import _lib as L


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from precision_moe_grouped_gb300 import build
        try:
            build.build()
        except (RuntimeError, FileNotFoundError) as e:  # no nvcc on this machine
            pytest.skip(f"cannot build libmoe.so here: {e}")
    return P.load()


def ashape(T=64, NA=4, r=16, H=256, N=128, kind=L.MOE_DTYPE_BF16):
    return L.AdapterShape(T, NA, r, H, N, kind)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), L.MOE_ERR_INVALID_ARG), (dict(T=(1 << 30) + 1), L.MOE_ERR_UNSUPPORTED),
    (dict(NA=0), L.MOE_ERR_INVALID_ARG),
    (dict(NA=1025), L.MOE_ERR_INVALID_ARG), (dict(r=0), L.MOE_ERR_INVALID_ARG),
    (dict(r=136), L.MOE_ERR_INVALID_ARG), (dict(r=12), L.MOE_ERR_MISALIGNED),
    (dict(H=0), L.MOE_ERR_INVALID_ARG), (dict(H=100), L.MOE_ERR_MISALIGNED),
    (dict(N=36), L.MOE_ERR_MISALIGNED), (dict(N=(1 << 20) + 8), L.MOE_ERR_UNSUPPORTED),
    (dict(kind=2), L.MOE_ERR_INVALID_ARG)])
def test_adapter_shapes(lib, bad, code):
    s = ashape(**bad)
    assert lib.moe_adapter_workspace_size(s, 0) == 0 and lib.moe_last_error()
    p = 0x100000
    args = [s, p, 1 << 10, p, p, p, None, None, 0, p, 1 << 10, p, 1 << 30, None]
    assert lib.moe_adapter_forward(*args) == code


def test_adapter_workspace(lib):
    assert lib.moe_adapter_workspace_size(ashape(), 0) == 256          # unused
    assert lib.moe_adapter_workspace_size(ashape(T=1024), 0) == 256
    assert lib.moe_adapter_workspace_size(ashape(T=1025), 0) > 256
    assert lib.moe_adapter_workspace_size(ashape(T=65, r=72), 0) > 256
    big = lib.moe_adapter_workspace_size(ashape(T=5000), 0)
    assert big > 5000 * 16 * 2 * 3 and big % 256 == 0
    assert lib.moe_adapter_workspace_size(ashape(T=5000), 1) > big
    assert lib.moe_adapter_workspace_size(ashape(T=1), 1) > 0


def forward(lib, s, x=0x100000, ld_x=256, ids=0x200000, a=0x300000, b=0x400000, scale=None,
            base=0x500000, ld_base=128, out=0x600000, ld_out=128, ws=0x700000, n=1 << 30):
    return lib.moe_adapter_forward(s, x, ld_x, ids, a, b, scale, base, ld_base, out, ld_out, ws, n, None)


def backward(lib, s, dout=0x100000, ld_dout=128, x=0x200000, ld_x=256, ids=0x300000, a=0x400000,
             b=0x500000, base=None, ld_base=0, dx=0x600000, ld_dx=256, da=0x700000, db=0x800000,
             ws=0x900000, n=1 << 30):
    return lib.moe_adapter_backward(s, dout, ld_dout, x, ld_x, ids, a, b, None, base, ld_base, dx,
                                    ld_dx, da, db, ws, n, None)


def test_adapter_refusals(lib):
    s = ashape(T=5000)
    for k in ("x", "ids", "a", "b", "out", "ws"):
        assert forward(lib, s, **{k: None}) == L.MOE_ERR_INVALID_ARG, k
    for k in ("x", "a", "b", "out", "base"):
        assert forward(lib, s, **{k: 0x100008}) == L.MOE_ERR_MISALIGNED, k
    assert forward(lib, s, ids=0x100002) == L.MOE_ERR_MISALIGNED
    assert forward(lib, s, scale=0x100002) == L.MOE_ERR_MISALIGNED
    assert forward(lib, s, ws=0x100010) == L.MOE_ERR_MISALIGNED
    for k in ("ld_x", "ld_base", "ld_out"):
        assert forward(lib, s, **{k: 64}) == L.MOE_ERR_INVALID_ARG, k      # below the row
        assert forward(lib, s, **{k: 1004}) == L.MOE_ERR_MISALIGNED, k
        assert forward(lib, s, **{k: (1 << 31) + 8}) == L.MOE_ERR_INVALID_ARG, k
    need = lib.moe_adapter_workspace_size(s, 0)
    assert forward(lib, s, n=need - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL
    assert forward(lib, ashape(T=0), x=None, ids=None, a=None, b=None, out=None, ws=None) == L.MOE_OK
    assert backward(lib, s, da=None) == L.MOE_ERR_INVALID_ARG              # one of the pair
    assert backward(lib, s, dout=None) == L.MOE_ERR_INVALID_ARG
    assert backward(lib, s, dx=0x200000) == L.MOE_ERR_INVALID_ARG          # x itself
    assert backward(lib, s, dx=0x100000) == L.MOE_ERR_INVALID_ARG          # dout itself
    assert backward(lib, s, da=0x700004) == L.MOE_ERR_MISALIGNED
    assert backward(lib, s, base=0x600000, ld_base=100) == L.MOE_ERR_INVALID_ARG
    assert backward(lib, s, n=lib.moe_adapter_workspace_size(s, 1) - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL
    assert backward(lib, ashape(T=0), da=None, db=None) == L.MOE_OK


def balance(lib, s, z=0x100000, ids=0x200000, mask=None, seq=None, w=None, dw=None, loss=0x300000,
            counts=0x400000, dz=0x500000, ws=0x600000, n=1 << 30):
    return lib.moe_balance_loss(s, z, ids, mask, seq, w, dw, loss, counts, dz, ws, n, None)


def test_balance_refusals(lib):
    good = dict(num_tokens=5000, num_experts=16, top_k=2, num_sequences=1, coef=1.0)
    for bad in (dict(num_tokens=-1), dict(num_experts=0), dict(num_experts=1025), dict(top_k=0),
                dict(top_k=17), dict(num_sequences=0), dict(coef=float("inf")),
                dict(num_tokens=(1 << 30), top_k=2)):
        s = L.BalanceShape(**(good | bad))
        assert lib.moe_balance_workspace_size(s) == 0, bad
        assert balance(lib, s) == L.MOE_ERR_INVALID_ARG, bad
    s = L.BalanceShape(**good)
    for k in ("z", "ids", "loss", "counts", "ws"):
        assert balance(lib, s, **{k: None}) == L.MOE_ERR_INVALID_ARG, k
    for k in ("z", "ids", "loss", "counts", "dz", "seq"):
        assert balance(lib, s, **{k: 0x100002}) == L.MOE_ERR_MISALIGNED, k
    assert balance(lib, s, w=0x100000) == L.MOE_ERR_INVALID_ARG
    assert balance(lib, s, ws=0x100010) == L.MOE_ERR_MISALIGNED
    assert balance(lib, s, n=lib.moe_balance_workspace_size(s) - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL
    assert lib.moe_balance_workspace_size(L.BalanceShape(**(good | dict(num_tokens=100)))) == 256
    many = L.BalanceShape(**(good | dict(num_sequences=3)))
    assert balance(lib, many) == L.MOE_ERR_INVALID_ARG                     # no offsets


def adamw(lib, count=1, null=False, **kw):
    o = L.AdamwOptions(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1,
                       state_bits=32, grad_dtype=L.MOE_DTYPE_F32)
    t = (L.AdamwTensor * max(1, count))()
    for e in t:
        e.param, e.grad, e.m, e.v, e.n = 0x100000, 0x200000, 0x300000, 0x400000, 10
    for k, v in kw.items():
        if hasattr(o, k):
            setattr(o, k, v)
        else:
            setattr(t[0], k, v)
    return lib.moe_adamw_step(None if null else t, count, o, None)


def test_adamw_refusals(lib):
    for bad in (dict(step=0), dict(state_bits=16), dict(grad_dtype=7), dict(beta1=1.0), dict(beta2=-0.1),
                dict(lr=float("nan")), dict(eps=-1.0), dict(weight_decay=float("inf")), dict(n=-1),
                dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(state_bits=8),
                dict(count=-1), dict(null=True)):
        assert adamw(lib, **bad) == L.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(param=0x100002), dict(grad=0x100002), dict(m=0x100001), dict(v=0x100002),
                dict(param_bf16=0x100001), dict(grad_scale=0x100002)):
        assert adamw(lib, **bad) == L.MOE_ERR_MISALIGNED, bad
    assert adamw(lib, count=0, null=True) == L.MOE_OK
    assert adamw(lib, n=0, param=None) == L.MOE_OK                         # nothing to do
    o = L.AdamwOptions(step=1, state_bits=32)
    o.reserved[1] = 1
    assert lib.moe_adamw_step(None, 0, o, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_adamw_step(None, 0, None, None) == L.MOE_ERR_INVALID_ARG


def test_no_device_gives_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these pointers must not reach it")
    assert forward(lib, ashape(T=5000)) == L.MOE_ERR_CUDA
    assert forward(lib, ashape()) == L.MOE_ERR_CUDA
    assert backward(lib, ashape(T=500)) == L.MOE_ERR_CUDA
    assert balance(lib, L.BalanceShape(100, 16, 2, 1, 1.0)) == L.MOE_ERR_CUDA
    assert adamw(lib) == L.MOE_ERR_CUDA


def test_binding_refuses_host_tensors(lib):
    a, b = torch.zeros(2, 8, 16, dtype=torch.bfloat16), torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    with pytest.raises(P.MoeError, match="CUDA"):
        P.LowRankAdapters(a, b)
    with pytest.raises(P.MoeError):
        P.BalanceLoss(8, 2)(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(P.MoeError, match="CUDA"):
        P.AdamW([torch.zeros(4)], [torch.zeros(4)])
    with pytest.raises(P.MoeError):
        P.BalanceLoss(8, 9)


def test_binding_refuses_what_is_no_tensor(lib):
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for z in (None, 3.0, torch.zeros(())):
        with pytest.raises(P.MoeError, match="logits"):
            P.BalanceLoss(8, 2)(z, ids)
    for params, grads in ((None, []), ([None], []), ([], None)):
        with pytest.raises(P.MoeError, match="list of tensors"):
            P.AdamW(params, grads)


def test_structs_match_the_header(tmp_path):
    """The binding's structures have the sizes and offsets C gives them."""
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = {"moe_adapter_shape": L.AdapterShape, "moe_balance_shape": L.BalanceShape,
             "moe_adamw_tensor": L.AdamwTensor, "moe_adamw_options": L.AdamwOptions}
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe.h"', "int main(void) {"]
    want = []
    for c, s in names.items():
        src.append(f'printf("%lu\\n", (unsigned long)sizeof({c}));')
        want.append(ctypes.sizeof(s))
        for f, _ in s._fields_:
            src.append(f'printf("%lu\\n", (unsigned long)offsetof({c}, {f}));')
            want.append(getattr(s, f).offset)
    src.append("return 0; }")
    (tmp_path / "s.c").write_text("\n".join(src))
    subprocess.run([cc, "-std=c99", "-I", os.path.join(root, "include"), str(tmp_path / "s.c"), "-o",
                    str(tmp_path / "s")], check=True)
    out = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == want
