"""The gated feed-forward block's and the orthogonalised step's entry points
without a GPU: sizes, limits and refusals of the C ABI, which come before any
CUDA call, the C structures' layout, and where their kernels read their inputs."""
import ctypes
import os
import re
import subprocess

import pytest

import precision_moe_grouped_gb300 as P
from precision_moe_grouped_gb300 import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "precision_moe_grouped_gb300", "csrc")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from precision_moe_grouped_gb300 import build
        try:
            build.build()
        except (RuntimeError, FileNotFoundError) as e:  # no nvcc on this machine
            pytest.skip(f"cannot build libmoe.so here: {e}")
    return P.load()


# ------------------------------------------------------- feed-forward block
@pytest.mark.parametrize("T,H,I,code", [
    (-1, 64, 64, L.MOE_ERR_INVALID_ARG), (4, 0, 64, L.MOE_ERR_INVALID_ARG), (4, 64, 0, L.MOE_ERR_INVALID_ARG),
    (4, -8, 64, L.MOE_ERR_INVALID_ARG), (4, 60, 64, L.MOE_ERR_MISALIGNED), (4, 64, 12, L.MOE_ERR_MISALIGNED),
    ((1 << 24) + 1, 64, 64, L.MOE_ERR_UNSUPPORTED), (4, (1 << 17) + 8, 64, L.MOE_ERR_UNSUPPORTED),
    (4, 64, (1 << 17) + 8, L.MOE_ERR_UNSUPPORTED)])
def test_ffn_shapes(lib, T, H, I, code):
    s = L.FfnShape(T, H, I)
    for backward in (0, 1):
        assert lib.moe_ffn_workspace_size(s, backward) == 0 and lib.moe_last_error()
    p = 0x100000
    assert lib.moe_ffn_forward(s, p, 1 << 20, p, p, None, 0, p, 1 << 20, p, 1 << 40, p, None) == code
    assert lib.moe_ffn_backward(s, p, 1 << 20, p, 1 << 20, p, p, None, 0, p, 1 << 20, p, p, p, 1 << 40, p,
                                None) == code
    assert lib.moe_ffn_forward(None, p, 64, p, p, None, 0, p, 64, p, 1 << 40, p, None) == L.MOE_ERR_INVALID_ARG


def test_ffn_workspace(lib):
    size = lambda T, b, H=2048, I=1024: lib.moe_ffn_workspace_size(L.FfnShape(T, H, I), b)   # noqa: E731
    for b in (0, 1):
        for T in (0, 1, 32, 33, 256, 257, 5000, 1 << 24):
            assert size(T, b) % 256 == 0 and size(T, b) >= max(256, 2 * T * 1024)
    assert size(1, 0) == 2048                                         # h alone
    assert size(5000, 1) >= 5000 * 1024 * (2 + 4 + 4)                 # h, dg and du, dh in float
    assert size(1 << 24, 1, 1 << 17, 1 << 17) >= (1 << 41) * 10       # in 64 bits


def forward(lib, s, x=0x100000, ld_x=64, wgu=0x200000, wd=0x300000, base=None, ld_base=64, out=0x400000, ld_out=64,
            ws=0x500000, n=1 << 40, status=0x600000):
    return lib.moe_ffn_forward(s, x, ld_x, wgu, wd, base, ld_base, out, ld_out, ws, n, status, None)


def backward(lib, s, dout=0x100000, ld_dout=64, x=0x200000, ld_x=64, wgu=0x300000, wd=0x400000, base=None, ld_base=64,
             dx=0x500000, ld_dx=64, dwgu=0x600000, dwd=0x700000, ws=0x800000, n=1 << 40, status=0x900000):
    return lib.moe_ffn_backward(s, dout, ld_dout, x, ld_x, wgu, wd, base, ld_base, dx, ld_dx, dwgu, dwd, ws, n,
                                status, None)


def test_ffn_tokens_of_weights_gradients(lib):
    """Sums over the tokens are refused beyond their limit, dx alone is not."""
    for T, code in ((1 << 16, L.MOE_ERR_WORKSPACE_TOO_SMALL), ((1 << 16) + 1, L.MOE_ERR_UNSUPPORTED)):
        assert backward(lib, L.FfnShape(T, 64, 32), n=0) == code
        assert backward(lib, L.FfnShape(T, 64, 32), n=0, dwgu=None, dwd=None) == L.MOE_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("T", [3, 100, 1000])
def test_ffn_refusals(lib, T):
    s = L.FfnShape(T, 64, 32)
    for k in ("x", "wgu", "wd", "out", "ws", "status"):
        assert forward(lib, s, **{k: None}) == L.MOE_ERR_INVALID_ARG, k
    for k in ("x", "wgu", "wd", "out", "base", "ws"):
        assert forward(lib, s, **{k: 0x100008}) == L.MOE_ERR_MISALIGNED, k
    assert forward(lib, s, status=0x600002) == L.MOE_ERR_MISALIGNED
    assert forward(lib, s, ws=0x500010) == L.MOE_ERR_MISALIGNED
    for k in ("ld_x", "ld_out"):
        assert forward(lib, s, **{k: 56}) == L.MOE_ERR_INVALID_ARG, k          # below the row
        assert forward(lib, s, **{k: 1 << 31}) == L.MOE_ERR_INVALID_ARG, k
        assert forward(lib, s, **{k: 68}) == L.MOE_ERR_MISALIGNED, k
    assert forward(lib, s, base=0x700000, ld_base=56) == L.MOE_ERR_INVALID_ARG
    need = lib.moe_ffn_workspace_size(s, 0)
    assert forward(lib, s, n=need - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL
    for k in ("x", "dout", "wgu", "wd", "ws", "status"):
        assert backward(lib, s, **{k: None}) == L.MOE_ERR_INVALID_ARG, k
    for k in ("x", "dout", "dx", "wgu", "wd", "base", "dwgu", "dwd"):
        assert backward(lib, s, **{k: 0x100008}) == L.MOE_ERR_MISALIGNED, k
    for k in ("dwgu", "dwd"):
        assert backward(lib, s, **{k: None}) == L.MOE_ERR_INVALID_ARG, k        # one of the pair
    assert backward(lib, s, dx=0x100000) == L.MOE_ERR_INVALID_ARG               # dout itself
    assert backward(lib, s, dx=0x200000) == L.MOE_ERR_INVALID_ARG               # x itself
    assert backward(lib, s, ld_dx=56) == L.MOE_ERR_INVALID_ARG
    assert backward(lib, s, base=0x500000, ld_base=36) == L.MOE_ERR_INVALID_ARG
    assert backward(lib, s, n=lib.moe_ffn_workspace_size(s, 1) - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL
    assert backward(lib, s, dx=None, dwgu=None, dwd=None) == L.MOE_OK           # nothing to compute


def test_ffn_without_tokens(lib):
    s = L.FfnShape(0, 64, 32)
    assert forward(lib, s, x=None, wgu=None, wd=None, out=None, ws=None, n=0, status=None) == L.MOE_OK
    assert backward(lib, s, dout=None, x=None, dwgu=None, dwd=None, ws=None, n=0, status=None) == L.MOE_OK


# ------------------------------------------------------ orthogonalised step
NS = (3.4445, -4.7750, 2.0315)


def options(**kw):
    o = L.MuonOptions()
    o.lr, o.momentum, o.weight_decay, o.eps, o.ns_steps, o.nesterov = 1e-3, 0.95, 0.1, 1e-7, 5, 1
    o.coefficients[:] = kw.pop("coefficients", NS)
    o.grad_dtype = L.MOE_DTYPE_F32
    for k, v in kw.items():
        if k == "reserved":
            o.reserved[v] = 1
        else:
            setattr(o, k, v)
    return o


def tensor(param=0x100000, grad=0x200000, momentum=0x300000, copy=None, count=1, rows=100, cols=80, reserved=0):
    return L.MuonTensor(param, grad, momentum, copy, count, rows, cols, reserved)


def step(lib, t, o, ws=0x400000, n=1 << 50, status=0x500000):
    table = (L.MuonTensor * len(t))(*t)
    return lib.moe_muon_step(table, len(t), o, ws, n, status, None), lib.moe_muon_workspace_size(table, len(t), o)


@pytest.mark.parametrize("bad,code", [
    (dict(lr=float("nan")), L.MOE_ERR_INVALID_ARG), (dict(weight_decay=float("inf")), L.MOE_ERR_INVALID_ARG),
    (dict(momentum=1.0), L.MOE_ERR_INVALID_ARG), (dict(momentum=-0.1), L.MOE_ERR_INVALID_ARG),
    (dict(eps=0.0), L.MOE_ERR_INVALID_ARG), (dict(eps=0.9e-16), L.MOE_ERR_INVALID_ARG),
    (dict(ns_steps=0), L.MOE_ERR_INVALID_ARG), (dict(ns_steps=13), L.MOE_ERR_INVALID_ARG),
    (dict(grad_dtype=2), L.MOE_ERR_INVALID_ARG), (dict(update_scale=2), L.MOE_ERR_INVALID_ARG),
    (dict(reserved=0), L.MOE_ERR_INVALID_ARG), (dict(reserved=1), L.MOE_ERR_INVALID_ARG),
    (dict(grad_scale=0x100002), L.MOE_ERR_MISALIGNED),
    (dict(coefficients=(1.5, -0.5, 0.0)), L.MOE_ERR_UNSUPPORTED),                # c = 0
    (dict(coefficients=(1.5, 0.0, 0.0)), L.MOE_ERR_UNSUPPORTED),
    (dict(coefficients=(1.5, -0.65, 0.01)), L.MOE_ERR_UNSUPPORTED),              # |b| > 64 |c|
    (dict(coefficients=(30.0, -1.0, 1.0)), L.MOE_ERR_UNSUPPORTED),               # grows without bound
    (dict(coefficients=(float("nan"), -1.0, 1.0)), L.MOE_ERR_UNSUPPORTED),
    (dict(coefficients=(3.0, float("nan"), 1.0)), L.MOE_ERR_UNSUPPORTED)])
def test_muon_options(lib, bad, code):
    assert step(lib, [tensor()], options(**bad)) == (code, 0)
    assert lib.moe_last_error()


@pytest.mark.parametrize("bad,code", [
    (dict(count=-1), L.MOE_ERR_INVALID_ARG), (dict(rows=-1), L.MOE_ERR_INVALID_ARG),
    (dict(cols=-1), L.MOE_ERR_INVALID_ARG), (dict(reserved=1), L.MOE_ERR_INVALID_ARG),
    (dict(param=None), L.MOE_ERR_INVALID_ARG), (dict(grad=None), L.MOE_ERR_INVALID_ARG),
    (dict(momentum=None), L.MOE_ERR_INVALID_ARG), (dict(param=0x100002), L.MOE_ERR_MISALIGNED),
    (dict(grad=0x100001), L.MOE_ERR_MISALIGNED), (dict(momentum=0x100002), L.MOE_ERR_MISALIGNED),
    (dict(copy=0x100001), L.MOE_ERR_MISALIGNED), (dict(rows=(1 << 20) + 1), L.MOE_ERR_UNSUPPORTED),
    (dict(cols=(1 << 20) + 1), L.MOE_ERR_UNSUPPORTED), (dict(rows=32769, cols=32769), L.MOE_ERR_UNSUPPORTED),
    (dict(count=(1 << 31) - 1, rows=300, cols=300), L.MOE_ERR_UNSUPPORTED)])
def test_muon_tensors(lib, bad, code):
    assert step(lib, [tensor(rows=20, cols=20), tensor(**bad)], options()) == (code, 0)
    assert lib.moe_last_error()


def test_muon_refusals(lib):
    for shape in (dict(rows=16, cols=700), dict(rows=333, cols=100)):
        t = [tensor(**shape)]
        o = options()
        rc, need = step(lib, t, o, ws=None)
        assert rc == L.MOE_ERR_INVALID_ARG and need >= 256 and need % 256 == 0
        assert step(lib, t, o, ws=0x400010)[0] == L.MOE_ERR_MISALIGNED
        assert step(lib, t, o, n=need - 1)[0] == L.MOE_ERR_WORKSPACE_TOO_SMALL
        assert step(lib, t, o, status=None)[0] == L.MOE_ERR_INVALID_ARG
        assert step(lib, t, o, status=0x500001)[0] == L.MOE_ERR_MISALIGNED
    o = options()
    assert lib.moe_muon_step(None, 1, o, None, 0, None, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_muon_step(None, -1, o, None, 0, None, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_muon_step(None, 0, None, None, 0, None, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_muon_step(None, 0, o, None, 0, None, None) == L.MOE_OK
    for empty in (dict(count=0), dict(rows=0), dict(cols=0)):
        assert step(lib, [tensor(**empty, param=None, grad=None, momentum=None)], o, ws=None, n=0,
                    status=None)[0] == L.MOE_OK


def test_muon_workspace_is_shared(lib):
    """Matrices of one shape add up, other shapes in turn reuse the memory (up to 256 MB is shared at once)."""
    o = options()
    size = lambda *t: step(lib, list(t), o, ws=None)[1]                          # noqa: E731
    one, two = size(tensor(rows=2048, cols=7168)), size(tensor(rows=2048, cols=7168, count=2))
    assert 1.9 * one < two < 2.1 * one and one >= 8 * 2048 * 7168
    assert size(tensor(rows=2048, cols=7168), tensor(rows=7168, cols=2048)) == two     # turned, the same shape
    assert size(tensor(rows=2048, cols=7168), tensor(rows=1024, cols=7168)) == one
    assert size(tensor(count=5, rows=8, cols=1 << 20)) < 1 << 27


@pytest.mark.parametrize("count", [300, 304, 400, 3000])
def test_muon_long_matrix_among_many(lib, count):
    """A matrix of 2^20 columns is shared out to blocks by its length, however many matrices there are besides: each
    block's sum of u u^T has a place in the workspace, beside a matrix's Q."""
    o, place = options(), 4 * 64 * 64
    size = lambda *t: step(lib, list(t), o, ws=None)[1]                          # noqa: E731
    tiles = count * 112 + 16384                                                  # of 64 columns
    blocks = count + 16384 * 304 // tiles // 2                                   # half of its fair share at least
    assert size(tensor(rows=64, cols=7168, count=count), tensor(rows=64, cols=1 << 20)) >= place * (blocks + count + 1)


def test_muon_resident_matrices_take_no_workspace(lib):
    """What stays in a cluster's shared memory has no sums in the workspace, whatever it stands beside."""
    o = options()
    size = lambda *t: step(lib, list(t), o, ws=None)[1]                          # noqa: E731
    pools = [tensor(count=1 << 22, rows=1, cols=1), tensor(count=48, rows=16, cols=7168), tensor(count=48, rows=4096, cols=16),
             tensor(count=500, rows=64, cols=4096), tensor(rows=8, cols=20000), tensor(count=70, rows=300, cols=33)]
    for t in pools:
        assert size(t) == 256
    # ... but for few matrices that go with a longer one of their size
    long = tensor(rows=8, cols=70000), tensor(rows=20, cols=40000)
    assert size(*pools, *long) == size(*long) > 256
    assert size(long[1], tensor(count=600, rows=300, cols=17)) == size(long[1])
    assert size(long[0], tensor(count=9, rows=300, cols=16)) > size(long[0])


GIB = 1 << 30


@pytest.mark.parametrize("rows,cols", [(2048, 7168), (7168, 2048), (100, 1000), (65, 65), (512, 512), (384, 1 << 17)])
def test_muon_workspace_does_not_grow_with_the_matrices(lib, rows, cols):
    """Matrices of one shape run in slices of up to 4 GiB of workspace (one matrix at least), but for the shares of
    few long sums (up to 38 of 256 x 256 floats a tile of the Gram matrix: 13 MB)."""
    o = options()
    size = lambda *t: step(lib, list(t), o, ws=None)[1]                          # noqa: E731
    one = size(tensor(rows=rows, cols=cols))
    sizes = [size(tensor(rows=rows, cols=cols, count=n)) for n in (2, 5, 30, 1000, 20000)]
    assert all(0 < n <= max(one, 4 * GIB) + (16 << 20) for n in sizes)
    assert max(sizes) > 2 * GIB
    # several tensors of the shape, turned or not, are one group
    assert size(*(tensor(rows=rows, cols=cols, count=400), tensor(rows=cols, cols=rows, count=600))) == sizes[3]


def test_muon_workspace_of_a_model(lib):
    """Shared experts of 61 layers, and the matrices of 256 experts."""
    o = options()
    layers = [tensor(rows=2048, cols=7168, count=2), tensor(rows=7168, cols=2048)] * 61
    experts = [tensor(rows=2048, cols=7168, count=512), tensor(rows=7168, cols=2048, count=256)]
    for t in (layers, experts):
        assert 0 < step(lib, t, o, ws=None)[1] <= 4 * GIB + (16 << 20)


def test_structures_match_the_header():
    """Sizes and offsets of the C structures, as a C compiler lays them out."""
    fields = {"moe_ffn_shape": L.FfnShape, "moe_muon_tensor": L.MuonTensor, "moe_muon_options": L.MuonOptions}
    lines = []
    for name, c in fields.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in c._fields_]
    src = ('#include <stddef.h>\n#include <stdio.h>\n#include "moe.h"\nint main(void) {\n' + "\n".join(lines) +
           "\nreturn 0; }\n")
    import tempfile
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "a")
        subprocess.run(["gcc", "-x", "c", "-", "-I", os.path.join(ROOT, "include"), "-o", exe], input=src, text=True,
                       check=True)
        said = dict(line.split() for line in subprocess.run([exe], capture_output=True, text=True,
                                                            check=True).stdout.splitlines())
    for name, c in fields.items():
        assert int(said[name]) == ctypes.sizeof(c)
        for f in c._fields_:
            assert int(said[f"{name}.{f[0]}"]) == getattr(c, f[0]).offset, (name, f[0])


# ------------------------------------------------ inputs behind the grid wait
def body(source, name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, source)).read())
    at = re.search(r"__global__[^;{]*\b%s\(" % name, text).end()
    at = text.index("{", at)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError("unbalanced")


@pytest.mark.parametrize("source,name,inputs", [
    ("muon.cu", "muon_momentum_kernel", ("a.m +", "grad_scale", "grad_at")),
    ("muon_small.cu", "muon_small_gram_kernel", ("f.fetch", "grad_scale")),
    ("muon_small.cu", "muon_cluster_kernel", ("f.fetch", "grad_scale", "pp["))])
def test_first_kernels_read_behind_the_wait(source, name, inputs):
    """What a call's first kernel reads may be written by the kernel before it on the stream."""
    text = body(source, name)
    ahead = text[:text.index("griddep_wait()")]
    assert text.count("griddep_wait()") == 1
    for word in inputs:
        assert word in text and word not in ahead, (name, word)


def test_early_operands_are_never_of_a_first_kernel():
    """A dense product's producer passes over its grid wait for an operand named early: only in launches that follow
    another one of their call, and only for weights.  The small batches' first product waits before any load."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "ffn.cu")).read())
    assert text.count("l.early = ") == 2
    turned = text.index("l.early = dense::kEarlyA;")
    assert text.rindex("join_gate_kernel,", 0, turned) > 0 and "w.t_down, wd" in text[turned:turned + 200]
    whole = text.index("l.early = dense::kEarlyB;")
    assert text.rindex("dense::launch<EpiGate>", 0, whole) > 0 and "w.down" in text[whole:whole + 200]
    up = body("ffn.cu", "decode_kernel")
    first = up.index("if constexpr (!DOWN) {\n    griddep_wait();")
    assert first < up.index("load_w") and first < up.index("load_x")
