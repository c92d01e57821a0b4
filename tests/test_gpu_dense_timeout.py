"""Bounded waits of the dense products that run out: tests/native/stalled_products.cu
runs their kernels with an epilogue that stalls for longer than the limit.  The status
word says so, the kernel ends by itself, and the context works on."""
import ctypes
import os
import subprocess
import time

import pytest
import torch

import precision_moe_grouped_gb300 as P
import test_gpu_ffn as F
import test_gpu_muon as M
from precision_moe_grouped_gb300 import _lib as L

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "precision_moe_grouped_gb300", "csrc")
MS = 1_000_000


@pytest.fixture(scope="module")
def stalled(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("stalled") / "stalled.so")
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                    "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-shared", "-o", out,
                    os.path.join(ROOT, "tests", "native", "stalled_products.cu"), os.path.join(CSRC, "dense.cu"), "-lcudart"],
                   check=True)
    lib = ctypes.CDLL(out)
    lib.stalled_product.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint64,
                                    ctypes.c_int, ctypes.c_void_p]
    return lib.stalled_product


@pytest.mark.parametrize("which", [0, 1, 2], ids=["dense", "terms", "chain"])
def test_a_wait_that_runs_out(cuda_ok, stalled, which):
    s = F.make(300, 264, 136, seed=1)
    op = P.GatedFFN(s["wgu"], s["wd"])
    grad = M.inputs("noise", (100, 200), 1)

    def work():
        p = torch.zeros_like(grad)
        muon = P.Muon([p], [grad], lr=1.0)
        muon.step()
        assert muon.device_status() == 0
        return op(s["x"], base=s["base"]), p

    want = work()
    mem = torch.zeros(4 << 20, dtype=torch.uint8, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for limit, stall, code in ((1000 * MS, 2 * MS, L.MOE_OK), (MS, 5 * MS, L.MOE_ERR_DEVICE_TIMEOUT)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        t = time.perf_counter()
        assert stalled(which, mem.data_ptr(), status.data_ptr(), limit, stall, sms, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert time.perf_counter() - t < 2
        assert int(status) == code
        for a, b in zip(work(), want):
            assert torch.equal(a, b)
    assert op.device_status() == 0
