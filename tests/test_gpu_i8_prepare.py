"""The 8-bit product's kernels may be unusable (another compiler gives them fewer registers than
their warps hand around): the other operators still run.  The library is linked again from its
own objects, with the function that prepares those kernels replaced by one that fails."""
import glob
import os
import subprocess

import pytest
import torch

import dense_gemm_bf16_gb300 as dg
from dense_gemm_bf16_gb300 import _abi, _build

pytestmark = pytest.mark.gpu

PREPARE = "_ZN2dg10i8_prepareEv"
INVALID_CONFIGURATION = 9


@pytest.fixture(scope="module")
def crippled(tmp_path_factory):
    dg.build()
    work = tmp_path_factory.mktemp("i8")
    stub, path = str(work / "stub.cpp"), str(work / "libcrippled.so")
    with open(stub, "w") as f:
        f.write(f'extern "C" int __wrap_{PREPARE}() {{ return {INVALID_CONFIGURATION}; }}\n')
    objects = sorted(glob.glob(os.path.join(_build.OBJ_DIR, "*.cu.o")))
    assert objects
    subprocess.run([_build.nvcc()] + _build.ARCH + ["-shared", "-Xcompiler", "-fPIC", "-Xlinker",
                                                    f"--wrap={PREPARE}", "-o", path, stub] + objects,
                   check=True, capture_output=True, text=True)
    return _abi._load(path)


def test_other_operators_run_where_the_8_bit_product_cannot(crippled):
    st = torch.cuda.current_stream().cuda_stream
    x = torch.randn((6, 64), device="cuda:0")
    q, qs = torch.empty((6, 64), dtype=torch.int8, device="cuda:0"), torch.empty(6, device="cuda:0")
    assert crippled.gemm_i8_quantize(2, 6, 64, x.data_ptr(), 64, q.data_ptr(), 64, qs.data_ptr(), st) == 0
    want, scales = dg.i8_quantize(x)
    assert torch.equal(q, want) and torch.equal(qs, scales)
    slots = torch.arange(6, dtype=torch.int32, device="cuda:0").reshape(3, 2)
    y = torch.empty((3, 64), device="cuda:0")
    assert crippled.gemm_expert_combine(2, 3, 64, 2, x.data_ptr(), 6, 64, slots.data_ptr(), 0, 0, 0,
                                        y.data_ptr(), 64, 2, st) == 0
    assert torch.equal(y, dg.expert_combine(x, slots))
    a = torch.randn((6, 64), device="cuda:0").bfloat16()
    b = torch.randn((2, 64, 32), device="cuda:0").bfloat16()
    offsets = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda:0")
    c = torch.empty((6, 32), dtype=torch.bfloat16, device="cuda:0")
    assert crippled.gemm_grouped(0, 2, 6, 32, 64, a.data_ptr(), 64, b.data_ptr(), 32, 0, 64 * 32,
                                 c.data_ptr(), 32, 0, offsets.data_ptr(), 1.0, 0.0, 0, 0, 0, 0, 0, st) == 0
    assert torch.equal(c, dg.grouped_gemm(a, b, offsets))
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda:0")
    kept = torch.full((6, 6), 7.0, device="cuda:0")
    assert crippled.gemm_i8(3, 1, 6, 6, 64, q.data_ptr(), 64, qs.data_ptr(), q.data_ptr(), 64, 0,
                            qs.data_ptr(), 0, kept.data_ptr(), 6, 2, 0, 0, 0, 0, ws.data_ptr(),
                            ws.numel(), st) == dg.Status.ERR_CUDA
    torch.cuda.synchronize()
    assert bool((kept == 7).all()) and crippled.gemm_check_device_status(st) == 0
