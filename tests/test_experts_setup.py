"""When the grouped products cannot be set up on a device, the other entries still work.

The failure is made at link time: the library's own objects, but for the one that holds the grouped products' launches,
with a set-up in its place that returns the error a failing CUDA call would give.
"""
import os
import subprocess
import sys

import pytest

from dense_fp32_gemm_f32_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = """
#include "api_internal.h"
#include "experts.h"
namespace gb300 {
namespace detail {
int experts_tc_set_up(DeviceState&) { return SGEMM_ERR_CUDA; }
int grouped_tc(const GroupedCall&, int, DeviceState&, cudaStream_t) { return SGEMM_OK; }  // (never to be reached)
}  // namespace detail
}  // namespace gb300
"""

SCRIPT = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
import dense_fp32_gemm_f32_gb300 as g
from dense_fp32_gemm_f32_gb300 import _lib
_lib._build.build = lambda *a, **k: sys.argv[2]
A, B = torch.randn((300, 200), device="cuda"), torch.randn((200, 260), device="cuda")
want, bound = A.double() @ B.double(), A.double().abs() @ B.double().abs()
for f in (g.sgemm_f32, g.sgemm_3xtf32):
    assert ((f(A, B).double() - want).abs() <= 5e-5 * bound).all(), f
codes, scales = g.sgemm_mxfp4_quantize(A)  # (sets nothing up)
assert g.sgemm_mxfp4_dequantize(codes, scales, cols=200).shape == A.shape
o = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
for call in (lambda: g.sgemm_grouped(A, B[None], o), lambda: g.sgemm_grouped_wgrad(A, A, o),
             lambda: g.sgemm_mxfp4(codes, scales, codes, scales)):
    try:
        call()
    except g.SgemmError as e:
        assert e.status == _lib.ERR_CUDA
    else:
        raise AssertionError("a call without its set-up was let through")
assert g.check_status() == 0
print("ok")
"""


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    build.build()
    objects = [os.path.join(build.OUT_DIR, os.path.splitext(s)[0] + ".o") for s in build.SOURCES if s != "experts_tc.cu"]
    if not all(map(os.path.exists, objects)):
        build.build(force=True)
    at = tmp_path_factory.mktemp("stub")
    src, lib = at / "stub.cu", at / "libstub.so"
    src.write_text(STUB)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-Xcompiler", "-fPIC", "-I", build.CSRC, "-shared", "-o", str(lib),
                    str(src), *objects, "-cudart", "static"], check=True, capture_output=True)
    return str(lib)


@pytest.mark.gpu
def test_other_entries_work(library):
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT, library], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]
