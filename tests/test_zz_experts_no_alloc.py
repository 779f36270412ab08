"""The entry points that the header lists as non-allocating take no device memory, also on streams not seen before.

Run in a process of its own, so that no earlier pool's cache can hide an allocation.
"""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import json, sys
import torch
sys.path.insert(0, sys.argv[1])
import dense_fp32_gemm_f32_gb300 as g

cases = []
for T, E, K, N in ((3, 2, 200, 264), (700, 3, 4096, 1000), (40, 1, 40000, 136)):
    x, w = torch.randn((T, K + 1), device="cuda")[:, 1:], torch.randn((E, N, K), device="cuda").to(torch.bfloat16)
    o = torch.tensor([T * e // E for e in range(E + 1)], dtype=torch.int32, device="cuda")
    a, b, r = g.sgemm_mxfp4_quantize(x, o), g.sgemm_mxfp4_quantize(w), g.sgemm_mxfp4_quantize(x)
    cases.append((x, w, o, a, b, r, torch.empty((T, N), device="cuda"), torch.empty((T, K), dtype=torch.float16, device="cuda")))

def calls(stream):
    for x, w, o, a, b, r, y, v in cases:
        g.sgemm_mxfp4_quantize(x, o, codes=a[0], scales=a[1], stream=stream)
        g.sgemm_mxfp4_quantize(x, codes=r[0], scales=r[1], stream=stream)
        g.sgemm_mxfp4_quantize(w, codes=b[0], scales=b[1], stream=stream)
        g.sgemm_mxfp4_grouped(*a, *b, o, y, stream=stream)
        g.sgemm_mxfp4(*r, b[0][0], b[1][0], y, stream=stream)
        g.sgemm_mxfp4_dequantize(*a, o, cols=v.shape[1], out=v, stream=stream)
        g.sgemm_mxfp4_dequantize(*r, cols=v.shape[1], out=v, stream=stream)

streams = [torch.cuda.Stream() for _ in range(5)]
calls(streams[0])  # (set-up, loading of the kernels)
torch.cuda.synchronize()
before = torch.cuda.mem_get_info()[0]
for s in streams[1:]:
    calls(s)
torch.cuda.synchronize()
after = torch.cuda.mem_get_info()[0]
assert g.check_status() == 0
print(json.dumps([before, after]))
"""


@pytest.mark.gpu
def test_no_device_memory_is_taken():
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    before, after = json.loads(r.stdout.strip().splitlines()[-1])
    assert after == before
