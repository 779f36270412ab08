"""The entry points of routing and updates that their headers list as non-allocating take no device memory, also on streams
not seen before.

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
from dense_fp32_gemm_f32_gb300 import _lib

lib = _lib.load()
rows = []
for T, E, k, H in ((3, 4, 2, 40), (700, 64, 4, 1001), (20000, 8, 1, 256)):
    logits = torch.randn((T, E), device="cuda")
    r = g.sgemm_route(logits, k)
    x = torch.randn((T, H), device="cuda")
    y, out, dy = torch.zeros((T * k, H), device="cuda"), torch.zeros((T, H), device="cuda"), torch.zeros((T * k, H), device="cuda")
    rows.append((T, E, k, H, logits, r, x, y, out, dy, torch.zeros((T, k), device="cuda"), torch.zeros((T, E), device="cuda")))
updates = []
for E, M, N in ((3, 100, 120), (2, 128, 2048), (2, 300, 260), (1, 260, 5000), (9, 64, 64)):
    x = torch.randn((E, M, N), device="cuda")
    n = lib.sgemm_orthogonalize_workspace(0, E, M, N, 5)
    updates.append((E, M, N, x, torch.zeros_like(x), n, torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")))

def calls(stream):
    s = stream.cuda_stream
    for T, E, k, H, logits, r, x, y, out, dy, dw, dl in rows:
        e, w, o, q = (t.data_ptr() for t in r)
        R = T * k
        for rc in (lib.sgemm_spread(0, T, k, R, H, x.data_ptr(), H, q, E, o, y.data_ptr(), H, s),
                   lib.sgemm_combine(0, T, k, R, H, y.data_ptr(), H, q, w, out.data_ptr(), H, s),
                   lib.sgemm_combine_grad(0, T, k, R, H, out.data_ptr(), H, y.data_ptr(), H, q, w, E, o, dy.data_ptr(), H, dw.data_ptr(), s),
                   lib.sgemm_route_grad(0, 0, T, E, k, logits.data_ptr(), E, e, dw.data_ptr(), 0, 1.0, dl.data_ptr(), E, s)):
            _lib.check(rc, "rows")
    for E, M, N, x, y, n, ws in updates:
        _lib.check(lib.sgemm_orthogonalize(0, E, M, N, x.data_ptr(), N, M * N, 5, 3.4445, -4.7750, 2.0315, 1e-7, y.data_ptr(), N, M * N,
                                           ws.data_ptr() if n else None, n, s), "update")

torch.cuda.synchronize()
streams = [torch.cuda.Stream() for _ in range(4)]
calls(streams[0])  # (set-up, loading of the kernels)
torch.cuda.synchronize()
before = torch.cuda.mem_get_info()[0]
for s in streams[1:]:
    calls(s)
    torch.cuda.synchronize()  # (the calls' outputs and scratch are the same on every stream)
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
