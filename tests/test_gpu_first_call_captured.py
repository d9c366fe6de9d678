"""The first calls of a process made inside a stream capture: whatever the library looks up
or configures once must be allowed there. A process of its own."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from int4_q4_gemv_b200 import build as B

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import torch
from int4_q4_gemv_b200 import q4g as Q
torch.manual_seed(0)
B, H, D, P, C, V = 5, 16, 512, 300, 40, 5000
new = lambda *s: torch.randn(*s, device="cuda").half()
k, v, q = new(P, 1, D) * 0.2, new(P, 1, D), new(B, H, D) * 0.4
ok, ov = new(B, C, 1, D) * 0.2, new(B, C, 1, D)
codes = [torch.zeros(P, 1, D, dtype=torch.int8, device="cuda") for _ in range(2)]
scales = [torch.zeros(P, 1, device="cuda") for _ in range(2)]
lens = torch.tensor([0, 1, 17, 40, 33], dtype=torch.int32, device="cuda")
nb = Q.q4g_flash_decode_shared_workspace_bytes(B, H, 1, D)
ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
out = torch.zeros(2, B, H, D, dtype=torch.float16, device="cuda")
x = torch.randn(2, V, device="cuda")
t = torch.tensor([3, 4999], dtype=torch.int32, device="cuda")
lp, ids = torch.zeros(2, device="cuda"), torch.zeros(2, 4, dtype=torch.int32, device="cuda")
p = lambda *ts: [t.data_ptr() for t in ts]

def calls():
    st = torch.cuda.current_stream().cuda_stream
    cache = p(codes[0], scales[0], codes[1], scales[1])
    Q.q4g_kv_write_linear_i8(*p(k, v), P, D, 1, D, 0, 0, P, *cache, st)
    Q.q4g_flash_decode_shared(q.data_ptr(), B, H, 1, D, *p(k, v), P, *p(ok, ov), C, *p(lens, out[0], ws), nb, st)
    Q.q4g_flash_decode_shared_i8(q.data_ptr(), B, H, 1, D, *cache, P, 0, 0, 0, 0, 0, 0, *p(out[1], ws), nb, st)
    Q.q4g_token_logprobs(x.data_ptr(), 2, V, V, 1.0, *p(t, lp), 0, 4, ids.data_ptr(), 0, st)

s = torch.cuda.Stream()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    calls()
g.replay()
torch.cuda.synchronize()
got = [a.clone() for a in (out, lp, ids, *codes, *scales)]
assert bool((out != 0).any()) and bool((lp != 0).all())
for a in (out, lp, ids, *codes, *scales):
    a.zero_()
calls()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (out, lp, ids, *codes, *scales)))
Q.q4g_model_check(0, 0)
print("captured and eager calls agree")
"""


def test_first_calls_inside_a_capture():
    B.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "agree" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
