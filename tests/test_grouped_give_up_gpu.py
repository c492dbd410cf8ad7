"""The bounded waits of the grouped products and of the product with adapters run out: the accumulators' barriers wait for an
arrival that never comes (GMMFR_TEST_STALL_NS, read once, so each of the two runs is a process of its own).  Every form
ends by itself, sets the timeout bit, and leaves the context usable."""
import json
import os
import subprocess
import sys

import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = """
import json, time, torch
from moe_grouped_gemm_mxfp8_gb300 import binding as B

g = torch.Generator().manual_seed(1)
def randn(*shape, scale=0.05):
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()

s = torch.cuda.current_stream().cuda_stream
seen = {}
def call(name, handle, f):
    t0 = time.time()
    f()
    torch.cuda.synchronize()
    took = time.time() - t0
    seen[name] = [B.gmmfr_check_device_errors(handle._spaces[s][0], s), took]

for sizes in ([3, 0, 40, 1], [700, 300, 0, 2500]):
    for dtype in (torch.bfloat16, torch.float32):
        for transposed in (False, True):
            h = B.GroupedLinear(randn(4, 512, 1032), transposed=transposed, out_dtype=dtype, grad_dtype=dtype)
            K, N = (512, 1032) if transposed else (1032, 512)
            M = sum(sizes)
            x, dy, groups = randn(M, K), randn(M, N), torch.tensor(sizes, device="cuda")
            name = f"{M} {dtype} {transposed}"
            call("y " + name, h, lambda: h(x, groups))
            call("dx " + name, h, lambda: h.grad_input(dy, groups))
            call("dw " + name, h, lambda: h.grad_weight(dy, x, groups))
for M, N, K, act, dtype in ((40, 4096, 4096, "none", torch.bfloat16), (100, 40000, 1024, "swiglu", torch.bfloat16), (128, 300, 7168, "silu", torch.float32),
                            (300, 520, 1032, "none", torch.bfloat16), (1030, 4096, 2048, "none", torch.bfloat16), (5000, 2048, 1024, "swiglu", torch.float32)):
    rows = 2 * N if act == "swiglu" else N
    h = B.LoraLinear(randn(rows, K), randn(20, 24, K), randn(20, rows, 24), activation=act, out_dtype=dtype)
    ids = torch.randint(-1, 20, (M,), generator=g, dtype=torch.int32).cuda()
    x = randn(M, K)
    call(f"lora {M} {N} {K} {act}", h, lambda: h(x, ids))
x = torch.randn(1000, 1000, device="cuda")
print(json.dumps([seen, bool(torch.isfinite(x @ x).all())]))
"""


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.load()


def _run(**env):
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, cwd=ROOT, timeout=240,
                       env={**os.environ, "PYTHONPATH": ROOT, **env})
    assert r.returncode == 0, r.stderr[-2000:]
    seen, usable = json.loads(r.stdout.strip().splitlines()[-1])
    assert usable
    return seen


def test_the_calls_are_clean():
    for name, (bits, took) in _run().items():
        assert bits == 0, (name, bits)


def test_waits_that_run_out_end_the_call_with_the_timeout_bit():
    for name, (bits, took) in _run(GMMFR_TEST_STALL_NS="20000000").items():
        assert bits == B.DEV_TIMEOUT, (name, bits)
        assert took < 20, (name, took)
