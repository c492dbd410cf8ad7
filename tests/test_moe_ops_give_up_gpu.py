"""The bounded waits of the router, the layer and the dense product run out: the accumulators' barriers wait for an arrival
that never comes (GMMFR_TEST_STALL_NS, read once, so each of the two runs is a process of its own).  Every form ends by
itself, sets the timeout bit, and leaves the context usable."""
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
def call(name, handle, x):
    t0 = time.time()
    handle(x)
    torch.cuda.synchronize()
    took = time.time() - t0
    seen[name] = [B.gmmfr_check_device_errors(handle._spaces[s][0], s), took]

E, H, I = 16, 512, 128
wg, w13, w2 = randn(E, H), randn(E, H, 2 * I), randn(E, I, H)
codes = [torch.randint(0, 120, t.shape, dtype=torch.uint8, generator=g).cuda() for t in (w13, w2)]
scales = [torch.full((E, -(-k // 64), n, 2), 115, dtype=torch.uint8, device="cuda") for k, n in ((H, 2 * I), (I, H))]
for T in (1, 40):
    call(f"layer bf16 {T}", B.MoeLayer(wg, w13, w2, topk=4), randn(T, H))
    call(f"layer mxfp8 {T}", B.MoeLayer(wg, codes[0], codes[1], scales[0], scales[1], topk=4), randn(T, H))
for E2 in (64, 300):
    call(f"gate pair {E2}", B.MoeGate(randn(E2, 2048), topk=4), randn(60000, 2048))
call("stream", B.Linear(randn(300, 1024)), randn(100, 1024))
call("stream, many tiles", B.Linear(randn(40000, 1024), activation="swiglu"), randn(100, 1024))
call("pair", B.Linear(randn(4096, 2048)), randn(5000, 2048))
call("pair, short stages", B.Linear(randn(64, 2048)), randn(300, 2048))
call("pair and rows beside it", B.Linear(randn(4096, 2048)), randn(1030, 2048))
for M, N, K, act in ((100, 40000, 1024, "swiglu"), (60, 300, 7168, "none"), (5000, 4096, 2048, "none"), (1030, 4096, 2048, "swiglu")):
    call(f"float32 {M} x {N} x {K}", B.Linear(randn(2 * N if act == "swiglu" else N, K), activation=act, out_dtype=torch.float32), randn(M, K))
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


def test_waits_that_run_out_end_the_call_with_the_timeout_bit():
    for name, (bits, took) in _run(GMMFR_TEST_STALL_NS="20000000").items():
        assert bits == B.DEV_TIMEOUT, (name, bits)
        assert took < 20, (name, took)


def test_the_same_calls_are_clean_otherwise():
    for name, (bits, took) in _run().items():
        assert bits == 0, (name, bits)
