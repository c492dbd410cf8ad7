"""Batches whose every row has an adapter of its own: a list of a tile's adapters up to its last entry (128 of the stream form, 256 of
the pair form, 128 to a tile of the sums), walked once and, with more ranks, several times.

Tolerances as in the parity tests of the product with adapters.
"""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod
from oracle import grouped as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.load()


def _f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("r", [8, 40])
@pytest.mark.parametrize("M,N,K,L,each", [(128, 264, 520, 128, 1), (127, 520, 1032, 140, 1), (65, 136, 264, 65, 1), (256, 264, 328, 256, 1),
                                          (300, 520, 264, 300, 1), (255, 136, 520, 255, 1), (1030, 264, 264, 200, 1), (600, 264, 328, 97, 6)])
def test_an_adapter_for_every_row(M, N, K, L, each, r, out):
    g = torch.Generator().manual_seed(M + r)
    x, w, a, b = ((torch.randn(s, generator=g) * f).to(torch.bfloat16).cuda()
                  for s, f in (((M, K), 1), ((N, K), K ** -0.5), ((L, r, K), K ** -0.5), ((L, N, r), r ** -0.5)))
    order = torch.randperm(L, generator=g)
    ids = order[torch.arange(M) // each % L].to(torch.int32).cuda()
    assert len(ids[:256].unique()) == min(M, 256, L) or each > 1
    scale = torch.linspace(0.5, 2.0, L, device="cuda")
    h = B.LoraLinear(w, a, b, scale=scale, out_dtype=out)
    y = h(x, ids)
    s = torch.cuda.current_stream().cuda_stream
    assert B.gmmfr_check_device_errors(h._spaces[s][0], s) == 0
    ref, absb = O.lora_linear(_f64(x), _f64(w), _f64(a), _f64(b), _f64(scale), ids.cpu().numpy())
    if out == torch.bfloat16:
        tol = (K / 8 * 2.0 ** -23 + 2.0 ** -17 + r * 2.0 ** -23) * absb + 2.0 ** -8 * np.abs(ref)
    else:
        tol = (K / 8 + 3 * r / 8) * 2.0 ** -23 * absb + 2.0 ** -20 * np.abs(ref)
    err = np.abs(_f64(y) - ref)
    assert np.all(err <= tol), (float(err.max()), float((err / (tol + 1e-30)).max()))
