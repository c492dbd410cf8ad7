"""Dense products whose K is no multiple of 8, with NaN and infinities wherever a row ends: behind x, behind the weights,
and in the columns between a row and the next.

Tolerance as in the parity tests: FP32 sums K / 8 * 2^-23 of the absolute sum, one BF16 rounding 2^-8.
"""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod
from oracle import moe as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.load()


def _f64(t):
    return t.detach().cpu().double().numpy()


def _rows(g, rows, K, pitch, scale=1.0):
    """[rows, K] of row stride `pitch`, everything else in the buffer (a row's worth behind it too) NaN or infinite."""
    buf = torch.full((rows * pitch + 64,), float("nan"), dtype=torch.bfloat16)
    buf[1::3] = float("inf")
    buf = buf.cuda()
    t = buf.as_strided((rows, K), (pitch, 1))
    t.copy_((torch.randn((rows, K), generator=g) * scale).to(torch.bfloat16))
    return t


def _check(x, w, act):
    y = B.Linear(w, activation=act)(x)
    ref, absb = O.linear(_f64(x), _f64(w), activation=act)
    err = np.abs(_f64(y) - ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + x.shape[1] / 8 * 2.0 ** -23 * absb + 1e-30)


@pytest.mark.parametrize("K", [1, 7, 9, 33, 1285, 2047])
@pytest.mark.parametrize("M", [1, 5, 20, 40, 300])
def test_rows_that_end_inside_a_16_byte_piece(M, K):
    g = torch.Generator().manual_seed(M * K)
    up = (K + 7) // 8 * 8
    for N in (1, 70):
        for px, pw in ((up, up), (up + 8, K), (K, up), (K, K)):
            for act in ("none", "swiglu"):
                rows = 2 * N if act == "swiglu" else N
                _check(_rows(g, M, K, px), _rows(g, rows, K, pw, scale=K ** -0.5), act)


@pytest.mark.parametrize("M", [1, 2, 32])
def test_one_weight_row(M):
    g = torch.Generator().manual_seed(M)
    for K in (3, 515, 4097):
        _check(_rows(g, M, K, K), _rows(g, 1, K, K, scale=K ** -0.5), "gelu")


def _entry(x, w, workspace, unaligned=0, **kw):
    """The C entry itself, on a workspace of the caller's."""
    M, K = x.shape
    N = w.shape[0]
    p = B.LinearProblem(**{**dict(M=M, N=N, K=K, ldx=x.stride(0), ldw=w.stride(0), ld_residual=0, ld_out=0, activation=0,
                                  out_type=B.DT_F32, unaligned=unaligned), **kw})
    need = B.gmmfr_linear_workspace_size(p)
    assert workspace.numel() >= need
    out = torch.empty((M, N), device="cuda")
    B.gmmfr_linear(p, x.data_ptr(), w.data_ptr(), None, None, out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                   torch.cuda.current_stream().cuda_stream)
    return out


def test_a_refused_call_enqueues_nothing():
    g = torch.Generator().manual_seed(1)
    x, w = _rows(g, 300, 129, 131), _rows(g, 64, 129, 136)
    ws = torch.full((1 << 20,), 0xA5, dtype=torch.uint8, device="cuda")
    with pytest.raises(B.GmmfrError):
        _entry(x, w, ws, ldw=1 << 40)  # a row stride that no tensor copy takes; x is copied to the workspace first
    torch.cuda.synchronize()
    assert (ws == 0xA5).all()


@pytest.mark.parametrize("M", [1, 20, 60, 300])
def test_only_what_is_off_a_boundary_is_copied(M):
    g = torch.Generator().manual_seed(M)
    K, N = 264, 48
    x, w = (torch.randn((r, K + 8), generator=g).to(torch.bfloat16).cuda() for r in (M, N))
    copies = {"x": M * K * 2, "w": N * K * 2}
    for off_x, off_w in ((0, 0), (1, 0), (0, 3), (5, 1)):
        xs, wsl = x[:, off_x:off_x + K], w[:, off_w:off_w + K]
        ws = torch.full((1 << 20,), 0xA5, dtype=torch.uint8, device="cuda")
        out = _entry(xs, wsl, ws, unaligned=1)
        ref, absb = O.linear(_f64(xs), _f64(wsl))
        assert np.all(np.abs(_f64(out) - ref) <= 2.0 ** -20 * np.abs(ref) + K / 8 * 2.0 ** -23 * absb + 1e-30)
        written = ws[4096:].ne(0xA5).sum().item()  # behind the error words
        want = (copies["x"] if off_x else 0) + (copies["w"] if off_w else 0)
        assert 0.98 * want <= written <= want, (off_x, off_w, written, want)
