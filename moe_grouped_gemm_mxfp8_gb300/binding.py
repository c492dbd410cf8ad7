"""ctypes binding of the gmmfr C ABI (include/gmmfr.h).

Argument marshalling only: every step of the computation runs in the CUDA
library.  The functions named like the C entry points take raw device
addresses (int) or None; :func:`tensor_args` and :func:`run` turn torch
tensors into those.  The library is loaded on first use; if it has not been
built, loading raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libgmmfr.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE = range(6)
E4M3, E5M2 = 0, 1
INDEX_I64, INDEX_I32 = 0, 1
DETERMINISTIC = 1
DEV_BAD_GROUP_LIST, DEV_BAD_ROW_INDEX, DEV_TIMEOUT, DEV_BAD_EXPERT_ID = 1, 2, 4, 8
PROFILE_SLOTS = 5
PROFILE_SLOT_NAMES = ("prep", "route", "gemm", "combine", "call")

# exported entry points, as declared in include/gmmfr.h
ENTRY_POINTS = (
    "gmmfr_prepared_weights_size", "gmmfr_prepare_weights", "gmmfr_workspace_size",
    "gmmfr_grouped_matmul_finalize_routing", "gmmfr_check_device_errors", "gmmfr_last_error",
    "gmmfr_profile_begin", "gmmfr_profile_end", "gmmfr_grouped_matmul_finalize_routing_static_scratch",
    "gmmfr_static_scratch_check_device_errors",
    "gmmfr_moe_route_workspace_size", "gmmfr_moe_route",
    "gmmfr_ffn_prepared_weights_size", "gmmfr_ffn_prepare_weights", "gmmfr_ffn_workspace_size",
    "gmmfr_llada2_moe_grouped_gemm",
    "gmmfr_moe_gate_workspace_size", "gmmfr_moe_gate",
    "gmmfr_ffn_prepared_weights_size_mx", "gmmfr_ffn_prepare_weights_mx",
    "gmmfr_moe_layer_workspace_size", "gmmfr_moe_layer",
    "gmmfr_linear_workspace_size", "gmmfr_linear",
)
GATE_SCORING = {"softmax": 0, "sigmoid": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5}
LAYER_MAX_TOKENS = 64


DT_U8, DT_E4M3, DT_E5M2, DT_E2M1X2, DT_E8M0, DT_I64, DT_I32, DT_F32, DT_BF16 = range(9)
MAX_DIMS = 4


class Tensor(ctypes.Structure):
    """Mirror of gmmfr_tensor: a non-owning view of dense device memory."""
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * MAX_DIMS), ("strides", ctypes.c_int64 * MAX_DIMS)]


def raw_view(data, dtype: int, shape, strides=None) -> Tensor:
    """A view of `data` (an address, or None) with the given dtype code, shape and strides
    (dense row-major when not given)."""
    shape = tuple(int(x) for x in shape)
    if strides is None:
        strides, acc = [], 1
        for d in reversed(shape):
            strides.insert(0, acc)
            acc *= d
    t = Tensor()
    t.data = data
    t.dtype = dtype
    t.ndim = len(shape)
    for i, (d, st) in enumerate(zip(shape, strides)):
        t.shape[i] = d
        t.strides[i] = int(st)
    return t


class Problem(ctypes.Structure):
    """Mirror of gmmfr_problem."""
    _fields_ = [
        ("M", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64),
        ("E", ctypes.c_int64), ("batch", ctypes.c_int64),
        ("x1_format", ctypes.c_int32), ("x2_format", ctypes.c_int32),
        ("transpose_x2", ctypes.c_int32), ("scale_per_expert", ctypes.c_int32),
        ("group_list_type", ctypes.c_int32), ("row_index_type", ctypes.c_int32),
        ("shared_rows", ctypes.c_int64), ("shared_offset", ctypes.c_int64),
        ("shared_weight", ctypes.c_float), ("flags", ctypes.c_uint32),
        ("expected_tokens_per_expert", ctypes.c_int64),
    ]


class RouteProblem(ctypes.Structure):
    """Mirror of gmmfr_route_problem."""
    _fields_ = [
        ("batch", ctypes.c_int64), ("topk", ctypes.c_int64), ("K", ctypes.c_int64), ("E", ctypes.c_int64),
        ("ids_type", ctypes.c_int32), ("group_list_type", ctypes.c_int32),
    ]


class FfnProblem(ctypes.Structure):
    """Mirror of gmmfr_ffn_problem."""
    _fields_ = [("N", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64), ("E", ctypes.c_int64)]


class GateProblem(ctypes.Structure):
    """Mirror of gmmfr_gate_problem."""
    _fields_ = [
        ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("E", ctypes.c_int64), ("topk", ctypes.c_int64),
        ("ldx", ctypes.c_int64), ("scoring", ctypes.c_int32), ("n_group", ctypes.c_int32),
        ("topk_group", ctypes.c_int32), ("group_top", ctypes.c_int32), ("renormalise", ctypes.c_int32),
        ("ids_type", ctypes.c_int32), ("scale", ctypes.c_float),
    ]


class LayerProblem(ctypes.Structure):
    """Mirror of gmmfr_layer_problem."""
    _fields_ = [("gate", GateProblem), ("I", ctypes.c_int64), ("shared_I", ctypes.c_int64),
                ("ld_residual", ctypes.c_int64), ("ld_out", ctypes.c_int64), ("weight_type", ctypes.c_int32)]


class LinearProblem(ctypes.Structure):
    """Mirror of gmmfr_linear_problem."""
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("ldx", ctypes.c_int64),
                ("ldw", ctypes.c_int64), ("ld_residual", ctypes.c_int64), ("ld_out", ctypes.c_int64),
                ("activation", ctypes.c_int32), ("out_type", ctypes.c_int32), ("unaligned", ctypes.c_int32)]


class GmmfrError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"gmmfr status {status}: {message}")
        self.status = status


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load the library (once).  Raises if it is missing: there is no fallback."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"gmmfr CUDA library not built ({path}); run __graft_entry__.build()")
            lib = ctypes.CDLL(path)
            P = ctypes.POINTER(Problem)
            vp, sz = ctypes.c_void_p, ctypes.c_size_t
            lib.gmmfr_prepared_weights_size.argtypes = [P, ctypes.POINTER(sz)]
            T = ctypes.POINTER(Tensor)
            lib.gmmfr_prepare_weights.argtypes = [P, T, T, vp, sz, vp]
            lib.gmmfr_workspace_size.argtypes = [P, ctypes.c_int, ctypes.POINTER(sz)]
            lib.gmmfr_grouped_matmul_finalize_routing.argtypes = [P] + [T] * 10 + [vp, sz, vp, sz, vp]
            lib.gmmfr_grouped_matmul_finalize_routing_static_scratch.argtypes = [P] + [T] * 7 + [vp, sz, vp]
            lib.gmmfr_static_scratch_check_device_errors.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
            RP = ctypes.POINTER(RouteProblem)
            lib.gmmfr_moe_route_workspace_size.argtypes = [RP, ctypes.POINTER(sz)]
            lib.gmmfr_moe_route.argtypes = [RP] + [vp] * 11 + [sz, vp]
            FP = ctypes.POINTER(FfnProblem)
            lib.gmmfr_ffn_prepared_weights_size.argtypes = [FP, ctypes.POINTER(sz)]
            lib.gmmfr_ffn_prepare_weights.argtypes = [FP, vp, vp, vp, sz, vp]
            lib.gmmfr_ffn_workspace_size.argtypes = [FP, ctypes.POINTER(sz)]
            lib.gmmfr_llada2_moe_grouped_gemm.argtypes = [FP, vp, vp, vp, vp, vp, sz, vp]
            GP, LP, DP = ctypes.POINTER(GateProblem), ctypes.POINTER(LayerProblem), ctypes.POINTER(LinearProblem)
            lib.gmmfr_moe_gate_workspace_size.argtypes = [GP, ctypes.POINTER(sz)]
            lib.gmmfr_moe_gate.argtypes = [GP] + [vp] * 7 + [sz, vp]
            lib.gmmfr_ffn_prepared_weights_size_mx.argtypes = [FP, ctypes.POINTER(sz)]
            lib.gmmfr_ffn_prepare_weights_mx.argtypes = [FP] + [vp] * 5 + [sz, vp]
            lib.gmmfr_moe_layer_workspace_size.argtypes = [LP, ctypes.POINTER(sz)]
            lib.gmmfr_moe_layer.argtypes = [LP] + [vp] * 6 + [sz, vp, sz] + [vp] * 3 + [sz, vp]
            lib.gmmfr_linear_workspace_size.argtypes = [DP, ctypes.POINTER(sz)]
            lib.gmmfr_linear.argtypes = [DP] + [vp] * 6 + [sz, vp]
            lib.gmmfr_check_device_errors.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
            lib.gmmfr_last_error.restype = ctypes.c_char_p
            lib.gmmfr_profile_begin.argtypes = [ctypes.c_int]
            lib.gmmfr_profile_end.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_int,
                                              ctypes.POINTER(ctypes.c_int)]
            for name in ENTRY_POINTS:
                if name != "gmmfr_last_error":
                    getattr(lib, name).restype = ctypes.c_int
            _lib = lib
    return _lib


def gmmfr_last_error() -> str:
    return load().gmmfr_last_error().decode()


def _check(status: int) -> None:
    if status != OK:
        raise GmmfrError(status, gmmfr_last_error())


def make_problem(*, M, K, N, E, batch, x1_format=E4M3, x2_format=E4M3, transpose_x2=False,
                 scale_per_expert=False, group_list_type=1, row_index_type=INDEX_I64, shared_rows=0,
                 shared_offset=0, shared_weight=1.0, deterministic=False,
                 expected_tokens_per_expert=0) -> Problem:
    return Problem(M=M, K=K, N=N, E=E, batch=batch, x1_format=x1_format, x2_format=x2_format,
                   transpose_x2=int(bool(transpose_x2)), scale_per_expert=int(bool(scale_per_expert)),
                   group_list_type=group_list_type, row_index_type=row_index_type,
                   shared_rows=shared_rows, shared_offset=shared_offset, shared_weight=shared_weight,
                   flags=DETERMINISTIC if deterministic else 0,
                   expected_tokens_per_expert=expected_tokens_per_expert)


def problem_from_spec(spec, deterministic: bool = False, row_index_type: int = INDEX_I64) -> Problem:
    """gmmfr_problem for a workloads.Spec."""
    return make_problem(M=spec.M, K=spec.K, N=spec.N, E=spec.E, batch=spec.batch, x1_format=spec.x1_dtype,
                        x2_format=spec.x2_dtype, transpose_x2=spec.transpose_x2,
                        scale_per_expert=spec.scale_per_expert, group_list_type=spec.group_list_type,
                        row_index_type=row_index_type, shared_rows=spec.n_shared,
                        shared_offset=spec.shared_offset, shared_weight=spec.shared_weight,
                        deterministic=deterministic)


def gmmfr_prepared_weights_size(problem: Problem) -> int:
    n = ctypes.c_size_t()
    _check(load().gmmfr_prepared_weights_size(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def _ref(view: Optional[Tensor]):
    return None if view is None else ctypes.byref(view)


def gmmfr_prepare_weights(problem: Problem, x2: Optional[Tensor], scale: Optional[Tensor], prepared: Optional[int],
                          prepared_bytes: int, stream: Optional[int] = None) -> None:
    _check(load().gmmfr_prepare_weights(ctypes.byref(problem), _ref(x2), _ref(scale), prepared, prepared_bytes,
                                        stream))


def gmmfr_workspace_size(problem: Problem, have_prepared: bool) -> int:
    n = ctypes.c_size_t()
    _check(load().gmmfr_workspace_size(ctypes.byref(problem), int(bool(have_prepared)), ctypes.byref(n)))
    return n.value


def gmmfr_grouped_matmul_finalize_routing(problem: Problem, x1, x2, scale, pertoken_scale, group_list, logit,
                                          row_index, shared_input, bias, out, prepared, prepared_bytes, workspace,
                                          workspace_bytes, stream=None) -> None:
    """Tensor arguments are Tensor views (or None); prepared and workspace are addresses."""
    _check(load().gmmfr_grouped_matmul_finalize_routing(
        ctypes.byref(problem), _ref(x1), _ref(x2), _ref(scale), _ref(pertoken_scale), _ref(group_list), _ref(logit),
        _ref(row_index), _ref(shared_input), _ref(bias), _ref(out), prepared, prepared_bytes, workspace,
        workspace_bytes, stream))


def gmmfr_grouped_matmul_finalize_routing_static_scratch(problem: Problem, x1, pertoken_scale, group_list, logit,
                                                         row_index, shared_input, out, prepared, prepared_bytes,
                                                         stream=None) -> None:
    """The operator with the library's own 16 MiB device scratch instead of a
    caller workspace (for callers that cannot allocate); needs prepared weights."""
    _check(load().gmmfr_grouped_matmul_finalize_routing_static_scratch(
        ctypes.byref(problem), _ref(x1), _ref(pertoken_scale), _ref(group_list), _ref(logit), _ref(row_index),
        _ref(shared_input), _ref(out), prepared, prepared_bytes, stream))


def gmmfr_static_scratch_check_device_errors(stream=None) -> int:
    """Synchronises `stream`; returns the device error bits of the last static-scratch call
    on the current device (0 when clean)."""
    bits = ctypes.c_uint32()
    st = load().gmmfr_static_scratch_check_device_errors(stream, ctypes.byref(bits))
    if st not in (OK, ERR_DEVICE):
        _check(st)
    return bits.value


def gmmfr_moe_route_workspace_size(problem: RouteProblem) -> int:
    n = ctypes.c_size_t()
    _check(load().gmmfr_moe_route_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def gmmfr_moe_route(problem: RouteProblem, topk_ids, topk_weights, x, x_scale, x1, pertoken_scale, group_list,
                    row_index, logit, perm, workspace, workspace_bytes, stream=None) -> None:
    _check(load().gmmfr_moe_route(ctypes.byref(problem), topk_ids, topk_weights, x, x_scale, x1, pertoken_scale,
                                  group_list, row_index, logit, perm, workspace, workspace_bytes, stream))


def gmmfr_ffn_prepared_weights_size(problem: FfnProblem) -> int:
    n = ctypes.c_size_t()
    _check(load().gmmfr_ffn_prepared_weights_size(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def gmmfr_ffn_prepare_weights(problem: FfnProblem, w13_flat, w2_flat, prepared, prepared_bytes, stream=None) -> None:
    _check(load().gmmfr_ffn_prepare_weights(ctypes.byref(problem), w13_flat, w2_flat, prepared, prepared_bytes, stream))


def gmmfr_ffn_workspace_size(problem: FfnProblem) -> int:
    n = ctypes.c_size_t()
    _check(load().gmmfr_ffn_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def gmmfr_llada2_moe_grouped_gemm(problem: FfnProblem, sorted_tokens, prepared, expert_cumsum, result, workspace,
                                  workspace_bytes, stream=None) -> None:
    _check(load().gmmfr_llada2_moe_grouped_gemm(ctypes.byref(problem), sorted_tokens, prepared, expert_cumsum,
                                                result, workspace, workspace_bytes, stream))


def gmmfr_moe_gate_workspace_size(problem: GateProblem) -> int:
    n = ctypes.c_size_t()
    _check(load().gmmfr_moe_gate_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def gmmfr_moe_gate(problem: GateProblem, x, weight, select_bias, topk_ids, topk_weights, logits, workspace,
                   workspace_bytes, stream=None) -> None:
    _check(load().gmmfr_moe_gate(ctypes.byref(problem), x, weight, select_bias, topk_ids, topk_weights, logits,
                                 workspace, workspace_bytes, stream))


def gmmfr_ffn_prepared_weights_size_mx(problem: FfnProblem) -> int:
    n = ctypes.c_size_t()
    _check(load().gmmfr_ffn_prepared_weights_size_mx(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def gmmfr_ffn_prepare_weights_mx(problem: FfnProblem, w13, w13_scale, w2, w2_scale, prepared, prepared_bytes,
                                 stream=None) -> None:
    _check(load().gmmfr_ffn_prepare_weights_mx(ctypes.byref(problem), w13, w13_scale, w2, w2_scale, prepared,
                                               prepared_bytes, stream))


def gmmfr_moe_layer_workspace_size(problem: LayerProblem) -> int:
    n = ctypes.c_size_t()
    _check(load().gmmfr_moe_layer_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def gmmfr_moe_layer(problem: LayerProblem, x, gate_weight, select_bias, residual, out, prepared, prepared_bytes,
                    shared_prepared, shared_prepared_bytes, topk_ids, topk_weights, workspace, workspace_bytes,
                    stream=None) -> None:
    _check(load().gmmfr_moe_layer(ctypes.byref(problem), x, gate_weight, select_bias, residual, out, prepared,
                                  prepared_bytes, shared_prepared, shared_prepared_bytes, topk_ids, topk_weights,
                                  workspace, workspace_bytes, stream))


def gmmfr_linear_workspace_size(problem: LinearProblem) -> int:
    n = ctypes.c_size_t()
    _check(load().gmmfr_linear_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def gmmfr_linear(problem: LinearProblem, x, weight, bias, residual, out, workspace, workspace_bytes,
                 stream=None) -> None:
    _check(load().gmmfr_linear(ctypes.byref(problem), x, weight, bias, residual, out, workspace, workspace_bytes,
                               stream))


def gmmfr_check_device_errors(workspace: int, stream: Optional[int] = None) -> int:
    """Synchronises `stream`; returns the device error bits (0 when clean)."""
    bits = ctypes.c_uint32()
    st = load().gmmfr_check_device_errors(workspace, stream, ctypes.byref(bits))
    if st not in (OK, ERR_DEVICE):
        _check(st)
    return bits.value


def gmmfr_profile_begin(max_calls: int) -> None:
    _check(load().gmmfr_profile_begin(max_calls))


def gmmfr_profile_end(max_calls: int):
    """Per recorded call, the kernel times in ms by slot (-1 when not run)."""
    buf = (ctypes.c_float * (max_calls * PROFILE_SLOTS))()
    n = ctypes.c_int()
    _check(load().gmmfr_profile_end(buf, len(buf), ctypes.byref(n)))
    return [[buf[c * PROFILE_SLOTS + s] for s in range(PROFILE_SLOTS)] for c in range(n.value)]


# ---------------------------------------------------------------------------- torch marshalling
def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("gmmfr takes device tensors")
    if not t.is_contiguous():
        raise ValueError("gmmfr takes contiguous tensors")
    return t.data_ptr()


def _dtype_code(t) -> int:
    import torch
    codes = {torch.uint8: DT_U8, torch.int64: DT_I64, torch.int32: DT_I32, torch.float32: DT_F32,
             torch.bfloat16: DT_BF16, torch.float8_e4m3fn: DT_E4M3, torch.float8_e5m2: DT_E5M2}
    for name, code in (("float8_e8m0fnu", DT_E8M0), ("float4_e2m1fn_x2", DT_E2M1X2)):
        if hasattr(torch, name):
            codes[getattr(torch, name)] = code
    if t.dtype not in codes:
        raise ValueError(f"gmmfr has no element type for {t.dtype}")
    return codes[t.dtype]


def view(t) -> Optional[Tensor]:
    """The gmmfr_tensor view of a device tensor (None for None).  The library checks its
    element type, rank, shape and layout against the problem."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("gmmfr takes device tensors")
    return raw_view(t.data_ptr(), _dtype_code(t), tuple(t.shape), tuple(t.stride()))


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _in_pool_of(stream):
    """Allocations within come from the memory pool of the stream that is going to use them (None: the current one).  A
    block of another stream's pool may be one that this stream's kernels still use."""
    import torch
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _handed_over(stream, *tensors) -> None:
    """Results of a call on `stream` are going to be used on the current stream."""
    import torch
    if stream is not None:
        for t in tensors:
            t.record_stream(torch.cuda.current_stream(t.device))


def prepare_weights(problem: Problem, x2, scale, stream=None):
    """Allocate (torch) and fill the prepared-weight buffer for x2/scale."""
    import torch
    n = gmmfr_prepared_weights_size(problem)
    with _in_pool_of(stream):
        buf = torch.empty(max(n, 16), dtype=torch.uint8, device=x2.device)
    _handed_over(stream, buf)
    gmmfr_prepare_weights(problem, view(x2), view(scale), _ptr(buf), n, _stream(stream))
    return buf


def workspace(problem: Problem, have_prepared: bool, device) -> "torch.Tensor":
    import torch
    n = gmmfr_workspace_size(problem, have_prepared)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def run(problem: Problem, inputs: dict, out, prepared=None, ws=None, stream=None) -> None:
    """One call of the operator on device tensors (``inputs`` as made by
    workloads.make_inputs); accumulates into ``out`` in place."""
    if ws is None:
        with _in_pool_of(stream):
            ws = workspace(problem, prepared is not None, out.device)
    gmmfr_grouped_matmul_finalize_routing(
        problem, view(inputs["x1"]), view(inputs["x2"]) if prepared is None else None,
        view(inputs["scale"]) if prepared is None else None, view(inputs["pertoken_scale"]),
        view(inputs["group_list"]), view(inputs.get("logit")), view(inputs["row_index"]),
        view(inputs.get("shared_input")), view(inputs.get("bias")), view(out), _ptr(prepared),
        0 if prepared is None else prepared.numel(), _ptr(ws), ws.numel(), _stream(stream))
    return ws


def run_static_scratch(problem: Problem, inputs: dict, out, prepared, stream=None) -> None:
    """One call of the allocation-free entry point on device tensors."""
    gmmfr_grouped_matmul_finalize_routing_static_scratch(
        problem, view(inputs["x1"]), view(inputs["pertoken_scale"]), view(inputs["group_list"]),
        view(inputs.get("logit")), view(inputs["row_index"]), view(inputs.get("shared_input")), view(out),
        _ptr(prepared), prepared.numel(), _stream(stream))


def route(topk_ids, topk_weights, x, x_scale, E: int, group_list_type: int = 1, stream=None, ws=None):
    """Run the routing step on device tensors; returns (dict of outputs, workspace)."""
    import torch
    batch, topk = topk_ids.shape
    K = x.shape[1]
    rp = RouteProblem(batch=batch, topk=topk, K=K, E=E,
                      ids_type=INDEX_I32 if topk_ids.dtype == torch.int32 else INDEX_I64,
                      group_list_type=group_list_type)
    M = batch * topk
    dev = x.device
    with _in_pool_of(stream):
        o = dict(x1=torch.empty((M, K), dtype=torch.uint8, device=dev),
                 pertoken_scale=torch.empty((M,) + tuple(x_scale.shape[1:]), dtype=torch.uint8, device=dev),
                 group_list=torch.empty(E, dtype=torch.int64, device=dev),
                 row_index=torch.empty(M, dtype=torch.int64, device=dev),
                 logit=torch.empty(M, dtype=torch.float32, device=dev),
                 perm=torch.empty(M, dtype=torch.int32, device=dev))
        if ws is None:
            ws = torch.empty(max(gmmfr_moe_route_workspace_size(rp), 256), dtype=torch.uint8, device=dev)
    _handed_over(stream, *o.values())
    gmmfr_moe_route(rp, _ptr(topk_ids), _ptr(topk_weights), _ptr(x), _ptr(x_scale), _ptr(o["x1"]),
                    _ptr(o["pertoken_scale"]), _ptr(o["group_list"]), _ptr(o["row_index"]), _ptr(o["logit"]),
                    _ptr(o["perm"]), _ptr(ws), ws.numel(), _stream(stream))
    return o, ws


def ffn_prepare(H: int, I: int, E: int, w13_flat, w2_flat, stream=None):
    """Prepared-weight buffer (torch uint8) for the grouped FFN."""
    import torch
    fp = FfnProblem(N=0, H=H, I=I, E=E)
    n = gmmfr_ffn_prepared_weights_size(fp)
    with _in_pool_of(stream):
        buf = torch.empty(n, dtype=torch.uint8, device=w13_flat.device)
    _handed_over(stream, buf)
    gmmfr_ffn_prepare_weights(fp, _ptr(w13_flat), _ptr(w2_flat), _ptr(buf), n, _stream(stream))
    return buf


def ffn(sorted_tokens, prepared, expert_cumsum, H: int, I: int, E: int, result=None, ws=None, stream=None):
    """Run the grouped FFN on device tensors; returns (result, workspace)."""
    import torch
    N = sorted_tokens.shape[0]
    fp = FfnProblem(N=N, H=H, I=I, E=E)
    with _in_pool_of(stream):
        new = result is None
        if new:
            result = torch.zeros((N, H), dtype=torch.bfloat16, device=sorted_tokens.device)
        if ws is None:
            ws = torch.empty(gmmfr_ffn_workspace_size(fp), dtype=torch.uint8, device=sorted_tokens.device)
    if new:
        _handed_over(stream, result)
    gmmfr_llada2_moe_grouped_gemm(fp, _ptr(sorted_tokens), _ptr(prepared), _ptr(expert_cumsum), _ptr(result),
                                  _ptr(ws), ws.numel(), _stream(stream))
    return result, ws


def ffn_prepare_mx(H: int, I: int, E: int, w13, w13_scale, w2, w2_scale, stream=None):
    """Prepared-weight buffer (torch uint8) of MXFP8 FFN weights: w13 [E, H, 2I], w2 [E, I, H] E4M3
    (or their bytes) with E8M0 scales (or their bytes) [E, ceil(K/64), columns, 2]."""
    import torch
    codes, exponents = ((torch.uint8, torch.int8, t) for t in (torch.float8_e4m3fn, getattr(torch, "float8_e8m0fnu", torch.uint8)))
    for name, t, shape, types in (("w13", w13, (E, H, 2 * I), codes), ("w13_scale", w13_scale, (E, -(-H // 64), 2 * I, 2), exponents),
                                  ("w2", w2, (E, I, H), codes), ("w2_scale", w2_scale, (E, -(-I // 64), H, 2), exponents)):
        if t is None or t.numel() != _numel(shape) or t.dtype not in types:
            got = None if t is None else f"{tuple(t.shape)} {t.dtype}"
            raise ValueError(f"{name}: {got}, expected {shape} of {' or '.join(str(d) for d in dict.fromkeys(types))}")
    fp = FfnProblem(N=0, H=H, I=I, E=E)
    n = gmmfr_ffn_prepared_weights_size_mx(fp)
    with _in_pool_of(stream):
        buf = torch.empty(n, dtype=torch.uint8, device=w13.device)
    _handed_over(stream, buf)
    gmmfr_ffn_prepare_weights_mx(fp, _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(buf), n,
                                 _stream(stream))
    return buf


# ------------------------------------------------------------- handles of the router, the layer, the product
# A call of a handle costs the host as little as Python allows (its GPU work may be a few microseconds):
# what does not change between calls is marshalled once, in the constructor.
def _numel(shape) -> int:
    n = 1
    for d in shape:
        n *= d
    return n


def _refuse(name, t, want, device):
    if t.get_device() < 0:
        raise ValueError("gmmfr takes device tensors")
    if t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, its handle on cuda:{device}")
    raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} strides {t.stride()}, expected {want}")


def _rows(t, name: str, rows, cols: int, dtype, device: int):
    """The row stride of a 2-D tensor [rows, cols] (rows None: any) on cuda:`device` whose rows are contiguous; 0 when
    they are dense, or there is one, which has no stride to speak of."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 2 or shape[1] != cols or t.get_device() != device or (rows is not None and shape[0] != rows):
        _refuse(name, t, f"[{'rows' if rows is None else rows}, {cols}] {dtype}", device)
    if t.is_contiguous():
        return 0
    ld, inner = t.stride()
    if shape[0] > 1:
        # an expanded row (stride 0) is not a row of its own
        if ld < cols or (inner != 1 and cols > 1):
            _refuse(name, t, "rows that are contiguous and do not overlap", device)
        return ld
    if inner != 1 and cols > 1:
        _refuse(name, t, "contiguous rows", device)
    return 0


def _dense(t, name: str, shape, dtype, device: int):
    """The address of a dense tensor of this shape on cuda:`device`, or None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or tuple(t.shape) != shape or t.get_device() != device or not t.is_contiguous():
        _refuse(name, t, f"dense {shape} {dtype}", device)
    return t.data_ptr()


class _Handle:
    """Workspaces of a handle, one per stream it has been called on (a workspace serves one call in
    flight at a time).  One that a larger call outgrows stays with the handle, since a CUDA graph captured on that
    stream writes to it: a handle is kept as long as the graphs it was captured in, and graphs captured on the same
    stream are replayed one after the other.  A handle serves one host thread at a time, and runs on the device
    of its weights, whichever is current."""

    def __init__(self, device):
        import torch
        if device.type != "cuda":
            raise ValueError("gmmfr takes device tensors")
        self._lib = load()
        self._device = device
        self._index = torch.cuda.current_device() if device.index is None else device.index
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._empty = torch.empty
        # what torch.empty ends in for a CUDA tensor, without its argument parsing and dispatch (half its time)
        guards = getattr(getattr(torch._C, "_dynamo", None), "guards", None)
        self._empty_here = getattr(guards, "_empty_strided_cuda", None)
        self._current = torch._C._cuda_getDevice
        self._spaces = {}
        self._outgrown = []

    def _grow(self, raw: int, need: int, stream):
        import torch
        old = self._spaces.get(raw)
        if old is not None:
            self._outgrown.append(old[4])
            need = max(need, 2 * old[3])  # so that all that are kept come to less than the newest
        with _in_pool_of(stream):
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device=self._device)
            if old is None:  # a stream that the weights are new to
                for t in self._weight_tensors():
                    t.record_stream(torch.cuda.current_stream(self._device))
        # the C call's arguments are kept as ctypes objects: converting Python integers costs more than setting them
        entry = (ctypes.c_void_p(ws.data_ptr()), ctypes.c_size_t(ws.numel()), ctypes.c_void_p(raw), ws.numel(), ws)
        self._spaces[raw] = entry
        return entry

    def _there(self, *args):
        """The same call with the handle's device as the current one: a launch goes to the current device."""
        import torch
        with torch.cuda.device(self._index):
            return self(*args)

    def _weight_tensors(self):
        return [t for t in self._keep if t is not None]

    def _entry(self, name):
        """The C entry, called with ctypes objects of its argument types alone."""
        return self._lib[name]

    def _new(self, shape, dtype, stream):
        if stream is not None:
            with _in_pool_of(stream):
                t = self._empty(shape, dtype=dtype, device=self._device)
            _handed_over(stream, t)
            return t
        if self._empty_here is not None:
            return self._empty_here(shape, (shape[1], 1), dtype)
        return self._empty(shape, dtype=dtype, device=self._device)


def _gate_problem(device, weight, topk, scoring, select_bias, n_group, topk_group, group_top, renormalise, scale) -> GateProblem:
    import torch
    if weight.dim() != 2:
        _refuse("weight", weight, "[E, H]", device)
    E, H = weight.shape
    _dense(weight, "weight", (E, H), torch.bfloat16, device)
    _dense(select_bias, "select_bias", (E,), torch.float32, device)
    if scoring not in GATE_SCORING:
        raise ValueError(f"scoring {scoring!r} is not one of {sorted(GATE_SCORING)}")
    return GateProblem(T=0, H=H, E=E, topk=topk, ldx=0, scoring=GATE_SCORING[scoring], n_group=n_group,
                       topk_group=topk_group, group_top=group_top, renormalise=int(bool(renormalise)),
                       ids_type=INDEX_I32, scale=scale)


class MoeGate(_Handle):
    """The router: ``gate(x)`` -> (topk_ids [T, topk], topk_weights [T, topk] float32), the inputs of
    :func:`route`.  ``weight`` [E, H] bfloat16; the rule is gmmfr_gate_problem's."""

    def __init__(self, weight, topk: int, scoring: str = "softmax", select_bias=None, n_group: int = 1,
                 topk_group: int = 1, group_top: int = 2, renormalise: bool = True, scale: float = 1.0,
                 ids_dtype=None):
        import torch
        super().__init__(weight.device)
        self._p = p = _gate_problem(self._index, weight, topk, scoring, select_bias, n_group, topk_group, group_top, renormalise, scale)
        self._ids_dtype = torch.int32 if ids_dtype is None else ids_dtype
        if self._ids_dtype not in (torch.int32, torch.int64):
            raise ValueError(f"ids_dtype {ids_dtype} is not int32 or int64")
        p.ids_type = INDEX_I32 if self._ids_dtype == torch.int32 else INDEX_I64
        self._keep = (weight, select_bias)
        self._wptr, self._bptr = weight.data_ptr(), _ptr(select_bias)
        self._bf16, self._f32 = torch.bfloat16, torch.float32
        self._H, self._E, self._topk = p.H, p.E, p.topk
        self._ref, self._fn = ctypes.byref(p), self._entry("gmmfr_moe_gate")
        self._cx, self._ci, self._ck, self._cl = (ctypes.c_void_p() for _ in range(4))
        self._cw, self._cb = ctypes.c_void_p(self._wptr), ctypes.c_void_p(self._bptr)
        gmmfr_moe_gate_workspace_size(p)  # refuses a rule that is out of range
        self._T, self._need = 0, 0

    @property
    def topk(self) -> int:
        return self._topk

    def __call__(self, x, ids=None, weights=None, logits=None, stream=None):
        p, dev = self._p, self._index
        if self._current() != dev:
            return self._there(x, ids, weights, logits, stream)
        p.ldx = _rows(x, "x", None, self._H, self._bf16, dev)
        T = x.shape[0]
        if T != self._T:
            self._T = -1  # until the size is known to be taken: the problem holds what a refused call left in it
            p.T = T
            self._need = gmmfr_moe_gate_workspace_size(p)
            self._T = T
        shape = (T, self._topk)
        if ids is None:
            ids = self._new(shape, self._ids_dtype, stream)
            iptr = ids.data_ptr()
        else:
            iptr = _dense(ids, "ids", shape, self._ids_dtype, dev)
        if weights is None:
            weights = self._new(shape, self._f32, stream)
            wptr = weights.data_ptr()
        else:
            wptr = _dense(weights, "weights", shape, self._f32, dev)
        lptr = None if logits is None else _dense(logits, "logits", (T, self._E), self._f32, dev)
        s = self._raw_stream(self._index) if stream is None else stream.cuda_stream
        ws = self._spaces.get(s)
        if ws is None or ws[3] < self._need:
            ws = self._grow(s, self._need, stream)
        cx, ci, ck, cl = self._cx, self._ci, self._ck, self._cl
        cx.value, ci.value, ck.value, cl.value = x.data_ptr(), iptr, wptr, lptr
        st = self._fn(self._ref, cx, self._cw, self._cb, ci, ck, cl, ws[0], ws[1], ws[2])
        if st:
            _check(st)
        return ids, weights


class MoeLayer(_Handle):
    """A whole MoE layer for up to 64 tokens, gate included: ``layer(x, residual=None)`` -> out [T, H].

    ``gate_weight`` [E, H]; ``w13`` [E, H, 2I] and ``w2`` [E, I, H] bfloat16, or E4M3 with
    ``w13_scale`` / ``w2_scale`` (E8M0, [E, ceil(K/64), columns, 2]); the shared expert's weights as
    [H, 2 shared_I] and [shared_I, H] of the same kind.  The weights are laid out once, here, on the current
    stream (calls on another are ordered after it by the caller, as after any kernel); the keyword arguments after
    them are the gate's."""

    def __init__(self, gate_weight, w13, w2, w13_scale=None, w2_scale=None, shared_w13=None, shared_w2=None,
                 shared_w13_scale=None, shared_w2_scale=None, *, topk: int, scoring: str = "softmax",
                 select_bias=None, n_group: int = 1, topk_group: int = 1, group_top: int = 2,
                 renormalise: bool = True, scale: float = 1.0):
        import torch
        super().__init__(gate_weight.device)
        gp = _gate_problem(self._index, gate_weight, topk, scoring, select_bias, n_group, topk_group, group_top, renormalise, scale)
        E, H, I = gp.E, gp.H, w2.shape[1]
        mx = w13_scale is not None or w2_scale is not None
        for name, t in (("w13", w13), ("w2", w2), ("w13_scale", w13_scale), ("w2_scale", w2_scale), ("shared_w13", shared_w13),
                        ("shared_w2", shared_w2), ("shared_w13_scale", shared_w13_scale), ("shared_w2_scale", shared_w2_scale)):
            if t is not None and t.get_device() != self._index:
                _refuse(name, t, "", self._index)
        if (shared_w13 is None) != (shared_w2 is None):
            raise ValueError("shared_w13 and shared_w2 come together")
        shared_I, self._shared = 0, None
        with torch.cuda.device(self._index):
            self._prepared = self._prepare(E, H, I, w13, w13_scale, w2, w2_scale, mx)
            if shared_w13 is not None:
                shared_I = shared_w2.shape[0]
                self._shared = self._prepare(1, H, shared_I, shared_w13, shared_w13_scale, shared_w2, shared_w2_scale, mx)
        self._p = p = LayerProblem(gate=gp, I=I, shared_I=shared_I, ld_residual=0, ld_out=0,
                                   weight_type=DT_E4M3 if mx else DT_BF16)
        self._g = p.gate
        self._keep = (gate_weight, select_bias, self._prepared, self._shared)
        self._wptr, self._bptr = gate_weight.data_ptr(), _ptr(select_bias)
        self._weights = (ctypes.c_void_p(self._prepared.data_ptr()), ctypes.c_size_t(self._prepared.numel()),
                         ctypes.c_void_p(_ptr(self._shared)),
                         ctypes.c_size_t(0 if self._shared is None else self._shared.numel()))
        self._bf16, self._i32, self._f32 = torch.bfloat16, torch.int32, torch.float32
        self._H, self._topk = H, gp.topk
        self._ref, self._fn = ctypes.byref(p), self._entry("gmmfr_moe_layer")
        self._cx, self._cr, self._co, self._ci, self._ck = (ctypes.c_void_p() for _ in range(5))
        self._cw, self._cb = ctypes.c_void_p(self._wptr), ctypes.c_void_p(self._bptr)
        # one workspace for every number of tokens: sizes called, or captured in graphs, in any order share it
        self._g.T = LAYER_MAX_TOKENS
        self._need = gmmfr_moe_layer_workspace_size(p)

    @property
    def prepared(self):
        """The routed experts' prepared weights (BF16 ones are what :func:`ffn` takes)."""
        return self._prepared

    @staticmethod
    def _prepare(E, H, I, w13, s13, w2, s2, mx):
        import torch
        if mx:
            return ffn_prepare_mx(H, I, E, w13, s13, w2, s2)
        for name, t, shape in (("w13", w13, (E, H, 2 * I)), ("w2", w2, (E, I, H))):
            if t is None or t.dtype != torch.bfloat16 or t.numel() != _numel(shape):
                got = None if t is None else f"{tuple(t.shape)} {t.dtype}"
                raise ValueError(f"{name}: {got}, expected {shape} bfloat16 (or E4M3 with its scales)")
        return ffn_prepare(H, I, E, w13, w2)

    def __call__(self, x, residual=None, out=None, topk_ids=None, topk_weights=None, stream=None):
        p, g, H, dev = self._p, self._g, self._H, self._index
        if self._current() != dev:
            return self._there(x, residual, out, topk_ids, topk_weights, stream)
        g.ldx = _rows(x, "x", None, H, self._bf16, dev)
        g.T = T = x.shape[0]
        rptr, p.ld_residual = None, 0
        if residual is not None:
            p.ld_residual = _rows(residual, "residual", T, H, self._bf16, dev)
            rptr = residual.data_ptr()
        if out is None:
            out = self._new((T, H), self._bf16, stream)
            p.ld_out = 0
        else:
            p.ld_out = _rows(out, "out", T, H, self._bf16, dev)
        iptr = None if topk_ids is None else _dense(topk_ids, "topk_ids", (T, self._topk), self._i32, dev)
        kptr = None if topk_weights is None else _dense(topk_weights, "topk_weights", (T, self._topk), self._f32, dev)
        s = self._raw_stream(self._index) if stream is None else stream.cuda_stream
        ws = self._spaces.get(s)
        if ws is None or ws[3] < self._need:
            ws = self._grow(s, self._need, stream)
        cx, cr, co, ci, ck = self._cx, self._cr, self._co, self._ci, self._ck
        cx.value, cr.value, co.value, ci.value, ck.value = x.data_ptr(), rptr, out.data_ptr(), iptr, kptr
        st = self._fn(self._ref, cx, self._cw, self._cb, cr, co, *self._weights, ci, ck, ws[0], ws[1], ws[2])
        if st:
            _check(st)
        return out


class Linear(_Handle):
    """The dense product: ``linear(x, residual=None)`` -> act(x @ weight.T + bias) + residual.

    ``weight`` [N, K] bfloat16 (rows may be strided); with ``activation="swiglu"`` [2N, K], the gate
    rows then the up rows, and ``bias`` [2N]."""

    def __init__(self, weight, bias=None, activation: str = "none", out_dtype=None):
        import torch
        super().__init__(weight.device)
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation {activation!r} is not one of {sorted(ACTIVATIONS)}")
        self._out = torch.bfloat16 if out_dtype is None else out_dtype
        if self._out not in (torch.bfloat16, torch.float32):
            raise ValueError(f"out_dtype {out_dtype} is not bfloat16 or float32")
        if weight.dim() != 2:
            _refuse("weight", weight, "[N, K]", self._index)
        rows, K = weight.shape
        ldw = _rows(weight, "weight", None, K, torch.bfloat16, self._index)
        if activation == "swiglu" and rows % 2:
            raise ValueError(f"weight: {rows} rows; swiglu takes gate and up rows, an even number")
        self._bptr = _dense(bias, "bias", (rows,), torch.bfloat16, self._index)
        self._keep = (weight, bias)
        self._wptr = weight.data_ptr()
        self._K, self._N = K, rows // 2 if activation == "swiglu" else rows
        self._p = p = LinearProblem(M=0, N=self._N, K=K, ldx=0, ldw=ldw, ld_residual=0, ld_out=0,
                                    activation=ACTIVATIONS[activation],
                                    out_type=DT_F32 if self._out == torch.float32 else DT_BF16)
        self._bf16 = torch.bfloat16
        self._ref, self._fn = ctypes.byref(p), self._entry("gmmfr_linear")
        self._cx, self._cr, self._co = (ctypes.c_void_p() for _ in range(3))
        self._cw, self._cb = ctypes.c_void_p(self._wptr), ctypes.c_void_p(self._bptr)
        gmmfr_linear_workspace_size(p)
        self._seen, self._need = None, 0

    def __call__(self, x, residual=None, out=None, stream=None):
        p, N, dev = self._p, self._N, self._index
        if self._current() != dev:
            return self._there(x, residual, out, stream)
        ldx = _rows(x, "x", None, self._K, self._bf16, dev)
        M, xptr = x.shape[0], x.data_ptr()
        seen = (M, ldx, (xptr | self._wptr) & 15)
        if seen != self._seen:
            self._seen = None  # until the size is known to be taken: the problem holds what a refused call left in it
            p.M, p.ldx, p.unaligned = M, ldx, int(seen[2] != 0)
            self._need = gmmfr_linear_workspace_size(p)
            self._seen = seen
        rptr, p.ld_residual = None, 0
        if residual is not None:
            p.ld_residual = _rows(residual, "residual", M, N, self._bf16, dev)
            rptr = residual.data_ptr()
        if out is None:
            out = self._new((M, N), self._out, stream)
            p.ld_out = 0
        else:
            p.ld_out = _rows(out, "out", M, N, self._out, dev)
        s = self._raw_stream(self._index) if stream is None else stream.cuda_stream
        ws = self._spaces.get(s)
        if ws is None or ws[3] < self._need:
            ws = self._grow(s, self._need, stream)
        cx, cr, co = self._cx, self._cr, self._co
        cx.value, cr.value, co.value = xptr, rptr, out.data_ptr()
        st = self._fn(self._ref, cx, self._cw, self._cb, cr, co, ws[0], ws[1], ws[2])
        if st:
            _check(st)
        return out
