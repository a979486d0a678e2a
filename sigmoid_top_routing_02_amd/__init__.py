"""Python binding of libmoefp8.so, the MI355X (gfx950) DeepSeekMoE layer forward.

Thin ctypes marshalling over the C ABI declared in ``include/moe_fp8.h``:
every function here has the name of a C entry point, checks tensor dtypes,
devices and shapes, allocates outputs with torch when the caller passes none,
and hands raw device pointers plus torch's current HIP stream to the library.
All arithmetic runs in the library's HIP kernels; there is no fallback.  If
the shared library is missing the calls raise instead of computing anything.
"""
from __future__ import annotations

import ctypes
import os
from collections import namedtuple

import numpy as np

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoefp8.so")

MOE_BF16, MOE_F32 = 0, 1
_DTYPES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}
MOE_EPI_STORE_F32, MOE_EPI_SWIGLU_F32, MOE_EPI_SWIGLU_QUANT, MOE_EPI_SWIGLU_QUANT_Z = 0, 1, 2, 3
MOE_MX_STORE_F32, MOE_MX_STORE_BF16, MOE_MX_SWIGLU_BF16, MOE_MX_SWIGLU_QUANT = 0, 1, 2, 3

# every symbol the header declares (kept in step with include/moe_fp8.h)
EXPORTS = (
    "moe_status_string", "moe_last_error", "moe_version",
    "moe_router_topk", "moe_router_topk_grouped",
    "moe_seq_balance_loss_workspace_bytes", "moe_seq_balance_loss",
    "moe_dispatch_workspace_bytes", "moe_dispatch", "moe_dispatch_check", "moe_permute_rows",
    "fp8_quant_1x128", "fp8_quant_128x128",
    "moe_gemm_workspace_bytes", "grouped_gemm_fp8_blockscaled", "grouped_gemm_fp8_blockscaled_noalloc",
    "moe_fp8_mfma_accumulation_probe", "moe_combine", "moe_bias_update",
    "moe_packed_weight_bytes", "moe_prepare_expert_weights",
    "moe_layer_workspace_bytes", "moe_layer_forward",
    "moe_prepare_backward_weights", "moe_gate_backward", "moe_swiglu_backward", "moe_router_backward",
    "moe_wgrad_block_starts", "moe_wgrad_operands", "moe_wgrad_workspace_bytes", "moe_wgrad",
    "moe_add_rmsnorm", "moe_add_rmsnorm_backward_workspace_bytes", "moe_add_rmsnorm_backward",
    "mxfp4_quant_1x32", "mxfp4_dequant_1x32", "fp8_dequant_1x128", "grouped_gemm_mxfp4",
    "moe_balance_loss_workspace_bytes", "moe_balance_loss", "moe_balance_loss_backward",
    "moe_router_logits_backward_workspace_bytes", "moe_router_logits_backward",
    "grouped_gemm_fp8_swiglu_zq", "moe_swiglu_backward_zq", "moe_wgrad_operands_zq",
    "moe_add_layernorm", "moe_add_layernorm_backward_workspace_bytes", "moe_add_layernorm_backward",
)


class MoEError(RuntimeError):
    pass


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libmoefp8.so and declare the C signatures (no GPU needed)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise MoEError(f"{path} is missing: build it with sigmoid_top_routing_02_amd/build.py")
    L = ctypes.CDLL(path)
    P, I64, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    sig = {
        "moe_status_string": ([I32], ctypes.c_char_p),
        "moe_last_error": ([], ctypes.c_char_p),
        "moe_version": ([], I32),
        "moe_router_topk": ([P, P, P, I64, I32, I32, I32, P, P, P, P], I32),
        "moe_router_topk_grouped": ([P, P, P, I64, I32, I32, I32, I32, I32, P, P, P, P], I32),
        "moe_seq_balance_loss_workspace_bytes": ([I64, I32], SZ),
        "moe_seq_balance_loss": ([P, P, I64, I32, I32, I32, F32, P, P, SZ, P], I32),
        "moe_dispatch_workspace_bytes": ([I64, I32], SZ),
        "moe_dispatch": ([P, I64, I32, I32, I32, P, P, P, P, P, SZ, P], I32),
        "moe_dispatch_check": ([P, P, P, P, P, I64, I32, I32, I32, P, P], I32),
        "moe_permute_rows": ([P, I32, P, I64, I32, P, P], I32),
        "fp8_quant_1x128": ([P, I32, I64, I32, P, P, P], I32),
        "fp8_quant_128x128": ([P, I64, I32, P, P, P], I32),
        "moe_gemm_workspace_bytes": ([I32, I64, I32, I32], SZ),
        "grouped_gemm_fp8_blockscaled": ([P, P, P, P, I32, I64, P, P, I32, I32, I32, P, P, P, P, SZ, P], I32),
        "grouped_gemm_fp8_blockscaled_noalloc": ([P, P, P, P, I32, I64, P, P, I32, I32, I32, P, P, P, P], I32),
        "moe_fp8_mfma_accumulation_probe": ([P, P, I32, I32, I32, I32, P, P], I32),
        "moe_combine": ([P, P, I32, I64, P, P, I64, I32, I32, P, P], I32),
        "moe_bias_update": ([P, P, I32, I64, F32, P], I32),
        "moe_packed_weight_bytes": ([I32, I32, I32], SZ),
        "moe_prepare_expert_weights": ([P, P, P, I32, I32, I32, I32, P, P], I32),
        "moe_layer_workspace_bytes": ([I64, I32, I32, I32, I32], SZ),
        "moe_layer_forward": ([P, P, P, P, I64, I32, I32, I32, I32, P, P, P, SZ, P], I32),
        "moe_prepare_backward_weights": ([P, I32, I32, I32, P, P], I32),
        "moe_gate_backward": ([P, P, I64, P, P, P, P, I64, I32, I32, I32, P, P, P, P, P], I32),
        "moe_swiglu_backward": ([P, P, I64, I32, P, P, P], I32),
        "moe_router_backward": ([P, P, I64, P, P, P, P, P, P, P, P, I64, I32, I32, I32, P, P, P], I32),
        "moe_wgrad_block_starts": ([P, I32, P, P], I32),
        "moe_wgrad_operands": ([P, P, P, P, P, P, P, P, P, I32, I32, I64, I32, I32, I32, I64,
                                P, P, P, P, P, P, P, P, P], I32),
        "moe_wgrad_workspace_bytes": ([I32, I32, I32], SZ),
        "moe_add_rmsnorm": ([P, I32, P, I32, P, I32, I64, I32, F32, P, P, P, P, P, P], I32),
        "moe_add_rmsnorm_backward_workspace_bytes": ([I64, I32], SZ),
        "moe_add_rmsnorm_backward": ([P, I32, P, I32, P, I32, P, P, I64, I32, P, I32, P, P, SZ, P], I32),
        "mxfp4_quant_1x32": ([P, I32, I64, I32, P, P, P], I32),
        "mxfp4_dequant_1x32": ([P, P, I64, I32, P, I32, P], I32),
        "fp8_dequant_1x128": ([P, P, I64, I32, P, I32, P], I32),
        "grouped_gemm_mxfp4": ([P, P, I64, P, P, I32, I64, P, P, I32, I32, I32, P, P, P, P], I32),
        "moe_balance_loss_workspace_bytes": ([I64, I32], SZ),
        "moe_balance_loss": ([P, P, P, I32, I64, I32, I32, F32, P, P, P, P, SZ, P], I32),
        "moe_balance_loss_backward": ([P, P, P, I32, I64, I32, I32, F32, P, P, P, P], I32),
        "moe_router_logits_backward_workspace_bytes": ([I64, I32, I32], SZ),
        "moe_router_logits_backward": ([P, P, P, I64, I32, I32, P, P, P, P, P, SZ, P], I32),
        "grouped_gemm_fp8_swiglu_zq": ([P, P, P, P, I32, I64, P, P, I32, I32, P, P, P, P, P, SZ, P], I32),
        "moe_swiglu_backward_zq": ([P, P, P, I64, I32, P, P, P], I32),
        "moe_wgrad_operands_zq": ([P, P, P, P, P, P, P, P, P, P, I32, I32, I64, I32, I32, I32, I64,
                                   P, P, P, P, P, P, P, P, P], I32),
        "moe_add_layernorm": ([P, I32, P, I32, P, P, I32, I64, I32, F32, P, P, P, P, P, P, P], I32),
        "moe_add_layernorm_backward_workspace_bytes": ([I64, I32], SZ),
        "moe_add_layernorm_backward": ([P, I32, P, I32, P, I32, P, P, P, I64, I32, P, I32, P, P, P, SZ, P], I32),
        "moe_wgrad": ([P, I32, I32, I32, I32, P, P, P, P, P, P, P, P, P, P, P, SZ, P], I32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(status: int, name: str):
    if status != 0:
        L = load_library()
        raise MoEError(f"{name}: {L.moe_status_string(status).decode()} ({status}): "
                       f"{L.moe_last_error().decode()}")


try:                                # the current stream's handle without a Stream object around it
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
except ImportError:                 # a torch built without GPU support: every call refuses its tensors first
    def _raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise MoEError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise MoEError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _want(t, dtype, shape, name):
    if t.dtype != dtype:
        raise MoEError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise MoEError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _new(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


# ---------------------------------------------------------------- router
def moe_router_topk(u, centroids, bias, K, scores=None, topk_idx=None, topk_gate=None,
                    n_groups=1, topk_groups=1):
    """u bf16 [T,d], centroids bf16 [E,d], bias f32 [E] -> (idx i32 [T,K], gate f32 [T,K], scores f32 [T,E]).
    n_groups > 1 calls the group-limited variant (moe_router_topk_grouped)."""
    T, d = u.shape
    E = centroids.shape[0]
    _want(u, torch.bfloat16, (T, d), "u")
    _want(centroids, torch.bfloat16, (E, d), "centroids")
    _want(bias, torch.float32, (E,), "bias")
    scores = _new((T, E), torch.float32, u) if scores is None else scores
    topk_idx = _new((T, K), torch.int32, u) if topk_idx is None else topk_idx
    topk_gate = _new((T, K), torch.float32, u) if topk_gate is None else topk_gate
    _want(scores, torch.float32, (T, E), "scores")
    _want(topk_idx, torch.int32, (T, K), "topk_idx")
    _want(topk_gate, torch.float32, (T, K), "topk_gate")
    L = load_library()
    if n_groups == 1:
        _check(L.moe_router_topk(_ptr(u), _ptr(centroids), _ptr(bias), T, d, E, K, _ptr(scores),
                                 _ptr(topk_idx), _ptr(topk_gate), _stream()), "moe_router_topk")
    else:
        _check(L.moe_router_topk_grouped(_ptr(u), _ptr(centroids), _ptr(bias), T, d, E, K, n_groups,
                                         topk_groups, _ptr(scores), _ptr(topk_idx), _ptr(topk_gate),
                                         _stream()), "moe_router_topk_grouped")
    return topk_idx, topk_gate, scores


def moe_seq_balance_loss(scores, topk_idx, seq_len, alpha, ws=None):
    """Per-sequence balance loss (f32 [T/seq_len]) from the router's scores
    f32 [T,E] and topk_idx i32 [T,K]."""
    T, E = scores.shape
    K = topk_idx.shape[1]
    _want(scores, torch.float32, (T, E), "scores")
    _want(topk_idx, torch.int32, (T, K), "topk_idx")
    if seq_len < 1 or T % seq_len:
        raise MoEError("moe_seq_balance_loss: T must be a multiple of seq_len")
    loss = _new((T // seq_len,), torch.float32, scores)
    L = load_library()
    if ws is None:
        ws = _new((max(L.moe_seq_balance_loss_workspace_bytes(T, seq_len), 256),), torch.uint8, scores)
    _check(L.moe_seq_balance_loss(_ptr(scores), _ptr(topk_idx), T, E, K, seq_len, alpha, _ptr(loss),
                                  _ptr(ws), ws.numel(), _stream()), "moe_seq_balance_loss")
    return loss


# ---------------------------------------------------------------- dispatch
def moe_dispatch_workspace_bytes(T, E):
    return load_library().moe_dispatch_workspace_bytes(T, E)


def moe_dispatch(topk_idx, E, include_shared=True, ws=None):
    """-> (expert_count [E], group_offset [E+1(+1)], row_token [R], slot_row [T,K]), int32."""
    T, K = topk_idx.shape
    _want(topk_idx, torch.int32, (T, K), "topk_idx")
    sh = 1 if include_shared else 0
    R = T * K + sh * T
    count = _new((E,), torch.int32, topk_idx)
    go = _new((E + 1 + sh,), torch.int32, topk_idx)
    row_token = _new((max(R, 1),), torch.int32, topk_idx)
    slot_row = _new((T, K), torch.int32, topk_idx)
    L = load_library()
    nb = L.moe_dispatch_workspace_bytes(T, E)
    if ws is None:
        ws = _new((max(nb, 256),), torch.uint8, topk_idx)
    _check(L.moe_dispatch(_ptr(topk_idx), T, K, E, sh, _ptr(count), _ptr(go), _ptr(row_token),
                          _ptr(slot_row), _ptr(ws), ws.numel(), _stream()), "moe_dispatch")
    return count, go, row_token[:R], slot_row


MOE_CHECK_BITS = {
    "count_sum": 1 << 0, "offsets_not_monotone": 1 << 1, "first_offset": 1 << 2, "count_ne_offsets": 1 << 3,
    "routed_total": 1 << 4, "shared_group": 1 << 5, "negative_count": 1 << 6, "slot_row": 1 << 7,
    "shared_rows": 1 << 8,
}


def moe_dispatch_check(expert_count, group_offset, T, K, topk_idx=None, row_token=None, slot_row=None):
    """The debug status word of a dispatch result: a uint32 bitmask
    (MOE_CHECK_BITS) left on the device in an int32 [1] tensor; 0 = every
    invariant holds."""
    E = expert_count.numel()
    sh = group_offset.numel() - E - 1
    if sh not in (0, 1):
        raise MoEError("group_offset must hold E+1 or E+2 entries")
    _want(expert_count, torch.int32, (E,), "expert_count")
    _want(group_offset, torch.int32, (E + 1 + sh,), "group_offset")
    if topk_idx is not None:
        _want(topk_idx, torch.int32, (T, K), "topk_idx")
        _want(slot_row, torch.int32, (T, K), "slot_row")
        if row_token.dtype != torch.int32 or row_token.numel() < T * K + sh * T:
            raise MoEError("row_token: int32 with T*K (+T) entries expected")
    status = _new((1,), torch.int32, expert_count)
    L = load_library()
    _check(L.moe_dispatch_check(_ptr(expert_count), _ptr(group_offset), _ptr(topk_idx), _ptr(row_token),
                                _ptr(slot_row), T, K, E, sh, _ptr(status), _stream()), "moe_dispatch_check")
    return status


def moe_permute_rows(x, row_token, out=None):
    rows = row_token.shape[0]
    T, d = x.shape
    dt = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}[x.dtype]
    out = _new((rows, d), x.dtype, x) if out is None else out
    _want(out, x.dtype, (rows, d), "out")
    L = load_library()
    _check(L.moe_permute_rows(_ptr(x), dt, _ptr(row_token), rows, d, _ptr(out), _stream()),
           "moe_permute_rows")
    return out


# ---------------------------------------------------------------- quantisers
def fp8_quant_1x128(x, q=None, scale=None):
    """x bf16/f32 [rows, cols] -> (q uint8 [rows, cols], scale f32 [rows, cols/128])."""
    rows, cols = x.shape
    dt = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}[x.dtype]
    q = _new((rows, cols), torch.uint8, x) if q is None else q
    scale = _new((rows, cols // 128), torch.float32, x) if scale is None else scale
    _want(q, torch.uint8, (rows, cols), "q")
    _want(scale, torch.float32, (rows, cols // 128), "scale")
    L = load_library()
    _check(L.fp8_quant_1x128(_ptr(x), dt, rows, cols, _ptr(q), _ptr(scale), _stream()),
           "fp8_quant_1x128")
    return q, scale


def fp8_quant_128x128(w, q=None, scale=None):
    rows, cols = w.shape
    _want(w, torch.float32, (rows, cols), "w")
    q = _new((rows, cols), torch.uint8, w) if q is None else q
    scale = _new((rows // 128, cols // 128), torch.float32, w) if scale is None else scale
    L = load_library()
    _check(L.fp8_quant_128x128(_ptr(w), rows, cols, _ptr(q), _ptr(scale), _stream()),
           "fp8_quant_128x128")
    return q, scale


# ---------------------------------------------------------------- grouped GEMM
def moe_gemm_workspace_bytes(G, M_total, N, K):
    return load_library().moe_gemm_workspace_bytes(G, M_total, N, K)


def grouped_gemm_fp8_blockscaled(a_q, a_scale, group_offset, M_total, b_q, b_scale,
                                 epi=MOE_EPI_STORE_F32, a_row_index=None, out=None, out_q=None,
                                 out_scale=None, ws=None):
    """a_q uint8 [*,K], a_scale f32 [*,K/128], group_offset i32 [G+1] (device),
    b_q uint8 [G,N,K], b_scale f32 [G,N/128,K/128]."""
    return _grouped_gemm(a_q, a_scale, group_offset, M_total, b_q, b_scale, epi, a_row_index, out, out_q,
                         out_scale, ws, noalloc=False)


def grouped_gemm_fp8_blockscaled_noalloc(a_q, a_scale, group_offset, M_total, b_q, b_scale,
                                         epi=MOE_EPI_STORE_F32, a_row_index=None, out=None, out_q=None,
                                         out_scale=None):
    """As grouped_gemm_fp8_blockscaled, through the C entry point that takes no
    workspace (its scratch is the library's static device array; the C call
    allocates nothing -- pass preallocated outputs to keep this binding from
    allocating them)."""
    return _grouped_gemm(a_q, a_scale, group_offset, M_total, b_q, b_scale, epi, a_row_index, out, out_q,
                         out_scale, None, noalloc=True)


def _grouped_gemm(a_q, a_scale, group_offset, M_total, b_q, b_scale, epi, a_row_index, out, out_q, out_scale,
                  ws, noalloc):
    G, N, K = b_q.shape
    if b_q.dtype != torch.uint8:
        raise MoEError(f"b_q: dtype {b_q.dtype}, expected torch.uint8")
    _want(b_scale, torch.float32, (G, N // 128, K // 128), "b_scale")
    if a_q.dim() != 2 or a_q.dtype != torch.uint8 or a_q.shape[1] != K:
        raise MoEError(f"a_q: {a_q.dtype} {tuple(a_q.shape)}, expected torch.uint8 [*, {K}]")
    _want(a_scale, torch.float32, (a_q.shape[0], K // 128), "a_scale")
    if group_offset.dtype != torch.int32 or group_offset.numel() < G + 1:
        raise MoEError("group_offset must be int32 with G+1 entries")
    # the rows each GEMM row reads: a gather through a_row_index, else row m
    # itself (the index values cannot be checked without reading them back)
    if a_row_index is None:
        if a_q.shape[0] < M_total:
            raise MoEError(f"a_q holds {a_q.shape[0]} rows, fewer than M_total = {M_total}")
    elif a_row_index.dtype != torch.int32 or a_row_index.numel() < M_total:
        raise MoEError(f"a_row_index: {a_row_index.dtype} with {a_row_index.numel()} entries, "
                       f"expected int32 with at least M_total = {M_total}")
    if epi == MOE_EPI_STORE_F32:
        out = _new((M_total, N), torch.float32, a_q) if out is None else out
        _want(out, torch.float32, (M_total, N), "out")
    elif epi == MOE_EPI_SWIGLU_F32:
        out = _new((M_total, N // 2), torch.float32, a_q) if out is None else out
        _want(out, torch.float32, (M_total, N // 2), "out")
    else:
        out_q = _new((M_total, N // 2), torch.uint8, a_q) if out_q is None else out_q
        out_scale = _new((M_total, N // 256), torch.float32, a_q) if out_scale is None else out_scale
        _want(out_q, torch.uint8, (M_total, N // 2), "out_q")
        _want(out_scale, torch.float32, (M_total, N // 256), "out_scale")
        if epi == MOE_EPI_SWIGLU_QUANT_Z:
            out = _new((M_total, N), torch.float32, a_q) if out is None else out
            _want(out, torch.float32, (M_total, N), "out")
        elif out is not None:
            _want(out, torch.float32, (M_total, N // 2), "out")
    L = load_library()
    if noalloc:
        _check(L.grouped_gemm_fp8_blockscaled_noalloc(
            _ptr(a_q), _ptr(a_scale), _ptr(a_row_index), _ptr(group_offset), G, M_total, _ptr(b_q),
            _ptr(b_scale), N, K, epi, _ptr(out), _ptr(out_q), _ptr(out_scale), _stream()),
            "grouped_gemm_fp8_blockscaled_noalloc")
    else:
        if ws is not None and ws.numel() < L.moe_gemm_workspace_bytes(G, M_total, N, K):
            raise MoEError("ws: smaller than moe_gemm_workspace_bytes")
        if ws is None:
            ws = _new((max(L.moe_gemm_workspace_bytes(G, M_total, N, K), 256),), torch.uint8, a_q)
        _check(L.grouped_gemm_fp8_blockscaled(
            _ptr(a_q), _ptr(a_scale), _ptr(a_row_index), _ptr(group_offset), G, M_total, _ptr(b_q),
            _ptr(b_scale), N, K, epi, _ptr(out), _ptr(out_q), _ptr(out_scale), _ptr(ws), ws.numel(),
            _stream()), "grouped_gemm_fp8_blockscaled")
    if epi == MOE_EPI_SWIGLU_QUANT:
        return out_q, out_scale
    if epi == MOE_EPI_SWIGLU_QUANT_Z:
        return out_q, out_scale, out
    return out


def moe_fp8_mfma_accumulation_probe(a_q, b_q, chained):
    """sum_k E4M3(a_q[m,k]) * E4M3(b_q[n,k]) with unit scales, FP32 [M, N]:
    chained=True carries one accumulator through the FP8 MFMA of every slice,
    chained=False adds each slice's MFMA result in FP32 (the GEMM's path)."""
    M, K = a_q.shape
    N = b_q.shape[0]
    _want(a_q, torch.uint8, (M, K), "a_q")
    _want(b_q, torch.uint8, (N, K), "b_q")
    out = _new((M, N), torch.float32, a_q)
    L = load_library()
    _check(L.moe_fp8_mfma_accumulation_probe(_ptr(a_q), _ptr(b_q), M, N, K, int(bool(chained)),
                                             _ptr(out), _stream()), "moe_fp8_mfma_accumulation_probe")
    return out


# ---------------------------------------------------------------- combine / bias
def moe_combine(u, y, topk_gate, slot_row, shared_row0=-1, out=None):
    T, d = u.shape
    K = topk_gate.shape[1]
    _want(u, torch.bfloat16, (T, d), "u")
    _want(topk_gate, torch.float32, (T, K), "topk_gate")
    _want(slot_row, torch.int32, (T, K), "slot_row")
    if y.dtype not in (torch.bfloat16, torch.float32) or y.dim() != 2 or y.shape[1] != d:
        raise MoEError(f"y: {y.dtype} {tuple(y.shape)}, expected bf16 or f32 [rows, {d}]")
    # rows read: shared_row0 + t for every token (the slot rows' values cannot
    # be checked without reading them back)
    if T > 0 and shared_row0 >= 0 and y.shape[0] < shared_row0 + T:
        raise MoEError(f"y holds {y.shape[0]} rows; the shared rows need {shared_row0 + T}")
    dt = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}[y.dtype]
    out = _new((T, d), torch.float32, u) if out is None else out
    _want(out, torch.float32, (T, d), "out")
    L = load_library()
    _check(L.moe_combine(_ptr(u), _ptr(y), dt, shared_row0, _ptr(topk_gate), _ptr(slot_row), T, K,
                         d, _ptr(out), _stream()), "moe_combine")
    return out


def moe_bias_update(bias, expert_count, total_assignments, gamma):
    """In-place update of bias (f32 [E]) from expert_count (i32 [E])."""
    E = bias.shape[0]
    _want(bias, torch.float32, (E,), "bias")
    _want(expert_count, torch.int32, (E,), "expert_count")
    L = load_library()
    _check(L.moe_bias_update(_ptr(bias), _ptr(expert_count), E, total_assignments, gamma, _stream()),
           "moe_bias_update")
    return bias


# ---------------------------------------------------------------- weights / layer
def moe_packed_weight_bytes(n_groups, d, I):
    return load_library().moe_packed_weight_bytes(n_groups, d, I)


def moe_prepare_expert_weights(w1, w3, w2, expert_index, n_groups, packed):
    I, d = w1.shape
    _want(w1, torch.float32, (I, d), "w1")
    _want(w3, torch.float32, (I, d), "w3")
    _want(w2, torch.float32, (d, I), "w2")
    L = load_library()
    _check(L.moe_prepare_expert_weights(_ptr(w1), _ptr(w3), _ptr(w2), expert_index, n_groups, d, I,
                                        _ptr(packed), _stream()), "moe_prepare_expert_weights")
    return packed


def packed_views(packed, n_groups, d, I):
    """Views of the packed weight buffer: (w13_q [G,2I,d], w2_q [G,d,I],
    w13_s [G,2I/128,d/128], w2_s [G,d/128,I/128]) -- the layout the header
    documents (each part starts on a 256-byte boundary)."""
    def al(x):
        return (x + 255) // 256 * 256
    G = n_groups
    o0 = 0
    o1 = o0 + al(G * 2 * I * d)
    o2 = o1 + al(G * d * I)
    o3 = o2 + al(G * (2 * I // 128) * (d // 128) * 4)
    w13q = packed[o0:o0 + G * 2 * I * d].view(G, 2 * I, d)
    w2q = packed[o1:o1 + G * d * I].view(G, d, I)
    w13s = packed[o2:o2 + G * (2 * I // 128) * (d // 128) * 4].view(torch.float32).view(G, 2 * I // 128, d // 128)
    w2s = packed[o3:o3 + G * (d // 128) * (I // 128) * 4].view(torch.float32).view(G, d // 128, I // 128)
    return w13q, w2q, w13s, w2s


def moe_layer_workspace_bytes(T, d, E, K, I):
    return load_library().moe_layer_workspace_bytes(T, d, E, K, I)


def moe_layer_forward(u, centroids, bias, packed, K, I, out=None, expert_count=None, ws=None):
    T, d = u.shape
    E = centroids.shape[0]
    _want(u, torch.bfloat16, (T, d), "u")
    _want(centroids, torch.bfloat16, (E, d), "centroids")
    _want(bias, torch.float32, (E,), "bias")
    L = load_library()
    need = L.moe_packed_weight_bytes(E + 1, d, I)
    if packed.dtype != torch.uint8 or packed.numel() < need:
        raise MoEError(f"packed weights: need {need} bytes of uint8")
    out = _new((T, d), torch.float32, u) if out is None else out
    if ws is None:
        ws = _new((max(L.moe_layer_workspace_bytes(T, d, E, K, I), 256),), torch.uint8, u)
    _check(L.moe_layer_forward(_ptr(u), _ptr(centroids), _ptr(bias), _ptr(packed), T, d, E, K, I,
                               _ptr(out), _ptr(expert_count), _ptr(ws), ws.numel(), _stream()),
           "moe_layer_forward")
    return out


# ---------------------------------------------------------------- backward (input gradient)
def moe_prepare_backward_weights(packed, n_groups, d, I, packed_t=None):
    """The packed weights transposed block by block (W13^T [G,d,2I], W2^T [G,I,d])."""
    L = load_library()
    need = L.moe_packed_weight_bytes(n_groups, d, I)
    packed_t = _new((need,), torch.uint8, packed) if packed_t is None else packed_t
    _check(L.moe_prepare_backward_weights(_ptr(packed), n_groups, d, I, _ptr(packed_t), _stream()),
           "moe_prepare_backward_weights")
    return packed_t


def moe_gate_backward(dh, y, topk_gate, slot_row, scores, topk_idx, shared_row0=-1):
    """-> (dy_q u8 [R,d], dy_scale f32 [R,d/128], dlogit f32 [T,K], row_dlogit f32 [R])."""
    T, d = dh.shape
    K = topk_gate.shape[1]
    E = scores.shape[1]
    R = y.shape[0]
    _want(dh, torch.float32, (T, d), "dh")
    _want(y, torch.float32, (R, d), "y")
    _want(topk_gate, torch.float32, (T, K), "topk_gate")
    _want(slot_row, torch.int32, (T, K), "slot_row")
    _want(scores, torch.float32, (T, E), "scores")
    _want(topk_idx, torch.int32, (T, K), "topk_idx")
    dy_q = _new((R, d), torch.uint8, dh)
    dy_s = _new((R, d // 128), torch.float32, dh)
    dlogit = _new((T, K), torch.float32, dh)
    row_dlogit = torch.zeros((R,), dtype=torch.float32, device=dh.device)
    L = load_library()
    _check(L.moe_gate_backward(_ptr(dh), _ptr(y), shared_row0, _ptr(topk_gate), _ptr(slot_row), _ptr(scores),
                               _ptr(topk_idx), T, K, d, E, _ptr(dy_q), _ptr(dy_s), _ptr(dlogit),
                               _ptr(row_dlogit), _stream()), "moe_gate_backward")
    return dy_q, dy_s, dlogit, row_dlogit


def moe_swiglu_backward(z, dh_row):
    """z f32 [R,2I] (interleaved gate/up), dh_row f32 [R,I] -> (dz_q u8 [R,2I], dz_scale f32 [R,2I/128])."""
    R, I2 = z.shape
    I = I2 // 2
    _want(z, torch.float32, (R, 2 * I), "z")
    _want(dh_row, torch.float32, (R, I), "dh_row")
    dz_q = _new((R, 2 * I), torch.uint8, z)
    dz_s = _new((R, 2 * I // 128), torch.float32, z)
    L = load_library()
    _check(L.moe_swiglu_backward(_ptr(z), _ptr(dh_row), R, I, _ptr(dz_q), _ptr(dz_s), _stream()),
           "moe_swiglu_backward")
    return dz_q, dz_s


def moe_router_backward(dh, dx, slot_row, dlogit, topk_idx, centroids, u, row_dlogit, row_token,
                        group_offset, shared_row0=-1):
    """-> (du f32 [T,d], de f32 [E,d])."""
    T, d = dh.shape
    K = slot_row.shape[1]
    E = centroids.shape[0]
    _want(u, torch.bfloat16, (T, d), "u")
    _want(centroids, torch.bfloat16, (E, d), "centroids")
    du = _new((T, d), torch.float32, dh)
    de = _new((E, d), torch.float32, dh)
    L = load_library()
    _check(L.moe_router_backward(_ptr(dh), _ptr(dx), shared_row0, _ptr(slot_row), _ptr(dlogit), _ptr(topk_idx),
                                 _ptr(centroids), _ptr(u), _ptr(row_dlogit), _ptr(row_token), _ptr(group_offset),
                                 T, K, d, E, _ptr(du), _ptr(de), _stream()), "moe_router_backward")
    return du, de


def moe_wgrad(dh, topk_gate, slot_row, row_token, z, dh_row, u, group_offset, shared_row0=-1):
    """Expert weight gradients -> (dW13 f32 [G, 2I, d] in W13's interleaved row
    order, dW2 f32 [G, d, I], the operand buffers, kb_start i32 [G+1] on the
    device).  moe_wgrad_block_starts places each expert's padded row blocks
    (on the device), moe_wgrad_operands builds the transposed operands, then
    moe_wgrad runs one K-grouped GEMM per weight over all experts.  Nothing is
    read back to the host: the buffers are sized by the bound
    ceil(R / 128) + G of the row-block count, so the whole chain can be
    captured in a graph."""
    return _wgrad(dh, topk_gate, slot_row, row_token, z, None, dh_row, u, group_offset, shared_row0)


def moe_wgrad_zq(dh, topk_gate, slot_row, row_token, z_q, z_scale, dh_row, u, group_offset, shared_row0=-1):
    """As moe_wgrad, from z kept in 8 bits (grouped_gemm_fp8_swiglu_zq): z_q uint8 [R, 2I], z_scale f32
    [R, 2I/128]; the operands come from moe_wgrad_operands_zq."""
    if z_q.dim() != 2:
        raise MoEError(f"z_q: shape {tuple(z_q.shape)}, expected two dimensions")
    if dh.dim() != 2 or topk_gate.dim() != 2:
        raise MoEError(f"dh: {tuple(dh.shape)}, topk_gate: {tuple(topk_gate.shape)}, expected [T, d] and [T, K]")
    (R, I2), (T, d), K = z_q.shape, dh.shape, topk_gate.shape[1]
    dev = _current(z_q, "z_q")
    for t, dtype, shape, name in (
            (z_q, torch.uint8, (R, I2), "z_q"), (z_scale, torch.float32, (R, I2 // 128), "z_scale"),
            (dh_row, torch.float32, (R, I2 // 2), "dh_row"), (dh, torch.float32, (T, d), "dh"),
            (u, torch.bfloat16, (T, d), "u"), (topk_gate, torch.float32, (T, K), "topk_gate"),
            (slot_row, torch.int32, (T, K), "slot_row"), (row_token, torch.int32, (R,), "row_token"),
            (group_offset, torch.int32, group_offset.shape, "group_offset")):
        _in(t, dtype, shape, name, dev)
    return _wgrad(dh, topk_gate, slot_row, row_token, z_q, z_scale, dh_row, u, group_offset, shared_row0)


def _wgrad(dh, topk_gate, slot_row, row_token, z, z_scale, dh_row, u, group_offset, shared_row0):
    T, d = dh.shape
    K = topk_gate.shape[1]
    R, I2 = z.shape
    I = I2 // 2
    G = group_offset.numel() - 1
    _want(group_offset, torch.int32, (G + 1,), "group_offset")
    n_kb = (R + 127) // 128 + G
    dev = dh.device
    cs_h, cs_x = (I // 128 + 3) // 4 * 4, (d // 128 + 3) // 4 * 4
    bufs = dict(
        dyT_q=torch.empty(max(d * 128 * n_kb, 16), dtype=torch.uint8, device=dev),
        dyT_s=torch.empty(max(d * n_kb, 4), dtype=torch.float32, device=dev),
        hT_q=torch.empty(max(I * 128 * n_kb, 16), dtype=torch.uint8, device=dev),
        hT_s=torch.empty(max(cs_h * n_kb, 4), dtype=torch.float32, device=dev),
        dzT_q=torch.empty(max(2 * I * 128 * n_kb, 16), dtype=torch.uint8, device=dev),
        dzT_s=torch.empty(max(2 * I * n_kb, 4), dtype=torch.float32, device=dev),
        xT_q=torch.empty(max(d * 128 * n_kb, 16), dtype=torch.uint8, device=dev),
        xT_s=torch.empty(max(cs_x * n_kb, 4), dtype=torch.float32, device=dev))
    L = load_library()
    kbs = torch.empty(G + 1, dtype=torch.int32, device=dev)
    _check(L.moe_wgrad_block_starts(_ptr(group_offset), G, _ptr(kbs), _stream()), "moe_wgrad_block_starts")
    name = "moe_wgrad_operands" if z_scale is None else "moe_wgrad_operands_zq"
    zs = (z,) if z_scale is None else (z, z_scale)
    _check(getattr(L, name)(*(_ptr(t) for t in (dh, topk_gate, slot_row, row_token, *zs, dh_row, u, group_offset, kbs)),
                            G, n_kb, T, K, d, I, shared_row0,
                            *(_ptr(bufs[k]) for k in ("dyT_q", "dyT_s", "hT_q", "hT_s", "dzT_q", "dzT_s",
                                                       "xT_q", "xT_s")), _stream()), name)
    dw13 = _new((G, 2 * I, d), torch.float32, dh)
    dw2 = _new((G, d, I), torch.float32, dh)
    ws = _new((max(L.moe_wgrad_workspace_bytes(G, d, I), 256),), torch.uint8, dh)
    _check(L.moe_wgrad(_ptr(kbs), G, n_kb, d, I,
                       *(_ptr(bufs[k]) for k in ("dyT_q", "dyT_s", "hT_q", "hT_s", "dzT_q", "dzT_s", "xT_q", "xT_s")),
                       _ptr(dw13), _ptr(dw2), _ptr(ws), ws.numel(), _stream()), "moe_wgrad")
    return dw13, dw2, bufs, kbs


# ---------------------------------------------------------------- residual + RMS norm
# The calls from here on are also made for single tokens, where the host's time
# is most of theirs: their checks pass over each tensor once (_in) and raise
# through _refuse, which finds out what was wrong.
RMSNorm = namedtuple("RMSNorm", "y h rstd q scale")
_INT_MAX = 2 ** 31 - 1              # ctypes hands a larger C int over modulo 2^32


def _too_large(name, n):
    raise MoEError(f"{name}: {n} is past a C int")


def _refuse(t, dtype, shape, name, dev):
    _want(t, dtype, shape, name)
    if not t.is_cuda:
        raise MoEError(f"{name}: tensor must live on the GPU")
    if t.get_device() != dev or dev != torch.cuda.current_device():
        raise MoEError(f"{name}: tensor on {t.device}, expected the current GPU, cuda:{torch.cuda.current_device()}, "
                       "for every tensor of a call")
    raise MoEError(f"{name}: tensor must be contiguous")


def _in(t, dtype, shape, name, dev):
    """The address of a tensor of this type and shape, contiguous and on GPU dev."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, dtype, shape, name, dev)
    return t.data_ptr()


def _out(t, dtype, shape, name, dev):
    """An output of this type and shape, allocated on GPU dev where t is None, and its address."""
    if t is None:
        t = torch.empty(*shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _in(t, dtype, shape, name, dev)


def _rows(t, name):
    """(rows, cols, MOE dtype, GPU) of a bf16 or FP32 matrix on the current GPU."""
    if t.dim() != 2:
        raise MoEError(f"{name}: shape {tuple(t.shape)}, expected two dimensions")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise MoEError(f"{name}: dtype {t.dtype}, expected torch.bfloat16 or torch.float32")
    rows, cols = t.shape
    if cols > _INT_MAX:
        _too_large(f"{name}'s columns", cols)
    return rows, cols, dt, _current(t, name)


def _current(t, name):
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        _refuse(t, t.dtype, t.shape, name, dev)
    return dev


def _dt(t, name):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise MoEError(f"{name}: dtype {t.dtype}, expected torch.bfloat16 or torch.float32")
    return dt


def moe_add_rmsnorm(x, weight, eps, residual=None, quant=False, h_out=None, y=None, q=None, scale=None, rstd=None):
    """h = x + residual, y = bf16(h / sqrt(mean(h^2) + eps) * weight) and, with quant, the FP8 1x128
    codes and scales of y.  x, residual bf16/f32 [T,d], weight bf16/f32 [d]
    -> RMSNorm(y bf16 [T,d], h of residual's type [T,d] or None, rstd f32 [T], q uint8 [T,d] or None,
    scale f32 [T,d/128] or None).  h_out may be residual, or x of the same type; y may be x or residual
    where that is bf16."""
    T, d, xd, dev = _rows(x, "x")
    shape = x.shape
    px = _in(x, x.dtype, shape, "x", dev)
    wd = _dt(weight, "weight")
    pw = _in(weight, weight.dtype, (d,), "weight", dev)
    pr = ph = pq = ps = None
    rd = MOE_F32
    if residual is not None:
        rd = _dt(residual, "residual")
        pr = _in(residual, residual.dtype, shape, "residual", dev)
        h_out, ph = _out(h_out, residual.dtype, shape, "h_out", dev)
    elif h_out is not None:
        raise MoEError("moe_add_rmsnorm: h_out without a residual")
    y, py = _out(y, torch.bfloat16, shape, "y", dev)
    rstd, prs = _out(rstd, torch.float32, (T,), "rstd", dev)
    if quant:
        q, pq = _out(q, torch.uint8, shape, "q", dev)
        scale, ps = _out(scale, torch.float32, (T, d // 128), "scale", dev)
    elif q is not None or scale is not None:
        raise MoEError("moe_add_rmsnorm: q or scale without quant")
    L = _lib or load_library()
    st = L.moe_add_rmsnorm(px, xd, pr, rd, pw, wd, T, d, eps, ph, py, pq, ps, prs, _raw_stream(dev))
    if st:
        _check(st, "moe_add_rmsnorm")
    return RMSNorm(y, h_out, rstd, q, scale)


def moe_add_rmsnorm_backward(dy, h, weight, rstd, dh=None, dx=None, dw=None, dx_dtype=None, ws=None):
    """dy, h bf16/f32 [T,d], weight bf16/f32 [d], rstd f32 [T], dh (the gradient of h_out) or None
    -> (dx [T,d] of dh's type, else dx_dtype, else dy's; dw f32 [d]).  dx is the gradient of x and of
    residual alike."""
    T, d, yd, dev = _rows(dy, "dy")
    shape = dy.shape
    if dx_dtype is None:
        dx_dtype = dh.dtype if dh is not None else dx.dtype if dx is not None else dy.dtype
    dx, pdx = _out(dx, dx_dtype, shape, "dx", dev)
    dw, pdw = _out(dw, torch.float32, (d,), "dw", dev)
    L = _lib or load_library()
    if ws is None:
        ws_bytes = max(L.moe_add_rmsnorm_backward_workspace_bytes(T, d), 16)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        pws = ws.data_ptr()
    else:
        ws_bytes, pws = ws.numel() * ws.element_size(), _in(ws, ws.dtype, ws.shape, "ws", dev)
    pdh = None if dh is None else _in(dh, dx_dtype, shape, "dh", dev)
    st = L.moe_add_rmsnorm_backward(
        _in(dy, dy.dtype, shape, "dy", dev), yd, _in(h, h.dtype, shape, "h", dev), _dt(h, "h"),
        _in(weight, weight.dtype, (d,), "weight", dev), _dt(weight, "weight"),
        _in(rstd, torch.float32, (T,), "rstd", dev), pdh, T, d, pdx, _dt(dx, "dx"), pdw, pws, ws_bytes,
        _raw_stream(dev))
    if st:
        _check(st, "moe_add_rmsnorm_backward")
    return dx, dw


# ---------------------------------------------------------------- MXFP4
def mxfp4_quant_1x32(x, q=None, scale=None):
    """x bf16/f32 [rows, cols] -> (q uint8 [rows, cols/2], two E2M1 codes to a byte, the even column in
    the low half; scale uint8 [rows, cols/32], E8M0)."""
    rows, cols, dt, dev = _rows(x, "x")
    q, pq = _out(q, torch.uint8, (rows, cols // 2), "q", dev)
    scale, ps = _out(scale, torch.uint8, (rows, cols // 32), "scale", dev)
    L = _lib or load_library()
    st = L.mxfp4_quant_1x32(_in(x, x.dtype, x.shape, "x", dev), dt, rows, cols, pq, ps, _raw_stream(dev))
    if st:
        _check(st, "mxfp4_quant_1x32")
    return q, scale


def _dequant(name, q, scale, cols, scale_dtype, per, dtype, out):
    """The shared part of the dequantisers: values [rows, cols], `per` of them under each scale."""
    rows = q.shape[0]
    dev = _current(q, "q")
    if cols > _INT_MAX:
        _too_large("columns", cols)
    if dtype not in _DTYPES:
        raise MoEError(f"{name}: dtype {dtype}, expected torch.bfloat16 or torch.float32")
    out, po = _out(out, dtype, (rows, cols), "out", dev)
    L = _lib or load_library()
    st = getattr(L, name)(_in(q, torch.uint8, q.shape, "q", dev), _in(scale, scale_dtype, (rows, cols // per), "scale", dev),
                          rows, cols, po, _DTYPES[dtype], _raw_stream(dev))
    if st:
        _check(st, name)
    return out


def mxfp4_dequant_1x32(q, scale, dtype=torch.bfloat16, out=None):
    """The values of mxfp4_quant_1x32's outputs, bf16 or f32 [rows, cols]."""
    if q.dim() != 2:
        raise MoEError(f"q: shape {tuple(q.shape)}, expected two dimensions")
    return _dequant("mxfp4_dequant_1x32", q, scale, 2 * q.shape[1], torch.uint8, 32, dtype, out)


def fp8_dequant_1x128(q, scale, dtype=torch.float32, out=None):
    """The values of fp8_quant_1x128's outputs, bf16 or f32 [rows, cols]."""
    if q.dim() != 2:
        raise MoEError(f"q: shape {tuple(q.shape)}, expected two dimensions")
    return _dequant("fp8_dequant_1x128", q, scale, q.shape[1], torch.float32, 128, dtype, out)


def grouped_gemm_mxfp4(a_q, a_scale, group_offset, M_total, b_q, b_scale, epi=MOE_MX_STORE_F32, a_row_index=None,
                       out=None, out_q=None, out_scale=None):
    """a_q uint8 [*,K/2], a_scale uint8 [*,K/32], group_offset i32 [G+1] (device), b_q uint8 [G,N,K/2],
    b_scale uint8 [G,N,K/32] -> out f32 or bf16 [M_total,N], h bf16 [M_total,N/2] (MOE_MX_SWIGLU_BF16), or
    (out_q uint8 [M_total,N/4], out_scale uint8 [M_total,N/64]) (MOE_MX_SWIGLU_QUANT)."""
    if b_q.dim() != 3 or a_q.dim() != 2:
        raise MoEError(f"a_q: {tuple(a_q.shape)}, b_q: {tuple(b_q.shape)}, expected [*, K/2] and [G, N, K/2]")
    G, N, half = b_q.shape
    K = half * 2
    rows = a_q.shape[0]
    if G > _INT_MAX or N > _INT_MAX or K > _INT_MAX:
        _too_large("G, N or K", max(G, N, K))
    dev = _current(b_q, "b_q")
    pi = None
    if a_row_index is not None:
        if a_row_index.dtype is not torch.int32 or a_row_index.numel() < M_total:
            raise MoEError(f"a_row_index: {a_row_index.dtype} with {a_row_index.numel()} entries, "
                           f"expected int32 with at least M_total = {M_total}")
        pi = _in(a_row_index, torch.int32, a_row_index.shape, "a_row_index", dev)
    if group_offset.dtype is not torch.int32 or group_offset.numel() < G + 1:
        raise MoEError("group_offset must be int32 with G+1 entries")
    po = pq = ps = None
    if epi == MOE_MX_SWIGLU_QUANT:
        out_q, pq = _out(out_q, torch.uint8, (M_total, N // 4), "out_q", dev)
        out_scale, ps = _out(out_scale, torch.uint8, (M_total, N // 64), "out_scale", dev)
        if out is not None:
            raise MoEError("grouped_gemm_mxfp4: this epilogue writes out_q and out_scale, not out")
    else:
        want = torch.float32 if epi == MOE_MX_STORE_F32 else torch.bfloat16
        shape = (M_total, N // 2 if epi == MOE_MX_SWIGLU_BF16 else N)
        out, po = _out(out, want, shape, "out", dev)
        if out_q is not None or out_scale is not None:
            raise MoEError("grouped_gemm_mxfp4: this epilogue writes out, not out_q or out_scale")
    L = _lib or load_library()
    st = L.grouped_gemm_mxfp4(
        _in(a_q, torch.uint8, (rows, half), "a_q", dev), _in(a_scale, torch.uint8, (rows, K // 32), "a_scale", dev),
        rows, pi, _in(group_offset, torch.int32, group_offset.shape, "group_offset", dev), G, M_total,
        _in(b_q, torch.uint8, b_q.shape, "b_q", dev), _in(b_scale, torch.uint8, (G, N, K // 32), "b_scale", dev), N, K,
        epi, po, pq, ps, _raw_stream(dev))
    if st:
        _check(st, "grouped_gemm_mxfp4")
    return (out_q, out_scale) if epi == MOE_MX_SWIGLU_QUANT else out


# ---------------------------------------------------------------- residual + layer norm
LayerNorm = namedtuple("LayerNorm", "y h mean rstd q scale")


def moe_add_layernorm(x, weight, eps, bias=None, residual=None, quant=False, h_out=None, y=None, q=None, scale=None,
                      mean=None, rstd=None):
    """h = x + residual, y = bf16((h - mean(h)) / sqrt(var(h) + eps) * weight + bias) and, with quant, the FP8
    1x128 codes and scales of y.  x, residual bf16/f32 [T,d], weight and bias (or None) bf16/f32 [d]
    -> LayerNorm(y bf16 [T,d], h of residual's type [T,d] or None, mean f32 [T], rstd f32 [T],
    q uint8 [T,d] or None, scale f32 [T,d/128] or None).  h_out may be residual, or x of the same type; y may
    be x or residual where that is bf16."""
    T, d, xd, dev = _rows(x, "x")
    shape = x.shape
    px = _in(x, x.dtype, shape, "x", dev)
    wd = _dt(weight, "weight")
    pw = _in(weight, weight.dtype, (d,), "weight", dev)
    pb = None if bias is None else _in(bias, weight.dtype, (d,), "bias", dev)
    pr = ph = pq = ps = None
    rd = MOE_F32
    if residual is not None:
        rd = _dt(residual, "residual")
        pr = _in(residual, residual.dtype, shape, "residual", dev)
        h_out, ph = _out(h_out, residual.dtype, shape, "h_out", dev)
    elif h_out is not None:
        raise MoEError("moe_add_layernorm: h_out without a residual")
    y, py = _out(y, torch.bfloat16, shape, "y", dev)
    mean, pm = _out(mean, torch.float32, (T,), "mean", dev)
    rstd, prs = _out(rstd, torch.float32, (T,), "rstd", dev)
    if quant:
        q, pq = _out(q, torch.uint8, shape, "q", dev)
        scale, ps = _out(scale, torch.float32, (T, d // 128), "scale", dev)
    elif q is not None or scale is not None:
        raise MoEError("moe_add_layernorm: q or scale without quant")
    L = _lib or load_library()
    st = L.moe_add_layernorm(px, xd, pr, rd, pw, pb, wd, T, d, eps, ph, py, pq, ps, pm, prs, _raw_stream(dev))
    if st:
        _check(st, "moe_add_layernorm")
    return LayerNorm(y, h_out, mean, rstd, q, scale)


def moe_add_layernorm_backward(dy, h, weight, mean, rstd, dh=None, bias_grad=True, dx=None, dw=None, db=None,
                               dx_dtype=None, ws=None):
    """dy, h bf16/f32 [T,d], weight bf16/f32 [d], mean, rstd f32 [T], dh (the gradient of h_out) or None
    -> (dx [T,d] of dh's type, else dx_dtype, else dy's; dw f32 [d]; db f32 [d], None without bias_grad).
    dx is the gradient of x and of residual alike."""
    T, d, yd, dev = _rows(dy, "dy")
    shape = dy.shape
    if dx_dtype is None:
        dx_dtype = dh.dtype if dh is not None else dx.dtype if dx is not None else dy.dtype
    dx, pdx = _out(dx, dx_dtype, shape, "dx", dev)
    dw, pdw = _out(dw, torch.float32, (d,), "dw", dev)
    pdb = None
    if bias_grad:
        db, pdb = _out(db, torch.float32, (d,), "db", dev)
    elif db is not None:
        raise MoEError("moe_add_layernorm_backward: db without bias_grad")
    L = _lib or load_library()
    if ws is None:
        ws_bytes = max(L.moe_add_layernorm_backward_workspace_bytes(T, d), 16)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        pws = ws.data_ptr()
    else:
        ws_bytes, pws = ws.numel() * ws.element_size(), _in(ws, ws.dtype, ws.shape, "ws", dev)
    pdh = None if dh is None else _in(dh, dx_dtype, shape, "dh", dev)
    st = L.moe_add_layernorm_backward(
        _in(dy, dy.dtype, shape, "dy", dev), yd, _in(h, h.dtype, shape, "h", dev), _dt(h, "h"),
        _in(weight, weight.dtype, (d,), "weight", dev), _dt(weight, "weight"),
        _in(mean, torch.float32, (T,), "mean", dev), _in(rstd, torch.float32, (T,), "rstd", dev), pdh, T, d, pdx,
        _dt(dx, "dx"), pdw, pdb, pws, ws_bytes, _raw_stream(dev))
    if st:
        _check(st, "moe_add_layernorm_backward")
    return dx, dw, db


# ---------------------------------------------------------------- balance loss over packed sequences
BalanceLoss = namedtuple("BalanceLoss", "loss seq_count expert_count")


def _scratch(ws, nbytes, dev):
    """(tensor, address, bytes) of a call's scratch, allocated where one is needed and not given."""
    if ws is None and nbytes == 16:                   # the call takes none
        return None, None, 0
    if ws is None:
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
        return ws, ws.data_ptr(), max(nbytes, 16)
    return ws, _in(ws, ws.dtype, ws.shape, "ws", dev), ws.numel() * ws.element_size()


def _sequences(scores, seq_start):
    """(T, E, n_seq, address of seq_start, GPU) of a balance loss's arguments."""
    if scores.dim() != 2:
        raise MoEError(f"scores: shape {tuple(scores.shape)}, expected two dimensions")
    T, E = scores.shape
    dev = _current(scores, "scores")
    if E > _INT_MAX:
        _too_large("scores' columns", E)
    if seq_start is None:
        return T, E, 1, None, dev
    if seq_start.dim() != 1 or seq_start.numel() < 2:
        raise MoEError(f"seq_start: shape {tuple(seq_start.shape)}, expected [n_seq + 1] with a sequence at least")
    n_seq = seq_start.numel() - 1
    if n_seq > _INT_MAX:
        _too_large("sequences", n_seq)
    return T, E, n_seq, _in(seq_start, torch.int32, (n_seq + 1,), "seq_start", dev), dev


def moe_balance_loss(scores, topk_idx, alpha, seq_start=None, loss=None, seq_count=None, expert_count=None, ws=None):
    """The balance loss of each of the sequences [seq_start[q], seq_start[q+1]) of a packed batch, and the
    experts' counts.  scores f32 [T,E], topk_idx i32 [T,K], seq_start i32 [n_seq+1] on the device (None: one
    sequence of all T tokens) -> BalanceLoss(loss f32 [n_seq], seq_count i32 [n_seq,E], expert_count i32 [E])."""
    T, E, n_seq, pstart, dev = _sequences(scores, seq_start)
    if topk_idx.dim() != 2:
        raise MoEError(f"topk_idx: shape {tuple(topk_idx.shape)}, expected two dimensions")
    K = topk_idx.shape[1]
    if K > _INT_MAX:
        _too_large("topk_idx's columns", K)
    loss, pl = _out(loss, torch.float32, (n_seq,), "loss", dev)
    seq_count, pc = _out(seq_count, torch.int32, (n_seq, E), "seq_count", dev)
    expert_count, pe = _out(expert_count, torch.int32, (E,), "expert_count", dev)
    L = _lib or load_library()
    ws, pws, ws_bytes = _scratch(ws, L.moe_balance_loss_workspace_bytes(T, n_seq), dev)
    st = L.moe_balance_loss(_in(scores, torch.float32, (T, E), "scores", dev), _in(topk_idx, torch.int32, (T, K), "topk_idx", dev),
                            pstart, n_seq, T, E, K, alpha, pl, pc, pe, pws, ws_bytes, _raw_stream(dev))
    if st:
        _check(st, "moe_balance_loss")
    return BalanceLoss(loss, seq_count, expert_count)


def moe_balance_loss_backward(scores, seq_count, K, alpha, seq_start=None, dloss=None, dlogits_in=None, dlogits=None):
    """The balance loss's gradient with respect to the router's logits, f32 [T,E], added to dlogits_in (None:
    zeros; may be dlogits itself).  seq_count as moe_balance_loss gave it, dloss f32 [n_seq] the gradient of
    each sequence's loss (None: ones)."""
    T, E, n_seq, pstart, dev = _sequences(scores, seq_start)
    if not 0 < K <= _INT_MAX:
        raise MoEError(f"moe_balance_loss_backward: K={K}")
    pd = None if dloss is None else _in(dloss, torch.float32, (n_seq,), "dloss", dev)
    pi = None if dlogits_in is None else _in(dlogits_in, torch.float32, (T, E), "dlogits_in", dev)
    dlogits, po = _out(dlogits, torch.float32, (T, E), "dlogits", dev)
    L = _lib or load_library()
    st = L.moe_balance_loss_backward(_in(scores, torch.float32, (T, E), "scores", dev),
                                     _in(seq_count, torch.int32, (n_seq, E), "seq_count", dev), pstart, n_seq, T, E, K,
                                     alpha, pd, pi, po, _raw_stream(dev))
    if st:
        _check(st, "moe_balance_loss_backward")
    return dlogits


def moe_router_logits_backward(dlogits, u, centroids, du_in=None, de_in=None, du=None, de=None, want_du=True,
                               want_de=True, ws=None):
    """dlogits f32 [T,E], u bf16 [T,d], centroids bf16 [E,d] -> (du f32 [T,d] = du_in + dlogits . centroids,
    de f32 [E,d] = de_in + dlogits^T . u); du may be du_in and de de_in.  None in the place of one that is not
    wanted."""
    if dlogits.dim() != 2 or u.dim() != 2:
        raise MoEError(f"dlogits: {tuple(dlogits.shape)}, u: {tuple(u.shape)}, expected [T, E] and [T, d]")
    T, E = dlogits.shape
    d = u.shape[1]
    if E > _INT_MAX or d > _INT_MAX:
        _too_large("E or d", max(E, d))
    dev = _current(dlogits, "dlogits")
    pdu = pde = None
    if want_du:
        du, pdu = _out(du, torch.float32, (T, d), "du", dev)
    elif du is not None or du_in is not None:
        raise MoEError("moe_router_logits_backward: du or du_in without want_du")
    L = _lib or load_library()
    if want_de:
        de, pde = _out(de, torch.float32, (E, d), "de", dev)
    elif de is not None or de_in is not None:
        raise MoEError("moe_router_logits_backward: de or de_in without want_de")
    ws, pws, ws_bytes = _scratch(ws, L.moe_router_logits_backward_workspace_bytes(T, d, E), dev)
    pui = None if du_in is None else _in(du_in, torch.float32, (T, d), "du_in", dev)
    pei = None if de_in is None else _in(de_in, torch.float32, (E, d), "de_in", dev)
    st = L.moe_router_logits_backward(_in(dlogits, torch.float32, (T, E), "dlogits", dev),
                                      _in(u, torch.bfloat16, (T, d), "u", dev),
                                      _in(centroids, torch.bfloat16, (E, d), "centroids", dev), T, d, E, pui, pei, pdu, pde,
                                      pws, ws_bytes, _raw_stream(dev))
    if st:
        _check(st, "moe_router_logits_backward")
    return (du if want_du else None), (de if want_de else None)


# ---------------------------------------------------------------- activations kept in 8 bits
def grouped_gemm_fp8_swiglu_zq(a_q, a_scale, group_offset, M_total, b_q, b_scale, a_row_index=None, h_q=None,
                               h_scale=None, z_q=None, z_scale=None, ws=None):
    """grouped_gemm_fp8_blockscaled with MOE_EPI_SWIGLU_QUANT that keeps z in 8 bits
    -> (h_q uint8 [M_total,N/2], h_scale f32 [M_total,N/256], z_q uint8 [M_total,N], z_scale f32 [M_total,N/128])."""
    if b_q.dim() != 3 or a_q.dim() != 2:
        raise MoEError(f"a_q: {tuple(a_q.shape)}, b_q: {tuple(b_q.shape)}, expected [*, K] and [G, N, K]")
    G, N, K = b_q.shape
    rows = a_q.shape[0]
    if G > _INT_MAX or N > _INT_MAX or K > _INT_MAX:
        _too_large("G, N or K", max(G, N, K))
    dev = _current(b_q, "b_q")
    pi = None
    if a_row_index is not None:
        if a_row_index.dtype is not torch.int32 or a_row_index.numel() < M_total:
            raise MoEError(f"a_row_index: {a_row_index.dtype} with {a_row_index.numel()} entries, "
                           f"expected int32 with at least M_total = {M_total}")
        pi = _in(a_row_index, torch.int32, a_row_index.shape, "a_row_index", dev)
    elif rows < M_total:
        raise MoEError(f"a_q holds {rows} rows, fewer than M_total = {M_total}")
    if group_offset.dtype is not torch.int32 or group_offset.numel() < G + 1:
        raise MoEError("group_offset must be int32 with G+1 entries")
    h_q, phq = _out(h_q, torch.uint8, (M_total, N // 2), "h_q", dev)
    h_scale, phs = _out(h_scale, torch.float32, (M_total, N // 256), "h_scale", dev)
    z_q, pzq = _out(z_q, torch.uint8, (M_total, N), "z_q", dev)
    z_scale, pzs = _out(z_scale, torch.float32, (M_total, N // 128), "z_scale", dev)
    L = _lib or load_library()
    ws, pws, ws_bytes = _scratch(ws, L.moe_gemm_workspace_bytes(G, M_total, N, K), dev)
    st = L.grouped_gemm_fp8_swiglu_zq(
        _in(a_q, torch.uint8, (rows, K), "a_q", dev), _in(a_scale, torch.float32, (rows, K // 128), "a_scale", dev), pi,
        _in(group_offset, torch.int32, group_offset.shape, "group_offset", dev), G, M_total,
        _in(b_q, torch.uint8, b_q.shape, "b_q", dev), _in(b_scale, torch.float32, (G, N // 128, K // 128), "b_scale", dev),
        N, K, phq, phs, pzq, pzs, pws, ws_bytes, _raw_stream(dev))
    if st:
        _check(st, "grouped_gemm_fp8_swiglu_zq")
    return h_q, h_scale, z_q, z_scale


def moe_swiglu_backward_zq(z_q, z_scale, dh_row, dz_q=None, dz_scale=None):
    """moe_swiglu_backward from z kept in 8 bits: z_q uint8 [R,2I], z_scale f32 [R,2I/128], dh_row f32 [R,I]
    -> (dz_q uint8 [R,2I], dz_scale f32 [R,2I/128]), which may be z_q and z_scale themselves."""
    if z_q.dim() != 2:
        raise MoEError(f"z_q: shape {tuple(z_q.shape)}, expected two dimensions")
    R, I2 = z_q.shape
    if I2 > _INT_MAX:
        _too_large("z_q's columns", I2)
    dev = _current(z_q, "z_q")
    dz_q, pq = _out(dz_q, torch.uint8, (R, I2), "dz_q", dev)
    dz_scale, ps = _out(dz_scale, torch.float32, (R, I2 // 128), "dz_scale", dev)
    L = _lib or load_library()
    st = L.moe_swiglu_backward_zq(_in(z_q, torch.uint8, (R, I2), "z_q", dev),
                                  _in(z_scale, torch.float32, (R, I2 // 128), "z_scale", dev),
                                  _in(dh_row, torch.float32, (R, I2 // 2), "dh_row", dev), R, I2 // 2, pq, ps,
                                  _raw_stream(dev))
    if st:
        _check(st, "moe_swiglu_backward_zq")
    return dz_q, dz_scale
