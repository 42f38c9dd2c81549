"""Python binding of libbi: batch-invariant linear layers and RMSNorm for GB300.

Argument marshalling only: every function here checks dtypes and devices,
takes data pointers, sizes and the current CUDA stream from torch tensors and
calls the matching ``extern "C"`` entry point of ``libbi.so`` (declared in
``include/bi.h``). All arithmetic runs in the library's sm_103a kernels; there
is no CPU or PyTorch fallback. If the library is missing this module raises.

Names follow the C ABI: ``gemm_bf16``, ``grouped_gemm_bf16``, ``gemm_nvfp4``,
``quantize_nvfp4``, ``rmsnorm``, ``plan``, ``device_status``, ``check_wait_timeout``;
the 4-bit forms ``kv_int4_cache``, ``kv_int4_append``, ``kv_int4_read``,
``attention_decode_int4``, ``attention_extend_int4``, ``gemm_int4``; from the
projection to the attention ``rope_freqs``, ``rope``, ``qk_norm_rope``,
``kv_append``; with a sliding window ``attention_decode_window``,
``attention_extend_window``.
"""
from __future__ import annotations

import ctypes
import operator
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
# BI_LIBRARY=debug selects the debug build (bounds-checked kernels, same results)
LIB_PATH = os.path.join(_HERE, "libbi_debug.so" if os.environ.get("BI_LIBRARY") == "debug" else "libbi.so")

(BI_OK, BI_ERR_INVALID_ARG, BI_ERR_UNSUPPORTED, BI_ERR_MISALIGNED, BI_ERR_ARCH, BI_ERR_CUDA, BI_ERR_TIMEOUT,
 BI_ERR_BOUNDS) = range(8)
OP_GEMM_BF16, OP_GROUPED_GEMM_BF16, OP_GEMM_NVFP4, OP_RMSNORM, OP_QUANTIZE_NVFP4, OP_GROUPED_GEMM_SILU_BF16 = range(6)

_lock = threading.Lock()
_lib = None


class BiError(RuntimeError):
    """A libbi call returned a non-OK status."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class Plan(ctypes.Structure):
    _fields_ = [("op", ctypes.c_int32),
                ("block_m", ctypes.c_int32), ("block_n", ctypes.c_int32), ("block_k", ctypes.c_int32),
                ("mma_m", ctypes.c_int32), ("mma_n", ctypes.c_int32), ("mma_k", ctypes.c_int32),
                ("k_steps", ctypes.c_int32), ("split_k", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("smem_bytes", ctypes.c_int32),
                ("tiles_m", ctypes.c_int64), ("tiles_n", ctypes.c_int64),
                ("grid", ctypes.c_int32), ("reduce_tree", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_}


def load() -> ctypes.CDLL:
    """Load libbi.so (built by ``__graft_entry__.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libbi.so is not built ({LIB_PATH}); run __graft_entry__.build() first")
        lib = ctypes.CDLL(LIB_PATH)
        P, I64, I32, F, D = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_double
        sig = {
            "bi_gemm_bf16": [P, I64, P, I64, P, I64, I64, I64, I64, P],
            "bi_grouped_gemm_bf16": [P, P, P, P, I32, I64, I64, I64, P],
            "bi_grouped_gemm_silu_bf16": [P, P, P, P, I32, I64, I64, I64, P],
            "bi_gemm_nvfp4": [P, P, P, P, F, P, I64, I64, I64, P],
            "bi_rmsnorm": [P, P, P, P, I64, I64, F, P],
            "bi_quantize_nvfp4": [P, I64, F, P, P, I64, I64, P],
            "bi_moe_topk_softmax": [P, I64, I32, I32, I32, P, P, P],
            "bi_moe_align": [P, I64, I32, I32, P, P, P, P],
            "bi_moe_gather": [P, I64, I64, P, I64, P, P],
            "bi_silu_mul": [P, I64, I64, P, P],
            "bi_moe_combine": [P, I64, P, P, I64, I32, I64, P, P],
            "bi_rank_sum_rmsnorm": [P, I32, P, P, P, P, I64, I64, F, P],
            "bi_attention_decode": [P, P, P, P, I32, I64, P, I64, I32, I32, I32, I32, I32, F, P, I64, P, P],
            "bi_attention_decode_workspace_size": [I64, I32, I32],
            "bi_attention_decode_noalloc": [P, P, P, P, I32, I64, P, I64, I32, I32, I32, I32, I32, F, P, P],
            "bi_debug_build": [],
            "bi_last_bounds_line": [],
            "bi_check_bounds": [I32, I32, P],
            "bi_attention_extend": [P, P, I32, P, P, P, I32, I64, P, I64, I32, I32, I32, I32, I32, I32, F, P, P],
            "bi_kv_int4_append": [P, I64, P, I64, I64, P, P, P, P, P, I64, I32, I32, I32, P],
            "bi_kv_int4_read": [P, P, P, P, I64, I32, I32, I32, P, I64, P, I64, P, I64, P],
            "bi_attention_decode_int4": [P, P, P, P, P, P, I32, I64, P, I64, I32, I32, I32, I32, I32, F, P, I64, P, P],
            "bi_attention_extend_int4": [P, P, I32, P, P, P, P, P, I32, I64, P, I64, I32, I32, I32, I32, I32, I32, F, P,
                                         I64, P, P],
            "bi_attention_extend_int4_workspace_size": [I64, I32, I32, I32, I32],
            "bi_gemm_int4": [P, I64, P, P, P, P, I64, I64, I64, I64, I64, P],
            "bi_rope_freqs": [I32, I32, D, D, D, D, D, P, P, ctypes.POINTER(F)],
            "bi_rope": [P, I64, P, I64, I32, I32, P, P, I64, P],
            "bi_qk_norm_rope": [P, I64, P, I64, P, P, F, P, I64, I32, I32, I32, P, P, I64, P, I64, P],
            "bi_kv_append": [P, I64, P, I64, I64, P, P, F, P, P, P, P, I64, I32, I32, I32, P, I64, P, I32, P, I64, P],
            "bi_attention_decode_window_workspace_size": [I64, I32, I32, I32, I32],
            "bi_attention_decode_window": [P, P, P, P, I32, I64, P, I64, I32, I32, I32, I32, I32, F, I32, I32, P, I64, P, P],
            "bi_attention_extend_window_workspace_size": [I64, I32, I32, I32, I32, I32, I32],
            "bi_attention_extend_window_batch_workspace_size": [I64, I64, I32, I32, I32, I32, I32, I32],
            "bi_attention_extend_window": [P, P, I32, P, P, P, I32, I64, P, I64, I32, I32, I32, I32, I32, I32, F, I32, I32,
                                           P, I64, P, P],
            "bi_plan": [I32, I64, I64, I64, I32, ctypes.POINTER(Plan)],
            "bi_device_status": [P],
            "bi_check_wait_timeout": [ctypes.c_uint32, P],
            "bi_status_string": [ctypes.c_int],
            "bi_version": [],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        lib.bi_status_string.restype = ctypes.c_char_p
        lib.bi_attention_decode_workspace_size.restype = ctypes.c_int64
        for name in ("bi_attention_extend_int4_workspace_size", "bi_attention_decode_window_workspace_size",
                     "bi_attention_extend_window_workspace_size", "bi_attention_extend_window_batch_workspace_size"):
            getattr(lib, name).restype = ctypes.c_int64
        _bind_torch()
        _lib = lib
        return lib


# What the calls over heads and the windowed ones use of torch, bound once by load(): where a call takes a few
# microseconds, looking them up is a tenth of it.
_bfloat16 = _int64 = _int32 = _uint8 = _empty_like = _current_device = _raw_stream = None


def _bind_torch():
    global _bfloat16, _int64, _int32, _uint8, _empty_like, _current_device, _raw_stream
    import torch
    _bfloat16, _int64, _int32, _uint8, _empty_like = torch.bfloat16, torch.int64, torch.int32, torch.uint8, torch.empty_like
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda device: torch.cuda.current_stream(device).cuda_stream)


def status_string(status: int) -> str:
    return load().bi_status_string(status).decode()


def version() -> int:
    return int(load().bi_version())


def _check(status: int, where: str):
    if status != BI_OK:
        raise BiError(status, where)


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, dtype, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def gemm_bf16(X, W, Y=None, stream=None):
    """Y[M,N] = X[M,K] W[N,K]^T (bf16 in/out, fp32 accumulate), batch-invariant.

    X and W may be row-strided views (unit column stride); Y is allocated if None."""
    import torch
    _dev(X, torch.bfloat16, "X"), _dev(W, torch.bfloat16, "W")
    if X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[1]:
        raise ValueError(f"shape mismatch X{tuple(X.shape)} W{tuple(W.shape)}")
    if X.stride(1) != 1 or W.stride(1) != 1:
        raise ValueError("X and W need unit column stride")
    M, K = X.shape
    N = W.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _dev(Y, torch.bfloat16, "Y")
    if Y.shape != (M, N) or Y.stride(1) != 1:
        raise ValueError("Y must be [M, N] with unit column stride")
    _check(load().bi_gemm_bf16(_ptr(X), X.stride(0), _ptr(W), W.stride(0), _ptr(Y), Y.stride(0), M, N, K,
                               _stream(stream)), "bi_gemm_bf16")
    return Y


def grouped_gemm_bf16(X, W, offsets, Y=None, stream=None):
    """Per-expert Y[r] = X[r] W[e]^T for rows r in [offsets[e], offsets[e+1]).

    X [rows,K], W [E,N,K] bf16 (contiguous); offsets int32 [E+1] on the device."""
    import torch
    _dev(X, torch.bfloat16, "X"), _dev(W, torch.bfloat16, "W"), _dev(offsets, torch.int32, "offsets")
    if not (X.is_contiguous() and W.is_contiguous() and offsets.is_contiguous()):
        raise ValueError("X, W and offsets must be contiguous")
    E, N, K = W.shape
    rows = X.shape[0]
    if X.shape[1] != K or offsets.numel() != E + 1:
        raise ValueError("shape mismatch")
    if Y is None:
        Y = torch.empty((rows, N), dtype=torch.bfloat16, device=X.device)
    _dev(Y, torch.bfloat16, "Y")
    if Y.shape != (rows, N) or not Y.is_contiguous():
        raise ValueError("Y must be contiguous [rows, N]")
    _check(load().bi_grouped_gemm_bf16(_ptr(X), _ptr(W), _ptr(Y), _ptr(offsets), E, rows, N, K, _stream(stream)),
           "bi_grouped_gemm_bf16")
    return Y


def grouped_gemm_silu_bf16(X, W, offsets, act=None, stream=None):
    """MoE gate_up with SiLU-mul fused: act[r] = silu(X[r] Wg[e]^T) * (X[r] Wu[e]^T),
    gate and up rounded to bf16 first, for rows r in [offsets[e], offsets[e+1]).

    X [rows,K], W [E,2I,K] bf16 (gate rows then up rows; contiguous); offsets int32 [E+1]."""
    import torch
    _dev(X, torch.bfloat16, "X"), _dev(W, torch.bfloat16, "W"), _dev(offsets, torch.int32, "offsets")
    if not (X.is_contiguous() and W.is_contiguous() and offsets.is_contiguous()):
        raise ValueError("X, W and offsets must be contiguous")
    E, N2, K = W.shape
    rows, I = X.shape[0], N2 // 2
    if X.shape[1] != K or offsets.numel() != E + 1 or N2 % 2:
        raise ValueError("shape mismatch")
    if act is None:
        act = torch.empty((rows, I), dtype=torch.bfloat16, device=X.device)
    _dev(act, torch.bfloat16, "act")
    if act.shape != (rows, I) or not act.is_contiguous():
        raise ValueError("act must be contiguous [rows, I]")
    _check(load().bi_grouped_gemm_silu_bf16(_ptr(X), _ptr(W), _ptr(act), _ptr(offsets), E, rows, I, K,
                                            _stream(stream)), "bi_grouped_gemm_silu_bf16")
    return act


def gemm_nvfp4(A, A_sf, B, B_sf, alpha: float, Y=None, stream=None):
    """Y[M,N] = alpha * dequant(A) dequant(B)^T, e2m1 codes packed two per byte
    (uint8 [rows, K/2]) with e4m3 block scales (uint8, interleaved 128x4 layout)."""
    import torch
    for t, n in ((A, "A"), (A_sf, "A_sf"), (B, "B"), (B_sf, "B_sf")):
        _dev(t, torch.uint8, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    M, KB = A.shape
    N = B.shape[0]
    K = KB * 2
    if B.shape[1] != KB:
        raise ValueError("A and B disagree on K")
    c4 = -(-(K // 16) // 4) * 4
    if A_sf.numel() < -(-M // 128) * 128 * c4 or B_sf.numel() < -(-N // 128) * 128 * c4:
        raise ValueError("scale buffers are smaller than the interleaved layout needs")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _dev(Y, torch.bfloat16, "Y")
    if Y.shape != (M, N) or not Y.is_contiguous():
        raise ValueError("Y must be contiguous [M, N]")
    _check(load().bi_gemm_nvfp4(_ptr(A), _ptr(A_sf), _ptr(B), _ptr(B_sf), float(alpha), _ptr(Y), M, N, K,
                                _stream(stream)), "bi_gemm_nvfp4")
    return Y


def quantize_nvfp4(X, global_scale: float, Q=None, Q_sf=None, stream=None):
    """NVFP4-quantise bf16 rows X [M, K] with a per-tensor global scale.

    Returns (Q uint8 [M, K/2] packed e2m1, Q_sf uint8 interleaved 128x4 scales
    for ceil(M/128)*128 rows), ready for gemm_nvfp4."""
    import torch
    _dev(X, torch.bfloat16, "X")
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be [M, K] with unit column stride")
    M, K = X.shape
    if Q is None:
        Q = torch.empty((M, K // 2), dtype=torch.uint8, device=X.device)
    if Q_sf is None:
        Q_sf = torch.zeros(-(-M // 128) * 128 * (K // 16), dtype=torch.uint8, device=X.device)
    _dev(Q, torch.uint8, "Q"), _dev(Q_sf, torch.uint8, "Q_sf")
    if Q.shape != (M, K // 2) or not Q.is_contiguous() or Q_sf.numel() < -(-M // 128) * 128 * (K // 16):
        raise ValueError("output buffers have the wrong size")
    _check(load().bi_quantize_nvfp4(_ptr(X), X.stride(0), float(global_scale), _ptr(Q), _ptr(Q_sf), M, K,
                                    _stream(stream)), "bi_quantize_nvfp4")
    return Q, Q_sf


def moe_topk_softmax(logits, k: int, renormalize: bool = True, stream=None):
    """Router: (topk_ids int32 [T, k], topk_weights float32 [T, k]) from float32 logits [T, E]."""
    import torch
    _dev(logits, torch.float32, "logits")
    if logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError("logits must be contiguous [T, E]")
    T, E = logits.shape
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(load().bi_moe_topk_softmax(_ptr(logits), T, E, k, int(bool(renormalize)), _ptr(ids), _ptr(w),
                                      _stream(stream)), "bi_moe_topk_softmax")
    return ids, w


def moe_align(topk_ids, E: int, stream=None):
    """(expert_offsets int32 [E+1], row_token int32 [T*k], pos int32 [T, k])."""
    import torch
    _dev(topk_ids, torch.int32, "topk_ids")
    T, k = topk_ids.shape
    off = torch.empty(E + 1, dtype=torch.int32, device=topk_ids.device)
    row_token = torch.empty(T * k, dtype=torch.int32, device=topk_ids.device)
    pos = torch.empty((T, k), dtype=torch.int32, device=topk_ids.device)
    _check(load().bi_moe_align(_ptr(topk_ids.contiguous()), T, k, E, _ptr(off), _ptr(row_token), _ptr(pos),
                               _stream(stream)), "bi_moe_align")
    return off, row_token, pos


def moe_gather(hidden, row_token, out=None, stream=None):
    """X_sorted[r] = hidden[row_token[r]]."""
    import torch
    _dev(hidden, torch.bfloat16, "hidden"), _dev(row_token, torch.int32, "row_token")
    T, H = hidden.shape
    rows = row_token.numel()
    if out is None:
        out = torch.empty((rows, H), dtype=torch.bfloat16, device=hidden.device)
    _check(load().bi_moe_gather(_ptr(hidden), T, H, _ptr(row_token), rows, _ptr(out), _stream(stream)),
           "bi_moe_gather")
    return out


def silu_mul(gate_up, out=None, stream=None):
    """act = silu(gate) * up for bf16 rows [gate | up]."""
    import torch
    _dev(gate_up, torch.bfloat16, "gate_up")
    rows, I2 = gate_up.shape
    if out is None:
        out = torch.empty((rows, I2 // 2), dtype=torch.bfloat16, device=gate_up.device)
    _check(load().bi_silu_mul(_ptr(gate_up), rows, I2 // 2, _ptr(out), _stream(stream)), "bi_silu_mul")
    return out


def moe_combine(Y_sorted, pos, topk_weights, out=None, stream=None):
    """out[t] = sum_i w[t, i] * Y_sorted[pos[t, i]] in rank order (fp32), bf16."""
    import torch
    _dev(Y_sorted, torch.bfloat16, "Y_sorted"), _dev(pos, torch.int32, "pos")
    _dev(topk_weights, torch.float32, "topk_weights")
    rows, H = Y_sorted.shape
    T, k = pos.shape
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=Y_sorted.device)
    _check(load().bi_moe_combine(_ptr(Y_sorted), rows, _ptr(pos), _ptr(topk_weights), T, k, H, _ptr(out),
                                 _stream(stream)), "bi_moe_combine")
    return out


def rmsnorm(x, w, eps: float, residual=None, out=None, stream=None):
    """out = bf16(h / sqrt(mean(h^2) + eps) * w), h = bf16(x + residual) (written
    back to residual) or x. x, residual, out contiguous bf16 [M, H]; w bf16 [H]."""
    import torch
    _dev(x, torch.bfloat16, "x"), _dev(w, torch.bfloat16, "w")
    if not x.is_contiguous() or not w.is_contiguous() or x.dim() != 2:
        raise ValueError("x must be contiguous [M, H]; w contiguous [H]")
    M, H = x.shape
    if w.numel() != H:
        raise ValueError("w must have H elements")
    if residual is not None:
        _dev(residual, torch.bfloat16, "residual")
        if residual.shape != x.shape or not residual.is_contiguous():
            raise ValueError("residual must be contiguous [M, H]")
    if out is None:
        out = torch.empty_like(x)
    _dev(out, torch.bfloat16, "out")
    if out.shape != x.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous [M, H]")
    _check(load().bi_rmsnorm(_ptr(x), _ptr(residual) if residual is not None else None, _ptr(w), _ptr(out), M, H,
                             float(eps), _stream(stream)), "bi_rmsnorm")
    return out


def rank_sum_rmsnorm(parts, w, eps: float, residual=None, sum_out=None, out=None, stream=None):
    """Deterministic all-reduce + RMSNorm over a list of R ranks' partial rows
    (bf16 [M, H] CUDA tensors on this GPU), summed in list (rank) order."""
    import torch
    R = len(parts)
    if R < 1:
        raise ValueError("need at least one rank")
    for r, t in enumerate(parts):
        _dev(t, torch.bfloat16, f"parts[{r}]")
        if t.shape != parts[0].shape or not t.is_contiguous():
            raise ValueError("all parts must be contiguous and the same shape")
    M, H = parts[0].shape
    _dev(w, torch.bfloat16, "w")
    if out is None:
        out = torch.empty_like(parts[0])
    ptrs = (ctypes.c_void_p * R)(*[t.data_ptr() for t in parts])
    _check(load().bi_rank_sum_rmsnorm(ptrs, R, _ptr(residual) if residual is not None else None, _ptr(w),
                                      _ptr(sum_out) if sum_out is not None else None, _ptr(out), M, H, float(eps),
                                      _stream(stream)), "bi_rank_sum_rmsnorm")
    return out


def attention_decode_workspace_size(B: int, Hq: int, max_seq_len: int) -> int:
    return int(load().bi_attention_decode_workspace_size(B, Hq, max_seq_len))


def attention_decode(Q, K_cache, V_cache, block_table, seq_lens, max_seq_len: int, scale: float,
                     workspace=None, O=None, stream=None):
    """Batch-invariant decode attention over a paged KV cache (see bi.h).

    Q bf16 [B, Hq, 128]; K_cache, V_cache bf16 [blocks, block_size, Hkv, 128];
    block_table int32 [B, max_blocks]; seq_lens int32 [B]. The workspace
    (uint8, device) is allocated with torch if not given."""
    import torch
    _dev(Q, torch.bfloat16, "Q"), _dev(K_cache, torch.bfloat16, "K_cache"), _dev(V_cache, torch.bfloat16, "V_cache")
    _dev(block_table, torch.int32, "block_table"), _dev(seq_lens, torch.int32, "seq_lens")
    for t, n in ((Q, "Q"), (K_cache, "K_cache"), (V_cache, "V_cache"), (block_table, "block_table")):
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    B, Hq, D = Q.shape
    nblk, bs, Hkv, D2 = K_cache.shape
    if D2 != D or V_cache.shape != K_cache.shape or block_table.shape[0] != B or seq_lens.numel() != B:
        raise ValueError("shape mismatch")
    need = attention_decode_workspace_size(B, Hq, max_seq_len)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=Q.device)
    if O is None:
        O = torch.empty_like(Q)
    _check(load().bi_attention_decode(_ptr(Q), _ptr(K_cache), _ptr(V_cache), _ptr(block_table), block_table.shape[1],
                                      nblk, _ptr(seq_lens), B, Hq, Hkv, D, bs, max_seq_len, float(scale),
                                      _ptr(workspace), workspace.numel(), _ptr(O), _stream(stream)),
           "bi_attention_decode")
    return O


def attention_extend(Q, cu_q, K_cache, V_cache, block_table, seq_lens, max_seq_len: int, max_q_len: int,
                     scale: float, O=None, stream=None):
    """Batch-invariant causal extend (prefill) attention over a paged KV cache (see bi.h).

    Q bf16 [total_q, Hq, 128] (each sequence's new tokens, in sequence order);
    cu_q int32 [B+1]; K_cache, V_cache bf16 [blocks, block_size, Hkv, 128];
    block_table int32 [B, max_blocks]; seq_lens int32 [B] (new tokens included)."""
    import torch
    _dev(Q, torch.bfloat16, "Q"), _dev(K_cache, torch.bfloat16, "K_cache"), _dev(V_cache, torch.bfloat16, "V_cache")
    _dev(cu_q, torch.int32, "cu_q"), _dev(block_table, torch.int32, "block_table"), _dev(seq_lens, torch.int32, "seq_lens")
    for t, n in ((Q, "Q"), (K_cache, "K_cache"), (V_cache, "V_cache"), (block_table, "block_table"), (cu_q, "cu_q")):
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    T, Hq, D = Q.shape
    nblk, bs, Hkv, D2 = K_cache.shape
    B = seq_lens.numel()
    if D2 != D or V_cache.shape != K_cache.shape or block_table.shape[0] != B or cu_q.numel() != B + 1:
        raise ValueError("shape mismatch")
    if O is None:
        O = torch.empty_like(Q)
    _check(load().bi_attention_extend(_ptr(Q), _ptr(cu_q), T, _ptr(K_cache), _ptr(V_cache), _ptr(block_table),
                                      block_table.shape[1], nblk, _ptr(seq_lens), B, Hq, Hkv, D, bs, max_seq_len,
                                      max_q_len, float(scale), _ptr(O), _stream(stream)), "bi_attention_extend")
    return O


class KVInt4Cache:
    """One layer's paged 4-bit K/V cache (see bi.h): codes uint8 [blocks, Hkv,
    block_size, 64], scales bfloat16 [blocks, Hkv, block_size, 4], for keys and
    for values; iterating gives the four tensors."""
    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "_dims")

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        import torch
        rows = None
        for t, d, w, n in ((k_codes, torch.uint8, 64, "k_codes"), (k_scales, torch.bfloat16, 4, "k_scales"),
                           (v_codes, torch.uint8, 64, "v_codes"), (v_scales, torch.bfloat16, 4, "v_scales")):
            _dev(t, d, n)
            rows = rows or tuple(t.shape[:3])
            if tuple(t.shape) != rows + (w,) or not t.is_contiguous() or t.device != k_codes.device:
                raise ValueError(f"{n} must be contiguous [blocks, Hkv, block_size, {w}], the same blocks, heads, block "
                                 f"size and device for keys and values; got {tuple(t.shape)}")
            object.__setattr__(self, n, t)
        object.__setattr__(self, "_dims", rows + (k_codes.get_device(),))   # what the calls need of the checked tensors

    def __setattr__(self, name, value):
        raise AttributeError("a KVInt4Cache's tensors are fixed; make a new one")

    def __iter__(self):
        return iter((self.k_codes, self.k_scales, self.v_codes, self.v_scales))


def kv_int4_cache(num_blocks: int, block_size: int, Hkv: int, device="cuda") -> KVInt4Cache:
    """An empty 4-bit K/V cache (every row reads as zeros)."""
    import torch
    rows = (num_blocks, Hkv, block_size)
    return KVInt4Cache(*(torch.zeros(rows + (w,), dtype=d, device=device)
                         for w, d in ((64, torch.uint8), (4, torch.bfloat16)) * 2))


def _current_raw_stream(device: int) -> int:
    """The current stream's handle (without making a Stream object, where torch offers that)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device) if raw is not None else torch.cuda.current_stream(device).cuda_stream


def _cache_dims(cache):
    """(blocks, Hkv, block_size, device) of a cache."""
    if not isinstance(cache, KVInt4Cache):
        raise TypeError("cache must be a KVInt4Cache")
    return cache._dims


def _launch_on(cache, tensors, stream):
    """(raw stream, cache arguments) for a call on the current device; the tensors and the cache (None for a call
    without one), which have passed their checks of type, have to be there."""
    import torch
    cur = torch.cuda.current_device()
    if cache is not None and cache._dims[3] != cur:
        raise ValueError(f"the cache must be on the current device cuda:{cur}, it is on cuda:{cache._dims[3]}")
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"tensors must be on the current device cuda:{cur}, got {t.device}")
    raw = _current_raw_stream(cur) if stream is None else stream.cuda_stream
    if cache is None:
        return raw, ()
    return raw, (cache.k_codes.data_ptr(), cache.k_scales.data_ptr(), cache.v_codes.data_ptr(), cache.v_scales.data_ptr())


def _new(shape, dtype, like, stream):
    """An uninitialised tensor of `stream` (None: the current one), which the current stream may use as well."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    current = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(current)
    return t


def _typed(t, dtype, name, contiguous=True):
    """The tensor, of this type; contiguous if asked for (the device is checked by _launch_on)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}, got {t.dtype} on {t.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _kv_rows(t, T, Hkv, name):
    """Token stride of bf16 rows [T, Hkv, 128] whose heads are contiguous within a token."""
    import torch
    _typed(t, torch.bfloat16, name, contiguous=False)
    if t.shape != (T, Hkv, 128):
        raise ValueError(f"{name} must be [T, Hkv, 128] = {(T, Hkv, 128)}, got {tuple(t.shape)}")
    st = t.stride()
    if T and (st[2] != 1 or (Hkv > 1 and st[1] != 128)):
        raise ValueError(f"{name}: the heads of a token must be contiguous (a token stride is allowed)")
    return st[0] if T > 1 else Hkv * 128


def _slots(slots):
    import torch
    _typed(slots, torch.int64, "slots")
    if slots.dim() != 1:
        raise ValueError("slots must be [T]")
    return slots.shape[0]


def kv_int4_append(K, V, slots, cache: KVInt4Cache, stream=None) -> KVInt4Cache:
    """Quantise tokens' keys and values into the 4-bit cache (see bi.h); returns the cache.

    K, V bf16 [T, Hkv, 128] (a token stride is allowed: slices of a fused
    projection); slots int64 [T]: block * block_size + offset, -1 to skip a
    token. The slots of one call must differ."""
    T = _slots(slots)
    nblk, Hkv, bs, _ = _cache_dims(cache)
    ldk, ldv = _kv_rows(K, T, Hkv, "K"), _kv_rows(V, T, Hkv, "V")
    raw, c = _launch_on(cache, (K, V, slots), stream)
    _check(load().bi_kv_int4_append(K.data_ptr(), ldk, V.data_ptr(), ldv, T, slots.data_ptr(), *c, nblk, Hkv, 128, bs, raw),
           "bi_kv_int4_append")
    return cache


def kv_int4_read(cache: KVInt4Cache, slots, K=None, V=None, stream=None):
    """(K, V) bf16 [T, Hkv, 128]: the values held at `slots` (int64 [T]; -1 gives zeros)."""
    import torch
    T = _slots(slots)
    nblk, Hkv, bs, _ = _cache_dims(cache)
    ldk = _kv_rows(K, T, Hkv, "K") if K is not None else Hkv * 128
    ldv = _kv_rows(V, T, Hkv, "V") if V is not None else Hkv * 128
    raw, c = _launch_on(cache, (slots, K, V), stream)
    if K is None:
        K = _new((T, Hkv, 128), torch.bfloat16, slots, stream)
    if V is None:
        V = _new((T, Hkv, 128), torch.bfloat16, slots, stream)
    _check(load().bi_kv_int4_read(*c, nblk, Hkv, 128, bs, slots.data_ptr(), T, K.data_ptr(), ldk, V.data_ptr(), ldv, raw),
           "bi_kv_int4_read")
    return K, V


def _attention_int4_args(Q, block_table, seq_lens, workspace, O):
    """Checks shared by the 4-bit attention calls: Q's shape."""
    import torch
    _typed(Q, torch.bfloat16, "Q"), _typed(block_table, torch.int32, "block_table"), _typed(seq_lens, torch.int32, "seq_lens")
    shape, tab = Q.shape, block_table.shape
    if len(shape) != 3 or shape[2] != 128 or len(tab) != 2 or tab[0] != seq_lens.numel():
        raise ValueError(f"shape mismatch Q{tuple(shape)} block_table{tuple(tab)} seq_lens{tuple(seq_lens.shape)}")
    if workspace is not None:
        _typed(workspace, torch.uint8, "workspace")
    if O is not None and _typed(O, torch.bfloat16, "O").shape != shape:
        raise ValueError("O must have Q's shape")
    return shape


def attention_decode_int4(Q, cache: KVInt4Cache, block_table, seq_lens, max_seq_len: int, scale: float,
                          workspace=None, O=None, stream=None):
    """Decode attention over the 4-bit cache: the bits of ``attention_decode`` over a bf16 cache of the same values.

    Q bf16 [B, Hq, 128]; block_table int32 [B, max_blocks]; seq_lens int32 [B].
    The workspace (uint8, ``attention_decode_workspace_size`` bytes) is
    allocated with torch if not given."""
    import torch
    B, Hq, D = _attention_int4_args(Q, block_table, seq_lens, workspace, O)
    nblk, Hkv, bs, _ = _cache_dims(cache)
    raw, c = _launch_on(cache, (Q, block_table, seq_lens, workspace, O), stream)
    if seq_lens.shape != (B,):
        raise ValueError("one query token a sequence: seq_lens must be [B], B the rows of Q")
    if workspace is None:
        workspace = _new(max(attention_decode_workspace_size(B, Hq, max_seq_len), 16), torch.uint8, Q, stream)
    if O is None:
        O = _new((B, Hq, D), torch.bfloat16, Q, stream)
    _check(load().bi_attention_decode_int4(Q.data_ptr(), *c, block_table.data_ptr(), block_table.shape[1], nblk,
                                           seq_lens.data_ptr(), B, Hq, Hkv, D, bs, max_seq_len, float(scale),
                                           workspace.data_ptr(), workspace.numel(), O.data_ptr(), raw),
           "bi_attention_decode_int4")
    return O


def attention_extend_int4_workspace_size(total_q: int, Hq: int, Hkv: int, max_seq_len: int, max_q_len: int) -> int:
    return int(load().bi_attention_extend_int4_workspace_size(total_q, Hq, Hkv, max_seq_len, max_q_len))


def attention_extend_int4(Q, cu_q, cache: KVInt4Cache, block_table, seq_lens, max_seq_len: int, max_q_len: int,
                          scale: float, workspace=None, O=None, stream=None):
    """Causal extend (prefill) attention over the 4-bit cache: the bits of ``attention_extend`` over a bf16 cache
    of the same values.

    Q bf16 [total_q, Hq, 128]; cu_q int32 [B+1]; block_table int32 [B, max_blocks];
    seq_lens int32 [B], the new tokens (already in the cache) included;
    max_q_len the most new tokens of a sequence (the work is laid out for that
    many of each). The workspace (uint8, ``attention_extend_int4_workspace_size``
    bytes) is allocated with torch if not given."""
    import torch
    T, Hq, D = _attention_int4_args(Q, block_table, seq_lens, workspace, O)
    B = _typed(cu_q, torch.int32, "cu_q").numel() - 1
    nblk, Hkv, bs, _ = _cache_dims(cache)
    raw, c = _launch_on(cache, (Q, cu_q, block_table, seq_lens, workspace, O), stream)
    if seq_lens.shape != (B,):
        raise ValueError("cu_q must have one entry more than seq_lens")
    if workspace is None:
        need = attention_extend_int4_workspace_size(T, Hq, Hkv, max_seq_len, max_q_len)
        workspace = _new(need, torch.uint8, Q, stream) if need > 0 else None
    if O is None:
        O = _new((T, Hq, D), torch.bfloat16, Q, stream)
    _check(load().bi_attention_extend_int4(Q.data_ptr(), cu_q.data_ptr(), T, *c, block_table.data_ptr(),
                                           block_table.shape[1], nblk, seq_lens.data_ptr(), B, Hq, Hkv, D, bs, max_seq_len,
                                           max_q_len, float(scale), workspace.data_ptr() if workspace is not None else None,
                                           workspace.numel() if workspace is not None else 0, O.data_ptr(), raw),
           "bi_attention_extend_int4")
    return O


def gemm_int4(X, W, scales, zeros=None, Y=None, stream=None):
    """Y[M,N] = X[M,K] dequant(W)[N,K]^T, batch-invariant, for 4-bit weights with group scales.

    X bf16 [M, K] (may be a row-strided view); W uint8 [N, K/2], two codes a
    byte, low nibble for even k; scales bf16 [N, K/g]; zeros uint8 [N, K/g] or
    None (8 throughout). A weight is (code - zero) * scale. Made for few rows:
    beyond 32, ``gemm_bf16`` over bf16 weights is faster (see bi.h)."""
    import torch
    _typed(X, torch.bfloat16, "X", contiguous=False), _typed(W, torch.uint8, "W"), _typed(scales, torch.bfloat16, "scales")
    xs, ws, ss = X.shape, W.shape, scales.shape
    if len(xs) != 2 or len(ws) != 2 or len(ss) != 2 or xs[1] != 2 * ws[1] or ss[0] != ws[0]:
        raise ValueError(f"shape mismatch X{tuple(xs)} W{tuple(ws)} scales{tuple(ss)}")
    (M, K), (N, groups) = xs, ss
    if X.stride(1) != 1:
        raise ValueError("X needs unit column stride")
    if groups < 1 or K % groups:
        raise ValueError("scales must divide K into groups")
    if zeros is not None and _typed(zeros, torch.uint8, "zeros").shape != ss:
        raise ValueError("zeros must have scales' shape")
    if Y is not None and (_typed(Y, torch.bfloat16, "Y", contiguous=False).shape != (M, N) or Y.stride(1) != 1):
        raise ValueError("Y must be [M, N] with unit column stride")
    raw, _ = _launch_on(None, (X, W, scales, zeros, Y), stream)
    if Y is None:
        Y = _new((M, N), torch.bfloat16, X, stream)
    _check(load().bi_gemm_int4(X.data_ptr(), X.stride(0) if M > 1 else K, W.data_ptr(), scales.data_ptr(),
                               zeros.data_ptr() if zeros is not None else None, Y.data_ptr(), Y.stride(0) if M > 1 else N,
                               M, N, K, K // groups, raw), "bi_gemm_int4")
    return Y


class _Rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("factor", ctypes.c_float)]


class RopeFreqs:
    """The frequencies of a rotation (made by ``rope_freqs``): turns int64 [rotary_dim / 2] on the GPU, turns per
    position in units of 2^-64, and how they are used."""
    __slots__ = ("turns", "rotary_dim", "interleaved", "factor", "_ref")

    def __init__(self, turns, rotary_dim: int, interleaved: bool = False, factor: float = 1.0):
        import torch
        _typed(turns, torch.int64, "turns")
        if tuple(turns.shape) != (rotary_dim // 2,) or rotary_dim % 2:
            raise ValueError(f"turns must be [rotary_dim / 2] = [{rotary_dim / 2:g}], got {tuple(turns.shape)}")
        for n, v in (("turns", turns), ("rotary_dim", int(rotary_dim)), ("interleaved", bool(interleaved)), ("factor", float(factor))):
            object.__setattr__(self, n, v)
        object.__setattr__(self, "_ref", ctypes.byref(_Rope(turns.data_ptr(), self.rotary_dim, self.interleaved, self.factor)))

    def __setattr__(self, name, value):
        raise AttributeError("a RopeFreqs is fixed; make a new one")


_ROPE_SCALING = {None: 0, "none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


def rope_freqs(rotary_dim: int, base: float = 10000.0, interleaved: bool = False, scaling=None, scale: float = 1.0,
               original_length: float = 0.0, low=None, high=None, factor=None, freqs=None, device="cuda") -> RopeFreqs:
    """Frequencies base^(-2i / rotary_dim) for ``rope``, ``qk_norm_rope`` and ``kv_append`` (formulas in bi.h).

    scaling for longer contexts, by `scale`: None, "linear", "ntk", "bands" (by turns over original_length: low 1,
    high 4 by default) or "yarn" (low 1, high 32). freqs: rotary_dim / 2 frequencies (radians a position) to use
    instead. factor: what cos and sin are multiplied by (None: 1, or what yarn gives)."""
    import torch
    if freqs is not None:
        kind, given = 5, [float(x) for x in freqs]
        if scaling is not None or 2 * len(given) != rotary_dim:
            raise ValueError("freqs must be rotary_dim / 2 numbers, without a scaling")
        given = (ctypes.c_double * len(given))(*given)
    else:
        if scaling not in _ROPE_SCALING:
            raise ValueError(f"scaling must be one of {sorted(k for k in _ROPE_SCALING if k)}, got {scaling!r}")
        kind, given = _ROPE_SCALING[scaling], None
    turns = torch.zeros(max(rotary_dim // 2, 1), dtype=torch.int64)
    m = ctypes.c_float()
    _check(load().bi_rope_freqs(rotary_dim, kind, base, scale, original_length, 1.0 if low is None else low,
                                (32.0 if scaling == "yarn" else 4.0) if high is None else high, given, turns.data_ptr(),
                                ctypes.byref(m)), "bi_rope_freqs")
    return RopeFreqs(turns.to(device), rotary_dim, interleaved, m.value if factor is None else factor)


# A call's checks are a good part of its time where it is short, so each of the following looks at a tensor once and
# leaves the wording of what is wrong to _refuse.
def _refuse(t, dtype, name, cur, what):
    """Raises what is wrong with a tensor that should be contiguous, of this type and on this device, else ValueError(what)."""
    _typed(t, dtype, name, contiguous=False)
    if t.get_device() != cur:
        raise ValueError(f"tensors must be on the current device cuda:{cur}, {name} is on {t.device}")
    raise ValueError(f"{name} must be {what}, got {tuple(t.shape)} with strides {t.stride()}")


def _tensor(t, dtype, shape, name, cur):
    """Checks a contiguous tensor of this type, device and shape (None: any)."""
    try:
        if t.dtype is dtype and t.get_device() == cur and t.is_contiguous() and (shape is None or t.shape == shape):
            return
    except AttributeError:
        pass                                             # not a tensor
    _refuse(t, dtype, name, cur, "contiguous" + (f" {tuple(shape)}" if shape is not None else ""))


def _heads(t, name, cur, T=-1, D=-1, H=-1):
    """(T, heads, D, token stride) of bf16 heads [T, H, D] that are contiguous within a token (-1: any size)."""
    try:
        (t_, h, d), (st, sh, sd) = t.shape, t.stride()
        if (t.dtype is _bfloat16 and t.get_device() == cur and (T < 0 or (t_ == T and d == D)) and (H < 0 or h == H) and
                ((sd == 1 and (sh == d or h == 1)) or not t_ * h)):
            return t_, h, d, st if t_ > 1 else h * d
    except (AttributeError, TypeError, ValueError):
        pass                                             # not a tensor, or not of three dimensions
    sizes = ", ".join(n if v < 0 else str(v) for n, v in (("T", T), ("heads", H), ("head_dim", D)))
    _refuse(t, _bfloat16, name, cur, f"[{sizes}], the heads of a token contiguous (a token stride is allowed)")


def _rope_args(positions, freqs, T, cur):
    """Pointers of the positions and the rotation, both or neither given."""
    if freqs is None:
        if positions is not None:
            raise ValueError("positions without freqs")
        return None, None
    if not isinstance(freqs, RopeFreqs):
        raise TypeError("freqs must be a RopeFreqs")
    _tensor(positions, _int64, (T,), "positions", cur)
    if freqs.turns.get_device() != cur:
        raise ValueError(f"freqs must be on the current device cuda:{cur}, they are on {freqs.turns.device}")
    return positions.data_ptr(), freqs._ref


def _out(like, stream):
    """A new tensor of a checked tensor's shape and type, contiguous, for a call on `stream`."""
    return _empty_like(like) if stream is None else _new(like.shape, like.dtype, like, stream)


def rope(X, positions, freqs: RopeFreqs, Y=None, stream=None):
    """Rotary positions: Y[t, h] = X[t, h] turned by positions[t].

    X bf16 [T, H, head_dim] (a token stride is allowed); positions int64 [T]. Y may be X (in place)."""
    call = load()
    cur = _current_device()
    T, H, D, ldx = _heads(X, "X", cur)
    if freqs is None:
        raise TypeError("freqs must be a RopeFreqs")
    pos, c = _rope_args(positions, freqs, T, cur)
    if Y is None:
        Y, ldy = _out(X, stream), H * D
    else:
        ldy = _heads(Y, "Y", cur, T, D, H)[3]
    raw = _raw_stream(cur) if stream is None else stream.cuda_stream
    st = call.bi_rope(X.data_ptr(), ldx, pos, T, H, D, c, Y.data_ptr(), ldy, raw)
    if st:
        raise BiError(st, "bi_rope")
    return Y


def qk_norm_rope(Q, K, q_weight, k_weight, eps: float, positions=None, freqs=None, Q_out=None, K_out=None, stream=None):
    """(Q_out, K_out): every query and key head normed (x / sqrt(mean x^2 + eps) * weight) and turned by its position.

    Q bf16 [T, Hq, head_dim], K [T, Hkv, head_dim] (token strides allowed); weights bf16 [head_dim];
    positions int64 [T]; freqs None: the norms alone. Q_out may be Q and K_out K (in place)."""
    call = load()
    cur = _current_device()
    T, Hq, D, ldq = _heads(Q, "Q", cur)
    _, Hkv, _, ldk = _heads(K, "K", cur, T, D)
    _tensor(q_weight, _bfloat16, (D,), "q_weight", cur)
    _tensor(k_weight, _bfloat16, (D,), "k_weight", cur)
    pos, c = _rope_args(positions, freqs, T, cur)
    if Q_out is None:
        Q_out, ldqo = _out(Q, stream), Hq * D
    else:
        ldqo = _heads(Q_out, "Q_out", cur, T, D, Hq)[3]
    if K_out is None:
        K_out, ldko = _out(K, stream), Hkv * D
    else:
        ldko = _heads(K_out, "K_out", cur, T, D, Hkv)[3]
    raw = _raw_stream(cur) if stream is None else stream.cuda_stream
    st = call.bi_qk_norm_rope(Q.data_ptr(), ldq, K.data_ptr(), ldk, q_weight.data_ptr(), k_weight.data_ptr(), eps, pos, T,
                                Hq, Hkv, D, c, Q_out.data_ptr(), ldqo, K_out.data_ptr(), ldko, raw)
    if st:
        raise BiError(st, "bi_qk_norm_rope")
    return Q_out, K_out


def kv_append(K, V, slots, K_cache, V_cache, positions=None, freqs=None, k_weight=None, eps: float = 1e-6, Q=None,
              q_weight=None, Q_out=None, stream=None):
    """Store tokens' keys and values in the paged bf16 cache, the keys normed (k_weight) and turned (positions, freqs)
    on the way; with Q, norm and turn the same tokens' queries in the same launch. Returns Q_out (None without Q).

    K, V bf16 [T, Hkv, head_dim] and Q [T, Hq, head_dim] (token strides allowed: slices of a fused projection);
    slots int64 [T]: block * block_size + offset, -1 to store nothing for a token (its query is computed all the
    same). The slots of one call must differ. K_cache, V_cache bf16 [blocks, block_size, Hkv, head_dim]. Q_out may be Q."""
    call = load()
    cur = _current_device()
    T, Hkv, D, ldk = _heads(K, "K", cur)
    ldv = _heads(V, "V", cur, T, D, Hkv)[3]
    _tensor(slots, _int64, (T,), "slots", cur)
    _tensor(K_cache, _bfloat16, None, "K_cache", cur)
    shape = K_cache.shape
    if len(shape) != 4 or shape[2] != Hkv or shape[3] != D:
        raise ValueError(f"K_cache must be [blocks, block_size, {Hkv}, {D}], got {tuple(shape)}")
    _tensor(V_cache, _bfloat16, shape, "V_cache", cur)
    if k_weight is not None:
        _tensor(k_weight, _bfloat16, (D,), "k_weight", cur)
    pos, c = _rope_args(positions, freqs, T, cur)
    if Q is not None:
        _, Hq, _, ldq = _heads(Q, "Q", cur, T, D)
        if q_weight is not None:
            _tensor(q_weight, _bfloat16, (D,), "q_weight", cur)
        if Q_out is None:
            Q_out, ldqo = _out(Q, stream), Hq * D
        else:
            ldqo = _heads(Q_out, "Q_out", cur, T, D, Hq)[3]
        queries = Q.data_ptr(), ldq, None if q_weight is None else q_weight.data_ptr(), Hq, Q_out.data_ptr(), ldqo
    elif q_weight is not None or Q_out is not None:
        raise ValueError("q_weight and Q_out belong to Q")
    else:
        queries = None, 0, None, 0, None, 0
    raw = _raw_stream(cur) if stream is None else stream.cuda_stream
    st = call.bi_kv_append(K.data_ptr(), ldk, V.data_ptr(), ldv, T, slots.data_ptr(),
                             None if k_weight is None else k_weight.data_ptr(), eps, pos, c, K_cache.data_ptr(),
                             V_cache.data_ptr(), shape[0], Hkv, D, shape[1], *queries, raw)
    if st:
        raise BiError(st, "bi_kv_append")
    return Q_out


def _attention_window_args(Q, K_cache, V_cache, block_table, seq_lens, workspace, O, cur):
    """Checks shared by the windowed calls: Q's and the cache's shapes, the rows of the table."""
    _tensor(Q, _bfloat16, None, "Q", cur)
    _tensor(K_cache, _bfloat16, None, "K_cache", cur)
    _tensor(block_table, _int32, None, "block_table", cur)
    shape, cache, table = Q.shape, K_cache.shape, block_table.shape
    if len(shape) != 3 or shape[2] != 128 or len(cache) != 4 or cache[3] != 128 or len(table) != 2:
        raise ValueError(f"Q must be [tokens, Hq, 128], K_cache [blocks, block_size, Hkv, 128], block_table [B, max_blocks]; got "
                         f"{tuple(shape)}, {tuple(cache)}, {tuple(table)}")
    _tensor(V_cache, _bfloat16, cache, "V_cache", cur)
    _tensor(seq_lens, _int32, (table[0],), "seq_lens", cur)
    if workspace is not None:
        _tensor(workspace, _uint8, None, "workspace", cur)
    if O is not None:
        _tensor(O, _bfloat16, shape, "O", cur)
    return shape, cache, table


def _most(x) -> int:
    """A number as 32 bits hold it (what is past them is refused, or counts as the largest)."""
    x = operator.index(x)
    return x if 0 <= x < 1 << 31 else -1 if x < 0 else (1 << 31) - 1


def _window(window, sinks):
    """Both as 32-bit numbers: anything past the longest sequence counts as that, anything below 0 is refused by the call."""
    window, sinks = operator.index(window), operator.index(sinks)
    if 0 < window <= 1 << 30 and 0 <= sinks <= 1 << 30:
        return window, sinks
    return max(-1, min(window, 1 << 30)), max(-1, min(sinks, 1 << 30))


def attention_decode_window_workspace_size(B: int, Hq: int, max_seq_len: int, window: int, sinks: int = 0) -> int:
    window, sinks = _window(window, sinks)
    return int(load().bi_attention_decode_window_workspace_size(B, Hq, _most(max_seq_len), window, sinks))


def attention_decode_window(Q, K_cache, V_cache, block_table, seq_lens, max_seq_len: int, scale: float, window: int,
                            sinks: int = 0, workspace=None, O=None, stream=None):
    """``attention_decode`` where a token sees the last `window` tokens (itself among them) and the first `sinks`.

    Table entries of blocks out of sight may be anything (-1 once given back). The workspace (uint8,
    ``attention_decode_window_workspace_size`` bytes) is allocated with torch if not given."""
    call = load()
    cur = _current_device()
    (B, Hq, D), (nblk, bs, Hkv, _), table = _attention_window_args(Q, K_cache, V_cache, block_table, seq_lens, workspace, O, cur)
    if table[0] != B:
        raise ValueError("one query token a sequence: block_table must be [B, max_blocks], B the rows of Q")
    window, sinks = _window(window, sinks)
    if workspace is None:
        workspace = _new(max(attention_decode_window_workspace_size(B, Hq, max_seq_len, window, sinks), 16), _uint8, Q, stream)
    if O is None:
        O = _out(Q, stream)
    raw = _raw_stream(cur) if stream is None else stream.cuda_stream
    st = call.bi_attention_decode_window(Q.data_ptr(), K_cache.data_ptr(), V_cache.data_ptr(), block_table.data_ptr(),
                                           table[1], nblk, seq_lens.data_ptr(), B, Hq, Hkv, D, bs, _most(max_seq_len), scale, window,
                                           sinks, workspace.data_ptr(), workspace.numel(), O.data_ptr(), raw)
    if st:
        raise BiError(st, "bi_attention_decode_window")
    return O


def attention_extend_window_workspace_size(total_q: int, Hq: int, Hkv: int, max_seq_len: int, max_q_len: int, window: int,
                                           sinks: int = 0, B=None) -> int:
    """Bytes for a call over B sequences, 0 where it splits nothing; without B, enough for any number of them, 0 past 512 MB."""
    window, sinks = _window(window, sinks)
    sizes = total_q, Hq, Hkv, _most(max_seq_len), _most(max_q_len), window, sinks
    if B is None:
        return int(load().bi_attention_extend_window_workspace_size(*sizes))
    return int(load().bi_attention_extend_window_batch_workspace_size(B, *sizes))


def attention_extend_window(Q, cu_q, K_cache, V_cache, block_table, seq_lens, max_seq_len: int, max_q_len: int, scale: float,
                            window: int, sinks: int = 0, workspace=None, O=None, stream=None):
    """``attention_extend`` where a token sees the last `window` tokens (itself among them) and the first `sinks`: the
    bits of ``attention_decode_window`` of each token's cut sequence.

    Table entries of blocks out of every new token's sight may be anything. The workspace (uint8,
    ``attention_extend_window_workspace_size`` bytes for these B sequences) is allocated with torch if not given."""
    call = load()
    cur = _current_device()
    (T, Hq, D), (nblk, bs, Hkv, _), table = _attention_window_args(Q, K_cache, V_cache, block_table, seq_lens, workspace, O, cur)
    B = table[0]
    _tensor(cu_q, _int32, (B + 1,), "cu_q", cur)
    window, sinks = _window(window, sinks)
    if workspace is None:
        need = attention_extend_window_workspace_size(T, Hq, Hkv, max_seq_len, max_q_len, window, sinks, B)
        workspace = _new(need, _uint8, Q, stream) if need > 0 else None
    if O is None:
        O = _out(Q, stream)
    raw = _raw_stream(cur) if stream is None else stream.cuda_stream
    st = call.bi_attention_extend_window(Q.data_ptr(), cu_q.data_ptr(), T, K_cache.data_ptr(), V_cache.data_ptr(),
                                           block_table.data_ptr(), table[1], nblk, seq_lens.data_ptr(), B, Hq, Hkv, D, bs,
                                           _most(max_seq_len), _most(max_q_len), scale, window, sinks,
                                           workspace.data_ptr() if workspace is not None else None,
                                           workspace.numel() if workspace is not None else 0, O.data_ptr(), raw)
    if st:
        raise BiError(st, "bi_attention_extend_window")
    return O


def plan(op: int, M: int, N: int, K: int, num_sms: int = 0) -> dict:
    """Launch plan for these sizes (num_sms=0: the current device's SM count)."""
    p = Plan()
    _check(load().bi_plan(op, M, N, K, num_sms, ctypes.byref(p)), "bi_plan")
    return p.as_dict()


def debug_build() -> bool:
    """True when the loaded library is the bounds-checked debug build."""
    return bool(load().bi_debug_build())


def last_bounds_line() -> int:
    """Source line of the failed bounds check the last device_status() reported (0 if none)."""
    return int(load().bi_last_bounds_line())


def check_bounds(index: int, limit: int, stream=None) -> None:
    """Write element `index` of a library-owned 64-element array under a
    bounds check against `limit` (debug build: index >= limit is skipped and
    recorded; device_status() then returns BI_ERR_BOUNDS)."""
    _check(load().bi_check_bounds(index, limit, _stream(stream)), "bi_check_bounds")


def device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status code."""
    return int(load().bi_device_status(_stream(stream)))


def check_wait_timeout(limit_us: int, stream=None):
    """Launch the bounded-wait check kernel (see bi.h)."""
    _check(load().bi_check_wait_timeout(limit_us, _stream(stream)), "bi_check_wait_timeout")
