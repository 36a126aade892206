"""Python binding of libcsa2 -- the CSA2 decode hot path over an FP4 main KV
cache, as hand-written CUDA kernels for GB300 (sm_103a).

Argument marshalling only: every function passes torch tensors' device
pointers, shapes and the current CUDA stream to the C ABI declared in
``include/csa2.h`` and raises ``Csa2Error`` on a non-OK status.  Since the C
calls see bare pointers, the binding first refuses (TypeError / ValueError)
tensors whose element size does not match what the call reads or writes and
buffers smaller than the call touches.  There is no CPU fallback: if the
shared library is missing the import fails loudly.

Names follow the C ABI: ``csa2_quantize_kv_fp4``, ``csa2_rope_quantize_kv_fp4``
(RoPE fused ahead of the quantiser), ``csa2_index_score``, ``csa2_build_pool``,
``csa2_topk``, ``csa2_index_topk`` (fused decode indexer),
``csa2_index_topk_dense`` (fused indexer for many query tokens),
``csa2_sparse_attn_fp4`` (and ``csa2_sparse_attn_fp4_noalloc``),
``csa2_swa_attn_fp8`` (sliding-window branch and merge), the paged 8-bit
cache's ``csa2_build_slots`` (block tables and slot maps),
``csa2_quantize_kv_fp8_paged`` (append) and ``csa2_paged_attn_fp8`` (attention;
``paged.PagedCache`` keeps the buffers and calls the three in order),
``csa2_selftest_bounded_wait`` and the ``*_workspace_bytes`` helpers.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa2.so")

MODE_FULL, MODE_REINDEX, MODE_REUSE = 0, 1, 2
BF16, FP8_E4M3, FP32, FP16 = 0, 1, 2, 3
FLAG_BAD_INDEX, FLAG_BAD_POOL, FLAG_BAD_SLOT, FLAG_TIMEOUT = 0x1, 0x2, 0x4, 0x8
FLAG_NO_BLOCKS, FLAG_NONFINITE = 0x10, 0x20
INDEX_HEADS, INDEX_DIM, POOL_BLOCK, MAX_POOL, MAX_K = 4, 64, 8, 2048, 2048

STATUS = {0: "CSA2_OK", 1: "CSA2_ERR_INVALID_ARG", 2: "CSA2_ERR_UNSUPPORTED", 3: "CSA2_ERR_WORKSPACE",
          4: "CSA2_ERR_CUDA", 5: "CSA2_ERR_DEVICE_FLAG", 6: "CSA2_ERR_TIMEOUT"}


class Csa2Error(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), detail))
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError("libcsa2.so is not built (run __graft_entry__.build() or "
                          "python sparse_attention_fp4_quantize_gb300/build.py)")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, u64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "csa2_quantize_kv_fp4": ([P, i64, i32, i64, P, i64, P, P, P, P], i32),
        "csa2_rope_quantize_kv_fp4": ([P, i64, i32, i64, P, P, i64, i32, P, i64, P, P, P, P], i32),
        "csa2_index_score": ([i32, i32, i32, i64, P, i32, P, P, i32, P, P, i32, P, P, P], i32),
        "csa2_build_pool": ([i32, i32, i64, P, P, i32, i32, P, P, u64, P], i32),
        "csa2_build_pool_workspace_bytes": ([i32, i32, i64, i32], u64),
        "csa2_topk": ([i32, i32, i32, i64, P, P, P, i32, i32, P, P, u64, P], i32),
        "csa2_topk_workspace_bytes": ([i32, i32, i64, i32], u64),
        "csa2_index_topk": ([i32, i32, i32, i64, P, i32, P, P, i32, P, P, i32, i32, P, P, i32, P, P], i32),
        "csa2_index_topk_dense": ([i32, i32, i64, P, i32, P, P, i32, P, i32, P, P, P, u64, P], i32),
        "csa2_index_topk_dense_workspace_bytes": ([i32, i32, i64, i32], u64),
        "csa2_sparse_attn_fp4": ([i32, i32, i32, i32, i32, i32, P, P, P, i64, P, i32, P, f32, P, i32, P, P,
                                  P, u64, P], i32),
        "csa2_sparse_attn_workspace_bytes": ([i32, i32, i32, i32, i32, i32], u64),
        "csa2_sparse_attn_fp4_prefetch": ([i32, i32, i32, i32, i32, i32, P, P, P, i64, P, i32, P, f32, P, i32, P, P,
                                           P, u64, P, P, P], i32),
        "csa2_swa_attn_fp8": ([i32, i32, i32, i32, i32, P, P, i32, P, f32, P, P, P, P, P, P], i32),
        "csa2_sparse_attn_fp4_noalloc": ([i32, i32, i32, i32, i32, i32, P, P, P, i64, P, i32, P, f32, P, i32, P,
                                          P, P], i32),
        "csa2_sparse_attn_noalloc_max_scratch_bytes": ([], u64),
        "csa2_build_slots": ([i32, i32, i64, i32, i64, i64, P, P, P, P, P, P, P, P, P, P, P, P], i32),
        "csa2_quantize_kv_fp8_paged": ([P, P, i32, i64, i32, i32, i64, i64, i64, i64, P, i64, i32, P, P, P, P, P, P],
                                       i32),
        "csa2_paged_attn_fp8": ([i32, i64, i32, i32, i32, i32, P, i64, i64, P, P, P, P, i64, i32, P, i32, i64, P, P,
                                 i32, i32, f32, P, P, P, P, u64, P], i32),
        "csa2_paged_attn_workspace_bytes": ([i32, i64, i32, i32, i32, i32], u64),
        "csa2_selftest_bounded_wait": ([ctypes.c_uint32, P, P], i32),
        "csa2_status_string": ([i32], ctypes.c_char_p),
        "csa2_last_error": ([], ctypes.c_char_p),
        "csa2_version": ([], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def exported_symbols():
    return ["csa2_quantize_kv_fp4", "csa2_rope_quantize_kv_fp4", "csa2_index_score", "csa2_build_pool", "csa2_build_pool_workspace_bytes",
            "csa2_topk", "csa2_topk_workspace_bytes", "csa2_index_topk", "csa2_index_topk_dense",
            "csa2_index_topk_dense_workspace_bytes", "csa2_sparse_attn_fp4", "csa2_sparse_attn_workspace_bytes",
            "csa2_sparse_attn_fp4_prefetch", "csa2_swa_attn_fp8",
            "csa2_sparse_attn_fp4_noalloc", "csa2_sparse_attn_noalloc_max_scratch_bytes",
            "csa2_build_slots", "csa2_quantize_kv_fp8_paged", "csa2_paged_attn_fp8",
            "csa2_paged_attn_workspace_bytes",
            "csa2_selftest_bounded_wait", "csa2_status_string", "csa2_last_error", "csa2_version"]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(rc: int):
    if rc != 0:
        raise Csa2Error(rc, _lib.csa2_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return FP8_E4M3
    if t.dtype in (torch.bfloat16, torch.int16):
        return BF16
    raise TypeError("indexer tensors must be FP8 E4M3 (uint8/float8_e4m3fn) or bf16 (bfloat16/int16 bits)")


def _on_device(t) -> bool:
    return t.is_cuda


def _cuda(*ts):
    for t in ts:
        if t is not None and (not _on_device(t) or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def _elem(t, name, sizes, floating=None):
    """The C call reads or writes t's memory as elements of one of these
    byte sizes (and of this kind, when given)."""
    if t is None:
        return
    if t.element_size() not in sizes or (floating is not None and t.is_floating_point() != floating):
        raise TypeError("%s: %s elements do not fit this call" % (name, t.dtype))


def _bf16(t, name):
    """The C call reads t as bf16 values: only torch.bfloat16 or its int16
    bit patterns are accepted (a float16 tensor has the same element size
    but other values)."""
    if t is not None and t.dtype not in (torch.bfloat16, torch.int16):
        raise TypeError("%s: %s elements are not bf16 (pass torch.bfloat16 or int16 bit patterns)" % (name, t.dtype))


def _room(t, name, n):
    """t must hold every element the call touches (the C side sees only a pointer)."""
    if t is not None and t.numel() < n:
        raise ValueError("%s holds %d elements, the call touches %d" % (name, t.numel(), n))


def _flag(err_flag):
    _elem(err_flag, "err_flag", (4,), False)
    _room(err_flag, "err_flag", 1)


def _indexer_operands(q_idx, w, k_idx, kv_len, B, T, N):
    _elem(q_idx, "q_idx", (1, 2))
    _elem(k_idx, "k_idx", (1, 2))
    _elem(w, "w", (4,), True)
    _elem(kv_len, "kv_len", (4,), False)
    _room(q_idx, "q_idx", B * T * INDEX_HEADS * INDEX_DIM)
    _room(k_idx, "k_idx", B * N * INDEX_DIM)
    _room(w, "w", B * T * INDEX_HEADS)
    _room(kv_len, "kv_len", B * T)


def csa2_selftest_bounded_wait(err_flag, max_polls=4096, stream=None):
    """The kernels' bounded mbarrier wait on an arrival that never comes:
    sets FLAG_TIMEOUT in err_flag (int32/uint32 CUDA tensor) and returns."""
    _cuda(err_flag)
    _check(_lib.csa2_selftest_bounded_wait(int(max_polls), _ptr(err_flag), _stream(stream)))


def version() -> int:
    return _lib.csa2_version()


def _plane_args(kv, codes, scales, dst_slot, err_flag, R, D, n_slots):
    _bf16(kv, "kv")
    _elem(codes, "codes", (1,))
    _elem(scales, "scales", (1,))
    _elem(dst_slot, "dst_slot", (8,), False)
    _flag(err_flag)
    if codes.dim() != 2 or codes.shape[1] != D // 2:
        raise ValueError("codes must be [slots, D/2] = [*, %d], got %s" % (D // 2, tuple(codes.shape)))
    _room(scales, "scales", n_slots * (D // 16))
    _room(dst_slot, "dst_slot", R)


def csa2_quantize_kv_fp4(kv, codes, scales, dst_slot=None, err_flag=None, stream=None):
    """kv bf16 [R, D] (or int16 bits) -> codes uint8 [S, D/2], scales uint8 [S, D/16]."""
    _cuda(codes, scales, dst_slot, err_flag)
    R, D = kv.shape
    if not _on_device(kv) or kv.stride(1) != 1:
        raise ValueError("kv must be a CUDA tensor with contiguous rows (any row stride)")
    n_slots = codes.shape[0]
    _plane_args(kv, codes, scales, dst_slot, err_flag, R, D, n_slots)
    _check(_lib.csa2_quantize_kv_fp4(_ptr(kv), R, D, kv.stride(0), _ptr(dst_slot), n_slots, _ptr(codes),
                                     _ptr(scales), _ptr(err_flag), _stream(stream)))


def csa2_rope_quantize_kv_fp4(kv, pos, cos_sin, codes, scales, dst_slot=None, err_flag=None, stream=None):
    """Pre-RoPE kv bf16 [R, D] (or int16 bits), pos int32 [R], cos_sin fp32
    [n_pos, rope_dim/2, 2] -> codes uint8 [S, D/2], scales uint8 [S, D/16]."""
    _cuda(kv, pos, cos_sin, codes, scales, dst_slot, err_flag)
    R, D = kv.shape
    _plane_args(kv, codes, scales, dst_slot, err_flag, R, D, codes.shape[0])
    _elem(pos, "pos", (4,), False)
    _elem(cos_sin, "cos_sin", (4,), True)
    _room(pos, "pos", R)
    if cos_sin.dim() != 3 or cos_sin.shape[2] != 2:
        raise ValueError("cos_sin must be [n_pos, rope_dim/2, 2], got %s" % (tuple(cos_sin.shape),))
    n_pos, half = cos_sin.shape[0], cos_sin.shape[1]
    _check(_lib.csa2_rope_quantize_kv_fp4(_ptr(kv), R, D, D, _ptr(pos), _ptr(cos_sin), n_pos, 2 * half,
                                          _ptr(dst_slot), codes.shape[0], _ptr(codes), _ptr(scales),
                                          _ptr(err_flag), _stream(stream)))


def csa2_index_score(mode, q_idx, w, k_idx, kv_len, scores, pool_blocks=None, err_flag=None, stream=None):
    """q_idx [B,T,4,64], w fp32 [B,T,4], k_idx [B,N,64], kv_len int32 [B*T] ->
    scores fp32 [B,T,N] (FULL) or [B,T,8P] (REINDEX)."""
    _cuda(q_idx, w, k_idx, kv_len, scores, pool_blocks, err_flag)
    B, T = q_idx.shape[0], q_idx.shape[1]
    N = k_idx.shape[1]
    P = 0 if pool_blocks is None else pool_blocks.shape[-1]
    if int(mode) != MODE_REUSE:
        _indexer_operands(q_idx, w, k_idx, kv_len, B, T, N)
        _elem(scores, "scores", (4,), True)
        _elem(pool_blocks, "pool_blocks", (4,), False)
        _flag(err_flag)
        _room(scores, "scores", B * T * (8 * P if int(mode) == MODE_REINDEX else N))
        _room(pool_blocks, "pool_blocks", B * T * P)
    _check(_lib.csa2_index_score(int(mode), B, T, N, _ptr(q_idx), _dtype_code(q_idx), _ptr(w), _ptr(k_idx),
                                 _dtype_code(k_idx), _ptr(kv_len), _ptr(pool_blocks), P, _ptr(scores),
                                 _ptr(err_flag), _stream(stream)))


def csa2_build_pool(scores, kv_len, pool_blocks, workspace=None, stream=None):
    """scores fp32 [B,T,N], kv_len int32 [B*T] -> pool_blocks int32 [B,T,P]."""
    _cuda(scores, kv_len, pool_blocks, workspace)
    B, T, N = scores.shape
    P = pool_blocks.shape[-1]
    _elem(scores, "scores", (4,), True)
    _elem(kv_len, "kv_len", (4,), False)
    _elem(pool_blocks, "pool_blocks", (4,), False)
    _room(kv_len, "kv_len", B * T)
    _room(pool_blocks, "pool_blocks", B * T * P)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.csa2_build_pool(B, T, N, _ptr(scores), _ptr(kv_len), P, POOL_BLOCK, _ptr(pool_blocks),
                                _ptr(workspace), ws, _stream(stream)))


def csa2_topk(mode, scores, idx, kv_len=None, pool_blocks=None, workspace=None, stream=None):
    """scores fp32 [B,T,M] -> idx int32 [B,T,K]."""
    _cuda(scores, idx, kv_len, pool_blocks, workspace)
    B, T, M = scores.shape
    K = idx.shape[-1]
    P = 0 if pool_blocks is None else pool_blocks.shape[-1]
    if int(mode) != MODE_REUSE:
        _elem(scores, "scores", (4,), True)
        for t, name in ((idx, "idx"), (kv_len, "kv_len"), (pool_blocks, "pool_blocks")):
            _elem(t, name, (4,), False)
        _room(idx, "idx", B * T * K)
        _room(kv_len, "kv_len", B * T)
        _room(pool_blocks, "pool_blocks", B * T * P)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.csa2_topk(int(mode), B, T, M, _ptr(scores), _ptr(kv_len), _ptr(pool_blocks), P, K, _ptr(idx),
                          _ptr(workspace), ws, _stream(stream)))


def csa2_index_topk(mode, q_idx, w, k_idx, kv_len, idx, pool_blocks=None, pool_out=None, err_flag=None,
                    stream=None):
    """Fused decode indexer (FP8): the scores of csa2_index_score feed the
    Top-K of csa2_topk (and, for FULL with pool_out, the pool of
    csa2_build_pool) without being written out.  q_idx [B,T,4,64], w fp32
    [B,T,4], k_idx [B,N,64], kv_len int32 [B*T] -> idx int32 [B,T,K]
    (+ pool_out int32 [B,T,P_out])."""
    _cuda(q_idx, w, k_idx, kv_len, idx, pool_blocks, pool_out, err_flag)
    B, T = q_idx.shape[0], q_idx.shape[1]
    N = k_idx.shape[1]
    P = 0 if pool_blocks is None else pool_blocks.shape[-1]
    P_out = 0 if pool_out is None else pool_out.shape[-1]
    if int(mode) != MODE_REUSE:
        if q_idx.element_size() == 1 and k_idx.element_size() == 1:   # other dtypes: rejected by the call
            _indexer_operands(q_idx, w, k_idx, kv_len, B, T, N)
        for t, name in ((idx, "idx"), (pool_blocks, "pool_blocks"), (pool_out, "pool_out")):
            _elem(t, name, (4,), False)
        _flag(err_flag)
        _room(idx, "idx", B * T * idx.shape[-1])
        _room(pool_blocks, "pool_blocks", B * T * P)
        _room(pool_out, "pool_out", B * T * P_out)
    _check(_lib.csa2_index_topk(int(mode), B, T, N, _ptr(q_idx), _dtype_code(q_idx), _ptr(w), _ptr(k_idx),
                                _dtype_code(k_idx), _ptr(kv_len), _ptr(pool_blocks), P, idx.shape[-1], _ptr(idx),
                                _ptr(pool_out), P_out, _ptr(err_flag), _stream(stream)))


def csa2_index_topk_dense_workspace_bytes(B, T, N, K) -> int:
    return int(_lib.csa2_index_topk_dense_workspace_bytes(B, T, N, K))


def csa2_index_topk_dense(q_idx, w, k_idx, kv_len, idx, workspace=None, err_flag=None, stream=None):
    """Fused dense indexer for many query tokens (FP8, Full mode): the Top-K
    of csa2_index_score's scores, as csa2_topk selects it, without the score
    matrix.  q_idx [B,T,4,64], w fp32 [B,T,4], k_idx [B,N,64], kv_len int32
    [B*T] -> idx int32 [B,T,K].  workspace: a CUDA byte tensor of at least
    csa2_index_topk_dense_workspace_bytes(B, T, N, K) bytes (allocated here
    when None)."""
    _cuda(q_idx, w, k_idx, kv_len, idx, workspace, err_flag)
    B, T = q_idx.shape[0], q_idx.shape[1]
    N, K = k_idx.shape[1], idx.shape[-1]
    if q_idx.element_size() == 1 and k_idx.element_size() == 1:       # other dtypes: rejected by the call
        _indexer_operands(q_idx, w, k_idx, kv_len, B, T, N)
    _elem(idx, "idx", (4,), False)
    _flag(err_flag)
    _room(idx, "idx", B * T * K)
    if workspace is None:
        workspace = torch.empty(max(1, csa2_index_topk_dense_workspace_bytes(B, T, N, K)), dtype=torch.uint8,
                                device=idx.device)
    ws = workspace.numel() * workspace.element_size()
    _check(_lib.csa2_index_topk_dense(B, T, N, _ptr(q_idx), _dtype_code(q_idx), _ptr(w), _ptr(k_idx),
                                      _dtype_code(k_idx), _ptr(kv_len), K, _ptr(idx), _ptr(err_flag),
                                      _ptr(workspace), ws, _stream(stream)))


def csa2_swa_attn_fp8(q, swa_kv, swa_len, out, sm_scale, o_sparse=None, lse_sparse=None, lse=None, err_flag=None,
                      stream=None):
    """Sliding-window branch: q bf16 [B,T,H,D], swa_kv E4M3 [B,W,D] (uint8 or
    float8_e4m3fn), swa_len int32 [B*T] -> out fp32 [B,T,H,dv] (and lse),
    merged with (o_sparse, lse_sparse) when given; out may be o_sparse."""
    _cuda(q, swa_kv, swa_len, out, o_sparse, lse_sparse, lse, err_flag)
    B, T, H, D = q.shape
    W = swa_kv.shape[1]
    dv = out.shape[-1]
    _bf16(q, "q")
    _elem(swa_kv, "swa_kv", (1,))
    _elem(swa_len, "swa_len", (4,), False)
    for t, name in ((out, "out"), (o_sparse, "o_sparse"), (lse_sparse, "lse_sparse"), (lse, "lse")):
        _elem(t, name, (4,), True)
    _flag(err_flag)
    _room(swa_kv, "swa_kv", B * W * D)
    _room(swa_len, "swa_len", B * T)
    _room(out, "out", B * T * H * dv)
    _room(o_sparse, "o_sparse", B * T * H * dv)
    _room(lse_sparse, "lse_sparse", B * T * H)
    _room(lse, "lse", B * T * H)
    _check(_lib.csa2_swa_attn_fp8(B, T, H, D, out.shape[-1], _ptr(q), _ptr(swa_kv), W, _ptr(swa_len),
                                  float(sm_scale), _ptr(o_sparse), _ptr(lse_sparse), _ptr(out), _ptr(lse),
                                  _ptr(err_flag), _stream(stream)))


def csa2_sparse_attn_workspace_bytes(B, T, H, D, dv, K) -> int:
    return int(_lib.csa2_sparse_attn_workspace_bytes(B, T, H, D, dv, K))


def _attn_args(q, codes, scales, N, idx, out, kv_len, lse, err_flag, B, T, H, D, dv, K):
    _bf16(q, "q")
    _elem(codes, "codes", (1,))
    _elem(scales, "scales", (1,))
    _elem(idx, "idx", (4,), False)
    _elem(kv_len, "kv_len", (4,), False)
    _elem(out, "out", (4,), True)
    _elem(lse, "lse", (4,), True)
    _flag(err_flag)
    _room(codes, "codes", B * int(N) * (D // 2))
    _room(scales, "scales", B * int(N) * (D // 16))
    _room(idx, "idx", B * T * K)
    _room(kv_len, "kv_len", B * T)
    _room(out, "out", B * T * H * dv)
    _room(lse, "lse", B * T * H)


def csa2_sparse_attn_fp4(mode, q, codes, scales, N, idx, out, sm_scale, kv_len=None, lse=None, err_flag=None,
                         workspace=None, stream=None):
    """q bf16 [B,T,H,D]; codes [B*N, D/2], scales [B*N, D/16]; idx int32
    [B,T,K] -> out fp32 [B,T,H,dv], lse fp32 [B,T,H] (optional)."""
    _cuda(q, codes, scales, idx, out, kv_len, lse, err_flag, workspace)
    B, T, H, D = q.shape
    dv = out.shape[-1]
    K = idx.shape[-1]
    _attn_args(q, codes, scales, N, idx, out, kv_len, lse, err_flag, B, T, H, D, dv, K)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.csa2_sparse_attn_fp4(int(mode), B, T, H, D, dv, _ptr(q), _ptr(codes), _ptr(scales), int(N),
                                     _ptr(idx), K, _ptr(kv_len), float(sm_scale), _ptr(out), FP32, _ptr(lse),
                                     _ptr(err_flag), _ptr(workspace), ws, _stream(stream)))


def csa2_sparse_attn_fp4_prefetch(mode, q, codes, scales, N, idx, out, sm_scale, next_codes=None, next_scales=None,
                                  kv_len=None, lse=None, err_flag=None, workspace=None, stream=None):
    """csa2_sparse_attn_fp4 plus an L2 prefetch hint: the rows idx selects in
    (next_codes, next_scales), the planes of the layer that attends next with
    the same indices."""
    _cuda(q, codes, scales, idx, out, kv_len, lse, err_flag, workspace, next_codes, next_scales)
    B, T, H, D = q.shape
    dv = out.shape[-1]
    K = idx.shape[-1]
    _attn_args(q, codes, scales, N, idx, out, kv_len, lse, err_flag, B, T, H, D, dv, K)
    if (next_codes is None) != (next_scales is None):
        raise ValueError("next_codes and next_scales go together")
    if next_codes is not None:
        _elem(next_codes, "next_codes", (1,))
        _elem(next_scales, "next_scales", (1,))
        _room(next_codes, "next_codes", B * int(N) * (D // 2))
        _room(next_scales, "next_scales", B * int(N) * (D // 16))
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.csa2_sparse_attn_fp4_prefetch(int(mode), B, T, H, D, dv, _ptr(q), _ptr(codes), _ptr(scales), int(N),
                                              _ptr(idx), K, _ptr(kv_len), float(sm_scale), _ptr(out), FP32,
                                              _ptr(lse), _ptr(err_flag), _ptr(workspace), ws, _ptr(next_codes),
                                              _ptr(next_scales), _stream(stream)))


def workspace_for_attn(B, T, H, D, dv, K, device="cuda"):
    """Allocate (through torch) the scratch csa2_sparse_attn_fp4 needs, or None."""
    n = csa2_sparse_attn_workspace_bytes(B, T, H, D, dv, K)
    return None if n == 0 else torch.empty(n, dtype=torch.uint8, device=device)


def csa2_sparse_attn_fp4_noalloc(mode, q, codes, scales, N, idx, out, sm_scale, kv_len=None, lse=None,
                                 err_flag=None, stream=None):
    """csa2_sparse_attn_fp4 for callers that may not allocate device memory:
    the split-KV scratch is the library's built-in array (see the header)."""
    _cuda(q, codes, scales, idx, out, kv_len, lse, err_flag)
    B, T, H, D = q.shape
    dv = out.shape[-1]
    K = idx.shape[-1]
    _attn_args(q, codes, scales, N, idx, out, kv_len, lse, err_flag, B, T, H, D, dv, K)
    _check(_lib.csa2_sparse_attn_fp4_noalloc(int(mode), B, T, H, D, dv, _ptr(q), _ptr(codes), _ptr(scales), int(N),
                                             _ptr(idx), K, _ptr(kv_len), float(sm_scale), _ptr(out), FP32,
                                             _ptr(lse), _ptr(err_flag), _stream(stream)))


def noalloc_max_scratch_bytes() -> int:
    return int(_lib.csa2_sparse_attn_noalloc_max_scratch_bytes())


# ------------------------------------------------------------------ paged 8-bit cache
# A serving loop makes these calls a few times per layer and step, on kernels of
# a few microseconds: one comparison per property and tensor, the reason for a
# refusal is worked out afterwards.
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
_ROWS = {torch.bfloat16: BF16, torch.int16: BF16, torch.float16: FP16}


def _refuse(t, name, dtype, shape, dev, dense):
    if t.dtype is not dtype:
        raise TypeError("%s: %s elements do not fit this call (%s)" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.get_device() != dev:
        raise ValueError("tensors must be CUDA tensors of one device (%s is on %s)" % (name, t.device))
    raise ValueError("%s must be contiguous" % name if dense else "%s: strides do not fit this call" % name)


def _arg(t, name, dtype, shape, dev):
    """Pointer of a tensor of this dtype and shape without gaps, on device dev."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _refuse(t, name, dtype, shape, dev, True)


def _opt(t, name, dtype, shape, dev):
    return None if t is None else _arg(t, name, dtype, shape, dev)


def _flag_arg(err_flag, dev):
    if err_flag is None:
        return None
    _flag(err_flag)
    if err_flag.get_device() != dev:
        raise ValueError("tensors must be CUDA tensors of one device (err_flag is on %s)" % err_flag.device)
    return err_flag.data_ptr()


def _rows_arg(x, name, dtype, shape, dev):
    """(pointer, token stride, head stride) of rows [T, H, D] with contiguous channels."""
    if x.dtype is not dtype or x.shape != shape or x.get_device() != dev:
        _refuse(x, name, dtype, shape, dev, False)
    st, sh, sd = x.stride()
    if sd != 1:
        raise ValueError("%s must have contiguous channels" % name)
    # the stride of an extent of one says nothing
    return x.data_ptr(), st if shape[0] > 1 else shape[1] * shape[2], sh if shape[1] > 1 else shape[2]


def _table_arg(t, shape, dev):
    """(pointer, row stride) of a block table whose rows have no gaps between entries."""
    st, s1 = t.stride()
    if t.dtype is not _I32 or t.get_device() != dev or (s1 != 1 and shape[1] > 1):
        _refuse(t, "block_table", _I32, shape, dev, False)
    return t.data_ptr(), st if shape[0] > 1 else shape[1]


def _planes_args(k_codes, v_codes, k_scale, v_scale, dev):
    shape = k_codes.shape
    if len(shape) != 4:
        raise ValueError("k_codes must be [n_blocks, Hkv, S, D], got %s" % (tuple(shape),))
    kd, vd = k_codes.dtype, v_codes.dtype
    if not (kd is torch.uint8 or kd is torch.float8_e4m3fn) or not (vd is torch.uint8 or vd is torch.float8_e4m3fn):
        raise TypeError("k_codes and v_codes must be E4M3 (uint8 or float8_e4m3fn), got %s and %s" % (kd, vd))
    return (_arg(k_codes, "k_codes", kd, shape, dev), _arg(v_codes, "v_codes", vd, shape, dev),
            _arg(k_scale, "k_scale", _F32, shape[:2], dev), _arg(v_scale, "v_scale", _F32, shape[:2], dev))


def _device_of(t):
    dev = t.get_device()
    if dev < 0 and not _on_device(t):
        raise ValueError("tensors must be CUDA tensors")
    return dev


def _launch(fn, dev, stream, *args):
    """Call the C function on device dev, on the given stream or that device's current one."""
    if dev < 0:                                   # no such device: a stand-in for the library
        return _check(fn(*args, _stream(stream)))
    s = _stream(stream) if stream is not None else torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc != 0:
        _check(rc)


def csa2_build_slots(kv_len, new_len, block_table, free_list, free_count, block_size, kv_len_out, free_count_out,
                     cu_len, positions, slots, err_flag=None, stream=None):
    """Block tables and slot maps of a step from the requests' lengths.
    kv_len, new_len int32 [B] (new_len < 0: the request has ended), block_table
    int32 [B, M] (updated in place), free_list int32 [capacity] with
    free_count int32 [1] ids on it -> kv_len_out int32 [B], free_count_out
    int32 [1] (may be the inputs), cu_len int32 [B + 1], positions int32 [T] or
    None, slots int64 [T]."""
    dev = _device_of(kv_len)
    B, M = block_table.shape
    (T,), (cap,) = slots.shape, free_list.shape
    one = (B,)
    table, stride = _table_arg(block_table, (B, M), dev)
    _launch(_lib.csa2_build_slots, dev, stream, B, M, stride, block_size, T, cap,
            _arg(kv_len, "kv_len", _I32, one, dev), _arg(new_len, "new_len", _I32, one, dev), table,
            _arg(free_list, "free_list", _I32, (cap,), dev), _arg(free_count, "free_count", _I32, (1,), dev),
            _arg(kv_len_out, "kv_len_out", _I32, one, dev), _arg(free_count_out, "free_count_out", _I32, (1,), dev),
            _arg(cu_len, "cu_len", _I32, (B + 1,), dev), _opt(positions, "positions", _I32, (T,), dev),
            _arg(slots, "slots", _I64, (T,), dev), _flag_arg(err_flag, dev))


def csa2_quantize_kv_fp8_paged(k, v, slots, k_codes, v_codes, k_scale, v_scale, err_flag=None, stream=None):
    """k, v bf16 (or int16 bits) or fp16 [T, Hkv, D] (any token and head
    strides that are multiples of 8), slots int64 [T] -> k_codes, v_codes
    uint8 or float8_e4m3fn [n_blocks, Hkv, S, D], k_scale, v_scale fp32
    [n_blocks, Hkv], updated in place."""
    dev = _device_of(k)
    kc, vc, ks, vs = _planes_args(k_codes, v_codes, k_scale, v_scale, dev)
    n, H, S, D = k_codes.shape
    (T,) = slots.shape
    dt = _ROWS.get(k.dtype)
    if dt is None:
        raise TypeError("k and v must be bf16 (or int16 bits) or fp16, got %s" % k.dtype)
    kp, kt, kh = _rows_arg(k, "k", k.dtype, (T, H, D), dev)
    vp, vt, vh = _rows_arg(v, "v", k.dtype, (T, H, D), dev)
    _launch(_lib.csa2_quantize_kv_fp8_paged, dev, stream, kp, vp, dt, T, H, D, kt, kh, vt, vh,
            _arg(slots, "slots", _I64, (T,), dev), n, S, kc, vc, ks, vs, _flag_arg(err_flag, dev))


def csa2_paged_attn_workspace_bytes(B, T, Hq, Hkv, D, max_new) -> int:
    return int(_lib.csa2_paged_attn_workspace_bytes(B, T, Hq, Hkv, D, max_new))


def workspace_for_paged_attn(B, T, Hq, Hkv, D, max_new, device="cuda"):
    """Allocate (through torch) the scratch csa2_paged_attn_fp8 needs, or None."""
    n = csa2_paged_attn_workspace_bytes(B, T, Hq, Hkv, D, max_new)
    return None if n == 0 else torch.empty(n, dtype=torch.uint8, device=device)


def csa2_paged_attn_fp8(q, k_codes, v_codes, k_scale, v_scale, block_table, kv_len, cu_len, out, sm_scale, max_new,
                        window=0, lse=None, err_flag=None, workspace=None, stream=None):
    """Causal attention of a ragged batch over the paged cache.  q bf16 (or
    int16 bits) or fp16 [T, Hq, D] (any token and head strides that are
    multiples of 8), planes as csa2_quantize_kv_fp8_paged, block_table int32
    [B, M], kv_len int32 [B], cu_len int32 [B + 1] -> out [T, Hq, D] of q's
    type, lse fp32 [T, Hq].  max_new: upper bound of a request's rows (a
    hint).  workspace: a CUDA byte tensor of at least
    csa2_paged_attn_workspace_bytes bytes (allocated here when None)."""
    dev = _device_of(q)
    kc, vc, ks, vs = _planes_args(k_codes, v_codes, k_scale, v_scale, dev)
    n, H, S, D = k_codes.shape
    T, Hq = q.shape[:2]
    B, M = block_table.shape
    dt = _ROWS.get(q.dtype)
    if dt is None:
        raise TypeError("q must be bf16 (or int16 bits) or fp16, got %s" % q.dtype)
    if H < 1 or Hq % H:
        raise ValueError("%d query heads do not divide over %d KV heads" % (Hq, H))
    shape = (T, Hq, D)
    qp, qt, qh = _rows_arg(q, "q", q.dtype, shape, dev)
    table, stride = _table_arg(block_table, (B, M), dev)
    if workspace is None:                         # of the stream that uses it, which may not be the current one
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=q.device)
        with torch.cuda.stream(stream):
            workspace = workspace_for_paged_attn(B, T, Hq, H, D, max_new, device=q.device)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _launch(_lib.csa2_paged_attn_fp8, dev, stream, B, T, Hq, H, D, dt, qp, qt, qh, kc, vc, ks, vs, n, S, table, M,
            stride, _arg(kv_len, "kv_len", _I32, (B,), dev), _arg(cu_len, "cu_len", _I32, (B + 1,), dev), max_new,
            window, sm_scale, _arg(out, "out", q.dtype, shape, dev), _opt(lse, "lse", _F32, (T, Hq), dev),
            _flag_arg(err_flag, dev),
            None if workspace is None else _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev), ws)
