"""Thin Python binding of libsparse_attn.so (C ABI in include/sparse_attn.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  There
is no CPU or library fallback: if the shared library is missing or a call
fails, an exception is raised.

Functions take torch tensors on the current CUDA device and launch on
``torch.cuda.current_stream()``; outputs are allocated with torch unless given.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsparse_attn.so")
_lib = None

SA_OK, SA_EINVAL, SA_EUNSUPPORTED, SA_ECUDA, SA_ETIMEOUT = range(5)
SA_F32, SA_E4M3, SA_BF16 = range(3)

EXPORTS = (
    "sa_status_string", "sa_version", "sa_check_device_error", "sa_index_scores", "sa_topk_select",
    "sa_sparse_mla_workspace_size", "sa_sparse_mla_prefill_workspace_size", "sa_sparse_mla_decode",
    "sa_sparse_mla_prefill",
    "sa_block_mean_pool", "sa_block_sparse_attn", "sa_sparse_mla_decode_static",
    "sa_dense_mla_workspace_size", "sa_dense_mla_decode", "sa_mla_absorb_query", "sa_mla_up_project",
    "sa_nsa_compress", "sa_nsa_decode", "sa_csa_compress", "sa_csa_window_index",
    "sa_index_scores_hist", "sa_topk_select_hist", "sa_set_wait_limit_ns",
    "sa_index_candidates", "sa_topk_from_candidates", "sa_sparse_mla_decode_bf16", "sa_sparse_mla_prefill_bf16",
    "sa_mla_up_project_bf16", "sa_qk_norm_rope", "sa_mla_cache_write", "sa_mla_cache_read",
    "sa_sparse_mla_q8_workspace_size", "sa_sparse_mla_q8", "sa_dense_mla_q8_workspace_size", "sa_dense_mla_q8",
    "sa_tree_mla_workspace_size", "sa_tree_mla_decode",
)

# Size of the library's static device array behind sparse_mla_decode_static
# (SA_STATIC_SCRATCH_BYTES in include/sparse_attn.h).
STATIC_SCRATCH_BYTES = (40 << 20) + (256 << 10)


class SparseAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        name = lib().sa_status_string(status).decode()
        super().__init__(f"{fn} returned {name} ({status})")
        self.status = status


def lib():
    """Load the shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sparse_attention_07_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        L.sa_status_string.restype = ctypes.c_char_p
        L.sa_status_string.argtypes = [I]
        L.sa_version.restype = I
        L.sa_check_device_error.argtypes = [ctypes.POINTER(I), P]
        L.sa_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
        L.sa_index_scores.argtypes = [P, P, P, I64, I, P, I, P, P, I, I, I, I64, P, P]
        L.sa_topk_select.argtypes = [P, I64, P, I, I, P, P]
        L.sa_index_scores_hist.argtypes = [P, P, P, I64, I, P, I, P, P, I, I, I, I64, P, P, P]
        L.sa_topk_select_hist.argtypes = [P, I64, P, I, I, P, P, P]
        L.sa_index_candidates.argtypes = [P, P, P, I64, I, P, I, P, I, I, I, I, I64, P, P, P, P]
        L.sa_topk_from_candidates.argtypes = [P, I64, P, P, I, I, P, P, P]
        L.sa_sparse_mla_workspace_size.restype = SZ
        L.sa_sparse_mla_workspace_size.argtypes = [I, I, I, I]
        L.sa_sparse_mla_decode.argtypes = [P, P, P, I64, P, I64, I64, P, I, P, P, I, I, I, I, I, F, P, P, P, SZ, P]
        L.sa_sparse_mla_prefill_workspace_size.restype = SZ
        L.sa_sparse_mla_prefill_workspace_size.argtypes = [I, I, I, I]
        L.sa_sparse_mla_prefill.argtypes = [P, P, P, I64, P, I64, I64, P, I, P, P, I, I, I, I, I, F, P, P, P, SZ, P]
        L.sa_sparse_mla_decode_bf16.argtypes = L.sa_sparse_mla_decode.argtypes
        L.sa_sparse_mla_prefill_bf16.argtypes = L.sa_sparse_mla_prefill.argtypes
        L.sa_dense_mla_workspace_size.restype = SZ
        L.sa_dense_mla_workspace_size.argtypes = [I, I, I, I]
        L.sa_dense_mla_decode.argtypes = [P, P, P, I64, P, I64, I64, P, I, P, P, I, I, I, I, I, F, P, P, P, SZ, P]
        L.sa_mla_absorb_query.argtypes = [P, P, I, I, I, I, P, P]
        L.sa_mla_up_project.argtypes = [P, P, I, I, I, I, P, P]
        L.sa_mla_up_project_bf16.argtypes = [P, P, I, I, I, I, P, P]
        L.sa_sparse_mla_decode_static.argtypes = [P, P, P, I64, P, I64, I64, P, I, P, P, I, I, I, I, I, F, P, P, P]
        L.sa_block_mean_pool.argtypes = [P, I64, I64, I64, I, I, I, I, I, P, I64, P]
        L.sa_block_sparse_attn.argtypes = [P, P, I64, P, P, I64, I64, I64, I, I, I, I, I, I, I, I, F, P, P, P]
        L.sa_nsa_compress.argtypes = [P, P, I64, I64, I64, I, I, I, I, I, P, P, I64, P]
        L.sa_nsa_decode.argtypes = [P, P, P, I64, I64, I64, P, P, I64, P, I, I, I, I, I, I, I, I, F, P, P, P]
        L.sa_csa_compress.argtypes = [P, P, P, P, I64, I64, P, P, I, I, I, I, I, I, P, I, I64, I64, P]
        L.sa_csa_window_index.argtypes = [P, I, I, P, I, I, P, P]
        L.sa_qk_norm_rope.argtypes = [P, I64, I64, P, I64, I64, I, P, I64, I64, P, I64, I64, I, I, P, P, I, F, P, P,
                                      I64, P, I, I, I, I, I, P]
        L.sa_mla_cache_write.argtypes = [P, I64, P, I64, I, P, I, F, P, P, I64, P, I, P, I, I64, P, I64, P, I64, I64,
                                         P, I, P, P, I, I, I, P]
        L.sa_mla_cache_read.argtypes = [P, I, I64, P, I64, P, I64, I64, P, I, P, P, I, I, I, I, P, P, P]
        L.sa_sparse_mla_q8.argtypes = [P, P, P, I64, P, I64, P, I64, I64, P, I, P, P, I, I, I, I, I, F, P, I, P, P,
                                       SZ, P]
        L.sa_dense_mla_q8.argtypes = L.sa_sparse_mla_q8.argtypes
        L.sa_tree_mla_decode.argtypes = [P, P, P, I, I64, P, I64, P, I64, I64, P, I, P, P, P, P, I, I, I, I, I, I, F,
                                         P, I, P, P, SZ, P]
        for name, args in (("sparse_mla_q8", [I, I, I]), ("dense_mla_q8", [I, I, I]), ("tree_mla", [I, I, I, I])):
            getattr(L, f"sa_{name}_workspace_size").argtypes = args
            getattr(L, f"sa_{name}_workspace_size").restype = SZ
        for name in EXPORTS:
            if name not in ("sa_status_string", "sa_version") and not name.endswith("_workspace_size"):
                getattr(L, name).restype = I
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream():
    # current_stream() builds a Stream object: 3.2 us a call against 0.3
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _check(fn: str, st: int):
    if st != SA_OK:
        raise SparseAttnError(fn, st)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SA_F32
    if t.dtype == torch.float8_e4m3fn:
        return SA_E4M3
    raise TypeError(f"unsupported indexer dtype {t.dtype}")


def check_device_error() -> int:
    """Synchronise the current stream; return (and clear) the device error word."""
    code = ctypes.c_int(0)
    st = lib().sa_check_device_error(ctypes.byref(code), _stream())
    if st not in (SA_OK, SA_ETIMEOUT):
        raise SparseAttnError("sa_check_device_error", st)
    return code.value


def set_wait_limit_ns(limit_ns: int) -> None:
    """Time limit of the kernels' waits on other parties for the current GPU
    (0: the default of one second).  Synchronous."""
    _check("sa_set_wait_limit_ns", lib().sa_set_wait_limit_ns(int(limit_ns)))


HIST_BINS = 4096


def topk_histogram(rows: int, device) -> torch.Tensor:
    """A zeroed [rows, 4096] int32 buffer for index_scores(hist=...) and
    topk_select(hist=...): the Top-K leaves it zeroed, so one serves every step."""
    return torch.zeros(rows, HIST_BINS, dtype=torch.int32, device=device)


def index_scores(q_idx, w, k_idx_cache, n_visible, pages_per_seq: int, page_table=None, seq_of_row=None,
                 scores=None, scores_ld: Optional[int] = None, hist=None):
    """Lightning-indexer scores [rows, scores_ld] fp32 (entries past n_visible untouched).
    With `hist` (zeroed [rows, 4096] int32) it also counts each row's first
    Top-K digit, for topk_select(hist=...)."""
    rows, H_I, d_I = q_idx.shape
    ld = scores_ld or pages_per_seq * 64
    if scores is None:
        scores = torch.empty(rows, ld, dtype=torch.float32, device=q_idx.device)
    pool_pages = k_idx_cache.shape[0] // 64
    args = (_p(q_idx), _p(w), _p(k_idx_cache), pool_pages, _dtype_code(q_idx), _p(page_table), pages_per_seq,
            _p(seq_of_row), _p(n_visible), rows, H_I, d_I, scores.stride(0), _p(scores))
    if hist is None:
        st = lib().sa_index_scores(*args, _stream())
        _check("sa_index_scores", st)
    else:
        st = lib().sa_index_scores_hist(*args, _p(hist), _stream())
        _check("sa_index_scores_hist", st)
    return scores


def topk_select(scores, n_valid, k: int, idx_out=None, hist=None):
    """Exact Top-K positions [rows, k] int32, ascending, -1 padded.  With
    `hist` (as filled by index_scores(hist=...)) the selection starts from it
    and clears it."""
    rows = scores.shape[0]
    if idx_out is None:
        idx_out = torch.empty(rows, k, dtype=torch.int32, device=scores.device)
    if hist is None:
        st = lib().sa_topk_select(_p(scores), scores.stride(0), _p(n_valid), rows, k, _p(idx_out), _stream())
        _check("sa_topk_select", st)
    else:
        st = lib().sa_topk_select_hist(_p(scores), scores.stride(0), _p(n_valid), rows, k, _p(hist), _p(idx_out),
                                       _stream())
        _check("sa_topk_select_hist", st)
    return idx_out


def candidate_buffers(rows: int, cand_ld: int, device):
    """(cand [rows, cand_ld] uint64 as int64, cand_cnt [rows] int32 zeroed,
    hist [rows, 4096] int32 zeroed) for index_candidates / topk_from_candidates:
    the Top-K leaves the counts zeroed, so one set serves every step."""
    return (torch.empty(rows, cand_ld, dtype=torch.int64, device=device),
            torch.zeros(rows, dtype=torch.int32, device=device),
            torch.zeros(rows, HIST_BINS, dtype=torch.int32, device=device))


def index_candidates(q_idx, w, k_idx_cache, n_visible, pages_per_seq: int, k: int, cand, cand_cnt, hist,
                     page_table=None):
    """Indexer scores of one query row per sequence, kept only where they can
    still be among the row's k largest: cand[r, :cand_cnt[r]] holds
    (order key << 32) | (0xFFFFFFFF - position) (read as int64), and hist
    counts every score's first digit."""
    rows, H_I, d_I = q_idx.shape
    pool_pages = k_idx_cache.shape[0] // 64
    st = lib().sa_index_candidates(_p(q_idx), _p(w), _p(k_idx_cache), pool_pages, _dtype_code(q_idx),
                                   _p(page_table), pages_per_seq, _p(n_visible), rows, H_I, d_I, k,
                                   cand.stride(0), _p(cand), _p(cand_cnt), _p(hist), _stream())
    _check("sa_index_candidates", st)
    return cand


def topk_from_candidates(cand, cand_cnt, n_valid, k: int, hist, idx_out=None):
    """Exact Top-K positions [rows, k] int32 (as topk_select) from the output of
    index_candidates; clears hist and cand_cnt."""
    rows = cand.shape[0]
    if idx_out is None:
        idx_out = torch.empty(rows, k, dtype=torch.int32, device=cand.device)
    st = lib().sa_topk_from_candidates(_p(cand), cand.stride(0), _p(cand_cnt), _p(n_valid), rows, k, _p(hist),
                                       _p(idx_out), _stream())
    _check("sa_topk_from_candidates", st)
    return idx_out


def sparse_mla_workspace_size(rows: int, H: int, k: int, d_c: int = 512) -> int:
    return int(lib().sa_sparse_mla_workspace_size(rows, H, k, d_c))


def _plain_cache(c_cache):
    if c_cache.dtype == torch.float8_e4m3fn:
        raise ValueError("an e4m3 cache needs c_scale")


def _mla_args(q_lat, q_rope, c_cache, kr_cache, idx, out, lse):
    _plain_cache(c_cache)
    rows, H, d_c = q_lat.shape
    d_R = q_rope.shape[2]
    k = idx.shape[1]
    if out is None:
        out = torch.empty(rows, H, d_c, dtype=torch.float32, device=q_lat.device)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"sparse MLA output must be float32 or bfloat16, not {out.dtype}")
    pool_pages = c_cache.shape[0] // 64
    return rows, H, d_c, d_R, k, out, lse, pool_pages


def sparse_mla_decode(q_lat, q_rope, c_cache, kr_cache, idx, scale: float, pages_per_seq: int, page_table=None,
                      seq_of_row=None, out=None, lse=None, workspace=None, c_scale=None):
    """Sparse MLA (latent aggregate) [rows, H, d_c], fp32 (or bf16 when `out`
    is a bf16 tensor); optional lse [rows, H].  With `c_scale` the cache is the
    quantised one of mla_cache_write (workspace: sparse_mla_q8_workspace_size)."""
    if c_scale is not None:
        return _sparse_mla_q8(q_lat, q_rope, c_cache, c_scale, kr_cache, idx, scale, pages_per_seq, page_table,
                              seq_of_row, out, lse, workspace)
    rows, H, d_c, d_R, k, out, lse, pool_pages = _mla_args(q_lat, q_rope, c_cache, kr_cache, idx, out, lse)
    need = sparse_mla_workspace_size(rows, H, k, d_c)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_lat.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    name = "sa_sparse_mla_decode_bf16" if out.dtype == torch.bfloat16 else "sa_sparse_mla_decode"
    st = getattr(lib(), name)(_p(q_lat), _p(q_rope), _p(c_cache), c_cache.stride(0), _p(kr_cache),
                              kr_cache.stride(0), pool_pages, _p(page_table), pages_per_seq, _p(seq_of_row),
                              _p(idx), rows, H, k, d_c, d_R, float(scale), _p(out), _p(lse), _p(workspace),
                              wbytes, _stream())
    _check(name, st)
    return out


def sparse_mla_prefill_workspace_size(rows: int, H: int, k: int, d_c: int = 512) -> int:
    return int(lib().sa_sparse_mla_prefill_workspace_size(rows, H, k, d_c))


def sparse_mla_prefill(q_lat, q_rope, c_cache, kr_cache, idx, scale: float, pages_per_seq: int, page_table=None,
                       seq_of_row=None, out=None, lse=None, workspace=None, c_scale=None):
    """sparse_mla_decode for many rows: one key split per row, but with `c_scale`
    as many as sparse_mla_decode takes (workspace: sparse_mla_q8_workspace_size)."""
    if c_scale is not None:
        return _sparse_mla_q8(q_lat, q_rope, c_cache, c_scale, kr_cache, idx, scale, pages_per_seq, page_table,
                              seq_of_row, out, lse, workspace)
    rows, H, d_c, d_R, k, out, lse, pool_pages = _mla_args(q_lat, q_rope, c_cache, kr_cache, idx, out, lse)
    if workspace is None and rows > 0:
        workspace = torch.empty(sparse_mla_prefill_workspace_size(rows, H, k, d_c), dtype=torch.uint8,
                                device=q_lat.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    name = "sa_sparse_mla_prefill_bf16" if out.dtype == torch.bfloat16 else "sa_sparse_mla_prefill"
    st = getattr(lib(), name)(_p(q_lat), _p(q_rope), _p(c_cache), c_cache.stride(0), _p(kr_cache),
                              kr_cache.stride(0), pool_pages, _p(page_table), pages_per_seq, _p(seq_of_row),
                              _p(idx), rows, H, k, d_c, d_R, float(scale), _p(out), _p(lse), _p(workspace),
                              wbytes, _stream())
    _check(name, st)
    return out


def dense_mla_workspace_size(rows: int, H: int, L_max: int, d_c: int = 512) -> int:
    return int(lib().sa_dense_mla_workspace_size(rows, H, L_max, d_c))


def dense_mla_decode(q_lat, q_rope, c_cache, kr_cache, n_visible, L_max: int, scale: float, pages_per_seq: int,
                     page_table=None, seq_of_row=None, out=None, lse=None, workspace=None, c_scale=None):
    """Dense MLA over every visible position (the short-sequence mode): row r
    attends to positions 0 .. n_visible[r]-1.  [rows, H, d_c] fp32.  With
    `c_scale` the cache is the quantised one of mla_cache_write (`out` may then
    be bf16; workspace: dense_mla_q8_workspace_size)."""
    if c_scale is not None:
        return _dense_mla_q8(q_lat, q_rope, c_cache, c_scale, kr_cache, n_visible, L_max, scale, pages_per_seq,
                             page_table, seq_of_row, out, lse, workspace)
    _plain_cache(c_cache)
    rows, H, d_c = q_lat.shape
    d_R = q_rope.shape[2]
    if out is None:
        out = torch.empty(rows, H, d_c, dtype=torch.float32, device=q_lat.device)
    pool_pages = c_cache.shape[0] // 64
    if workspace is None and rows > 0:
        workspace = torch.empty(dense_mla_workspace_size(rows, H, L_max, d_c), dtype=torch.uint8,
                                device=q_lat.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().sa_dense_mla_decode(_p(q_lat), _p(q_rope), _p(c_cache), c_cache.stride(0), _p(kr_cache),
                                   kr_cache.stride(0), pool_pages, _p(page_table), pages_per_seq, _p(seq_of_row),
                                   _p(n_visible), rows, H, L_max, d_c, d_R, float(scale), _p(out), _p(lse),
                                   _p(workspace), wbytes, _stream())
    _check("sa_dense_mla_decode", st)
    return out


def mla_absorb_query(q_c, U_K, q_lat=None):
    """q_lat[r,h,:] = U_K[h]^T q_c[r,h,:]: q_c [rows,H,d_C] bf16, U_K [H,d_C,d_c] bf16 -> [rows,H,d_c] bf16."""
    rows, H, d_C = q_c.shape
    d_c = U_K.shape[2]
    if q_lat is None:
        q_lat = torch.empty(rows, H, d_c, dtype=torch.bfloat16, device=q_c.device)
    _check("sa_mla_absorb_query", lib().sa_mla_absorb_query(_p(q_c), _p(U_K), rows, H, d_C, d_c, _p(q_lat), _stream()))
    return q_lat


def mla_up_project(o_lat, U_V, out=None):
    """out[r,h,:] = U_V[h] o_lat[r,h,:]: o_lat [rows,H,d_c] fp32 or bf16, U_V [H,d_v,d_c] bf16 -> [rows,H,d_v] fp32."""
    rows, H, d_c = o_lat.shape
    d_v = U_V.shape[1]
    if out is None:
        out = torch.empty(rows, H, d_v, dtype=torch.float32, device=o_lat.device)
    if o_lat.dtype == torch.bfloat16:
        name = "sa_mla_up_project_bf16"
    elif o_lat.dtype == torch.float32:
        name = "sa_mla_up_project"
    else:
        raise TypeError(f"o_lat must be float32 or bfloat16, not {o_lat.dtype}")
    _check(name, getattr(lib(), name)(_p(o_lat), _p(U_V), rows, H, d_c, d_v, _p(out), _stream()))
    return out


def sparse_mla_decode_static(q_lat, q_rope, c_cache, kr_cache, idx, scale: float, pages_per_seq: int,
                             page_table=None, seq_of_row=None, out=None, lse=None):
    """sparse_mla_decode without a workspace: for callers that cannot allocate
    device memory, the split-key partial states go to the library's static
    device array (STATIC_SCRATCH_BYTES).  Calls share that array, so calls that
    may overlap on the GPU must be ordered on one stream.  ``out`` and ``lse``
    can be passed in so that the call itself allocates nothing."""
    rows, H, d_c, d_R, k, out, lse, pool_pages = _mla_args(q_lat, q_rope, c_cache, kr_cache, idx, out, lse)
    need = sparse_mla_workspace_size(rows, H, k, d_c)
    if need > STATIC_SCRATCH_BYTES:
        raise ValueError(f"sparse_mla_decode_static: {rows} rows x {H} heads x k={k} need {need} bytes of "
                         f"split-key state, the static array holds {STATIC_SCRATCH_BYTES}; "
                         "use sparse_mla_decode with a workspace")
    st = lib().sa_sparse_mla_decode_static(_p(q_lat), _p(q_rope), _p(c_cache), c_cache.stride(0), _p(kr_cache),
                                           kr_cache.stride(0), pool_pages, _p(page_table), pages_per_seq,
                                           _p(seq_of_row), _p(idx), rows, H, k, d_c, d_R, float(scale), _p(out),
                                           _p(lse), _stream())
    _check("sa_sparse_mla_decode_static", st)
    return out


def block_mean_pool(K, block: int = 64, pooled=None):
    """Mean-pooled complete blocks: K [B, L, H, D] bf16 -> [B, H, L//block, D] fp32."""
    B, L, H, D = K.shape
    nb = L // block
    if pooled is None:
        pooled = torch.empty(B, H, max(nb, 1), D, dtype=torch.float32, device=K.device)
    st = lib().sa_block_mean_pool(_p(K), K.stride(0), K.stride(1), K.stride(2), B, L, H, D, block, _p(pooled),
                                  pooled.shape[2], _stream())
    _check("sa_block_mean_pool", st)
    return pooled


def block_sparse_attn(q, pooled, K, V, block: int, top_blocks: int, sink_blocks: int, window: int, scale: float,
                      out=None, sel_blocks=None):
    """Block-sparse decode of the query at position L-1: out [B, H, D] fp32."""
    B, L, H, D = K.shape
    if out is None:
        out = torch.empty(B, H, D, dtype=torch.float32, device=q.device)
    st = lib().sa_block_sparse_attn(_p(q), _p(pooled), pooled.shape[2], _p(K), _p(V), K.stride(0), K.stride(1),
                                    K.stride(2), B, H, D, L, block, top_blocks, sink_blocks, window, float(scale),
                                    _p(out), _p(sel_blocks), _stream())
    _check("sa_block_sparse_attn", st)
    return out


def nsa_compress(K, V, block: int = 64, Kc=None, Vc=None):
    """NSA compressed cache: bf16 block means of K and V [B, L, H_kv, D] ->
    Kc, Vc [B, H_kv, L//block, D] bf16 (complete blocks only)."""
    B, L, Hkv, D = K.shape
    nb = L // block
    if Kc is None:
        Kc = torch.empty(B, Hkv, max(nb, 1), D, dtype=torch.bfloat16, device=K.device)
    if Vc is None:
        Vc = torch.empty_like(Kc)
    if V.stride() != K.stride() or not (Kc.is_contiguous() and Vc.is_contiguous()):
        raise ValueError("K and V must share one layout; Kc and Vc must be contiguous")
    st = lib().sa_nsa_compress(_p(K), _p(V), K.stride(0), K.stride(1), K.stride(2), B, L, Hkv, D, block, _p(Kc),
                               _p(Vc), Kc.shape[2], _stream())
    _check("sa_nsa_compress", st)
    return Kc, Vc


def nsa_decode(q, K, V, Kc, Vc, gates, block: int, top_blocks: int, window: int, scale: float, out=None,
               sel_blocks=None):
    """NSA three-branch decode of the query at position L-1 of every head:
    q [B, H, D] bf16, K and V [B, L, H_kv, D] bf16, Kc and Vc from
    nsa_compress, gates [B, H, 3] fp32 -> out [B, H, D] fp32."""
    B, L, Hkv, D = K.shape
    H = q.shape[1]
    if V.stride() != K.stride() or not (Kc.is_contiguous() and Vc.is_contiguous()):
        raise ValueError("K and V must share one layout; Kc and Vc must be contiguous")
    if out is None:
        out = torch.empty(B, H, D, dtype=torch.float32, device=q.device)
    st = lib().sa_nsa_decode(_p(q), _p(K), _p(V), K.stride(0), K.stride(1), K.stride(2), _p(Kc), _p(Vc),
                             Kc.shape[2], _p(gates), B, H, Hkv, D, L, block,
                             top_blocks, window, float(scale), _p(out), _p(sel_blocks), _stream())
    _check("sa_nsa_decode", st)
    return out


def csa_compress(Ca, Cb, Za, Zb, Ba, Bb, m: int, out, out_seq_stride: int, out_row_stride: int, g0: int = 0,
                 g1: Optional[int] = None):
    """CSA compressed entries g0 .. g1-1 of every sequence: streams [S, L, c]
    bf16 (one layout for all four), biases [m, c] fp32; written into `out`
    (bf16 or e4m3) at s*out_seq_stride + g*out_row_stride (elements)."""
    S, L, c = Ca.shape
    if not (Cb.stride() == Za.stride() == Zb.stride() == Ca.stride()):
        raise ValueError("the four streams must share one layout")
    g1 = L // m if g1 is None else g1
    code = 1 if out.dtype == torch.float8_e4m3fn else (2 if out.dtype == torch.bfloat16 else -1)
    st = lib().sa_csa_compress(_p(Ca), _p(Cb), _p(Za), _p(Zb), Ca.stride(0), Ca.stride(1), _p(Ba), _p(Bb), S, L, m,
                               c, g0, g1, _p(out), code, out_seq_stride, out_row_stride, _stream())
    _check("sa_csa_compress", st)
    return out


def csa_window_index(topk_idx, raw_len, window: int, win_base: int, idx_out=None):
    """[rows, k + window] int32: the selected entries, then the window slots."""
    rows, k = topk_idx.shape
    if idx_out is None:
        idx_out = torch.empty(rows, k + window, dtype=torch.int32, device=topk_idx.device)
    st = lib().sa_csa_window_index(_p(topk_idx), rows, k, _p(raw_len), window, win_base, _p(idx_out), _stream())
    _check("sa_csa_window_index", st)
    return idx_out


def _need(t, name: str, dtypes, shape=None, contiguous=True):
    """Check one tensor argument: on the current device, of an allowed dtype,
    of the given shape and, unless strides are passed on, contiguous."""
    dev = t.get_device()  # (-1: not on a GPU)
    if dev >= 0 and dev == torch._C._cuda_getDevice() and t.dtype in dtypes and (
            shape is None or t.shape == shape) and (not contiguous or t.is_contiguous()):
        return
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current CUDA device, not on {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


# (torch before 2.7 has no float8_e8m0fnu)
_SCALE_TYPES = (torch.uint8,) + ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ())
_POOL_TYPES = (torch.float8_e4m3fn, torch.bfloat16)
_IO_TYPES = (torch.bfloat16, torch.float32)
_F32, _BF16, _I32 = (torch.float32,), (torch.bfloat16,), (torch.int32,)


def _need_cache(c_cache, c_scale, kr_cache, pages_per_seq, page_table, seq_of_row, rows):
    """Check a latent cache; return (dtype code, c_ld, scale_ld, kr_ld, pool_pages)."""
    n = c_cache.shape[0]
    quantised = c_cache.dtype == torch.float8_e4m3fn
    if quantised != (c_scale is not None):
        raise ValueError("an e4m3 cache needs c_scale, a bf16 cache has none")
    if n == 0 or n % 64:
        raise ValueError(f"the cache holds whole pages of 64 rows, not {n} rows")
    _need(c_cache, "c_cache", _POOL_TYPES, (n, 512), False)
    _need(kr_cache, "kr_cache", _BF16, (n, 64), False)
    (c_ld, one), (kr_ld, one_kr), s_ld = c_cache.stride(), kr_cache.stride(), 0
    if quantised:
        _need(c_scale, "c_scale", _SCALE_TYPES, (n, 4), False)
        s_ld, one_s = c_scale.stride()
        one *= one_s
    if one != 1 or one_kr != 1:
        raise ValueError("the dims of a cache row must be contiguous")
    if seq_of_row is not None:
        _need(seq_of_row, "seq_of_row", _I32, (rows,))
    if page_table is not None:
        seqs = page_table.shape[0]
        _need(page_table, "page_table", _I32, (seqs, pages_per_seq))
        if seq_of_row is None and seqs < rows:
            raise ValueError(f"page_table has {seqs} sequences for {rows} rows")
    return SA_E4M3 if quantised else SA_BF16, c_ld, s_ld, kr_ld, n // 64


def _need_tables(cos, sin, half) -> int:
    """Check the tables of `half` pairs; return their number of positions."""
    shape = (cos.shape[0], half)
    _need(cos, "cos", _F32, shape)
    _need(sin, "sin", _F32, shape)
    return shape[0]


def _heads_out(x, out):
    """(output of per-head rows x [tokens, H, D], made when not given, token
    and head strides of x and of it)."""
    tokens, H, D = x.shape
    xt, xh, one = x.stride()
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        ot, oh = H * D, D
    else:
        _need(out, "output", (x.dtype,), (tokens, H, D), contiguous=False)
        ot, oh, one_out = out.stride()
        if (ot == 0 and tokens > 1) or (oh == 0 and H > 1):
            raise ValueError("an output must not be a broadcast view")
        one *= one_out
    if D > 1 and one != 1:
        raise ValueError("the dims of a head must be contiguous")
    return out, (x.data_ptr(), xt, xh, out.data_ptr(), ot, oh, H)


def _code(t) -> int:
    return SA_F32 if t.dtype == torch.float32 else SA_BF16


def qk_norm_rope(q, k, cos, sin, positions, q_weight=None, k_weight=None, eps: float = 1e-6, norm: bool = True,
                 rope_start: int = 0, interleaved: bool = False, q_out=None, k_out=None):
    """Per-head RMS norm (skipped if not `norm`) and rotary rotation of queries
    q [tokens, H_q, D] and keys k [tokens, H_k, D] (or None), bf16 or fp32, in
    one launch.  Dims rope_start .. rope_start + 2*cos.shape[1] - 1 are rotated
    by row positions[t] of cos and sin [n_pos, rope_dims/2] fp32, in split
    halves or interleaved pairs; cos = sin = None: no rotation.  Token and
    head strides are free; q_out and k_out may be q and k.  Returns (q_out, k_out)."""
    tokens, _, D = q.shape
    _need(q, "q", _IO_TYPES, None, False)
    q_out, queries = _heads_out(q, q_out)
    keys = (None, 0, 0, None, 0, 0, 0)
    if k is not None:
        _need(k, "k", (q.dtype,), (tokens, k.shape[1], D), False)
        k_out, keys = _heads_out(k, k_out)
    else:
        k_out = None
    if q_weight is not None:
        _need(q_weight, "q_weight", _F32, (D,))
    if k_weight is not None:
        _need(k_weight, "k_weight", _F32, (D,))
    n_pos = half = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None and cos.shape[1]:
        half = cos.shape[1]
        n_pos = _need_tables(cos, sin, half)
        _need(positions, "positions", _I32, (tokens,))
    st = lib().sa_qk_norm_rope(*queries, *keys, _code(q), _p(q_weight), _p(k_weight), 1 if norm else 0, eps, _p(cos),
                               _p(sin), n_pos, _p(positions), tokens, D, rope_start, 2 * half, 1 if interleaved else 0,
                               _stream())
    _check("sa_qk_norm_rope", st)
    return q_out, k_out


def mla_cache_write(c, kr, c_cache, kr_cache, slots, pages_per_seq: int, cos, sin, positions=None, weight=None,
                    eps: float = 1e-6, norm: bool = True, interleaved: bool = False, c_scale=None, page_table=None,
                    seq_of_row=None):
    """Write tokens into the latent cache: c [tokens, 512] RMS-normalised
    (skipped if not `norm`) and stored as bf16, or as e4m3 codes with a scale
    byte per 128 dims when c_scale ([rows, 4] uint8 or float8_e8m0fnu) is
    given; kr [tokens, 64] rotated by row positions[t] (None: slots[t]) of
    cos and sin [n_pos, 32].  slots [tokens] int32: position of the token in
    sequence seq_of_row[t] (None: t), -1: skip the token; two tokens of one
    call must not name the same row.  Without `norm` a weight still applies."""
    tokens = c.shape[0]
    _need(c, "c", _IO_TYPES, (tokens, 512), False)
    _need(kr, "kr", (c.dtype,), (tokens, 64), False)
    if c.stride(1) != 1 or kr.stride(1) != 1:
        raise ValueError("the dims of a token must be contiguous")
    _need(slots, "slots", _I32, (tokens,))
    if positions is not None:
        _need(positions, "positions", _I32, (tokens,))
    if weight is not None:
        _need(weight, "weight", _F32, (512,))
    n_pos = _need_tables(cos, sin, 32)
    dt, c_ld, s_ld, kr_ld, pool = _need_cache(c_cache, c_scale, kr_cache, pages_per_seq, page_table, seq_of_row, tokens)
    c_in_ld, kr_in_ld = (c.stride(0), kr.stride(0)) if tokens > 1 else (512, 64)
    st = lib().sa_mla_cache_write(_p(c), c_in_ld, _p(kr), kr_in_ld, _code(c), _p(weight),
                                  1 if norm else 0, eps, _p(cos), _p(sin), n_pos, _p(positions),
                                  int(bool(interleaved)), _p(c_cache), dt, c_ld, _p(c_scale), s_ld, _p(kr_cache), kr_ld,
                                  pool, _p(page_table), pages_per_seq, _p(seq_of_row), _p(slots), tokens, 512, 64,
                                  _stream())
    _check("sa_mla_cache_write", st)


def mla_cache_read(c_cache, kr_cache, idx, pages_per_seq: int, c_scale=None, page_table=None, seq_of_row=None,
                   c_out=None, kr_out=None):
    """Rows of the latent cache at positions idx [rows, k] int32 (-1: zeros) of
    sequence seq_of_row[r], as bf16: (c [rows, k, 512], kr [rows, k, 64])."""
    rows, k = idx.shape
    _need(idx, "idx", _I32)
    dt, c_ld, s_ld, kr_ld, pool = _need_cache(c_cache, c_scale, kr_cache, pages_per_seq, page_table, seq_of_row, rows)
    if c_out is None:
        c_out = torch.empty(rows, k, 512, dtype=torch.bfloat16, device=idx.device)
    else:
        _need(c_out, "c_out", _BF16, (rows, k, 512))
    if kr_out is None:
        kr_out = torch.empty(rows, k, 64, dtype=torch.bfloat16, device=idx.device)
    else:
        _need(kr_out, "kr_out", _BF16, (rows, k, 64))
    st = lib().sa_mla_cache_read(_p(c_cache), dt, c_ld, _p(c_scale), s_ld, _p(kr_cache), kr_ld, pool, _p(page_table),
                                 pages_per_seq, _p(seq_of_row), _p(idx), rows, k, 512, 64, _p(c_out), _p(kr_out),
                                 _stream())
    _check("sa_mla_cache_read", st)
    return c_out, kr_out


def sparse_mla_q8_workspace_size(rows: int, H: int, k: int) -> int:
    return int(lib().sa_sparse_mla_q8_workspace_size(rows, H, k))


def dense_mla_q8_workspace_size(rows: int, H: int, L_max: int) -> int:
    return int(lib().sa_dense_mla_q8_workspace_size(rows, H, L_max))


def tree_mla_workspace_size(B: int, T: int, H: int, L_max: int) -> int:
    return int(lib().sa_tree_mla_workspace_size(B, T, H, L_max))


def _latent_io(q_lat, q_rope, out, lse, workspace, need: int):
    """Check queries [..., H, 512] / [..., H, 64]; make the output and the workspace when not given."""
    lead = tuple(q_lat.shape[:-1])
    _need(q_lat, "q_lat", _BF16, lead + (512,))
    _need(q_rope, "q_rope", _BF16, lead + (64,))
    if out is None:
        out = torch.empty(lead + (512,), dtype=torch.float32, device=q_lat.device)
    else:
        _need(out, "out", _IO_TYPES, lead + (512,))
    if lse is not None:
        _need(lse, "lse", _F32, lead)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_lat.device)
    if workspace is not None:
        _need(workspace, "workspace", (workspace.dtype,))
    return out, workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def _sparse_mla_q8(q_lat, q_rope, c_cache, c_scale, kr_cache, idx, scale, pages_per_seq, page_table, seq_of_row, out,
                   lse, workspace):
    rows, H, _ = q_lat.shape
    k = idx.shape[1]
    _need(idx, "idx", _I32, (rows, k))
    out, workspace, wbytes = _latent_io(q_lat, q_rope, out, lse, workspace, sparse_mla_q8_workspace_size(rows, H, k))
    _, c_ld, s_ld, kr_ld, pool = _need_cache(c_cache, c_scale, kr_cache, pages_per_seq, page_table, seq_of_row, rows)
    st = lib().sa_sparse_mla_q8(_p(q_lat), _p(q_rope), _p(c_cache), c_ld, _p(c_scale), s_ld, _p(kr_cache), kr_ld, pool,
                                _p(page_table), pages_per_seq, _p(seq_of_row), _p(idx), rows, H, k, 512, 64,
                                float(scale), _p(out), _code(out), _p(lse), _p(workspace), wbytes, _stream())
    _check("sa_sparse_mla_q8", st)
    return out


def _dense_mla_q8(q_lat, q_rope, c_cache, c_scale, kr_cache, n_visible, L_max, scale, pages_per_seq, page_table,
                  seq_of_row, out, lse, workspace):
    rows, H, _ = q_lat.shape
    _need(n_visible, "n_visible", _I32, (rows,))
    out, workspace, wbytes = _latent_io(q_lat, q_rope, out, lse, workspace, dense_mla_q8_workspace_size(rows, H, L_max))
    _, c_ld, s_ld, kr_ld, pool = _need_cache(c_cache, c_scale, kr_cache, pages_per_seq, page_table, seq_of_row, rows)
    st = lib().sa_dense_mla_q8(_p(q_lat), _p(q_rope), _p(c_cache), c_ld, _p(c_scale), s_ld, _p(kr_cache), kr_ld, pool,
                               _p(page_table), pages_per_seq, _p(seq_of_row), _p(n_visible), rows, H, L_max, 512, 64,
                               float(scale), _p(out), _code(out), _p(lse), _p(workspace), wbytes, _stream())
    _check("sa_dense_mla_q8", st)
    return out


def tree_mla_decode(q_lat, q_rope, c_cache, kr_cache, n_past, tree_mask, L_max: int, scale: float, pages_per_seq: int,
                    n_draft=None, c_scale=None, page_table=None, seq_of_row=None, out=None, lse=None, workspace=None):
    """MLA attention of drafted tokens: q_lat [B, T, H, 512], q_rope [B, T, H, 64]
    bf16.  Token i of tree b attends to cached positions 0 .. n_past[b]-1 and to
    the drafted tokens j < n_draft[b] (None: T), cached at n_past[b] + j, with
    tree_mask[b, i, j] nonzero (uint8 or bool [B, T, T]; None: j <= i).  The
    cache is bf16, or e4m3 with `c_scale`.  [B, T, H, 512] fp32 (or bf16 when
    `out` is a bf16 tensor); rows i >= n_draft[b] are left as they were."""
    B, T, H, _ = q_lat.shape
    _need(n_past, "n_past", _I32, (B,))
    if n_draft is not None:
        _need(n_draft, "n_draft", _I32, (B,))
    if tree_mask is not None:
        _need(tree_mask, "tree_mask", (torch.uint8, torch.bool), (B, T, T))
    out, workspace, wbytes = _latent_io(q_lat, q_rope, out, lse, workspace, tree_mla_workspace_size(B, T, H, L_max))
    dt, c_ld, s_ld, kr_ld, pool = _need_cache(c_cache, c_scale, kr_cache, pages_per_seq, page_table, seq_of_row, B)
    st = lib().sa_tree_mla_decode(_p(q_lat), _p(q_rope), _p(c_cache), dt, c_ld, _p(c_scale), s_ld, _p(kr_cache), kr_ld,
                                  pool, _p(page_table), pages_per_seq, _p(seq_of_row), _p(n_past), _p(n_draft),
                                  _p(tree_mask), B, T, H, L_max, 512, 64, float(scale), _p(out), _code(out), _p(lse),
                                  _p(workspace), wbytes, _stream())
    _check("sa_tree_mla_decode", st)
    return out
