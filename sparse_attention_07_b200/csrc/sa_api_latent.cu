// sa_api_latent.cu — C ABI of the operators around the latent cache
// (include/sparse_attn.h): argument checks on the host, then the launches.
#include <cmath>

#include "sa_device.cuh"
#include "sa_internal.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxPoolRows = int64_t(1) << 31;
constexpr int kMaxKeys = 1 << 30;  // of one row: tiles of them are counted in 32 bits

}  // namespace

using namespace sa;

extern "C" {

sa_status sa_qk_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                          int64_t q_out_token_stride, int64_t q_out_head_stride, int H_q, const void* k,
                          int64_t k_token_stride, int64_t k_head_stride, void* k_out, int64_t k_out_token_stride,
                          int64_t k_out_head_stride, int H_k, sa_dtype dtype, const float* q_weight,
                          const float* k_weight, int norm, float eps, const float* cos, const float* sin,
                          int64_t n_pos, const int32_t* positions, int tokens, int D, int rope_start, int rope_dims,
                          int interleaved, sa_stream_t stream) {
    if (tokens < 0 || H_q < 0 || H_k < 0 || D < 1 || rope_start < 0 || rope_dims < 0 || rope_dims % 2 != 0 ||
        rope_start > D - rope_dims || !(eps >= 0.f) || !std::isfinite(eps))
        return SA_EINVAL;
    if (dtype != SA_F32 && dtype != SA_BF16) return SA_EUNSUPPORTED;
    if (D > 512) return SA_EUNSUPPORTED;
    if (tokens == 0 || H_q + static_cast<int64_t>(H_k) == 0) return SA_OK;
    if ((H_q && (!q || !q_out)) || (H_k && (!k || !k_out))) return SA_EINVAL;
    if (rope_dims && (!cos || !sin || !positions || n_pos < 1)) return SA_EINVAL;
    const size_t e = dtype == SA_F32 ? 4 : 2;
    if (!aligned(q, e) || !aligned(q_out, e) || !aligned(k, e) || !aligned(k_out, e) || !aligned(q_weight, 4) ||
        !aligned(k_weight, 4) || !aligned(cos, 4) || !aligned(sin, 4) || !aligned(positions, 4))
        return SA_EINVAL;
    if (static_cast<int64_t>(tokens) * (H_q + static_cast<int64_t>(H_k)) > (int64_t(1) << 32)) return SA_EUNSUPPORTED;
    NormRopeArgs a = {};
    a.q = q;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.q_out = q_out;
    a.qo_ts = q_out_token_stride;
    a.qo_hs = q_out_head_stride;
    a.Hq = H_q;
    a.k = k;
    a.k_ts = k_token_stride;
    a.k_hs = k_head_stride;
    a.k_out = k_out;
    a.ko_ts = k_out_token_stride;
    a.ko_hs = k_out_head_stride;
    a.Hk = H_k;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.norm = norm;
    a.eps = eps;
    a.cos = cos;
    a.sin = sin;
    a.n_pos = n_pos;
    a.positions = positions;
    a.tokens = tokens;
    a.D = D;
    a.start = rope_start;
    a.rot = rope_dims;
    a.interleaved = interleaved;
    a.err = device_error_word();
    return norm_rope_launch(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

// The cache arguments shared by the calls below.
static sa_status check_cache(const void* c_cache, sa_dtype cache_dtype, int64_t c_ld, const uint8_t* c_scale,
                             int64_t scale_ld, const void* kr_cache, int64_t kr_ld, int64_t pool_pages,
                             const int32_t* page_table, int pages_per_seq, const int32_t* seq_of_row, int d_c, int d_R) {
    if (pages_per_seq < 1 || pool_pages < 1 || !c_cache || !kr_cache) return SA_EINVAL;
    if ((cache_dtype != SA_BF16 && cache_dtype != SA_E4M3) || d_c != 512 || d_R != 64) return SA_EUNSUPPORTED;
    if ((cache_dtype == SA_E4M3) != (c_scale != nullptr)) return SA_EINVAL;
    if (c_ld < d_c || kr_ld < d_R || kr_ld % 8 != 0 || !aligned(c_cache, 16) || !aligned(kr_cache, 16)) return SA_EINVAL;
    if (c_ld % (cache_dtype == SA_E4M3 ? 16 : 8) != 0) return SA_EINVAL;
    if (c_scale && (scale_ld < d_c / 128 || scale_ld % 4 != 0 || !aligned(c_scale, 4))) return SA_EINVAL;
    if (!aligned(page_table, 4) || !aligned(seq_of_row, 4)) return SA_EINVAL;
    if (pool_pages > kMaxPoolRows / 64 || c_ld > INT32_MAX || kr_ld > INT32_MAX) return SA_EUNSUPPORTED;
    return SA_OK;
}

sa_status sa_mla_cache_write(const void* c, int64_t c_in_ld, const void* kr, int64_t kr_in_ld, sa_dtype in_dtype,
                             const float* weight, int norm, float eps, const float* cos, const float* sin,
                             int64_t n_pos, const int32_t* positions, int interleaved, void* c_cache,
                             sa_dtype cache_dtype, int64_t c_ld, uint8_t* c_scale, int64_t scale_ld, void* kr_cache,
                             int64_t kr_ld, int64_t pool_pages, const int32_t* page_table, int pages_per_seq,
                             const int32_t* seq_of_row, const int32_t* slots, int tokens, int d_c, int d_R,
                             sa_stream_t stream) {
    if (tokens < 0 || !(eps >= 0.f) || !std::isfinite(eps) || n_pos < 1) return SA_EINVAL;
    if (tokens == 0) return SA_OK;
    const sa_status s = check_cache(c_cache, cache_dtype, c_ld, c_scale, scale_ld, kr_cache, kr_ld, pool_pages,
                                    page_table, pages_per_seq, seq_of_row, d_c, d_R);
    if (s != SA_OK) return s;
    if (in_dtype != SA_BF16 && in_dtype != SA_F32) return SA_EUNSUPPORTED;
    if (!c || !kr || !cos || !sin || !slots) return SA_EINVAL;
    const int64_t per16 = in_dtype == SA_F32 ? 4 : 8;  // elements per 16 bytes
    if (c_in_ld < d_c || kr_in_ld < d_R || c_in_ld % per16 != 0 || !aligned(c, 16) ||
        !aligned(kr, in_dtype == SA_F32 ? 4 : 2) || !aligned(weight, 16) || !aligned(cos, 4) || !aligned(sin, 4) ||
        !aligned(positions, 4) || !aligned(slots, 4))
        return SA_EINVAL;
    CacheWriteArgs a = {};
    a.c = c;
    a.c_in_ld = c_in_ld;
    a.kr = kr;
    a.kr_in_ld = kr_in_ld;
    a.weight = weight;
    a.norm = norm;
    a.eps = eps;
    a.cos = cos;
    a.sin = sin;
    a.n_pos = n_pos;
    a.positions = positions;
    a.interleaved = interleaved;
    a.c_cache = c_cache;
    a.c_ld = c_ld;
    a.c_scale = c_scale;
    a.s_ld = scale_ld;
    a.kr_cache = kr_cache;
    a.kr_ld = kr_ld;
    a.pool_pages = pool_pages;
    a.page_table = page_table;
    a.pages_per_seq = pages_per_seq;
    a.seq_of_row = seq_of_row;
    a.slots = slots;
    a.tokens = tokens;
    a.err = device_error_word();
    return mla_cache_write_launch(a, in_dtype, reinterpret_cast<cudaStream_t>(stream));
}

sa_status sa_mla_cache_read(const void* c_cache, sa_dtype cache_dtype, int64_t c_ld, const uint8_t* c_scale,
                            int64_t scale_ld, const void* kr_cache, int64_t kr_ld, int64_t pool_pages,
                            const int32_t* page_table, int pages_per_seq, const int32_t* seq_of_row,
                            const int32_t* idx, int rows, int k, int d_c, int d_R, void* c_out, void* kr_out,
                            sa_stream_t stream) {
    if (rows < 0 || k < 0) return SA_EINVAL;
    if (rows == 0 || k == 0) return SA_OK;
    const sa_status s = check_cache(c_cache, cache_dtype, c_ld, c_scale, scale_ld, kr_cache, kr_ld, pool_pages,
                                    page_table, pages_per_seq, seq_of_row, d_c, d_R);
    if (s != SA_OK) return s;
    if (!idx || !c_out || !aligned(idx, 4) || !aligned(c_out, 16) || !aligned(kr_out, 16)) return SA_EINVAL;
    CacheReadArgs a = {};
    a.c_cache = c_cache;
    a.c_ld = c_ld;
    a.c_scale = c_scale;
    a.s_ld = scale_ld;
    a.kr_cache = kr_cache;
    a.kr_ld = kr_ld;
    a.pool_pages = pool_pages;
    a.page_table = page_table;
    a.pages_per_seq = pages_per_seq;
    a.seq_of_row = seq_of_row;
    a.idx = idx;
    a.rows = rows;
    a.k = k;
    a.c_out = c_out;
    a.kr_out = kr_out;
    a.err = device_error_word();
    return mla_cache_read_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

static sa_status latent_attn(const void* q_lat, const void* q_rope, const void* c_cache, sa_dtype cache_dtype,
                             int64_t c_ld, const uint8_t* c_scale, int64_t scale_ld, const void* kr_cache,
                             int64_t kr_ld, int64_t pool_pages, const int32_t* page_table, int pages_per_seq,
                             const int32_t* seq_of_row, const int32_t* idx, const int32_t* n_past,
                             const int32_t* n_draft, const uint8_t* tree_mask, bool tree, int B, int T, int H, int k,
                             int d_c, int d_R, float scale, void* out, sa_dtype out_dtype, float* lse, void* workspace,
                             size_t workspace_bytes, sa_stream_t stream) {
    if (B < 0 || T < 1 || H < 1 || k < 1 || !std::isfinite(scale)) return SA_EINVAL;
    if (B == 0) return SA_OK;
    const sa_status s = check_cache(c_cache, cache_dtype, c_ld, c_scale, scale_ld, kr_cache, kr_ld, pool_pages,
                                    page_table, pages_per_seq, seq_of_row, d_c, d_R);
    if (s != SA_OK) return s;
    if (H > 128 || T > SA_TREE_MAX_TOKENS || k > kMaxKeys || (out_dtype != SA_F32 && out_dtype != SA_BF16)) return SA_EUNSUPPORTED;
    // (a length read on the device is cut to the page table and one page, which 32 bits hold)
    if (pages_per_seq > kMaxKeys / 64) return SA_EUNSUPPORTED;
    if (!q_lat || !q_rope || !out || (!idx && !n_past)) return SA_EINVAL;
    if (!aligned(q_lat, 16) || !aligned(q_rope, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(idx, 4) ||
        !aligned(n_past, 4) || !aligned(n_draft, 4))
        return SA_EINVAL;
    if (static_cast<int64_t>(B) * T > (int64_t(1) << 24)) return SA_EUNSUPPORTED;
    const size_t need = mla_latent_workspace_bytes(B, T, H, k);
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return SA_EINVAL;
    LatentArgs a = {};
    a.q_lat = q_lat;
    a.q_rope = q_rope;
    a.c_cache = c_cache;
    a.c_ld = c_ld;
    a.c_scale = c_scale;
    a.s_ld = scale_ld;
    a.kr_cache = kr_cache;
    a.kr_ld = kr_ld;
    a.page_table = page_table;
    a.pages_per_seq = pages_per_seq;
    a.pool_pages = pool_pages;
    a.seq_of_row = seq_of_row;
    a.idx = idx;
    a.k = k;
    a.n_past = n_past;
    a.n_draft = n_draft;
    a.tree_mask = tree_mask;
    a.tree = tree;
    a.B = B;
    a.T = T;
    a.H = H;
    a.scale = scale;
    a.out = out_dtype == SA_F32 ? static_cast<float*>(out) : nullptr;
    a.out_bf16 = out_dtype == SA_F32 ? nullptr : out;
    a.lse = lse;
    a.err = device_error_word();
    return mla_latent_launch(a, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t sa_sparse_mla_q8_workspace_size(int rows, int H, int k) {
    if (rows < 1 || H < 1 || k < 1 || k > kMaxKeys) return 0;
    return mla_latent_workspace_bytes(rows, 1, H, k);
}

sa_status sa_sparse_mla_q8(const void* q_lat, const void* q_rope, const void* c_cache, int64_t c_ld,
                           const uint8_t* c_scale, int64_t scale_ld, const void* kr_cache, int64_t kr_ld,
                           int64_t pool_pages, const int32_t* page_table, int pages_per_seq,
                           const int32_t* seq_of_row, const int32_t* idx, int rows, int H, int k, int d_c, int d_R,
                           float scale, void* out, sa_dtype out_dtype, float* lse, void* workspace,
                           size_t workspace_bytes, sa_stream_t stream) {
    if (rows > 0 && !idx) return SA_EINVAL;
    return latent_attn(q_lat, q_rope, c_cache, SA_E4M3, c_ld, c_scale, scale_ld, kr_cache, kr_ld, pool_pages,
                       page_table, pages_per_seq, seq_of_row, idx, nullptr, nullptr, nullptr, false, rows, 1, H, k,
                       d_c, d_R, scale, out, out_dtype, lse, workspace, workspace_bytes, stream);
}

size_t sa_dense_mla_q8_workspace_size(int rows, int H, int L_max) { return sa_tree_mla_workspace_size(rows, 1, H, L_max); }

sa_status sa_dense_mla_q8(const void* q_lat, const void* q_rope, const void* c_cache, int64_t c_ld,
                          const uint8_t* c_scale, int64_t scale_ld, const void* kr_cache, int64_t kr_ld,
                          int64_t pool_pages, const int32_t* page_table, int pages_per_seq, const int32_t* seq_of_row,
                          const int32_t* n_visible, int rows, int H, int L_max, int d_c, int d_R, float scale,
                          void* out, sa_dtype out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                          sa_stream_t stream) {
    return latent_attn(q_lat, q_rope, c_cache, SA_E4M3, c_ld, c_scale, scale_ld, kr_cache, kr_ld, pool_pages,
                       page_table, pages_per_seq, seq_of_row, nullptr, n_visible, nullptr, nullptr, false, rows, 1, H,
                       L_max, d_c, d_R, scale, out, out_dtype, lse, workspace, workspace_bytes, stream);
}

size_t sa_tree_mla_workspace_size(int B, int T, int H, int L_max) {
    if (B < 1 || T < 1 || H < 1 || L_max < 1 || L_max > kMaxKeys) return 0;
    return mla_latent_workspace_bytes(B, T, H, L_max);
}

sa_status sa_tree_mla_decode(const void* q_lat, const void* q_rope, const void* c_cache, sa_dtype cache_dtype,
                             int64_t c_ld, const uint8_t* c_scale, int64_t scale_ld, const void* kr_cache,
                             int64_t kr_ld, int64_t pool_pages, const int32_t* page_table, int pages_per_seq,
                             const int32_t* seq_of_row, const int32_t* n_past, const int32_t* n_draft,
                             const uint8_t* tree_mask, int B, int T, int H, int L_max, int d_c, int d_R, float scale,
                             void* out, sa_dtype out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                             sa_stream_t stream) {
    return latent_attn(q_lat, q_rope, c_cache, cache_dtype, c_ld, c_scale, scale_ld, kr_cache, kr_ld, pool_pages,
                       page_table, pages_per_seq, seq_of_row, nullptr, n_past, n_draft, tree_mask, true, B, T, H,
                       L_max, d_c, d_R, scale, out, out_dtype, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
