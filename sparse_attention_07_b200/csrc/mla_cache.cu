// mla_cache.cu — the latent cache written and read back.
//
// Write, per token: c -> y = c * rsqrt(mean(c^2) + eps) * w over the 512
// latent dims (or y = c), stored as bf16, or quantised per 128 dims: the scale
// is the smallest power of two 2^(e-127) with max|y| <= 448 * scale, the codes
// are y / scale rounded to e4m3 (nearest, ties to even) straight from fp32.  A
// power of two costs at most one bit of e4m3's range against a free scale and
// makes code * scale exact in bf16, so reading back adds no rounding.  The
// 64-dim RoPE key is rotated by cos/sin of the token's position and stored as
// bf16.  Row = page_table[seq][slot / 64] * 64 + slot % 64.
//
// Read: rows of the cache, gathered by position, as bf16.
//
// Both are bound by HBM on long chunks and by latency on short ones.  Write:
// one warp per token, 16 consecutive dims per lane, so a quantisation block is
// eight lanes (its maximum is three shuffles) and a quantised row leaves in
// one 512-byte warp store; 4096 tokens written and read back take 8.2 us, 32
// tokens 5.5 (launches, and the chain slot, page, row).
// Read: two slots per warp, all their loads in flight together; 61440 rows of
// the quantised cache take 21.5 us (5.2 TB/s; four slots per warp 23.3, one
// 22.9: the warps are short and most of their time is the chain index, page,
// row).
#include <cuda_fp8.h>

#include "sa_device.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kPage = 64;
constexpr int kDc = 512;
constexpr int kDr = 64;
constexpr int kThreads = 128;

// Pool row of a position, or -2 when it lies past the page table or its page
// is outside the pool.
__device__ __forceinline__ int64_t cache_row(const int32_t* table, int pages_per_seq, int64_t pool_pages, int seq, int p) {
    if (p / kPage >= pages_per_seq) return -2;
    const int64_t at = static_cast<int64_t>(seq) * pages_per_seq + p / kPage;
    const int64_t pg = table ? table[at] : at;
    if (pg < 0 || pg >= pool_pages) return -2;
    return pg * kPage + (p % kPage);
}

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]);
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 f = reinterpret_cast<const float4*>(p)[i];
        v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
}
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[i];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads) mla_cache_write_kernel(const CacheWriteArgs a) {
    const int token = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (token >= a.tokens) return;
    const int slot = a.slots[token];
    if (slot < 0) return;  // padded token
    const int seq = a.seq_of_row ? a.seq_of_row[token] : token;
    const int pos = a.positions ? a.positions[token] : slot;
    float v[16], w[16];
    load16(static_cast<const T*>(a.c) + token * a.c_in_ld + lane * 16, v);
    // RoPE pair of this lane: dims (2 lane, 2 lane + 1) or (lane, lane + 32)
    const T* kr = static_cast<const T*>(a.kr) + token * a.kr_in_ld;
    const int i0 = a.interleaved ? 2 * lane : lane, i1 = a.interleaved ? 2 * lane + 1 : lane + 32;
    const float ka = to_f(kr[i0]), kb = to_f(kr[i1]);
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = 1.f;
    if (a.weight) load16(a.weight + lane * 16, w);
    const bool pos_ok = pos >= 0 && pos < a.n_pos;
    const float cs = a.cos[static_cast<int64_t>(pos_ok ? pos : 0) * 32 + lane];
    const float sn = a.sin[static_cast<int64_t>(pos_ok ? pos : 0) * 32 + lane];
    const int64_t row = cache_row(a.page_table, a.pages_per_seq, a.pool_pages, seq, slot);
    if (lane == 0 && !pos_ok) record_error(a.err, kErrRopePos);
    if (row < 0) {
        if (lane == 0) record_error(a.err, kErrMlaIndex);
        return;
    }
    float r = 1.f;
    if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) ss += v[j] * v[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float f = norm_factor(ss * (1.f / kDc), a.eps);
        if (f != 1.f) {  // (of the whole warp alike)
            ss = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] *= f, ss += v[j] * v[j];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
        r = rsqrtf(ss * (1.f / kDc) + a.eps * f * f);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = v[j] * r * w[j];
    if (a.c_scale) {
        float m = 0.f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            m = fmaxf(m, fabsf(v[j]));
            bad |= !isfinite(v[j]);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        bad = (__ballot_sync(0xffffffffu, bad) >> (lane & 24) & 0xFFu) != 0;
        // m = f * 2^k: scale 2^(k-8), doubled when f > 1.75 (448 = 1.75 * 2^8)
        const uint32_t u = __float_as_uint(m);
        int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        e = m == 0.f ? 127 : max(e, 1);
        const float inv = bad ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = bad ? 0.f : v[4 * j + i] * inv;
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(t[0], t[1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(t[2], t[3]), __NV_SATFINITE, __NV_E4M3);
            q[j] = lo | (hi << 16);
        }
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.c_cache) + row * a.c_ld + lane * 16) =
            make_uint4(q[0], q[1], q[2], q[3]);
        if ((lane & 7) == 0) a.c_scale[row * a.s_ld + (lane >> 3)] = static_cast<uint8_t>(bad ? 255 : e);
    } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.c_cache) + row * a.c_ld + lane * 16);
        dst[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                            pack_bf16x2(v[6], v[7]));
        dst[1] = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                            pack_bf16x2(v[14], v[15]));
    }
    const float ra = ka * cs - kb * sn, rb = kb * cs + ka * sn;
    __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(a.kr_cache) + row * a.kr_ld;
    if (a.interleaved) {
        *reinterpret_cast<uint32_t*>(ko + 2 * lane) = pack_bf16x2(ra, rb);
    } else {
        ko[lane] = __float2bfloat16_rn(ra);
        ko[lane + 32] = __float2bfloat16_rn(rb);
    }
}

// Warp = kSlots consecutive slots of the flat [rows * k] index array.
constexpr int kSlots = 2;
template <bool kQ8>
__global__ void __launch_bounds__(kThreads) mla_cache_read_kernel(const CacheReadArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t total = static_cast<int64_t>(a.rows) * a.k;
    const int64_t o0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kSlots;
    if (o0 >= total) return;
    const int n = static_cast<int>(min(static_cast<int64_t>(kSlots), total - o0));
    int64_t row = -1;  // lane i < kSlots: slot o0 + i
    if (lane < n) {
        const int64_t o = o0 + lane;
        const int p = a.idx[o];
        if (p >= 0) {
            // a 64-bit division only where the count needs one
            const int r = static_cast<int>(total >> 32 ? o / a.k : static_cast<uint32_t>(o) / static_cast<uint32_t>(a.k));
            const int seq = a.seq_of_row ? a.seq_of_row[r] : r;
            row = cache_row(a.page_table, a.pages_per_seq, a.pool_pages, seq, p);
            if (row < 0) {
                record_error(a.err, kErrMlaIndex);
                row = 0;
            }
        }
    }
    constexpr int kPieces = kQ8 ? 1 : 2;
    uint4 u[kSlots][kPieces];
    uint32_t sc[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int64_t ri = __shfl_sync(0xffffffffu, row, i);
        sc[i] = 0;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) u[i][p] = make_uint4(0u, 0u, 0u, 0u);
        if (ri >= 0) {
            if (kQ8) {
                u[i][0] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c_cache) + ri * a.c_ld + lane * 16);
                sc[i] = a.c_scale[ri * a.s_ld + (lane >> 3)];
            } else {
#pragma unroll
                for (int p = 0; p < kPieces; ++p)
                    u[i][p] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.c_cache) + ri * a.c_ld +
                                                              p * 256 + lane * 8);
            }
        }
    }
    const int64_t rk = __shfl_sync(0xffffffffu, row, lane >> 3);  // RoPE keys: eight lanes per slot (none past kSlots)
    uint4 kr = make_uint4(0u, 0u, 0u, 0u);
    if (rk >= 0)
        kr = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.kr_cache) + rk * a.kr_ld + (lane & 7) * 8);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.c_out) + o0 * kDc;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        if (i >= n) break;
        if (kQ8) {
            const uint32_t s2 = q8_scale_bf16x2(sc[i]);
            const uint2 a0 = e4m3x4_to_bf16x4(u[i][0].x, s2), a1 = e4m3x4_to_bf16x4(u[i][0].y, s2);
            const uint2 a2 = e4m3x4_to_bf16x4(u[i][0].z, s2), a3 = e4m3x4_to_bf16x4(u[i][0].w, s2);
            uint4* dst = reinterpret_cast<uint4*>(out + i * kDc + lane * 16);
            dst[0] = make_uint4(a0.x, a0.y, a1.x, a1.y);
            dst[1] = make_uint4(a2.x, a2.y, a3.x, a3.y);
        } else {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) *reinterpret_cast<uint4*>(out + i * kDc + p * 256 + lane * 8) = u[i][p];
        }
    }
    if (a.kr_out && (lane >> 3) < n)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.kr_out) + (o0 + (lane >> 3)) * kDr + (lane & 7) * 8) = kr;
}

}  // namespace

sa_status mla_cache_write_launch(const CacheWriteArgs& a, sa_dtype dt, cudaStream_t st) {
    const unsigned blocks = static_cast<unsigned>((a.tokens + 3) / 4);
    if (dt == SA_F32)
        mla_cache_write_kernel<float><<<blocks, kThreads, 0, st>>>(a);
    else
        mla_cache_write_kernel<__nv_bfloat16><<<blocks, kThreads, 0, st>>>(a);
    return launch_status(cudaGetLastError());
}

sa_status mla_cache_read_launch(const CacheReadArgs& a, cudaStream_t st) {
    constexpr int64_t kPerBlock = kThreads / 32 * kSlots;
    const int64_t blocks = (static_cast<int64_t>(a.rows) * a.k + kPerBlock - 1) / kPerBlock;
    if (blocks > 0x7FFFFFFF) return SA_EUNSUPPORTED;
    if (a.c_scale)
        mla_cache_read_kernel<true><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a);
    else
        mla_cache_read_kernel<false><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a);
    return launch_status(cudaGetLastError());
}

}  // namespace sa
