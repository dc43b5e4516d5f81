// mla_latent.cu — MLA attention over the quantised latent cache (selected or
// all positions), and of a tree of drafted tokens over the quantised or the
// bf16 cache.
//
//   z_j = (q_lat . c_j + q_rope . kr_j) * scale,  out = sum_j softmax(z)_j c_j
//
// One warp per (row, head): lane l owns latent dims 16 l .. 16 l + 15 and RoPE
// dims 2 l, 2 l + 1; the keys go by one at a time under an online softmax.
#include "sa_device.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kPage = 64;

__device__ __forceinline__ int64_t latent_row(const LatentArgs& a, int seq, int p) {
    if (p / kPage >= a.pages_per_seq) return -2;
    const int64_t at = static_cast<int64_t>(seq) * a.pages_per_seq + p / kPage;
    const int64_t pg = a.page_table ? a.page_table[at] : at;
    if (pg < 0 || pg >= a.pool_pages) return -2;
    return pg * kPage + (p % kPage);
}

__device__ __forceinline__ void unpack8(uint4 u, float* v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__global__ void __launch_bounds__(128) mla_latent_kernel(const LatentArgs a) {
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t rows = static_cast<int64_t>(a.B) * a.T;
    if (item >= rows * a.H) return;
    const int64_t r = item / a.H;
    const int b = static_cast<int>(r / a.T), i = static_cast<int>(r % a.T);
    const int seq = a.seq_of_row ? a.seq_of_row[b] : b;
    const int nd = a.tree ? (a.n_draft ? a.n_draft[b] : a.T) : 0;
    if (a.tree && i >= nd) return;
    const int past = a.idx ? 0 : a.n_past[b];
    const int n = a.idx ? a.k : past + nd;
    float q[16], acc[16];
    const uint4* ql = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q_lat) + item * 512 + lane * 16);
    unpack8(ql[0], q);
    unpack8(ql[1], q + 8);
    const uint32_t qr = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q_rope) + item * 64)[lane];
    const float q0 = __uint_as_float(qr << 16), q1 = __uint_as_float(qr & 0xFFFF0000u);
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.f;
    float m = -INFINITY, l = 0.f;
    const float c2 = a.scale * 1.4426950408889634f;
    for (int t = 0; t < n; ++t) {
        int p = t;
        if (a.idx) {
            p = a.idx[r * a.k + t];
            if (p < 0) continue;
        } else if (t >= past) {
            const int j = t - past;
            if (!(a.tree_mask ? a.tree_mask[r * a.T + j] != 0 : j <= i)) continue;
        }
        int64_t row = latent_row(a, seq, p);
        if (row < 0) {
            if (lane == 0) record_error(a.err, kErrMlaIndex);
            row = 0;
        }
        float c[16];
        if (a.c_scale) {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c_cache) + row * a.c_ld + lane * 16);
            const uint32_t s2 = q8_scale_bf16x2(a.c_scale[row * a.s_ld + (lane >> 3)]);
            const uint2 a0 = e4m3x4_to_bf16x4(u.x, s2), a1 = e4m3x4_to_bf16x4(u.y, s2);
            const uint2 a2 = e4m3x4_to_bf16x4(u.z, s2), a3 = e4m3x4_to_bf16x4(u.w, s2);
            unpack8(make_uint4(a0.x, a0.y, a1.x, a1.y), c);
            unpack8(make_uint4(a2.x, a2.y, a3.x, a3.y), c + 8);
        } else {
            const uint4* u = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.c_cache) + row * a.c_ld + lane * 16);
            unpack8(u[0], c);
            unpack8(u[1], c + 8);
        }
        const uint32_t kr = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.kr_cache) + row * a.kr_ld)[lane];
        float z = q0 * __uint_as_float(kr << 16) + q1 * __uint_as_float(kr & 0xFFFF0000u);
#pragma unroll
        for (int j = 0; j < 16; ++j) z += q[j] * c[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        z *= c2;
        if (z > m) {
            const float f = exp2f(m - z);
            l *= f;
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[j] *= f;
            m = z;
        }
        const float w = exp2f(z - m);
        l += w;
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[j] += w * c[j];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (a.out_bf16) {
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = pack_bf16x2(acc[2 * j] * inv, acc[2 * j + 1] * inv);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out_bf16) + item * 512 + lane * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
        float4* dst = reinterpret_cast<float4*>(a.out + item * 512 + lane * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            dst[j] = make_float4(acc[4 * j] * inv, acc[4 * j + 1] * inv, acc[4 * j + 2] * inv, acc[4 * j + 3] * inv);
    }
    if (a.lse && lane == 0) a.lse[item] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t mla_latent_workspace_bytes(int, int, int, int, bool) { return 0; }

sa_status mla_latent_launch(const LatentArgs& a, void*, size_t, cudaStream_t st) {
    const int64_t items = static_cast<int64_t>(a.B) * a.T * a.H;
    mla_latent_kernel<<<static_cast<unsigned>((items + 3) / 4), 128, 0, st>>>(a);
    return launch_status(cudaGetLastError());
}

}  // namespace sa
