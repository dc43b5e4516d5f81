// norm_rope.cu — per-head RMS norm of queries and keys with the rotary
// rotation in the same pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w                    (per head, fp32)
//   out[d] = y[d], and for the pairs (a, b) of dims [start, start + rot):
//   out[a] = y[a] cos - y[b] sin,  out[b] = y[b] cos + y[a] sin
// with cos, sin of the token's position, pairs (i, i + rot/2) or, interleaved,
// (2i, 2i + 1).  Rounded once, to the storage type, at the end.
//
// Bound by HBM on chunks (each element read once and written once) and by
// launch and load latency on a decode step.  Each thread owns eight
// consecutive dims of a head (16-byte loads) and, for split pairs, loads the
// eight partner dims a second time: they are in lines its own lane group reads
// anyway, so that costs an L1 hit and no shuffle.  The cos/sin and weight
// values of a thread's dims stay in registers over up to kHeads heads of one
// token, whose loads are all in flight together.
#include "sa_device.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kThreads = 128;
constexpr int kVec = 8;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Position of a token, checked against the tables (row 0 and a recorded error
// when outside).
__device__ __forceinline__ int64_t table_row(const NormRopeArgs& a, int token) {
    const int p = a.positions[token];
    if (p < 0 || p >= a.n_pos) {
        record_error(a.err, kErrRopePos);
        return 0;
    }
    return p;
}

// One lane group (a power of two of lanes, `lanes` = D / 8 of them live) per
// (token, up to kHeads heads of q or of k).
template <typename T, int kHeads>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a, int group, int lanes) {
    const int per_cta = kThreads / group;
    const int nq = (a.Hq + kHeads - 1) / kHeads, nk = (a.Hk + kHeads - 1) / kHeads;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * per_cta + threadIdx.x / group;
    const int l = threadIdx.x % group;
    const bool live = item < static_cast<int64_t>(a.tokens) * (nq + nk);
    const int token = live ? static_cast<int>(item / (nq + nk)) : 0;
    const int part = live ? static_cast<int>(item % (nq + nk)) : 0;
    const bool is_k = part >= nq;
    const int h0 = (is_k ? part - nq : part) * kHeads, H = is_k ? a.Hk : a.Hq;
    const int d = l * kVec;
    const bool in = live && l < lanes;
    const T* x = static_cast<const T*>(is_k ? a.k : a.q) + token * (is_k ? a.k_ts : a.q_ts);
    T* y = static_cast<T*>(is_k ? a.k_out : a.q_out) + token * (is_k ? a.ko_ts : a.qo_ts);
    const int64_t hs = is_k ? a.k_hs : a.q_hs, ohs = is_k ? a.ko_hs : a.qo_hs;
    const float* w = is_k ? a.k_weight : a.q_weight;
    const int half = a.rot / 2, dr = d - a.start;
    const bool rot = in && dr >= 0 && dr < a.rot;
    const bool split = rot && !a.interleaved;
    const int dp = split ? (dr < half ? d + half : d - half) : d;  // the partner dims' start

    float v[kHeads][8], u[kHeads][8];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (in && h0 + i < H) {
            load8(x + (h0 + i) * hs + d, v[i]);
            if (split) load8(x + (h0 + i) * hs + dp, u[i]);
        }
    float wv[8], wu[8], c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) wv[j] = wu[j] = 1.f;
    if (in && w) {
        load8(w + d, wv);
        if (split) load8(w + dp, wu);
    }
    if (rot) {
        const int64_t row = table_row(a, token) * half;
        if (a.interleaved) {
            const float4 c4 = *reinterpret_cast<const float4*>(a.cos + row + dr / 2);
            const float4 s4 = *reinterpret_cast<const float4*>(a.sin + row + dr / 2);
            c[0] = c[1] = c4.x, c[2] = c[3] = c4.y, c[4] = c[5] = c4.z, c[6] = c[7] = c4.w;
            s[0] = s[1] = s4.x, s[2] = s[3] = s4.y, s[4] = s[5] = s4.z, s[6] = s[7] = s4.w;
        } else {
            load8(a.cos + row + (dr < half ? dr : dr - half), c);
            load8(a.sin + row + (dr < half ? dr : dr - half), s);
        }
    }
    __syncwarp();  // every load of the warp precedes its stores (the call may be in place)
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        float r = 1.f;
        if (a.norm) {
            float ss = 0.f;
            if (in && h0 + i < H)
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
            for (int o = group / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            r = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
        }
        if (!(in && h0 + i < H)) continue;
        float o8[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o8[j] = v[i][j] * r * wv[j];
        if (split) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = u[i][j] * r * wu[j];
                o8[j] = dr < half ? o8[j] * c[j] - p * s[j] : o8[j] * c[j] + p * s[j];
            }
        } else if (rot) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float p = o8[j], q = o8[j + 1];
                o8[j] = p * c[j] - q * s[j];
                o8[j + 1] = q * c[j] + p * s[j];
            }
        }
        store8(y + (h0 + i) * ohs + d, o8);
    }
}

// Any D up to 512, any strides and alignment: one warp per head, lane owns
// dims lane, lane + 32, ...
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const NormRopeArgs a) {
    constexpr int kMost = 16;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (item >= static_cast<int64_t>(a.tokens) * (a.Hq + a.Hk)) return;
    const int token = static_cast<int>(item / (a.Hq + a.Hk));
    int h = static_cast<int>(item % (a.Hq + a.Hk));
    const bool is_k = h >= a.Hq;
    if (is_k) h -= a.Hq;
    const T* x = static_cast<const T*>(is_k ? a.k : a.q) + token * (is_k ? a.k_ts : a.q_ts) + h * (is_k ? a.k_hs : a.q_hs);
    T* y = static_cast<T*>(is_k ? a.k_out : a.q_out) + token * (is_k ? a.ko_ts : a.qo_ts) + h * (is_k ? a.ko_hs : a.qo_hs);
    const float* w = is_k ? a.k_weight : a.q_weight;
    const int half = a.rot / 2;
    float v[kMost], u[kMost];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int d = lane + 32 * i, dr = d - a.start;
        v[i] = u[i] = 0.f;
        if (d < a.D) {
            v[i] = to_f(x[d]);
            if (dr >= 0 && dr < a.rot) u[i] = to_f(x[a.interleaved ? a.start + (dr ^ 1) : (dr < half ? d + half : d - half)]);
            ss += v[i] * v[i];
        }
    }
    __syncwarp();  // every load of the head precedes its stores (the call may be in place)
    float r = 1.f;
    if (a.norm) {
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
    }
    const int64_t row = a.rot ? table_row(a, token) * half : 0;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int d = lane + 32 * i, dr = d - a.start;
        if (d >= a.D) break;
        float o = v[i] * r * (w ? w[d] : 1.f);
        if (dr >= 0 && dr < a.rot) {
            const bool first = a.interleaved ? (dr & 1) == 0 : dr < half;
            const int dp = a.interleaved ? a.start + (dr ^ 1) : (first ? d + half : d - half);
            const int t = a.interleaved ? dr / 2 : (first ? dr : dr - half);
            const float p = u[i] * r * (w ? w[dp] : 1.f), c = a.cos[row + t], s = a.sin[row + t];
            o = first ? o * c - p * s : o * c + p * s;
        }
        put(y + d, o);
    }
}

template <typename T>
sa_status launch(const NormRopeArgs& a, cudaStream_t st) {
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    constexpr int kE = 16 / sizeof(T);  // elements per 16 bytes
    const int64_t strides = a.q_ts | a.q_hs | a.qo_ts | a.qo_hs | (a.Hk ? a.k_ts | a.k_hs | a.ko_ts | a.ko_hs : 0);
    // eight-dim pieces never straddle a border of the rotated range or of its halves
    const bool whole = a.D % 8 == 0 && a.D <= 256 && a.start % 8 == 0 &&
                       (a.interleaved ? a.rot % 8 == 0 : a.rot % 16 == 0);
    const bool vec = whole && strides % kE == 0 && al(a.q) && al(a.q_out) && al(a.q_weight) && al(a.k_weight) &&
                     (!a.Hk || (al(a.k) && al(a.k_out))) && (!a.rot || (al(a.cos) && al(a.sin)));
    if (!vec) {
        const int64_t warps = static_cast<int64_t>(a.tokens) * (a.Hq + a.Hk);
        norm_rope_any_kernel<T><<<static_cast<unsigned>((warps + 3) / 4), kThreads, 0, st>>>(a);
        return launch_status(cudaGetLastError());
    }
    const int lanes = a.D / kVec;
    int group = 1;
    while (group < lanes) group *= 2;
    const int64_t one = static_cast<int64_t>(a.tokens) * (a.Hq + a.Hk) * group / kThreads;
    auto blocks = [&](int heads) {
        const int64_t items = static_cast<int64_t>(a.tokens) * ((a.Hq + heads - 1) / heads + (a.Hk + heads - 1) / heads);
        return static_cast<unsigned>((items * group + kThreads - 1) / kThreads);
    };
    // four heads per group once that still fills every SM several times over
    if (one >= 4 * 8 * sm_count())
        norm_rope_kernel<T, 4><<<blocks(4), kThreads, 0, st>>>(a, group, lanes);
    else
        norm_rope_kernel<T, 1><<<blocks(1), kThreads, 0, st>>>(a, group, lanes);
    return launch_status(cudaGetLastError());
}

}  // namespace

sa_status norm_rope_launch(const NormRopeArgs& a, sa_dtype dt, cudaStream_t st) {
    return dt == SA_F32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace sa
