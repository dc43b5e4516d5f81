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
// launch and load latency on a decode step.  A lane owns two pieces of four
// consecutive dims of a head, each piece one load: for split pairs the piece at
// d and the one at d + rot/2, so both dims of a pair are in the lane that rotates
// them, with no shuffle, no second load, and a call in place needs no ordering
// between lanes.  The cos/sin and weight values of a
// lane's dims stay in registers over up to kHeads heads of one token, whose
// loads are all in flight together.  4096 tokens x 36 heads of 128 in bf16 take
// 19.9 us (3.9 TB/s; issue slots 69 percent busy), 1021 tokens x 129
// heads of 192 in fp32 36.7 us (5.5 TB/s), eight tokens 2.7 us.
#include "sa_device.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kThreads = 128;
constexpr int kVec = 4;  // dims of a piece

// A piece as it was loaded: 16 bytes of fp32 or 8 of bf16.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    using type = float4;
};
template <>
struct Raw<__nv_bfloat16> {
    using type = uint2;
};
template <typename T>
__device__ __forceinline__ typename Raw<T>::type load_piece(const T* p) {
    return *reinterpret_cast<const typename Raw<T>::type*>(p);
}
__device__ __forceinline__ void unpack(const float4& p, float (&v)[4]) { v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w; }
__device__ __forceinline__ void unpack(const uint2& p, float (&v)[4]) {
    v[0] = __uint_as_float(p.x << 16), v[1] = __uint_as_float(p.x & 0xFFFF0000u);
    v[2] = __uint_as_float(p.y << 16), v[3] = __uint_as_float(p.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store_piece(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_piece(__nv_bfloat16* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
// Times a power of two.
__device__ __forceinline__ void scale_piece(float4& p, float f) { p.x *= f, p.y *= f, p.z *= f, p.w *= f; }
__device__ __forceinline__ void scale_piece(uint2& p, float f) {
    const uint32_t f2 = pack_bf16x2(f, f);
    p.x = hmul2_bf16(p.x, f2), p.y = hmul2_bf16(p.y, f2);
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Row of the tables for position p (row 0 and a recorded error when outside).
__device__ __forceinline__ int64_t table_row(const NormRopeArgs& a, int p) {
    if (p < 0 || p >= a.n_pos) {
        record_error(a.err, kErrRopePos);
        return 0;
    }
    return p;
}

// One lane group (a power of two of lanes, `lanes` = D / 8 of them live) per
// (token, up to kHeads heads of q or of k).  Lanes below rot / 8 own the
// rotated dims, the others the rest of the head in order.
template <typename T, int kHeads, bool kInter>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a, int lg_group, int lanes) {
    const uint32_t nq = (a.Hq + kHeads - 1) / kHeads, nk = (a.Hk + kHeads - 1) / kHeads, parts = nq + nk;
    const uint64_t item = (static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x) >> lg_group;
    const int l = threadIdx.x & ((1 << lg_group) - 1);
    // the caller has checked that tokens * heads <= 2^32: a 32-bit division serves
    const uint32_t tok = static_cast<uint32_t>(item) / parts;
    const bool in = item >> 32 == 0 && tok < static_cast<uint32_t>(a.tokens) && l < lanes;
    const int token = in ? static_cast<int>(tok) : 0;
    const uint32_t part = in ? static_cast<uint32_t>(item) - tok * parts : 0;
    const bool is_k = part >= nq;
    const int h0 = static_cast<int>(is_k ? part - nq : part) * kHeads;
    const int n = in ? (is_k ? a.Hk : a.Hq) - h0 : 0;  // heads left for this group
    const int half = a.rot / 2;
    const bool rot = in && l * 8 < a.rot;
    int da, db;  // where the lane's two pieces start
    if (rot) {
        da = a.start + l * (kInter ? 8 : 4);
        db = da + (kInter ? 4 : half);
    } else {
        da = l * 8 - a.rot, db = da + 4;
        if (da >= a.start) da += a.rot;
        if (db >= a.start) db += a.rot;
    }
    const int pos = rot ? a.positions[token] : 0;

    using Raw4 = typename Raw<T>::type;
    Raw4 pa[kHeads], pb[kHeads];
    const int64_t hs = is_k ? a.k_hs : a.q_hs;
    const T* x = static_cast<const T*>(is_k ? a.k : a.q) + token * (is_k ? a.k_ts : a.q_ts) + h0 * hs + da;
#pragma unroll
    for (int i = 0; i < kHeads; ++i, x += hs) {
        pa[i] = pb[i] = Raw4{};
        if (i < n) pa[i] = load_piece(x), pb[i] = load_piece(x + (db - da));
    }
    float wa[4], wb[4], c[4], s[4];
    const float* w = is_k ? a.k_weight : a.q_weight;
#pragma unroll
    for (int j = 0; j < 4; ++j) wa[j] = wb[j] = c[j] = 1.f, s[j] = 0.f;
    if (in && w) unpack(load_piece(w + da), wa), unpack(load_piece(w + db), wb);
    if (rot) {
        const int64_t at = table_row(a, pos) * half + l * 4;  // four pairs either way
        unpack(load_piece(a.cos + at), c), unpack(load_piece(a.sin + at), s);
    }
    float r[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        float va[4], vb[4];
        unpack(pa[i], va), unpack(pb[i], vb);
        r[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i] += va[j] * va[j] + vb[j] * vb[j];
    }
    for (int o = 1 << lg_group >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < kHeads; ++i) r[i] += __shfl_xor_sync(0xffffffffu, r[i], o);
    const float inv = 1.f / static_cast<float>(a.D);
    bool outside = false;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) outside |= norm_factor(r[i] * inv, a.eps) != 1.f;
    if (__builtin_expect(a.norm && __any_sync(0xffffffffu, outside && n > 0), 0)) {
        // some head's sum of squares left fp32's range: scaled, and summed again
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const float f = norm_factor(r[i] * inv, a.eps);
            scale_piece(pa[i], f), scale_piece(pb[i], f);
            float va[4], vb[4], sum = 0.f;
            unpack(pa[i], va), unpack(pb[i], vb);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += va[j] * va[j] + vb[j] * vb[j];
            for (int o = 1 << lg_group >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            r[i] = rsqrtf(sum * inv + a.eps * f * f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kHeads; ++i) r[i] = a.norm ? rsqrtf(r[i] * inv + a.eps) : 1.f;
    }
    const int64_t ohs = is_k ? a.ko_hs : a.qo_hs;
    T* y = static_cast<T*>(is_k ? a.k_out : a.q_out) + token * (is_k ? a.ko_ts : a.qo_ts) + h0 * ohs + da;
#pragma unroll
    for (int i = 0; i < kHeads; ++i, y += ohs) {
        if (i >= n) break;
        float va[4], vb[4];
        unpack(pa[i], va), unpack(pb[i], vb);
#pragma unroll
        for (int j = 0; j < 4; ++j) va[j] *= r[i] * wa[j], vb[j] *= r[i] * wb[j];
        if (rot) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // pair j: split (a[j], b[j]); interleaved (2j, 2j + 1) of the eight dims
                float& p = kInter ? (j < 2 ? va[2 * j] : vb[2 * j - 4]) : va[j];
                float& q = kInter ? (j < 2 ? va[2 * j + 1] : vb[2 * j - 3]) : vb[j];
                const float o = p * c[j] - q * s[j];
                q = q * c[j] + p * s[j];
                p = o;
            }
        }
        store_piece(y, va), store_piece(y + (db - da), vb);
    }
}

// Any D up to 512, any strides and alignment: one warp per head, lane owns
// dims lane, lane + 32, ...  (4096 tokens x 36 heads in bf16: 116 us for 124 dims,
// 121 for 128 at odd addresses; 120 dims 20 us above.)
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
        float mean = ss / static_cast<float>(a.D), eps = a.eps;
        const float f = norm_factor(mean, eps);
        if (__builtin_expect(f != 1.f, 0)) {  // (of the whole warp alike)
            ss = 0.f;
#pragma unroll
            for (int i = 0; i < kMost; ++i) v[i] *= f, u[i] *= f, ss += v[i] * v[i];
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            mean = ss / static_cast<float>(a.D);
            eps = eps * f * f;
        }
        r = rsqrtf(mean + eps);
    }
    const int64_t row = a.rot ? table_row(a, a.positions[token]) * half : 0;
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
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & (sizeof(T) * kVec - 1)) == 0; };
    auto al16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    constexpr int kMany = 4;
    const int64_t strides = a.q_ts | a.q_hs | a.qo_ts | a.qo_hs | (a.Hk ? a.k_ts | a.k_hs | a.ko_ts | a.ko_hs : 0);
    // pieces of four dims never straddle a border of the rotated range or of its halves, and pair up
    const bool whole = a.D % 8 == 0 && a.D <= 256 && a.rot % 8 == 0 && a.start % 4 == 0;
    const bool vec = whole && strides % kVec == 0 && al(a.q) && al(a.q_out) && al16(a.q_weight) && al16(a.k_weight) &&
                     (!a.Hk || (al(a.k) && al(a.k_out))) && (!a.rot || (al16(a.cos) && al16(a.sin)));
    if (!vec) {
        const int64_t warps = static_cast<int64_t>(a.tokens) * (a.Hq + a.Hk);
        norm_rope_any_kernel<T><<<static_cast<unsigned>((warps + 3) / 4), kThreads, 0, st>>>(a);
        return launch_status(cudaGetLastError());
    }
    const int lanes = a.D / (2 * kVec);
    int lg_group = 0;
    while (1 << lg_group < lanes) ++lg_group;
    auto blocks = [&](int heads) {
        const int64_t items = static_cast<int64_t>(a.tokens) * ((a.Hq + heads - 1) / heads + (a.Hk + heads - 1) / heads);
        return static_cast<unsigned>(((items << lg_group) + kThreads - 1) / kThreads);
    };
    // Four heads per group once that still gives every SM a block: 4096 tokens
    // x 36 heads of 128 in bf16 take 19.9 us (one head: 32, two: 24.6, eight:
    // 23.4), 256 tokens 3.5 us (one head: 4.1).
    const bool many = blocks(kMany) >= static_cast<unsigned>(sm_count());
    auto go = [&](auto kernel) { kernel<<<blocks(many ? kMany : 1), kThreads, 0, st>>>(a, lg_group, lanes); };
    if (a.interleaved)
        many ? go(norm_rope_kernel<T, kMany, true>) : go(norm_rope_kernel<T, 1, true>);
    else
        many ? go(norm_rope_kernel<T, kMany, false>) : go(norm_rope_kernel<T, 1, false>);
    return launch_status(cudaGetLastError());
}

}  // namespace

sa_status norm_rope_launch(const NormRopeArgs& a, sa_dtype dt, cudaStream_t st) {
    return dt == SA_F32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace sa
