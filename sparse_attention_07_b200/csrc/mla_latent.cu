// mla_latent.cu — MLA attention over the quantised latent cache (selected or
// all positions), and of a tree of drafted tokens over the quantised or the
// bf16 cache.
//
//   z_j = (q_lat . c_j + q_rope . kr_j) * scale,  out = sum_j softmax(z)_j c_j
//
// One CTA pair per (128 query rows, key split).  The 128 rows are the heads of
// one query, or, for drafted tokens with H <= 64 heads, of several tokens of
// one tree: they share the prefix, so it is read once for all of them.
//  * The pair's rows are split 64 / 64 and both products run as cta_group::2
//    MMAs with M = 128: a CTA holds the whole output of its 64 rows (512 dims
//    fp32 = 256 tensor-memory columns, rows folded over the 128 lanes) and
//    their scores and softmax state, so nothing is exchanged between the two
//    but the cache rows themselves.
//  * Keys go by in tiles of 64.  Each CTA loads 32 of them, once, with plain
//    16-byte loads (the next tile's are in flight while this one is stored),
//    turns e4m3 codes into bf16 exactly, and stores them twice: all 576 dims as
//    its half of the B operand of the score product (K-major), and the 512
//    latent dims as rows of the V operand (MN-major), 256 dims here and 256
//    into the partner's shared memory, since each CTA supplies half the dims of
//    the aggregation.
//  * Four softmax warps: thread = (row, half of the tile's keys).  Online base-2
//    softmax; the two threads of a row exchange tile maxima through shared
//    memory, O is rescaled only when a maximum grows by more than 2^8.  P goes
//    to shared memory as bf16 (the normaliser sums the rounded values, so the
//    weights applied add up to one; lse uses the fp32 sum).
//  * One thread of the even CTA issues scores(t + 1) before aggregation(t).
//  * A drafted row that holds a non-finite value stays out of V and makes its
//    scores NaN instead: tokens that see it get NaN, tokens that do not are
//    untouched (0 * NaN would reach them through the product).
//  * Few items split their keys over several pairs; partial states go to a
//    workspace and a combine kernel merges them in split order.
#include "sa_device.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kPage = 64;
constexpr int kNK = 64;    // keys per tile
constexpr int kOwn = 32;   // keys of a tile that one CTA loads
constexpr int kRows = 64;  // query rows per CTA
constexpr int kQSlice = kRows * 128, kKSlice = kOwn * 128, kVSlice = kNK * 128;  // 64 dims each
constexpr int kKStage = 9 * kKSlice, kVStage = 4 * kVSlice;
constexpr int kStages = 2;
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 9 * kQSlice;
constexpr int kOffV = kOffK + kStages * kKStage;
constexpr int kOffP = kOffV + kStages * kVStage;
constexpr int kSmem = kOffP + kRows * 128 + 1024;
constexpr int kORow = 512 * 4 + 16;  // an output row staged in the K and V rings (padded)
constexpr int kSmxWarps = 4, kProdWarps = 8;
constexpr int kMmaWarp = kSmxWarps + kProdWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0;    // two 256-dim products, 128 columns each
constexpr uint32_t kColS = 256;  // two score buffers of 32 columns
constexpr float kRescaleLog2 = 8.0f;
constexpr int kMaxSplits = 32;

static_assert(kOffK % 1024 == 0 && kOffV % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms are 1024-byte aligned");
static_assert(kSmem <= 232448 - 3072, "shared memory budget");
static_assert(kRows * kORow <= kStages * (kKStage + kVStage), "the output rows fit in the rings");

struct Args {
    LatentArgs a;
    int tokens_per_item;  // P: tokens of a tree in one item's 128 rows
    int groups;           // items per tree
    int nsplit;
    float* ws_o;   // [item][nsplit][128][512]
    float* ws_ml;  // [item][nsplit][128][4]: m, l of bf16 P, l of fp32 P
};

// What one item covers.
struct Item {
    int b, i0, seq, past, nd, n_keys, tokens;
};

__device__ __forceinline__ Item item_of(const Args& ka, int item) {
    const LatentArgs& a = ka.a;
    Item it;
    it.b = item / ka.groups;
    it.i0 = (item % ka.groups) * ka.tokens_per_item;
    it.seq = a.seq_of_row ? a.seq_of_row[it.b] : it.b;
    it.nd = a.tree ? max(min(a.n_draft ? a.n_draft[it.b] : a.T, a.T), 0) : 0;
    it.past = a.idx ? 0 : max(a.n_past[it.b], 0);
    it.n_keys = a.idx ? a.k : it.past + it.nd;
    it.tokens = min(ka.tokens_per_item, (a.tree ? it.nd : a.T) - it.i0);  // <= 0: nothing to do
    return it;
}

__device__ __forceinline__ int latent_row(const LatentArgs& a, int seq, int p) {
    if (p / kPage >= a.pages_per_seq) return -2;
    const int64_t at = static_cast<int64_t>(seq) * a.pages_per_seq + p / kPage;
    const int64_t pg = a.page_table ? a.page_table[at] : at;
    if (pg < 0 || pg >= a.pool_pages) return -2;
    return static_cast<int>(pg * kPage + (p % kPage));
}

__device__ __forceinline__ bool bf16x2_bad(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

template <int N>
__device__ __forceinline__ float tree_max(const float (&s)[N]) {
    float v[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v[i] = fmaxf(s[i], s[i + N / 2]);
#pragma unroll
    for (int w = N / 4; w > 0; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) v[i] = fmaxf(v[i], v[i + w]);
    return v[0];
}

__device__ __forceinline__ void st_smem_v4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// One tile's rows of a producer warp (4 keys) as loaded: lane l holds 16
// consecutive dims of an e4m3 row, or 16-byte pieces l and l + 32 of a bf16 row;
// kr: piece l % 8 of key l / 8.
template <bool kQ8>
struct Loaded {
    uint4 c[4][kQ8 ? 1 : 2];
    uint32_t sc[kQ8 ? 4 : 1];
    uint4 kr;
};

template <bool kQ8>
__device__ __forceinline__ void load_tile(const LatentArgs& a, int rows4, int lane, Loaded<kQ8>& x) {
    // rows4: lane i < 4 of each group of 4 lanes holds the pool row of key i (negative: zeros)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = __shfl_sync(0xffffffffu, rows4, i);
        if (kQ8) {
            x.c[i][0] = make_uint4(0u, 0u, 0u, 0u);
            x.sc[i] = 127u;
            if (row >= 0) {
                x.c[i][0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c_cache) + row * a.c_ld) + lane);
                x.sc[i] = __ldg(a.c_scale + row * a.s_ld + (lane >> 3));
            }
        } else {
#pragma unroll
            for (int p = 0; p < (kQ8 ? 1 : 2); ++p) {
                x.c[i][p] = make_uint4(0u, 0u, 0u, 0u);
                if (row >= 0)
                    x.c[i][p] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.c_cache) + row * a.c_ld) +
                                      lane + 32 * p);
            }
        }
    }
    const int row = __shfl_sync(0xffffffffu, rows4, lane >> 3);
    x.kr = make_uint4(0u, 0u, 0u, 0u);
    if (row >= 0)
        x.kr = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.kr_cache) + row * a.kr_ld) + (lane & 7));
}

template <bool kQ8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) mla_latent_kernel(const Args ka) {
    pdl_trigger();
    const LatentArgs& a = ka.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // filled by both CTAs' warps, waited for by the issuing thread (the even CTA's copies are used)
    __shared__ uint64_t bar_kfull[kStages], bar_vfull[kStages], bar_sfree[2], bar_pfull;
    // arrived on in both CTAs when a product is done: scores(t) -> bar_s[t & 1] (K stage free, scores
    // readable), aggregation(t) -> bar_o[t & 1] (V stage and P free, O updated)
    __shared__ uint64_t bar_s[2], bar_o[2], bar_final;
    __shared__ float s_max[2][128];
    __shared__ float2 s_sum[128];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ volatile int s_fail[2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int cl = blockIdx.x >> 1;
    const int item = cl / ka.nsplit, split = cl % ka.nsplit;
    const Item it = item_of(ka, item);
    if (it.tokens <= 0) return;  // both CTAs of the pair alike
    const int tiles = (it.n_keys + kNK - 1) / kNK;
    const int t0 = static_cast<int>(static_cast<int64_t>(split) * tiles / ka.nsplit);
    const int nt = static_cast<int>(static_cast<int64_t>(split + 1) * tiles / ka.nsplit) - t0;
    WaitCtx wc{a.err, &s_abort};

    if (tid == 0) {
        s_abort = 0;
        s_fail[0] = s_fail[1] = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_kfull[i], 2 * kProdWarps);
            mbar_init(&bar_vfull[i], 2 * kProdWarps);
            mbar_init(&bar_sfree[i], 2 * kSmxWarps);
            mbar_init(&bar_s[i], 1);
            mbar_init(&bar_o[i], 1);
        }
        mbar_init(&bar_pfull, 2 * kSmxWarps);
        mbar_init(&bar_final, 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(&s_tmem, kTmemCols);
        tmem_relinquish_pair();
    }

    // ---- producers: pool rows of the next eight tiles, one (tile, key) per lane
    const int pw = warp - kSmxWarps;
    const bool producer = pw >= 0 && pw < kProdWarps;
    auto resolve = [&](int t) {  // lane l: tile t + l / 4, own key 4 pw + l % 4
        const int tt = t + (lane >> 2);
        if (tt >= nt) return -1;
        const int slot = (t0 + tt) * kNK + static_cast<int>(rank) * kOwn + 4 * pw + (lane & 3);
        if (slot >= it.n_keys) return -1;
        const int p = a.idx ? a.idx[static_cast<int64_t>(it.b) * a.k + slot] : slot;
        if (p < 0) return -1;
        const int row = latent_row(a, it.seq, p);
        if (row < 0) record_error(a.err, kErrMlaIndex);
        return max(row, 0);
    };
    int rows8 = -1, rows8_next = -1;
    Loaded<kQ8> x;
    if (producer) {
        rows8 = resolve(0);
        rows8_next = resolve(8);
        load_tile<kQ8>(a, rows8, lane, x);
    }

    // ---- the query rows, as the K-major A operand: row r of this CTA, 16-byte
    // piece c of its 72 (512 latent dims, then 64 RoPE dims)
    {
        uint8_t* sQ = sm + kOffQ;
        for (int i = tid; i < kRows * 72; i += kThreads) {
            const int r = i / 72, c = i % 72;
            const int m = static_cast<int>(rank) * kRows + r;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (m < it.tokens * a.H) {
                const int64_t qrow = (static_cast<int64_t>(it.b) * a.T + it.i0) * a.H + m;
                v = c < 64 ? __ldg(static_cast<const uint4*>(a.q_lat) + qrow * 64 + c)
                           : __ldg(static_cast<const uint4*>(a.q_rope) + qrow * 8 + (c - 64));
            }
            *reinterpret_cast<uint4*>(sQ + (c >> 3) * kQSlice + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();  // the TMEM address and the barriers are in place here
    cluster_sync_all();  // and in the partner, and both queries are written
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (nt == 0) {
        // no keys: fall through (the softmax warps write the empty result)
    } else if (producer) {
        const uint32_t kfull0 = mapa_u32(smem_u32(&bar_kfull[0]), 0), vfull0 = mapa_u32(smem_u32(&bar_vfull[0]), 0);
        // this lane's dim slices and where their V copy goes: slice s (64 dims)
        // belongs to CTA (s % 4) / 2, as its slice 2 (s / 4) + s % 2
        constexpr int kPieces = 2;  // 16-byte bf16 pieces per row and lane
        uint32_t koff[kPieces], voff[kPieces];
        const uint32_t vb[2] = {mapa_u32(smem_u32(sm + kOffV), 0), mapa_u32(smem_u32(sm + kOffV), 1)};
        int chunk[kPieces];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            // e4m3: dims 16 lane ..: pieces 2 lane, 2 lane + 1 (odd slices store theirs in the other
            // order, so that the eight lanes of a store phase touch distinct banks); bf16: lane, lane + 32
            const int c = kQ8 ? 2 * lane + (p ^ ((lane >> 2) & 1)) : lane + 32 * p;
            const int s = c >> 3;
            chunk[p] = c & 7;
            koff[p] = smem_u32(sm + kOffK) + s * kKSlice;
            voff[p] = vb[(s & 3) >> 1] + (2 * (s >> 2) + (s & 1)) * kVSlice;
        }
        const uint32_t kroff = smem_u32(sm + kOffK) + 8 * kKSlice;
        for (int t = 0; t < nt; ++t) {
            const int st = t & 1;
            const uint32_t par = static_cast<uint32_t>(((t >> 1) & 1) ^ 1);
            // bf16 pieces of this tile
            uint4 w[4][kPieces];
            uint4 kr = x.kr;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kQ8) {
                    const uint32_t s2 = q8_scale_bf16x2(x.sc[i]);
                    const uint2 a0 = e4m3x4_to_bf16x4(x.c[i][0].x, s2), a1 = e4m3x4_to_bf16x4(x.c[i][0].y, s2);
                    const uint2 a2 = e4m3x4_to_bf16x4(x.c[i][0].z, s2), a3 = e4m3x4_to_bf16x4(x.c[i][0].w, s2);
                    const uint4 lo = make_uint4(a0.x, a0.y, a1.x, a1.y), hi = make_uint4(a2.x, a2.y, a3.x, a3.y);
                    const bool odd = (lane >> 2) & 1;
                    w[i][0] = odd ? hi : lo;
                    w[i][1] = odd ? lo : hi;
                } else {
#pragma unroll
                    for (int p = 0; p < kPieces; ++p) w[i][p] = x.c[i][kQ8 ? 0 : p];
                }
            }
            // the next tile's loads
            if (t + 1 < nt) {
                const int u = (t + 1) & 7;
                if (u == 0) {
                    rows8 = rows8_next;
                    rows8_next = resolve(t + 9);
                }
                load_tile<kQ8>(a, __shfl_sync(0xffffffffu, rows8, 4 * u + (lane & 3)), lane, x);
            }
            // drafted rows with non-finite contents: out of V, NaN in K
            uint32_t bad = 0;
            const int own0 = (t0 + t) * kNK + static_cast<int>(rank) * kOwn + 4 * pw;  // this warp's first slot
            if (a.tree && own0 + 3 >= it.past) {
                const uint32_t kb = __ballot_sync(0xffffffffu, bf16x2_bad(kr.x) | bf16x2_bad(kr.y) | bf16x2_bad(kr.z) |
                                                                   bf16x2_bad(kr.w));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    bool any = (kb >> (8 * i) & 0xFFu) != 0;
#pragma unroll
                    for (int p = 0; p < kPieces; ++p)
                        any |= bf16x2_bad(w[i][p].x) | bf16x2_bad(w[i][p].y) | bf16x2_bad(w[i][p].z) | bf16x2_bad(w[i][p].w);
                    if (__any_sync(0xffffffffu, any) && own0 + i >= it.past) bad |= 1u << i;
                }
                if (bad >> (lane >> 3) & 1u) kr = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
            }
            if (t >= kStages && !warp_wait(&bar_s[st], par, wc, kErrLatWait | 1)) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = 4 * pw + i;
#pragma unroll
                for (int p = 0; p < kPieces; ++p)
                    st_smem_v4(koff[p] + st * kKStage + j * 128 + ((chunk[p] ^ (j & 7)) << 4), w[i][p]);
            }
            {
                const int j = 4 * pw + (lane >> 3);
                st_smem_v4(kroff + st * kKStage + j * 128 + (((lane & 7) ^ (j & 7)) << 4), kr);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(kfull0 + 8 * st);
            if (t >= kStages && !warp_wait(&bar_o[st], par, wc, kErrLatWait | 2)) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = static_cast<int>(rank) * kOwn + 4 * pw + i;
                if (bad >> i & 1u) w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int p = 0; p < kPieces; ++p)
                    st_cluster_v4(voff[p] + st * kVStage + j * 128 + ((chunk[p] ^ (j & 7)) << 4), w[i][p].x, w[i][p].y,
                                  w[i][p].z, w[i][p].w);
            }
            fence_proxy_async_cluster();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(vfull0 + 8 * st);
        }
    } else if (warp == kMmaWarp) {
        if (rank == 0 && lane == 0) {
            constexpr uint32_t id_qk = idesc_f32acc(1, 1, false, false, 128, kNK);
            constexpr uint32_t id_pv = idesc_f32acc(1, 1, false, true, 128, 256);
            bool ok = true;
            for (int t = 0; ok && t <= nt; ++t) {
                if (t < nt) {  // scores(t)
                    const int st = t & 1;
                    const uint32_t ph = static_cast<uint32_t>((t >> 1) & 1);
                    ok = mbar_wait<true>(&bar_kfull[st], ph, wc, kErrLatWait | 3) &&
                         (t < 2 || mbar_wait<true>(&bar_sfree[st], ph ^ 1, wc, kErrLatWait | 4));
                    if (!ok) break;
                    fence_proxy_async_cluster();
                    tc_fence_after();
                    for (int bb = 0; bb < 9; ++bb) {
                        const uint64_t qd = sdesc(smem_u32(sm + kOffQ + bb * kQSlice), 16, 1024, kSw128);
                        const uint64_t kd = sdesc(smem_u32(sm + kOffK + st * kKStage + bb * kKSlice), 16, 1024, kSw128);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_bf16_pair(tmem + kColS + 32 * st, qd + 2 * kk, kd + 2 * kk, id_qk, (bb | kk) != 0 ? 1u : 0u);
                    }
                    tc_commit_pair(&bar_s[st]);
                }
                if (t > 0) {  // aggregation(t - 1)
                    const int u = t - 1, st = u & 1;
                    ok = mbar_wait<true>(&bar_vfull[st], static_cast<uint32_t>((u >> 1) & 1), wc, kErrLatWait | 5) &&
                         mbar_wait<true>(&bar_pfull, static_cast<uint32_t>(u & 1), wc, kErrLatWait | 6);
                    if (!ok) break;
                    fence_proxy_async_cluster();
                    tc_fence_after();
                    const uint64_t pd = sdesc(smem_u32(sm + kOffP), 16, 1024, kSw128);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint64_t vd = sdesc(smem_u32(sm + kOffV + st * kVStage + 2 * j * kVSlice), kVSlice, 1024, kSw128);
#pragma unroll
                        for (int kk = 0; kk < kNK / 16; ++kk)
                            mma_bf16_pair(tmem + kColO + 128 * j, pd + 2 * kk, vd + 128 * kk, id_pv,
                                          (u > 0 || kk > 0) ? 1u : 0u);
                    }
                    tc_commit_pair(&bar_o[st]);
                }
            }
            // every product has finished (fixed limit) before the pair tears down
            int dummy = 0;
            WaitCtx dw(a.err, reinterpret_cast<volatile int*>(&dummy), kWaitLimitNs);
            tc_commit_pair(&bar_final);
            mbar_wait(&bar_final, 0, dw, kErrLatWait | 7);
        } else if (lane == 0) {
            // the last arrival this CTA gets (the even CTA's waits all have limits, so it comes)
            int dummy = 0;
            WaitCtx dw(a.err, reinterpret_cast<volatile int*>(&dummy), 4 * kWaitLimitNs);
            mbar_wait(&bar_final, 0, dw, kErrLatWait | 12);
        }
        __syncwarp();
    }
    if (warp < kSmxWarps) {
        // ---------------------------------------------- softmax + output
        const int r = tid & 63, hf = tid >> 6;  // row of this CTA, half of the keys (and of the output dims)
        const int m_row = static_cast<int>(rank) * kRows + r;
        const bool live = m_row < it.tokens * a.H;
        const int token = it.i0 + (live ? m_row / a.H : 0);
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t sfree0 = mapa_u32(smem_u32(&bar_sfree[0]), 0), pfull0 = mapa_u32(smem_u32(&bar_pfull), 0);
        const uint32_t prow = smem_u32(sm + kOffP) + r * 128;
        const float c2 = a.scale * 1.4426950408889634f;  // scores in base-2 units
        float m = -INFINITY, l = 0.f, lx = 0.f;
        bool ok = true;
        // which of this thread's 32 keys of tile t it attends to
        auto visible = [&](int t) -> uint32_t {
            const int s0 = (t0 + t) * kNK + hf * 32;
            if (a.idx) {
                const int s = s0 + lane;
                return __ballot_sync(0xffffffffu, s < a.k && a.idx[static_cast<int64_t>(it.b) * a.k + s] >= 0);
            }
            if (s0 + 32 <= it.past) return 0xffffffffu;
            uint32_t v = s0 < it.past ? (1u << (it.past - s0)) - 1u : 0u;
            const int n = min(32, it.n_keys - s0);
            const uint8_t* mk = a.tree_mask ? a.tree_mask + (static_cast<int64_t>(it.b) * a.T + token) * a.T : nullptr;
            for (int j = max(0, it.past - s0); j < n; ++j) {
                const int d = s0 + j - it.past;
                if (mk ? mk[d] != 0 : d <= token) v |= 1u << j;
            }
            return v;
        };
        uint32_t vis = nt > 0 ? visible(0) : 0u;
        for (int t = 0; t < nt; ++t) {
            const int sb = t & 1;
            ok = ok && warp_wait(&bar_s[sb], static_cast<uint32_t>((t >> 1) & 1), wc, kErrLatWait | 8);
            float s[32];
            if (ok) {
                tc_fence_after();
                uint32_t v[32];
                tmem_ld32(tmem + lane_base + kColS + 32 * sb, v);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(sfree0 + 8 * sb);
#pragma unroll
                for (int j = 0; j < 32; ++j) s[j] = (vis >> j & 1u) ? __uint_as_float(v[j]) * c2 : -INFINITY;
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) s[j] = -INFINITY;
                if (lane == 0) s_fail[sb] = 1;
            }
            const float mx = tree_max(s);
            s_max[sb][tid] = mx;
            named_sync(1, 32 * kSmxWarps);
            // a failed wait before this barrier is seen by all four warps after it (the flag
            // of the next tile is another word), so they leave the loop together
            if (s_fail[sb]) {
                ok = false;
                break;
            }
            const float top = fmaxf(mx, s_max[sb][tid ^ 64]);
            if (t + 1 < nt) vis = visible(t + 1);
            const bool grow = top > m + kRescaleLog2;
            if (__any_sync(0xffffffffu, grow)) {
                const float m_new = grow ? top : m;
                const float alpha = grow ? (m == -INFINITY ? 0.f : fast_exp2(m - m_new)) : 1.f;
                if (t > 0) {  // O holds the tiles before t
                    ok = warp_wait(&bar_o[(t - 1) & 1], static_cast<uint32_t>(((t - 1) >> 1) & 1), wc, kErrLatWait | 9);
                    if (ok) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 256; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(tmem + lane_base + kColO + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                            tmem_st32(tmem + lane_base + kColO + c, o);
                        }
                        tmem_st_wait();
                    }
                }
                l *= alpha;
                lx *= alpha;
                m = m_new;
            }
            const float mref = m == -INFINITY ? 0.f : m;  // masked keys are -inf and give exactly 0
            uint32_t pk[16];
            float lb = 0.f, lf = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float p0 = fast_exp2(s[2 * j] - mref), p1 = fast_exp2(s[2 * j + 1] - mref);
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
                lb += __low2float(b2) + __high2float(b2);
                lf += p0 + p1;
                pk[j] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            l += lb;
            lx += lf;
            // aggregation(t - 1) has read P
            if (ok && t > 0)
                ok = warp_wait(&bar_o[(t - 1) & 1], static_cast<uint32_t>(((t - 1) >> 1) & 1), wc, kErrLatWait | 10);
            if (ok) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    st_smem_v4(prow + (((4 * hf + q) ^ (r & 7)) << 4),
                               make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]));
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(pfull0);
            }
        }
        // ---- both halves' sums, then the rows out: staged in the idle rings, bulk copies
        s_sum[tid] = make_float2(l, lx);
        named_sync(1, 32 * kSmxWarps);
        l += s_sum[tid ^ 64].x;
        lx += s_sum[tid ^ 64].y;
        if (ok && nt > 0)
            ok = warp_wait(&bar_o[(nt - 1) & 1], static_cast<uint32_t>(((nt - 1) >> 1) & 1), wc, kErrLatWait | 11);
        if (ok && !*wc.abort) {
            tc_fence_after();
            const bool partial = ka.nsplit > 1;
            const bool bf = !partial && a.out_bf16 != nullptr;
            const bool empty = l == 0.f;  // (a NaN sum is not empty)
            const float inv = empty || partial ? 1.f : 1.f / l;
            uint8_t* srow = sm + kOffK + r * kORow;
            const int e = bf ? 2 : 4;
#pragma unroll 1
            for (int c = 0; c < 256; c += 32) {
                const int d = (c >> 7) * 256 + hf * 128 + (c & 127);
                uint32_t o[32];
                if (nt > 0) {
                    tmem_ld32(tmem + lane_base + kColO + c, o);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    float f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = empty ? 0.f : __uint_as_float(o[j + i]) * inv;
                    if (bf)
                        *reinterpret_cast<uint2*>(srow + 2 * (d + j)) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
                    else
                        *reinterpret_cast<float4*>(srow + 4 * (d + j)) = make_float4(f[0], f[1], f[2], f[3]);
                }
            }
            fence_proxy_async_smem();
            if (live) {
                const int64_t orow = (static_cast<int64_t>(it.b) * a.T + it.i0) * a.H + m_row;
                const int64_t wrow = (static_cast<int64_t>(item) * ka.nsplit + split) * 128 + m_row;
                uint8_t* dst = partial ? reinterpret_cast<uint8_t*>(ka.ws_o + wrow * 512)
                                       : (bf ? static_cast<uint8_t*>(a.out_bf16) + orow * 1024
                                             : reinterpret_cast<uint8_t*>(a.out + orow * 512));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int d = j * 256 + hf * 128;
                    bulk_copy_s2g(dst + d * e, srow + d * e, 128 * e);
                }
                if (hf == 0) {
                    if (partial) {
                        *reinterpret_cast<float4*>(ka.ws_ml + wrow * 4) = make_float4(m, l, lx, 0.f);
                    } else if (a.lse) {
                        a.lse[orow] = empty ? -INFINITY : (m + log2f(lx)) * 0.6931471805599453f;
                    }
                }
                bulk_wait_all();
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // no more remote arrivals, stores or products in either CTA
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

// Merge the split partial states: one warp per query row, lane owns dims
// 4 lane + 128 p.
constexpr int kCombThreads = 256;

__global__ void __launch_bounds__(kCombThreads) mla_latent_combine_kernel(const Args ka) {
    pdl_wait();
    const LatentArgs& a = ka.a;
    const int64_t orow = static_cast<int64_t>(blockIdx.x) * (kCombThreads / 32) + (threadIdx.x >> 5);
    if (orow >= static_cast<int64_t>(a.B) * a.T * a.H) return;
    const int lane = threadIdx.x & 31;
    const int h = static_cast<int>(orow % a.H), token = static_cast<int>(orow / a.H % a.T);
    const int b = static_cast<int>(orow / a.H / a.T);
    if (a.tree && a.n_draft && token >= a.n_draft[b]) return;
    const int item = b * ka.groups + token / ka.tokens_per_item;
    const int64_t w0 = static_cast<int64_t>(item) * ka.nsplit * 128 + token % ka.tokens_per_item * a.H + h;
    // lane s holds split s's state
    float ms = -INFINITY, ls = 0.f, xs = 0.f;
    if (lane < ka.nsplit) {
        const float4 v = *reinterpret_cast<const float4*>(ka.ws_ml + (w0 + static_cast<int64_t>(lane) * 128) * 4);
        ms = v.x, ls = v.y, xs = v.z;
    }
    float top = ls != 0.f ? ms : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float wgt = ls != 0.f ? exp2f(ms - top) : 0.f;
    float L = ls * wgt, LX = xs * wgt;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        L += __shfl_xor_sync(0xffffffffu, L, o);
        LX += __shfl_xor_sync(0xffffffffu, LX, o);
    }
    float4 acc[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) acc[p] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < ka.nsplit; ++s) {
        const float w = __shfl_sync(0xffffffffu, wgt, s);
        if (__shfl_sync(0xffffffffu, ls, s) == 0.f) continue;
        const float4* src = reinterpret_cast<const float4*>(ka.ws_o + (w0 + static_cast<int64_t>(s) * 128) * 512) + lane;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float4 v = src[32 * p];
            acc[p].x += v.x * w, acc[p].y += v.y * w, acc[p].z += v.z * w, acc[p].w += v.w * w;
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const float x = acc[p].x * inv, y = acc[p].y * inv, z = acc[p].z * inv, w = acc[p].w * inv;
        if (a.out_bf16)
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out_bf16) + orow * 1024 + 256 * p + 8 * lane) =
                make_uint2(pack_bf16x2(x, y), pack_bf16x2(z, w));
        else
            *reinterpret_cast<float4*>(a.out + orow * 512 + 128 * p + 4 * lane) = make_float4(x, y, z, w);
    }
    if (a.lse && lane == 0) a.lse[orow] = L == 0.f ? -INFINITY : (top + log2f(LX)) * 0.6931471805599453f;
}

int tokens_per_item(int T, int H) {
    const int p = 128 / H;
    return p < 1 ? 1 : (p < T ? p : T);
}

// Key splits of an item: as many as fill the GPU's CTA pairs, each of at least
// three tiles.
int splits(int64_t items, int k) {
    const int64_t pairs = sm_count() / 2;
    const int tiles = (k + kNK - 1) / kNK;
    int64_t ns = items >= pairs ? 1 : pairs / items;
    if (ns > tiles / 3) ns = tiles / 3;
    if (ns > kMaxSplits) ns = kMaxSplits;
    return ns < 1 ? 1 : static_cast<int>(ns);
}

size_t state_bytes(int64_t items, int ns) { return static_cast<size_t>(items) * ns * 128 * (512 + 4) * 4; }

template <bool kQ8>
cudaError_t launch(const Args& ka, int64_t items, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(mla_latent_kernel<kQ8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    mla_latent_kernel<kQ8><<<static_cast<unsigned>(2 * items * ka.nsplit), kThreads, kSmem, st>>>(ka);
    return cudaGetLastError();
}

}  // namespace

size_t mla_latent_workspace_bytes(int B, int T, int H, int k) {
    const int P = tokens_per_item(T, H);
    const int64_t items = static_cast<int64_t>(B) * ((T + P - 1) / P);
    const int ns = splits(items, k);
    return ns > 1 ? state_bytes(items, ns) : 0;
}

sa_status mla_latent_launch(const LatentArgs& a, void* ws, size_t ws_bytes, cudaStream_t st) {
    Args ka = {};
    ka.a = a;
    ka.tokens_per_item = tokens_per_item(a.T, a.H);
    ka.groups = (a.T + ka.tokens_per_item - 1) / ka.tokens_per_item;
    const int64_t items = static_cast<int64_t>(a.B) * ka.groups;
    ka.nsplit = splits(items, a.k);
    if (ka.nsplit > 1) {
        if (!ws || ws_bytes < state_bytes(items, ka.nsplit)) return SA_EINVAL;
        ka.ws_o = static_cast<float*>(ws);
        ka.ws_ml = ka.ws_o + static_cast<size_t>(items) * ka.nsplit * 128 * 512;
    }
    cudaError_t e = a.c_scale ? launch<true>(ka, items, st) : launch<false>(ka, items, st);
    if (e == cudaSuccess && ka.nsplit > 1) {
        const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.H;
        constexpr int kPer = kCombThreads / 32;
        e = launch_pdl(mla_latent_combine_kernel, dim3(static_cast<unsigned>((rows + kPer - 1) / kPer)), dim3(kCombThreads), 0,
                       st, ka);
    }
    return launch_status(e);
}

}  // namespace sa
