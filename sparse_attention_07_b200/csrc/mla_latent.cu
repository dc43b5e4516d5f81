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
//  * Keys go by in tiles of 64.  A CTA supplies 32 rows of each as its half of the
//    score product's B operand (576 dims, K-major, two stages) and 256 dims of all
//    64 as its half of the aggregation's (MN-major).  bf16 rows (of a prefix: whole
//    pages) are TMA-loaded into the operands.  e4m3 rows are loaded to registers by
//    sixteen warps, whole lines, turned into bf16 there, exactly, and stored to the
//    operands, eight warps each; one warp resolves their pool rows and scales, two
//    report stored operands.  Latent dims stand in the order 0, 2, 1, 3 of each four
//    (fewer shifts), and in odd 64-dim slices with neighbouring groups of eight
//    swapped (banks), in the query and the output columns alike.
//  * Eight softmax warps: thread = (row, quarter of the tile's keys).  Online base-2
//    softmax; the four threads of a row exchange tile maxima through shared
//    memory, O is rescaled only when a maximum grows by more than 2^8.  P goes
//    to shared memory as bf16, as the tensor cores take it (half a step, 2^-8, of
//    each weight); the normaliser is the sum of the weights as rounded, so that
//    the weights applied sum to 1, and the lse uses the fp32 values.  (Two sums cost
//    5 us of 1024 x 2048 rows; with one, 2^15 keys of one sign were off by 5e-4,
//    with two by 2e-4.)
//  * One thread of the even CTA issues scores(t + 1) before aggregation(t).
//  * Drafted rows are masked token by token, so a row that some token must not see
//    may be in the tile; non-finite contents of such a row are zeroed in the
//    aggregation operand (0 * NaN would reach every token) and NaN in the score
//    operand (an infinity alone can score -inf, as if masked): the tokens that see
//    the row get NaN, through its score.
//  * Few items split their keys over several pairs; partial states go to a
//    workspace and a combine kernel merges them in split order.
//  * Many short selections go to the pairs in turn (kMany): the tiles of a pair's items
//    are one stream for the roles, the loading warps bring the next query when an
//    item's scores are done, and its output leaves straight from tensor memory while
//    the next item's tiles are under way.
//
// Measured (device time, replayed graph): 1024 queries x 2048 selected e4m3 rows x
// 128 heads in 0.90 ms (649 TFLOP/s), 74 of them (one per pair) in 64 us: 1.56 us
// per tile and 14 us around them.  The tensor cores are at work for 30 percent of
// that.  What is left is the hand-over from role to role: an earlier version, of
// 63.6 us, still took 54.4 with conversion, row loads, seven eighths of the products
// and the exponentials left out.  So the warps are many (28, of 72
// registers) and their loops short: fewer or longer ones ran slower (sixteen warps
// of 128 registers 87 us; a second tile of rows in flight per warp, as copies or
// as a doubled loop, 79 to 83; loading warps taking turns with double the rows 70),
// softmax groups that alternate tiles and issuing products by readiness the same.
#include <algorithm>

#include "sa_device.cuh"
#include "sa_internal.h"
#include "sa_wait.h"

namespace sa {
namespace {

constexpr int kPage = 64;
constexpr int kNK = 64;    // keys per tile
constexpr int kOwn = 32;   // keys of a tile that one CTA loads
constexpr int kRows = 64;  // query rows per CTA
constexpr int kQSlice = kRows * 128, kKSlice = kOwn * 128, kVSlice = kNK * 128;  // 64 dims each
constexpr int kVStage = 4 * kVSlice;
constexpr int kORow = 512 * 4 + 16;  // a staged output row (padded)
constexpr int kSmxWarps = 8, kLoadWarps = 8;  // loading warps of either operand
constexpr int kKWarp0 = kSmxWarps, kVWarp0 = kKWarp0 + kLoadWarps;
constexpr int kMmaWarp = kVWarp0 + kLoadWarps;
constexpr int kTmaWarp = kMmaWarp + 1;     // bf16: loads; e4m3: rows resolved
constexpr int kReportWarp = kTmaWarp + 1;  // and the next: e4m3: stored operands reported, scores' and aggregation's
constexpr int kThreads = 32 * (kReportWarp + 2);

template <bool kQ8>
struct Smem {
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + 9 * kQSlice;
    static constexpr int kOffR = kOffK + 2 * 8 * kKSlice;
    static constexpr int kOffV = kOffR + 2 * kKSlice;
    static constexpr int kOffP = kOffV + 2 * kVStage;
    static constexpr int kEnd = kOffP + kRows * 128;
    static constexpr int kBytes = kEnd + 1024;
    static_assert(kRows * kORow <= kEnd, "the output rows fit");
    static_assert(kOffK % 1024 == 0 && kOffR % 1024 == 0 && kOffV % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms are 1024-byte aligned");
    static_assert(kBytes <= 232448 - 4096, "shared memory budget");
};

// Tiles whose rows are resolved ahead: the warps of the score operand run up to three
// tiles ahead of the aggregation's.
constexpr int kRing = 4;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0;    // two 256-dim products, 128 columns each
constexpr uint32_t kColS = 256;  // two score buffers of 32 columns
constexpr float kRescaleLog2 = 8.0f;
constexpr int kMaxSplits = 32;
// Keys of a split at most (as far as kMaxSplits go): the tensor cores cut off what
// of a product lies below 2^-25 of the sum it is added to, so the output of n keys
// of the same sign falls short by n 2^-27 (measured, one split: 2e-3 at 2^18, 8e-3
// at 2^20, 3.3e-2 at 2^22; 16 splits of the last 2e-3).
constexpr int kLongKeys = 1 << 18;

// Tensor maps of the bf16 pools: latent rows in boxes of 64 dims by 32 rows (c) and
// by 64 rows (cv), RoPE keys by 32 rows, 128-byte swizzle.
struct Maps {
    CUtensorMap c, cv, kr;
};

struct Args {
    LatentArgs a;
    int tokens_per_item;  // P: tokens of a tree in one item's 128 rows
    int groups;           // items per tree
    int nsplit;           // key splits at most, and at least (an item's own: Item)
    int base;
    int items, stride;  // stride > 0 (selections): a pair takes items p, p + stride, ... of them, of equal tiles
    float* ws_o;   // [item][nsplit][128][512]
    float* ws_ml;  // [item][nsplit][128][2]: m, l
};

// Waits of this kernel.  Their code is small, since some thirty of them are inlined
// in the roles' loops: a wait that runs out leaves its site in the CTA's abort word,
// and the CTA's end records it.
struct Waits {
    volatile int* abort;
    uint32_t limit_ns;

    __device__ __forceinline__ static uint32_t now() {
        uint32_t t;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
        return t;
    }
    // kCluster: for reports of operands from both CTAs of the pair (mbar_arrive_remote).
    template <bool kCluster>
    __device__ __forceinline__ static bool poll(uint64_t* b, uint32_t parity) {
        return kCluster ? mbar_try_wait_acq_cluster(b, parity) : mbar_try_wait(b, parity);
    }
    // (one lane)
    template <bool kCluster = false>
    __device__ __forceinline__ bool one(uint64_t* b, uint32_t parity, int site) const {
        if (poll<kCluster>(b, parity)) return true;
        const uint32_t t0 = now();
#pragma unroll 1
        while (!poll<kCluster>(b, parity)) {
            if (*abort) return false;
            if (wait32_over(t0, now(), limit_ns)) {
                *abort = site;
                return false;
            }
        }
        return true;
    }
    // (one lane) Without the abort word: for a role's own work in flight.
    __device__ __forceinline__ static bool own(uint64_t* b, uint32_t parity, uint32_t limit_ns) {
        if (mbar_try_wait(b, parity)) return true;
        const uint32_t t0 = now();
#pragma unroll 1
        while (!mbar_try_wait(b, parity))
            if (wait32_over(t0, now(), limit_ns)) return false;
        return true;
    }
    // The whole warp leaves together.
    template <bool kCluster = false>
    __device__ __forceinline__ bool warp(uint64_t* b, uint32_t parity, int site) const {
        if (__all_sync(0xffffffffu, poll<kCluster>(b, parity))) return true;
        int ok = 1;
        if ((threadIdx.x & 31) == 0) ok = one<kCluster>(b, parity, site) ? 1 : 0;
        return __shfl_sync(0xffffffffu, ok, 0) != 0;
    }
    __device__ __forceinline__ bool operator()(uint64_t* b, uint32_t parity, int site) const { return warp(b, parity, site); }
    // For operands reported by both CTAs of the pair.
    __device__ __forceinline__ bool pair(uint64_t* b, uint32_t parity, int site) const { return warp<true>(b, parity, site); }
};

// What one item covers.
struct Item {
    int b, i0, seq, past, nd, n_keys, tokens, splits;
};

__device__ __forceinline__ Item item_of(const Args& ka, int item) {
    const LatentArgs& a = ka.a;
    Item it;
    it.b = item / ka.groups;
    it.i0 = (item % ka.groups) * ka.tokens_per_item;
    it.seq = a.seq_of_row ? a.seq_of_row[it.b] : it.b;
    it.nd = a.tree ? max(min(a.n_draft ? a.n_draft[it.b] : a.T, a.T), 0) : 0;
    // (no further than the page table: what lies behind is recorded where it is resolved, for 64 positions)
    it.past = a.idx ? 0 : static_cast<int>(min(static_cast<int64_t>(max(a.n_past[it.b], 0)), a.pages_per_seq * int64_t(kPage) + kPage));
    it.n_keys = a.idx ? a.k : it.past + it.nd;
    it.tokens = min(ka.tokens_per_item, (a.tree ? it.nd : a.T) - it.i0);  // <= 0: nothing to do
    it.splits = min(max(ka.base, (it.n_keys + kLongKeys - 1) / kLongKeys), ka.nsplit);
    return it;
}

// Pool row of a slot of a row's keys in three steps, each one load that has
// a while to land: the slot's position (-1: none), the page that holds it, the
// row.  A broken page table is recorded and row 0 of the pool read instead.
__device__ __forceinline__ int key_page(const LatentArgs& a, int seq, int pos) {
    if (pos < 0 || pos / kPage >= a.pages_per_seq) return -1;
    const int64_t at = static_cast<int64_t>(seq) * a.pages_per_seq + pos / kPage;
    return a.page_table ? a.page_table[at] : (at < a.pool_pages ? static_cast<int>(at) : -1);
}
__device__ __forceinline__ int key_row(const LatentArgs& a, int pos, int page, bool& broken) {
    const bool ok = page >= 0 && page < a.pool_pages;
    if (pos >= 0 && !ok) broken = true;
    return pos < 0 ? -1 : ok ? page * kPage + (pos % kPage) : 0;
}

// Pool rows and scale words of 32 keys (lane = key) of the tiles to come, of one item
// after the other: the next tile's are known, the one after has its page under way, the
// third its position.
template <bool kQ8, bool kMany>
struct Rows {
    int row, next, pos2, page2, pos3, seq3;
    uint32_t sc, sc_next;
    int b, seq, t;  // the tile whose position comes next
    bool broken;

    __device__ __forceinline__ uint32_t scale_word(const LatentArgs& a, int r) const {
        return kQ8 && r >= 0 ? __ldg(reinterpret_cast<const uint32_t*>(a.c_scale + r * a.s_ld)) : 0x7F7F7F7Fu;
    }
    // slot: the lane's key of an item's tile 0
    __device__ __forceinline__ int position(const Args& ka, const Item& it, int nt, int slot) {
        const LatentArgs& a = ka.a;
        if (kMany && t == nt) {
            t = 0;
            b += ka.stride;
            if (b < ka.items) seq = a.seq_of_row ? a.seq_of_row[b] : b;
        }
        const int at = slot + t * kNK;
        int pos = -1;
        if ((kMany ? b < ka.items : t < nt) && at < it.n_keys) pos = a.idx ? a.idx[static_cast<int64_t>(b) * a.k + at] : at;
        seq3 = seq;
        ++t;
        return pos;
    }
    __device__ __forceinline__ void start(const Args& ka, const Item& it, int nt, int slot) {
        const LatentArgs& a = ka.a;
        b = it.b, seq = it.seq, t = 0;
        const int p0 = position(ka, it, nt, slot), s0 = seq3, p1 = position(ka, it, nt, slot), s1 = seq3;
        pos2 = position(ka, it, nt, slot);
        const int s2 = seq3;
        pos3 = position(ka, it, nt, slot);
        const int g0 = key_page(a, s0, p0), g1 = key_page(a, s1, p1);
        page2 = key_page(a, s2, pos2);
        broken = false;
        row = key_row(a, p0, g0, broken);
        next = key_row(a, p1, g1, broken);
        sc = scale_word(a, row);
        sc_next = scale_word(a, next);
    }
    __device__ __forceinline__ void advance(const Args& ka, const Item& it, int nt, int slot) {
        const LatentArgs& a = ka.a;
        row = next;
        sc = sc_next;
        next = key_row(a, pos2, page2, broken);
        sc_next = scale_word(a, next);
        pos2 = pos3;
        page2 = key_page(a, seq3, pos2);
        pos3 = position(ka, it, nt, slot);
    }
};

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

// Volatile: issued a tile ahead of its use, where it stands, and not sunk to it.
__device__ __forceinline__ uint4 ld_row16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ld_smem_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Sixteen e4m3 dims -> two 16-byte bf16 pieces, each four in the order 0, 2, 1, 3.
__device__ __forceinline__ void convert16(uint4 u, uint32_t f, uint4& lo, uint4& hi) {
    const uint2 v0 = e4m3x4_to_bf16x4_0213(u.x, f), v1 = e4m3x4_to_bf16x4_0213(u.y, f);
    const uint2 v2 = e4m3x4_to_bf16x4_0213(u.z, f), v3 = e4m3x4_to_bf16x4_0213(u.w, f);
    lo = make_uint4(v0.x, v0.y, v1.x, v1.y);
    hi = make_uint4(v2.x, v2.y, v3.x, v3.y);
}
__device__ __forceinline__ void times4(uint4& v, uint32_t f) {
    v = make_uint4(hmul2_bf16(v.x, f), hmul2_bf16(v.y, f), hmul2_bf16(v.z, f), hmul2_bf16(v.w, f));
}

// The loads of the last of `issued` tiles, one per stage, have landed (fixed limit).
__device__ __forceinline__ void drain(int* abort_word, uint64_t* bars, int stages, int issued, int lane) {
    if (lane == 0) {
#pragma unroll 1
        for (int t = max(0, issued - stages); t < issued; ++t)
            if (!Waits::own(&bars[t % stages], static_cast<uint32_t>(t / stages & 1), static_cast<uint32_t>(kWaitLimitNs)))
                *abort_word = 14;
    }
    __syncwarp();
}

__device__ __forceinline__ bool bad4(uint4 v) {
    return bf16x2_bad(v.x) | bf16x2_bad(v.y) | bf16x2_bad(v.z) | bf16x2_bad(v.w);
}

// A 16-byte piece of a drafted row's operand, of the aggregation (v) or of the scores.
__device__ __forceinline__ void clean_piece(uint32_t at, uint4 piece, bool v) {
    const uint32_t w = v ? 0u : 0x7FC07FC0u;
    if (bad4(piece)) st_smem_v4(at, make_uint4(w, w, w, w));
}

// An item's query rows (its first is row q0 of the queries, `rows` of them this CTA's) by warp w
// of n, as the K-major A operand: row r of this CTA, 16-byte piece c of its 72 (512 latent dims,
// then 64 RoPE dims); rows that are not live are zero.
template <bool kQ8>
__device__ __forceinline__ void load_queries(const LatentArgs& a, uint32_t sQ, int64_t q0, int rows, int w, int n) {
    const int lane = threadIdx.x & 31;
    // a negative scale is moved to the queries: the softmax takes maxima of unscaled scores
    const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0u;
    // a warp per row, two rows in flight: pieces lane, lane + 32, and in eight lanes lane + 64
#pragma unroll 1
    for (int r0 = w; r0 < kRows; r0 += 2 * n) {
        uint4 x[2][3];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = r0 + k * n;
            const uint4* lat = static_cast<const uint4*>(a.q_lat) + (q0 + r) * 64 + lane;
            const uint4* rope = static_cast<const uint4*>(a.q_rope) + (q0 + r) * 8 + lane;
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                x[k][j] = make_uint4(0u, 0u, 0u, 0u);
                if (r < min(rows, kRows) && (j < 2 || lane < 8)) x[k][j] = __ldg(j < 2 ? lat + 32 * j : rope);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = r0 + k * n;
            if (r >= kRows) break;
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                uint4 v = x[k][j];
                v = make_uint4(v.x ^ sign, v.y ^ sign, v.z ^ sign, v.w ^ sign);
                if (kQ8 && j < 2)
                    v = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                                   __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
                if (j < 2 || lane < 8)
                    st_smem_v4(sQ + ((lane >> 3) + 4 * j) * kQSlice + r * 128 + (((lane & 7) ^ (r & 7) ^ (kQ8 && j < 2 ? lane >> 3 & 1 : 0)) << 4), v);
            }
        }
    }
}
// kMany: several items per pair (selections over the quantised cache).
template <bool kQ8, bool kMany>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) mla_latent_kernel(const __grid_constant__ Args ka, const __grid_constant__ Maps maps) {
    pdl_trigger();
    using S = Smem<kQ8>;
    const LatentArgs& a = ka.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bar_rows[kRing], bar_rowsfree[kRing];  // e4m3: rows and scale words of a tile's keys
    __shared__ __align__(16) int s_row[kRing][kNK];
    __shared__ __align__(16) uint32_t s_scale[kRing][kNK];
    __shared__ uint64_t bar_kst[2], bar_vst[2];      // bf16: an operand's loads have landed
    __shared__ uint64_t bar_kdone[2], bar_vdone[2];        // e4m3: the loading warps have stored an operand
    // a stage is visible to the tensor cores, the scores are read, P is written: waited for by the
    // issuing thread (the even CTA's copies are used)
    __shared__ uint64_t bar_kfull[2], bar_vfull[2], bar_sfree[2], bar_pfull;
    // arrived on in both CTAs when a product is done: scores(t) -> bar_s[t & 1] (K stage free, scores
    // readable), aggregation(t) -> bar_o[t & 1] (V stage and P free, O updated)
    __shared__ uint64_t bar_s[2], bar_o[2], bar_final;
    // the next item's query is in place, the last one's output is read (the even CTA's copies)
    __shared__ uint64_t bar_query, bar_ofree;
    __shared__ float s_max[2][32 * kSmxWarps];
    __shared__ float s_sum[2][32 * kSmxWarps];  // of a thread's weights, and of them as rounded
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ Item s_it;  // (drafted tokens' masks read it: no registers for it in the loops)
    __shared__ int s_t0;
    __shared__ volatile int s_fail[2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int cl = blockIdx.x >> 1;
    const int item = cl % ka.items, split = cl / ka.items;  // (splits that a short row does not have come last)
    const Item it = item_of(ka, item);
    if (it.tokens <= 0 || split >= it.splits) return;  // both CTAs of the pair alike
    const int tiles = (it.n_keys + kNK - 1) / kNK;
    // (2^24 tiles, and 32 splits, stay below 2^31)
    const int t0 = split * tiles / it.splits, nt = (split + 1) * tiles / it.splits - t0;
    // the tiles of all of this pair's items are one stream for the roles (stages and barriers go on from
    // item to item): nt of each
    const int n_items = kMany ? (ka.items - item + ka.stride - 1) / ka.stride : 1;
    const int all = nt * n_items;
    const Waits wait{&s_abort, wait32_limit(wait_limit_of(a.err))};

    if (tid == 0) {
        s_abort = 0;
        s_it = it;
        s_t0 = t0;
        s_fail[0] = s_fail[1] = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_kdone[i], kLoadWarps);
            mbar_init(&bar_vdone[i], kLoadWarps);
            mbar_init(&bar_kst[i], 1);
            mbar_init(&bar_vst[i], 1);
            mbar_init(&bar_kfull[i], 2);
            mbar_init(&bar_vfull[i], 2);
            mbar_init(&bar_sfree[i], 2 * kSmxWarps);
            mbar_init(&bar_s[i], 1);
            mbar_init(&bar_o[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&bar_rows[i], 2);  // halves
            mbar_init(&bar_rowsfree[i], 2 * kLoadWarps);
        }
        mbar_init(&bar_pfull, 2 * kSmxWarps);
        mbar_init(&bar_final, 1);
        mbar_init(&bar_query, 4 * kLoadWarps);
        mbar_init(&bar_ofree, 2 * kSmxWarps);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(&s_tmem, kTmemCols);
        tmem_relinquish_pair();
    }

    const uint32_t kbase = smem_u32(sm + S::kOffK), vbase = smem_u32(sm + S::kOffV);
    const int own0 = static_cast<int>(rank) * kOwn, other0 = kOwn - own0;  // this CTA's keys of a tile, the partner's
    // keys of a tile whose rows a warp resolves: e4m3: this CTA's half and the partner's; bf16: the first
    Rows<kQ8, kMany> keys, others;
    if (warp >= kTmaWarp) {
        if (!kQ8 && warp == kTmaWarp && lane == 0) {
            tma_prefetch_desc(&maps.c);
            tma_prefetch_desc(&maps.cv);
            tma_prefetch_desc(&maps.kr);
        }
        if (warp == kTmaWarp) keys.start(ka, it, nt, t0 * kNK + (kQ8 ? own0 : 0) + lane);
        if (kQ8 && warp == kTmaWarp) others.start(ka, it, nt, t0 * kNK + other0 + lane);
    } else if (warp < kTmaWarp) {
        load_queries<kQ8>(a, smem_u32(sm + S::kOffQ), (static_cast<int64_t>(it.b) * a.T + it.i0) * a.H + rank * kRows,
                          it.tokens * a.H - static_cast<int>(rank) * kRows, warp, kTmaWarp);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();  // the TMEM address and the barriers are in place here
    cluster_sync_all();  // and in the partner, and both queries are written
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (nt <= 0) {
        // no keys: fall through (the softmax warps write the empty result)
    } else if (kQ8 && warp == kTmaWarp) {
        // ------------------------------------------ e4m3: pool rows and scales, as far ahead as the ring goes
#pragma unroll 1
        for (int h = 0; h < 2 * all; ++h) {  // half tiles: the lanes' own keys, then the partner's
            const int t = h >> 1, st = t % kRing, key0 = h & 1 ? other0 : own0;
            if (t >= kRing && !wait(&bar_rowsfree[st], static_cast<uint32_t>(t / kRing & 1) ^ 1, 5)) break;
            s_row[st][key0 + lane] = keys.row;
            s_scale[st][key0 + lane] = keys.sc;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_rows[st]);
            keys.advance(ka, it, nt, t0 * kNK + key0 + lane);
            const Rows<kQ8, kMany> x = keys;  // (one copy of the code for both)
            keys = others;
            others = x;
        }
        if (keys.broken || others.broken) record_error(a.err, kErrMlaIndex);
        __syncwarp();
    } else if (kQ8 && warp >= kReportWarp) {
        // ------------------------------------------ e4m3: operands made visible and reported as they are stored
        // (a fence in a loading thread would wait for its stores and loads; an operand's bytes are in this
        // CTA, so the report to the issuing thread orders no more than that)
        if (lane == 0) {
            const bool v = warp != kReportWarp;
            uint64_t* done = v ? bar_vdone : bar_kdone;
            const uint32_t full = mapa_u32(smem_u32(v ? &bar_vfull[0] : &bar_kfull[0]), 0);
#pragma unroll 1
            for (int t = 0; t < all; ++t) {
                if (!wait.one(&done[t & 1], static_cast<uint32_t>(t >> 1 & 1), 6)) break;
                fence_proxy_async_smem();
                mbar_arrive_remote(full + 8 * (t & 1));
            }
        }
        __syncwarp();
    } else if (!kQ8 && warp == kTmaWarp) {
        // ------------------------------------------ bf16: loads
        int issued = 0, issued_v = 0;
        {
            // A tile is one page: the row of the tile's key 0 (keys past the last one are masked, and
            // cleaned in the aggregation operand).  The score operand of a tile comes before the
            // aggregation operand of the tile before it, as their stages become free.
            int row0 = 0;
            for (int t = 0; t <= nt; ++t) {
                const uint32_t par = static_cast<uint32_t>((t >> 1) & 1) ^ 1;  // tile t - 2's products
                const int row1 = row0, st = t & 1;
                if (t < nt) {
                    row0 = __shfl_sync(0xffffffffu, keys.row, 0);
                    if (t >= 2 && !wait(&bar_s[st], par, 1)) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&bar_kst[st], 9 * kKSlice);
                        for (int sl = 0; sl < 8; ++sl)
                            tma_load_2d(sm + S::kOffK + (8 * st + sl) * kKSlice, &maps.c, &bar_kst[st], 64 * sl, row0 + own0);
                        tma_load_2d(sm + S::kOffR + st * kKSlice, &maps.kr, &bar_kst[st], 0, row0 + own0);
                    }
                    __syncwarp();
                    issued = t + 1;
                    keys.advance(ka, it, nt, t0 * kNK + lane);
                }
                if (t >= 1) {
                    const int u = t - 1, vs = u & 1;
                    if (u >= 2 && !wait(&bar_o[vs], static_cast<uint32_t>((u >> 1) & 1) ^ 1, 2)) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&bar_vst[vs], kVStage);
                        for (int sl = 0; sl < 4; ++sl)
                            tma_load_2d(sm + S::kOffV + vs * kVStage + sl * kVSlice, &maps.cv, &bar_vst[vs],
                                        256 * (sl >> 1) + 128 * static_cast<int>(rank) + 64 * (sl & 1), row1);
                    }
                    __syncwarp();
                    issued_v = t;
                }
            }
            if (keys.broken) record_error(a.err, kErrMlaIndex);
            drain(&s_abort, bar_kst, 2, issued, lane);
            drain(&s_abort, bar_vst, 2, issued_v, lane);
        }
    } else if (kQ8 && warp >= kKWarp0 && warp < kMmaWarp) {
        // ------------------------------------------ e4m3 rows into an operand.  Scores: own rows 4 lw ..
        // 4 lw + 3 of a tile, a row of 32 pieces of 16 dims per load; aggregation: rows 8 lw .. 8 lw + 3 of it in
        // the lower half warp, 8 lw + 4 .. in the upper, the 16 pieces of this CTA's 256 dims.  Loads are
        // whole 128-byte lines.  A piece becomes two 16-byte ones of the operand, the later one first in odd
        // 64-dim slices: so the eight lanes of a store phase, which span two slices, touch distinct banks.
        const bool v = warp >= kVWarp0;
        const int lw = warp - (v ? kVWarp0 : kKWarp0);
        const int row0 = v ? 8 * lw + 4 * (lane >> 4) : own0 + 4 * lw;     // of the tile
        const int blk = v ? lane >> 3 & 1 : lane >> 3;                     // 128-dim block of the lane's pieces
        const uint8_t* src0 = static_cast<const uint8_t*>(a.c_cache) + (v ? 256 * blk + 128 * rank : 128 * blk) + 16 * (lane & 7);
        const int sc_shift = v ? 16 * blk + 8 * static_cast<int>(rank) : 8 * blk;
        const uint32_t sl = 2 * blk + (lane >> 2 & 1);                     // 64-dim slice of the lane's pieces
        const uint32_t atom = v ? 8 * lw : 8 * (lw >> 1), r0 = v ? 4 * (lane >> 4) : 4 * (lw & 1);  // row0 in the operand
        const uint32_t dst0 = (v ? vbase : kbase) + sl * (v ? kVSlice : kKSlice) + (atom + r0) * 128 +
                              ((2 * (lane & 3) + (sl & 1) ^ r0) << 4);
        const uint32_t stage = v ? kVStage : 8 * kKSlice;
        const int rr = 4 * lw + (lane >> 3);  // own row whose RoPE piece lane % 8 this lane moves (scores)
        const uint32_t rdst = smem_u32(sm + S::kOffR) + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4);
        uint64_t* freed = v ? bar_o : bar_s;
        // The next tile's loads are under way while the warp waits for its stage.
        uint4 u[4], kr = make_uint4(0u, 0u, 0u, 0u);
        int4 row;  // pool rows (-1: none) and scale words of rows row0 .. row0 + 3
        uint4 sc;
        auto fetch = [&](int t) {
            const int st = t % kRing;
            if (!wait(&bar_rows[st], static_cast<uint32_t>(t / kRing & 1), 7)) return false;
            row = *reinterpret_cast<const int4*>(&s_row[st][row0]);
            sc = *reinterpret_cast<const uint4*>(&s_scale[st][row0]);
            int rope = 0;
            if (!v) rope = s_row[st][own0 + rr];
            // (a slot without a row loads row 0: its scores are masked, its factor in the aggregation is 0)
            const int rows[4] = {row.x, row.y, row.z, row.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = ld_row16(src0 + static_cast<uint64_t>(static_cast<uint32_t>(max(rows[i], 0))) * static_cast<uint32_t>(a.c_ld));
            if (!v)
                kr = ld_row16(static_cast<const __nv_bfloat16*>(a.kr_cache) + 8 * (lane & 7) +
                              static_cast<uint64_t>(static_cast<uint32_t>(max(rope, 0))) * static_cast<uint32_t>(a.kr_ld));
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_rowsfree[st]);
            return true;
        };
        bool ok = true;
        int t = 0;
#pragma unroll 1
        for (int n = 0; ok && n < n_items; ++n) {
            if (n > 0) {  // the next item's query, when the last scores are done
                if (!wait(&bar_s[(t - 1) & 1], static_cast<uint32_t>((t - 1) >> 1 & 1), 7)) break;
                load_queries<kQ8>(a, smem_u32(sm + S::kOffQ), static_cast<int64_t>(it.b + n * ka.stride) * a.H + rank * kRows,
                                  a.H - static_cast<int>(rank) * kRows, warp - kKWarp0, 2 * kLoadWarps);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(mapa_u32(smem_u32(&bar_query), 0));
            }
            ok = fetch(t);
#pragma unroll 1
            for (int left = nt; ok && left > 0; --left, ++t) {
                const int tf = t - 2;  // the tile whose products free the stage
                if (tf >= 0 && !wait(&freed[tf & 1], static_cast<uint32_t>(tf >> 1 & 1), 8)) {
                    ok = false;
                    break;
                }
                const uint32_t at = dst0 + (t & 1) * stage;
                const bool big = __any_sync(0xffffffffu, ((sc.x | sc.y | sc.z | sc.w) & 0x80808080u) != 0);
                const int rows[4] = {row.x, row.y, row.z, row.w};
                const uint32_t scs[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t e = scs[i] >> sc_shift & 255u;
                    uint4 lo, hi;
                    convert16(u[i], rows[i] < 0 ? 0u : q8_factor_bf16x2(e), lo, hi);
                    if (big) {  // scales of 2 and above: some may need a second factor
                        const uint32_t f2 = q8_excess_bf16x2(e);
                        times4(lo, f2);
                        times4(hi, f2);
                    }
                    const uint32_t dst = (at + i * 128) ^ (i << 4);  // (the swizzle's lower two bits)
                    st_smem_v4(dst, lo);
                    st_smem_v4(dst ^ 16, hi);
                }
                if (!v) st_smem_v4(rdst + (t & 1) * kKSlice, kr);
                // drafted rows' non-finite pieces (codes reach 448: only with scales above 1) stay out of the
                // aggregation and are NaN in the scores
                if (big && a.tree && (s_t0 + t + 1) * kNK > s_it.past) {
#pragma unroll 1
                    for (int i = max(0, s_it.past - (s_t0 + t) * kNK - row0); i < 4; ++i) {
                        const uint32_t dst = (at + i * 128) ^ (i << 4);
                        clean_piece(dst, ld_smem_v4(dst), v);
                        clean_piece(dst ^ 16, ld_smem_v4(dst ^ 16), v);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(v ? &bar_vdone[t & 1] : &bar_kdone[t & 1]);
                if (left > 1) ok = fetch(t + 1);
            }
        }
    } else if (!kQ8 && (warp == kKWarp0 || warp == kVWarp0)) {
        // ------------------------------------------ bf16 operands reported (and cleaned)
        const bool v = warp == kVWarp0;
        uint64_t* landed = v ? bar_vst : bar_kst;
        const uint32_t full = mapa_u32(smem_u32(v ? &bar_vfull[0] : &bar_kfull[0]), 0);
        for (int t = 0; t < nt; ++t) {
            const int st = t & 1;
            if (!wait(&landed[st], static_cast<uint32_t>(t >> 1 & 1), 13)) break;
            const int pos0 = (t0 + t) * kNK + (v ? 0 : own0);  // of the operand's row 0
            if ((t0 + t + 1) * kNK > it.past) {  // 16-byte pieces, row after row
                const uint32_t at0 = v ? vbase + st * kVStage : kbase + st * 8 * kKSlice, slice = v ? kVSlice : kKSlice;
                const int rows = v ? kNK : min(kOwn, it.n_keys - pos0);  // (scores of keys past the last are masked)
                const int lg = v ? 5 : 6;
#pragma unroll 1
                for (int q0 = max(0, it.past - pos0) << lg; q0 < rows * (1 << lg); q0 += 128) {  // four pieces a lane at once
                    uint32_t at[4];
                    uint4 w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int q = q0 + 32 * k + lane, j = q >> lg, p = q & ((1 << lg) - 1);
                        at[k] = at0 + (p >> 3) * slice + j * 128 + (((p & 7) ^ (j & 7)) << 4);
                        w[k] = j < rows ? ld_smem_v4(at[k]) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) clean_piece(at[k], w[k], v);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive_remote(full + 8 * st);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (rank == 0) {
            constexpr uint32_t id_qk = idesc_f32acc(1, 1, false, false, 128, kNK);
            constexpr uint32_t id_pv = idesc_f32acc(1, 1, false, true, 128, 256);
            const uint64_t qd = sdesc(smem_u32(sm + S::kOffQ), 16, 1024, kSw128);
            const uint64_t kd0 = sdesc(smem_u32(sm + S::kOffK), 16, 1024, kSw128);
            const uint64_t rd0 = sdesc(smem_u32(sm + S::kOffR), 16, 1024, kSw128);
            const uint64_t pd = sdesc(smem_u32(sm + S::kOffP), 16, 1024, kSw128);
            const uint64_t vd0 = sdesc(smem_u32(sm + S::kOffV), kVSlice, 1024, kSw128);
            bool ok = true;
            int g = 0;  // tiles before the item's
#pragma unroll 1
            for (int n = 0; ok && n < n_items; ++n, g += nt) {
                // the next item's query is in place
                if (n > 0 && !wait.pair(&bar_query, static_cast<uint32_t>(n & 1) ^ 1, 3)) break;
#pragma unroll 1
                for (int u = 0; u <= nt; ++u) {
                    if (u < nt) {  // scores(u)
                        const int t = g + u, sb = t & 1;
                        ok = wait.pair(&bar_kfull[sb], static_cast<uint32_t>(t >> 1 & 1), 3) &&
                             (t < 2 || wait(&bar_sfree[sb], static_cast<uint32_t>(t >> 1 & 1) ^ 1, 4));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t kd = kd0 + static_cast<uint32_t>(sb * (8 * kKSlice >> 4));
                        const uint64_t rd = rd0 + static_cast<uint32_t>(sb * (kKSlice >> 4));
                        const uint32_t sc = tmem + kColS + 32 * sb;
                        if (elect_one()) {
#pragma unroll 1
                            for (int sl = 0; sl < 9; ++sl) {  // 64-dim slices, 16 dims each
                                const uint64_t qs = qd + sl * (kQSlice >> 4), ks = sl < 8 ? kd + sl * (kKSlice >> 4) : rd;
#pragma unroll
                                for (int i = 0; i < 4; ++i) mma_bf16_pair(sc, qs + 2 * i, ks + 2 * i, id_qk, (sl | i) != 0 ? 1u : 0u);
                            }
                            tc_commit_pair(&bar_s[sb]);
                        }
                        __syncwarp();
                    }
                    if (u > 0) {  // aggregation(u - 1)
                        const int t = g + u - 1, st = t & 1;
                        ok = wait.pair(&bar_vfull[st], static_cast<uint32_t>(t >> 1 & 1), 5) &&
                             wait.pair(&bar_pfull, static_cast<uint32_t>(t & 1), 6) &&
                             (u > 1 || n == 0 || wait(&bar_ofree, static_cast<uint32_t>(n & 1) ^ 1, 6));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vd = vd0 + static_cast<uint32_t>(st * (kVStage >> 4));
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)  // 256 dims i / 4, 16 keys each
                                mma_bf16_pair(tmem + kColO + 128 * (i >> 2), pd + 2 * (i & 3),
                                              vd + (i >> 2) * (2 * kVSlice >> 4) + 128 * (i & 3), id_pv,
                                              u > 1 || (i & 3) != 0 ? 1u : 0u);
                            tc_commit_pair(&bar_o[st]);
                        }
                        __syncwarp();
                    }
                }
            }
            if (elect_one()) tc_commit_pair(&bar_final);
            __syncwarp();
        }
    }
    if (warp < kSmxWarps) {
        // ---------------------------------------------- softmax + output
        // row of this CTA; the row's half of the keys (and of the output dims), by tensor-memory lane; quarter of them
        const int r = tid & 63, hf = tid >> 6 & 1, qd = tid >> 7;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t sfree0 = mapa_u32(smem_u32(&bar_sfree[0]), 0), pfull0 = mapa_u32(smem_u32(&bar_pfull), 0);
        const uint32_t prow = smem_u32(sm + S::kOffP) + r * 128;
        // scores in base-2 units (the queries carry the sign; never 0, so that masked scores stay -inf)
        const float c2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-37f);
        bool ok = true;
        // which of this thread's 16 keys of the item's tile t its row attends to.  Selections: the
        // slots of eight tiles are loaded eight tiles ahead (the fence that publishes P waits for
        // loads in flight): the half's 32 of a tile per load, lane u holding tile u's mask, or, with
        // registers short (kMany), this thread's 16 of two tiles, lane u holding tiles 2 u and 2 u + 1.
        constexpr int kLoads = kMany ? 4 : 8;
        int slots[kLoads];
        uint32_t vis8 = 0;
        auto load_slots = [&](int n, int t) {  // of the pair's n-th item
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int tile = kMany ? t + 2 * u + (lane >> 4) : t + u;
                const int s = (s_t0 + tile) * kNK + hf * 32 + (kMany ? qd * 16 + (lane & 15) : lane);
                slots[u] = tile < nt && s < a.k ? a.idx[static_cast<int64_t>(s_it.b + n * ka.stride) * a.k + s] : -1;
            }
        };
        auto next_slots = [&](int n, int t) {
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const uint32_t v = __ballot_sync(0xffffffffu, slots[u] >= 0);
                if (lane == u) vis8 = v;
            }
            load_slots(n, t + 8);
        };
        auto visible = [&](int n, int t) -> uint32_t {
            if (a.idx) {
                if ((t & 7) == 0) next_slots(n, t);
                if (kMany) return __shfl_sync(0xffffffffu, vis8, t >> 1 & 3) >> (16 * (t & 1)) & 0xFFFFu;
                return __shfl_sync(0xffffffffu, vis8, t & 7) >> (16 * qd) & 0xFFFFu;
            }
            const int s0 = (s_t0 + t) * kNK + hf * 32 + qd * 16, past = s_it.past;
            if (s0 + 16 <= past) return 0xFFFFu;
            const int m_row = static_cast<int>(cluster_rank()) * kRows + r;
            const int token = s_it.i0 + (m_row < s_it.tokens * a.H ? m_row / a.H : 0);
            uint32_t v = s0 < past ? (1u << (past - s0)) - 1u : 0u;
            const int keys = min(16, s_it.n_keys - s0);
            const uint8_t* mk = a.tree_mask ? a.tree_mask + (static_cast<int64_t>(s_it.b) * a.T + token) * a.T : nullptr;
#pragma unroll 1
            for (int j = max(0, past - s0); j < keys; ++j) {
                const int d = s0 + j - past;
                if (mk ? mk[d] != 0 : d <= token) v |= 1u << j;
            }
            return v;
        };
        if (a.idx) load_slots(0, 0);
        int t = 0;  // of the pair's tiles
#pragma unroll 1
        for (int n = 0; n < n_items; ++n) {
            float m = -INFINITY, l = 0.f, lr = 0.f;  // lr: the sum of the rounded weights
            bool failed = false;
#pragma unroll 1
            for (int u = 0; u < nt; ++u, ++t) {
                const int sb = t & 1;
                const uint32_t vis = visible(n, u);
                ok = ok && wait(&bar_s[sb], static_cast<uint32_t>((t >> 1) & 1), 8);
                float s[16];
                if (ok) {
                    tc_fence_after();
                    uint32_t v[16];
                    tmem_ld16(tmem + lane_base + kColS + 32 * sb + 16 * qd, v);
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(sfree0 + 8 * sb);
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = __uint_as_float(v[j]);
                    if (!__all_sync(0xffffffffu, vis == 0xFFFFu)) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (!(vis >> j & 1u)) s[j] = -INFINITY;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = -INFINITY;
                    if (lane == 0) s_fail[sb] = 1;
                }
                const float mx = tree_max(s) * c2;
                s_max[sb][tid] = mx;
                named_sync(1, 32 * kSmxWarps);
                // a failed wait before this barrier is seen by all four warps after it (the flag
                // of the next tile is another word), so they leave the loop together
                if (s_fail[sb]) {
                    ok = false;
                    failed = true;
                    break;
                }
                const float top = fmaxf(fmaxf(mx, s_max[sb][tid ^ 64]), fmaxf(s_max[sb][tid ^ 128], s_max[sb][tid ^ 192]));
                const bool grow = top > m + kRescaleLog2;
                if (__any_sync(0xffffffffu, grow)) {
                    const float m_new = grow ? top : m;
                    const float alpha = grow ? (m == -INFINITY ? 0.f : fast_exp2(m - m_new)) : 1.f;
                    if (u > 0) {  // O holds the item's tiles before this one
                        ok = wait(&bar_o[(t - 1) & 1], static_cast<uint32_t>((t - 1) >> 1 & 1), 9);
                        if (ok) {
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 128 * qd; c < 128 * qd + 128; c += 32) {
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
                    lr *= alpha;
                    m = m_new;
                }
                const float mref = m == -INFINITY ? 0.f : m;  // masked keys are -inf and give exactly 0
                uint32_t pk[8];
                float sum = 0.f, sumr = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p0 = fast_exp2(s[2 * j] * c2 - mref), p1 = fast_exp2(s[2 * j + 1] * c2 - mref);
                    sum += p0 + p1;
                    pk[j] = pack_bf16x2(p0, p1);
                    sumr += __uint_as_float(pk[j] << 16) + __uint_as_float(pk[j] & 0xFFFF0000u);
                }
                l += sum;
                lr += sumr;
                // aggregation(t - 1) has read P
                if (ok && t > 0)
                    ok = wait(&bar_o[(t - 1) & 1], static_cast<uint32_t>((t - 1) >> 1 & 1), 10);
                if (ok) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        st_smem_v4(prow + (((4 * hf + 2 * qd + q) ^ (r & 7)) << 4),
                                   make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]));
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(pfull0);
                }
            }
            // ---- the row's sums, then the rows out: staged over the idle operands, bulk copies
            s_sum[0][tid] = l;
            s_sum[1][tid] = lr;
            named_sync(1, 32 * kSmxWarps);
            l = (s_sum[0][r] + s_sum[0][r + 64]) + (s_sum[0][r + 128] + s_sum[0][r + 192]);  // (one order in all four)
            lr = (s_sum[1][r] + s_sum[1][r + 64]) + (s_sum[1][r + 128] + s_sum[1][r + 192]);
            const int m_row = static_cast<int>(cluster_rank()) * kRows + r;
            const bool live = m_row < s_it.tokens * a.H;
            const int64_t orow = (static_cast<int64_t>(s_it.b + n * ka.stride) * a.T + s_it.i0) * a.H + m_row;
            const bool last = n + 1 == n_items;
            uint8_t* dst = nullptr;
            if (ok && nt > 0)
                ok = wait(&bar_o[(t - 1) & 1], static_cast<uint32_t>((t - 1) >> 1 & 1), 11);
            if (ok && !*wait.abort) {
                tc_fence_after();
                const bool partial = s_it.splits > 1;
                const int64_t wrow = (static_cast<int64_t>(item) * ka.nsplit + split) * 128 + m_row;
                const bool empty = l == 0.f;  // (a NaN sum is not empty)
                // divided by the rounded weights' sum; a split's share of the row is that of its weights
                const float inv = empty ? 1.f : (partial ? l : 1.f) / lr;
                const bool bf = !partial && a.out_bf16 != nullptr;
                dst = partial ? reinterpret_cast<uint8_t*>(ka.ws_o + wrow * 512)
                              : (bf ? static_cast<uint8_t*>(a.out_bf16) + orow * 1024 : reinterpret_cast<uint8_t*>(a.out + orow * 512));
                // a thread's 128 dims: the last item's staged over the idle operands (bulk copies), the others', while
                // the next item's tiles are under way, straight to memory
                uint8_t* to = last ? sm + r * kORow : dst;
                constexpr int kCols = kMany ? 16 : 32;
#pragma unroll 1
                for (int c = 128 * qd; c < 128 * qd + 128; c += kCols) {
                    const int d = qd * 256 + hf * 128 + (c & 127);
                    const int swap = kQ8 ? (c & 64) >> 3 : 0;  // groups of eight dims are swapped in odd slices
                    uint32_t o[kCols];
                    if (nt > 0) {
                        if constexpr (kMany)
                            tmem_ld16(tmem + lane_base + kColO + c, o);
                        else
                            tmem_ld32(tmem + lane_base + kColO + c, o);
                        tmem_ld_wait();
                    }
                    if (live) {
#pragma unroll
                        for (int j = 0; j < kCols; j += 8) {
                            float f[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int at = kQ8 && ((i & 3) == 1 || (i & 3) == 2) ? i ^ 3 : i;  // dims in the order 0, 2, 1, 3
                                f[i] = empty ? 0.f : __uint_as_float(o[j + at]) * inv;
                            }
                            if (bf) {
                                *reinterpret_cast<uint4*>(to + 2 * (d + (j ^ swap))) =
                                    make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
                            } else {
                                float4* at = reinterpret_cast<float4*>(to + 4 * (d + (j ^ swap)));
                                at[0] = make_float4(f[0], f[1], f[2], f[3]);
                                at[1] = make_float4(f[4], f[5], f[6], f[7]);
                            }
                        }
                    }
                    __syncwarp();  // (the loads are the whole warp's)
                }
                if (live && tid < kRows) {
                    if (partial)
                        *reinterpret_cast<float2*>(ka.ws_ml + wrow * 2) = make_float2(m, l);
                    else if (a.lse)
                        a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                }
                tc_fence_before();
                __syncwarp();
                if (kMany && lane == 0) mbar_arrive_cluster_relaxed(mapa_u32(smem_u32(&bar_ofree), 0));  // O is read
                if (last) fence_proxy_async_smem();
            }
            if (failed) break;  // (all eight warps)
            if (last) {
                named_sync(1, 32 * kSmxWarps);  // the threads of a row have staged it (one bulk copy per row)
                if (ok && !*wait.abort && live && tid < kRows) {
                    bulk_copy_s2g(dst, sm + r * kORow, s_it.splits == 1 && a.out_bf16 ? 1024 : 2048);
                    bulk_wait_all();
                }
            } else {
                load_slots(n + 1, 0);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        // Every product has finished, and the last arrival this CTA gets has come, before the pair tears down.  The
        // roles have ended, so what is left is work in flight (fixed limit), and for the odd CTA the even one's way
        // to its last commit, which a wait of the even one's may hold up (kMaxWait32Ns at most).
        if (lane == 0) {
            if (nt > 0 && !Waits::own(&bar_final, 0, static_cast<uint32_t>(rank ? 3 * kWaitLimitNs : kWaitLimitNs))) s_abort = 12;
            if (*wait.abort) record_error(a.err, kErrLatWait | *wait.abort);
        }
        __syncwarp();
    }
    cluster_sync_all();  // no more remote arrivals, stores or products in either CTA
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

// Merge the split partial states: one warp per query row and 128 of its dims,
// four per lane; the loads of eight splits are under way together.
constexpr int kCombThreads = 256;

__global__ void __launch_bounds__(kCombThreads) mla_latent_combine_kernel(const Args ka) {
    pdl_wait();
    const LatentArgs& a = ka.a;
    const int64_t orow = static_cast<int64_t>(blockIdx.x) * (kCombThreads / 128) + (threadIdx.x >> 7);
    const int p = threadIdx.x >> 5 & 3;  // quarter of the dims
    if (orow >= static_cast<int64_t>(a.B) * a.T * a.H) return;
    const int lane = threadIdx.x & 31;
    const int h = static_cast<int>(orow % a.H), token = static_cast<int>(orow / a.H % a.T);
    const int b = static_cast<int>(orow / a.H / a.T);
    if (a.tree && a.n_draft && token >= a.n_draft[b]) return;
    const int item = b * ka.groups + token / ka.tokens_per_item;
    const int splits = item_of(ka, item).splits;
    if (splits == 1) return;  // (written by its pair)
    const int64_t w0 = static_cast<int64_t>(item) * ka.nsplit * 128 + token % ka.tokens_per_item * a.H + h;
    // lane s holds split s's state
    float ms = -INFINITY, ls = 0.f;
    if (lane < splits) {
        const float2 v = *reinterpret_cast<const float2*>(ka.ws_ml + (w0 + static_cast<int64_t>(lane) * 128) * 2);
        ms = v.x, ls = v.y;
    }
    float top = ls != 0.f ? ms : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float wgt = ls != 0.f ? exp2f(ms - top) : 0.f;
    float L = ls * wgt;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4* src = reinterpret_cast<const float4*>(ka.ws_o + w0 * 512) + 32 * p + lane;
    for (int s0 = 0; s0 < splits; s0 += 8) {
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s0 + i < splits) v[i] = src[static_cast<int64_t>(s0 + i) * 128 * 128];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float w = __shfl_sync(0xffffffffu, wgt, s0 + i);  // (s0 + i < 32: weights past the splits are 0)
            acc.x += v[i].x * w, acc.y += v[i].y * w, acc.z += v[i].z * w, acc.w += v[i].w * w;
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const float x = acc.x * inv, y = acc.y * inv, z = acc.z * inv, w = acc.w * inv;
    if (a.out_bf16)
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out_bf16) + orow * 1024 + 256 * p + 8 * lane) =
            make_uint2(pack_bf16x2(x, y), pack_bf16x2(z, w));
    else
        *reinterpret_cast<float4*>(a.out + orow * 512 + 128 * p + 4 * lane) = make_float4(x, y, z, w);
    if (a.lse && p == 0 && lane == 0) a.lse[orow] = L == 0.f ? -INFINITY : (top + log2f(L)) * 0.6931471805599453f;
}

int tokens_per_item(int T, int H) {
    const int p = 128 / H;
    return p < 1 ? 1 : (p < T ? p : T);
}

// Key splits of every item: as many as fill the GPU's CTA pairs, each of at least
// three tiles.
int base_splits(int64_t items, int k) {
    const int64_t pairs = sm_count() / 2;
    const int tiles = (k + kNK - 1) / kNK;
    int64_t ns = items >= pairs ? 1 : pairs / items;
    if (ns > tiles / 3) ns = tiles / 3;
    if (ns > kMaxSplits) ns = kMaxSplits;
    return ns < 1 ? 1 : static_cast<int>(ns);
}

// Of the longest item: k may be a bound far above the lengths, so an item takes no
// more than its own length asks for (64 rows of 4096 positions 115 us; under a bound
// of 2^20 126, and 171 if they took the bound's splits).
int most_splits(int64_t items, int k) {
    const int of_length = static_cast<int>((static_cast<int64_t>(k) + kLongKeys - 1) / kLongKeys);
    return std::max(base_splits(items, k), std::min(of_length, kMaxSplits));
}

size_t state_bytes(int64_t items, int ns) { return static_cast<size_t>(items) * ns * 128 * (512 + 2) * 4; }

template <bool kQ8, bool kMany>
sa_status launch(const Args& ka, int64_t items, cudaStream_t st) {
    const LatentArgs& a = ka.a;
    Maps maps = {};
    if (!kQ8) {
        const uint64_t rows = static_cast<uint64_t>(a.pool_pages) * kPage;
        const uint64_t dims[2] = {512, rows}, rdims[2] = {64, rows};
        const uint64_t stride[1] = {static_cast<uint64_t>(a.c_ld) * 2}, rstride[1] = {static_cast<uint64_t>(a.kr_ld) * 2};
        const uint32_t half[2] = {64, kOwn}, whole[2] = {64, kNK};
        if (!encode_tiled(&maps.c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.c_cache, dims, stride, half, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_tiled(&maps.cv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.c_cache, dims, stride, whole, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_tiled(&maps.kr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.kr_cache, rdims, rstride, half, CU_TENSOR_MAP_SWIZZLE_128B))
            return SA_ECUDA;
    }
    const cudaError_t e = cudaFuncSetAttribute(mla_latent_kernel<kQ8, kMany>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<kQ8>::kBytes);
    if (e != cudaSuccess) return launch_status(e);
    const int64_t clusters = kMany ? ka.stride : items * ka.nsplit;
    mla_latent_kernel<kQ8, kMany><<<static_cast<unsigned>(2 * clusters), kThreads, Smem<kQ8>::kBytes, st>>>(ka, maps);
    return launch_status(cudaGetLastError());
}

}  // namespace

size_t mla_latent_workspace_bytes(int B, int T, int H, int k) {
    const int P = tokens_per_item(T, H);
    const int64_t items = static_cast<int64_t>(B) * ((T + P - 1) / P);
    const int ns = most_splits(items, k);
    return ns > 1 ? state_bytes(items, ns) : 0;
}

sa_status mla_latent_launch(const LatentArgs& a, void* ws, size_t ws_bytes, cudaStream_t st) {
    Args ka = {};
    ka.a = a;
    ka.tokens_per_item = tokens_per_item(a.T, a.H);
    ka.groups = (a.T + ka.tokens_per_item - 1) / ka.tokens_per_item;
    const int64_t items = static_cast<int64_t>(a.B) * ka.groups;
    ka.nsplit = most_splits(items, a.k);
    ka.base = base_splits(items, a.k);
    ka.items = static_cast<int>(items);
    // Short selections, more of them than pairs, go to the pairs in turn (equal tiles each), so that an item's
    // query and first rows load behind the output before: 500 rows x 128 heads of 64 / 256 / 512 slots take
    // 79 / 115 / 171 us against 100 / 137 / 184 with a pair for each, 768 the same, 1024 285 against 273 (a tile
    // takes 2.0 us there against 1.56: the loops around the tiles' cost registers); 100 rows of 64 / 200 / 400
    // 25 / 37 / 49 against 27 / 38 / 48.
    if (a.idx && ka.nsplit == 1) {
        const int64_t pairs = sm_count() / 2, tiles = (a.k + kNK - 1) / kNK;
        if (items > pairs && (tiles <= 4 || (tiles <= 8 && items > 2 * pairs))) ka.stride = static_cast<int>(pairs);
    }
    if (ka.nsplit > 1) {
        if (!ws || ws_bytes < state_bytes(items, ka.nsplit)) return SA_EINVAL;
        ka.ws_o = static_cast<float*>(ws);
        ka.ws_ml = ka.ws_o + static_cast<size_t>(items) * ka.nsplit * 128 * 512;
    }
    const sa_status s = !a.c_scale ? launch<false, false>(ka, items, st)
                        : ka.stride ? launch<true, true>(ka, items, st) : launch<true, false>(ka, items, st);
    if (s == SA_OK && ka.nsplit > 1) {
        const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.H;
        constexpr int kPer = kCombThreads / 128;
        return launch_status(launch_pdl(mla_latent_combine_kernel, dim3(static_cast<unsigned>((rows + kPer - 1) / kPer)),
                                        dim3(kCombThreads), 0, st, ka));
    }
    return s;
}

}  // namespace sa
