// Attention of drafted tokens against a paged bf16 cache (fa_decode_paged_tree; definition in
// fa.h): every query sees its sequence's cached tokens, itself and its ancestors in the tree.
//
// The R = (H / Hkv) * Nq query rows of a key/value head are the M of the products, 128 rows to a
// block, one or two blocks per CTA that share each tile of keys on its way through shared memory:
//   S (128 rows x BK keys) = Q K^T        both from shared memory
//   O (128 rows x d)      += P V          P, bf16, from tensor memory over S's own columns
// A thread owns one row, so the running maximum and sum of the softmax are per-thread work without
// exchange, and so is the mask: a tile of keys behind the cached ones is looked up in the row's
// bits of the nodes that it sees (a tile before them is not masked at all).  The reference of a
// row's exponents moves only when a score passes it by 2^8; then the thread rescales its row of O.
// P is rounded to bf16 (2^-8 at most of each term, the sum of the row is taken before that): V is
// bf16, the product takes both of one type, and O is rounded to bf16 at the end all the same (2-norm
// error of O 2.1 to 2.4e-3, and 1.65e-3 where P is in fp32; a second product with what the rounding left
// would double the work of P V, which two blocks of rows are bound by).
//
// Work is cut over the CTAs as fa_cut.cuh describes.  Twelve warps: eight of softmax, which also write
// the results, two that issue products, one of which also brings the queries and makes the trees (which,
// below), and one each for the TMA copies of K and of V (issued one by one, a hundred clocks each: with one
// warp for both, pages of 16 made that the bound, B1 131072 keys R = 256 139 us).  Per CTA: a ring of
// K_0 V_0 K_1 V_1 ..., two S slots, one or two query buffers.
//
// Measured (GB300, with the merge; graph replay of one input, of which L2 keeps a part, then calls on
// inputs that change, and their rate):
//   B32 H32 Hkv8 Nq32 of 1..8192 keys   102 us, 103  5.5 TB/s  HBM between the items; 4 to 8k clocks for the
//                                                              results at the end of each, 10k to the first S
//   B1 H32 Hkv8 Nq64 131072 keys        110 us, 119  4.5 TB/s  3.1k clocks a tile: the chain of one block, 1.5k
//                                                              of softmax, 0.3k to P's being seen, 1.3k of P V
//                                                              and the next S, and the other block's turns;
//                                                              that is 81 to 87 us of 54 tiles, HBM alone takes
//                                                              80, and the ring holds two tiles only
//   B16 H64 Hkv8 Nq48 16384..32768      531 us, 573  2.9 TB/s  the same, 1.08 PFLOP/s; items of R = 256 and 128
//                                                              in turn, the latter with one block in flight
//   B8 H32 Hkv4 Nq4 d64 5000..32768      36 us, 37.7 4.3 TB/s  1.5k clocks a tile, of which HBM's rate needs
//                                                              1.4k, 9k to the first S, results, merge
//   B5 H16 Hkv2 Nq21 d256 101..2899      24 us, 24.5           parts: 3 tiles per CTA, whose results are as
//                                                              large as the keys and values that they read
//   B1 H32 Hkv8 Nq16 1000 keys         10.4 us, 10.8           latency of two launches: lengths, pages, first
//                                                              copies, results, merge
// Tried and slower: S slots of 64 keys, two per block (116 -> 197 us); a cluster of a CTA per block with
// the copies shared out and multicast (two tiles in the ring are too few: 150 us); one product of 256 rows
// by a pair of CTAs, each with half of K's rows and V's columns (330 us, the reason was not found); boxes of
// five dimensions that bring whole rows, half the copies (no difference); for up to 64 rows of d64 copies of
// them in every quarter of tensor memory, so that all warps share their softmax, P through shared memory
// (no difference with a warp for S and one for P V; a single short sequence 0.3 us slower); a round of the
// results' code before the first tile, to have it fetched (no difference in replay).
#include <type_traits>

#include "fa_cut.cuh"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr float kMoveLog2 = 8.0f;
constexpr int kMaxNodes = FA_MAX_TREE_NODES, kNodeWords = kMaxNodes / 32;

template <int D, int NB>  // NB: blocks of 128 rows in a CTA
struct TreeTile {
    static constexpr int DP = (D + 63) / 64 * 64;       // row width in shared memory
    static constexpr int NCH = DP / 64;                 // 128-byte swizzle spans per row
    static constexpr int BK = D == 256 ? 64 : 128;      // keys per tile
    static constexpr int RB = 128 * NB;                 // query rows per item
    // With one block, two softmax warpgroups, a thread for one half of the tile's keys each: the ring's V
    // slots are held for as long as a softmax takes (B32 R = 128 of 1..8192 keys: 120 -> 113 us).  With
    // two, a warpgroup for each (four: 115 -> 137 us, the MMA warp then issues late, and registers end).
    static constexpr int NH = NB == 1 ? 2 : 1;
    static constexpr int CB = BK / NH;                  // keys of a thread
    static constexpr int THREADS = 32 * 12;
    // (Two blocks: their softmax threads hold a row of 128 scores, the other warps little, so warpgroups
    // trade the launch's registers, 3 x 168, and every wait is inlined, as a called function has one
    // budget: 127 -> 113 us.)
    static constexpr bool TRADE = NB == 2;
    static constexpr int REG_SOFTMAX = 216, REG_OTHERS = 72;
    static_assert(2 * REG_SOFTMAX + REG_OTHERS <= 3 * 168, "registers of the launch");
    static constexpr uint32_t SPAN = BK * 128;
    static constexpr uint32_t SLOT = NCH * SPAN;
    static constexpr uint32_t Q_CHUNK = 128 * 128;
    static constexpr uint32_t Q_BLOCK = NCH * Q_CHUNK;
    static constexpr uint32_t Q_BYTES = NB * Q_BLOCK;
    static constexpr int QBUF = Q_BYTES <= 32 * 1024 ? 2 : 1;
    static constexpr uint32_t MISC = 24 * 1024;
    static constexpr int FIT = (int)((226 * 1024 - QBUF * Q_BYTES - MISC - 1024) / SLOT) / 2 * 2;
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;    // 128 KB of keys and values
    static constexpr uint32_t OFF_Q = STAGES * SLOT;
    static constexpr uint32_t OFF_MISC = OFF_Q + QBUF * Q_BYTES;
    static constexpr uint32_t SMEM = OFF_MISC + MISC + 1024;  // and room to align the start
    static constexpr uint32_t TM_O = 2 * BK;
    static constexpr uint32_t TM_USED = TM_O + NB * DP;
    static constexpr uint32_t TM_COLS = 512;
    static_assert(STAGES >= 4, "two tiles in the ring");
    static_assert(TM_USED <= 512, "tensor memory budget");
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

template <int STAGES, int NB>
struct TreeMisc {
    unsigned long long full[STAGES], empty[STAGES];
    // per block of rows, by its own tiles in turn: S is there, half of P, all of P, O is there.  (A warp may
    // come to wait for O of a tile before O of the last one is done, so these are two as well.)
    unsigned long long s_full[NB][2], p_half[NB][2], p_full[NB][2], pv_done[NB][2];
    unsigned long long q_full[2], q_empty[2], info_full[2], info_empty[2], done[2];
    uint32_t tmem;
    int abort;
    float trade[2][256];                  // what the threads of a row tell each other, by turns
    // per segment of this CTA's work, in turn:
    int bad_page[2], bad_tree[2];         // a page or a parent out of range
    int special_any[2];
    uint32_t special[2][kNodeWords];      // nodes whose values have infinities or NaN
    short up[kMaxNodes];                  // an ancestor, or -1
    alignas(16) uint32_t sees[2][kMaxNodes][kNodeWords];  // the nodes that a node sees, as bits
};

struct TreeArgs {
    static constexpr bool kKeepInfinities = true;  // a node's values may have them
    CUtensorMap tm_q, tm_k, tm_v;   // (d, B * H * Nq), box 64 x box_q; (d, page_size, num_pages *
                                    // Hkv), boxes 64 x box x 1
    const __nv_bfloat16 *v_cache;
    const int *block_table, *seq_lens, *parents;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o, *part_l;         // [CTA][2][item_rows][d], [CTA][2][item_rows]
    int4 *cuts;                     // [CTA]: the item that its range begins in the middle of: sequence,
                                    // number within it, its first CTA, its CTAs (0: none)
    FastDiv by_page;
    int B, H, Hkv, Nq, Nt, d, page_size, max_pages, num_pages;
    int R, row_blocks, item_rows;   // query rows per key/value head, items of up to RB of them
    int box, box_q;                 // rows of a TMA box
    int tile_log2;
    int start;
    int o_aligned;                  // o begins on 32 bytes (part_o always does)
    float scale_log2;
    int *status;
    unsigned long long limit_ns;
};

__device__ __forceinline__ bool len_ok(const TreeArgs &a, int len) {
    return len >= 0 && (long long)len <= (long long)a.page_size * a.max_pages;
}
__device__ __forceinline__ int tiles_of_len(const TreeArgs &a, int len) {
    return len_ok(a, len) ? (len + a.Nt + (1 << a.tile_log2) - 1) >> a.tile_log2 : 0;
}
// A sequence always has its nodes' tiles, so attention writes its rows.
__device__ __forceinline__ bool empty_len(const TreeArgs &, int) { return false; }

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// N = 2 or 4 steps of a product of 16 columns each, by one elected lane: as mma_ss_elect and
// mma_ts_elect, with one election for all.  Steps lie STEP_A and STEP_B units of 16 bytes apart (A in
// tensor memory: 8 columns); all but the first accumulate.
template <int N, uint32_t STEP_A, uint32_t STEP_B>
__device__ __forceinline__ void mma_ss_run(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    static_assert(N == 2 || N == 4, "steps of a run");
    if constexpr (N == 4)
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\telect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %10, 0;\n\tsetp.eq.b32 t, %10, %10;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %9, p;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %4, %9, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %5, %6, %9, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %7, %8, %9, t;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "l"(a + STEP_A), "l"(b + STEP_B), "l"(a + 2 * STEP_A), "l"(b + 2 * STEP_B),
            "l"(a + 3 * STEP_A), "l"(b + 3 * STEP_B), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\telect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, %6, %6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %5, p;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %4, %5, t;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "l"(a + STEP_A), "l"(b + STEP_B), "r"(idesc), "r"(accumulate)
            : "memory");
}
template <int N, uint32_t STEP_B>
__device__ __forceinline__ void mma_ts_run(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    static_assert(N == 2 || N == 4, "steps of a run");
    if constexpr (N == 4)
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\telect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %10, 0;\n\tsetp.eq.b32 t, %10, %10;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %9, p;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %4, %9, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], %6, %9, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%7], %8, %9, t;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(a + 8), "l"(b + STEP_B), "r"(a + 16), "l"(b + 2 * STEP_B), "r"(a + 24),
            "l"(b + 3 * STEP_B), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\telect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, %6, %6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %5, p;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %4, %5, t;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(a + 8), "l"(b + STEP_B), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Of a pair of bf16 values, the bits of those that are infinite or NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
    const uint32_t lo = (x & 0x7f80u) == 0x7f80u ? 0xffffu : 0u;
    const uint32_t hi = (x & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
    return lo | hi;
}

// 32 bytes of a thread's row, a whole sector of L2 (a warp's 16-byte stores to 32 rows leave every
// sector half written).
__device__ __forceinline__ void store32(void *dst, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

template <int D, int NB>
__global__ void __launch_bounds__(TreeTile<D, NB>::THREADS, 1)
    fa_tree_kernel(const __grid_constant__ TreeArgs a) {
    using T = TreeTile<D, NB>;
    constexpr int ST = T::STAGES, BK = T::BK, NH = T::NH, CB = T::CB, NCH = T::NCH, QBUF = T::QBUF;
    using Misc = TreeMisc<ST, NB>;
    static_assert(sizeof(Misc) <= T::MISC, "state fits behind the buffers");
    constexpr int kMmaWarp = 8, kTmaWarp = kMmaWarp + 1, kMmaWarp2 = kMmaWarp + 3;  // TMA: K, then V
    constexpr bool kIn = T::TRADE;
    extern __shared__ uint8_t tree_smem[];
    const uint32_t raw = smem_u32(tree_smem);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = tree_smem + (base - raw);
    Misc &ms = *reinterpret_cast<Misc *>(gbase + T::OFF_MISC);
    auto bar = [](unsigned long long &b) { return smem_u32(&b); };
    const uint32_t sQ = base + T::OFF_Q;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(bar(ms.full[s]), 1);
            mbar_init(bar(ms.empty[s]), 1);
        }
        for (int u = 0; u < 2; ++u) {
            for (int k = 0; k < NB; ++k) {
                mbar_init(bar(ms.s_full[k][u]), 1);
                mbar_init(bar(ms.p_full[k][u]), 4 * NH);  // one arrival per softmax warp
                if (NB == 2) mbar_init(bar(ms.p_half[k][u]), 4);  // P of the first half of the keys
                mbar_init(bar(ms.pv_done[k][u]), 1);
            }
            mbar_init(bar(ms.q_full[u]), 1);
            mbar_init(bar(ms.q_empty[u]), 1);
            mbar_init(bar(ms.info_full[u]), 1);
            mbar_init(bar(ms.info_empty[u]), 8);
        }
        for (int u = 0; u < 2; ++u) mbar_init(bar(ms.done[u]), 1);
        ms.abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&ms.tmem), T::TM_COLS);
        tmem_relinquish();
    }
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_desc(&a.tm_q);
        tma_prefetch_desc(&a.tm_k);
        tma_prefetch_desc(&a.tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem;
    const Guard g{a.status, &ms.abort, a.limit_ns};

    // What the kernels before this one wrote is there from here on.
    griddep_wait();
    griddep_launch_dependents();

    // Every warp finds the CTA's first tile for itself.
    Cut cut;
    Walk walk = start_walk(a, blockIdx.x, gridDim.x, &cut);
    Segment s{};
    auto rows_of = [&](const Segment &x) { return min(a.item_rows, a.R - x.rb * a.item_rows); };
    auto blocks_of = [&](const Segment &x) { return NB == 1 ? 1 : (rows_of(x) + 127) / 128; };

    if (warp == kMmaWarp2) {  // for the merge
        int4 item = make_int4(walk.b, walk.item, 0, 0);
        if (walk.left > 0 && walk.tile() > 0) {
            const int first = cut.first((int)blockIdx.x) - walk.tile();
            item.z = cut.owner(first);
            item.w = cut.owner(first + walk.nt - 1) - item.z + 1;
        }
        if (lane == 0) a.cuts[blockIdx.x] = item;
    }

    // ---------------------------------------------------------------- products
    constexpr uint32_t kIdescS = idesc_bf16_f32(128, BK, false, false);
    constexpr uint32_t kIdescO = idesc_bf16_f32(128, D, false, true);
    constexpr int kRun = CB / 16 < 4 ? CB / 16 : 4;
    const uint64_t d_q = sdesc_sw128(sQ, 16, 1024), d_k = sdesc_sw128(base, 16, 1024);
    const uint64_t d_v = sdesc_sw128(base, T::SPAN, 1024);
    struct Slot {  // a ring slot of K or V and the parity of its round
        int at;
        uint32_t round;
        __device__ __forceinline__ void advance() {
            at += 2;
            if (at >= ST) at -= ST, round ^= 1;
        }
    };
    auto product_s = [&](int qb, int blk, uint32_t at, int ring) {
        tc_fence_after();
        const uint64_t dq = desc_add(d_q, qb * T::Q_BYTES + blk * T::Q_BLOCK), dk = desc_add(d_k, ring * T::SLOT);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            mma_ss_run<4, 2, 2>(tmem + at * BK, desc_add(dq, c * T::Q_CHUNK), desc_add(dk, c * T::SPAN), kIdescS,
                                c > 0 ? 1u : 0u);
        if constexpr (D % 64 == 32)
            mma_ss_run<2, 2, 2>(tmem + at * BK, desc_add(dq, D / 64 * T::Q_CHUNK), desc_add(dk, D / 64 * T::SPAN),
                                kIdescS, 1u);
    };
    auto product_o = [&](int blk, uint32_t at, bool first, int ring, int from = 0, int to = T::BK / 16) {
        tc_fence_after();
        const uint64_t dv = desc_add(d_v, ring * T::SLOT);
#pragma unroll
        for (int ks = from; ks < to; ks += kRun) {
            const uint64_t dvk = desc_add(dv, ks * 2048);
            const uint32_t more = (!first || ks > 0) ? 1u : 0u;
            mma_ts_run<kRun, 128>(tmem + T::TM_O + blk * T::DP,
                                  tmem + at * BK + ks / (CB / 16) * CB + ks % (CB / 16) * 8, dvk, kIdescO, more);
        }
    };
    // Waits until every MMA that this warp has issued has completed (normal or aborted run).
    auto drain = [&](uint32_t done) {
        tc_commit_elect(done);
        volatile int never = 0;
        const Guard g2{a.status, &never, kWaitLimitNs};
        mbar_wait_warp<kIn>(done, 0, g2, SITE_DEC_DRAIN);
    };

    // ------------------------------------------------------ queries and trees
    // The query rows of segment n, x; rows behind them in the last box are other heads', or zeros
    // past the tensor, and what they give is dropped.
    auto put_queries = [&](const Segment &x, uint32_t n) {
        const int qb = (int)(n % QBUF), nb = blocks_of(x);
        if (n >= (uint32_t)QBUF &&
            !mbar_wait_warp<kIn>(bar(ms.q_empty[qb]), ((n / QBUF) - 1) & 1, g, SITE_DEC_EMPTY))
            return false;
        if (lane == 0) {
            const uint32_t fb = bar(ms.q_full[qb]);
            mbar_arrive_expect_tx(fb, (uint32_t)(nb * NCH * a.box_q) * 128u);
            const int row0 = (int)(((long long)x.b * a.Hkv + x.kvh) * a.R + (long long)x.rb * a.item_rows);
            for (int k = 0; k < nb; ++k)
                for (int c = 0; c < NCH; ++c)
                    tma_load_3d(sQ + qb * T::Q_BYTES + k * T::Q_BLOCK + c * T::Q_CHUNK, &a.tm_q, fb, c * 64,
                                row0 + 128 * k, 0);
        }
        __syncwarp();
        return true;
    };
    // After an abort: queries under way have to land before the CTA exits.
    auto drain_queries = [&](uint32_t sent) {
        if (!*g.abort) return;
        volatile int never = 0;
        const Guard g2{a.status, &never, kWaitLimitNs};
        for (uint32_t i = sent > (uint32_t)QBUF ? sent - QBUF : 0; i < sent; ++i)
            mbar_wait_warp<kIn>(bar(ms.q_full[i % QBUF]), (i / QBUF) & 1, g2, SITE_DEC_DRAIN);
    };
    // What a node sees, as bits: itself and, in rounds that double the reach, what the farthest ancestor
    // that it has come to sees.  Lane i has nodes i, 32 + i, ...; a parent's number is below its child's,
    // so from the last 32 nodes to the first each round reads what the one before it left.
    auto put_tree = [&](const Segment &x, uint32_t n) {
        const int ib = n & 1;
        if (n >= 2 && !mbar_wait_warp<kIn>(bar(ms.info_empty[ib]), ((n >> 1) - 1) & 1, g, SITE_DEC_EMPTY))
            return false;
        if (lane < kNodeWords) ms.special[ib][lane] = 0;
        bool bad = false;
        if (a.parents) {
            const int *parents = a.parents + (size_t)x.b * a.Nt;
            const int groups = (a.Nt + 31) / 32;
            bool any = false;
            for (int k = 0; k < groups; ++k) {
                const int j = 32 * k + lane;
                int up = j < a.Nt ? parents[j] : -2;
                const bool is = up >= -1;
                if (up >= j || (up >= 0 && parents[up] < -1)) {
                    bad = true;
                    up = -1;
                }
                if (up < -1) up = -1;
                any = any || up >= 0;
                ms.up[j] = (short)up;
#pragma unroll
                for (int w = 0; w < kNodeWords; w += 4)
                    *reinterpret_cast<uint4 *>(&ms.sees[ib][j][w]) = make_uint4(0u, 0u, 0u, 0u);
                if (is) ms.sees[ib][j][k] = 1u << lane;
            }
            bad = __any_sync(kFull, bad);
            __syncwarp();
            while (__any_sync(kFull, any)) {
                any = false;
                for (int k = groups - 1; k >= 0; --k) {
                    const int j = 32 * k + lane, up = ms.up[j];
                    uint4 far[kNodeWords / 4] = {};
                    int next = -1;
                    if (up >= 0) {
#pragma unroll
                        for (int w = 0; w < kNodeWords / 4; ++w)
                            far[w] = *reinterpret_cast<const uint4 *>(&ms.sees[ib][up][4 * w]);
                        next = ms.up[up];
                    }
                    __syncwarp();
                    if (up >= 0) {
#pragma unroll
                        for (int w = 0; w < kNodeWords / 4; ++w) {
                            uint4 *to = reinterpret_cast<uint4 *>(&ms.sees[ib][j][4 * w]);
                            const uint4 y = *to;
                            *to = make_uint4(far[w].x | y.x, far[w].y | y.y, far[w].z | y.z, far[w].w | y.w);
                        }
                        ms.up[j] = (short)next;
                        any = any || next >= 0;
                    }
                    __syncwarp();
                }
            }
        }
        if (lane == 0) {
            ms.bad_tree[ib] = bad;
            ms.special_any[ib] = 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ms.info_full[ib]));
        return true;
    };
    auto check_lengths = [&]() {
        if (blockIdx.x != 0) return;
        bool good = true;
        for (int b = lane; b < a.B; b += 32) good = good && len_ok(a, a.seq_lens[b]);
        if (!__all_sync(kFull, good) && lane == 0) {
            atomicCAS(a.status + 1, 0, SITE_TREE_BAD_LEN);
            atomicExch(a.status, FA_ERR_BAD_INDEX);
        }
    };

    // One block: a warp for S = Q K^T, the queries and the trees, one for O += P V.  (A warp with all
    // products takes 1.5k to 1.9k clocks to issue those of a tile, of waits, commits and descriptors: B32
    // R = 128 of 1..8192 keys 104 -> 101 us, B4 R = 32 of d96 14.0 -> 12.2.)  Two blocks: all products from
    // one warp, in a fixed order (taken as they get ready: B1 R = 256 of 131072 keys 115 -> 111 us), the
    // other prepares.  (From two warps, by kind or by block, products mix on their way, which slows both:
    // 125 to 137 us.)
    if (warp == kTmaWarp || warp == kTmaWarp + 1) {
        // ------------------------------------------------------------ K, or V
        if constexpr (T::TRADE) setmaxnreg_dec<T::REG_OTHERS>();
        // A tile is a run of boxes of `box` rows (the largest power of two that divides a page's
        // rows, so a box never straddles two pages); lane i looks up and copies box i (and i +
        // 32, ... of pages that allow only tiny boxes).  Boxes behind the last node are not copied.
        const bool is_v = warp != kTmaWarp;
        const CUtensorMap *map = is_v ? &a.tm_v : &a.tm_k;
        uint32_t n = is_v, seg = 0;  // ring slots up to this warp's next; segments begun
        bool ok = true;
        const int boxes = BK / a.box;
        for (; ok && walk.next(a, &s); ++seg) {
            const int ib = seg & 1, len = a.seq_lens[s.b], keys = len + a.Nt;
            const int *bt = a.block_table + (size_t)s.b * a.max_pages;
            // page of the key that is `at` keys into tile t, -1 where there is none
            auto page_at = [&](int t, int at) {
                const int key = t * BK + at;
                if (t >= s.t1 || key >= keys) return -1;
                const uint32_t i = a.by_page.div((uint32_t)key);
                return i < (uint32_t)a.max_pages ? __ldg(bt + i) : -1;
            };
            auto valid = [&](int page) { return page >= 0 && page < a.num_pages; };
            int pg = lane < boxes ? page_at(s.t0, lane * a.box) : -1;
            if (!is_v) {
                if (seg >= 2)  // `bad_page` of the segment before the last has been read
                    ok = mbar_wait_warp<kIn>(bar(ms.info_empty[ib]), ((seg >> 1) - 1) & 1, g, SITE_DEC_EMPTY);
                if (!ok) break;
                if (lane == 0) ms.bad_page[ib] = 0;
                __syncwarp();
            }
#pragma unroll 1
            for (int t = s.t0; ok && t < s.t1; ++t, n += 2) {
                const int pg_next = lane < boxes ? page_at(t + 1, lane * a.box) : -1;
                const int slot = (int)(n % ST);
                ok = n < (uint32_t)ST ||
                     mbar_wait_warp<kIn>(bar(ms.empty[slot]), ((n / ST) - 1) & 1, g, SITE_DEC_EMPTY);
                if (!ok) break;
                const uint32_t fb = bar(ms.full[slot]), dst = base + slot * T::SLOT;
#pragma unroll 1
                for (int i0 = 0; i0 < boxes; i0 += 32) {
                    const int i = i0 + lane, key = t * BK + i * a.box;
                    const int page = i0 == 0 ? pg : page_at(t, i * a.box);
                    const bool copy = i < boxes && valid(page);
                    if (!is_v && !copy && i < boxes && key < keys) {
                        // wrong if it holds a token: places without a node do not
                        bool token = key < len || !a.parents;
                        for (int j = key - len; !token && j < min(key - len + a.box, a.Nt); ++j)
                            token = a.parents[(size_t)s.b * a.Nt + j] >= -1;
                        if (token) ms.bad_page[ib] = 1;
                    }
                    const int mine = __popc(__ballot_sync(kFull, copy));
                    __syncwarp();  // lane 0's arrival passes on what any lane has found
                    if (lane == 0) {
                        // the phase's one arrival comes with its last boxes
                        const uint32_t bytes = (uint32_t)(mine * a.box) * (uint32_t)(NCH * 128);
                        if (i0 + 32 < boxes) mbar_expect_tx(fb, bytes);
                        else mbar_arrive_expect_tx(fb, bytes);
                    }
                    __syncwarp();
                    if (copy) {
                        const int y = key - (int)a.by_page.div((uint32_t)key) * a.page_size;
                        const int z = page * a.Hkv + s.kvh;
                        const uint32_t to = dst + i * a.box * 128;
#pragma unroll
                        for (int c = 0; c < NCH; ++c) tma_load_3d(to + c * T::SPAN, map, fb, c * 64, y, z);
                    }
                    __syncwarp();
                }
                pg = pg_next;
            }
        }
        if (*g.abort) {
            // let every copy still in flight land before the CTA exits
            volatile int never = 0;
            const Guard g2{a.status, &never, kWaitLimitNs};
            for (uint32_t i = n > (uint32_t)ST ? n - ST : is_v; i < n; i += 2)
                mbar_wait_warp<kIn>(bar(ms.full[i % ST]), (i / ST) & 1, g2, SITE_DEC_DRAIN);
        }
    } else if (NB == 1 && warp == kMmaWarp) {
        // -------------------------------------- issuer of S = Q K^T, queries and trees
        uint32_t seg = 0, unit = 0, sent = 0;
        bool ok = true;
        Slot k_slot{0, 0};
        Segment sa{};  // one ahead, whose queries come while there is room for them
        bool more = walk.next(a, &sa);
        auto put_next = [&]() {
            if (!ok || !more) return;
            ok = put_queries(sa, sent);
            sent += ok;
        };
        put_next();
        for (; ok && more; ++seg) {
            s = sa;
            more = walk.next(a, &sa);
            const int qb = (int)(seg % QBUF);
            if (QBUF == 2) put_next();
            // the first one while the first copies are under way, later ones behind the first S
            if (seg == 0) ok = ok && put_tree(s, 0);
            ok = ok && mbar_wait_warp<kIn>(bar(ms.q_full[qb]), (seg / QBUF) & 1, g, SITE_DEC_MMA);
#pragma unroll 1
            for (int t = s.t0; ok && t < s.t1; ++t, ++unit) {
                ok = mbar_wait_warp<kIn>(bar(ms.full[k_slot.at]), k_slot.round, g, SITE_DEC_FULL);
                // the slot of S is free behind the product with V of the tile before the last
                if (ok && unit >= 2)
                    ok = mbar_wait_warp<kIn>(bar(ms.pv_done[0][unit & 1]), ((unit - 2) >> 1) & 1, g, SITE_DEC_MMA);
                if (!ok) break;
                product_s(qb, 0, unit & 1, k_slot.at);
                tc_commit_elect(bar(ms.s_full[0][unit & 1]));
                tc_commit_elect(bar(ms.empty[k_slot.at]));
                k_slot.advance();
                if (t == s.t0 && seg > 0) ok = put_tree(s, seg);
            }
            tc_commit_elect(bar(ms.q_empty[qb]));
            if (QBUF == 1) put_next();
        }
        drain_queries(sent);
        drain(bar(ms.done[0]));
    } else if (NB == 1 && warp == kMmaWarp2) {
        // ------------------------------------------------------------ issuer of O += P V
        check_lengths();
        uint32_t unit = 0;
        bool ok = true;
        Slot v_slot{1, 0};
        while (ok && walk.next(a, &s)) {
#pragma unroll 1
            for (int t = s.t0; ok && t < s.t1; ++t, ++unit) {
                ok = mbar_wait_warp<kIn>(bar(ms.p_full[0][unit & 1]), (unit >> 1) & 1, g, SITE_DEC_MMA) &&
                     mbar_wait_warp<kIn>(bar(ms.full[v_slot.at]), v_slot.round, g, SITE_DEC_FULL);
                if (!ok) break;
                product_o(0, unit & 1, t == s.t0, v_slot.at);
                tc_commit_elect(bar(ms.pv_done[0][unit & 1]));
                tc_commit_elect(bar(ms.empty[v_slot.at]));
                v_slot.advance();
            }
        }
        drain(bar(ms.done[1]));
    } else if (NB == 2 && warp == kMmaWarp) {
        // ------------------------------------------------------------ issuer of all products
        if constexpr (T::TRADE) setmaxnreg_dec<T::REG_OTHERS>();
        check_lengths();
        // A fixed order: a block's P V, S of its next tile, then the same of the other block.
        uint32_t m0 = 0, m1 = 0;  // tiles of each block
        bool ok = true;
        Slot k_slot{0, 0}, v_slot{1, 0};
        auto here = [&](const Slot &slot) {
            return mbar_wait_warp<kIn>(bar(ms.full[slot.at]), slot.round, g, SITE_DEC_FULL);
        };
        auto have_half = [&](int blk, uint32_t m) {
            return mbar_wait_warp<kIn>(bar(ms.p_half[blk][m & 1]), (m >> 1) & 1, g, SITE_DEC_MMA);
        };
        auto have_p = [&](int blk, uint32_t m) {
            return mbar_wait_warp<kIn>(bar(ms.p_full[blk][m & 1]), (m >> 1) & 1, g, SITE_DEC_MMA);
        };
        for (uint32_t seg = 0; ok && walk.next(a, &s); ++seg) {
            const int qb = (int)(seg % QBUF);
            ok = mbar_wait_warp<kIn>(bar(ms.q_full[qb]), (seg / QBUF) & 1, g, SITE_DEC_MMA) && here(k_slot);
            if (!ok) break;
            if (blocks_of(s) == 2) {  // a slot of S for each
                product_s(qb, 0, 0, k_slot.at);
                tc_commit_elect(bar(ms.s_full[0][m0 & 1]));
                product_s(qb, 1, 1, k_slot.at);
                tc_commit_elect(bar(ms.s_full[NB - 1][m1 & 1]));
                tc_commit_elect(bar(ms.empty[k_slot.at]));
                k_slot.advance();
#pragma unroll 1
                for (int t = s.t0; t < s.t1; ++t, ++m0, ++m1) {
                    const bool next = t + 1 < s.t1;
                    ok = have_half(0, m0) && here(v_slot);
                    if (!ok) break;
                    product_o(0, 0, t == s.t0, v_slot.at, 0, BK / 32);
                    ok = have_p(0, m0);
                    if (!ok) break;
                    product_o(0, 0, false, v_slot.at, BK / 32, BK / 16);
                    tc_commit_elect(bar(ms.pv_done[0][m0 & 1]));
                    if (next) {
                        ok = here(k_slot);
                        if (!ok) break;
                        product_s(qb, 0, 0, k_slot.at);
                        tc_commit_elect(bar(ms.s_full[0][(m0 + 1) & 1]));
                    }
                    ok = have_half(NB - 1, m1);
                    if (!ok) break;
                    product_o(1, 1, t == s.t0, v_slot.at, 0, BK / 32);
                    ok = have_p(NB - 1, m1);
                    if (!ok) break;
                    product_o(1, 1, false, v_slot.at, BK / 32, BK / 16);
                    tc_commit_elect(bar(ms.pv_done[NB - 1][m1 & 1]));
                    if (next) {
                        product_s(qb, 1, 1, k_slot.at);
                        tc_commit_elect(bar(ms.s_full[NB - 1][(m1 + 1) & 1]));
                        tc_commit_elect(bar(ms.empty[k_slot.at]));
                        k_slot.advance();
                    }
                    tc_commit_elect(bar(ms.empty[v_slot.at]));
                    v_slot.advance();
                }
            } else {  // both slots in turn, S a tile ahead
                int ts = s.t0;
#pragma unroll 1
                for (int t = s.t0; t < s.t1; ++t, ++m0) {
#pragma unroll 1
                    for (; ts < s.t1 && ts < t + 2; ++ts) {
                        ok = here(k_slot);
                        if (!ok) break;
                        product_s(qb, 0, (ts - s.t0) & 1, k_slot.at);
                        tc_commit_elect(bar(ms.s_full[0][(m0 + (uint32_t)(ts - t)) & 1]));
                        tc_commit_elect(bar(ms.empty[k_slot.at]));
                        k_slot.advance();
                    }
                    ok = ok && have_p(0, m0) && here(v_slot);
                    if (!ok) break;
                    product_o(0, (t - s.t0) & 1, t == s.t0, v_slot.at);
                    tc_commit_elect(bar(ms.pv_done[0][m0 & 1]));
                    tc_commit_elect(bar(ms.empty[v_slot.at]));
                    v_slot.advance();
                }
            }
            tc_commit_elect(bar(ms.q_empty[qb]));
        }
        drain(bar(ms.done[0]));
    } else if (NB == 2 && warp == kMmaWarp2) {
        // ------------------------------------------------------------ queries and trees
        if constexpr (T::TRADE) setmaxnreg_dec<T::REG_OTHERS>();
        uint32_t sent = 0;
        bool ok = true;
        for (uint32_t seg = 0; ok && walk.next(a, &s); ++seg) {
            if (QBUF == 2 || seg == 0) {
                ok = put_queries(s, seg);
                sent += ok;
            }
            ok = ok && put_tree(s, seg);
            if (ok && QBUF == 1 && seg > 0) {
                ok = put_queries(s, seg);
                sent += ok;
            }
        }
        drain_queries(sent);
    } else {
        // ------------------------------------------------------------ softmax, results
        if constexpr (T::TRADE) setmaxnreg_inc<T::REG_SOFTMAX>();
        // Every warp runs every step even after a wait has given up (waits then return soon).
        const int wg = NH == 1 ? warp >> 2 : 0, h = NH == 1 ? 0 : warp >> 2, w4 = warp & 3;  // block of rows, half of the keys
        const int kk = threadIdx.x & 127;  // row of the block; lane of S and O; key of a tile's V
        const int pair = 1 + w4;           // barrier of the two warps that share 32 rows
        const int turn = h * 128 + kk;     // this thread's place in what they tell each other
        const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
        const uint32_t t_o = tmem + lane_base + T::TM_O + wg * T::DP;
        const float c_s = a.scale_log2;
        uint32_t seg = 0, m = 0, tiles = 0;  // this block's tiles; the CTA's
        while (walk.next(a, &s)) {
            const int ib = seg & 1, len = a.seq_lens[s.b], nb = blocks_of(s);
            const int r0 = s.rb * a.item_rows + wg * 128, rows = min(128, rows_of(s) - wg * 128);  // may be none
            const bool mine = w4 * 32 < rows;                                   // this warp has rows
            const int node = a.Nt - a.Nq + (r0 + kk) % a.Nq;                    // this thread's row
            const int full_tiles = len >> (D == 256 ? 6 : 7);
            bool informed = false;
            auto inform = [&]() {
                if (!informed) mbar_wait_warp<kIn>(bar(ms.info_full[ib]), (seg >> 1) & 1, g, SITE_DEC_MMA);
                informed = true;
            };
            // word k of the bits of nodes that node j sees; the cached keys stand before them
            auto sees = [&](int j, int k) -> uint32_t {
                if (k < 0) return 0xffffffffu;
                if (k >= kNodeWords) return 0u;
                if (a.parents) return ms.sees[ib][j][k];
                const int n = j + 1 - 32 * k;
                return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
            };
            auto is_node = [&](int j) { return j < a.Nt && (!a.parents || (ms.sees[ib][j][j >> 5] >> (j & 31) & 1u)); };
            float m_ref = kUnseen, l = 0.f;
            if (rows > 0) {
#pragma unroll 1
                for (int t = s.t0; t < s.t1; ++t, ++m) {
                    const bool partly = t >= full_tiles;
                    if (partly) inform();
                    mbar_wait_warp<kIn>(bar(ms.s_full[wg][m & 1]), (m >> 1) & 1, g, SITE_DEC_MMA);
                    tc_fence_after();
                    if (mine) {
                        const uint32_t at = NB == 1 ? m & 1 : nb == 2 ? wg : (t - s.t0) & 1;  // slot of S
                        const uint32_t t_s = tmem + lane_base + at * BK + h * CB;
                        uint32_t sr[CB / 32][32];
#pragma unroll
                        for (int c = 0; c < CB / 32; ++c) {
                            tmem_ld32(t_s + c * 32, sr[c]);
                        }
#pragma unroll
                        for (int c = 0; c < CB / 32; ++c) tmem_wait_ld(sr[c]);
                        float x[CB];
#pragma unroll
                        for (int c = 0; c < CB / 32; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[c * 32 + e] = __uint_as_float(sr[c][e]);
                        if (partly) {
                            const int n0 = t * BK + h * CB - len;  // node of the first key, or below 0
#pragma unroll
                            for (int c = 0; c < CB / 32; ++c) {
                                const int at = (n0 + 32 * c) >> 5, sh = (n0 + 32 * c) & 31;
                                const uint32_t w = __funnelshift_r(sees(node, at), sees(node, at + 1), sh);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(w >> e & 1u)) x[c * 32 + e] = -INFINITY;
                            }
                        }
                        float mp0 = -INFINITY, mp1 = -INFINITY;
#pragma unroll
                        for (int c = 0; c < CB; c += 4) {
                            mp0 = fmax3(mp0, x[c], x[c + 1]);
                            mp1 = fmax3(mp1, x[c + 2], x[c + 3]);
                        }
                        float top = fmaxf(mp0, mp1);
                        if constexpr (NH == 2) {  // of both halves, which then take the same steps
                            ms.trade[m & 1][turn] = top;
                            named_barrier_sync(pair, 64);
                            top = fmaxf(top, ms.trade[m & 1][turn ^ 128]);
                        }
                        top *= c_s;
                        float alpha = 1.f;
                        const bool move = top > m_ref + kMoveLog2;
                        if (move) {
                            alpha = ex2(m_ref - top);
                            m_ref = top;
                        }
                        auto rescale = [&]() {
                            if (t > s.t0 && __any_sync(kFull, move)) {
                                // O <- alpha O once the product before is complete
                                mbar_wait_warp<kIn>(bar(ms.pv_done[wg][(m - 1) & 1]), ((m - 1) >> 1) & 1, g, SITE_DEC_MMA);
                                tc_fence_after();
                                const uint64_t a2 = f32x2_splat(alpha);
    #pragma unroll 1
                                for (int c = h; c < D / 32; c += NH) {
                                    uint32_t o[32];
                                    tmem_ld32(t_o + c * 32, o);
                                    tmem_wait_ld(o);
    #pragma unroll
                                    for (int e = 0; e < 32; e += 2) {
                                        float x0 = __uint_as_float(o[e]), x1 = __uint_as_float(o[e + 1]);
                                        mul_f32x2(x0, x1, a2);
                                        o[e] = __float_as_uint(x0);
                                        o[e + 1] = __float_as_uint(x1);
                                    }
                                    tmem_st32(t_o + c * 32, o);
                                }
                            }
                        };
                        if constexpr (NB == 2) rescale();
                        float sp0 = 0.f, sp1 = 0.f;
                        const uint64_t c2 = f32x2_splat(c_s), nm2 = f32x2_splat(-m_ref);
                        auto exponentials = [&](int from, int to) {
#pragma unroll
                            for (int c = from; c < to; c += 2) {
                                fma_f32x2(x[c], x[c + 1], c2, nm2);
                                x[c] = ex2(x[c]);
                                x[c + 1] = ex2(x[c + 1]);
                                add_f32x2(sp0, sp1, x[c], x[c + 1]);
                            }
                        };
                        auto put_p = [&](int c) {  // as bf16 pairs over the first half of the thread's own columns
                            uint32_t pk[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) pk[e] = pack_bf16(x[64 * c + 2 * e], x[64 * c + 2 * e + 1]);
                            tmem_st32(t_s + c * 32, pk);
                        };
                        if constexpr (NB == 2) {
                            // the product with V begins on the first half of the keys while the second's
                            // exponentials are taken
                            exponentials(0, CB / 2);
                            put_p(0);
                            tmem_wait_st();
                            if (!partly) {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(bar(ms.p_half[wg][m & 1]));
                            }
                            exponentials(CB / 2, CB);
                            put_p(1);
                        } else {
                            exponentials(0, CB);
                        }
                        l = l * alpha + (sp0 + sp1);
                        if constexpr (CB == 64) {
                            put_p(0);
                        } else if constexpr (CB == 32) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) pk[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
                            tmem_st16(t_s, pk);
                        }
                        if constexpr (NB == 1) rescale();
                        tmem_wait_st();
                    }
                    if (wg == 0 && partly && kk < BK) {
                        // P is 0 where a row does not see the key, but 0 times an infinity or NaN of
                        // V would not be: rows of V that hold no token, whatever lies there, become 0;
                        // so do such values of nodes, which their rows get back at the end
                        const uint32_t i = 2 * (tiles + (uint32_t)(t - s.t0)) + 1;
                        const int slot = (int)(i % ST), key = t * BK + kk;
                        mbar_wait<kIn>(bar(ms.full[slot]), (i / ST) & 1, g, SITE_DEC_FULL);
                        uint8_t *v0 = gbase + slot * T::SLOT + kk * 128;
                        if (key >= len) {
                            const bool keep = is_node(key - len);
                            bool found = false;
#pragma unroll 1
                            for (int e = h * NCH * 8 / NH; e < (h + 1) * NCH * 8 / NH; ++e) {
                                uint4 *p = reinterpret_cast<uint4 *>(v0 + (e >> 3) * T::SPAN + (e & 7) * 16);
                                uint4 w = keep ? *p : make_uint4(0u, 0u, 0u, 0u);
                                const uint4 f = make_uint4(not_finite(w.x), not_finite(w.y), not_finite(w.z),
                                                           not_finite(w.w));
                                const bool here = (f.x | f.y | f.z | f.w) != 0u;
                                found |= here;
                                if (here || !keep) *p = make_uint4(w.x & ~f.x, w.y & ~f.y, w.z & ~f.z, w.w & ~f.w);
                            }
                            if (found) {
                                atomicOr(&ms.special[ib][(key - len) >> 5], 1u << ((key - len) & 31));
                                ms.special_any[ib] = 1;
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    tc_fence_before();
                    if (NB == 2 && lane == 0 && (partly || !mine)) mbar_arrive(bar(ms.p_half[wg][m & 1]));
                    if (lane == 0) mbar_arrive(bar(ms.p_full[wg][m & 1]));
                }
            }
            // ---- the segment's rows
            inform();
            if (rows > 0) mbar_wait_warp<kIn>(bar(ms.pv_done[wg][(m - 1) & 1]), ((m - 1) >> 1) & 1, g, SITE_DEC_MMA);
            tc_fence_after();
            const bool bad_page = *(volatile int *)&ms.bad_page[ib] != 0;
            const bool bad_tree = *(volatile int *)&ms.bad_tree[ib] != 0, bad = bad_page || bad_tree;
            if (bad && threadIdx.x == 0) {
                atomicCAS(a.status + 1, 0, bad_page ? SITE_TREE_BAD_PAGE : SITE_TREE_BAD_PARENT);
                atomicExch(a.status, FA_ERR_BAD_INDEX);
            }
            if (NH == 2 && mine) {  // the row's sum, of both halves
                ms.trade[m & 1][turn] = l;
                named_barrier_sync(pair, 64);
                l += ms.trade[m & 1][turn ^ 128];
                named_barrier_sync(pair, 64);  // both have read
            }
            if (mine && *g.abort == 0) {
                const bool whole = s.t0 == 0 && s.t1 == s.nt;
                if (!bad && !is_node(node)) l = 0.f;  // a place without a node
                const bool none = l == 0.f;
                const float inv = none ? 0.f : 1.f / l;
                const float l2 = none ? -INFINITY : m_ref + lg2(l);  // base 2
                const long long row = ((long long)s.b * a.Hkv + s.kvh) * a.R + r0 + kk;
                const size_t prow = ((size_t)blockIdx.x * 2 + (s.t0 == 0 ? 1 : 0)) * a.item_rows + wg * 128 + kk;
                const bool put = kk < rows && !bad;
                // (also into a part whose keys all have a score of -infinity: it weighs nothing, they stay)
                const bool special = *(volatile int *)&ms.special_any[ib] != 0 && !bad;
                const int *bt = a.block_table + (size_t)s.b * a.max_pages;
                __nv_bfloat16 *out = a.o + (size_t)row * D;
                float *part = a.part_o + prow * D;
                // (code that runs once per item is kept small: fetching it costs more than running it)
#pragma unroll 1
                for (int c = 32 * h; c < D; c += 32 * NH) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld32(t_o + c, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = none ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);
                    if (put && !whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) store32(part + c + e, o + e);
                    }
                    if (put && whole) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = pack_bf16(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                        if (a.o_aligned) {
                            store32(out + c, o);
                            store32(out + c + 16, o + 8);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<uint4 *>(out + c + 2 * e) =
                                    make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        }
                    }
                }
                if (special && put) {  // infinities and NaN of nodes' values that the row sees
                    for (int j = 0; j < a.Nt; ++j) {
                        if (!(ms.special[ib][j >> 5] & sees(node, j >> 5) & 1u << (j & 31))) continue;
                        const uint32_t key = (uint32_t)(len + j), i = a.by_page.div(key);
                        const __nv_bfloat16 *v =
                            a.v_cache + (((size_t)bt[i] * a.Hkv + s.kvh) * a.page_size + (key - i * a.page_size)) * D;
#pragma unroll 1
                        for (int c = 32 * h; c < D; c = c % 32 == 31 ? c + 32 * NH - 31 : c + 1) {
                            const float f = __bfloat162float(v[c]);
                            if (fabsf(f) < INFINITY) continue;
                            if (whole) out[c] = __float2bfloat16(__bfloat162float(out[c]) + f);
                            else part[c] += f;
                        }
                    }
                }
                if (kk < rows && h == 0) {
                    if (!whole) a.part_l[prow] = bad ? __uint_as_float(kBadPartial) : l2;
                    else if (!bad) a.lse[row] = l2 * kLn2;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(ms.info_empty[ib]));
            tiles += (uint32_t)(s.t1 - s.t0);
            ++seg;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, T::TM_COLS);
    }
}

// The items that were cut: L = log2 sum 2^(L_s), O = sum 2^(L_s - L) O_s.  Every cut lies where one of
// the attention kernel's CTAs begins, and each cut of an item takes its share of the item's rows, so
// an item of many parts has many CTAs to merge it.  A thread has four columns of a row, four parts
// in flight.
constexpr int kMergeThreads = 256, kMergeWorkers = 16;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) fa_tree_merge_kernel(const __grid_constant__ TreeArgs a) {
    constexpr int PER = D / 4, ROWS = kMergeThreads / PER, U = 4;
    const int at = threadIdx.x / PER, col = (threadIdx.x - at * PER) * 4;
    griddep_wait();
    griddep_launch_dependents();
    const int4 item = a.cuts[blockIdx.x];
    if (item.w == 0 || at >= ROWS) return;
    const int n = item.w, c0 = item.z;
    const int kvh = item.y / a.row_blocks, rb = item.y - kvh * a.row_blocks;
    const int worker = ((int)blockIdx.x - c0 - 1) * kMergeWorkers + blockIdx.y;
    const int rows = min(a.item_rows, a.R - rb * a.item_rows);
    const long long row0 = ((long long)item.x * a.Hkv + kvh) * a.R + (long long)rb * a.item_rows;
    for (int r = worker * ROWS + at; r < rows; r += (n - 1) * kMergeWorkers * ROWS) {
        float m = kUnseen, sum = 0.f, acc[4] = {};
        bool bad = false;
        for (int k0 = 0; k0 < n; k0 += U) {
            float w[U];
            float4 x[U];
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const int k = k0 + v;
                const size_t pr = ((size_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * a.item_rows + r;
                w[v] = k < n ? __ldcg(a.part_l + pr) : -INFINITY;
                x[v] = k < n ? __ldcg(reinterpret_cast<const float4 *>(a.part_o + pr * D + col))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float top = m;
#pragma unroll
            for (int v = 0; v < U; ++v) {
                bad = bad || __float_as_uint(w[v]) == kBadPartial;
                top = fmaxf(top, w[v]);
            }
            const float f = ex2(m - top);
            m = top;
            sum *= f;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] *= f;
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const float p = ex2(w[v] - top);
                sum += p;
                acc[0] = fmaf(p, x[v].x, acc[0]);
                acc[1] = fmaf(p, x[v].y, acc[1]);
                acc[2] = fmaf(p, x[v].z, acc[2]);
                acc[3] = fmaf(p, x[v].w, acc[3]);
            }
        }
        if (bad) continue;  // the sequence was rejected: nothing is written
        const float inv = sum == 0.f ? 0.f : reciprocal(sum);
        *reinterpret_cast<uint2 *>(a.o + (row0 + r) * D + col) =
            make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
        const float any = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        if (any != any && sum == sum)
            put_infinities<0, D, 4, 1>(a, ((size_t)c0 * 2 + 1) * a.item_rows + r, (size_t)c0 * 2 * a.item_rows + r, n,
                                       col, a.o + (row0 + r) * D + col);
        if (col == 0) a.lse[row0 + r] = sum == 0.f ? -INFINITY : (m + lg2(sum)) * kLn2;
    }
}

// Tiles of all items at the longest possible lengths.
template <int D, int NB>
long long tree_tiles(const TreeParams &p) {
    using T = TreeTile<D, NB>;
    const long long R = (long long)(p.H / p.Hkv) * p.Nq;
    const long long nt = ((long long)p.page_size * p.max_pages + p.Nt + T::BK - 1) / T::BK;
    const long long items = (long long)p.B * p.Hkv * ((R + T::RB - 1) / T::RB);
    return items >= (1LL << 31) ? items : items * nt;
}

// CTAs of a launch: one per SM, or the largest number of tiles there can be.
template <int D, int NB>
int tree_ctas(const TreeParams &p) {
    const long long n = tree_tiles<D, NB>(p);
    return n < p.num_sms ? (int)n : p.num_sms;
}

template <int D, int NB>
size_t tree_bytes(const TreeParams &p, size_t *l_offset) {
    const size_t ctas = tree_ctas<D, NB>(p), rows = ctas * 2 * TreeTile<D, NB>::RB;
    *l_offset = rows * D * sizeof(float);
    return *l_offset + rows * sizeof(float) + ctas * sizeof(int4) + 16;  // and room to begin on 32 bytes
}

template <int D, int NB>
int launch_t(const TreeParams &p, cudaStream_t stream) {
    using T = TreeTile<D, NB>;
    TreeArgs a{};
    a.tm_q = p.tm_q;
    a.tm_k = p.tm_k;
    a.tm_v = p.tm_v;
    a.v_cache = static_cast<const __nv_bfloat16 *>(p.v_cache);
    a.block_table = p.block_table;
    a.seq_lens = p.seq_lens;
    a.parents = p.parents;
    a.o = static_cast<__nv_bfloat16 *>(p.o);
    a.lse = p.lse;
    size_t l_offset;
    tree_bytes<D, NB>(p, &l_offset);
    char *const ws = static_cast<char *>(p.workspace) + (reinterpret_cast<uintptr_t>(p.workspace) % 32);
    a.part_o = reinterpret_cast<float *>(ws);
    a.part_l = reinterpret_cast<float *>(ws + l_offset);
    a.cuts = reinterpret_cast<int4 *>(a.part_l + (size_t)tree_ctas<D, NB>(p) * 2 * T::RB);
    a.by_page = fast_div((uint32_t)p.page_size);
    a.B = p.B;
    a.H = p.H;
    a.Hkv = p.Hkv;
    a.Nq = p.Nq;
    a.Nt = p.Nt;
    a.d = p.d;
    a.page_size = p.page_size;
    a.max_pages = p.max_pages;
    a.num_pages = p.num_pages;
    a.R = p.H / p.Hkv * p.Nq;
    a.row_blocks = (a.R + T::RB - 1) / T::RB;
    // items of one block share the rows evenly, so that none of a key/value head's is left for last (d256,
    // pages of 48: B2 Hkv2 R = 144 of 233..700 keys 16.8 -> 15.1 us, B5 Hkv2 R = 136 of up to 2900 keys 22.2
    // -> 21.5, R = 168 no difference); of two blocks, the fewest blocks in all are best
    a.item_rows = NB == 1 ? (a.R + a.row_blocks - 1) / a.row_blocks : T::RB;
    a.box = tree_box_rows(p);
    a.box_q = tree_query_box(p);
    a.tile_log2 = T::BK == 64 ? 6 : 7;
    // an item's start costs as much as two tiles (B32 Hkv8 R = 128 of 1..8192 keys, with 1, 2, 3: 107, 101.7,
    // 102 us; one sequence of 131072 keys 108, 110, 109)
    a.start = 2;
    a.o_aligned = reinterpret_cast<uintptr_t>(p.o) % 32 == 0;
    a.scale_log2 = p.scale_log2;
    a.status = p.status;
    a.limit_ns = kWaitLimitNs;
    auto kern = fa_tree_kernel<D, NB>;
    constexpr int kSmem = (int)T::SMEM;
    if (ensure_smem_attr(reinterpret_cast<const void *>(kern), kSmem) != FA_OK) return FA_ERR_CUDA;
    const int n_cta = tree_ctas<D, NB>(p);
    if (launch_dependent(kern, dim3((unsigned)n_cta), T::THREADS, kSmem, stream, 1, a) != FA_OK) return FA_ERR_CUDA;
    // Few rows: a CTA for each, which looks for its parts while the attention kernel still runs; many: the
    // listed cuts only (a CTA per row against the list: 512 rows of one sequence 10.0 and 11.0 us, of four
    // 11.5 and 16.3, 1024 rows of one sequence 19.8 and 22.2, 2048 rows of sixteen 30.9 and 28.1, 32768 rows
    // 167 and 101).
    const long long rows = (long long)p.B * p.H * p.Nq;
    if (rows <= 8LL * p.num_sms)
        return launch_dependent(fa_merge_row_kernel<(D + 31) / 32, 0, TreeArgs>, dim3((unsigned)rows),
                                32 * kRowWarps, 0, stream, 1, a, n_cta);
    return launch_dependent(fa_tree_merge_kernel<D>, dim3((unsigned)n_cta, kMergeWorkers), kMergeThreads, 0,
                            stream, 1, a);
}

// Calls f with the tile that serves the call: head dimension and blocks of 128 query rows (two against
// one, which copies the keys again for each block: B1 R = 256 of 131072 keys 111 and 171 us, B16 R = 384
// of 16384..32768 keys 528 and 677).
template <typename F>
auto with_tile(const TreeParams &p, F f) {
    using std::integral_constant;
    const bool two = (long long)(p.H / p.Hkv) * p.Nq > 128;
    using One = integral_constant<int, 1>;
    using Two = integral_constant<int, 2>;
    switch (p.d) {
        case 64: return two ? f(integral_constant<int, 64>(), Two()) : f(integral_constant<int, 64>(), One());
        case 96: return two ? f(integral_constant<int, 96>(), Two()) : f(integral_constant<int, 96>(), One());
        case 128: return two ? f(integral_constant<int, 128>(), Two()) : f(integral_constant<int, 128>(), One());
        default: return f(integral_constant<int, 256>(), One());  // O of a second block has no room
    }
}

}  // namespace

int tree_box_rows(const TreeParams &p) {
    const int most = p.d == 256 ? 64 : 128;
    int box = 1;
    while (box < most && p.page_size % (2 * box) == 0) box *= 2;
    return box;
}

int tree_query_box(const TreeParams &p) {
    const long long R = (long long)(p.H / p.Hkv) * p.Nq;
    return R >= 128 ? 128 : (int)(R + 7) / 8 * 8;
}

long long tree_max_tiles(const TreeParams &p) {
    return with_tile(p, [&](auto d, auto nb) {
        return tree_tiles<decltype(d)::value, decltype(nb)::value>(p);
    });
}

size_t tree_workspace_bytes(const TreeParams &p) {
    return with_tile(p, [&](auto d, auto nb) {
        size_t l_offset;
        return tree_bytes<decltype(d)::value, decltype(nb)::value>(p, &l_offset);
    });
}

int launch_tree(const TreeParams &p, cudaStream_t stream) {
    return with_tile(p, [&](auto d, auto nb) {
        return launch_t<decltype(d)::value, decltype(nb)::value>(p, stream);
    });
}

}  // namespace fa
