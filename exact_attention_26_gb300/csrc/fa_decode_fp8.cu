// Decode attention against a paged e4m3 cache (definition in fa.h), on the tensor cores
// straight from the codes.
//
// A decode step reads every cached byte once, so it is bound by HBM, and an 8-bit cache has
// two elements to work on per byte: widening the codes on CUDA cores (or into shared memory
// for a 16-bit product) costs more than the stream leaves room for.  Here no code is ever
// widened.  Both products run as tcgen05 kind::f8f6f4 with the cache as the M operand, as TMA
// left it in shared memory, and the few query rows as N:
//   S^T (128 keys x rows)  = K (keys x d, K-major)      Q^T
//   O^T (d x rows)        += V^T (V is keys x d: MN-major) P^T
// The other operand is made of e4m3 terms that carry the precision:
//   q, bf16 with 8 significant bits, scaled per row by a power of two into [128, 256), is
//   c1 + c2 / 16: e4m3 keeps 4 significant bits, and the remainder of rounding 8 bits to 4
//   has 4.  The sum is exact down to 2^-14 of the row's largest element and off by at most
//   2^-22 of it below.
//   p, fp32, times its key's value scale, is c1 + c2 / 16 + c3 / 256: relative error 2^-13,
//   and at most 2^-22 of the largest where the terms run into e4m3's smallest step.
// Every term is a column of N of its own; the columns are put together in fp32 after the
// product.  A thread owns one key of S^T, so the key scales, the mask, exp2 and the row sums
// are per-thread work, and the row maximum is needed only when a score passes the row's
// reference by 2^3 (then P would leave e4m3's range): the four softmax warps vote once per
// tile, and only a tile that does pass takes the maximum and rescales O^T.
//
// Work: the tiles of 128 keys of all (sequence, key/value head, block of RB rows), laid end to
// end, are cut evenly over the resident CTAs (a prefix sum over seq_lens on the device, so
// ragged batches balance and a captured launch follows the lengths).  A CTA writes finished
// rows directly and at most two partial results (the item its range begins in, the item it
// ends in), which a second kernel merges by log-sum-exp.
//
// Warps: 0-3 softmax and epilogue, 4 MMA issue and tensor memory, 5 TMA, 6 query terms.
// Per CTA: a ring of 16 KB slots (K_0 V_0 K_1 V_1 ...; 32 KB at d = 256) that runs across
// items, two S slots, two P buffers, two query buffers.
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kTile = 128;             // keys per tile: the M of S^T and the K of O^T
constexpr float kUnseen = -3.0e38f;    // reference of a row that has seen no key yet
constexpr float kMoveLog2 = 3.0f;      // the reference moves when a score passes it by 2^3 ...
constexpr float kOneP = 32.0f;         // ... so that p = 1 enters as 32 and at most 256 < 448
constexpr uint32_t kBadPartial = 0x7fc0bad1u;  // L of a partial result of a rejected sequence
constexpr int kThreads = 224;

// NCH: 128-byte chunks of a row (d <= 128: 1, d = 256: 2).  RB: query rows per CTA.
template <int NCH, int RB>
struct Dec8Tile {
    static constexpr int NS = 2 * RB;                    // columns of S^T: two terms of q
    static constexpr int NP = (3 * RB + 15) / 16 * 16;   // columns of O^T: three terms of p
    static constexpr int CTAS = (NCH == 1 && RB <= 32) ? 2 : 1;  // resident per SM
    static constexpr uint32_t CHUNK = kTile * 128;
    static constexpr uint32_t SLOT = NCH * CHUNK;
    static constexpr uint32_t Q_CHUNK = NS * 128;
    static constexpr uint32_t Q_BYTES = NCH * Q_CHUNK;   // of one of two buffers
    static constexpr uint32_t P_BYTES = NP * 128;        // of one of two buffers
    static constexpr uint32_t FIXED = 2 * Q_BYTES + 2 * P_BYTES;
    static constexpr uint32_t BUDGET = (CTAS == 2 ? 113u : 226u) * 1024u - 1024u - 4096u;
    static constexpr int STAGES = (int)((BUDGET - FIXED) / SLOT) > 10 ? 10 : (int)((BUDGET - FIXED) / SLOT);
    static constexpr uint32_t OFF_Q = STAGES * SLOT;
    static constexpr uint32_t OFF_P = OFF_Q + 2 * Q_BYTES;
    static constexpr uint32_t OFF_MISC = OFF_P + 2 * P_BYTES;
    static constexpr uint32_t TM_O = 2 * NS;             // after two S slots
    static constexpr uint32_t TM_USED = TM_O + NCH * NP;
    static constexpr uint32_t TM_COLS = TM_USED <= 64 ? 64 : TM_USED <= 128 ? 128 : TM_USED <= 256 ? 256 : 512;
    static_assert(STAGES >= 4, "two tiles in the ring");
    static_assert(TM_USED <= 512 && CTAS * TM_COLS <= 512, "tensor memory budget");
    static_assert(Q_CHUNK % 1024 == 0 && P_BYTES % 1024 == 0, "swizzle atoms stay aligned");
};

// Small per-CTA state behind the buffers.
template <int RB, int STAGES>
struct Dec8Misc {
    unsigned long long full[STAGES], empty[STAGES];
    unsigned long long q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2], done;
    uint32_t tmem;
    int abort;
    int bad;                        // the segment met a page out of range
    float vref;                     // power of two that the value scales are taken relative to
    long long g0, g1, g_b;          // this CTA's tiles; tiles before sequence b0
    int b0;
    alignas(16) float row_scale[2][RB];  // per query buffer: score -> base-2 exponent, before the key's scale
    alignas(16) int limit[2][RB];        // keys the row sees
    alignas(16) float mref[RB];          // reference of the row's scores, base 2
    alignas(16) float alpha[RB];         // old reference to new, as a factor
    alignas(16) float part[4][RB];       // per-warp maxima, then sums
    float vpart[4];
};

struct FastDiv {  // n / d for 0 <= n < 2^31
    uint32_t d, mul, shift;
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return d == 1 ? n : __umulhi(n, mul) >> shift;
    }
};

FastDiv fast_div(uint32_t d) {
    FastDiv f{d, 0, 0};
    if (d > 1) {
        uint32_t l = 0;
        while ((1ull << l) < d) ++l;  // ceil(log2 d)
        const uint32_t p = 31 + l;    // mul = ceil(2^p / d) < 2^32
        f.mul = (uint32_t)(((1ull << p) + d - 1) / d);
        f.shift = p - 32;
    }
    return f;
}

struct Dec8Args {
    CUtensorMap tm_k, tm_v;         // bytes (d, page_size, num_pages * Hkv), boxes 128 x box x 1
    const __nv_bfloat16 *q;
    const float *k_scale, *v_scale;
    const int *block_table, *seq_lens;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o, *part_l;         // [CTA][2][RB][d], [CTA][2][RB]
    FastDiv by_page, by_group;
    int B, H, Hkv, Nq, d, page_size, max_pages, num_pages, groups;
    int R, row_blocks;              // query rows per key/value head, blocks of RB of them
    int box;                        // rows per TMA box
    int causal;
    float scale_log2;
    int *status;
    unsigned long long limit_ns;
};

// ---------------------------------------------------------------- small PTX

// Columns [taddr, taddr + 8) or + 16 of the calling warp's 32 lanes.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]),
                   "=f"(r[6]), "=f"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait8(float (&r)[8]) {  // ties the registers to the wait
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]),
                   "+f"(r[6]), "+f"(r[7])
                 :
                 : "memory");
}

// Barrier 1 over the 128 softmax threads that also answers: does any of them say yes?
__device__ __forceinline__ bool vote_softmax(bool yes) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)yes)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void sync_softmax() { named_barrier_sync(1, 128); }

// e4m3 of two values (a in the low byte), and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return make_float2(lo, hi);
}

__device__ __forceinline__ void sts8(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Byte `x` (0..127) of row n of an operand of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(uint32_t base, int n, int x) {
    return base + n * 128 + ((((uint32_t)x >> 4) ^ (n & 7)) << 4) + (x & 15);
}

// ---------------------------------------------------------------- the schedule

__device__ __forceinline__ bool len_ok(const Dec8Args &a, int len) {
    return len >= 0 && (long long)len <= (long long)a.page_size * a.max_pages;
}
// Tiles of one (head, row block) item of sequence b.
__device__ __forceinline__ int tiles_of(const Dec8Args &a, int b) {
    const int len = a.seq_lens[b];
    return len_ok(a, len) ? (int)(((long long)len + kTile - 1) / kTile) : 0;
}

__device__ __forceinline__ long long warp_scan(long long v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// Tiles of all sequences (of one warp's call): total, and those before sequence `upto`.
__device__ __forceinline__ long long count_tiles(const Dec8Args &a, int upto, long long *before) {
    const int lane = threadIdx.x & 31;
    long long all = 0, pre = 0;
    for (int b = lane; b < a.B; b += 32) {
        const long long t = tiles_of(a, b);
        all += t;
        if (b < upto) pre += t;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(kFull, all, o);
        pre += __shfl_xor_sync(kFull, pre, o);
    }
    *before = pre;
    return all;
}

// CTA c of n takes tiles [total * c / n, total * (c + 1) / n), n at most the tiles there are,
// so that every one of the n has some.
__device__ __forceinline__ int busy_ctas(long long total, int n_cta) {
    return (int)(total < n_cta ? total : n_cta);
}
__device__ __forceinline__ long long first_tile(long long total, int c, int n) {
    return c < n ? total * c / n : total;
}
__device__ __forceinline__ int cta_of(long long total, long long g, int n) {
    return (int)(((g + 1) * n - 1) / total);
}

// A run of tiles of one item within this CTA's range.  Every role walks the same segments.
struct Segment {
    int b, kvh, rb;   // sequence, key/value head, row block
    int t0, t1, nt;   // tiles [t0, t1) of the item's nt
};
struct Walk {
    long long left;
    int b, item, t, nt;
    __device__ __forceinline__ bool next(const Dec8Args &a, Segment *s) {
        if (left <= 0) return false;
        while (t >= nt) {  // the next item that has tiles
            t = 0;
            if (++item >= a.Hkv * a.row_blocks || nt == 0) {
                item = 0;
                if (++b >= a.B) return false;  // not reached: `left` ends first
                nt = tiles_of(a, b);
            }
        }
        s->b = b;
        s->kvh = item / a.row_blocks;
        s->rb = item % a.row_blocks;
        s->t0 = t;
        s->t1 = (int)(left < nt - t ? t + left : nt);
        s->nt = nt;
        left -= s->t1 - t;
        t = s->t1;
        return true;
    }
};

// ---------------------------------------------------------------- the kernel

template <int NCH, int RB>
__global__ void __launch_bounds__(kThreads, Dec8Tile<NCH, RB>::CTAS)
    fa_decode8_kernel(const __grid_constant__ Dec8Args a) {
    using T = Dec8Tile<NCH, RB>;
    using Misc = Dec8Misc<RB, T::STAGES>;
    static_assert(sizeof(Misc) <= 4096, "state fits behind the buffers");
    constexpr int ST = T::STAGES;
    griddep_launch_dependents();  // the merge kernel may launch while the tiles run
    extern __shared__ uint8_t dec8_smem[];
    const uint32_t raw = smem_u32(dec8_smem);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = dec8_smem + (base - raw);
    Misc &ms = *reinterpret_cast<Misc *>(gbase + T::OFF_MISC);
    auto bar = [](unsigned long long &b) { return smem_u32(&b); };
    const uint32_t sQ = base + T::OFF_Q, sP = base + T::OFF_P;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(bar(ms.full[s]), 1);
            mbar_init(bar(ms.empty[s]), 1);
        }
        for (int u = 0; u < 2; ++u) {
            mbar_init(bar(ms.q_full[u]), 32);
            mbar_init(bar(ms.q_empty[u]), 2);  // the MMAs that read it, the softmax warps
            mbar_init(bar(ms.s_full[u]), 1);
            mbar_init(bar(ms.p_full[u]), 128);
            mbar_init(bar(ms.pv_done[u]), 1);
        }
        mbar_init(bar(ms.done), 1);
        ms.abort = 0;
        fence_mbar_init();
    }
    if (warp == 4) {
        tmem_alloc(smem_u32(&ms.tmem), T::TM_COLS);
        tmem_relinquish();
    }
    if (warp == 5 && lane == 0) {
        tma_prefetch_desc(&a.tm_k);
        tma_prefetch_desc(&a.tm_v);
    }
    if (warp == 6) {
        // this CTA's range of tiles, and the sequence it begins in
        long long pre;
        const long long ipb = (long long)a.Hkv * a.row_blocks;
        const long long total = count_tiles(a, 0, &pre) * ipb;
        const int n = busy_ctas(total, gridDim.x);
        const long long g0 = first_tile(total, blockIdx.x, n);
        const long long g1 = first_tile(total, blockIdx.x + 1, n);
        long long run = 0;
        for (int b = 0; b < a.B; b += 32) {
            const long long mine = b + lane < a.B ? tiles_of(a, b + lane) * ipb : 0;
            const long long incl = run + warp_scan(mine, lane);
            const unsigned m = __ballot_sync(kFull, incl > g0);
            if (m || b + 32 >= a.B) {
                const int k = m ? __ffs(m) - 1 : 31;
                if (lane == k) {
                    ms.b0 = min(b + lane, a.B - 1);
                    ms.g_b = incl - mine;
                    ms.g0 = g0;
                    ms.g1 = g1;
                }
                break;
            }
            run = __shfl_sync(kFull, incl, 31);
        }
        if (blockIdx.x == 0) {
            bool ok = true;
            for (int b = lane; b < a.B; b += 32) ok = ok && len_ok(a, a.seq_lens[b]);
            if (!__all_sync(kFull, ok) && lane == 0) {
                atomicCAS(a.status + 1, 0, SITE_DEC8_BAD_LEN);
                atomicExch(a.status, FA_ERR_BAD_INDEX);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem;
    const Guard g{a.status, &ms.abort, a.limit_ns};
    Walk walk;
    walk.left = ms.g1 - ms.g0;
    walk.b = ms.b0;
    walk.nt = walk.left > 0 ? tiles_of(a, walk.b) : 0;
    walk.item = walk.left > 0 ? (int)((ms.g0 - ms.g_b) / walk.nt) : 0;
    walk.t = walk.left > 0 ? (int)((ms.g0 - ms.g_b) % walk.nt) : 0;
    Segment s;

    if (warp == 5) {
        // ------------------------------------------------------------ TMA producer
        // The whole warp runs the loop.  A tile is a run of boxes of `box` rows (the largest
        // power of two that divides the page size, so a box never straddles two pages); lane i
        // looks up and copies boxes i, i + 32, ...  Boxes behind the last key are not copied.
        const int per_tile = kTile / a.box;
        uint32_t n = 0;  // ring slots used so far
        bool ok = true;
        while (ok && walk.next(a, &s)) {
            const int len = a.seq_lens[s.b];
            const int *bt = a.block_table + (size_t)s.b * a.max_pages;
            auto look = [&](int t, int (&pg)[4]) {  // pages of this lane's boxes of tile t
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int bx = lane + 32 * i;
                    const long long key = (long long)t * kTile + (long long)bx * a.box;
                    pg[i] = (bx < per_tile && t < s.t1 && key < len)
                                ? __ldg(bt + a.by_page.div((uint32_t)key)) : -1;
                    if (pg[i] >= a.num_pages) pg[i] = -1;
                }
            };
            int pg[4], pg_next[4];
            look(s.t0, pg);
            for (int t = s.t0; ok && t < s.t1; ++t) {
                look(t + 1, pg_next);
                int mine = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) mine += pg[i] >= 0 ? 1 : 0;
                const uint32_t bytes =
                    (uint32_t)__reduce_add_sync(kFull, mine) * (uint32_t)a.box * 128u * NCH;
#pragma unroll
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    const int slot = (int)(n % ST);
                    ok = n < (uint32_t)ST ||
                         mbar_wait_warp(bar(ms.empty[slot]), ((n / ST) - 1) & 1, g, SITE_DEC_EMPTY);
                    if (!ok) break;
                    const uint32_t fb = bar(ms.full[slot]);
                    if (lane == 0) {
                        if (bytes) mbar_arrive_expect_tx(fb, bytes);
                        else mbar_arrive(fb);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (pg[i] < 0) continue;
                        const int row = (lane + 32 * i) * a.box;
                        const uint32_t key = (uint32_t)(t * kTile + row);
                        const int y = (int)(key - a.by_page.div(key) * (uint32_t)a.page_size);
                        const uint32_t dst = base + slot * T::SLOT + row * 128;
#pragma unroll
                        for (int c = 0; c < NCH; ++c)
                            tma_load_3d(dst + c * T::CHUNK, kv ? &a.tm_v : &a.tm_k, fb, c * 128, y,
                                        pg[i] * a.Hkv + s.kvh);
                    }
                    ++n;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) pg[i] = pg_next[i];
            }
        }
        if (*g.abort) {
            // let every copy still in flight land before the CTA exits
            volatile int never = 0;
            const Guard g2{a.status, &never, kWaitLimitNs};
            for (uint32_t i = n > (uint32_t)ST ? n - ST : 0; i < n; ++i)
                mbar_wait_warp(bar(ms.full[i % ST]), (i / ST) & 1, g2, SITE_DEC_DRAIN);
        }
    } else if (warp == 4) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t kIdescS = idesc_e4m3_f32(128, T::NS);
        constexpr uint32_t kIdescO = idesc_e4m3_f32(128, T::NP) | (1u << 15);  // A is MN-major
        const int ksteps = a.d / 32;
        Walk ahead = walk;   // segments of S, up to two tiles ahead of O
        Segment sa;
        bool more = ahead.next(a, &sa);
        int ta = more ? sa.t0 : 0;
        uint32_t js = 0, seg = 0;  // tiles whose S is issued; segments begun
        bool ok = true;
        auto issue_s = [&]() {
            const int u = js & 1, qb = seg & 1;
            const uint32_t i = 2 * js;
            const int slot = (int)(i % ST);
            if (ta == sa.t0) ok = ok && mbar_wait_warp(bar(ms.q_full[qb]), (seg >> 1) & 1, g, SITE_DEC_MMA);
            ok = ok && mbar_wait_warp(bar(ms.full[slot]), (i / ST) & 1, g, SITE_DEC_FULL);
            if (!ok) return;
            tc_fence_after();
            const uint64_t dk = sdesc_sw128(base + slot * T::SLOT, 16, 1024);
            const uint64_t dq = sdesc_sw128(sQ + qb * T::Q_BYTES, 16, 1024);
            for (int ks = 0; ks < ksteps; ++ks)
                mma_ss_elect_f8(tmem + u * T::NS, desc_add(dk, (ks >> 2) * T::CHUNK + (ks & 3) * 32),
                                desc_add(dq, (ks >> 2) * T::Q_CHUNK + (ks & 3) * 32), kIdescS,
                                ks > 0 ? 1u : 0u);
            tc_commit_elect(bar(ms.s_full[u]));
            tc_commit_elect(bar(ms.empty[slot]));
            ++js;
            if (++ta == sa.t1) {
                tc_commit_elect(bar(ms.q_empty[qb]));
                ++seg;
                more = ahead.next(a, &sa);
                ta = more ? sa.t0 : 0;
            }
        };
        if (more) issue_s();
        if (more && ok) issue_s();
        uint32_t j = 0;
        while (ok && walk.next(a, &s)) {
            for (int t = s.t0; ok && t < s.t1; ++t, ++j) {
                const int u = j & 1;
                const uint32_t i = 2 * j + 1;
                const int slot = (int)(i % ST);
                ok = mbar_wait_warp(bar(ms.p_full[u]), (j >> 1) & 1, g, SITE_DEC_MMA) &&
                     mbar_wait_warp(bar(ms.full[slot]), (i / ST) & 1, g, SITE_DEC_FULL);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dv = sdesc_sw128(base + slot * T::SLOT, T::CHUNK, 1024);
                const uint64_t dp = sdesc_sw128(sP + u * T::P_BYTES, 16, 1024);
#pragma unroll
                for (int c = 0; c < NCH; ++c)
#pragma unroll
                    for (int ks = 0; ks < kTile / 32; ++ks)
                        mma_ss_elect_f8(tmem + T::TM_O + c * T::NP, desc_add(dv, c * T::CHUNK + ks * 4096),
                                        desc_add(dp, ks * 32), kIdescO, (t > s.t0 || ks > 0) ? 1u : 0u);
                tc_commit_elect(bar(ms.pv_done[u]));
                tc_commit_elect(bar(ms.empty[slot]));
                if (more) issue_s();
            }
        }
        // fires once every MMA issued above has completed (normal or aborted run)
        tc_commit_elect(bar(ms.done));
        volatile int never = 0;
        const Guard g2{a.status, &never, kWaitLimitNs};
        mbar_wait_warp(bar(ms.done), 0, g2, SITE_DEC_DRAIN);
    } else if (warp == 6) {
        // ------------------------------------------------------------ query terms
        const int E = a.d == 96 ? 4 : a.d / 32;  // elements per lane
        const bool on = lane * E < a.d;
        uint32_t seg = 0;
        bool ok = true;
        while (ok && walk.next(a, &s)) {
            const int qb = seg & 1;
            ok = seg < 2 || mbar_wait_warp(bar(ms.q_empty[qb]), ((seg >> 1) - 1) & 1, g, SITE_DEC_EMPTY);
            if (!ok) break;
            const int len = a.seq_lens[s.b];
            const int r0 = s.rb * RB, rows = min(RB, a.R - r0);
            const long long row0 = ((long long)s.b * a.H + (long long)s.kvh * (a.H / a.Hkv)) * a.Nq + r0;
            const uint32_t sq = sQ + qb * T::Q_BYTES;
#pragma unroll 1
            for (int r8 = 0; r8 < RB; r8 += 8) {
                uint32_t w[8][NCH == 2 ? 4 : 2];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w[e][0] = w[e][1] = 0u;
                    if constexpr (NCH == 2) w[e][2] = w[e][3] = 0u;
                    if (r8 + e < rows && on) {
                        const __nv_bfloat16 *p = a.q + (row0 + r8 + e) * a.d + lane * E;
                        if constexpr (NCH == 2) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(p);
                            w[e][0] = x.x; w[e][1] = x.y; w[e][2] = x.z; w[e][3] = x.w;
                        } else if (E == 4) {
                            const uint2 x = *reinterpret_cast<const uint2 *>(p);
                            w[e][0] = x.x; w[e][1] = x.y;
                        } else {
                            w[e][0] = *reinterpret_cast<const uint32_t *>(p);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = r8 + e;
                    uint32_t am = 0;
#pragma unroll
                    for (int i = 0; i < (NCH == 2 ? 4 : 2); ++i)
                        am = max(am, max(w[e][i] & 0x7fffu, (w[e][i] >> 16) & 0x7fffu));
                    am = __reduce_max_sync(kFull, am);
                    // row scale 2^(e - 7) of the largest magnitude's exponent e; a row with a
                    // NaN or an infinity becomes NaN
                    const uint32_t ex = max((int)(am >> 7) - 7, 1);
                    const float inv = __uint_as_float((254u - ex) << 23);
                    const bool finite = am < 0x7f80u;
#pragma unroll
                    for (int i = 0; i < (NCH == 2 ? 4 : 2); i += 2) {
                        float x[4], y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t u = w[e][i + k / 2];
                            x[k] = __uint_as_float(k % 2 ? (u & 0xffff0000u) : (u << 16)) * inv;
                            if (!finite) x[k] = __uint_as_float(0x7fc00000u);
                        }
                        const uint32_t c1 = pack_e4m3x4(x[0], x[1], x[2], x[3]);
                        const float2 lo = from_e4m3x2(c1 & 0xffffu), hi = from_e4m3x2(c1 >> 16);
                        y[0] = (x[0] - lo.x) * 16.f;
                        y[1] = (x[1] - lo.y) * 16.f;
                        y[2] = (x[2] - hi.x) * 16.f;
                        y[3] = (x[3] - hi.y) * 16.f;
                        const uint32_t c2 = pack_e4m3x4(y[0], y[1], y[2], y[3]);
                        if (on) {
                            const int col = lane * E + 2 * i;  // byte of the row
                            const uint32_t q0 = sq + (col >> 7) * T::Q_CHUNK;
                            const int n1 = (r >> 3) * 16 + (r & 7);
                            const uint32_t a1 = swizzled(q0, n1, col & 127), a2 = swizzled(q0, n1 + 8, col & 127);
                            if (NCH == 1 && E == 2) {
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(a1), "h"((uint16_t)c1) : "memory");
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(a2), "h"((uint16_t)c2) : "memory");
                            } else {
                                asm volatile("st.shared.u32 [%0], %1;" ::"r"(a1), "r"(c1) : "memory");
                                asm volatile("st.shared.u32 [%0], %1;" ::"r"(a2), "r"(c2) : "memory");
                            }
                        }
                    }
                    if (lane == e) {
                        ms.row_scale[qb][r] = __uint_as_float(ex << 23) * a.scale_log2;
                        ms.limit[qb][r] = a.causal && r < rows
                                              ? min(len, len - a.Nq + 1 + (r0 + r) % a.Nq) : len;
                    }
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(bar(ms.q_full[qb]));
            ++seg;
        }
    } else {
        // ------------------------------------------------------------ softmax, epilogue
        // All four warps run every step even after a wait has given up (waits then return at
        // once), so that none is left behind at a barrier.
        const int tid = threadIdx.x;  // key of the tile; lane of O^T (head dimension)
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        uint32_t j = 0, seg = 0;
        float l[RB];
        while (walk.next(a, &s)) {
            const int qb = seg & 1;
            const int len = a.seq_lens[s.b];
            const int r0 = s.rb * RB, rows = min(RB, a.R - r0);
            const int *bt = a.block_table + (size_t)s.b * a.max_pages;
            const int full_keys = a.causal ? len - a.Nq + 1 : len;  // keys that every row sees
            // page of this thread's key of tile t (-1: none, -2: out of range), and its scales
            auto page_of = [&](int t) {
                const long long key = (long long)t * kTile + tid;
                if (t >= s.t1 || key >= len) return -1;
                const int pg = __ldg(bt + a.by_page.div((uint32_t)key));
                return pg >= 0 && pg < a.num_pages ? pg : -2;
            };
            auto scales_of = [&](int t, int pg, float &ks, float &vs) {
                ks = vs = 0.f;
                if (pg < 0) return;
                const uint32_t key = (uint32_t)(t * kTile + tid);
                const uint32_t row = key - a.by_page.div(key) * (uint32_t)a.page_size;
                const size_t at = ((size_t)pg * a.Hkv + s.kvh) * a.groups + a.by_group.div(row);
                ks = __ldg(a.k_scale + at);
                vs = __ldg(a.v_scale + at);
            };
            int pg = page_of(s.t0), pg1 = page_of(s.t0 + 1);
            float ks, vs, ks1, vs1;
            scales_of(s.t0, pg, ks, vs);
            if (tid < RB) ms.mref[tid] = kUnseen;
            if (tid == 0) {
                ms.vref = 0.f;
                ms.bad = 0;
            }
#pragma unroll
            for (int r = 0; r < RB; ++r) l[r] = 0.f;
            mbar_wait_warp(bar(ms.q_full[qb]), (seg >> 1) & 1, g, SITE_DEC_MMA);
            sync_softmax();
            for (int t = s.t0; t < s.t1; ++t, ++j) {
                const int u = j & 1;
                const int key = t * kTile + tid;
                const int pg2 = page_of(t + 2);
                scales_of(t + 1, pg1, ks1, vs1);
                mbar_wait_warp(bar(ms.s_full[u]), (j >> 1) & 1, g, SITE_DEC_MMA);
                tc_fence_after();
                float x[RB];
#pragma unroll
                for (int q = 0; q < RB / 8; ++q) {
                    float c1[8], c2[8];
                    tmem_ld8(tmem + lane_base + u * T::NS + q * 16, c1);
                    tmem_ld8(tmem + lane_base + u * T::NS + q * 16 + 8, c2);
                    tmem_wait8(c1);
                    tmem_wait8(c2);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[q * 8 + e] = fmaf(c2[e], 0.0625f, c1[e]) * (ms.row_scale[qb][q * 8 + e] * ks);
                }
                if ((t + 1) * (long long)kTile > full_keys) {  // some row does not see every key
#pragma unroll
                    for (int r = 0; r < RB; ++r)
                        if (key >= ms.limit[qb][r]) x[r] = -INFINITY;
                }
                bool move = vs > ms.vref || pg == -2;
#pragma unroll
                for (int r = 0; r < RB; ++r) move = move || x[r] > ms.mref[r] + kMoveLog2;
                if (vote_softmax(move)) {
                    // new references: the tile's maximum where it passes the old one by 2^3
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        float m = x[r];
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                        if (lane == (r & 31)) ms.part[warp][r] = m;
                    }
                    float vm = vs;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) vm = fmaxf(vm, __shfl_xor_sync(kFull, vm, o));
                    if (lane == 0) ms.vpart[warp] = vm;
                    if (pg == -2) ms.bad = 1;
                    const float v_old = ms.vref;
                    sync_softmax();
                    vm = fmaxf(fmaxf(ms.vpart[0], ms.vpart[1]), fmaxf(ms.vpart[2], ms.vpart[3]));
                    float v_new = v_old;
                    if (vm > v_old)  // the power of two at or above, and kOneP / v_new stays finite
                        v_new = fmaxf(__uint_as_float((__float_as_uint(vm) + 0x7fffffu) & 0x7f800000u),
                                      0x1p-120f);
                    if (tid < RB) {
                        const float m_old = ms.mref[tid];
                        const float m = fmaxf(fmaxf(ms.part[0][tid], ms.part[1][tid]),
                                              fmaxf(ms.part[2][tid], ms.part[3][tid]));
                        const bool up = m > m_old + kMoveLog2;
                        ms.alpha[tid] = up ? ex2(m_old - m) : 1.f;
                        if (up) ms.mref[tid] = m;
                    }
                    if (tid == 0) ms.vref = v_new;
                    sync_softmax();
#pragma unroll
                    for (int r = 0; r < RB; ++r) l[r] *= ms.alpha[r];
                    if (t > s.t0) {  // O^T to the new references, once PV of the tile before is done
                        const float fv = v_new > 0.f ? v_old / v_new : 1.f;
                        mbar_wait_warp(bar(ms.pv_done[(j - 1) & 1]), ((j - 1) >> 1) & 1, g, SITE_DEC_MMA);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < NCH; ++c)
#pragma unroll 1
                            for (int n = 0; n < 3 * RB / 8; ++n) {
                                float o[8];
                                const uint32_t at = tmem + lane_base + T::TM_O + c * T::NP + n * 8;
                                tmem_ld8(at, o);
                                tmem_wait8(o);
#pragma unroll
                                for (int e = 0; e < 8; ++e) o[e] *= ms.alpha[n / 3 * 8 + e] * fv;
                                tmem_st8(at, o);
                            }
                        tmem_wait_st();
                    }
                }
                if (j >= 2)  // the P buffer's last reader
                    mbar_wait_warp(bar(ms.pv_done[u]), ((j >> 1) - 1) & 1, g, SITE_DEC_MMA);
                const float vref = ms.vref;
                const float fv = vref > 0.f ? vs * (kOneP / vref) : 0.f;
                const uint32_t p0 = sP + u * T::P_BYTES;
#pragma unroll
                for (int r = 0; r < RB; r += 2) {
                    const float pa = ex2(x[r] - ms.mref[r]), pb = ex2(x[r + 1] - ms.mref[r + 1]);
                    l[r] += pa;
                    l[r + 1] += pb;
                    float wa = pa * fv, wb = pb * fv;
                    const int n = (r >> 3) * 24 + (r & 7);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const uint32_t c = to_e4m3x2(wa, wb);
                        sts8(swizzled(p0, n + 8 * k, tid), c & 0xffu);
                        sts8(swizzled(p0, n + 8 * k + 1, tid), c >> 8);
                        if (k < 2) {
                            const float2 f = from_e4m3x2(c);
                            wa = (wa - f.x) * 16.f;
                            wb = (wb - f.y) * 16.f;
                        }
                    }
                }
                if ((t + 1) * (long long)kTile > len) {
                    // rows of V behind the last key: whatever lies there, P is 0 and V must not be NaN
                    const uint32_t i = 2 * j + 1;
                    const int slot = (int)(i % ST);
                    mbar_wait_warp(bar(ms.full[slot]), (i / ST) & 1, g, SITE_DEC_FULL);
                    if (key >= len) {
#pragma unroll
                        for (int c = 0; c < NCH; ++c)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4 *>(gbase + slot * T::SLOT + c * T::CHUNK + tid * 128 +
                                                           e * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(bar(ms.p_full[u]));
                pg = pg1;
                pg1 = pg2;
                ks = ks1;
                vs = vs1;
            }
            // ---- the segment's rows: sums over all keys, then O^T columns
            const uint32_t jl = j - 1;
            mbar_wait_warp(bar(ms.pv_done[jl & 1]), (jl >> 1) & 1, g, SITE_DEC_MMA);
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                float v = l[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
                if (lane == (r & 31)) ms.part[warp][r] = v;
            }
            sync_softmax();
            const bool whole = s.t0 == 0 && s.t1 == s.nt;
            const bool bad = ms.bad != 0;
            const bool dead = *g.abort != 0;
            const size_t prow = ((size_t)blockIdx.x * 2 + (s.t0 == 0 ? 1 : 0)) * RB;
            const long long row0 = ((long long)s.b * a.H + (long long)s.kvh * (a.H / a.Hkv)) * a.Nq + r0;
            const float ov = ms.vref * (1.f / kOneP);
            if (bad && tid == 0) {
                atomicCAS(a.status + 1, 0, SITE_DEC8_BAD_PAGE);
                atomicExch(a.status, FA_ERR_BAD_INDEX);
            }
            if (tid < rows && !dead) {
                const float sum = (ms.part[0][tid] + ms.part[1][tid]) + (ms.part[2][tid] + ms.part[3][tid]);
                const float l2 = sum == 0.f ? -INFINITY : ms.mref[tid] + lg2(sum);  // base 2
                if (!whole) a.part_l[prow + tid] = bad ? __uint_as_float(kBadPartial) : l2;
                else if (!bad) a.lse[row0 + tid] = l2 * kLn2;
            }
#pragma unroll 1
            for (int c = 0; c < NCH; ++c) {
                const int dd = c * 128 + tid;
#pragma unroll 1
                for (int q = 0; q < RB / 8; ++q) {
                    float o0[8], o1[8], o2[8];
                    __syncwarp();
                    const uint32_t at = tmem + lane_base + T::TM_O + c * T::NP + q * 24;
                    tmem_ld8(at, o0);
                    tmem_ld8(at + 8, o1);
                    tmem_ld8(at + 16, o2);
                    tmem_wait8(o0);
                    tmem_wait8(o1);
                    tmem_wait8(o2);
                    if (dd >= a.d || dead || bad) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = q * 8 + e;
                        if (r >= rows) break;
                        const float sum = (ms.part[0][r] + ms.part[1][r]) + (ms.part[2][r] + ms.part[3][r]);
                        const float inv = sum == 0.f ? 0.f : ov / sum;
                        const float o = fmaf(fmaf(o2[e], 0.0625f, o1[e]), 0.0625f, o0[e]) * inv;
                        if (whole) a.o[(row0 + r) * a.d + dd] = __float2bfloat16(o);
                        else a.part_o[(prow + r) * a.d + dd] = o;
                    }
                }
            }
            tc_fence_before();
            sync_softmax();  // the state above is free for the next segment
            if (tid == 0) mbar_arrive(bar(ms.q_empty[qb]));
            ++seg;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, T::TM_COLS);
    }
}

// Merge of the partial results of the items that were cut, one warp per query row:
// L = log2 sum 2^(L_s), O = sum 2^(L_s - L) O_s.  Rows of empty sequences are written here.
template <int NCH, int RB>
__global__ void __launch_bounds__(128)
    fa_decode8_merge_kernel(const __grid_constant__ Dec8Args a, int n_cta, long long n_rows) {
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= n_rows) return;
    const int i = (int)(row % a.Nq);
    const long long bh = row / a.Nq;
    const int b = (int)(bh / a.H), h = (int)(bh % a.H), group = a.H / a.Hkv;
    const int len = a.seq_lens[b];
    const long long ipb = (long long)a.Hkv * a.row_blocks;
    long long before;
    const long long total = count_tiles(a, b, &before) * ipb;
    griddep_wait();  // every partial result is written
    if (!len_ok(a, len)) return;
    __nv_bfloat16 *o = a.o + row * a.d;
    if (len == 0) {
        for (int c = lane; c < a.d; c += 32) o[c] = __float2bfloat16(0.f);
        if (lane == 0) a.lse[row] = -INFINITY;
        return;
    }
    const int r = (h % group) * a.Nq + i, nt = tiles_of(a, b);
    const long long first =
        before * ipb + ((long long)(h / group) * a.row_blocks + r / RB) * nt;
    const int n = busy_ctas(total, n_cta);
    const int c0 = cta_of(total, first, n), c1 = cta_of(total, first + nt - 1, n);
    if (c0 == c1) return;  // written directly
    auto prow = [&](int c) { return ((size_t)c * 2 + (c == c0 ? 1 : 0)) * RB + r % RB; };
    float m = -INFINITY;
    bool bad = false;
    for (int c = c0 + lane; c <= c1; c += 32) {
        const float x = __ldcg(a.part_l + prow(c));
        bad = bad || __float_as_uint(x) == kBadPartial;
        m = fmaxf(m, x);
    }
    if (__any_sync(kFull, bad)) return;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
    if (m == -INFINITY) m = 0.f;  // the row sees no key: every weight is 0
    constexpr int E = NCH == 2 ? 8 : 4;
    float acc[E], wsum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int cb = c0; cb <= c1; cb += 32) {
        const int n = min(32, c1 - cb + 1);
        const float w = lane < n ? ex2(__ldcg(a.part_l + prow(cb + lane)) - m) : 0.f;
        for (int k = 0; k < n; ++k) {
            const float wk = __shfl_sync(kFull, w, k);
            const float *po = a.part_o + prow(cb + k) * a.d;
            wsum += wk;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = lane + 32 * e;
                if (c < a.d) acc[e] = fmaf(wk, __ldcg(po + c), acc[e]);
            }
        }
    }
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (lane + 32 * e < a.d) o[lane + 32 * e] = __float2bfloat16(acc[e] * inv);
    if (lane == 0) a.lse[row] = wsum == 0.f ? -INFINITY : (m + lg2(wsum)) * kLn2;
}

// CTAs of a launch: all that are resident, or the largest number of tiles there can be.
template <int NCH, int RB>
int dec8_ctas(const Decode8Params &p) {
    const long long R = (long long)(p.H / p.Hkv) * p.Nq;
    const long long nt = ((long long)p.page_size * p.max_pages + kTile - 1) / kTile;
    const long long items = (long long)p.B * p.Hkv * ((R + RB - 1) / RB);
    const long long most = (long long)p.num_sms * Dec8Tile<NCH, RB>::CTAS;
    return (int)(items >= most || items * nt >= most ? most : items * nt);
}

template <int NCH, int RB>
size_t dec8_bytes(const Decode8Params &p, size_t *l_offset) {
    const size_t rows = (size_t)dec8_ctas<NCH, RB>(p) * 2 * RB;
    *l_offset = rows * p.d * sizeof(float);  // a multiple of 16
    return *l_offset + rows * sizeof(float);
}

template <int NCH, int RB>
int launch_t(const Decode8Params &p, cudaStream_t stream) {
    using T = Dec8Tile<NCH, RB>;
    Dec8Args a{};
    a.tm_k = p.tm_k;
    a.tm_v = p.tm_v;
    a.q = static_cast<const __nv_bfloat16 *>(p.q);
    a.k_scale = p.k_scale;
    a.v_scale = p.v_scale;
    a.block_table = p.block_table;
    a.seq_lens = p.seq_lens;
    a.o = static_cast<__nv_bfloat16 *>(p.o);
    a.lse = p.lse;
    size_t l_offset;
    dec8_bytes<NCH, RB>(p, &l_offset);
    a.part_o = static_cast<float *>(p.workspace);
    a.part_l = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + l_offset);
    a.by_page = fast_div((uint32_t)p.page_size);
    a.by_group = fast_div((uint32_t)p.group);
    a.B = p.B;
    a.H = p.H;
    a.Hkv = p.Hkv;
    a.Nq = p.Nq;
    a.d = p.d;
    a.page_size = p.page_size;
    a.max_pages = p.max_pages;
    a.num_pages = p.num_pages;
    a.groups = p.page_size / p.group;
    a.R = p.H / p.Hkv * p.Nq;
    a.row_blocks = (a.R + RB - 1) / RB;
    a.box = decode8_box_rows(p.page_size);
    a.causal = p.causal;
    a.scale_log2 = p.scale_log2;
    a.status = p.status;
    a.limit_ns = kWaitLimitNs;
    auto kern = fa_decode8_kernel<NCH, RB>;
    constexpr int kSmem = (int)(T::OFF_MISC + 4096 + 1024);
    if (ensure_smem_attr(reinterpret_cast<const void *>(kern), kSmem) != FA_OK) return FA_ERR_CUDA;
    const int n_cta = dec8_ctas<NCH, RB>(p);
    kern<<<n_cta, kThreads, kSmem, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    // a programmatic dependent: launched as the last CTAs start, it waits for the whole grid
    const long long rows = (long long)p.B * p.H * p.Nq;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fa_decode8_merge_kernel<NCH, RB>, a, n_cta, rows) != cudaSuccess)
        return FA_ERR_CUDA;
    return FA_OK;
}

// Calls f with the tile that serves R query rows per key/value head of dimension d.
template <typename F>
auto with_tile(int d, long long R, F f) {
    if (d == 256) {
        if (R <= 8) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 8>());
        return f(std::integral_constant<int, 2>(), std::integral_constant<int, 32>());
    }
    if (R <= 8) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
    if (R <= 32) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 32>());
    return f(std::integral_constant<int, 1>(), std::integral_constant<int, 64>());
}

}  // namespace

int decode8_box_rows(int page_size) {
    int box = 1;
    while (box < kTile && page_size % (2 * box) == 0) box *= 2;
    return box;
}

size_t decode8_workspace_bytes(const Decode8Params &p) {
    return with_tile(p.d, (long long)(p.H / p.Hkv) * p.Nq, [&](auto nch, auto rb) {
        size_t l_offset;
        return dec8_bytes<decltype(nch)::value, decltype(rb)::value>(p, &l_offset);
    });
}

int launch_decode8(const Decode8Params &p, cudaStream_t stream) {
    return with_tile(p.d, (long long)(p.H / p.Hkv) * p.Nq, [&](auto nch, auto rb) {
        return launch_t<decltype(nch)::value, decltype(rb)::value>(p, stream);
    });
}

}  // namespace fa
