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
//   c1 + c2 / 32: e4m3 keeps 4 significant bits, and the remainder of rounding 8 bits to 4
//   has 4 and is at most 8, so 32 times it is in range.  c2 / 32 has steps of 2^-14: the sum is
//   exact from 2^-7 up, which is 2^-14 of the row's largest element or less, and off by at most
//   2^-15 below, 2^-22 of the largest or less.
//   p, fp32, times its key's value scale, is rounded to f16 and split into three e5m2 terms:
//   e5m2 is f16's upper byte, so the first two are byte selections and the remainders exact
//   subtractions; the third, of 2^5 times what they leave (less than 2^-5 of p), is rounded to
//   nearest.  Relative error at most 2^-9 + 2^-11 (a rounding to bf16 would be off by 2^-8);
//   where the first two run into e5m2's smallest step, 2^-16, they leave up to that, of which the
//   third is off by 2^-20: 2^-24 of the row's largest p times the largest scale it sees (or 2^-84
//   of any).
// Every term is a column of N of its own; the columns are put together in fp32 after the
// product.  A thread owns one key of S^T, so the key scales, the mask, exp2 and the row sums
// are per-thread work, and the row maximum is needed only when a score passes the row's
// reference by 2^6 (then P would leave e5m2's range): the softmax warps vote once per tile,
// and only a tile that does pass takes the maximum and rescales O^T.  A thread's terms of one
// key are contiguous in P (MN-major, like V), so they leave in 16-byte stores.
//
// Work: the tiles of 128 keys of all (sequence, key/value head, block of RB rows), laid end to
// end, are cut evenly over the resident CTAs (a prefix sum over seq_lens on the device, so
// ragged batches balance and a captured launch follows the lengths).  A CTA writes finished
// rows directly and at most two partial results (the item its range begins in, the item it
// ends in), which a second kernel merges by log-sum-exp.
//
// Warps: one or more softmax warpgroups of up to 16 rows each (they also write the results),
// then one each for MMA issue and tensor memory, TMA, key and value scales, and query terms.
// Per CTA: a ring of 16 KB slots (K_0 V_0 K_1 V_1 ...; 32 KB at d = 256) that runs across
// items, two S slots, two P buffers, two query buffers, three tiles of scales.
//
// Measured (GB300, graph replay, caches larger than L2, d = 128 and one query unless stated):
//   B8 H32 Hkv32 32768 keys   320-325 us  6.6-6.7 TB/s   HBM
//   B1 H32 Hkv8 131072 keys    48 us      5.6 TB/s       37 us of stream; the rest is launch,
//                                                        first tile, partials and merge
//   B32 H32 Hkv8 1..8192 keys  49 us      5.6 TB/s       the same, twice an item per CTA
//   B32 H16 Hkv8 30000 d64    166 us      6.0 TB/s       two keys to a row of a tile (pages of 32)
//   B8 H32 Hkv4 Nq4 d64        38 us      2.1 TB/s       32 rows per head: 16 tiles of 1.2 us per
//                                                        CTA; fixed work per step of 128 keys and
//                                                        16 scores a thread, and TMA's half rows
//                                                        (issue slots 53% busy); then as above
//   B1 H32 Hkv8 1000 keys       6.5 us                   latency of two launches
// Alone, the chain of a softmax warp takes 0.7k clocks (8 rows) to 0.9k (16 rows) per tile of 128
// keys, against 1.3k clocks in which its bytes arrive at d = 128 for one of two CTAs on the SM.
// Code that runs once per item is kept small: fetching it cold costs more than running it
// (unrolled copy and scale loops: 54 -> 60 us for the ragged batch).
#include <type_traits>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kTile = 128;             // keys per step: the M of S^T and the K of O^T
constexpr float kUnseen = -3.0e38f;    // reference of a row that has seen no key yet
// e5m2 reaches from 2^-16 to 57344, and p times the value scale is placed in it so that neither
// reference moves often: the rows' references move when a score passes them by 2^6, the value
// scales' (first 8 to 16 times the largest) when a scale passes it, and p = 2^6 at the reference
// scale is 2^15.  The wider the threshold, the fewer tiles rescale.
constexpr float kMoveLog2 = 6.0f;
constexpr float kOneP = 512.0f;        // p = 1 at the reference scale
constexpr uint32_t kBadPartial = 0x7fc0bad1u;  // L of a partial result of a rejected sequence
constexpr int kScaleStages = 3;

// NCH: 128-byte chunks of a row (d <= 128: 1, d = 256: 2).  RB: query rows per CTA.
// PACK: keys per 128-byte row of a tile.  With two (d = 64, even pages) TMA copies rows twice as
// long, half as many; a tile holds 256 keys and is worked on in two steps, of the even keys and
// of the odd ones.  K's halves are chosen by the column that S^T's products begin at; the
// products with V take whole rows, so each step has columns of O^T of its own, of which the
// lanes of its half are O and the others are not read, and the halves meet in the epilogue.
template <int NCH, int RB, int PACK>
struct Dec8Tile {
    static constexpr int RW = RB < 16 ? RB : 16;         // rows of a softmax warpgroup
    static constexpr int NWG = RB / RW;
    static constexpr int NS = 2 * RB;                    // columns of S^T: two terms of q
    static constexpr int NP = (3 * RB + 15) / 16 * 16;   // columns of O^T: three terms of p
    static constexpr int CTAS = (NCH == 1 && RB <= 32) ? 2 : 1;  // resident per SM
    static constexpr int THREADS = 32 * (4 * NWG + 4);
    // A wait that calls a function costs the registers that calls clobber.  Where registers are
    // short, waits are inlined (B8 H32 Hkv4 Nq4 19000 keys d128: 46.5 -> 42.3 us).
    static constexpr bool INLINE_WAITS = NCH == 1 && RB >= 32;
    static constexpr int TK = PACK * kTile;              // keys of a tile
    static constexpr uint32_t CHUNK = kTile * 128;
    static constexpr uint32_t SLOT = NCH * CHUNK;
    static constexpr uint32_t Q_CHUNK = NS * 128;
    static constexpr uint32_t Q_BYTES = NCH * Q_CHUNK;   // of one of two buffers
    static constexpr uint32_t P_CHUNK = kTile * 32;      // 32 columns of every key
    static constexpr uint32_t P_BYTES = (NP + 31) / 32 * P_CHUNK;  // of one of two buffers
    static constexpr uint32_t MISC = RB > 32 ? 9216 : 8192;
    static constexpr uint32_t FIXED = 2 * Q_BYTES + 2 * P_BYTES + MISC + 1024;
    static constexpr uint32_t BUDGET = (CTAS == 2 ? 113u : 226u) * 1024u;
    static constexpr int FIT = (int)((BUDGET - FIXED) / SLOT);
    // five where two CTAs share an SM: that keeps the HBM busy (6: 322 us, 5: 316 us, 4: 327 us
    // for B8 H32 Nk32768 d128) and leaves the merge kernel's CTAs room to start early
    static constexpr int MOST = CTAS == 2 ? 5 : 10;
    static constexpr int STAGES = FIT > MOST ? MOST : FIT;
    static constexpr uint32_t OFF_Q = STAGES * SLOT;
    static constexpr uint32_t OFF_P = OFF_Q + 2 * Q_BYTES;
    static constexpr uint32_t OFF_MISC = OFF_P + 2 * P_BYTES;
    static constexpr uint32_t SMEM = OFF_MISC + MISC + 1024;  // and room to align the start
    static constexpr uint32_t TM_O = 2 * NS;             // after two S slots
    static constexpr uint32_t TM_USED = TM_O + NCH * PACK * NP;
    static constexpr uint32_t TM_COLS = TM_USED <= 64 ? 64 : TM_USED <= 128 ? 128 : TM_USED <= 256 ? 256 : 512;
    static_assert(NCH == 1 || PACK == 1, "only half rows are packed");
    static_assert(PACK == 1 || (NWG == 1 && P_BYTES >= RB * 64 * sizeof(float)),
                  "room for the halves of O to meet in a buffer of P");
    static_assert(STAGES >= 4, "two tiles in the ring");
    static_assert(TM_USED <= 512 && CTAS * TM_COLS <= 512, "tensor memory budget");
    static_assert(Q_CHUNK % 1024 == 0 && P_BYTES % 1024 == 0, "swizzle atoms stay aligned");
};

// Small per-CTA state behind the buffers.
template <int NCH, int RB, int STAGES, int NWG, int TK>
struct Dec8Misc {
    unsigned long long full[STAGES], empty[STAGES];
    unsigned long long q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2], done;
    unsigned long long scale_full[kScaleStages], scale_empty[kScaleStages];
    uint32_t tmem;
    int abort;
    int bad[2];                     // per query buffer: the segment met a page out of range
    alignas(16) float k_scale[kScaleStages][TK];  // of keys 0, 2^run, ... of a tile
    alignas(16) float v_scale[kScaleStages][TK];
    alignas(16) float row_scale[2][RB];  // per query buffer: score -> base-2 exponent, before the key's scale
    alignas(16) int limit[2][RB];        // keys the row sees
    int len[2];                          // per query buffer: the sequence's length
    alignas(16) float nref[RB];          // minus the reference of the row's scores, base 2
    alignas(16) float alpha[RB];         // old reference to new, as a factor
    // causal calls: log2 of what a row's terms of p are divided by, to make room for value scales
    // above the common reference, and the row's factor of O^T when that or the reference moves
    alignas(16) float room[RB], alpha_o[RB];
    alignas(16) float part[4][RB];       // per-warp maxima, then sums
    float vpart[NWG][4];
    // causal calls, per query buffer: columns of O that a NaN code of V makes NaN in a row, where
    // not every row sees its key (elsewhere the product does it), as bits; and whether there are
    // any.  One warpgroup marks them for all, and may be a segment ahead of the others' epilogues,
    // so they are cleared with the buffer's queries, which waits for every warpgroup.
    uint32_t nan_cols[2][RB][NCH * 4];
    int nan_any[2];
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
    CUtensorMap tm_k, tm_v;         // bytes (d, page_size, num_pages * Hkv), boxes 128 x box x 1;
                                    // packed (2 d, page_size / 2, num_pages * Hkv)
    const __nv_bfloat16 *q;
    const float *k_scale, *v_scale;
    const int *block_table, *seq_lens;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o, *part_l;         // [CTA][2][RB][d], [CTA][2][RB]
    FastDiv by_page, by_group;
    int B, H, Hkv, Nq, d, page_size, max_pages, num_pages, groups;
    int R, row_blocks;              // query rows per key/value head, blocks of RB of them
    int box;                        // 128-byte rows per TMA box
    int tile_log2;                  // log2 of the keys per tile
    int start;                      // tiles that an item's start counts as in the cut, up to 3
    int run;                        // log2 of the keys that one entry of the scales stands for
    float scale_log2;
    int *status;
    unsigned long long limit_ns;
};

// ---------------------------------------------------------------- small PTX

// Columns [taddr, taddr + N) of the calling warp's 32 lanes (N = 8, 16 or 32), without waiting.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]),
                   "=f"(r[6]), "=f"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
        "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
          "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
          "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]),
        "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
        : "memory");
}
// Wait for this thread's tcgen05.ld; the registers are tied to the wait.
__device__ __forceinline__ void tmem_wait(float (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]),
                   "+f"(r[6]), "+f"(r[7])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait(float (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]),
                   "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]),
                   "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
                 :
                 : "memory");
}

// Barrier `id` over the 128 threads of a warpgroup that also answers: does any of them say yes?
__device__ __forceinline__ bool vote_group(int id, bool yes) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)yes), "r"(id)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ float warp_max(float x) {  // NaN is passed over
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / x to 2^-23 (x normal), which O's rounding to bf16 hides, without a divide's code.
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 1 / x of a power of two, 2^-126 to 2^126: exponents e and -e.
__device__ __forceinline__ float inverse2(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

// e4m3 of two f16 values (16 bits), and back, exactly.
__device__ __forceinline__ uint32_t e4m3x2_of(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_of(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    return h;
}
// Two floats as f16x2 (a in the low half).
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b), "f"(a));
    return h;
}
// h * 32 and (h - c) * 32 on f16 pairs: exact for the remainder of rounding h to c.
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t times32(uint32_t h) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x50005000u));
    return r;
}
__device__ __forceinline__ uint32_t remainder32(uint32_t h, uint32_t c) { return times32(sub_f16x2(h, c)); }
// e5m2 of two f16 values, to nearest even.
__device__ __forceinline__ uint32_t e5m2x2_of(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}

// The sum over the warp of eight values per lane: every lane gets that of value
// (lane >> 2) & 7, with 9 shuffles: each exchange halves the values a lane keeps.
__device__ __forceinline__ float warp_sum8(const float (&v)[8], int lane) {
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
    float x[4], y[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = (b4 ? v[i + 4] : v[i]) + __shfl_xor_sync(kFull, b4 ? v[i] : v[i + 4], 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        y[i] = (b3 ? x[i + 2] : x[i]) + __shfl_xor_sync(kFull, b3 ? x[i] : x[i + 2], 8);
    float z = (b2 ? y[1] : y[0]) + __shfl_xor_sync(kFull, b2 ? y[0] : y[1], 4);
    z += __shfl_xor_sync(kFull, z, 2);
    z += __shfl_xor_sync(kFull, z, 1);
    return z;
}

// (x0, x1) <- (x0, x1) * (a0, a1) + (c0, c1).
__device__ __forceinline__ void fma_pairs(float &x0, float &x1, float a0, float a1, float c0, float c1) {
    asm("{\n\t.reg .b64 x, a, c;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\t"
        "mov.b64 c, {%4, %5};\n\tfma.rn.f32x2 x, x, a, c;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(a0), "f"(a1), "f"(c0), "f"(c1));
}

// 4-byte asynchronous copy global -> shared, or 4 zero bytes; the thread's earlier ones
// arrive once on `bar` when they are done.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool copy) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(copy ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Has the phase of this parity completed?  Does not wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// MN-major operand with the 32-byte swizzle: rows of 32 bytes (32 columns of one key), 8 rows
// per 256-byte atom (`sbo` between atoms), `lbo` between runs of 32 columns.
__device__ __forceinline__ uint64_t sdesc_sw32(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)6 << 61;
    return d;
}
// Address of the 16-byte column group c of a key in such an operand (the swizzle exchanges a
// row's halves where bit 7 of the address is set: every other four rows).
__device__ __forceinline__ uint32_t p_addr(uint32_t base, uint32_t chunk, int c, int key) {
    return base + (c >> 1) * chunk + key * 32 + ((((uint32_t)c & 1u) ^ (((uint32_t)key >> 2) & 1u)) << 4);
}

// Byte `x` (0..127) of row n of an operand of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(uint32_t base, int n, int x) {
    return base + n * 128 + ((((uint32_t)x >> 4) ^ (n & 7)) << 4) + (x & 15);
}

// ---------------------------------------------------------------- the schedule

__device__ __forceinline__ bool len_ok(const Dec8Args &a, int len) {
    return len >= 0 && (long long)len <= (long long)a.page_size * a.max_pages;
}
// Tiles of one (head, row block) item of a sequence.
__device__ __forceinline__ int tiles_of_len(const Dec8Args &a, int len) {
    return len_ok(a, len) ? (int)(((long long)len + (1 << a.tile_log2) - 1) >> a.tile_log2) : 0;
}
__device__ __forceinline__ int tiles_of(const Dec8Args &a, int b) { return tiles_of_len(a, a.seq_lens[b]); }

// The cut is even in tiles and item starts: an item that begins inside a CTA's range costs it
// the results of the one before and a new set of queries, and counts as a.start tiles.  With few
// tiles per CTA the finest cut is better.
// (Positions below count both: item i's tile t is at its base + start + t.)
__device__ __forceinline__ int start_of(const Dec8Args &a, int tiles, int n_cta) {
    return tiles >= 4 * n_cta && tiles < (1 << 29) ? a.start : 0;
}

// Tiles (of one head and row block) and non-empty sequences, of all and of those before `upto`;
// one warp.
struct Count {
    int tiles, full, tiles_before, full_before;
};
__device__ __forceinline__ Count count_tiles(const Dec8Args &a, int upto) {
    const int lane = threadIdx.x & 31;
    Count c{};
    for (int b = lane; b < a.B; b += 32) {
        const int t = tiles_of(a, b);
        c.tiles += t;
        c.full += t > 0;
        if (b < upto) c.tiles_before += t, c.full_before += t > 0;
    }
    return Count{__reduce_add_sync(kFull, c.tiles), __reduce_add_sync(kFull, c.full),
                 __reduce_add_sync(kFull, c.tiles_before), __reduce_add_sync(kFull, c.full_before)};
}

// An even cut of `total` positions over the n CTAs that get any: the first `more` of them take
// one more than the others.
struct Cut {
    int n, each, more;
    Cut() = default;
    __device__ __forceinline__ Cut(int total, int n_cta) {
        n = min(total, n_cta);
        each = n ? total / n : 0;
        more = total - each * n;
    }
    __device__ __forceinline__ int first(int c) const { return c * each + min(c, more); }
    __device__ __forceinline__ int owner(int g) const {  // the CTA of position g
        const int big = more * (each + 1);
        return g < big ? g / (each + 1) : more + (g - big) / each;
    }
};

// A run of tiles of one item within this CTA's range.  Every role walks the same segments.
struct Segment {
    int b, kvh, rb;   // sequence, key/value head, row block
    int t0, t1, nt;   // tiles [t0, t1) of the item's nt
};
struct Walk {
    int left, b, item, at, nt, start;  // positions left, and the next one's place in its item
    int len_next;  // of sequence b + 1, under way while b is worked on
    __device__ __forceinline__ int tile() const { return max(at - start, 0); }
    __device__ __forceinline__ bool next(const Dec8Args &a, Segment *s) {
        while (left > 0) {
            if (nt == 0 || at >= start + nt) {  // the next item
                at = 0;
                if (++item >= a.Hkv * a.row_blocks || nt == 0) {
                    item = 0;
                    if (++b >= a.B) return false;  // not reached: `left` ends first
                    nt = tiles_of_len(a, len_next);
                    if (b + 1 < a.B) len_next = a.seq_lens[b + 1];
                }
                if (nt == 0) continue;
            }
            const int end = min(start + nt, at + left);
            s->t0 = tile();
            left -= end - at;
            at = end;
            s->t1 = tile();
            if (s->t1 == s->t0) continue;  // the range ends in the item's start
            s->b = b;
            s->kvh = a.row_blocks == 1 ? item : item / a.row_blocks;
            s->rb = item - s->kvh * a.row_blocks;
            s->nt = nt;
            return true;
        }
        return false;
    }
};

// Where CTA c of n_cta begins, and the cut; one warp.
__device__ __forceinline__ Walk start_walk(const Dec8Args &a, int c, int n_cta, Cut *the_cut) {
    const int lane = threadIdx.x & 31, ipb = a.Hkv * a.row_blocks;
    Walk w{};
    // the first 32 sequences' tiles stay in a register: most batches are no larger
    const int nt0 = lane < a.B ? tiles_of(a, lane) : 0;
    int mine = nt0, full = nt0 > 0;
    for (int b = lane + 32; b < a.B; b += 32) {
        const int nt = tiles_of(a, b);
        mine += nt;
        full += nt > 0;
    }
    mine = __reduce_add_sync(kFull, mine) * ipb;
    full = __reduce_add_sync(kFull, full) * ipb;
    w.start = start_of(a, mine, n_cta);
    const Cut cut(mine + w.start * full, n_cta);
    *the_cut = cut;
    if (c >= cut.n) return w;
    int g = cut.first(c);
    w.left = cut.first(c + 1) - g;
    for (int b = 0; b < a.B; b += 32) {
        const int nt = b == 0 ? nt0 : b + lane < a.B ? tiles_of(a, b + lane) : 0;
        const int size = (nt > 0 ? nt + w.start : 0) * ipb;
        int incl = size;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned m = __ballot_sync(kFull, incl > g);
        if (m) {
            const int k = __ffs(m) - 1;
            w.b = b + k;
            w.nt = __shfl_sync(kFull, nt, k);
            g -= __shfl_sync(kFull, incl - size, k);
            w.item = g / (w.nt + w.start);
            w.at = g - w.item * (w.nt + w.start);
            if (w.b + 1 < a.B) w.len_next = a.seq_lens[w.b + 1];
            break;
        }
        g -= __shfl_sync(kFull, incl, 31);
    }
    return w;
}

// ---------------------------------------------------------------- the kernel

// CAUSAL: rows of one item see different numbers of keys.  A kernel of its own, because what that
// needs (marks of NaN values, room for value scales) lies in code that runs once per item, where
// its size alone costs time (B256 of 1..600 keys, one query: 60 us without it, 68 us with).
template <int NCH, int RB, int PACK, bool CAUSAL>
__global__ void __launch_bounds__(Dec8Tile<NCH, RB, PACK>::THREADS, Dec8Tile<NCH, RB, PACK>::CTAS)
    fa_decode8_kernel(const __grid_constant__ Dec8Args a) {
    using T = Dec8Tile<NCH, RB, PACK>;
    using Misc = Dec8Misc<NCH, RB, T::STAGES, T::NWG, T::TK>;
    static_assert(sizeof(Misc) <= T::MISC, "state fits behind the buffers");
    constexpr int ST = T::STAGES, RW = T::RW, NWG = T::NWG, TK = T::TK;
    constexpr int kMmaWarp = 4 * NWG, kTmaWarp = kMmaWarp + 1, kAuxWarp = kMmaWarp + 2, kQueryWarp = kMmaWarp + 3;
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
            mbar_init(bar(ms.q_full[u]), 4 * NWG);
            mbar_init(bar(ms.q_empty[u]), 1 + NWG);  // the MMAs that read it, the warpgroups
            mbar_init(bar(ms.s_full[u]), 1);
            mbar_init(bar(ms.p_full[u]), 4 * NWG);   // one arrival per softmax warp
            mbar_init(bar(ms.pv_done[u]), 1);
        }
        for (int u = 0; u < kScaleStages; ++u) {
            mbar_init(bar(ms.scale_full[u]), 64);    // per lane: its copies, its other writes
            mbar_init(bar(ms.scale_empty[u]), 1);
        }
        mbar_init(bar(ms.done), 1);
        ms.abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&ms.tmem), T::TM_COLS);
        tmem_relinquish();
    }
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_desc(&a.tm_k);
        tma_prefetch_desc(&a.tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem;
    const Guard g{a.status, &ms.abort, a.limit_ns};

    // What the kernels before this one wrote is there from here on; the merge kernel may launch,
    // not earlier: it reads seq_lens without a wait of its own.
    griddep_wait();
    griddep_launch_dependents();

    // Every warp finds the CTA's first tile for itself (none waits for another's answer), and the
    // two that fetch page numbers the first of those.
    Cut cut;
    Walk walk = start_walk(a, blockIdx.x, gridDim.x, &cut);
    Segment s{};
    bool some = false;      // s is the CTA's first segment
    int len = 0;            // s's length and table row
    const int *bt = nullptr;
    const int boxes = kTile / a.box, entries = TK >> a.run;  // of a tile
    auto open = [&] {
        len = a.seq_lens[s.b];
        bt = a.block_table + (size_t)s.b * a.max_pages;
    };
    // page of the key that is `at` keys into tile t (-1 behind the last key or past this segment)
    auto page_at = [&](int t, int at) {
        const uint32_t key = (uint32_t)t * TK + (uint32_t)at;
        return t < s.t1 && key < (uint32_t)len ? __ldg(bt + a.by_page.div(key)) : -1;
    };
    int pg = -1;            // of this lane's first box, or scale entry, of a tile
    auto first_page = [&](int t) {
        if (warp == kTmaWarp) return lane < boxes ? page_at(t, lane * a.box * PACK) : -1;
        return page_at(t, lane << a.run);
    };
    if (warp == kTmaWarp || warp == kAuxWarp || warp == kQueryWarp) {
        some = walk.next(a, &s);
        if (some && warp != kQueryWarp) {
            open();
            pg = first_page(s.t0);
        }
    }
    if (warp == kMmaWarp && blockIdx.x == 0) {
        bool ok = true;
        for (int b = lane; b < a.B; b += 32) ok = ok && len_ok(a, a.seq_lens[b]);
        if (!__all_sync(kFull, ok) && lane == 0) {
            atomicCAS(a.status + 1, 0, SITE_DEC8_BAD_LEN);
            atomicExch(a.status, FA_ERR_BAD_INDEX);
        }
    }
    // Query terms of rows r, r + step, ... below RB of segment s into buffer qb, one warp.  A row
    // is scaled by the power of two that brings its largest magnitude into [128, 256); a row
    // with a NaN or an infinity becomes NaN.  N rows at a time, the next ones' loads under way:
    // one for the softmax warps, whose first segment waits for them (unrolled, code that runs
    // once takes longer to fetch than to execute), four for the query warp, alone with all RB.
    auto put_queries = [&](auto at_once, int qb, int r_first, int step) {
        constexpr int N = decltype(at_once)::value, W = NCH == 2 ? 4 : 2;
        const int E = a.d == 96 ? 4 : a.d / 32;  // elements per lane
        const bool on = lane * E < a.d;
        const int r0 = s.rb * RB, rows = min(RB, a.R - r0);
        const __nv_bfloat16 *src =
            a.q + (((long long)s.b * a.Hkv + s.kvh) * a.R + r0) * a.d + lane * E;
        auto load = [&](int r, uint32_t (&w)[W]) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = 0u;
            if (r >= rows || !on) return;
            const __nv_bfloat16 *p = src + (long long)r * a.d;
            if constexpr (NCH == 2) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p);
                w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            } else if (E == 4) {
                const uint2 x = *reinterpret_cast<const uint2 *>(p);
                w[0] = x.x; w[1] = x.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t *>(p);
            }
        };
        const int len = a.seq_lens[s.b];
        for (int r = r_first + lane * step; r < rows; r += 32 * step)  // all rows at once into L2
            for (int x = 0; x < a.d; x += 64) prefetch_l2(src + (long long)r * a.d - lane * E + x);
        uint32_t rows_w[N][W], next[N][W];
#pragma unroll
        for (int e = 0; e < N; ++e) load(r_first + e * step, rows_w[e]);
#pragma unroll 1
        for (int rn = r_first; rn < RB; rn += N * step) {
#pragma unroll
            for (int e = 0; e < N; ++e) load(rn + (N + e) * step, next[e]);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int r = rn + e * step;
                const uint32_t (&w)[W] = rows_w[e];
                uint32_t c1[W / 2], c2[W / 2], ex = 1;
#pragma unroll
                for (int i = 0; i < W / 2; ++i) c1[i] = c2[i] = 0u;
                if (r < rows) {
                    uint32_t am = 0;
#pragma unroll
                    for (int i = 0; i < W; ++i) am = max(am, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
                    am = __reduce_max_sync(kFull, am);
                    ex = max((int)(am >> 7) - 7, 1);
                    const float inv = __uint_as_float((254u - ex) << 23);
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        if (i % 2 && E == 2) continue;
                        // 8 significant bits fit f16, and so do both remainders
                        uint32_t h = pack_f16(__uint_as_float(w[i] << 16) * inv,
                                              __uint_as_float(w[i] & 0xffff0000u) * inv);
                        if (am >= 0x7f80u) h = 0x7fff7fffu;
                        const uint32_t c = e4m3x2_of(h);
                        const uint32_t d = e4m3x2_of(remainder32(h, f16x2_of(c)));
                        c1[i / 2] |= c << (16 * (i % 2));
                        c2[i / 2] |= d << (16 * (i % 2));
                    }
                }
                if (on) {
                    const int n1 = r / RW * (2 * RW) + r % RW;
#pragma unroll
                    for (int i = 0; i < W / 2; ++i) {
                        const int col = lane * E + 4 * i;  // byte of the row
                        const uint32_t q0 = sQ + qb * T::Q_BYTES + (col >> 7) * T::Q_CHUNK;
                        const uint32_t a1 = swizzled(q0, n1, col & 127), a2 = swizzled(q0, n1 + RW, col & 127);
                        if (NCH == 1 && E == 2) {
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(a1), "h"((uint16_t)c1[i]) : "memory");
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(a2), "h"((uint16_t)c2[i]) : "memory");
                        } else {
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(a1), "r"(c1[i]) : "memory");
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(a2), "r"(c2[i]) : "memory");
                        }
                    }
                }
                if (lane == 0) ms.row_scale[qb][r] = __uint_as_float(ex << 23) * a.scale_log2;
            }
#pragma unroll
            for (int e = 0; e < N; ++e)
#pragma unroll
                for (int i = 0; i < W; ++i) rows_w[e][i] = next[e][i];
        }
        if (r_first == 0) {
            for (int r = lane; r < RB; r += 32)
                ms.limit[qb][r] = CAUSAL && r < rows ? min(len, len - a.Nq + 1 + (r0 + r) % a.Nq) : len;
            if (CAUSAL)
                for (int i = lane; i < RB * NCH * 4; i += 32) ms.nan_cols[qb][i / (NCH * 4)][i % (NCH * 4)] = 0u;
            if (lane == 0) {
                ms.len[qb] = len;
                ms.nan_any[qb] = 0;
            }
        }
    };

    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ TMA producer
        // The whole warp runs the loop.  A tile is a run of boxes of `box` rows (the largest
        // power of two that divides a page's rows, so a box never straddles two pages); lane i
        // looks up and copies box i (and i + 32, ... of pages that allow only tiny boxes).  Boxes
        // behind the last key are not copied.  Page numbers are fetched one tile ahead and looked
        // at only when they are used.
        uint32_t n = 0;  // ring slots used so far
        bool ok = true;
        for (bool first = true; ok && some; first = false, some = walk.next(a, &s)) {
            if (!first) {
                open();
                pg = first_page(s.t0);
            }
#pragma unroll 1
            for (int t = s.t0; ok && t < s.t1; ++t) {
                const int pg_next = first_page(t + 1);
                auto page_of = [&](int i) { return i < 32 ? pg : page_at(t, i * a.box * PACK); };
                auto valid = [&](int page) { return page >= 0 && page < a.num_pages; };
                int mine = 0;
#pragma unroll 1
                for (int i = lane; i < boxes; i += 32) mine += valid(page_of(i)) ? 1 : 0;
                const uint32_t bytes =
                    (uint32_t)__reduce_add_sync(kFull, mine) * (uint32_t)a.box * 128u * NCH;
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const int slot = (int)(n % ST);
                    ok = n < (uint32_t)ST ||
                         mbar_wait_warp<T::INLINE_WAITS>(bar(ms.empty[slot]), ((n / ST) - 1) & 1, g, SITE_DEC_EMPTY);
                    if (!ok) break;
                    const uint32_t fb = bar(ms.full[slot]);
                    const CUtensorMap *map = kv ? &a.tm_v : &a.tm_k;
                    if (lane == 0) {
                        if (bytes) mbar_arrive_expect_tx(fb, bytes);
                        else mbar_arrive(fb);
                    }
                    __syncwarp();
#pragma unroll 1
                    for (int i = lane; i < boxes; i += 32) {
                        const int page = page_of(i), row = i * a.box;
                        if (!valid(page)) continue;
                        const uint32_t key = (uint32_t)(t * TK + row * PACK);
                        const int y = (int)(key - a.by_page.div(key) * (uint32_t)a.page_size) / PACK;
                        const uint32_t dst = base + slot * T::SLOT + row * 128;
#pragma unroll
                        for (int c = 0; c < NCH; ++c)
                            tma_load_3d(dst + c * T::CHUNK, map, fb, c * 128, y, page * a.Hkv + s.kvh);
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
            for (uint32_t i = n > (uint32_t)ST ? n - ST : 0; i < n; ++i)
                mbar_wait_warp<T::INLINE_WAITS>(bar(ms.full[i % ST]), (i / ST) & 1, g2, SITE_DEC_DRAIN);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t kIdescS = idesc_e4m3_f32(128, T::NS);
        constexpr uint32_t kIdescO = idesc_e4m3_f32(128, T::NP) | (1u << 10) | (3u << 15);  // B e5m2; both MN-major
        const int ksteps = a.d / 32;
        Walk ahead = walk;   // segments of S, up to two steps ahead of O
        Segment sa;
        bool more = ahead.next(a, &sa);
        int ta = more ? sa.t0 : 0;
        uint32_t js = 0, seg = 0;  // steps whose S is issued; segments begun
        bool ok = true;
        // a ring slot of K or V and the parity of its round, two slots further with every tile
        struct Slot {
            int at;
            uint32_t round;
            __device__ __forceinline__ void advance() {
                at += 2;
                if (at >= ST) at -= ST, round ^= 1;
            }
        };
        Slot k_slot{0, 0}, v_slot{1, 0};
        const uint64_t d_ring = sdesc_sw128(base, 16, 1024), d_q = sdesc_sw128(sQ, 16, 1024);
        const uint64_t d_v = sdesc_sw128(base, T::CHUNK, 1024), d_p = sdesc_sw32(sP, T::P_CHUNK, 256);
        auto issue_s = [&]() {
            const int u = js & 1, qb = seg & 1, half = (int)(js % PACK);
            if (ta == sa.t0)
                ok = ok && mbar_wait_warp<T::INLINE_WAITS>(bar(ms.q_full[qb]), (seg >> 1) & 1, g, SITE_DEC_MMA);
            if (half == 0)
                ok = ok && mbar_wait_warp<T::INLINE_WAITS>(bar(ms.full[k_slot.at]), k_slot.round, g, SITE_DEC_FULL);
            if (!ok) return;
            tc_fence_after();
            const uint64_t dk = desc_add(d_ring, k_slot.at * T::SLOT + half * 64);
            const uint64_t dq = desc_add(d_q, qb * T::Q_BYTES);
#pragma unroll
            for (int ks = 0; ks < NCH * 4 / PACK; ++ks)
                if (PACK == 2 || NCH == 2 || ks < ksteps)
                    mma_ss_elect_f8(tmem + u * T::NS, desc_add(dk, (ks >> 2) * T::CHUNK + (ks & 3) * 32),
                                    desc_add(dq, (ks >> 2) * T::Q_CHUNK + (ks & 3) * 32), kIdescS,
                                    ks > 0 ? 1u : 0u);
            tc_commit_elect(bar(ms.s_full[u]));
            ++js;
            if (half + 1 < PACK) return;
            tc_commit_elect(bar(ms.empty[k_slot.at]));
            k_slot.advance();
            if (++ta == sa.t1) {
                tc_commit_elect(bar(ms.q_empty[qb]));
                ++seg;
                more = ahead.next(a, &sa);
                ta = more ? sa.t0 : 0;
            }
        };
        // S of a segment whose queries are not there yet is not waited for while O of the tiles
        // before it can be issued.  (B75 Hkv16 R = 16 d256, one tile per item: 61 -> 50 us.)
        auto ready = [&]() {
            return (ta != sa.t0 || __all_sync(kFull, mbar_test(bar(ms.q_full[seg & 1]), (seg >> 1) & 1)));
        };
        uint32_t j = 0;
        while (ok && walk.next(a, &s)) {
            for (int t = s.t0; ok && t < s.t1; t += (int)(++j % PACK == 0)) {
                const int u = j & 1, half = (int)(j % PACK);
#pragma unroll 1
                while (ok && more && (js == j || (js == j + 1 && ready()))) issue_s();
                ok = ok && mbar_wait_warp<T::INLINE_WAITS>(bar(ms.p_full[u]), (j >> 1) & 1, g, SITE_DEC_MMA);
                // every softmax warp has read the tile's scales
                if (half + 1 == PACK && lane == 0) mbar_arrive(bar(ms.scale_empty[j / PACK % kScaleStages]));
                if (half == 0)
                    ok = ok && mbar_wait_warp<T::INLINE_WAITS>(bar(ms.full[v_slot.at]), v_slot.round, g, SITE_DEC_FULL);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dv = desc_add(d_v, v_slot.at * T::SLOT), dp = desc_add(d_p, u * T::P_BYTES);
#pragma unroll
                for (int c = 0; c < NCH; ++c)
#pragma unroll
                    for (int ks = 0; ks < kTile / 32; ++ks)
                        mma_ss_elect_f8(tmem + T::TM_O + (c + half) * T::NP, desc_add(dv, c * T::CHUNK + ks * 4096),
                                        desc_add(dp, ks * 1024), kIdescO, (t > s.t0 || ks > 0) ? 1u : 0u);
                tc_commit_elect(bar(ms.pv_done[u]));
                if (half + 1 == PACK) {
                    tc_commit_elect(bar(ms.empty[v_slot.at]));
                    v_slot.advance();
                }
            }
        }
        // fires once every MMA issued above has completed (normal or aborted run)
        tc_commit_elect(bar(ms.done));
        volatile int never = 0;
        const Guard g2{a.status, &never, kWaitLimitNs};
        mbar_wait_warp<T::INLINE_WAITS>(bar(ms.done), 0, g2, SITE_DEC_DRAIN);
    } else if (warp == kAuxWarp) {
        // ------------------------------------------------------ key and value scales
        uint32_t seg = 0, j = 0;
        bool ok = true;
        for (; ok && some; ++seg, some = walk.next(a, &s)) {
            const int qb = seg & 1;
            if (seg >= 1) {
                open();
                pg = first_page(s.t0);
                if (seg >= 2)  // `bad` of the segment before the last has been read
                    ok = mbar_wait_warp<T::INLINE_WAITS>(bar(ms.q_empty[qb]), ((seg >> 1) - 1) & 1, g, SITE_DEC_EMPTY);
                if (!ok) break;
            }
            if (lane == 0) ms.bad[qb] = 0;
            __syncwarp();
            for (int t = s.t0; ok && t < s.t1; ++t, ++j) {
                const int pg_next = first_page(t + 1);
                const int st = (int)(j % kScaleStages);
                ok = j < kScaleStages || mbar_wait_warp<T::INLINE_WAITS>(bar(ms.scale_empty[st]), ((j / kScaleStages) - 1) & 1,
                                                        g, SITE_DEC_EMPTY);
                if (!ok) break;
#pragma unroll 1
                for (int i = lane; i < entries; i += 32) {
                    const int at = i << a.run;
                    const int page = i < 32 ? pg : page_at(t, at);
                    const uint32_t key = (uint32_t)(t * TK + at);
                    const bool here = key < (uint32_t)len, valid = page >= 0 && page < a.num_pages;
                    if (here && !valid) ms.bad[qb] = 1;
                    const bool copy = here && valid;  // keys not there: scale 0
                    const uint32_t row = key - a.by_page.div(key) * (uint32_t)a.page_size;
                    const size_t from = copy ? ((size_t)page * a.Hkv + s.kvh) * a.groups + a.by_group.div(row) : 0;
                    cp_async4(smem_u32(&ms.k_scale[st][i]), a.k_scale + from, copy);
                    cp_async4(smem_u32(&ms.v_scale[st][i]), a.v_scale + from, copy);
                }
                __syncwarp();
                cp_async_arrive(bar(ms.scale_full[st]));
                mbar_arrive(bar(ms.scale_full[st]));
                pg = pg_next;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kQueryWarp) {
        // ------------------------------------------------------ query terms
        // Of the segments after the first, whose rows the softmax warps, idle then, share out: a
        // warp of its own, because 32 rows take one warp longer than several tiles take the others
        // (B8 H32 Hkv4 Nq4 d64: 41.7 us, and 44.6 us when the warp of the scales did it between
        // two items).
        bool ok = true;
        if (some) some = walk.next(a, &s);
        for (uint32_t seg = 1; some; ++seg, some = walk.next(a, &s)) {
            const int qb = seg & 1;
            if (seg >= 2) ok = mbar_wait_warp<T::INLINE_WAITS>(bar(ms.q_empty[qb]), ((seg >> 1) - 1) & 1, g, SITE_DEC_EMPTY);
            if (!ok) break;
            put_queries(std::integral_constant<int, 4>(), qb, 0, 1);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_n(bar(ms.q_full[qb]), 4 * NWG);
        }
    } else {
        // ------------------------------------------------------------ softmax, epilogue
        // Every warp runs every step even after a wait has given up (waits then return at
        // once), so that none is left behind at a barrier.
        const int wg = warp >> 2, w4 = warp & 3;
        const int kk = threadIdx.x & 127;  // key of the step; lane of O^T (head dimension)
        const int rw0 = wg * RW;           // this warpgroup's rows of the CTA's
        const int id = 1 + wg;             // its named barrier
        const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
        const uint32_t t_s = tmem + lane_base + wg * 2 * RW;
        const uint32_t t_o = tmem + lane_base + T::TM_O + wg * 3 * RW;
        uint32_t j = 0, seg = 0;
        float l[RW];
        while (walk.next(a, &s)) {
            const int qb = seg & 1;
            const int r0 = s.rb * RB + rw0, rows = min(RW, a.R - r0);  // may be none
            if (seg == 0) {
                put_queries(std::integral_constant<int, 1>(), 0, warp, 4 * NWG);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ms.q_full[0]));
            }
            if (kk < RW) ms.nref[rw0 + kk] = -kUnseen;
            // kOneP / vref (0: none yet), vref the power of two that value scales are taken relative
            // to; and what a scale may not pass, vref, or -1 where some row's terms are divided
            float vmul = 0.f, vmax = 0.f;
            auto vref_of = [&] { return !CAUSAL ? vmax : vmul > 0.f ? kOneP * inverse2(vmul) : 0.f; };
#pragma unroll
            for (int r = 0; r < RW; ++r) l[r] = 0.f;
            mbar_wait_warp<T::INLINE_WAITS>(bar(ms.q_full[qb]), (seg >> 1) & 1, g, SITE_DEC_MMA);
            named_barrier_sync(id, 128);
            const int len = ms.len[qb];
            const int full_keys = CAUSAL ? len - a.Nq + 1 : len;  // keys that every row sees
            const int full_tiles = max(full_keys, 0) / TK;          // of those only
            for (int t = s.t0; t < s.t1; t += (int)(++j % PACK == 0)) {
                const int u = j & 1, half = (int)(j % PACK);
                const uint32_t jt = j / PACK;
                const int at = kk * PACK + half, key = t * TK + at;
                const int st = (int)(jt % kScaleStages);
                const bool first = t == s.t0 && half == 0;
                mbar_wait<T::INLINE_WAITS>(bar(ms.scale_full[st]), (jt / kScaleStages) & 1, g, SITE_DEC_FULL);
                float ks = ms.k_scale[st][at >> a.run], vs = ms.v_scale[st][at >> a.run];
                mbar_wait<T::INLINE_WAITS>(bar(ms.s_full[u]), (j >> 1) & 1, g, SITE_DEC_MMA);
                __syncwarp();
                tc_fence_after();
                const bool partly = t >= full_tiles;  // some row sees less
                // base-2 exponents of the rows' scores of this thread's key; with REF less the
                // references
                float x[RW];
                auto scores = [&](auto ref) {
                    float c1[RW];
                    tmem_ld(t_s + u * T::NS, c1);
                    tmem_ld(t_s + u * T::NS + RW, x);
                    tmem_wait(c1);
                    tmem_wait(x);
                    const uint64_t k32 = f32x2_splat(1.f / 32.f), ks2 = f32x2_splat(ks);
#pragma unroll
                    for (int r = 0; r < RW; r += 4) {
                        const float4 rs = *reinterpret_cast<const float4 *>(&ms.row_scale[qb][rw0 + r]);
                        float f[4] = {rs.x, rs.y, rs.z, rs.w};
                        float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
                        if constexpr (decltype(ref)::value)
                            m = *reinterpret_cast<const float4 *>(&ms.nref[rw0 + r]);
                        mul_f32x2(f[0], f[1], ks2);
                        mul_f32x2(f[2], f[3], ks2);
                        fma_f32x2(x[r], x[r + 1], k32, c1[r], c1[r + 1]);
                        fma_f32x2(x[r + 2], x[r + 3], k32, c1[r + 2], c1[r + 3]);
                        fma_pairs(x[r], x[r + 1], f[0], f[1], m.x, m.y);
                        fma_pairs(x[r + 2], x[r + 3], f[2], f[3], m.z, m.w);
                    }
                    if (partly) {
#pragma unroll
                        for (int r = 0; r < RW; ++r)
                            if (key >= ms.limit[qb][rw0 + r]) x[r] = -INFINITY;
                    }
                };
                bool move = first;  // which always sets them
                if (!move) {
                    scores(std::true_type());
                    float top = fmaxf(x[0], x[1]);
#pragma unroll
                    for (int r = 2; r < RW; r += 2) top = fmax3(top, x[r], x[r + 1]);
                    move = vote_group(id, top > kMoveLog2 || vs > vmax);
                }
                if (move) {
                    // new references: the step's maximum where it passes the old one by 2^6
                    __syncwarp();  // a vote's barrier does not bring a warp's lanes together
                    scores(std::false_type());
                    // Where not every row sees the key, its value scale must not push the others'
                    // terms out of e5m2's range: it counts for the common reference as 2^-60 of
                    // itself, and where it is above that still, the rows that see the key divide
                    // their terms.  Then every step up to the item's end comes here.
                    const bool some_see = CAUSAL && partly && key >= full_keys;
                    const float vs_all = some_see && vs > 0.f ? fmaxf(vs * 0x1p-60f, 0x1p-126f) : vs;
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        const float m = warp_max(x[r]);
                        if (lane == r) ms.part[w4][rw0 + r] = m;
                    }
                    const float vm_warp = warp_max(vs_all);
                    if (lane == 0) ms.vpart[wg][w4] = vm_warp;
                    const bool roomy = vmax < 0.f;
                    const float v_old = vref_of();
                    float vref = v_old;
                    __syncwarp();
                    named_barrier_sync(id, 128);
                    const float vm = fmaxf(fmaxf(ms.vpart[wg][0], ms.vpart[wg][1]),
                                           fmaxf(ms.vpart[wg][2], ms.vpart[wg][3]));
                    // a power of two 8 to 16 times the largest scale, so that it seldom moves
                    // again (p's terms have the room), and kOneP / v_new stays finite
                    if (vm > v_old) {
                        vref = fmaxf(__uint_as_float(__float_as_uint(vm) & 0x7f800000u) * 16.f, 0x1p-110f);
                        vmul = kOneP * inverse2(vref);
                    }
                    vmax = vref;
                    float room = 0.f;
                    if (kk < RW) {
                        const int r = rw0 + kk;
                        const float m_old = -ms.nref[r];
                        const float m = fmaxf(fmaxf(ms.part[0][r], ms.part[1][r]),
                                              fmaxf(ms.part[2][r], ms.part[3][r]));
                        const bool up = m > m_old + kMoveLog2;
                        const float down = up ? m_old - m : 0.f;  // log2 of alpha
                        ms.alpha[r] = ex2(down);
                        if (up) ms.nref[r] = -m;
                        if (CAUSAL && partly) {
                            // what the row's terms are divided by: the largest scale among the keys
                            // of the tile that it sees and others do not, over the reference, or
                            // what earlier ones leave of it
                            const int from = max(full_keys - t * TK, 0), to = min(ms.limit[qb][r] - t * TK, TK);
                            float top = 0.f;
                            if (from < to)
                                for (int i = from >> a.run; i <= (to - 1) >> a.run; ++i) top = fmaxf(top, ms.v_scale[st][i]);
                            auto log_over = [](float x, float y) {  // of powers of two
                                return (float)((int)(__float_as_uint(x) >> 23) - (int)(__float_as_uint(y) >> 23));
                            };
                            const float old = roomy ? ms.room[r] : 0.f;
                            const float left = roomy ? old + down - log_over(vref, v_old) : 0.f;
                            room = fmaxf(ceilf(left), top > vref ? log_over(top, vref) + 1.f : 0.f);
                            ms.alpha_o[r] = ex2(down + old - room);
                            ms.room[r] = room;
                        }
                    }
                    const bool divide = vote_group(id, room > 0.f);
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        l[r] *= ms.alpha[rw0 + r];
                        x[r] += ms.nref[rw0 + r];
                    }
                    if (CAUSAL && divide) {
                        vmax = -1.f;
#pragma unroll
                        for (int r = 0; r < RW; ++r) {  // the sum keeps p itself
                            const float p = ex2(x[r]);
                            x[r] -= ms.room[rw0 + r];
                            l[r] += p - ex2(x[r]);
                        }
                    }
                    if (!first) {  // O^T to the new references, once PV of the step before is done
                        const float fo = vref > 0.f ? v_old * inverse2(vref) : 1.f;
                        const float *alpha = CAUSAL && partly ? ms.alpha_o : ms.alpha;
                        mbar_wait_warp<T::INLINE_WAITS>(bar(ms.pv_done[(j - 1) & 1]), ((j - 1) >> 1) & 1, g, SITE_DEC_MMA);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < NCH * PACK; ++c)
#pragma unroll 1
                            for (int n = 0; n < 3 * RW; n += RW) {
                                float o[RW];
                                const uint32_t at = t_o + c * T::NP + n;
                                tmem_ld(at, o);
                                tmem_wait(o);
#pragma unroll
                                for (int e = 0; e < RW; ++e) o[e] *= alpha[rw0 + e] * fo;
                                tmem_st(at, o);
                            }
                        tmem_wait_st();
                    }
                }
                const uint64_t fv2 = f32x2_splat(vs * vmul);
                uint32_t term[3][RW / 4];
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    uint32_t h[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float pa = ex2(x[r + 2 * k]), pb = ex2(x[r + 2 * k + 1]);
                        add_f32x2(l[r + 2 * k], l[r + 2 * k + 1], pa, pb);
                        mul_f32x2(pa, pb, fv2);
                        h[k] = pack_f16(pa, pb);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {  // the upper bytes, and what they leave
                        term[e][r / 4] = __byte_perm(h[0], h[1], 0x7531);
                        h[0] = sub_f16x2(h[0], h[0] & 0xff00ff00u);
                        h[1] = sub_f16x2(h[1], h[1] & 0xff00ff00u);
                    }
                    term[2][r / 4] = e5m2x2_of(times32(h[0])) | e5m2x2_of(times32(h[1])) << 16;
                }
                // the buffer's last reader, PV of step j - 2, was issued before S of this step, whose
                // commit covers all that was issued before it
                const uint32_t p0 = sP + u * T::P_BYTES;
                if constexpr (RW == 8) {
                    sts128(p_addr(p0, T::P_CHUNK, 0, kk), term[0][0], term[0][1], term[1][0], term[1][1]);
                    sts128(p_addr(p0, T::P_CHUNK, 1, kk), term[2][0], term[2][1], 0u, 0u);
                } else {
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        sts128(p_addr(p0, T::P_CHUNK, 3 * wg + e, kk), term[e][0], term[e][1], term[e][2],
                               term[e][3]);
                }
                if (wg == 0 && partly) {
                    // P is 0 where a row does not see the key, but 0 times a NaN of V would not be:
                    // rows of V behind the last key, whatever lies there, become 0; so do the NaN
                    // codes of keys that some rows see and others do not, and the rows that
                    // do are noted
                    const uint32_t i = 2 * jt + 1;
                    const int slot = (int)(i % ST);
                    mbar_wait_warp<T::INLINE_WAITS>(bar(ms.full[slot]), (i / ST) & 1, g, SITE_DEC_FULL);
                    const uint32_t v0 = base + slot * T::SLOT + kk * 128;
                    constexpr int kGroups = NCH * 8 / PACK;  // of 16 columns
                    auto group = [&](int e) { return ((e & 7) + half * kGroups ^ (kk & 7)) << 4; };
                    if (key >= len) {
#pragma unroll
                        for (int e = 0; e < kGroups; ++e)
                            sts128(v0 + (e >> 3) * T::CHUNK + group(e), 0u, 0u, 0u, 0u);
                    } else if (key >= full_keys) {
                        auto codes = [&](int e) {
                            return reinterpret_cast<uint4 *>(gbase + slot * T::SLOT + (e >> 3) * T::CHUNK + kk * 128 +
                                                             group(e));
                        };
                        // a NaN code is 7f or ff: adding 1 to its low 7 bits sets the eighth
                        auto nan_of = [](uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
                        uint32_t any = 0;
#pragma unroll 4
                        for (int e = 0; e < kGroups; ++e) {
                            const uint4 w = *codes(e);
                            any |= nan_of(w.x) | nan_of(w.y) | nan_of(w.z) | nan_of(w.w);
                        }
                        if (any) {
#pragma unroll 1
                            for (int e = 0; e < kGroups * 4; ++e) {  // four columns at a time
                                uint32_t *x = reinterpret_cast<uint32_t *>(codes(e >> 2)) + (e & 3);
                                const uint32_t nan = nan_of(*x);
                                if (nan == 0) continue;
                                *x &= ~((nan >> 7) * 255u);
                                ms.nan_any[qb] = 1;
                                const uint32_t bits = (nan >> 7 & 1u) | (nan >> 14 & 2u) | (nan >> 21 & 4u) | (nan >> 28 & 8u);
                                for (int r = 0; r < RB; ++r)
                                    if (key < ms.limit[qb][r]) atomicOr(&ms.nan_cols[qb][r][e >> 3], bits << (4 * (e & 7)));
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ms.p_full[u]));
            }
            // ---- the segment's rows: sums over all keys, then O^T columns
            const uint32_t jl = j - 1;
#pragma unroll
            for (int q = 0; q < RW; q += 8) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = l[q + e];
                const float sum = warp_sum8(v, lane);
                if ((lane & 3) == 0) ms.part[w4][rw0 + q + (lane >> 2)] = sum;
            }
            __syncwarp();
            named_barrier_sync(id, 128);
            const bool whole = s.t0 == 0 && s.t1 == s.nt;
            const bool bad = ms.bad[qb] != 0;
            const bool dead = *g.abort != 0;
            const size_t prow = ((size_t)blockIdx.x * 2 + (s.t0 == 0 ? 1 : 0)) * RB + rw0;
            const long long row0 = ((long long)s.b * a.Hkv + s.kvh) * a.R + r0;
            if (bad && threadIdx.x == 0) {
                atomicCAS(a.status + 1, 0, SITE_DEC8_BAD_PAGE);
                atomicExch(a.status, FA_ERR_BAD_INDEX);
            }
            if (kk < RW) {
                const int r = rw0 + kk;
                const float sum = (ms.part[0][r] + ms.part[1][r]) + (ms.part[2][r] + ms.part[3][r]);
                const float l2 = sum == 0.f ? -INFINITY : lg2(sum) - ms.nref[r];  // base 2
                ms.alpha[r] = sum == 0.f ? 0.f : vref_of() * (1.f / kOneP) * reciprocal(sum);
                if (vmax < 0.f) ms.alpha[r] *= ex2(ms.room[r]);
                if (kk < rows && !dead) {
                    if (!whole) a.part_l[prow + kk] = bad ? __uint_as_float(kBadPartial) : l2;
                    else if (!bad) a.lse[row0 + kk] = l2 * kLn2;
                }
            }
            mbar_wait_warp<T::INLINE_WAITS>(bar(ms.pv_done[jl & 1]), (jl >> 1) & 1, g, SITE_DEC_MMA);
            tc_fence_after();
            named_barrier_sync(id, 128);
            const int upper = PACK == 2 ? w4 >> 1 : 0;  // lanes of the odd keys' half
#pragma unroll 1
            for (int c = 0; c < NCH; ++c) {
                const int dd = c * 128 + kk;
#pragma unroll 1
                for (int q = 0; q < RW && q < rows; q += 8) {
                    float o0[8], o1[8], o2[8];
                    __syncwarp();
                    const uint32_t at = t_o + (c + upper) * T::NP + q;
                    tmem_ld(at, o0);
                    tmem_ld(at + RW, o1);
                    tmem_ld(at + 2 * RW, o2);
                    tmem_wait(o0);
                    tmem_wait(o1);
                    tmem_wait(o2);
                    const float4 f0 = *reinterpret_cast<const float4 *>(&ms.alpha[rw0 + q]);
                    const float4 f1 = *reinterpret_cast<const float4 *>(&ms.alpha[rw0 + q + 4]);
                    const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) o0[e] += fmaf(o2[e], 0x1p-5f, o1[e]);
                    if constexpr (PACK == 2) {  // the odd keys' part, through a buffer of P, idle now
                        float *part = reinterpret_cast<float *>(gbase + T::OFF_P) + q * 64 + (kk & 63);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (upper) part[e * 64] = o0[e];
                        named_barrier_sync(id, 128);
                        if (upper) continue;
#pragma unroll
                        for (int e = 0; e < 8; ++e) o0[e] += part[e * 64];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) o0[e] *= f[e];
                    if (CAUSAL && ms.nan_any[qb]) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (ms.nan_cols[qb][rw0 + q + e][dd >> 5] >> (dd & 31) & 1u) o0[e] = NAN;
                    }
                    const int here = dd < a.d && !dead && !bad ? rows - q : 0;
                    if (whole) {
                        __nv_bfloat16 *out = a.o + (row0 + q) * a.d + dd;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (e < here) out[e * a.d] = __float2bfloat16(o0[e]);
                    } else {
                        float *out = a.part_o + (prow + q) * a.d + dd;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (e < here) out[e * a.d] = o0[e];
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            named_barrier_sync(id, 128);  // the state above is free for the next segment
            if (kk == 0) mbar_arrive(bar(ms.q_empty[qb]));
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

// Merge of the partial results of the items that were cut: L = log2 sum 2^(L_s),
// O = sum 2^(L_s - L) O_s.  Both kernels below are bound by latency: find the partials before
// waiting for the attention kernel, then one or two rounds of loads.  (What they read before that
// wait is seq_lens only, written by nothing later than the kernels before the attention kernel,
// which has waited for those before it lets a merge start.)

// The running result of one warp over partials first, first + step, ... of a row's n: reference,
// sum and output columns lane, lane + 32, ...; U partials with their L in flight at a time.
template <int E, int U, typename Row>
__device__ __forceinline__ void merge_part(const Dec8Args &a, Row prow, int first, int step, int n, float &m,
                                           float &sum, float (&acc)[E], bool &bad) {
    const int lane = threadIdx.x & 31;
    m = kUnseen;
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int k0 = first; k0 < n; k0 += step * U) {
        float w[U], x[U][E];
#pragma unroll
        for (int v = 0; v < U; ++v) {
            const int k = k0 + step * v;
            const bool in = k < n;
            const size_t pr = prow(in ? k : k0);
            w[v] = in ? __ldcg(a.part_l + pr) : -INFINITY;
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[v][e] = in && lane + 32 * e < a.d ? __ldcg(a.part_o + pr * a.d + lane + 32 * e) : 0.f;
        }
        float top = m;
#pragma unroll
        for (int v = 0; v < U; ++v) {
            bad = bad || __float_as_uint(w[v]) == kBadPartial;
            top = fmaxf(top, w[v]);
        }
        const float f = ex2(m - top);
        sum *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
        for (int v = 0; v < U; ++v) {
            const float wk = ex2(w[v] - top);
            sum += wk;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wk, x[v][e], acc[e]);
        }
        m = top;
    }
}

template <int E>
__device__ __forceinline__ void merge_out(const Dec8Args &a, long long row, float m, float sum,
                                          const float (&acc)[E]) {
    const int lane = threadIdx.x & 31;
    const float inv = sum == 0.f ? 0.f : reciprocal(sum);
    __nv_bfloat16 *o = a.o + row * a.d;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (lane + 32 * e < a.d) o[lane + 32 * e] = __float2bfloat16(acc[e] * inv);
    if (lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (m + lg2(sum)) * kLn2;
}

// One row by the CTA's eight warps: row r of its block, whose n partials the attention kernel's
// CTAs from c0 on left (n == 0: an empty sequence).  The warps' running results meet in `sh`.
constexpr int kRowWarps = 8;
template <int E>
struct RowShared {
    float acc[kRowWarps][E * 32], sum[kRowWarps], max[kRowWarps];
};
template <int E, int RB>
__device__ __forceinline__ void merge_row(const Dec8Args &a, RowShared<E> &sh, int c0, int r, int n, long long row) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    float m, sum, acc[E];
    merge_part<E, 4>(
        a, [&](int k) { return ((size_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * RB + r; }, warp, kRowWarps, n, m, sum,
        acc, bad);
#pragma unroll
    for (int e = 0; e < E; ++e) sh.acc[warp][lane + 32 * e] = acc[e];
    if (lane == 0) {
        sh.sum[warp] = sum;
        sh.max[warp] = bad ? INFINITY : m;
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int v = 0; v < kRowWarps; ++v) m = fmaxf(m, sh.max[v]);
    if (m == INFINITY) return;  // the sequence was rejected: nothing is written
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int v = 0; v < kRowWarps; ++v) {
        const float f = ex2(sh.max[v] - m);
        sum = fmaf(sh.sum[v], f, sum);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(sh.acc[v][lane + 32 * e], f, acc[e]);
    }
    merge_out(a, row, m, sum, acc);  // an empty sequence: sum 0
}

// A CTA for each row, which may have dozens of partials (a long sequence alone in the launch).
template <int NCH, int RB>
__global__ void __launch_bounds__(32 * kRowWarps)
    fa_decode8_merge_row_kernel(const __grid_constant__ Dec8Args a, int n_cta) {
    constexpr int E = NCH == 2 ? 8 : 4;  // columns lane, lane + 32, ... of a row
    __shared__ RowShared<E> sh;
    __shared__ int s_row, s_c0, s_n;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x;
    if (warp == 0) {
        const int i = row % a.Nq, bh = row / a.Nq, b = bh / a.H, h = bh - b * a.H, group = a.H / a.Hkv;
        const int nt = tiles_of(a, b), kvh = h / group, r = (h - kvh * group) * a.Nq + i;
        const int ipb = a.Hkv * a.row_blocks;
        int c0 = 0, n = 0;
        const Count count = count_tiles(a, b);
        const int start = start_of(a, count.tiles * ipb, n_cta);
        const Cut cut((count.tiles + start * count.full) * ipb, n_cta);
        if (nt > 0) {
            const int first = (count.tiles_before + start * count.full_before) * ipb +
                              (kvh * a.row_blocks + r / RB) * (nt + start) + start;
            c0 = cut.owner(first);
            n = cut.owner(first + nt - 1) - c0 + 1;
        }
        if (lane == 0) {
            s_row = r % RB;
            s_c0 = c0;
            s_n = n > 1 || a.seq_lens[b] == 0 ? n : -1;  // -1: written directly, or rejected
        }
    }
    griddep_wait();  // every partial result is written
    griddep_launch_dependents();
    __syncthreads();
    if (s_n >= 0) merge_row<E, RB>(a, sh, s_c0, s_row, s_n, row);
}

// Many rows, most of which were not cut.  Every cut lies where one of the attention kernel's
// CTAs begins, so there is a CTA here for each of those (times blocks of eight rows).  The first
// cut of an item merges it, one warp per row; in an item of many cuts (a long sequence among
// short ones) each takes some of the rows, with all of its warps.
constexpr int kCutRows = 8, kManyCuts = 16;
static_assert(kCutRows == kRowWarps, "the same CTA does both");
template <int NCH, int RB>
__global__ void __launch_bounds__(32 * kCutRows)
    fa_decode8_merge_cut_kernel(const __grid_constant__ Dec8Args a, int n_cta) {
    constexpr int E = NCH == 2 ? 8 : 4;
    __shared__ RowShared<E> sh;
    __shared__ int s_b, s_item, s_c0, s_n;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x;  // the CTA whose beginning this is
    if (warp == 0) {
        Cut cut;
        const Walk w = start_walk(a, c, n_cta, &cut);
        int c0 = 0, n = 0;
        if (c > 0 && w.left > 0 && w.tile() > 0) {
            const int first = cut.first(c) - w.tile();  // the item's first tile
            c0 = cut.owner(first);
            n = cut.owner(first + w.nt - 1) - c0 + 1;
        }
        if (lane == 0) {
            s_b = w.b;
            s_item = w.item;
            s_c0 = c0;
            s_n = n;
        }
    }
    griddep_wait();
    griddep_launch_dependents();
    __syncthreads();
    if (blockIdx.y == 0) {
        for (int b = c; b < a.B; b += gridDim.x) {
            if (a.seq_lens[b] != 0) continue;
            const long long row0 = (long long)b * a.H * a.Nq, rows = (long long)a.H * a.Nq;
            for (long long i = threadIdx.x; i < rows * a.d; i += blockDim.x)
                a.o[row0 * a.d + i] = __float2bfloat16(0.f);
            for (long long i = threadIdx.x; i < rows; i += blockDim.x) a.lse[row0 + i] = -INFINITY;
        }
    }
    const int n = s_n, c0 = s_c0, nth = c - c0 - 1;  // the item's nth cut, from 0
    const int kvh = a.row_blocks == 1 ? s_item : s_item / a.row_blocks, rb = s_item - kvh * a.row_blocks;
    const int r0 = blockIdx.y * kCutRows, rows = min(min(kCutRows, RB - r0), a.R - rb * RB - r0);
    const long long row0 = ((long long)s_b * a.Hkv + kvh) * a.R + rb * RB + r0;
    if (n > kManyCuts) {
        for (int i = nth; i < rows; i += n - 1) {
            merge_row<E, RB>(a, sh, c0, r0 + i, n, row0 + i);
            __syncthreads();
        }
    } else if (n > 0 && nth == 0 && warp < rows) {
        bool bad = false;
        float m, sum, acc[E];
        merge_part<E, 4>(
            a, [&](int k) { return ((size_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * RB + r0 + warp; }, 0, 1, n, m, sum,
            acc, bad);
        if (!bad) merge_out(a, row0 + warp, m, sum, acc);
    }
}

// CTAs of a launch: all that are resident, or the largest number of tiles there can be.
template <int NCH, int RB, int PACK>
int dec8_ctas(const Decode8Params &p) {
    const long long R = (long long)(p.H / p.Hkv) * p.Nq;
    const int tk = Dec8Tile<NCH, RB, PACK>::TK;
    const long long nt = ((long long)p.page_size * p.max_pages + tk - 1) / tk;
    const long long items = (long long)p.B * p.Hkv * ((R + RB - 1) / RB);
    const long long most = (long long)p.num_sms * Dec8Tile<NCH, RB, PACK>::CTAS;
    return (int)(items >= most || items * nt >= most ? most : items * nt);
}

template <int NCH, int RB, int PACK>
size_t dec8_bytes(const Decode8Params &p, size_t *l_offset) {
    const size_t rows = (size_t)dec8_ctas<NCH, RB, PACK>(p) * 2 * RB;
    *l_offset = rows * p.d * sizeof(float);  // a multiple of 16
    return *l_offset + rows * sizeof(float);
}

template <int NCH, int RB, int PACK>
int launch_t(const Decode8Params &p, cudaStream_t stream) {
    using T = Dec8Tile<NCH, RB, PACK>;
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
    dec8_bytes<NCH, RB, PACK>(p, &l_offset);
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
    a.box = decode8_box_rows(p.page_size / PACK);
    a.tile_log2 = PACK == 2 ? 8 : 7;
    // Measured, counted as 0, 1, 2 (and 3) tiles, in an earlier state whose calls of many short
    // sequences took 8% longer: one sequence of 131072 keys among 199 of 20, H32
    // Hkv8, 94, 74, 62 us; B256 of 1..600 keys 70.6, 66.0, 65.0; B32 of 1..8192 keys 49.0, 49.3,
    // 49.2 (0.8 more with 3).  With more rows a start costs more (0, 2, 3, 4 of B8 Hkv4 19000 keys
    // d64: R = 16 25.1, 23.8, 24.0, 24.4; R = 32 40.5, 39.6, 38.7, 38.6; R = 64 61.2, 63.2, 55.9, 60.6).
    a.start = RB > 8 ? 3 : 2;
    a.run = p.group % 4 == 0 ? 2 : 0;  // four keys of a tile share a page and a group, or none do
    a.scale_log2 = p.scale_log2;
    a.status = p.status;
    a.limit_ns = kWaitLimitNs;
    // a single query is the last token: it sees every key with either mask
    auto kern = p.causal && p.Nq > 1 ? fa_decode8_kernel<NCH, RB, PACK, true>
                                     : fa_decode8_kernel<NCH, RB, PACK, false>;
    constexpr int kSmem = (int)T::SMEM;
    if (ensure_smem_attr(reinterpret_cast<const void *>(kern), kSmem) != FA_OK) return FA_ERR_CUDA;
    const int n_cta = dec8_ctas<NCH, RB, PACK>(p);
    if (launch_dependent(kern, dim3((unsigned)n_cta), T::THREADS, kSmem, stream, 1, a) != FA_OK) return FA_ERR_CUDA;
    // the merge that has fewer CTAs (B32 H32 Hkv8, 1024 rows against 304 cuts: 50.7 us by rows,
    // 49.3 by cuts; B8 H32 Hkv4 Nq4, 1024 against 1216: 39.0 by rows, 39.9 by cuts)
    const long long rows = (long long)p.B * p.H * p.Nq;
    const int blocks = ((a.R < RB ? a.R : RB) + kCutRows - 1) / kCutRows;
    if (rows <= (long long)n_cta * blocks)
        return launch_dependent(fa_decode8_merge_row_kernel<NCH, RB>, dim3((unsigned)rows), 32 * kRowWarps, 0,
                                stream, 1, a, n_cta);
    return launch_dependent(fa_decode8_merge_cut_kernel<NCH, RB>, dim3((unsigned)n_cta, (unsigned)blocks),
                            32 * kCutRows, 0, stream, 1, a, n_cta);
}

// Tiles of 128 keys of all items in blocks of rb rows at the longest possible lengths.
long long most_tiles(const Decode8Params &p, int rb) {
    const long long R = (long long)(p.H / p.Hkv) * p.Nq;
    const long long nt = ((long long)p.page_size * p.max_pages + kTile - 1) / kTile;
    const long long items = (long long)p.B * p.Hkv * ((R + rb - 1) / rb);
    return items >= (1LL << 31) ? items : items * nt;
}

// Two keys to a row of a tile where a key is half of one, up to 16 query rows leave the time
// to copies, and every CTA may get more than two tiles of 128 keys; with less work, a finer cut
// is worth more.  (Hkv8 d64 R4, one key and two: B1 1000 keys 6.4 and 7.2 us, 16000 keys 11.9
// and 12.0 us; B32 of 1..1000 keys 20.7 and 17.1 us; B32 H16 of 30000 keys 238 and 170 us.  A
// key's number plus a tile's stays below 2^31.)
bool packs(const Decode8Params &p) {
    return p.d == 64 && (long long)(p.H / p.Hkv) * p.Nq <= 16 && p.page_size % 2 == 0 &&
           (long long)p.page_size * p.max_pages < (1LL << 31) - 256 && most_tiles(p, 16) > 4LL * p.num_sms;
}

// Calls f with the tile that serves the call's query rows per key/value head: the constants
// NCH, RB and PACK.
template <typename F>
auto with_tile(const Decode8Params &p, F f) {
    using std::integral_constant;
    using One = integral_constant<int, 1>;
    using Two = integral_constant<int, 2>;
    const long long R = (long long)(p.H / p.Hkv) * p.Nq;
    if (p.d == 256) {
        if (R <= 8) return f(Two(), integral_constant<int, 8>(), One());
        if (R <= 16) return f(Two(), integral_constant<int, 16>(), One());
        return f(Two(), integral_constant<int, 32>(), One());
    }
    if (packs(p)) {
        if (R <= 8) return f(One(), integral_constant<int, 8>(), Two());
        return f(One(), integral_constant<int, 16>(), Two());
    }
    if (R <= 8) return f(One(), integral_constant<int, 8>(), One());
    if (R <= 16) return f(One(), integral_constant<int, 16>(), One());
    if (R <= 32) return f(One(), integral_constant<int, 32>(), One());
    return f(One(), integral_constant<int, 64>(), One());
}

}  // namespace

int decode8_pack(const Decode8Params &p) {
    return with_tile(p, [](auto, auto, auto pack) { return (int)pack; });
}

int decode8_box_rows(int rows) {
    int box = 1;
    while (box < kTile && rows % (2 * box) == 0) box *= 2;
    return box;
}

long long decode8_max_tiles(const Decode8Params &p) {
    return with_tile(p, [&](auto, auto rb, auto) { return most_tiles(p, rb); });
}

size_t decode8_workspace_bytes(const Decode8Params &p) {
    return with_tile(p, [&](auto nch, auto rb, auto pack) {
        size_t l_offset;
        return dec8_bytes<decltype(nch)::value, decltype(rb)::value, decltype(pack)::value>(p, &l_offset);
    });
}

int launch_decode8(const Decode8Params &p, cudaStream_t stream) {
    return with_tile(p, [&](auto nch, auto rb, auto pack) {
        return launch_t<decltype(nch)::value, decltype(rb)::value, decltype(pack)::value>(p, stream);
    });
}

}  // namespace fa
