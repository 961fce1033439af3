// The cut of a decode launch over a paged cache, and the merge of what it leaves in parts.
//
// The tiles of all (sequence, key/value head, block of query rows) items, laid end to end, are cut
// evenly over the launch's CTAs (a prefix sum over seq_lens on the device, so ragged batches
// balance and a captured launch follows the lengths).  A CTA writes finished rows directly and at
// most two partial results (the item its range begins in, the item it ends in), which a merge
// kernel joins by log-sum-exp.
//
// Shared by kernels whose argument block `Args` has B, H, Hkv, Nq, d, R (query rows per
// key/value head), row_blocks, start, seq_lens, o, lse, part_o [CTA][2][RB][d], part_l
// [CTA][2][RB], and, found with it, tiles_of_len(a, len): the tiles of one item of a sequence
// (0 where the length is bad), and empty_len(a, len): has it no key, so that its rows are the
// merge's to write?  RB, the rows of an item, is a constant of the kernel, or 0 where it is
// a.item_rows.  Args::kKeepInfinities: an infinity in a part is the row's, however little the part
// weighs; d is a multiple of 32 then.
#pragma once

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kUnseen = -3.0e38f;    // reference of a row that has seen no key yet
constexpr uint32_t kBadPartial = 0x7fc0bad1u;  // L of a partial result of a rejected sequence

struct FastDiv {  // n / d for 0 <= n < 2^31
    uint32_t d, mul, shift;
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return d == 1 ? n : __umulhi(n, mul) >> shift;
    }
};

inline FastDiv fast_div(uint32_t d) {
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

// 1 / x to 2^-23 (x normal), which O's rounding to bf16 hides, without a divide's code.
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---------------------------------------------------------------- the schedule

template <typename Args>
__device__ __forceinline__ int tiles_of(const Args &a, int b) { return tiles_of_len(a, a.seq_lens[b]); }

// The cut is even in tiles and item starts: an item that begins inside a CTA's range costs it
// the results of the one before and a new set of queries, and counts as a.start tiles.  With few
// tiles per CTA the finest cut is better.
// (Positions below count both: item i's tile t is at its base + start + t.)
template <typename Args>
__device__ __forceinline__ int start_of(const Args &a, int tiles, int n_cta) {
    return tiles >= 4 * n_cta && tiles < (1 << 29) ? a.start : 0;
}

// Tiles (of one head and row block) and non-empty sequences, of all and of those before `upto`;
// one warp.
struct Count {
    int tiles, full, tiles_before, full_before;
};
template <typename Args>
__device__ __forceinline__ Count count_tiles(const Args &a, int upto) {
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
    template <typename Args>
    __device__ __forceinline__ bool next(const Args &a, Segment *s) {
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
template <typename Args>
__device__ __forceinline__ Walk start_walk(const Args &a, int c, int n_cta, Cut *the_cut) {
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

// ---------------------------------------------------------------- the merge

// Merge of the partial results of the items that were cut: L = log2 sum 2^(L_s),
// O = sum 2^(L_s - L) O_s.  Both kernels below are bound by latency: find the partials before
// waiting for the attention kernel, then one or two rounds of loads.  (What they read before that
// wait is seq_lens only, written by nothing later than the kernels before the attention kernel,
// which has waited for those before it lets a merge start.)

template <int RB, typename Args>
__device__ __forceinline__ int item_rows_of(const Args &a) {
    if constexpr (RB > 0) return RB;
    else return a.item_rows;
}

// Of COLUMNS columns of a row of D, STEP apart from `col` (at o) on, those that the merge of its n parts
// made NaN although no weight is: an infinity has met a weight of 0.  They become the sum of the
// parts' infinities (and NaN) as they are.  Part 0 is row pr0 of part_o, part k row pr1 and 2 k items' rows
// more.  (A function of its own, behind the merge and the stores: factors that spare infinities, in
// the merge, or this in line cost 1 to 2 us of B32 R = 128 of 1..8192 keys, B1 R = 256 of 131072
// keys and B5 Hkv2 R = 168 of d256; so it costs none.)
template <int RB, int D, int COLUMNS, int STEP, typename Args>
__device__ __noinline__ void put_infinities(const Args &a, size_t pr0, size_t pr1, int n, int col, __nv_bfloat16 *o) {
    for (int e = 0; e < COLUMNS * STEP; e += STEP) {
        float kept = 0.f;
        for (int k = 0; k < n; ++k) {
            const float x = __ldcg(a.part_o + (k == 0 ? pr0 : pr1 + (size_t)(2 * k) * item_rows_of<RB>(a)) * D + col + e);
            if (!(fabsf(x) < INFINITY)) kept += x;
        }
        if (kept != 0.f) o[e] = __float2bfloat16(kept);
    }
}

// The running result of one warp over partials first, first + step, ... of a row's n: reference,
// sum and output columns lane, lane + 32, ...; U partials with their L in flight at a time.
template <int E, int U, typename Args, typename Row>
__device__ __forceinline__ void merge_part(const Args &a, Row prow, int first, int step, int n, float &m,
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

template <int E, typename Args>
__device__ __forceinline__ void merge_out(const Args &a, long long row, float m, float sum,
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
template <int E, int RB, typename Args>
__device__ __forceinline__ void merge_row(const Args &a, RowShared<E> &sh, int c0, int r, int n, long long row) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    float m, sum, acc[E];
    merge_part<E, 4>(
        a, [&](int k) { return ((size_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * item_rows_of<RB>(a) + r; }, warp, kRowWarps, n,
        m, sum,
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
    if constexpr (Args::kKeepInfinities) {
        float any = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) any += acc[e];
        if (any != any && sum == sum)
            put_infinities<RB, 32 * E, E, 32>(a, ((size_t)c0 * 2 + 1) * item_rows_of<RB>(a) + r,
                                              (size_t)c0 * 2 * item_rows_of<RB>(a) + r, n, lane, a.o + row * a.d + lane);
    }
}

// A CTA for each row, which may have dozens of partials (a long sequence alone in the launch).
template <int E, int RB, typename Args>
__global__ void __launch_bounds__(32 * kRowWarps)
    fa_merge_row_kernel(const __grid_constant__ Args a, int n_cta) {
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
                              (kvh * a.row_blocks + r / item_rows_of<RB>(a)) * (nt + start) + start;
            c0 = cut.owner(first);
            n = cut.owner(first + nt - 1) - c0 + 1;
        }
        if (lane == 0) {
            s_row = r % item_rows_of<RB>(a);
            s_c0 = c0;
            s_n = n > 1 || empty_len(a, a.seq_lens[b]) ? n : -1;  // -1: written directly, or rejected
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
template <int E, int RB, typename Args>
__global__ void __launch_bounds__(32 * kCutRows)
    fa_merge_cut_kernel(const __grid_constant__ Args a, int n_cta) {
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
            if (!empty_len(a, a.seq_lens[b])) continue;
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

}  // namespace
}  // namespace fa
