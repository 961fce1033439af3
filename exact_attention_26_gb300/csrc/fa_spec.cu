// What follows the attention of drafted trees: the verification of the drafted tokens against the
// target's probabilities (fa_verify_tree), and bringing the accepted ones' rows of the paged cache
// together (fa_keep_path).  The definitions are in fa.h.
#include <cooperative_groups.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

namespace cg = cooperative_groups;

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void flag_index(int *status, int site) {
    atomicCAS(status + 1, 0, site);
    atomicExch(status, FA_ERR_BAD_INDEX);
}

// ------------------------------------------------------------------ verification
//
// A sequence's walk down its tree is a chain of decisions, each behind a rejection needing a sum
// over the vocabulary; nothing else of it takes time.  A cluster of CTAs owns a sequence: one warp
// of each walks (all the same way), and all their threads share the sums, each warp a contiguous
// part of the row, so that the sums also lead to the token at the end: the CTA, the warp, the step
// and the lane in which the running sum passes u times the whole.
//
// Sums are whole numbers: each weight p - a q is formed in fp32 pairs, to 2^-46 of p, and taken
// in multiples of 2^-44, so no order of summation and no number of CTAs changes a result, and
// where p and a q are nearly equal what is left of them is kept.  fp64 would not do: this GPU adds two doubles per
// clock and SM.  The numbers are cut out by adding a constant whose last place is the multiple wanted
// and summing the bit patterns: 13 fp32 and integer operations per element, against two dozen, half
// of them shifts, of a conversion to 64 bits (B64 Nt24 V128000, six sums one after another: 80 us).
//
// Measured (GB300; graph replay of one input, whose rows are then in L2, and calls on inputs that
// change): B1 Nt16 V32000 fp32 7.7 and 6.4 to 8.7 us, B64 Nt24 V128000 fp32 without repetition 45 and
// 61 to 63, B48 Nt9 V50021 bf16 certain drafts 8.3 and 8.8.  CTAs of 256 threads, four to an SM: a wave holds twice
// the sequences that it held with 512 threads, two to an SM (9.7, 47.5 and 9.2 us).

constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxNodes = FA_MAX_TREE_NODES;

// x as a probability: 0 for what is below 0 or NaN, 1 above 1.
__device__ __forceinline__ float probability(float x) { return __saturatef(x); }

// floor(u whole), for u of any size; below `whole` also from u = 1 on.
__device__ __forceinline__ unsigned long long share_of(float u, unsigned long long whole) {
    u = probability(u);
    const uint32_t w = __float_as_uint(u), by = 126u - (w >> 23);  // u = m 2^-64-by
    const unsigned long long m = (unsigned long long)((w & 0x7fffffu) | 0x800000u) << 40;
    return u >= 1.f ? __umul64hi(~0ull, whole) : by < 64 ? __umul64hi(m, whole) >> by : 0ull;
}

// A weight of 0 .. 1 is k1 2^-22 + k2 2^-44: the bit patterns of kCut1 + k1 2^-22 and of kCut2 +
// k2 2^-44, floats whose last places those are.
constexpr float kCut1 = 3.0f, kCut2 = 1.5f * 0x1p-21f;
constexpr uint32_t kBits1 = 0x40400000u, kBits2 = 0x35400000u;
__device__ __forceinline__ long long weight_of(uint32_t k1, uint32_t k2) {  // of sums of up to 2^8
    return ((long long)(int)k1 << 22) + (int)k2;
}

template <typename P>
struct Row;  // the VEC probabilities of 16 bytes
template <>
struct Row<float> {
    static constexpr int VEC = 4;
    __device__ static float get(const uint4 &w, int i) {
        return probability(__uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w));
    }
    __device__ static float one(const float *p) { return probability(*p); }
};
template <>
struct Row<__nv_bfloat16> {
    static constexpr int VEC = 8;
    __device__ static float get(const uint4 &w, int i) {
        const uint32_t x = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
        return probability(__uint_as_float(i & 1 ? x & 0xffff0000u : x << 16));
    }
    __device__ static float one(const __nv_bfloat16 *p) { return probability(__bfloat162float(*p)); }
};

// What is left of the target's probabilities: max(p - a q, 0), or p without the rejected tokens.
struct Left {
    int cur;                     // the node after which they are
    float a_hi, a_lo;            // a, their sum
    int n_gone;
    int count;                   // nodes accepted so far
    int stop;                    // 1: this sum is for the token at the end
};

struct VerifyShared {
    int parents[kMaxNodes], tokens[kMaxNodes], gone[kMaxNodes];
    float u[kMaxNodes], px[kMaxNodes], qx[kMaxNodes], gone_p[kMaxNodes];
    unsigned long long warp_sum[kVerifyWarps];
    unsigned long long cta_sum[2][8];  // of every CTA of the cluster, by turns
    int bad;
    Left left;
};

template <typename P, bool DRAFT>
struct Weights {
    static constexpr int VEC = Row<P>::VEC;
    const P *p, *q;               // the node's rows
    const VerifyShared &sh;
    const Left &l;
    int V;

    // 16 bytes of both rows from element i0 on; 0 outside the rows (before them lies the row
    // before, or nothing; the first unit's elements there are passed over in `get`)
    struct Raw {
        uint4 a, b;
    };
    __device__ __forceinline__ Raw load(int i0) const {
        Raw r;
        r.b = make_uint4(0u, 0u, 0u, 0u);
        if (i0 + VEC <= V) {
            r.a = __ldg(reinterpret_cast<const uint4 *>(p + i0));
            if (DRAFT) r.b = __ldg(reinterpret_cast<const uint4 *>(q + i0));
        } else {
            uint32_t x[4] = {}, y[4] = {};
            constexpr int PER = VEC / 4;  // elements per word
            for (int e = 0; e < VEC; ++e) {
                if (i0 + e >= V) break;
                if (PER == 1) {
                    x[e] = reinterpret_cast<const uint32_t *>(p)[i0 + e];
                    if (DRAFT) y[e] = reinterpret_cast<const uint32_t *>(q)[i0 + e];
                } else {
                    x[e / PER] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[i0 + e] << 16 * (e % PER);
                    if (DRAFT) y[e / PER] |= (uint32_t)reinterpret_cast<const uint16_t *>(q)[i0 + e] << 16 * (e % PER);
                }
            }
            r.a = make_uint4(x[0], x[1], x[2], x[3]);
            r.b = make_uint4(y[0], y[1], y[2], y[3]);
        }
        return r;
    }

    // k1 and k2 of the weight of an element, as bit patterns
    __device__ __forceinline__ void cut(float x, float y, uint32_t &k1, uint32_t &k2) const {
        float w = x, rest = 0.f;  // the weight, as a sum
        if (DRAFT) {
            if (l.a_hi == 1.f && l.a_lo == 0.f) {
                x = fmaxf(x, y);
                w = x - y;
                rest = (x - w) - y;
            } else {
                // x - (h + lo); (x - d) - h is what d = x - h was rounded by, exactly so from x = h / 2 on,
                // and below that d decides.  The sign is the pair's: lo may outweigh an x below h.
                const float h = l.a_hi * y, lo = fmaf(l.a_lo, y, fmaf(l.a_hi, y, -h)), d = x - h;
                const float e = ((x - d) - h) - lo;
                w = d + e;
                rest = e - (w - d);
                if (!(w > 0.f)) w = rest = 0.f;
            }
        }
        const float t1 = w + kCut1;
        const float t2 = ((w - (t1 - kCut1)) + rest) + kCut2;
        k1 = __float_as_uint(t1);
        k2 = __float_as_uint(t2);
    }
    // their weights
    __device__ __forceinline__ void get(const Raw &r, int i0, uint32_t (&k1)[VEC], uint32_t (&k2)[VEC]) const {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            cut(Row<P>::get(r.a, e), DRAFT ? Row<P>::get(r.b, e) : 0.f, k1[e], k2[e]);
            k1[e] -= kBits1;
            k2[e] -= kBits2;
        }
        if (i0 < 0) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (i0 + e < 0) k1[e] = k2[e] = 0u;
        }
    }
    // without the tokens that are out
    __device__ __forceinline__ void drop_gone(int i0, unsigned long long (&w)[VEC]) const {
        for (int k = 0; k < l.n_gone; ++k) {
            const int at = sh.gone[k] - i0;
            if ((unsigned)at >= (unsigned)VEC) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e == at) w[e] = 0ull;
        }
    }
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

// The walk's numbers as sums of two floats, 2^-47 relative (Dekker's and Knuth's exact sums, and
// products by FMA): fp64's chains of dependent operations, at a sixteenth of the rate, were 1.5 us
// of each step.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair join(float a, float b) {  // |a| >= |b|
    const float s = a + b;
    return {s, b - (s - a)};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    const float s = a.hi + b.hi, v = s - a.hi;
    return join(s, ((a.hi - (s - v)) + (b.hi - v)) + (a.lo + b.lo));
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) { return a + Pair{-b.hi, -b.lo}; }
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    const float p = a.hi * b.hi;
    return join(p, fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, fmaf(a.hi, b.hi, -p))));
}
__device__ __forceinline__ bool operator<(Pair a, Pair b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
__device__ __forceinline__ Pair pair_of(float x) { return {x, 0.f}; }
// A sum of weights, in multiples of 2^-44.
__device__ __forceinline__ Pair pair_of(unsigned long long sum) {
    const float hi = __ull2float_rz(sum);
    return {hi * 0x1p-44f, __ull2float_rn(sum - (unsigned long long)hi) * 0x1p-44f};
}
// 1 / x by Newton's iteration.
__device__ __forceinline__ Pair inverse(Pair x) {
    const Pair r = pair_of(__frcp_rn(x.hi)), one = pair_of(1.f);
    return r + r * (one - x * r);
}

template <typename P, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads, 4) fa_verify_kernel(const VerifyParams v) {
    constexpr int VEC = Row<P>::VEC;
    __shared__ VerifyShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int b = blockIdx.x / ctas, Nt = v.Nt, V = v.V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const P *target = static_cast<const P *>(v.target) + (size_t)b * Nt * V;
    const P *draft = DRAFT ? static_cast<const P *>(v.draft) + (size_t)b * Nt * V : nullptr;
    // The CTAs write into each other's shared memory, which takes that they run: every CTA says here
    // that it does, and waits for the others in front of its first write (`met`).
    cluster_arrive();
    bool met = false;
    griddep_wait();
    griddep_launch_dependents();

    // the tree, and both probabilities of every drafted token after its parent
    if (threadIdx.x == 0) sh.bad = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < Nt; j += kVerifyThreads) {
        const size_t at = (size_t)b * Nt + j;
        int up = v.parents ? v.parents[at] : j - 1;
        const int x = v.tokens[at];
        const bool is = up >= -1, root = j == 0;
        bool bad = is && (root ? up != -1 : up < 0 || up >= j || x < 0 || x >= V);
        if (is && !root && !bad && v.parents) bad = v.parents[(size_t)b * Nt + up] < -1;
        if (bad) sh.bad = 1;
        if (bad || !is || root) up = root && is && !bad ? -1 : -2;
        sh.parents[j] = up;
        sh.tokens[j] = x;
        sh.u[j] = v.uniform[at];
        if (up >= 0) {
            sh.px[j] = Row<P>::one(target + (size_t)up * V + x);
            sh.qx[j] = DRAFT ? Row<P>::one(draft + (size_t)up * V + x) : 1.f;
        }
    }
    __syncthreads();
    int *path = v.path + (size_t)b * Nt, *fresh = v.fresh + (size_t)b * Nt;
    if (sh.bad || sh.parents[0] < -1) {  // the same in every CTA of the cluster
        if (rank == 0) {
            for (int j = threadIdx.x; j < Nt; j += kVerifyThreads) path[j] = fresh[j] = -1;
            if (threadIdx.x == 0) {
                v.count[b] = 0;
                if (sh.bad) flag_index(v.status, SITE_VERIFY_BAD_TREE);
            }
        }
        cluster_wait();
        return;
    }

    // the walk's state, of warp 0
    int cur = 0, count = 1, j = 0;
    const Pair zero = pair_of(0.f), one = pair_of(1.f);
    Pair a = zero, used = zero, total = one;  // of the draft's to take off; of the rejected; left
    int n_gone = 0;
    bool stale = false;                       // `total` is not known yet
    if (warp == 0 && rank == 0 && lane == 0) path[0] = 0;
    int turn = 0;  // of cta_sum
    for (;;) {
        if (warp == 0) {
            for (;;) {
                // the next child of the node
                int next = -1;
                for (int base = j + 1; base < Nt && next < 0; base += 32) {
                    const unsigned m = __ballot_sync(kFull, base + lane < Nt && sh.parents[base + lane] == cur);
                    if (m) next = base + __ffs(m) - 1;
                }
                if (next < 0 || stale) {
                    if (lane == 0) {
                        const Left l{cur, a.hi, a.lo, n_gone, count, next < 0};
                        sh.left = l;
                    }
                    break;
                }
                j = next;
                const Pair p = pair_of(sh.px[j]), u = pair_of(sh.u[j]), q = pair_of(sh.qx[j]);
                Pair drawn = one;  // 1 - s of the definition
                bool accept;
                if (DRAFT) {
                    const Pair w = p - a * q;
                    accept = u * q * total < w;
                    if (!v.replacement && used.hi > 0.f) {
                        drawn = one - used;
                        if (drawn.hi < 0x1p-60f) drawn = pair_of(0x1p-60f);
                        accept = u * q * total < w * drawn;
                    }
                } else {
                    bool gone = false;
                    for (int k = lane; k < n_gone; k += 32) gone = gone || sh.gone[k] == sh.tokens[j];
                    if (__any_sync(kFull, gone)) continue;  // its weight is 0
                    accept = u * total < p;
                }
                if (accept) {
                    if (rank == 0 && lane == 0) {
                        path[count] = j;
                        fresh[count - 1] = sh.tokens[j];
                    }
                    cur = j;
                    ++count;
                    a = used = zero;
                    total = one;
                    n_gone = 0;
                } else if (DRAFT) {
                    a = a + (drawn.hi == 1.f && drawn.lo == 0.f ? total : total * inverse(drawn));
                    if (a.hi > 0x1p60f) a = pair_of(0x1p60f);
                    used = used + q;
                    stale = true;
                } else {
                    if (lane == 0) {
                        sh.gone[n_gone] = sh.tokens[j];
                        sh.gone_p[n_gone] = sh.px[j];
                    }
                    __syncwarp();
                    ++n_gone;
                    total = total - p;
                }
            }
        }
        __syncthreads();
        const Left l = sh.left;
        const size_t row = (size_t)l.cur * V;
        const int before = (int)(((size_t)b * Nt * V + row) % VEC);
        const Weights<P, DRAFT> weights{target + row, DRAFT ? draft + row : nullptr, sh, l, V};
        // this CTA's, and this warp's, part of the row in units of 16 bytes
        const int units = (V + before + VEC - 1) / VEC;
        const int per_warp = (units + ctas * kVerifyWarps - 1) / (ctas * kVerifyWarps);
        const int u0 = (rank * kVerifyWarps + warp) * per_warp, u1 = min(u0 + per_warp, units);
        unsigned long long sum = 0;
        constexpr int kAhead = VEC == 4 || !DRAFT ? 4 : 2;  // loads in flight
        for (int i = u0 + lane; i - lane < u1; i += 32 * kAhead) {
            typename Weights<P, DRAFT>::Raw raw[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                raw[k] = weights.load(i + 32 * k < u1 ? (i + 32 * k) * VEC - before : V);  // from V on, zeros
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                uint32_t k1[VEC], k2[VEC], s1 = 0, s2 = 0;
                weights.get(raw[k], (i + 32 * k) * VEC - before, k1, k2);
#pragma unroll
                for (int e = 0; e < VEC; ++e) s1 += k1[e], s2 += k2[e];
                sum += weight_of(s1, s2);
            }
        }
        if (!DRAFT) {  // the tokens that are out, of this warp's part
            for (int k = lane; k < l.n_gone; k += 32) {
                const int unit = (sh.gone[k] + before) / VEC;
                uint32_t k1, k2;
                weights.cut(sh.gone_p[k], 0.f, k1, k2);
                if (unit >= u0 && unit < u1) sum -= weight_of(k1 - kBits1, k2 - kBits2);
            }
        }
        sum = warp_sum(sum);
        if (lane == 0) sh.warp_sum[warp] = sum;
        __syncthreads();
        if (!met) cluster_wait();
        met = true;
        if (warp == 0) {
            const unsigned long long all = warp_sum(lane < kVerifyWarps ? sh.warp_sum[lane] : 0ull);
            if (lane < ctas) cluster.map_shared_rank(&sh, lane)->cta_sum[turn][rank] = all;
        }
        cluster.sync();
        unsigned long long whole = 0, here = 0;
        for (int r = 0; r < ctas; ++r) {
            if (r == rank) here = whole;
            whole += sh.cta_sum[turn][r];
        }
        const unsigned long long mine = sh.cta_sum[turn][rank];
        turn ^= 1;
        if (!l.stop) {
            total = pair_of(whole);
            stale = false;
            continue;
        }
        if (whole == 0 && (l.a_hi > 0.f || l.n_gone)) {  // the drafts left nothing: the target's own
            a = zero;
            n_gone = 0;
            stale = false;
            j = Nt;
            __syncthreads();
            continue;
        }
        // ---- the token whose part of the running sum holds u times the whole
        const unsigned long long goal = share_of(sh.u[0], whole);
        if (warp == 0 && rank == 0) {
            for (int i = count + lane; i < Nt; i += 32) path[i] = fresh[i] = -1;
            if (lane == 0) {
                v.count[b] = count;
                if (whole == 0) fresh[count - 1] = -1;
            }
        }
        if (goal < here || goal - here >= mine) break;
        // it is this CTA's: in the part of warp w, which all threads go through, a unit each
        unsigned long long left = goal - here;
        int w = 0;
        while (left >= sh.warp_sum[w]) left -= sh.warp_sum[w++];
        const int first = (rank * kVerifyWarps + w) * per_warp, end = min(first + per_warp, units);
        for (int base = first; base < end; base += kVerifyThreads) {
            unsigned long long x[VEC], sum = 0;
            const int unit = base + (int)threadIdx.x, i0 = unit * VEC - before;
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = 0ull;
            if (unit < end) {
                uint32_t k1[VEC], k2[VEC];
                weights.get(weights.load(i0), i0, k1, k2);
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[e] = weight_of(k1[e], k2[e]);
                if (!DRAFT) weights.drop_gone(i0, x);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum += x[e];
            unsigned long long run = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long y = __shfl_up_sync(kFull, run, o);
                if (lane >= o) run += y;
            }
            __syncthreads();  // the sums below are read
            if (lane == 31) sh.warp_sum[warp] = run;
            __syncthreads();
            unsigned long long all = 0;
            run -= sum;
            for (int k = 0; k < kVerifyWarps; ++k) {
                if (k < warp) run += sh.warp_sum[k];
                all += sh.warp_sum[k];
            }
            if (left >= all) {
                left -= all;
                continue;
            }
            if (left >= run && left - run < sum) {
                int found = i0;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    if (left >= run && left - run < x[e]) found = i0 + e;
                    run += x[e];
                }
                fresh[l.count - 1] = found;
            }
            break;
        }
        break;
    }
}

// ------------------------------------------------------------------ kept rows
//
// A copy of a few rows per sequence, head and layer: the metadata (path, pages) is a chain of
// dependent loads, so a CTA looks it up once and moves the rows of many layers and heads with it.
// The moves overlap (row 3's place may be row 7's new one): new places are never behind old ones
// and both ascend, so rows taken in order, each batch read before any of it is written, stay
// what they were.
//
// Measured (GB300, graph replay): 64 sequences of 24 layers (48 cache tensors), Hkv8 d128, 192 rows that
// move, 37.7 MB read and written: 10.2 us, behind a chain of lookups of about 3; one sequence 2.9 us (calls on inputs that change: 12 and 5.6 to
// 6.4).
// Small CTAs of few registers, as many as an SM holds, hide the lookups best: 128 threads with 4 loads in
// flight 10.2 us, 64 threads 10.7, 256 threads 10.8, with 8 loads in flight 11.9.

constexpr int kKeepThreads = 128, kKeepWarps = kKeepThreads / 32;
constexpr int kKeepInFlight = 4;  // 16-byte loads of a lane before the first store

__global__ void __launch_bounds__(kKeepThreads) fa_keep_kernel(const __grid_constant__ KeepParams k) {
    __shared__ long long s_src[kMaxNodes], s_dst[kMaxNodes];  // rows of the cache, of head 0
    __shared__ int s_n, s_bad;
    const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();
    griddep_launch_dependents();
    const int len = k.seq_lens[b], count = k.count[b];
    const long long room = (long long)k.page_size * k.max_pages;
    if (threadIdx.x == 0) {
        s_n = 0;
        s_bad = len < 0 || count < 0 || count > k.Nt || (long long)len + count > room;
    }
    __syncthreads();
    if (!s_bad) {
        const int *path = k.path + (size_t)b * k.Nt, *bt = k.block_table + (size_t)b * k.max_pages;
        for (int i = threadIdx.x; i < count; i += kKeepThreads) {
            const int node = path[i], before = i > 0 ? path[i - 1] : -1;
            bool bad = node <= before || node >= k.Nt;
            if (!bad) {  // also of a row that stays
                const uint32_t from = (uint32_t)(len + node), to = (uint32_t)(len + i), ps = (uint32_t)k.page_size;
                const uint32_t fp = from / ps, tp = to / ps;
                const int from_page = fp < (uint32_t)k.max_pages ? bt[fp] : -1, to_page = bt[tp];
                bad = from_page < 0 || from_page >= k.num_pages || to_page < 0 || to_page >= k.num_pages;
                s_src[i] = (long long)from_page * k.Hkv * k.page_size + (from - fp * ps);
                s_dst[i] = (long long)to_page * k.Hkv * k.page_size + (to - tp * ps);
            }
            if (bad) s_bad = 1;
            if (node == i) atomicMax(&s_n, i + 1);  // the leading rows stay
        }
    }
    __syncthreads();
    const bool bad = s_bad != 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        k.lens[b] = bad ? len : len + count;
        if (bad) flag_index(k.status, SITE_KEEP_BAD_PATH);
    }
    if (bad) return;
    // rows first .. count - 1 move (ascending nodes: once one moves, so do those behind it)
    const int first = s_n, m = count - first;
    if (m <= 0) return;
    const int lanes = k.d / 8, at_once = 32 / lanes;  // lanes of a row, rows of a step
    const int group = lane / lanes, col = (lane - group * lanes) * 8;
    const int batch = kKeepInFlight * at_once;
    const int heads = k.n_caches * k.Hkv;             // (cache, head) units
    // units of a batch: as many as there is room for, and no more than make work for every warp
    const int share = (heads + gridDim.x * kKeepWarps - 1) / (gridDim.x * kKeepWarps);
    const int per = m <= batch ? min(batch / m, share) : 1;
    for (int h0 = (blockIdx.x * kKeepWarps + warp) * per; h0 < heads; h0 += gridDim.x * kKeepWarps * per) {
        const int n = min(per, heads - h0) * m;       // rows of these units
        for (int r0 = 0; r0 < n; r0 += batch) {
            uint4 x[kKeepInFlight];
            __nv_bfloat16 *to[kKeepInFlight];
#pragma unroll
            for (int e = 0; e < kKeepInFlight; ++e) {
                const int r = r0 + e * at_once + group;
                to[e] = nullptr;
                if (group < at_once && r < n) {
                    const int unit = (int)((uint32_t)r / (uint32_t)m), i = first + r - unit * m;
                    const int c = (int)((uint32_t)(h0 + unit) / (uint32_t)k.Hkv), h = h0 + unit - c * k.Hkv;
                    __nv_bfloat16 *cache = static_cast<__nv_bfloat16 *>(k.cache[c]);
                    const long long head = (long long)h * k.page_size;
                    to[e] = cache + (s_dst[i] + head) * k.d + col;
                    x[e] = *reinterpret_cast<const uint4 *>(cache + (s_src[i] + head) * k.d + col);
                }
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < kKeepInFlight; ++e)
                if (to[e]) *reinterpret_cast<uint4 *>(to[e]) = x[e];
            __syncwarp();
        }
    }
}

template <typename P>
int launch_verify_t(const VerifyParams &v, int ctas, cudaStream_t stream) {
    const dim3 grid((unsigned)(v.B * ctas));
    return v.draft ? launch_dependent(fa_verify_kernel<P, true>, grid, kVerifyThreads, 0, stream, ctas, v)
                   : launch_dependent(fa_verify_kernel<P, false>, grid, kVerifyThreads, 0, stream, ctas, v);
}

}  // namespace

int launch_verify(const VerifyParams &v, cudaStream_t stream) {
    // CTAs per sequence: more while each still has 24 KB of a node's rows, and all of them are no more than
    // two waves (a sequence of many sums, alone at the end, then has more of the GPU), or, where drafts are
    // certain and a sequence has one sum, than one.  With 1, 2, 4, 8: V1000 fp32, two rows, B64 12.6, 14.8,
    // 14.7, 17.0 us; V8000 B64 32.8, 29.9, 30.5, 32.3; V32000 B1 19.4, 12.9, 9.1, 7.7, B256 88, 61, 55, 60;
    // V128000 B64 172, 98, 60, 45; V50021 bf16, one row, B48 12.3, 9.6, 8.4, 8.2, B256 16.7, 16.7, 20.9, 30.3.
    const long long bytes = (long long)v.V * (v.bf16 ? 2 : 4) * (v.draft ? 2 : 1);
    const long long most = (v.draft ? 7LL : 4LL) * v.num_sms;
    int ctas = 1;
    while (ctas < 8 && (long long)v.B * ctas * 2 <= most && bytes / (ctas * 2) >= 24000) ctas *= 2;
    return v.bf16 ? launch_verify_t<__nv_bfloat16>(v, ctas, stream) : launch_verify_t<float>(v, ctas, stream);
}

int launch_keep(const KeepParams &k, cudaStream_t stream) {
    // CTAs per sequence: all that the GPU holds at once, 16 to an SM (12, 16, 24 of them: 10.3, 10.2, 10.3
    // us for the 64 sequences above)
    const int heads = k.n_caches * k.Hkv, most = (heads + kKeepWarps - 1) / kKeepWarps;
    const int want = 16 * k.num_sms / k.B, n = want < 1 ? 1 : want < most ? want : most;
    return launch_dependent(fa_keep_kernel, dim3((unsigned)n, (unsigned)k.B), kKeepThreads, 0, stream, 1, k);
}

}  // namespace fa
