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
// Sums are exact: probabilities are held in 64-bit fixed point, 2^-60, in which a 24-bit
// significand is exact from 2^-37 up and smaller ones are off by less than 2^-60.  So no order of
// summation and no number of CTAs changes a result, and where p and q are nearly equal nothing is
// lost.  (In fp64 the sums would be ten times the work: this GPU adds two doubles per clock and SM.)

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxNodes = FA_MAX_TREE_NODES;

// floor(x 2^bits) of x >= 0, NaN and below as 0, 1 and above as 2^bits (bits 60), or one less
// (bits 64).
template <int BITS>
__device__ __forceinline__ unsigned long long to_fixed(float x) {
    if (!(x > 0.f)) return 0ull;
    if (x >= 1.f) return BITS == 64 ? ~0ull : 1ull << (BITS & 63);
    const uint32_t w = __float_as_uint(x);
    const int e = (int)(w >> 23) - 150 + BITS;  // x = m 2^(e - BITS)
    const unsigned long long m = (w & 0x7fffffu) | 0x800000u;  // a subnormal's is shifted out all the same
    return e >= 0 ? m << e : e > -24 ? m >> -e : 0ull;
}

__device__ __forceinline__ float probability(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }

template <typename P>
struct Row;  // the VEC probabilities of 16 bytes
template <>
struct Row<float> {
    static constexpr int VEC = 4;
    __device__ static float get(const uint4 &w, int i) {
        return __uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w);
    }
    __device__ static float one(const float *p) { return *p; }
};
template <>
struct Row<__nv_bfloat16> {
    static constexpr int VEC = 8;
    __device__ static float get(const uint4 &w, int i) {
        const uint32_t x = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
        return __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16);
    }
    __device__ static float one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
};

// What is left of the target's probabilities: max(p - a q, 0), or p without the rejected tokens.
struct Left {
    int cur;                     // the node after which they are
    unsigned long long a;        // a = a_fixed 2^-shift, of 62 significant bits; shift < 0: a is 1
    int shift;
    int n_gone;
    int count;                   // nodes accepted so far
    int stop;                    // 1: this sum is for the token at the end
};

struct VerifyShared {
    int parents[kMaxNodes], tokens[kMaxNodes], gone[kMaxNodes];
    float u[kMaxNodes], px[kMaxNodes], qx[kMaxNodes];
    unsigned long long warp_sum[kVerifyWarps];
    unsigned long long cta_sum[2][16];  // of every CTA of the cluster, by turns
    int bad;
    Left left;
};

template <typename P, bool DRAFT>
struct Weights {
    static constexpr int VEC = Row<P>::VEC;
    const P *p, *q;               // the node's rows
    const VerifyShared &sh;
    const Left &l;
    int V, before;                // elements of the first 16 bytes that lie before the row

    // the weights of elements i0 .. i0 + VEC - 1, which share 16 bytes; 0 outside the row
    __device__ __forceinline__ void get(int i0, unsigned long long (&w)[VEC]) const {
        float x[VEC], y[VEC];
        if (i0 + VEC <= V) {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p + i0));
            const uint4 b = DRAFT ? __ldg(reinterpret_cast<const uint4 *>(q + i0)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                x[e] = i0 + e >= 0 ? Row<P>::get(a, e) : 0.f;
                y[e] = DRAFT ? Row<P>::get(b, e) : 0.f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const bool in = i0 + e >= 0 && i0 + e < V;
                x[e] = in ? Row<P>::one(p + i0 + e) : 0.f;
                y[e] = in && DRAFT ? Row<P>::one(q + i0 + e) : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = to_fixed<60>(x[e]);
        if (DRAFT) {
            if (l.a) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    unsigned long long off = to_fixed<60>(y[e]);
                    if (l.shift >= 0) {
                        const unsigned long long hi = __umul64hi(l.a, off), lo = l.a * off;
                        off = hi >> l.shift ? ~0ull : l.shift == 0 ? lo : hi << (64 - l.shift) | lo >> l.shift;
                    }
                    w[e] = w[e] > off ? w[e] - off : 0ull;
                }
            }
        } else {
            for (int k = 0; k < l.n_gone; ++k) {
                const int at = sh.gone[k] - i0;
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (e == at) w[e] = 0ull;
            }
        }
    }
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

template <typename P, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads) fa_verify_kernel(const VerifyParams v) {
    constexpr int VEC = Row<P>::VEC;
    __shared__ VerifyShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int b = blockIdx.x / ctas, Nt = v.Nt, V = v.V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const P *target = static_cast<const P *>(v.target) + (size_t)b * Nt * V;
    const P *draft = DRAFT ? static_cast<const P *>(v.draft) + (size_t)b * Nt * V : nullptr;
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
            sh.px[j] = probability(Row<P>::one(target + (size_t)up * V + x));
            sh.qx[j] = DRAFT ? probability(Row<P>::one(draft + (size_t)up * V + x)) : 1.f;
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
        return;
    }

    // the walk's state, of warp 0
    int cur = 0, count = 1, j = 0;
    double a = 0.0, used = 0.0, total = 1.0;  // of the draft's to take off; of the rejected; left
    int n_gone = 0;
    bool stale = false;                       // `total` is not known yet
    if (warp == 0 && rank == 0 && lane == 0) path[0] = 0;
    // this CTA's, and this warp's, part of a row in units of 16 bytes
    int turn = 0;
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
                        Left l{cur, 0ull, -1, n_gone, count, next < 0};
                        if (a > 0.0) {
                            int e;
                            frexp(a, &e);  // a < 2^e
                            l.a = (unsigned long long)ldexp(a, 62 - e);
                            l.shift = a == 1.0 ? -1 : 62 - e;
                        }
                        sh.left = l;
                    }
                    break;
                }
                const double p = (double)sh.px[next], q = (double)sh.qx[next];
                double w, rest = 1.0, tried = q;  // q of what the draft draws from: all, or the rest
                if (DRAFT) {
                    w = fmax(p - a * q, 0.0);
                    if (!v.replacement && used > 0.0) {
                        rest = fmax(1.0 - used, 0x1p-60);
                        tried = q / rest;
                    }
                } else {
                    const int x = sh.tokens[next];
                    bool gone = false;
                    for (int k = 0; k < n_gone; ++k) gone = gone || sh.gone[k] == x;
                    w = gone ? 0.0 : p;
                }
                j = next;
                if ((double)sh.u[j] * tried * total < w) {
                    if (rank == 0 && lane == 0) {
                        path[count] = j;
                        fresh[count - 1] = sh.tokens[j];
                    }
                    cur = j;
                    ++count;
                    a = used = 0.0;
                    total = 1.0;
                    n_gone = 0;
                } else if (DRAFT) {
                    a = fmin(a + (rest == 1.0 ? total : total / rest), 0x1p60);
                    used += q;
                    stale = true;
                } else {
                    if (lane == 0) sh.gone[n_gone] = sh.tokens[j];
                    __syncwarp();
                    ++n_gone;
                    total -= w;
                }
            }
        }
        __syncthreads();
        const Left l = sh.left;
        const size_t row = (size_t)l.cur * V;
        const int before = (int)(((size_t)b * Nt * V + row) % VEC);
        const Weights<P, DRAFT> weights{target + row, DRAFT ? draft + row : nullptr, sh, l, V, before};
        const int units = (V + before + VEC - 1) / VEC;
        const int per_warp = (units + ctas * kVerifyWarps - 1) / (ctas * kVerifyWarps);
        const int u0 = (rank * kVerifyWarps + warp) * per_warp, u1 = min(u0 + per_warp, units);
        unsigned long long sum = 0;
        for (int i = u0 + lane; i < u1; i += 32) {
            unsigned long long w[VEC];
            weights.get(i * VEC - before, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum += w[e];
        }
        sum = warp_sum(sum);
        if (lane == 0) sh.warp_sum[warp] = sum;
        __syncthreads();
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
            total = (double)whole * 0x1p-60;
            stale = false;
            continue;
        }
        if (whole == 0 && (l.a || l.n_gone)) {  // the drafts left nothing: the target's own
            a = 0.0;
            n_gone = 0;
            stale = false;
            j = Nt;
            __syncthreads();
            continue;
        }
        // ---- the token whose part of the running sum holds u times the whole
        const unsigned long long goal = __umul64hi(to_fixed<64>(sh.u[0]), whole);
        if (warp == 0 && rank == 0) {
            for (int i = count + lane; i < Nt; i += 32) path[i] = fresh[i] = -1;
            if (lane == 0) {
                v.count[b] = count;
                if (whole == 0) fresh[count - 1] = -1;
            }
        }
        // (a CTA's own count is the same in all of them)
        if (goal >= here && goal - here < mine) {
            unsigned long long before_warp = here;
            for (int w = 0; w < warp; ++w) before_warp += sh.warp_sum[w];
            if (goal >= before_warp && goal - before_warp < sh.warp_sum[warp]) {
                unsigned long long left = goal - before_warp;
                for (int base = u0; base < u1; base += 32) {
                    unsigned long long w[VEC], lane_sum = 0;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) w[e] = 0ull;
                    const int i0 = (base + lane) * VEC - before;
                    if (base + lane < u1) weights.get(i0, w);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) lane_sum += w[e];
                    unsigned long long incl = lane_sum;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const unsigned long long y = __shfl_up_sync(kFull, incl, o);
                        if (lane >= o) incl += y;
                    }
                    const unsigned long long all = __shfl_sync(kFull, incl, 31);
                    if (left < all) {
                        unsigned long long run = incl - lane_sum;
                        if (left >= run && left < incl) {
                            int found = i0;
#pragma unroll
                            for (int e = 0; e < VEC; ++e) {
                                if (left >= run && left - run < w[e]) found = i0 + e;
                                run += w[e];
                            }
                            fresh[l.count - 1] = found;
                        }
                        break;
                    }
                    left -= all;
                }
            }
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

constexpr int kKeepThreads = 256, kKeepWarps = kKeepThreads / 32;
constexpr int kKeepInFlight = 8;  // 16-byte loads of a lane before the first store

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
            if (!bad && node != i) {
                const long long from = (long long)len + node, to = (long long)len + i;
                const int from_page = from < room ? bt[from / k.page_size] : -1, to_page = bt[to / k.page_size];
                bad = from_page < 0 || from_page >= k.num_pages || to_page < 0 || to_page >= k.num_pages;
                s_src[i] = (long long)from_page * k.Hkv * k.page_size + from % k.page_size;
                s_dst[i] = (long long)to_page * k.Hkv * k.page_size + to % k.page_size;
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
    const int per = m <= batch ? batch / m : 1;       // units of a batch
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
                    const int unit = r / m, i = first + r - unit * m;
                    const int c = (h0 + unit) / k.Hkv, h = h0 + unit - c * k.Hkv;
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
    // CTAs per sequence: more while they all fit the GPU at once and have a few thousand elements
    int ctas = 1;
    while (ctas < 8 && (long long)v.B * ctas * 2 <= 4LL * v.num_sms && v.V / (ctas * 2) >= 2048) ctas *= 2;
    return v.bf16 ? launch_verify_t<__nv_bfloat16>(v, ctas, stream) : launch_verify_t<float>(v, ctas, stream);
}

int launch_keep(const KeepParams &k, cudaStream_t stream) {
    // CTAs per sequence: about two waves of the GPU in all
    const int heads = k.n_caches * k.Hkv, most = (heads + kKeepWarps - 1) / kKeepWarps;
    const int want = (8 * k.num_sms + k.B - 1) / k.B;
    return launch_dependent(fa_keep_kernel, dim3((unsigned)(want < most ? want : most), (unsigned)k.B), kKeepThreads, 0,
                            stream, 1, k);
}

}  // namespace fa
