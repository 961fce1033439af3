// Filling and keeping a paged key/value cache: storing new tokens as e4m3 codes with a
// power-of-two scale per group of tokens and head, and the upkeep of the pages (listing
// the unused ones, forking sequences, compaction, copying).  The definitions are in fa.h.
#include <cooperative_groups.h>

#include <type_traits>

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

// ------------------------------------------------------------------ append
//
// A group's new codes need the group's largest magnitude first, so its rows are held in
// registers between the maximum and the conversion and read once: 2 bytes in, 1 byte out
// per element, bound by HBM.  A team of W warps owns one (group, head, key or value); a lane
// holds eight consecutive elements of a row (16-byte loads, 8-byte stores), so a warp covers
// one to four rows at a time and 16 in all.  Teams are handed out by windows of `window`
// consecutive rows of the call: a team walks the groups that begin in its window, which needs
// no list of the groups (their number is only known on the device).  The host sets the window
// to about the rows a group gets, so a window holds about one group whether the call stores
// prompts or one token per sequence.  Finding a group is a chain of dependent loads (offsets
// and lengths, page), during which a warp holds no data: many resident warps hide it, which
// the registers are kept few for.  Measured (GB300, graph replay, Hkv8 d128): 14083 tokens of
// seven prompts 18.9 us, 4.5 TB/s of 3 bytes per element (a wave of CTAs is latency for its
// first half; eight rows per warp and more warps 23 us, two heads per warp with the next
// one's rows under way 27 us); one token each for 128 sequences 3.4 us, latency.

template <int D>
struct RowLanes {
    static constexpr int E = 8;                // elements per lane
    static constexpr int PER_ROW = D / E;      // lanes of a row
    static constexpr int ROWS = 32 / PER_ROW;  // rows a warp covers at a time (d = 96: 2, 24 lanes)
    static constexpr int STEPS = 16 / ROWS;    // to cover 16 rows
    static_assert(16 % ROWS == 0, "whole steps");
};

constexpr int kAppendThreads = 256;

// Value of an e4m3 code (in the low byte): e4m3's exponent bias is 7 and bf16's 127, so the
// code's bits moved to a bf16's places read as value * 2^-120 (subnormals too).
__device__ __forceinline__ float e4m3_float(uint32_t c) {
    const uint32_t m = c & 0x7fu;
    const float v = __uint_as_float(((c & 0x80u) << 24) | (m << 20)) * 0x1p120f;
    return m == 0x7fu ? __uint_as_float(0x7fc00000u) : v;
}

__device__ __forceinline__ uint2 encode8(const float (&y)[8]) {
    return make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
}

// bf16 magnitudes order like the integers of their 15 bits; 0x7f80 and up are not finite.
constexpr uint32_t kNotFinite = 0x7f80u;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The larger magnitudes of two words' halves, as bits.
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint32_t u) {
    return max_u16x2(m, u & 0x7fff7fffu);
}
// The same without what is not finite.
__device__ __forceinline__ uint32_t max_finite_bits(uint32_t m, uint32_t u) {
    const uint32_t a = u & 0x7fffu, b = (u >> 16) & 0x7fffu;
    return max_u16x2(m, (a < kNotFinite ? a : 0u) | (b < kNotFinite ? b : 0u) << 16);
}

// The least power of two s >= 2^-126 with amax <= 448 s: amax = m 2^e, 448 = 1.75 * 2^8,
// so s = 2^(e - 8) where m <= 1.75 (mantissa 0x60 of 7 bits) and 2^(e - 7) above.
__device__ __forceinline__ float least_scale(uint32_t amax) {
    const int e = (int)(amax >> 7) - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0);  // biased by 127
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// A scale that was there, rounded up to a power of two (what this kernel stores is one already).
__device__ __forceinline__ float up_to_pow2(float s) {
    return __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u);
}

template <int D, int W>
__global__ void __launch_bounds__(kAppendThreads, D == 256 ? 2 : D == 96 ? 3 : 4) fa_append_kernel(const AppendParams p) {
    using L = RowLanes<D>;
    constexpr int STEPS = L::STEPS;
    constexpr int TEAMS = kAppendThreads / 32 / W;
    __shared__ uint32_t s_amax[TEAMS][W];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = warp / W, w = warp % W;
    const bool on = lane < L::PER_ROW * L::ROWS;
    const int sub = lane / L::PER_ROW, col = lane % L::PER_ROW * L::E;  // of the rows of a step
    // heads fastest: the CTAs that run together read whole rows of the call
    const int job_ctas = (2 * p.Hkv + TEAMS - 1) / TEAMS;
    const int job = (int)(blockIdx.x % job_ctas) * TEAMS + team;  // 2 h: keys of head h, 2 h + 1: values
    if (job >= 2 * p.Hkv) return;
    const int h = job >> 1;
    const __nv_bfloat16 *x =
        reinterpret_cast<const __nv_bfloat16 *>(job & 1 ? p.v : p.k) + (size_t)h * D + col;
    const long long stride = job & 1 ? p.v_stride : p.k_stride;
    uint8_t *cache = (job & 1 ? p.v_cache : p.k_cache) + col;
    float *scales = job & 1 ? p.v_scale : p.k_scale;
    const bool reports = job == 0 && w == 0 && lane == 0;
    const int G = p.group, ps = p.page_size, groups = ps / G;

    int t = (int)(blockIdx.x / job_ctas) * p.window;
    const int t_end = (int)min((long long)p.T, (long long)t + p.window);
    int b;
    if (p.cu_seqlens == nullptr) {
        b = t;
    } else {
        // the last b with cu[b] <= t (0 if there is none) among every 32nd, by steps of 32
        // pivots; the walk finds it among the 32 from there, which it holds in registers.  An
        // offset outside 0 .. T never counts, so the walk may begin early but not late.
        int lo = 0, n = (p.B + 31) / 32;
        while (n > 1) {
            const int step = (n + 31) / 32;
            const int i = lane * step;
            const int c = i < n ? p.cu_seqlens[(lo + i) * 32] : -1;
            const unsigned m = __ballot_sync(kFull, c >= 0 && c <= t);
            const int k = m ? 31 - __clz(m) : 0;
            lo += k * step;
            n = min(step, n - k * step);
        }
        b = lo * 32;
        if (blockIdx.x == 0 && job == 0 && w == 0) {
            bool ok = true;  // the offsets, checked once per call
            for (int i = lane; i < p.B; i += 32) {
                const int c0 = p.cu_seqlens[i], c1 = p.cu_seqlens[i + 1];
                ok = ok && c0 >= 0 && c0 <= c1 && c1 <= p.T;
            }
            if (!__all_sync(kFull, ok) && lane == 0) flag_index(p.status, SITE_APPEND_BAD_SEQ);
        }
    }
    // lane i holds the offsets and length of sequence held + i
    int held = b, my_c0 = 0, my_c1 = 0, my_len = 0;
    auto hold = [&] {
        held = b;
        const int i = b + lane;
        if (i < p.B) {
            my_c0 = p.cu_seqlens ? p.cu_seqlens[i] : i;
            my_c1 = p.cu_seqlens ? p.cu_seqlens[i + 1] : i + 1;
            my_len = p.seq_lens[i];
        }
    };
    hold();
    if (p.cu_seqlens) {
        const unsigned m = __ballot_sync(kFull, b + lane < p.B && my_c0 >= 0 && my_c0 <= t);
        if (m) b += 31 - __clz(m);
    }
    // Walk the groups that begin at rows t .. t_end - 1 (all values are uniform over the team).
    while (t < t_end && b < p.B) {
        if (b - held >= 32) hold();
        const int c0 = __shfl_sync(kFull, my_c0, b - held), c1 = __shfl_sync(kFull, my_c1, b - held);
        const int start = __shfl_sync(kFull, my_len, b - held);
        // an empty sequence, the end of this one, or one with a bad offset
        if (t >= c1 || c0 < 0 || c0 > c1 || c1 > p.T) {
            ++b;
            continue;
        }
        if (t < c0) {  // rows before the first sequence
            t = c0;
            continue;
        }
        const long long room = (long long)ps * p.max_pages;
        if (start < 0 || start + (long long)(c1 - c0) > room) {
            if (reports) flag_index(p.status, SITE_APPEND_BAD_SEQ);
            t = c1;
            continue;
        }
        const int pos = start + (t - c0);
        const int in_group = pos % G;
        const int cnt = min(G - in_group, c1 - t);  // rows of this group from t on
        if (t != c0 && in_group != 0) {             // begun in an earlier window
            t += cnt;
            continue;
        }
        const int page = p.block_table[(size_t)b * p.max_pages + pos / ps];
        const int g = pos % ps / G;
        // step i: rows row(i) of the new ones, loaded while the page number is on its way
        auto row = [&](int i) { return (i * W + w) * L::ROWS + sub; };
        uint4 u[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            u[i] = row(i) < cnt && on ? *reinterpret_cast<const uint4 *>(x + (t + row(i)) * stride)
                                      : make_uint4(0u, 0u, 0u, 0u);
        if (page < 0 || page >= p.num_pages) {
            if (reports) flag_index(p.status, SITE_APPEND_BAD_PAGE);
            t += cnt;
            continue;
        }
        const size_t ph = (size_t)page * p.Hkv + h;
        float *sc = scales + ph * groups + g;
        uint8_t *rows = cache + (ph * ps + (size_t)g * G) * D;  // of the group
        const float old = in_group ? *sc : 0.f;
        // the team's largest of a word's halves
        auto team_max = [&](uint32_t m) {
            m = __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16));
            if constexpr (W > 1) {
                if (lane == 0) s_amax[team][w] = m;
                named_barrier_sync(1 + team, 32 * W);
#pragma unroll
                for (int i = 0; i < W; ++i) m = max(m, s_amax[team][i]);
                named_barrier_sync(1 + team, 32 * W);  // everyone has read before it is written again
            }
            return m;
        };
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            m = max_bits(max_bits(m, u[i].x), u[i].y);
            m = max_bits(max_bits(m, u[i].z), u[i].w);
        }
        uint32_t amax = team_max(m);
        const bool odd = amax >= kNotFinite;
        if (odd) {  // something is not finite: the largest of the rest
            m = 0;
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                m = max_finite_bits(max_finite_bits(m, u[i].x), u[i].y);
                m = max_finite_bits(max_finite_bits(m, u[i].z), u[i].w);
            }
            amax = team_max(m);
        }
        const float s = fmaxf(least_scale(amax), up_to_pow2(old));
        if (in_group && s > old) {  // the codes that were there, at the larger scale
            const float ratio = old / s;
            for (int r = w * L::ROWS + sub; r < in_group; r += W * L::ROWS) {
                if (on) {
                    const uint2 c = *reinterpret_cast<const uint2 *>(rows + (size_t)r * D);
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = e4m3_float((e < 4 ? c.x : c.y) >> (8 * (e % 4))) * ratio;
                    *reinterpret_cast<uint2 *>(rows + (size_t)r * D) = encode8(y);
                }
            }
        }
        const uint64_t inv = f32x2_splat(1.f / s);  // exact, and so are the products
        uint8_t *out = rows + (size_t)in_group * D;
        auto put = [&](auto fix) {
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                if (row(i) < cnt && on) {
                    const uint32_t v[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[2 * e] = __uint_as_float(v[e] << 16);
                        y[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
                        mul_f32x2(y[2 * e], y[2 * e + 1], inv);
                    }
                    uint2 c = encode8(y);
                    if constexpr (decltype(fix)::value) {  // an infinity is stored as NaN
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            uint32_t &word = e < 4 ? c.x : c.y;
                            const int at = 8 * (e % 4);
                            if (!(fabsf(y[e]) < INFINITY)) word = (word & ~(0xffu << at)) | 0x7fu << at;
                        }
                    }
                    *reinterpret_cast<uint2 *>(out + (size_t)row(i) * D) = c;
                }
            }
        };
        if (odd) put(std::true_type());
        else put(std::false_type());
        if (w == 0 && lane == 0) *sc = s;
        t += cnt;
    }
}

template <int D, int W>
int launch_append_t(const AppendParams &p, cudaStream_t stream) {
    constexpr int TEAMS = kAppendThreads / 32 / W;
    const long long ctas = (2LL * p.Hkv + TEAMS - 1) / TEAMS * ((p.T - 1LL) / p.window + 1);
    if (ctas >= (1LL << 31)) return FA_ERR_INVALID_ARG;
    return launch_dependent(fa_append_kernel<D, W>, (unsigned)ctas, kAppendThreads, 0, stream, 1, p);
}

template <int D>
int launch_append_d(const AppendParams &p, cudaStream_t stream) {
    if (p.group <= 16) return launch_append_t<D, 1>(p, stream);
    if (p.group <= 32) return launch_append_t<D, 2>(p, stream);
    if (p.group <= 64) return launch_append_t<D, 4>(p, stream);
    return launch_append_t<D, 8>(p, stream);
}

// ------------------------------------------------------------- page bookkeeping
//
// Which pages are in use is a bitmap, and a page's new number a rank in it, so one cluster
// of CTAs does the whole plan in one launch with the bitmap in its shared memory: mark the
// pages of the table (atomics on the owner's words through distributed shared memory),
// count the bits of the words before each word, then write the lists.  A launch that is
// bound by latency: barriers and two passes over the table.  A small table is done sooner by
// one CTA, whose barriers are local (kOneCta below).  Measured (graph replay): the compaction
// plan of 12 x 20 entries and 300 pages 3.8 us (one CTA; 7.1 us as a cluster), of 192 x 63 and
// 23000 pages 11.3 us (cluster; 18.7 us in one CTA), against 200 us of copies.

constexpr int kPlanThreads = 1024;

template <int CTAS>
struct Bitmap {
    cg::cluster_group cluster;
    uint32_t *words, *before;  // this CTA's part: bits, and bits set before the word (globally)
    int per_cta;               // words per CTA

    __device__ void sync() {
        if constexpr (CTAS > 1) cluster.sync();
        else __syncthreads();
    }
    __device__ uint32_t *at(uint32_t *base, int word) {
        if constexpr (CTAS == 1) return base + word;
        else return cluster.map_shared_rank(base, word / per_cta) + word % per_cta;
    }
    __device__ void set(int page) { atomicOr(at(words, page >> 5), 1u << (page & 31)); }
    // pages in use below `page`
    __device__ int rank(int page) {
        const int w = page >> 5;
        return (int)*at(before, w) + __popc(*at(words, w) & ((1u << (page & 31)) - 1u));
    }
};

// Table entries (and four per word of the bitmap) up to which one CTA does the plan.
constexpr long long kOneCta = 5000;

// Entries of a table row that are in use.
__device__ __forceinline__ int used_entries(int len, int page_size, int max_pages, bool *bad) {
    const int need = len <= 0 ? 0 : (int)((uint32_t)(len - 1) / (uint32_t)page_size) + 1;
    *bad = len < 0 || need > max_pages;
    return min(need, max_pages);
}

template <int CTAS>
__global__ void __launch_bounds__(kPlanThreads) fa_pages_kernel(const PagesParams p, int per_cta) {
    extern __shared__ uint32_t plan_smem[];
    __shared__ int s_total, s_warp[kPlanThreads / 32];
    Bitmap<CTAS> bm{cg::this_cluster(), plan_smem, plan_smem + per_cta, per_cta};
    const int rank = CTAS > 1 ? (int)bm.cluster.block_rank() : 0;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t entries = (uint32_t)p.B * (uint32_t)p.max_pages;  // below 2^31
    const uint32_t first = (uint32_t)rank * kPlanThreads + tid;
    constexpr uint32_t kStep = CTAS * kPlanThreads;
    constexpr int U = 4;  // entries whose loads a thread has in flight

    for (int i = tid; i < per_cta; i += kPlanThreads) bm.words[i] = 0u;
    griddep_wait();
    griddep_launch_dependents();
    bm.sync();
    for (uint32_t i0 = first; i0 < entries; i0 += U * kStep) {
        int page[U];
        bool used[U];
#pragma unroll
        for (int v = 0; v < U; ++v) {
            const uint32_t i = i0 + v * kStep;
            used[v] = false;
            page[v] = 0;
            if (i >= entries) continue;
            const int b = (int)(i / (uint32_t)p.max_pages), col = (int)(i - (uint32_t)b * p.max_pages);
            bool bad;
            used[v] = col < used_entries(p.seq_lens[b], p.page_size, p.max_pages, &bad);
            if (bad && col == 0) flag_index(p.status, SITE_PAGES_BAD_LEN);
            page[v] = p.block_table[i];
        }
#pragma unroll
        for (int v = 0; v < U; ++v) {
            if (!used[v]) continue;
            if (page[v] >= 0 && page[v] < p.num_pages) bm.set(page[v]);
            else flag_index(p.status, SITE_PAGES_BAD_PAGE);
        }
    }
    bm.sync();

    // bits before each word: a thread's run of words, then the CTA's threads, then the CTAs
    const int run = (per_cta + kPlanThreads - 1) / kPlanThreads;
    const int w0 = min(tid * run, per_cta), w1 = min(w0 + run, per_cta);
    int mine = 0;
    for (int i = w0; i < w1; ++i) mine += __popc(bm.words[i]);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int v = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, v, o);
            if (lane >= o) v += y;
        }
        s_warp[lane] = v;
        if (lane == 31) s_total = v;
    }
    bm.sync();
    int base = incl - mine + (warp > 0 ? s_warp[warp - 1] : 0);
    int n_live = s_total;
    if constexpr (CTAS > 1) {
        n_live = 0;
        for (int r = 0; r < CTAS; ++r) {
            const int tot = *bm.cluster.map_shared_rank(&s_total, r);
            if (r < rank) base += tot;
            n_live += tot;
        }
    }
    for (int i = w0; i < w1; ++i) {
        bm.before[i] = (uint32_t)base;
        base += __popc(bm.words[i]);
    }
    bm.sync();

    if (p.pages) {
        const int n_free = p.num_pages - n_live;
        for (int i = warp; i < per_cta; i += kPlanThreads / 32) {
            const int page = (rank * per_cta + i) * 32 + lane;
            const uint32_t bits = bm.words[i];
            if (page < p.num_pages && !((bits >> lane) & 1u))
                p.pages[page - (int)bm.before[i] - __popc(bits & ((1u << lane) - 1u))] = page;
        }
        for (uint32_t i = n_free + first; i < (uint32_t)p.num_pages; i += kStep) p.pages[i] = -1;
        if (first == 0) p.counts[0] = n_free;
    } else {
        const int below = n_live < p.num_pages ? bm.rank(n_live) : n_live;
        const int moves = n_live - below;  // pages in use from n_live on = unused ones below it
        for (int i = warp; i < per_cta; i += kPlanThreads / 32) {
            const int page = (rank * per_cta + i) * 32 + lane;
            const uint32_t bits = bm.words[i];
            const bool in_use = (bits >> lane) & 1u;
            const int r = (int)bm.before[i] + __popc(bits & ((1u << lane) - 1u));
            if (page < n_live && !in_use) p.dst[page - r] = page;
            if (page >= n_live && page < p.num_pages && in_use) p.src[r - below] = page;
        }
        for (uint32_t i = moves + first; i < (uint32_t)p.cap; i += kStep) p.src[i] = p.dst[i] = -1;
        if (first == 0) {
            p.counts[0] = n_live;
            p.counts[1] = moves;
        }
        bm.sync();  // dst is complete
        for (uint32_t i0 = first; i0 < entries; i0 += U * kStep) {
            int page[U];
            bool moved[U];
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const uint32_t i = i0 + v * kStep;
                moved[v] = false;
                page[v] = 0;
                if (i >= entries) continue;
                const int b = (int)(i / (uint32_t)p.max_pages), col = (int)(i - (uint32_t)b * p.max_pages);
                bool bad;
                page[v] = p.block_table[i];
                moved[v] = col < used_entries(p.seq_lens[b], p.page_size, p.max_pages, &bad) &&
                           page[v] >= n_live && page[v] < p.num_pages;
            }
#pragma unroll
            for (int v = 0; v < U; ++v)
                if (moved[v]) page[v] = __ldcg(p.dst + (bm.rank(page[v]) - below));
#pragma unroll
            for (int v = 0; v < U; ++v)
                if (i0 + v * kStep < entries) p.new_table[i0 + v * kStep] = page[v];
        }
    }
    if constexpr (CTAS > 1) bm.sync();  // nobody reads this CTA's words any more
}

// One CTA per child.
__global__ void __launch_bounds__(128) fa_fork_kernel(const ForkParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int i = blockIdx.x;
    const int parent = p.parents[i];
    const bool known = parent >= 0 && parent < p.B;
    int need = 0, len = 0;
    if (known) {
        len = p.seq_lens[parent];
        bool bad;
        need = used_entries(len, p.page_size, p.max_pages, &bad);
        if (bad) {
            if (threadIdx.x == 0) flag_index(p.status, SITE_PAGES_BAD_LEN);
            len = len < 0 ? 0 : p.page_size * p.max_pages;
        }
    } else if (threadIdx.x == 0) {
        flag_index(p.status, SITE_PAGES_BAD_LEN);
    }
    const bool partial = need > 0 && len % p.page_size != 0;
    const int *from = p.block_table + (size_t)(known ? parent : 0) * p.max_pages;
    int *row = p.rows + (size_t)i * p.max_pages;
    for (int c = threadIdx.x; c < p.max_pages; c += blockDim.x) {
        int page = c < need ? from[c] : -1;
        if (c < need && (page < 0 || page >= p.num_pages)) {
            flag_index(p.status, SITE_PAGES_BAD_PAGE);
            page = -1;
        }
        if (partial && c == need - 1) {
            int to = p.fresh[i];
            if (to < 0 || to >= p.num_pages) {
                flag_index(p.status, SITE_PAGES_BAD_PAGE);
                to = -1;
            }
            p.src[i] = to < 0 ? -1 : page;
            p.dst[i] = page < 0 ? -1 : to;
            page = to;
        }
        row[c] = page;
    }
    if (threadIdx.x == 0) {
        p.lens[i] = len;
        if (!partial) p.src[i] = p.dst[i] = -1;
    }
}

// ---------------------------------------------------------------------- copies
//
// A copy is bound by HBM: 2 bytes of traffic per byte.  A page of all buffers is cut into
// units of 4 KB, one warp each (8 independent 16-byte loads per lane in flight); the small
// pages of the scales are units of their own.  Warps stride over the units, so one launch of
// resident CTAs serves any number of pairs, with their number on the device if it must be.
// Measured (GB300): 2500 pages of 4 layers, 1.3 GB of traffic, 200 us, 6.5 TB/s; 128 pages of
// 8 layers, 0.26 GB, 39 us, 6.8 TB/s.

constexpr int kCopyUnit = 4096;
constexpr int kCopyThreads = 256;

template <typename T>
__device__ __forceinline__ void copy_unit(const uint8_t *s, uint8_t *d, int bytes, int lane) {
    constexpr int N = 8;
    const T *a = reinterpret_cast<const T *>(s);
    T *b = reinterpret_cast<T *>(d);
    const int n = bytes / (int)sizeof(T);
    for (int i = lane; i < n; i += 32 * N) {
        T r[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (i + 32 * k < n) r[k] = a[i + 32 * k];
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (i + 32 * k < n) b[i + 32 * k] = r[k];
    }
}

__global__ void __launch_bounds__(kCopyThreads) fa_copy_pages_kernel(const __grid_constant__ CopyParams p) {
    const int lane = threadIdx.x & 31;
    const int per_pair = p.first_unit[p.n_caches];
    griddep_wait();
    griddep_launch_dependents();
    int n = p.n_pairs;
    if (p.count) n = max(0, min(n, *p.count));
    const long long units = (long long)n * per_pair;
    const long long step = (long long)gridDim.x * (kCopyThreads / 32);
    for (long long u = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units;
         u += step) {
        const int pair = (int)(u / per_pair), k = (int)(u % per_pair);
        const int from = p.src[pair];
        if (from == -1) continue;
        const int to = p.dst[pair];
        if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
            if (lane == 0) flag_index(p.status, SITE_COPY_BAD_PAGE);
            continue;
        }
        int lo = 0, hi = p.n_caches;  // the buffer of unit k: the last with first_unit <= k
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (p.first_unit[mid] <= k) lo = mid;
            else hi = mid;
        }
        const unsigned long long pb = p.page_bytes[lo];
        const unsigned long long off = (unsigned long long)(k - p.first_unit[lo]) * kCopyUnit;
        const int bytes = (int)min((unsigned long long)kCopyUnit, pb - off);
        uint8_t *base = static_cast<uint8_t *>(p.cache[lo]);
        const uint8_t *s = base + (unsigned long long)from * pb + off;
        uint8_t *d = base + (unsigned long long)to * pb + off;
        const unsigned long long align = reinterpret_cast<uintptr_t>(base) | pb;
        if ((align & 15) == 0) copy_unit<uint4>(s, d, bytes, lane);
        else if ((align & 3) == 0) copy_unit<uint32_t>(s, d, bytes, lane);
        else copy_unit<uint8_t>(s, d, bytes, lane);
    }
}

}  // namespace

int launch_append(const AppendParams &p, cudaStream_t stream) {
    switch (p.d) {
        case 64: return launch_append_d<64>(p, stream);
        case 96: return launch_append_d<96>(p, stream);
        case 128: return launch_append_d<128>(p, stream);
        case 256: return launch_append_d<256>(p, stream);
        default: return FA_ERR_UNSUPPORTED;
    }
}

int launch_pages(const PagesParams &p, cudaStream_t stream) {
    const int words = (p.num_pages + 31) / 32;
    const bool one = (long long)p.B * p.max_pages + 4LL * words <= kOneCta;
    const int ctas = one ? 1 : 8;
    const int per_cta = (words + ctas - 1) / ctas;
    auto kern = one ? fa_pages_kernel<1> : fa_pages_kernel<8>;
    const int smem = per_cta * 8;
    if (ensure_smem_attr(reinterpret_cast<const void *>(kern), smem) != FA_OK) return FA_ERR_CUDA;
    return launch_dependent(kern, (unsigned)ctas, kPlanThreads, (size_t)smem, stream, ctas, p, per_cta);
}

int launch_fork(const ForkParams &p, cudaStream_t stream) {
    return launch_dependent(fa_fork_kernel, (unsigned)p.n, 128, 0, stream, 1, p);
}

int launch_copy(CopyParams &p, cudaStream_t stream) {
    long long per_pair = 0;
    for (int c = 0; c < p.n_caches; ++c) {
        p.first_unit[c] = (int)per_pair;
        per_pair += (long long)((p.page_bytes[c] + kCopyUnit - 1) / kCopyUnit);
        if (per_pair >= (1LL << 31)) return FA_ERR_INVALID_ARG;
    }
    p.first_unit[p.n_caches] = (int)per_pair;
    constexpr int kWarps = kCopyThreads / 32;
    const long long units = per_pair * p.n_pairs;
    const long long most = (long long)p.num_sms * (2048 / kCopyThreads);
    const long long ctas = (units + kWarps - 1) / kWarps;
    return launch_dependent(fa_copy_pages_kernel, (unsigned)(ctas < most ? ctas : most), kCopyThreads, 0,
                            stream, 1, p);
}

}  // namespace fa
