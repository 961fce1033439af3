// Decode attention against a paged e4m3 cache (definition in fa.h).
//
// One CTA per query row: its warps take keys in turn, a lane holds E elements of a key, and
// each warp keeps its own running (max, sum, output), merged at the end.
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kWarps = 4;

__device__ __forceinline__ float e4m3_value(uint32_t c) {
    const uint32_t m = c & 0x7fu;
    const float v = __uint_as_float(((c & 0x80u) << 24) | (m << 20)) * 0x1p120f;
    return m == 0x7fu ? __uint_as_float(0x7fc00000u) : v;
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) fa_decode8_kernel(const Decode8Params p) {
    constexpr int E = (D == 96) ? 4 : D / 32, LANES = D / E;
    __shared__ float s_o[kWarps][D], s_m[kWarps], s_l[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool on = lane < LANES;
    const long long row = blockIdx.x;
    const int i = (int)(row % p.Nq), h = (int)(row / p.Nq % p.H), b = (int)(row / p.Nq / p.H);
    const int kvh = h / (p.H / p.Hkv);
    const int len = p.seq_lens[b], ps = p.page_size, groups = ps / p.group;
    if (len < 0 || len > (long long)ps * p.max_pages) {
        if (threadIdx.x == 0) {
            atomicCAS(p.status + 1, 0, SITE_DEC8_BAD_LEN);
            atomicExch(p.status, FA_ERR_BAD_INDEX);
        }
        return;
    }
    const int end = p.causal ? min(len, len - p.Nq + 1 + i) : len;
    const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(p.q) + row * D;
    float qv[E], acc[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
        qv[e] = on ? __bfloat162float(q[lane * E + e]) : 0.f;
        acc[e] = 0.f;
    }
    bool ok = true;
    for (int j = warp; j < end && ok; j += kWarps) {
        const int page = p.block_table[(size_t)b * p.max_pages + j / ps];
        if (page < 0 || page >= p.num_pages) {
            ok = false;
            break;
        }
        const size_t ph = (size_t)page * p.Hkv + kvh;
        const size_t at = (ph * ps + j % ps) * D + lane * E, sat = ph * groups + j % ps / p.group;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += on ? qv[e] * e4m3_value(p.k[at + e]) : 0.f;
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        s *= p.k_scale[sat] * p.scale_log2;
        const float mn = fmaxf(m, s), a = ex2(m - mn), w = ex2(s - mn), wv = w * p.v_scale[sat];
        m = mn;
        l = l * a + w;
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + (on ? wv * e4m3_value(p.v[at + e]) : 0.f);
    }
    if (on)
        for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
    s_m[warp] = m;
    s_l[warp] = l;
    if (!__syncthreads_and(ok)) {
        if (threadIdx.x == 0) {
            atomicCAS(p.status + 1, 0, SITE_DEC8_BAD_PAGE);
            atomicExch(p.status, FA_ERR_BAD_INDEX);
        }
        return;
    }
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    for (int w = 0; w < kWarps; ++w) L += s_m[w] == -INFINITY ? s_l[w] : s_l[w] * ex2(s_m[w] - M);
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        float o = 0.f;
        for (int w = 0; w < kWarps; ++w) o += s_m[w] == -INFINITY ? s_o[w][c] : s_o[w][c] * ex2(s_m[w] - M);
        reinterpret_cast<__nv_bfloat16 *>(p.o)[row * D + c] = __float2bfloat16(end > 0 ? o / L : 0.f);
    }
    if (threadIdx.x == 0) p.lse[row] = end > 0 ? (M + lg2(L)) * kLn2 : -INFINITY;
}

template <int D>
int launch_t(const Decode8Params &p, cudaStream_t stream) {
    fa_decode8_kernel<D><<<(unsigned)((long long)p.B * p.H * p.Nq), 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

int launch_decode8(const Decode8Params &p, cudaStream_t stream) {
    switch (p.d) {
        case 64: return launch_t<64>(p, stream);
        case 96: return launch_t<96>(p, stream);
        case 128: return launch_t<128>(p, stream);
        case 256: return launch_t<256>(p, stream);
        default: return FA_ERR_UNSUPPORTED;
    }
}

}  // namespace fa
