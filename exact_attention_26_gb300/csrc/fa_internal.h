// Declarations shared by the host API and the kernel translation units.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa.h"

namespace fa {

// Where a bounded wait gave up (second word of the device status record).
enum WaitSite : int {
    SITE_NONE = 0,
    SITE_FWD_LOAD_KV_EMPTY = 1,
    SITE_FWD_MMA_Q = 2,
    SITE_FWD_MMA_KV_FULL = 3,
    SITE_FWD_MMA_P_FULL = 4,
    SITE_FWD_SOFTMAX_S_FULL = 5,
    SITE_FWD_EPILOGUE_O_FULL = 6,
    SITE_FWD_DRAIN = 7,
    SITE_FWD_BAD_SEQ = 8,
    SITE_BWD_LOAD_EMPTY = 11,
    SITE_BWD_MMA_KV = 12,
    SITE_BWD_MMA_Q_FULL = 13,
    SITE_BWD_MMA_DS_FULL = 14,
    SITE_BWD_MMA_DQ_FREE = 15,
    SITE_BWD_SOFTMAX_S_FULL = 16,
    SITE_BWD_DQ_FULL = 17,
    SITE_BWD_EPILOGUE = 18,
    SITE_BWD_DRAIN = 19,
    SITE_BWD_BAD_SEQ = 20,
    SITE_BWD_SMEM_ALIGN = 26,
    SITE_FWD_SMEM_ALIGN = 27,
    SITE_DEC_FULL = 21,
    SITE_DEC_EMPTY = 22,
    SITE_DEC_DRAIN = 23,
    SITE_DEC_BAD_LEN = 24,
    SITE_DEC_BAD_PAGE = 25,
    SITE_DEC_MMA = 28,
    SITE_BWD_ITEM = 29,
    SITE_SELFTEST = 30,
    SITE_APPEND_BAD_SEQ = 31,
    SITE_APPEND_BAD_PAGE = 32,
    SITE_PAGES_BAD_LEN = 33,
    SITE_PAGES_BAD_PAGE = 34,
    SITE_COPY_BAD_PAGE = 35,
    SITE_DEC8_BAD_LEN = 36,
    SITE_DEC8_BAD_PAGE = 37,
    SITE_TREE_BAD_LEN = 38,
    SITE_TREE_BAD_PAGE = 39,
    SITE_TREE_BAD_PARENT = 40,
    SITE_VERIFY_BAD_TREE = 41,
    SITE_KEEP_BAD_PATH = 42,
};

// Default limit of one in-kernel wait.
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

struct FwdSegPlan;

struct FwdParams {
    CUtensorMap tm_q, tm_k, tm_v;  // 3-D maps over [BH][N][d] (q) and [B*Hkv][N][d] (k, v) bf16
    void *o;                       // bf16 [BH][N][d]
    float *lse;                    // fp32 [BH][N]
    int N, BH, d, causal;
    int H, group;                  // query heads per batch; query heads per key/value head
    const int *cu_seqlens;         // varlen: [B+1] sequence starts (token-major layout), else null
    int total_tokens;              // varlen: T
    float scale_log2;              // scale * log2(e)
    int fp8;                       // e4m3 inputs: tm_q/tm_k over bytes, tm_v over V^T [B*Hkv][d][Np]
    const float *q_descale, *k_descale, *v_descale;  // fp8: [BH][nqb], [B*Hkv][nqb], [B*Hkv]
    int kv_chunk;                  // > 0: key ranges cut into chunks of this many K/V tiles
    const FwdSegPlan *seg;         // non-null: key ranges cut by this balanced plan
    float *ws_o, *ws_l;            // kv_chunk > 0: partial O [BH][N][s_max][d], L [BH][N][s_max]
    int s_max;                     // chunks of the longest key range
    int *status;                   // device status record (2 ints)
    unsigned long long limit_ns;
    int num_sms;
};

// Key-range chunk in K/V tiles of the one-tile forward for B*H heads of N rows
// (0: no cut); `forced` > 0 asks for that many tiles (rounded up to the tiles of a
// row block on the diagonal).
int fwd_split_chunk(int d, int BH, int N, int causal, int num_sms, int forced);

// Balanced cut of the one-tile forward's key ranges: the row blocks, longest first,
// are laid end to end and cut into segments (a row block's K/V tiles
// [kv_lo, kv_lo + n)) so that every CTA's run of consecutive segments costs about
// the same (its tiles plus a fixed cost per segment); the kernel reads its run from
// the table and the merge kernel the segment count of each row block.
constexpr int kSegMaxCta = 256, kSegMax = 640, kSegMaxRows = 256, kSegMaxParts = 15;
struct FwdSegTable {
    int n_cta, max_per_cta;           // CTAs of the launch; segments of the busiest
    uint16_t start[kSegMaxCta + 1];   // CTA c runs segments [start[c], start[c + 1])
    uint32_t seg[kSegMax][2];         // bh | cb << 16;  kv_lo | n << 12 | s << 24 | ns << 28
};
struct FwdMergeNs {
    uint8_t ns[kSegMaxRows];          // segments of row block bh * n_cb + cb
};
struct FwdSegPlan {
    FwdSegTable tab;
    FwdMergeNs mns;
    int n_seg, s_max;                 // segments; most segments of one row block
    double cost;                      // predicted K/V-tile steps, merge included
};
// The balanced plan for B*H heads of N rows, or null when the library does not cut
// this way (the cut is not predicted 5% faster than no cut and faster than even
// chunks).  Plans are remembered per shape; the pointer stays valid.
const FwdSegPlan *fwd_seg_plan(int d, int BH, int N, int causal, int num_sms);
// Rows per TMA box of the forward's K and V tensor maps (the kernel loads a K/V
// tile of BN keys as BN / box boxes).
constexpr int fwd_kv_box_rows(int d) { return d == 256 ? 64 : 128; }

// e4m3 block quantiser: x bf16 [BH][N][d] -> codes [BH][N][d] (or [BH][d][Np]).
struct QuantParams {
    const void *x;
    void *codes;
    float *descale;        // [BH][n_groups]
    float *partial;        // workspace: per 128-row chunk maxima, [BH][n_chunks]
    const float *signs;    // incoherent processing: d signs (+-1), or null
    int BH, N, d, block_rows, transpose, Np;
};

int launch_quant(const QuantParams &p, cudaStream_t stream);

// Query rows per backward block of the kernel that serves head dim d (the box
// height of the q and dO tensor maps).
int bwd_block_q(int d);

struct BwdParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_do;  // 3-D maps over [BH][N][d] (q, do), [B*Hkv][N][d] (k, v)
    CUtensorMap tm_dq;                    // fp32 dq: (d, N, BH) box (32, 32, 1), or packed
                                          // (d, heads, T) box (32, 1, 32); tiled bulk adds
    const void *o, *dout;                 // bf16 [BH][N][d]
    const float *lse;                     // fp32 [BH][N]
    float *dq, *dk, *dv;                  // fp32 [BH][N][d]
    float *ws_delta, *ws_lse2;            // workspace, [BH][Npad] each
    int *ws_counter;                      // workspace: the main kernel's next unclaimed item
    int N, Npad, BH, d, causal;
    int H, group;                         // query heads per batch; query heads per k/v head
    const int *cu_seqlens;                // varlen: [B+1] sequence starts (token-major), else null
    int total_tokens;                     // varlen: T
    float scale, scale_log2;
    int *status;
    unsigned long long limit_ns;
    int num_sms;
};

// Query rows per backward q-block and the padding unit of the workspace vectors.
constexpr int kBwdPad = 128;
// Bytes at the end of the backward workspace for the work-item counter.
constexpr size_t kBwdCounterBytes = 16;

struct DecodeParams {
    // tensor-core path only: q as [1][BH*Nq][d] (boxes of 128 rows), k and v as
    // [B*Hkv][Nk][d] (boxes of 64 keys)
    CUtensorMap tm_q, tm_k, tm_v;
    const void *q;            // bf16 [BH][Nq][d]
    const void *k, *v;        // bf16 [B*Hkv][Nk][d], or paged [num_pages][Hkv][page_size][d]
    void *o;                  // bf16 [BH][Nq][d]
    float *lse;               // fp32 [BH][Nq]
    float *part_o, *part_l;   // workspace when S > 1: [B*Hkv][S][group*Nq][d], [..][S][group*Nq]
    const int *block_table;   // paged: [B][max_pages] physical page of each logical page
    const int *seq_lens;      // paged: [B] cached tokens of each sequence
    int BH, H, Nq, Nk, d;     // Nk: keys per head (paged: page_size * max_pages, an upper bound)
    int Hkv, group;           // key/value heads; query heads per key/value head (H = Hkv*group)
    int S, keys_per_split;    // key ranges [s*keys_per_split, ...) per CTA
    int paged, page_size, max_pages, num_pages;
    float scale_log2;
    int *status;
    unsigned long long limit_ns;
};

// New tokens into the paged e4m3 cache.
struct AppendParams {
    const void *k, *v;               // bf16 rows [T][Hkv][d] at the strides below (elements)
    long long k_stride, v_stride;
    uint8_t *k_cache, *v_cache;      // e4m3 [num_pages][Hkv][page_size][d]
    float *k_scale, *v_scale;        // [num_pages][Hkv][page_size / group]
    const int *block_table, *seq_lens;
    const int *cu_seqlens;           // [B+1], or null: one token each
    int B, T, Hkv, d, page_size, max_pages, num_pages, group;
    int window;                      // consecutive rows a team of warps looks after
    int *status;
};
int launch_append(const AppendParams &p, cudaStream_t stream);

// Page bookkeeping: the listing of unused pages (pages non-null) or the compaction plan.
struct PagesParams {
    const int *block_table, *seq_lens;
    int *pages;                      // free list [num_pages], or null
    int *new_table, *src, *dst;      // compaction: [B][max_pages], [cap], [cap]
    int *counts;                     // free: [1]; compaction: [2]
    int B, max_pages, page_size, num_pages, cap;
    int *status;
};
constexpr int kMaxPlanPages = 1 << 22;
int launch_pages(const PagesParams &p, cudaStream_t stream);

struct ForkParams {
    const int *block_table, *seq_lens, *parents, *fresh;
    int *rows, *lens, *src, *dst;
    int B, n, max_pages, page_size, num_pages;
    int *status;
};
int launch_fork(const ForkParams &p, cudaStream_t stream);

struct CopyParams {
    void *cache[FA_MAX_COPY_CACHES];
    unsigned long long page_bytes[FA_MAX_COPY_CACHES];
    int first_unit[FA_MAX_COPY_CACHES + 1];  // copy units of one pair before cache c
    int n_caches, num_pages, n_pairs;
    const int *src, *dst, *count;
    int *status;
    int num_sms;
};
int launch_copy(CopyParams &p, cudaStream_t stream);  // fills first_unit

// Attention over the paged e4m3 cache.
struct Decode8Params {
    CUtensorMap tm_k, tm_v;          // bytes (pack * d, rows = page_size / pack, num_pages * Hkv)
                                     // with pack = decode8_pack, boxes 128 x decode8_box_rows(rows) x 1
    const void *q;                   // bf16 [B][H][Nq][d]
    const float *k_scale, *v_scale;  // [num_pages][Hkv][page_size / group]
    const int *block_table, *seq_lens;
    void *o;                         // bf16 [B][H][Nq][d]
    float *lse;                      // [B][H][Nq]
    void *workspace;
    int B, H, Hkv, Nq, d, page_size, max_pages, num_pages, group, causal;
    float scale_log2;
    int *status;
    int num_sms;
};
int decode8_pack(const Decode8Params &p);  // keys per row of the tensor maps, of the sizes
int decode8_box_rows(int rows);
// Tiles of 128 keys of all items at the longest possible lengths; the kernels count in ints.
long long decode8_max_tiles(const Decode8Params &p);
size_t decode8_workspace_bytes(const Decode8Params &p);  // of its sizes and num_sms
int launch_decode8(const Decode8Params &p, cudaStream_t stream);

// Attention of drafted tokens over the paged bf16 cache.
struct TreeParams {
    CUtensorMap tm_q, tm_k, tm_v;    // q as one plane of B * H * Nq rows, boxes of tree_query_box rows;
                                     // k, v as num_pages * Hkv planes, boxes of tree_box_rows rows
    const void *v_cache;
    const int *block_table, *seq_lens;
    const int *parents;              // [B][Nt], or null: a chain
    void *o;                         // bf16 [B][H][Nq][d]
    float *lse;                      // [B][H][Nq]
    void *workspace;
    int B, H, Hkv, Nq, Nt, d, page_size, max_pages, num_pages;
    float scale_log2;
    int *status;
    int num_sms;
};
int tree_box_rows(const TreeParams &p);
int tree_query_box(const TreeParams &p);
// Tiles of all items at the longest possible lengths; the kernels count in ints.
long long tree_max_tiles(const TreeParams &p);
size_t tree_workspace_bytes(const TreeParams &p);  // of its sizes and num_sms
int launch_tree(const TreeParams &p, cudaStream_t stream);

// Verification of drafted tokens.
struct VerifyParams {
    const int *tokens, *parents;         // [B][Nt]; parents null: a chain
    const void *target, *draft;          // [B][Nt][V] fp32 or bf16; draft null: drafts are certain
    const float *uniform;                // [B][Nt]
    int *path, *fresh, *count;           // [B][Nt], [B][Nt], [B]
    int B, Nt, V, bf16, replacement;
    int *status;
    int num_sms;
};
int launch_verify(const VerifyParams &v, cudaStream_t stream);

// The accepted tokens' rows of a paged bf16 cache.
struct KeepParams {
    void *cache[FA_MAX_COPY_CACHES];     // bf16 [num_pages][Hkv][page_size][d]
    const int *block_table, *seq_lens, *path, *count;
    int *lens;                           // [B] out
    int n_caches, B, Nt, Hkv, d, page_size, max_pages, num_pages;
    int *status;
    int num_sms;
};
int launch_keep(const KeepParams &k, cudaStream_t stream);

// Devices the per-device caches of the host code cover (ordinals 0..63).
constexpr int kMaxCachedDevices = 64;

// Raise a kernel's dynamic shared memory limit to `bytes` once per (kernel,
// device): the attribute stays with the function in the device's context, so
// later launches skip the driver call.  FA_OK or FA_ERR_CUDA.
int ensure_smem_attr(const void *kernel, int bytes);

// Launch as a programmatic dependent of the stream's previous kernel: the CTAs may start (and
// set up what needs no memory of others) while that kernel ends, and wait for its results with
// griddepcontrol.wait.  Kernels launched this way make that wait before they read or write
// global memory, and let their own dependents start only after it, so a chain of them stays
// ordered: where one runs, all that the stream held before its predecessor is done.  Only for that
// reason may the merges of the paged e4m3 decode and of the trees' attention read seq_lens before
// their wait (the attention kernel that they follow does not write them, and what did is done).
template <typename... P, typename... A>
int launch_dependent(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem,
                     cudaStream_t stream, int cluster, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Registers per thread a kernel is launched with (cached per kernel), or -1.
int kernel_num_regs(const void *kernel);

int launch_fwd(const FwdParams &p, cudaStream_t stream);
int launch_bwd(const BwdParams &p, cudaStream_t stream);
int launch_decode(const DecodeParams &p, cudaStream_t stream);
// Decode with R = (H / Hkv) * Nq query rows per key/value head: whether the
// tensor-core kernel serves it, and the launch shape of the kernel that does.
bool decode_uses_mma(int d, int R, bool paged);
int decode_block_keys(int d, int R, bool paged);   // keys per pipeline stage
int decode_query_block(int d, int R, bool paged);  // query rows per decode CTA
int decode_ctas_per_sm(int d, int R, bool paged);  // resident decode CTAs per SM

}  // namespace fa
