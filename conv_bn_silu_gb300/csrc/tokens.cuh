// tokens.cuh -- declarations shared by the token operators' translation units
// (RMS norm, the paged cache, attention over it, 4-bit products).  Nothing
// here is part of the public ABI (include/cbs.h is).
#pragma once

#include <atomic>

#include "cbs_internal.cuh"
#include "status.cuh"

namespace cbs {

// The paged cache and a call's sequences as the kernels take them.
struct CacheArgs {
    void *k, *v;               // [num_pages][kv_heads][page][head_dim], bf16 or int8
    float *k_scale, *v_scale;  // [num_pages][kv_heads][page] (int8)
    int int8, num_pages, page_shift, kv_heads, head_dim;
    const int *new_start, *seq_lens, *page_table;
    int batch, max_pages, total;
    unsigned int *status;
};

#ifdef __CUDACC__
__device__ __forceinline__ float silu(float z) { return __fdiv_rn(z, 1.0f + expf(-z)); }

// The larger of two magnitudes, or NaN if one is (fmaxf would pass it over).
__device__ __forceinline__ float most_or_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Length of sequence b: what the array says, within what its table can hold.
__device__ __forceinline__ int seq_len(const CacheArgs &a, int b) {
    const int n = a.seq_lens[b];
    const long long cap = (long long)a.max_pages << a.page_shift;
    if (n < 0 || n > cap) {
        atomicOr(a.status, kStatusBadIndex);
        return n < 0 ? 0 : (int)cap;
    }
    return n;
}

// Page that holds position pos of sequence b, or -1 (and the status bit) when
// the table's entry is not a page of the pool.
__device__ __forceinline__ int page_of(const CacheArgs &a, int b, int pos) {
    const int slot = pos >> a.page_shift;
    const int p = slot < a.max_pages ? a.page_table[(size_t)b * a.max_pages + slot] : -1;
    if ((unsigned)p >= (unsigned)a.num_pages) {
        atomicOr(a.status, kStatusBadIndex);
        return -1;
    }
    return p;
}
#endif

struct NormLaunch {
    const void *x, *residual;   // residual nullable
    const float *weight;
    void *h, *y;                // h nullable
    float *scale;               // int8 output
    float eps;
    int rows, cols, in_bf16, out_int8;
};
cudaError_t launch_rmsnorm(const NormLaunch &L, cudaStream_t s);
constexpr int kNormMaxCols = 32768;

cudaError_t launch_dequantize_rows(const int8_t *q, const float *scale, void *out, int rows, int cols, int out_bf16,
                                   cudaStream_t s);

cudaError_t launch_cache_write(const CacheArgs &a, const void *k, long long k_stride, const void *v,
                               long long v_stride, int in_bf16, cudaStream_t s);
cudaError_t launch_cache_read(const CacheArgs &a, int max_len, void *k_out, void *v_out, int out_bf16, cudaStream_t s);

struct EvictLaunch {
    CacheArgs c;
    float *mass;                // [num_pages][kv_heads][page]
    const int *new_table;       // [batch][new_max_pages]
    int new_max_pages, keep, recent;
    int *kept, *new_lens;       // [batch][kv_heads][keep], [batch]
    int ctas;                   // of a cluster (set by the launch)
};
cudaError_t launch_evict(EvictLaunch L, cudaStream_t s);
// Positions of a CTA of eight at most: what its shared memory holds.
constexpr int kEvictRun = 48 * 1024;
constexpr long long kEvictMost = 8ll * kEvictRun;

struct W4Launch {
    const void *x;              // bf16, or int8 codes
    const float *x_scale;       // int8: [rows]
    const uint8_t *w;           // [n][k/2], packed
    const void *scales;         // bf16 [k/group][n]
    const uint8_t *zeros;       // [k/group][n], nullable (8)
    const float *bias;          // [n], nullable
    void *y;
    unsigned int *status;
    int rows, n, k, group, x_int8, out_bf16, act;
};
cbs_status launch_w4(const W4Launch &L, cudaStream_t s);
cudaError_t launch_w4_few(const W4Launch &L, cudaStream_t s);   // up to eight rows
cudaError_t launch_quantize_w4(const float *w, int n, int k, int group, uint8_t *packed, void *scales, cudaStream_t s);

struct W8Launch {
    const int8_t *x, *w;        // [rows][k], [n][k]
    const float *x_scale, *w_scale, *bias;   // [rows], [n], [n] (nullable)
    void *y;
    unsigned int *status;
    int rows, n, k, out_bf16, act;
};
cbs_status launch_w8(const W8Launch &L, cudaStream_t s);
cbs_status launch_w8_pair(const W8Launch &L, cudaStream_t s);    // tiles of 256 rows
cudaError_t launch_w8_few(const W8Launch &L, cudaStream_t s);   // up to sixteen rows
cudaError_t launch_quantize_w8(const float *w, int n, int k, int8_t *codes, float *scales, cudaStream_t s);

struct AttnLaunch {
    CacheArgs c;
    const void *q;              // bf16 [total][heads][head_dim], q_stride elements between tokens
    void *out;
    long long q_stride, out_stride;
    float scale_log2;           // softmax scale * log2(e)
    int group;                  // query heads of a key head
    unsigned int group_magic;   // ceil(2^32 / group): r / group for r group < 2^32 (group > 1)
    int heads, causal, window, max_new;
    int split, row_tiles;
    int cluster;                // few rows: the ranges are CTAs of a cluster
    float *partial;             // [batch][kv_heads][row_tiles][split][rows][head_dim], then (max, sum) of each row
    float2 *stats;
    unsigned int *counters;     // [batch][kv_heads][row_tiles]
    // A shared prefix: batch counts groups in the prefix's part, of `sequences` in all.
    const int *group_start;     // [groups + 1]
    int sequences;
    float *share;               // [total][heads][head_dim], unnormalised, and (max, sum)
    float2 *share_stats;
    // A weighed call: (max, 1 / sum) [total][heads]; the ranges' sums as `stats` lie;
    // scores [batch][kv_heads][rows_pad][len_pad] of the few-row kernels.
    float2 *row_stats;
    float *sums, *scores, *mass;
    int rows_pad, len_pad, fused;   // fused: the few-row kernels sum the weights up themselves
    float decay;
};
// set_max_dyn_smem, once in a context: a call's host time is a small call's whole
// time.  `done`: the kernel's own, the contexts it was set in.
using ContextOfDevice = std::atomic<unsigned long long>[64];
template <typename F>
cudaError_t set_max_dyn_smem_once(F *kern, int bytes, ContextOfDevice &done) {
    int dev = 0;
    unsigned long long ctx = 0;
    const bool known = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 && current_context_id(&ctx) == CBS_OK && ctx;
    if (known && done[dev].load(std::memory_order_relaxed) == ctx) return cudaSuccess;
    const cudaError_t e = set_max_dyn_smem(kern, bytes);
    if (e == cudaSuccess && known) done[dev].store(ctx, std::memory_order_relaxed);
    return e;
}

// The few-row kernels' CTAs an SM: as many as rings and registers fit.  (8 bits, heads of
// 128 at four in place of three, 64 x 1000 keys 30.5 -> 28.9 us, 16 x 4000 34.0 -> 35.0, and
// with tiles of 16 rows at three in place of two 84 -> 73; 64 at six in place of five, 64
// x 8000 keys: 97 -> 104.)
constexpr int attn_rows_ctas(int d, bool int8, int row_tile) {
    return d == 64 ? (int8 && row_tile == 8 ? 5 : 4) : int8 ? (row_tile == 16 ? 3 : 4) : 2;
}
cudaError_t launch_attn_rows(const AttnLaunch &L, int row_tile, cudaStream_t s);
// Tensor-core kernel: tiles of kAttnChunkRows rows.
cbs_status launch_attn_chunk(const AttnLaunch &L, cudaStream_t s);
// The same in the other modes (either kernel, by the plan's row tile), and the
// weights of a weighed call's keys.
cbs_status launch_attn_prefix(const AttnLaunch &L, int row_tile, cudaStream_t s);
cbs_status launch_attn_own(const AttnLaunch &L, int row_tile, cudaStream_t s);
cbs_status launch_attn_beside(const AttnLaunch &L, int row_tile, cudaStream_t s);
cudaError_t launch_join_shares(const AttnLaunch &L, const float *pre, const float2 *pre_stats, cudaStream_t s);   // L's and a prefix's
cbs_status launch_attn_weighed(const AttnLaunch &L, int row_tile, cudaStream_t s);
cbs_status launch_attn_weights(const AttnLaunch &L, cudaStream_t s);
constexpr int kAttnChunkRows = 256, kAttnChunkKeys = 128;
constexpr int kAttnClusterMost = 8;
constexpr int kAttnChunkSplitMost = kAttnClusterMost;   // ranges of keys: CTAs of one cluster

}  // namespace cbs
