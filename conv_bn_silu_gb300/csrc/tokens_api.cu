// tokens_api.cu -- the token operators' C entry points (include/cbs.h):
// argument checks, the attention's planning and dispatch to the kernels.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "tokens.cuh"

namespace cbs {
namespace {

cbs_status need(const void *p, const char *what) {
    if (!p) return fail(CBS_ERR_INVALID_ARG, "%s is NULL", what);
    if (!aligned16(p)) return fail(CBS_ERR_MISALIGNED, "%s is not 16-byte aligned", what);
    return CBS_OK;
}

cbs_status may(const void *p, const char *what) { return p ? need(p, what) : CBS_OK; }

cbs_status float_type(int prec, const char *what) {
    if (prec != CBS_FP32 && prec != CBS_BF16) return fail(CBS_ERR_INVALID_ARG, "%s must be FP32 or BF16", what);
    return CBS_OK;
}

cbs_status head_shape(int kv_heads, int head_dim) {
    if (kv_heads < 1 || head_dim < 1) return fail(CBS_ERR_INVALID_ARG, "bad heads (%d of %d)", kv_heads, head_dim);
    if (head_dim != 64 && head_dim != 128) return fail(CBS_ERR_UNSUPPORTED, "head_dim %d: 64 or 128", head_dim);
    return CBS_OK;
}

// Checks a cache and a call's sequences and lays them out for the kernels.
cbs_status cache_args(const cbs_cache *c, const cbs_sequences *s, bool starts, CacheArgs *a) {
    if (!c || !s) return fail(CBS_ERR_INVALID_ARG, "%s is NULL", c ? "sequences" : "cache");
    if (c->prec != CBS_BF16 && c->prec != CBS_INT8) return fail(CBS_ERR_INVALID_ARG, "a cache is BF16 or INT8");
    CBS_TRY(head_shape(c->kv_heads, c->head_dim));
    if (c->num_pages < 1) return fail(CBS_ERR_INVALID_ARG, "a cache needs a page");
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
        return fail(CBS_ERR_UNSUPPORTED, "page_size %d: 16, 32, 64, 128 or 256", c->page_size);
    if ((long long)c->num_pages * c->kv_heads > INT_MAX / c->page_size)
        return fail(CBS_ERR_UNSUPPORTED, "cache of over 2^31 rows");
    CBS_TRY(need(c->k, "k"));
    CBS_TRY(need(c->v, "v"));
    if (c->prec == CBS_INT8) {
        CBS_TRY(need(c->k_scale, "k_scale"));
        CBS_TRY(need(c->v_scale, "v_scale"));
    } else if (c->k_scale || c->v_scale) {
        return fail(CBS_ERR_INVALID_ARG, "scales given for a BF16 cache");
    }
    if (s->batch < 0 || s->max_pages < 0 || s->total < 0 || s->max_pages > INT_MAX / c->page_size)
        return fail(CBS_ERR_INVALID_ARG, "bad sequences (batch=%d max_pages=%d total=%d)", s->batch, s->max_pages, s->total);
    if (s->batch > 0) {
        if (starts && !s->new_start) return fail(CBS_ERR_INVALID_ARG, "new_start is NULL");
        if (!s->seq_lens) return fail(CBS_ERR_INVALID_ARG, "seq_lens is NULL");
        if (s->max_pages > 0 && !s->page_table) return fail(CBS_ERR_INVALID_ARG, "page_table is NULL");
        for (const void *p : {(const void *)s->new_start, (const void *)s->seq_lens, (const void *)s->page_table})
            if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(CBS_ERR_MISALIGNED, "an int32 array is not 4-byte aligned");
    }
    a->k = c->k; a->v = c->v; a->k_scale = c->k_scale; a->v_scale = c->v_scale;
    a->int8 = c->prec == CBS_INT8;
    a->num_pages = c->num_pages;
    a->page_shift = 0;
    while ((1 << a->page_shift) < c->page_size) ++a->page_shift;
    a->kv_heads = c->kv_heads; a->head_dim = c->head_dim;
    a->new_start = s->new_start; a->seq_lens = s->seq_lens; a->page_table = s->page_table;
    a->batch = s->batch; a->max_pages = s->max_pages; a->total = s->total;
    a->status = nullptr;
    return CBS_OK;
}

cbs_status status_word(CacheArgs *a) {
    a->status = device_status_word();
    if (!a->status) return fail(CBS_ERR_CUDA, "cannot resolve the device status word");
    return CBS_OK;
}

cbs_status token_stride(long long stride, long long least, const char *what) {
    if (stride < least) return fail(CBS_ERR_INVALID_ARG, "%s %lld < %lld elements of a token", what, stride, least);
    if (stride % 8) return fail(CBS_ERR_MISALIGNED, "%s %lld is not a multiple of 8", what, stride);
    return CBS_OK;
}

// Outputs must not lie on what other CTAs still read.
bool overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + b_bytes && y < x + a_bytes;
}

// Rows of `width` 16-bit elements, `total` of them: side by side in wider rows of
// one pitch is not on one another.  (Of two pitches, where the ranges meet, taken to be.)
bool rows_overlap(const void *a, long long a_stride, const void *b, long long b_stride, long long width, int total) {
    const auto bytes = [&](long long stride) { return (size_t)((total - 1) * stride + width) * 2; };
    if (!overlap(a, bytes(a_stride), b, bytes(b_stride))) return false;
    if (a_stride != b_stride) return true;
    const long long at = (static_cast<const char *>(b) - static_cast<const char *>(a)) / 2 % a_stride;
    const long long r = at < 0 ? at + a_stride : at;
    return r < width || r + width > a_stride;
}

constexpr int kGridMax = 65535;

// Most rows of a key head for the few-row kernel.  32 heads, 8 key heads of 128,
// few-row (the better of its two ways to join ranges) / chunk kernel in us, for 8,
// 16, 32, 64 rows: bf16 (tiles of 8 rows), one sequence of 4000 keys 11/13, 13/13,
// 18/14, 24/14; 16 of 4000 53/56, 82/56, 134/56, 238/57; 64 of 1000 59/79, 78/80,
// 127/82, 226/85.  8 bits (tiles of 16 from 16 rows on; the chunk kernel widens every
// code first): 11/19, 11/19, 14/19, 17/20; 46/119, 54/120, 100/120, 165/119; 50/126,
// 51/127, 94/126, 160/127.
constexpr int kAttnRowsMost = 8, kAttnRowsMostInt8 = 32;

size_t attn_counter_bytes(const cbs_attn_plan_t &p) {
    return ((size_t)p.desc.batch * p.desc.kv_heads * p.row_tiles * 4 + 255) / 256 * 256;
}
size_t attn_stat_rows(const cbs_attn_plan_t &p) {
    return (size_t)p.desc.batch * p.desc.kv_heads * p.row_tiles * p.split * p.row_tile;
}

}  // namespace
}  // namespace cbs

using namespace cbs;

extern "C" {

cbs_status cbs_cache_write(const cbs_cache *c, const cbs_sequences *s, const void *k, long long k_stride,
                           const void *v, long long v_stride, int in_prec, void *stream) {
    CacheArgs a;
    CBS_TRY(cache_args(c, s, true, &a));
    CBS_TRY(float_type(in_prec, "keys and values"));
    CBS_TRY(token_stride(k_stride, (long long)c->kv_heads * c->head_dim, "k_stride"));
    CBS_TRY(token_stride(v_stride, (long long)c->kv_heads * c->head_dim, "v_stride"));
    if (s->batch == 0 || s->total == 0) return CBS_OK;
    CBS_TRY(need(k, "k"));
    CBS_TRY(need(v, "v"));
    CBS_TRY(status_word(&a));
    return cuda_check(launch_cache_write(a, k, k_stride, v, v_stride, in_prec == CBS_BF16, (cudaStream_t)stream),
                      "cache write launch");
}

cbs_status cbs_cache_read(const cbs_cache *c, const cbs_sequences *s, int max_len, void *k_out, void *v_out,
                          int out_prec, void *stream) {
    CacheArgs a;
    CBS_TRY(cache_args(c, s, false, &a));
    CBS_TRY(float_type(out_prec, "output"));
    if (max_len < 0) return fail(CBS_ERR_INVALID_ARG, "max_len %d", max_len);
    if (s->batch > kGridMax || c->kv_heads > kGridMax)
        return fail(CBS_ERR_UNSUPPORTED, "%d sequences, %d heads: at most %d", s->batch, c->kv_heads, kGridMax);
    if (s->batch == 0 || max_len == 0) return CBS_OK;
    CBS_TRY(need(k_out, "k_out"));
    CBS_TRY(need(v_out, "v_out"));
    CBS_TRY(status_word(&a));
    return cuda_check(launch_cache_read(a, max_len, k_out, v_out, out_prec == CBS_BF16, (cudaStream_t)stream),
                      "cache read launch");
}

cbs_status cbs_attn_plan(const cbs_attn_desc *d, cbs_attn_plan_t *out) {
    if (!d || !out) return fail(CBS_ERR_INVALID_ARG, "%s is NULL", d ? "out" : "desc");
    if (d->batch < 0 || d->max_new < 0 || d->max_len < 0 || d->heads < 1 || d->window < 0 || d->force_split < 0 ||
        d->num_sms < 0)
        return fail(CBS_ERR_INVALID_ARG, "bad attention shape (batch=%d max_new=%d max_len=%d heads=%d window=%d)",
                    d->batch, d->max_new, d->max_len, d->heads, d->window);
    CBS_TRY(head_shape(d->kv_heads, d->head_dim));
    if (d->heads % d->kv_heads)
        return fail(CBS_ERR_INVALID_ARG, "%d heads do not share %d key heads evenly", d->heads, d->kv_heads);
    if (d->cache_prec != CBS_BF16 && d->cache_prec != CBS_INT8)
        return fail(CBS_ERR_INVALID_ARG, "a cache is BF16 or INT8");
    if (d->force_kernel < -1 || d->force_kernel > CBS_ATTN_CLUSTER)
        return fail(CBS_ERR_INVALID_ARG, "unknown attention kernel %d", d->force_kernel);
    cbs_attn_plan_t p;
    std::memset(&p, 0, sizeof(p));
    p.size = sizeof(p);
    p.abi_version = CBS_ABI_VERSION;
    p.desc = *d;
    const long long rows = (long long)d->max_new * (d->heads / d->kv_heads);
    const int rows_most = d->cache_prec == CBS_INT8 ? kAttnRowsMostInt8 : kAttnRowsMost;
    p.kernel = d->force_kernel >= 0 ? d->force_kernel : rows > rows_most ? CBS_ATTN_CHUNK : CBS_ATTN_ROWS;
    const bool chunk = p.kernel == CBS_ATTN_CHUNK;
    // (Tiles of 16 rows in 8 bits alone: a bf16 cache's call of more than eight takes
    // the chunk kernel, unless told otherwise.)
    p.row_tile = chunk ? kAttnChunkRows : rows <= 8 || d->cache_prec == CBS_BF16 ? 8 : 16;
    const long long tiles = (rows + p.row_tile - 1) / p.row_tile;
    if (tiles * d->kv_heads > kGridMax || d->batch > kGridMax)
        return fail(CBS_ERR_UNSUPPORTED, "%lld row tiles of %d heads, %d sequences: at most %d", tiles, d->kv_heads,
                    d->batch, kGridMax);
    if (rows * (d->heads / d->kv_heads) >= 1ll << 32)
        return fail(CBS_ERR_UNSUPPORTED, "%d new tokens of %d heads", d->max_new, d->heads);
    p.row_tiles = (int)std::max(tiles, 1ll);
    const int sms = d->num_sms > 0 ? d->num_sms : kDefaultNumSMs;
    const long long base = (long long)std::max(d->batch, 1) * d->kv_heads * p.row_tiles;
    const int keys = d->window > 0 ? (int)std::min<long long>(d->max_len, (long long)d->window + d->max_new) : d->max_len;
    if (d->force_split) {
        p.split = p.kernel == CBS_ATTN_ROWS ? d->force_split : std::min(d->force_split, kAttnClusterMost);
    } else if (chunk) {
        // One CTA an SM: the split with the least rounds of clusters times what a
        // range costs.  Of 152 SMs, that many clusters of x such CTAs run at once.
        // A key tile is one unit (1.6 us, head dimension 128), a range's start and
        // end 4.5, a cluster's join 2 and a fifth for each CTA.  64 tokens of 32
        // heads over 4096 keys of 8 key heads, 1 to 8 ranges: one sequence 60, 39,
        // 30, 26, 23, 22, 21, 22 us; four sequences 61, 40, 31, 28, 47, 45, 62, 64.
        // Less than a tenth is not worth a cluster: sequences are of unequal lengths.
        static constexpr int kAtOnce[kAttnChunkSplitMost] = {152, 76, 46, 36, 28, 23, 15, 15};
        const int key_tiles = std::max((keys + kAttnChunkKeys - 1) / kAttnChunkKeys, 1);
        long long best = 0;
        for (int x = 1; x <= std::min(key_tiles, kAttnChunkSplitMost); ++x) {
            const int at_once = std::max(kAtOnce[x - 1] * sms / 152, 1);
            const long long rounds = (base + at_once - 1) / at_once;
            const long long cost = rounds * ((key_tiles + x - 1) / x * 10 + 45 + (x > 1 ? 20 + 2 * x : 0));
            if (x == 1) best = cost - cost / 10, p.split = 1;
            else if (cost < best) best = cost, p.split = x;
        }
    } else {
        // At least a CTA for each SM if that leaves a range 64 keys, and up to
        // twelve if it leaves 640.  Tokens of 32 heads, 8 key heads, 1, 2, 4, ... 32
        // ranges: one sequence of 1000 keys 16, 12, 8.1, 6.8, 6.8, 9.8 us; one of 8192
        // 112, 59, 32, 19, 13, 14; 8 of 8192 140, 76, 55, 63, 57, 61 (12 ranges 52); 32
        // of 1024 29, 37, 34, 37, 51, 88.  8 bits: one of 1000 15, 11, 7.8, 6.8, 7.1, 10;
        // one of 8192 99, 54, 29, 18, 12, 15; 32 of 8192 194, 178, 146, 137, 150, 180.
        const long long few = std::min((sms + base - 1) / base, ((long long)keys + 63) / 64);
        const long long many = std::min((sms * 12ll + base - 1) / base, (long long)keys / 640);
        p.split = (int)std::max(1ll, std::max(few, many));
        // Up to eight ranges join in a cluster where it does not keep CTAs waiting (three
        // an SM; more are made eight if that leaves a range 512 keys at most, and five to
        // seven four).  Through the workspace / in a cluster: one token over 1000 keys, 8
        // ranges 6.8/5.7 us (16 ranges 6.8 through the workspace), over 4000 12.0/10.9 (19
        // ranges 10.1), two tokens over 1000 8.1/5.9; four sequences of 1000, 4 ranges
        // 8.3/7.3, 5 ranges 9.2/8.5; 16 of 1000, 2 ranges 16.8/15.5; 8 of 8000, 8 ranges
        // 62/60; 32 of 8000, 8 ranges 168/187.  8 bits: 6.9/5.7 (7.1), 11.4/10.2 (10.0),
        // 8.3/5.9; 8.0/7.0, 9.2/8.6; 16.5/15.2; 52/53; 135/159.
        const int most = std::min(p.split, kAttnClusterMost), x = most > 4 && most < 8 ? 4 : most;
        const bool fits = p.split <= kAttnClusterMost || keys <= 512 * kAttnClusterMost;
        if (d->force_kernel == CBS_ATTN_CLUSTER || (d->force_kernel < 0 && fits && base * x <= 3ll * sms)) {
            p.kernel = CBS_ATTN_CLUSTER;
            p.split = x;
        }
    }
    p.threads = chunk ? (d->cache_prec == CBS_INT8 ? 704 : 640) : 128;
    const long long ctas = base * p.split;
    if (ctas > INT_MAX) return fail(CBS_ERR_UNSUPPORTED, "%lld CTAs", ctas);
    p.grid_ctas = (int)ctas;
    if (p.split > 1 && p.kernel == CBS_ATTN_ROWS) {
        const size_t rows_all = attn_stat_rows(p);
        p.workspace_bytes = attn_counter_bytes(p) + (rows_all * 8 + 255) / 256 * 256 + rows_all * d->head_dim * 4;
    }
    *out = p;
    return CBS_OK;
}

cbs_status cbs_paged_attention(const cbs_attn_plan_t *p, const cbs_cache *c, const cbs_sequences *s, const void *q,
                               long long q_stride, float scale, void *out, long long out_stride, void *workspace,
                               size_t workspace_bytes, void *stream) {
    if (!p) return fail(CBS_ERR_INVALID_ARG, "plan is NULL");
    if (p->size != sizeof(cbs_attn_plan_t) || p->abi_version != CBS_ABI_VERSION)
        return fail(CBS_ERR_PLAN_MISMATCH, "plan of another library version");
    const cbs_attn_desc &d = p->desc;
    AttnLaunch L;
    std::memset(&L, 0, sizeof(L));
    CBS_TRY(cache_args(c, s, true, &L.c));
    if (c->prec != d.cache_prec || c->kv_heads != d.kv_heads || c->head_dim != d.head_dim || s->batch != d.batch)
        return fail(CBS_ERR_PLAN_MISMATCH, "the plan is for another cache or batch");
    const long long width = (long long)d.heads * d.head_dim;
    CBS_TRY(token_stride(q_stride, width, "q_stride"));
    CBS_TRY(token_stride(out_stride, width, "out_stride"));
    if (!std::isfinite(scale)) return fail(CBS_ERR_INVALID_ARG, "scale is not finite");
    if (s->total == 0) return CBS_OK;
    if (s->batch == 0) {   // all tokens are padding
        CBS_TRY(need(out, "out"));
        return cuda_check(cudaMemset2DAsync(out, (size_t)out_stride * 2, 0, (size_t)width * 2, s->total, (cudaStream_t)stream),
                          "zero padding");
    }
    if (d.max_new == 0) return fail(CBS_ERR_INVALID_ARG, "%d new tokens for a plan of none", s->total);
    CBS_TRY(need(q, "q"));
    CBS_TRY(need(out, "out"));
    if (p->workspace_bytes > 0) {
        if (!workspace || workspace_bytes < p->workspace_bytes)
            return fail(CBS_ERR_WORKSPACE, "workspace of %zu bytes, %zu required", workspace ? workspace_bytes : (size_t)0,
                        p->workspace_bytes);
        CBS_TRY(need(workspace, "workspace"));
    }
    if (rows_overlap(q, q_stride, out, out_stride, width, s->total)) return fail(CBS_ERR_INVALID_ARG, "out lies on q");
    CBS_TRY(status_word(&L.c));
    L.q = q; L.out = out; L.q_stride = q_stride; L.out_stride = out_stride;
    L.scale_log2 = scale * 1.44269504088896340736f;
    L.group = d.heads / d.kv_heads;
    L.group_magic = L.group > 1 ? (unsigned)(((1ull << 32) + L.group - 1) / L.group) : 0u;
    L.heads = d.heads; L.causal = d.causal != 0; L.window = d.window; L.max_new = d.max_new;
    L.split = p->split; L.row_tiles = p->row_tiles;
    L.cluster = p->kernel == CBS_ATTN_CLUSTER && p->split > 1;
    if (p->workspace_bytes > 0) {
        char *w = static_cast<char *>(workspace);
        L.counters = reinterpret_cast<unsigned int *>(w);
        L.stats = reinterpret_cast<float2 *>(w + attn_counter_bytes(*p));
        L.partial = reinterpret_cast<float *>(w + attn_counter_bytes(*p) + (attn_stat_rows(*p) * 8 + 255) / 256 * 256);
    }
    if (p->kernel == CBS_ATTN_CHUNK) return launch_attn_chunk(L, (cudaStream_t)stream);
    return cuda_check(launch_attn_rows(L, p->row_tile, (cudaStream_t)stream), "attention launch");
}

cbs_status cbs_rmsnorm(const void *x, const void *residual, const float *weight, void *h_out, void *y, float *scale,
                       int rows, int cols, float eps, int in_prec, int out_prec, void *stream) {
    CBS_TRY(float_type(in_prec, "input"));
    if (out_prec != in_prec && out_prec != CBS_INT8)
        return fail(CBS_ERR_INVALID_ARG, "output must be of the input's type or INT8");
    if (rows < 0 || cols < 1) return fail(CBS_ERR_INVALID_ARG, "bad norm shape (%d x %d)", rows, cols);
    if (cols > kNormMaxCols) return fail(CBS_ERR_UNSUPPORTED, "%d columns: at most %d", cols, kNormMaxCols);
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(CBS_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (h_out && !residual) return fail(CBS_ERR_INVALID_ARG, "h_out without a residual is x itself");
    if (rows == 0) return CBS_OK;
    CBS_TRY(need(x, "x"));
    CBS_TRY(may(residual, "residual"));
    CBS_TRY(need(weight, "weight"));
    CBS_TRY(may(h_out, "h_out"));
    CBS_TRY(need(y, "y"));
    if (out_prec == CBS_INT8) CBS_TRY(need(scale, "scale"));
    const size_t in_bytes = (size_t)rows * cols * (in_prec == CBS_BF16 ? 2 : 4);
    const size_t y_bytes = out_prec == CBS_INT8 ? (size_t)rows * cols : in_bytes;
    for (const void *in : {x, residual}) {
        if (h_out != in && overlap(h_out, in_bytes, in, in_bytes)) return fail(CBS_ERR_INVALID_ARG, "h_out lies across an input");
        if ((y != in || out_prec == CBS_INT8) && overlap(y, y_bytes, in, in_bytes))
            return fail(CBS_ERR_INVALID_ARG, "y lies on an input");
        if (out_prec == CBS_INT8 && overlap(scale, (size_t)rows * 4, in, in_bytes)) return fail(CBS_ERR_INVALID_ARG, "scale lies on an input");
    }
    if (overlap(y, y_bytes, h_out, in_bytes)) return fail(CBS_ERR_INVALID_ARG, "y lies on h_out");
    NormLaunch L;
    L.x = x; L.residual = residual; L.weight = weight; L.h = h_out; L.y = y; L.scale = scale;
    L.eps = eps; L.rows = rows; L.cols = cols; L.in_bf16 = in_prec == CBS_BF16; L.out_int8 = out_prec == CBS_INT8;
    return cuda_check(launch_rmsnorm(L, (cudaStream_t)stream), "norm launch");
}

cbs_status cbs_dequantize_rows(const int8_t *q, const float *scale, void *out, int rows, int cols, int out_prec,
                               void *stream) {
    CBS_TRY(float_type(out_prec, "output"));
    if (rows < 0 || cols < 1) return fail(CBS_ERR_INVALID_ARG, "bad shape (%d x %d)", rows, cols);
    if (rows == 0) return CBS_OK;
    CBS_TRY(need(q, "q"));
    CBS_TRY(need(scale, "scale"));
    CBS_TRY(need(out, "out"));
    const size_t count = (size_t)rows * cols, out_bytes = count * (out_prec == CBS_BF16 ? 2 : 4);
    if (overlap(out, out_bytes, q, count) || overlap(out, out_bytes, scale, (size_t)rows * 4))
        return fail(CBS_ERR_INVALID_ARG, "out lies on an input");
    return cuda_check(launch_dequantize_rows(q, scale, out, rows, cols, out_prec == CBS_BF16, (cudaStream_t)stream),
                      "dequantise launch");
}

static cbs_status w4_shape(int n, int k, int group) {
    if (n < 1 || k < 1) return fail(CBS_ERR_INVALID_ARG, "bad weight shape (%d x %d)", n, k);
    if (group != 32 && group != 64 && group != 128) return fail(CBS_ERR_UNSUPPORTED, "group %d: 32, 64 or 128", group);
    if (k % group) return fail(CBS_ERR_UNSUPPORTED, "k = %d is not a multiple of the group (%d)", k, group);
    return CBS_OK;
}

cbs_status cbs_linear_w4(const void *x, int x_prec, const float *x_scale, const void *w, const void *scales,
                         const void *zeros, const float *bias, void *y, int out_prec, int rows, int n, int k, int group,
                         int activation, void *stream) {
    if (x_prec != CBS_BF16 && x_prec != CBS_INT8) return fail(CBS_ERR_INVALID_ARG, "x must be BF16 or INT8");
    CBS_TRY(float_type(out_prec, "output"));
    CBS_TRY(w4_shape(n, k, group));
    if (activation != CBS_ACT_SILU && activation != CBS_ACT_IDENTITY)
        return fail(CBS_ERR_INVALID_ARG, "unknown activation %d", activation);
    if (rows < 0) return fail(CBS_ERR_INVALID_ARG, "%d rows", rows);
    if (rows > 16 * kGridMax) return fail(CBS_ERR_UNSUPPORTED, "%d rows: at most %d", rows, 16 * kGridMax);
    if (x_prec == CBS_BF16 && x_scale) return fail(CBS_ERR_INVALID_ARG, "x_scale given for BF16 inputs");
    if (rows == 0) return CBS_OK;
    CBS_TRY(need(x, "x"));
    if (x_prec == CBS_INT8) CBS_TRY(need(x_scale, "x_scale"));
    CBS_TRY(need(w, "w"));
    CBS_TRY(need(scales, "scales"));
    CBS_TRY(may(zeros, "zeros"));
    CBS_TRY(may(bias, "bias"));
    CBS_TRY(need(y, "y"));
    const size_t y_bytes = (size_t)rows * n * (out_prec == CBS_BF16 ? 2 : 4);
    if (overlap(y, y_bytes, x, (size_t)rows * k * (x_prec == CBS_BF16 ? 2 : 1)) || overlap(y, y_bytes, x_scale, (size_t)rows * 4))
        return fail(CBS_ERR_INVALID_ARG, "y lies on an input");
    W4Launch L;
    L.x = x; L.x_scale = x_scale; L.w = static_cast<const uint8_t *>(w); L.scales = scales;
    L.zeros = static_cast<const uint8_t *>(zeros); L.bias = bias; L.y = y;
    L.rows = rows; L.n = n; L.k = k; L.group = group; L.x_int8 = x_prec == CBS_INT8; L.out_bf16 = out_prec == CBS_BF16;
    L.act = activation;
    L.status = device_status_word();
    if (!L.status) return fail(CBS_ERR_CUDA, "cannot resolve the device status word");
    return launch_w4(L, (cudaStream_t)stream);
}

cbs_status cbs_quantize_w4(const float *w, int n, int k, int group, void *packed, void *scales, void *stream) {
    CBS_TRY(w4_shape(n, k, group));
    CBS_TRY(need(w, "w"));
    CBS_TRY(need(packed, "packed"));
    CBS_TRY(need(scales, "scales"));
    return cuda_check(launch_quantize_w4(w, n, k, group, static_cast<uint8_t *>(packed), scales, (cudaStream_t)stream),
                      "4-bit quantiser launch");
}

}  // extern "C"
