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
// few-row (the better of its two ways to join ranges) / chunk kernel in us on the GPU, for
// 8, 16, 32, 64 rows: bf16 (tiles of 8 rows), one sequence of 4000 keys 9.1/14, 10/14,
// 14/15, 16/15; 16 of 4000 47/58, 64/58, 94/58, 158/58; 64 of 1000 45/83, 60/84, 87/84,
// 153/86 (so sixteen rows would be faster in two of three).  8 bits (tiles of 16 from 16
// rows on; the chunk kernel widens every code first): 9.8/19, 11/19, 14/19, 17/20; 35/120,
// 49/120, 77/120, 135/120; 33/126, 45/127, 69/127, 126/127.
constexpr int kAttnRowsMost = 8, kAttnRowsMostInt8 = 32;

// Of 152 SMs with one CTA each, that many clusters of x of the chunk kernel's CTAs run at once.
long long chunk_rounds(long long base, int x, int sms) {
    static constexpr int kAtOnce[kAttnChunkSplitMost] = {152, 76, 46, 36, 28, 23, 15, 15};
    const int at_once = std::max(kAtOnce[x - 1] * sms / 152, 1);
    return (base + at_once - 1) / at_once;
}
int chunk_key_tiles(int keys) { return std::max((keys + kAttnChunkKeys - 1) / kAttnChunkKeys, 1); }

// Ranges of keys of the chunk kernel, for `base` row tiles of all sequences and heads.
int chunk_split(long long base, int keys, int sms) {
    // The split with the least rounds of clusters times what a range costs.  A key tile
    // is one unit (1.6 us, head dimension 128), a range's start and end 4.5, a cluster's
    // join 2 and a fifth for each CTA.  64 tokens of 32 heads over 4096 keys of 8 key
    // heads, 1 to 8 ranges: one sequence 60, 39, 30, 26, 23, 22, 21, 22 us; four
    // sequences 61, 40, 31, 28, 47, 45, 62, 64.
    // Less than a tenth is not worth a cluster: sequences are of unequal lengths.
    const int key_tiles = chunk_key_tiles(keys);
    long long best = 0;
    int split = 1;
    for (int x = 1; x <= std::min(key_tiles, kAttnChunkSplitMost); ++x) {
        const long long cost = chunk_rounds(base, x, sms) * ((key_tiles + x - 1) / x * 10 + 45 + (x > 1 ? 20 + 2 * x : 0));
        if (x == 1) best = cost - cost / 10;
        else if (cost < best) best = cost, split = x;
    }
    return split;
}

// Its time in nanoseconds, in the same terms: a key tile's by head dimension and type.
long long chunk_ns(const cbs_attn_desc &d, long long base, int x, int sms) {
    const int tile = d.cache_prec == CBS_INT8 ? (d.head_dim == 64 ? 2400 : 3000) : d.head_dim == 64 ? 1400 : 1600;
    return chunk_rounds(base, x, sms) * ((long long)((chunk_key_tiles(d.max_len) + x - 1) / x) * tile + 7200 + (x > 1 ? 3200 + 320 * x : 0));
}

// Ranges of a shared prefix, whose CTAs run beside those of the sequences' own part and
// keep their SMs from it: the least of the two parts' end.  The own part takes its bytes at
// 5.8 TB/s (few rows; sequences three quarters of the longest on average) or its tiles'
// time; beside it a prefix's takes a fifth longer.  64 streams over a prefix of 8192
// (bf16, own part of up to 1000 keys 45 us alone), 1, 2, 3, 4 and 8 ranges (8 to 64 CTAs,
// alone 107, 62, 47, 37, 27 us): 121, 73, 57, 52, 57 us; with the own part at 36 us alone
// 51 with four and 47.6 with five.
int prefix_split(const cbs_shared_plan_t &p, long long base, int sms) {
    const cbs_attn_desc &d = p.prefix.desc, &o = p.own.desc;
    const long long bytes = (long long)o.batch * o.max_len * 3 / 4 * d.kv_heads * d.head_dim * (d.cache_prec == CBS_INT8 ? 2 : 4);
    const long long own = p.own.kernel == CBS_ATTN_CHUNK ? chunk_ns(o, (long long)o.batch * o.kv_heads * p.own.row_tiles, p.own.split, sms)
                                                         : bytes / 5800;
    long long best = 0;
    int split = 1;
    for (int x = 1; x <= std::min(chunk_key_tiles(d.max_len), kAttnChunkSplitMost); ++x) {
        const long long prefix = chunk_ns(d, base, x, sms) * 6 / 5, end = std::max(prefix, own + prefix * std::min<long long>(base * x, sms) / sms);
        if (x == 1 || end < best) best = end, split = x;
    }
    return split;
}

size_t attn_counter_bytes(const cbs_attn_plan_t &p) {
    return ((size_t)p.desc.batch * p.desc.kv_heads * p.row_tiles * 4 + 255) / 256 * 256;
}
size_t attn_stat_rows(const cbs_attn_plan_t &p) {
    return (size_t)p.desc.batch * p.desc.kv_heads * p.row_tiles * p.split * p.row_tile;
}
size_t round256(size_t bytes) { return (bytes + 255) / 256 * 256; }

// A workspace's parts, as offsets.
struct WeighedParts { size_t row_stats, sums, scores, all; int rows_pad, len_pad; };
WeighedParts weighed_parts(const cbs_attn_plan_t &p) {
    const cbs_attn_desc &d = p.desc;
    WeighedParts w;
    w.rows_pad = (int)((long long)d.max_new * (d.heads / d.kv_heads));
    w.len_pad = (int)(std::max(d.max_len + 15ll, 16ll) / 16 * 16);
    w.row_stats = round256(p.workspace_bytes);
    w.sums = w.row_stats + round256((size_t)d.batch * d.max_new * d.heads * 8);
    w.scores = w.sums + (p.workspace_bytes ? round256(attn_stat_rows(p) * 4) : 0);
    w.all = w.scores + (p.kernel == CBS_ATTN_CHUNK ? 0 : (size_t)d.batch * d.kv_heads * w.rows_pad * w.len_pad * 4);
    return w;
}
struct SharedParts { size_t own, stats, share, own_stats, own_share, all; };
SharedParts shared_parts(const cbs_shared_plan_t &p) {
    SharedParts w;
    w.own = round256(p.prefix.workspace_bytes);
    w.stats = w.own + round256(p.own.workspace_bytes);
    w.share = w.stats + round256((size_t)p.max_total * p.desc.heads * 8);
    const size_t stats = w.share - w.stats, share = round256((size_t)p.max_total * p.desc.heads * p.desc.head_dim * 4);
    w.own_stats = w.share + share;
    w.own_share = w.own_stats + stats;
    w.all = w.own_share + share;
    return w;
}

// What a plan says of a launch.
void attn_fill(const cbs_attn_plan_t &p, AttnLaunch *L) {
    const cbs_attn_desc &d = p.desc;
    L->group = d.heads / d.kv_heads;
    L->group_magic = L->group > 1 ? (unsigned)(((1ull << 32) + L->group - 1) / L->group) : 0u;
    L->heads = d.heads; L->causal = d.causal != 0; L->window = d.window; L->max_new = d.max_new;
    L->split = p.split; L->row_tiles = p.row_tiles;
    L->cluster = p.kernel == CBS_ATTN_CLUSTER && p.split > 1;
}
void attn_workspace(const cbs_attn_plan_t &p, void *workspace, AttnLaunch *L) {
    if (p.workspace_bytes == 0) return;
    char *w = static_cast<char *>(workspace);
    L->counters = reinterpret_cast<unsigned int *>(w);
    L->stats = reinterpret_cast<float2 *>(w + attn_counter_bytes(p));
    L->partial = reinterpret_cast<float *>(w + attn_counter_bytes(p) + round256(attn_stat_rows(p) * 8));
}

// Checks of an attention call and its launch but for the workspace's parts and the
// status word; *run: there is something to compute.
cbs_status attn_call(const cbs_attn_plan_t &p, const cbs_cache *c, const cbs_sequences *s, const void *q, long long q_stride, float scale,
                     void *out, long long out_stride, void *workspace, size_t workspace_bytes, size_t needed, int batch,
                     cudaStream_t stream, AttnLaunch *L, bool *run) {
    *run = false;
    if (p.size != sizeof(cbs_attn_plan_t) || p.abi_version != CBS_ABI_VERSION)
        return fail(CBS_ERR_PLAN_MISMATCH, "plan of another library version");
    const cbs_attn_desc &d = p.desc;
    std::memset(L, 0, sizeof(*L));
    CBS_TRY(cache_args(c, s, true, &L->c));
    if (c->prec != d.cache_prec || c->kv_heads != d.kv_heads || c->head_dim != d.head_dim || s->batch != batch)
        return fail(CBS_ERR_PLAN_MISMATCH, "the plan is for another cache or batch");
    const long long width = (long long)d.heads * d.head_dim;
    CBS_TRY(token_stride(q_stride, width, "q_stride"));
    CBS_TRY(token_stride(out_stride, width, "out_stride"));
    if (!std::isfinite(scale)) return fail(CBS_ERR_INVALID_ARG, "scale is not finite");
    if (s->total == 0) return CBS_OK;
    if (s->batch == 0) {   // all tokens are padding
        CBS_TRY(need(out, "out"));
        return cuda_check(cudaMemset2DAsync(out, (size_t)out_stride * 2, 0, (size_t)width * 2, s->total, stream), "zero padding");
    }
    if (d.max_new == 0) return fail(CBS_ERR_INVALID_ARG, "%d new tokens for a plan of none", s->total);
    CBS_TRY(need(q, "q"));
    CBS_TRY(need(out, "out"));
    if (needed > 0) {
        if (!workspace || workspace_bytes < needed)
            return fail(CBS_ERR_WORKSPACE, "workspace of %zu bytes, %zu required", workspace ? workspace_bytes : (size_t)0, needed);
        CBS_TRY(need(workspace, "workspace"));
    }
    if (rows_overlap(q, q_stride, out, out_stride, width, s->total)) return fail(CBS_ERR_INVALID_ARG, "out lies on q");
    L->q = q; L->out = out; L->q_stride = q_stride; L->out_stride = out_stride;
    L->scale_log2 = scale * 1.44269504088896340736f;
    attn_fill(p, L);
    *run = true;
    return CBS_OK;
}

// few: 1 or 0 for the few-row kernels or the chunk kernel, -1 for what the rows say.
cbs_status attn_plan(const cbs_attn_desc *d, int few, cbs_attn_plan_t *out) {
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
    p.kernel = d->force_kernel >= 0 ? d->force_kernel : (few < 0 ? rows > rows_most : !few) ? CBS_ATTN_CHUNK : CBS_ATTN_ROWS;
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
        p.split = chunk_split(base, keys, sms);
    } else {
        // At least a CTA for each SM if that leaves a range 64 keys, and up to
        // twelve if it leaves 640.  Tokens of 32 heads, 8 key heads of 128, 1, 2, 4, 8, 12, 16
        // and 32 ranges joined through the workspace, us on the GPU: one sequence of 1000 keys
        // 12, 9.6, 6.9, 6.5, 7.7, 7.1, 10; one of 8192 79, 44, 24, 15, 12, 11, 14; 8 of 8192 89,
        // 52, 45, 49, 50, 54, 59; 32 of 1024 24, 30, 31, 35, 43, 50, 86.  8 bits: one of 1000 14,
        // 11, 7.7, 7.1, 8.2, 8.0, 12; one of 8192 92, 50, 27, 17, 14, 13, 14; 32 of 8192 135, 116,
        // 103, 107, 111, 115, 136.
        const long long few = std::min((sms + base - 1) / base, ((long long)keys + 63) / 64);
        const long long many = std::min((sms * 12ll + base - 1) / base, (long long)keys / 640);
        p.split = (int)std::max(1ll, std::max(few, many));
        // Up to eight ranges join in a cluster where it does not keep CTAs waiting (three
        // an SM, which calls of one token take in one round by one form of the kernel or the
        // other; more are made eight if that leaves a range 512 keys at most, and five to seven
        // four).  Through the workspace / in a cluster: one token over 1000 keys, 8 ranges
        // 6.4/5.1 us (16 ranges 7.1 through the workspace), over 4000 10.0/8.9 (19 ranges 9.5),
        // two tokens over 1000 8.0/5.2; four sequences of 1000, 4 ranges 7.0/6.1, 5 ranges
        // 8.2/7.0; 16 of 1000, 2 ranges 11.6/10.2; 8 of 8000, 8 ranges 48/47; 32 of 8000, 8 ranges
        // 162/183.  8 bits: 7.0/5.3 (8.1), 11.3/9.5 (9.8), 8.6/5.5; 7.6/6.5, 8.7/8.0; 13.0/11.5;
        // 36/34; 105/107.
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

// What a plan's call takes, in nanoseconds: a few-row tile's thousand keys by head
// dimension and type (in 8 bits a tile's start and end are worth 160 more), or the chunk
// kernel's tiles.
long long attn_ns(const cbs_attn_plan_t &p, int sms) {
    const cbs_attn_desc &d = p.desc;
    const long long base = (long long)std::max(d.batch, 1) * d.kv_heads * p.row_tiles;
    if (p.kernel == CBS_ATTN_CHUNK) return chunk_ns(d, base, p.split, sms);
    const bool int8 = d.cache_prec == CBS_INT8;
    const int thousand = int8 ? (d.head_dim == 64 ? 28 : 47) : d.head_dim == 64 ? 31 : 62;
    return 4500 + base * (d.max_len + (int8 ? 160 : 0)) / 1000 * thousand;
}

// The faster kernel for a part of a call whose rows are more than the few-row
// kernels' own: short sequences do not repay a chunk's start.  (`more`: what follows
// the few-row kernel less what follows the chunk kernel.)  Head dimension 64, bf16, few
// rows and chunks: 64 rows of 400 keys, two heads 4.3 and 9.2 us, 64 heads 8.0 and 9.4;
// 8 bits, 512 heads, 64 rows of 200 keys 25 and 43, of 1000 76 and 93, and 128 rows of 1000
// 141 and 95.
cbs_status attn_plan_by_time(const cbs_attn_desc *d, long long (*more)(const cbs_attn_plan_t &few, const cbs_attn_plan_t &chunk, int sms),
                             cbs_attn_plan_t *out) {
    CBS_TRY(attn_plan(d, -1, out));
    if (d->force_kernel >= 0) return CBS_OK;
    const int sms = d->num_sms > 0 ? d->num_sms : kDefaultNumSMs;
    // Of more than eight rows the many ranges that a few-row kernel joins through the
    // workspace take longer than eight in a cluster: 16 rows of 6000 keys, two heads of
    // 128 in 8 bits 56 and 14 us, in bf16 19 and 11.  (Given ranges stay as they are.)
    const auto in_clusters = [&](cbs_attn_plan_t *p) {
        const long long base = (long long)std::max(d->batch, 1) * d->kv_heads * p->row_tiles;
        if (d->force_split || p->kernel != CBS_ATTN_ROWS || p->split <= kAttnClusterMost || (long long)d->max_new * (d->heads / d->kv_heads) <= 8 ||
            d->max_len > 8192 || base * kAttnClusterMost > 3ll * sms)
            return;
        p->kernel = CBS_ATTN_CLUSTER;
        p->split = kAttnClusterMost;
        p->grid_ctas = (int)(base * p->split);
        p->workspace_bytes = 0;
    };
    if (out->kernel != CBS_ATTN_CHUNK) {
        in_clusters(out);
        return CBS_OK;
    }
    cbs_attn_plan_t few;
    if (attn_plan(d, 1, &few) != CBS_OK) return CBS_OK;   // (too many row tiles)
    in_clusters(&few);
    if (attn_ns(few, sms) + (more ? more(few, *out, sms) : 0) < attn_ns(*out, sms)) *out = few;
    return CBS_OK;
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

cbs_status cbs_cache_evict(const cbs_cache *c, const cbs_sequences *s, float *mass, const int32_t *new_table,
                           int new_max_pages, int keep, int recent, int32_t *kept, int32_t *new_lens, void *stream) {
    EvictLaunch L;
    std::memset(&L, 0, sizeof(L));
    CBS_TRY(cache_args(c, s, false, &L.c));
    if (keep < 1 || recent < 0 || recent > keep) return fail(CBS_ERR_INVALID_ARG, "keep %d, recent %d of them", keep, recent);
    if (keep > 1 << 30) return fail(CBS_ERR_UNSUPPORTED, "keep %d: at most 2^30", keep);
    if (new_max_pages < 0) return fail(CBS_ERR_INVALID_ARG, "new_max_pages %d", new_max_pages);
    const long long held = (long long)s->max_pages * c->page_size;
    if ((long long)new_max_pages * c->page_size < std::min<long long>(keep, held))
        return fail(CBS_ERR_INVALID_ARG, "%d new pages of %d do not hold %lld positions", new_max_pages, c->page_size,
                    std::min<long long>(keep, held));
    if (held > kEvictMost) return fail(CBS_ERR_UNSUPPORTED, "tables of %lld positions: at most %lld", held, kEvictMost);
    if (s->batch > kGridMax || c->kv_heads > kGridMax)
        return fail(CBS_ERR_UNSUPPORTED, "%d sequences, %d heads: at most %d", s->batch, c->kv_heads, kGridMax);
    if (s->batch == 0) return CBS_OK;
    CBS_TRY(need(mass, "mass"));
    CBS_TRY(need(kept, "kept"));
    CBS_TRY(need(new_lens, "new_lens"));
    if (!new_table && new_max_pages > 0) return fail(CBS_ERR_INVALID_ARG, "new_table is NULL");
    if (reinterpret_cast<uintptr_t>(new_table) & 3u) return fail(CBS_ERR_MISALIGNED, "new_table is not 4-byte aligned");
    // What one part of the call writes, others still read.
    const size_t rows = (size_t)c->num_pages * c->kv_heads * c->page_size, row = (size_t)c->head_dim * (c->prec == CBS_INT8 ? 1 : 2);
    const size_t kept_bytes = (size_t)s->batch * c->kv_heads * keep * 4, lens_bytes = (size_t)s->batch * 4;
    const struct { const void *p; size_t bytes; const char *what; } parts[] = {
        {c->k, rows * row, "k"}, {c->v, rows * row, "v"}, {c->k_scale, rows * 4, "k_scale"}, {c->v_scale, rows * 4, "v_scale"},
        {mass, rows * 4, "mass"}, {s->seq_lens, lens_bytes, "seq_lens"}, {s->page_table, (size_t)s->batch * s->max_pages * 4, "page_table"},
        {new_table, (size_t)s->batch * new_max_pages * 4, "new_table"}, {new_lens, lens_bytes, "new_lens"}, {kept, kept_bytes, "kept"}};
    constexpr int kParts = sizeof(parts) / sizeof(parts[0]);
    for (int out = 4; out < kParts; ++out) {
        if (out > 4 && out < 8) continue;   // inputs
        for (int other = 0; other < out; ++other)
            if (overlap(parts[out].p, parts[out].bytes, parts[other].p, parts[other].bytes))
                return fail(CBS_ERR_INVALID_ARG, "%s lies on %s", parts[out].what, parts[other].what);
    }
    CBS_TRY(status_word(&L.c));
    L.mass = mass; L.new_table = new_table; L.new_max_pages = new_max_pages;
    L.keep = keep; L.recent = recent; L.kept = kept; L.new_lens = new_lens;
    return cuda_check(launch_evict(L, (cudaStream_t)stream), "eviction launch");
}

cbs_status cbs_attn_plan(const cbs_attn_desc *d, cbs_attn_plan_t *out) { return attn_plan(d, -1, out); }

cbs_status cbs_paged_attention(const cbs_attn_plan_t *p, const cbs_cache *c, const cbs_sequences *s, const void *q,
                               long long q_stride, float scale, void *out, long long out_stride, void *workspace,
                               size_t workspace_bytes, void *stream) {
    if (!p) return fail(CBS_ERR_INVALID_ARG, "plan is NULL");
    AttnLaunch L;
    bool run;
    CBS_TRY(attn_call(*p, c, s, q, q_stride, scale, out, out_stride, workspace, workspace_bytes, p->workspace_bytes, p->desc.batch,
                      (cudaStream_t)stream, &L, &run));
    if (!run) return CBS_OK;
    CBS_TRY(status_word(&L.c));
    attn_workspace(*p, workspace, &L);
    if (p->kernel == CBS_ATTN_CHUNK) return launch_attn_chunk(L, (cudaStream_t)stream);
    return cuda_check(launch_attn_rows(L, p->row_tile, (cudaStream_t)stream), "attention launch");
}

cbs_status cbs_weighed_plan(const cbs_attn_desc *d, cbs_weighed_plan_t *out) {
    if (!d || !out) return fail(CBS_ERR_INVALID_ARG, "%s is NULL", d ? "out" : "desc");
    cbs_weighed_plan_t p;
    std::memset(&p, 0, sizeof(p));
    p.size = sizeof(p);
    p.abi_version = CBS_ABI_VERSION;
    // What comes after the attention: scores summed up, 5 us and some more with their
    // number, or the chunk's keys again, 5.5 us a round of them and 0.8 a tile of rows.
    CBS_TRY(attn_plan_by_time(d, [](const cbs_attn_plan_t &few, const cbs_attn_plan_t &chunk, int sms) -> long long {
        const cbs_attn_desc &d = few.desc;
        const long long rows = (long long)d.max_new * (d.heads / d.kv_heads), heads = (long long)d.batch * d.kv_heads;
        const long long ctas = heads * chunk_key_tiles(d.max_len), rounds = (ctas + 2 * sms - 1) / (2 * sms);
        return 5000 + heads * rows * d.max_len / 700 - rounds * (5500 + (rows + 127) / 128 * 800);
    }, &p.attention));
    if ((d->max_len + 15ll) / 16 * 16 > INT_MAX) return fail(CBS_ERR_UNSUPPORTED, "max_len %d", d->max_len);
    p.workspace_bytes = weighed_parts(p.attention).all;
    *out = p;
    return CBS_OK;
}

cbs_status cbs_weighed_attention(const cbs_weighed_plan_t *p, const cbs_cache *c, const cbs_sequences *s, const void *q,
                                 long long q_stride, float scale, void *out, long long out_stride, float *mass, float decay,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    if (!p) return fail(CBS_ERR_INVALID_ARG, "plan is NULL");
    if (p->size != sizeof(*p) || p->abi_version != CBS_ABI_VERSION)
        return fail(CBS_ERR_PLAN_MISMATCH, "plan of another library version");
    const cbs_attn_plan_t &a = p->attention;
    if (!std::isfinite(decay)) return fail(CBS_ERR_INVALID_ARG, "decay is not finite");
    AttnLaunch L;
    bool run;
    CBS_TRY(attn_call(a, c, s, q, q_stride, scale, out, out_stride, workspace, workspace_bytes, p->workspace_bytes, a.desc.batch,
                      (cudaStream_t)stream, &L, &run));
    if (!run) return CBS_OK;
    CBS_TRY(need(mass, "mass"));
    if (s->total > (long long)a.desc.batch * a.desc.max_new)
        return fail(CBS_ERR_INVALID_ARG, "%d tokens for a plan of %d sequences of %d", s->total, a.desc.batch, a.desc.max_new);
    const size_t rows = (size_t)c->num_pages * c->kv_heads * c->page_size, row = (size_t)c->head_dim * (c->prec == CBS_INT8 ? 1 : 2);
    const long long width = (long long)a.desc.heads * c->head_dim;
    const struct { const void *p; size_t bytes; const char *what; } others[] = {
        {c->k, rows * row, "k"}, {c->v, rows * row, "v"}, {c->k_scale, rows * 4, "k_scale"}, {c->v_scale, rows * 4, "v_scale"},
        {q, (size_t)((s->total - 1) * q_stride + width) * 2, "q"}, {out, (size_t)((s->total - 1) * out_stride + width) * 2, "out"},
        {workspace, p->workspace_bytes, "workspace"}, {s->new_start, ((size_t)s->batch + 1) * 4, "new_start"},
        {s->seq_lens, (size_t)s->batch * 4, "seq_lens"}, {s->page_table, (size_t)s->batch * s->max_pages * 4, "page_table"}};
    for (const auto &o : others)
        if (overlap(mass, rows * 4, o.p, o.bytes)) return fail(CBS_ERR_INVALID_ARG, "mass lies on %s", o.what);
    CBS_TRY(status_word(&L.c));
    attn_workspace(a, workspace, &L);
    const WeighedParts w = weighed_parts(a);
    char *at = static_cast<char *>(workspace);
    L.row_stats = reinterpret_cast<float2 *>(at + w.row_stats);
    L.sums = reinterpret_cast<float *>(at + w.sums);
    L.len_pad = w.len_pad;
    L.rows_pad = w.rows_pad;
    if (a.kernel != CBS_ATTN_CHUNK) L.scores = reinterpret_cast<float *>(at + w.scores);
    L.mass = mass;
    L.decay = decay;
    // Few rows in one tile: the CTAs of a cluster weigh their own keys, and so does one
    // CTA without ranges (on the GPU, by the kernel after them / by themselves: one token over
    // 1000 keys 9.3/7.8 us; 64 sequences of 300 17.8/16.6).  Of ranges joined by the CTA that
    // finishes last, that one would weigh all of them (32 sequences of up to 8192, 8 bits:
    // 107/121).
    L.fused = L.scores && a.row_tiles == 1 && (L.cluster || a.split == 1);
    CBS_TRY(launch_attn_weighed(L, a.row_tile, (cudaStream_t)stream));
    return L.fused ? CBS_OK : launch_attn_weights(L, (cudaStream_t)stream);
}

cbs_status cbs_shared_plan(const cbs_shared_desc *d, cbs_shared_plan_t *out) {
    if (!d || !out) return fail(CBS_ERR_INVALID_ARG, "%s is NULL", d ? "out" : "desc");
    if (d->groups < 0 || d->max_group_new < 0 || d->max_prefix < 0)
        return fail(CBS_ERR_INVALID_ARG, "bad groups (%d, of %d new tokens, prefixes of %d)", d->groups, d->max_group_new, d->max_prefix);
    cbs_shared_plan_t p;
    std::memset(&p, 0, sizeof(p));
    p.size = sizeof(p);
    p.abi_version = CBS_ABI_VERSION;
    p.desc = *d;
    cbs_attn_desc part = {d->batch, d->max_new, d->max_len, d->heads, d->kv_heads, d->head_dim, d->cache_prec, 1, 0, d->num_sms, -1, 0};
    CBS_TRY(attn_plan_by_time(&part, nullptr, &p.own));
    part.batch = d->groups; part.max_new = d->max_group_new; part.max_len = d->max_prefix; part.causal = 0;
    CBS_TRY(attn_plan_by_time(&part, nullptr, &p.prefix));
    const long long total = std::min((long long)d->batch * d->max_new, (long long)d->groups * d->max_group_new);
    if (total > INT_MAX) return fail(CBS_ERR_UNSUPPORTED, "%lld new tokens", total);
    p.max_total = (int)total;
    const SharedParts parts = shared_parts(p);
    p.zeroed_bytes = parts.stats;
    p.workspace_bytes = parts.all;
    *out = p;
    return CBS_OK;
}

cbs_status cbs_shared_attention(const cbs_shared_plan_t *p, const cbs_cache *c, const cbs_sequences *s, const cbs_prefixes *prefixes,
                                const void *q, long long q_stride, float scale, void *out, long long out_stride, void *workspace,
                                size_t workspace_bytes, void *stream) {
    if (!p || !prefixes) return fail(CBS_ERR_INVALID_ARG, "%s is NULL", p ? "prefixes" : "plan");
    if (p->size != sizeof(*p) || p->abi_version != CBS_ABI_VERSION)
        return fail(CBS_ERR_PLAN_MISMATCH, "plan of another library version");
    if (prefixes->groups != p->desc.groups) return fail(CBS_ERR_PLAN_MISMATCH, "the plan is for %d groups", p->desc.groups);
    AttnLaunch own;
    bool run;
    CBS_TRY(attn_call(p->own, c, s, q, q_stride, scale, out, out_stride, workspace, workspace_bytes, p->workspace_bytes, p->desc.batch,
                      (cudaStream_t)stream, &own, &run));
    if (!run) return CBS_OK;
    if (s->total > p->max_total) return fail(CBS_ERR_INVALID_ARG, "%d tokens for a plan of %d", s->total, p->max_total);
    cbs_sequences ps = {s->new_start, prefixes->prefix_lens, prefixes->page_table, prefixes->groups, prefixes->max_pages, s->total};
    AttnLaunch pre = own;
    CBS_TRY(cache_args(c, &ps, true, &pre.c));
    if (!prefixes->group_start) return fail(CBS_ERR_INVALID_ARG, "group_start is NULL");
    if (reinterpret_cast<uintptr_t>(prefixes->group_start) & 3u) return fail(CBS_ERR_MISALIGNED, "group_start is not 4-byte aligned");
    CBS_TRY(status_word(&own.c));
    pre.c.status = own.c.status;
    const SharedParts parts = shared_parts(*p);
    char *at = static_cast<char *>(workspace);
    attn_fill(p->prefix, &pre);
    long long prefix_base = 0;
    if (p->prefix.kernel == CBS_ATTN_CHUNK) {
        // Groups differ in size: the tiles that a call of so many tokens has, half of each
        // group's last one empty, are fewer than the largest group's for every group.
        const cbs_attn_desc &d = p->prefix.desc;
        const long long tiles = ((long long)s->total * pre.group / kAttnChunkRows) + (d.batch + 1) / 2;
        prefix_base = std::min<long long>(tiles, (long long)d.batch * pre.row_tiles) * d.kv_heads;
        pre.split = prefix_split(*p, prefix_base, d.num_sms > 0 ? d.num_sms : kDefaultNumSMs);
    }
    attn_workspace(p->prefix, at, &pre);
    attn_workspace(p->own, at + parts.own, &own);
    pre.group_start = prefixes->group_start;
    pre.sequences = s->batch;
    pre.share_stats = own.share_stats = reinterpret_cast<float2 *>(at + parts.stats);
    pre.share = own.share = reinterpret_cast<float *>(at + parts.share);
    CBS_TRY(launch_attn_prefix(pre, p->prefix.row_tile, (cudaStream_t)stream));
    // An own part of one round of CTAs waits for the prefixes' shares and joins them
    // itself; a longer one would wait with its first round, and is joined afterwards
    // (64 streams over a prefix of 8192, 8 ranges: 63 and 57 us).
    const bool chunk = p->prefix.kernel == CBS_ATTN_CHUNK;
    const int sms = p->desc.num_sms > 0 ? p->desc.num_sms : kDefaultNumSMs;
    const long long taken = chunk ? std::min<long long>(sms, prefix_base * pre.split) : 0;
    const int per_sm = p->own.kernel == CBS_ATTN_CHUNK ? 1 : attn_rows_ctas(p->desc.head_dim, p->desc.cache_prec == CBS_INT8, p->own.row_tile);
    if (p->own.grid_ctas <= (sms - taken) * per_sm) return launch_attn_own(own, p->own.row_tile, (cudaStream_t)stream);
    own.share_stats = reinterpret_cast<float2 *>(at + parts.own_stats);
    own.share = reinterpret_cast<float *>(at + parts.own_share);
    CBS_TRY(launch_attn_beside(own, p->own.row_tile, (cudaStream_t)stream));
    return cuda_check(launch_join_shares(own, pre.share, pre.share_stats, (cudaStream_t)stream), "join launch");
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

static cbs_status w8_shape(int n, int k) {
    if (n < 1 || k < 1) return fail(CBS_ERR_INVALID_ARG, "bad weight shape (%d x %d)", n, k);
    if (k % 16) return fail(CBS_ERR_UNSUPPORTED, "k = %d is not a multiple of 16", k);
    if (n > 1 << 30) return fail(CBS_ERR_UNSUPPORTED, "%d outputs: at most 2^30", n);
    // (Past this the additions' errors, k / 16 of 2^-23, are over 2^-11 of what is added up.)
    if (k > 1 << 16) return fail(CBS_ERR_UNSUPPORTED, "k = %d: at most 65536", k);
    return CBS_OK;
}

cbs_status cbs_linear_w8(const int8_t *x, const float *x_scale, const int8_t *w, const float *w_scale, const float *bias,
                         void *y, int out_prec, int rows, int n, int k, int activation, void *stream) {
    CBS_TRY(float_type(out_prec, "output"));
    CBS_TRY(w8_shape(n, k));
    if (activation != CBS_ACT_SILU && activation != CBS_ACT_IDENTITY)
        return fail(CBS_ERR_INVALID_ARG, "unknown activation %d", activation);
    if (rows < 0) return fail(CBS_ERR_INVALID_ARG, "%d rows", rows);
    if (rows > 256 * kGridMax) return fail(CBS_ERR_UNSUPPORTED, "%d rows: at most %d", rows, 256 * kGridMax);
    if (rows == 0) return CBS_OK;
    CBS_TRY(need(x, "x"));
    CBS_TRY(need(x_scale, "x_scale"));
    CBS_TRY(need(w, "w"));
    CBS_TRY(need(w_scale, "w_scale"));
    CBS_TRY(may(bias, "bias"));
    CBS_TRY(need(y, "y"));
    const size_t y_bytes = (size_t)rows * n * (out_prec == CBS_BF16 ? 2 : 4);
    const struct { const void *p; size_t bytes; } inputs[] = {
        {x, (size_t)rows * k}, {x_scale, (size_t)rows * 4}, {w, (size_t)n * k}, {w_scale, (size_t)n * 4}, {bias, (size_t)n * 4}};
    for (const auto &in : inputs)
        if (overlap(y, y_bytes, in.p, in.bytes)) return fail(CBS_ERR_INVALID_ARG, "y lies on an input");
    W8Launch L;
    L.x = x; L.x_scale = x_scale; L.w = w; L.w_scale = w_scale; L.bias = bias; L.y = y;
    L.rows = rows; L.n = n; L.k = k; L.out_bf16 = out_prec == CBS_BF16; L.act = activation;
    L.status = device_status_word();
    if (!L.status) return fail(CBS_ERR_CUDA, "cannot resolve the device status word");
    return launch_w8(L, (cudaStream_t)stream);
}

cbs_status cbs_quantize_w8(const float *w, int n, int k, int8_t *codes, float *scales, void *stream) {
    CBS_TRY(w8_shape(n, k));
    CBS_TRY(need(w, "w"));
    CBS_TRY(need(codes, "codes"));
    CBS_TRY(need(scales, "scales"));
    const size_t w_bytes = (size_t)n * k * 4;
    if (overlap(codes, (size_t)n * k, w, w_bytes) || overlap(scales, (size_t)n * 4, w, w_bytes) ||
        overlap(codes, (size_t)n * k, scales, (size_t)n * 4))
        return fail(CBS_ERR_INVALID_ARG, "an output lies on the weights or another");
    return cuda_check(launch_quantize_w8(w, n, k, codes, scales, (cudaStream_t)stream), "8-bit quantiser launch");
}

}  // extern "C"
