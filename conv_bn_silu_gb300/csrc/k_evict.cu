// k_evict.cu -- eviction from a paged cache by accumulated attention weight:
// of each sequence and key head the last `recent` positions and the heaviest
// others, `keep` in all, in order, to new pages.
//
// Two kernels.  The first chooses: a cluster takes a (sequence, head), each of
// its CTAs a run of the positions, whose weights become whole numbers of the same
// order in shared memory.  A radix selection finds the lightest weight that stays
// (11, 11 and 10 bits, from the top; the CTAs add their histograms up through
// distributed shared memory), and one scan over (heavier, equal) counts gives
// every position that stays its place, equal weights by position.  The second
// copies rows, sixteen bytes a thread: reading and writing them once bounds it.
//
// Measured, 16 sequences of up to 8192 positions, 4096 kept, 8 heads of 128: bf16 105 us;
// 8 bits 64 us, of which the choice takes 17 and the rows 47 (4.8 TB/s).
#include "tc_ptx.cuh"
#include "tc_warp.cuh"
#include "tokens.cuh"

namespace cbs {

namespace {

constexpr int kThreads = 1024, kBins = 2048, kMostCtas = 8, kRunLeast = 2048;
static_assert(kEvictRun * 4 + 3 * kBins * 4 + 1024 <= kMaxDynSmem, "a CTA's weights and its histogram");

// A weight as a whole number of the same order; a NaN above all.
__device__ __forceinline__ uint32_t ordered(float w) {
    if (w != w) return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.0f);   // (one zero)
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ int2 ld_cluster_pair(const int *p, uint32_t rank) {
    uint32_t a;
    int2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// Sum of a count over the threads before this one; one barrier.  `warps` is written
// anew by the next call but one.
__device__ __forceinline__ int scan(int v, int *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const auto inclusive = [&](int s) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(~0u, s, o);
            if (lane >= o) s += a;
        }
        return s;
    };
    const int s = inclusive(v);
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    const int before = __shfl_sync(~0u, inclusive(warps[lane]), warp ? warp - 1 : 0);
    return s - v + (warp ? before : 0);
}

// The same of a pair of counts, and over all threads.
struct Pair { int a, b; };
__device__ __forceinline__ Pair scan(Pair v, Pair &total, Pair *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const auto inclusive = [&](Pair s) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(~0u, s.a, o), b = __shfl_up_sync(~0u, s.b, o);
            if (lane >= o) s.a += a, s.b += b;
        }
        return s;
    };
    const Pair s = inclusive(v);
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    const Pair w = inclusive(warps[lane]);
    total = Pair{__shfl_sync(~0u, w.a, 31), __shfl_sync(~0u, w.b, 31)};
    const int from = warp ? warp - 1 : 0, a = __shfl_sync(~0u, w.a, from), b = __shfl_sync(~0u, w.b, from);
    return Pair{s.a - v.a + (warp ? a : 0), s.b - v.b + (warp ? b : 0)};
}

__global__ void __launch_bounds__(kThreads) evict_choose_kernel(const EvictLaunch L) {
    extern __shared__ __align__(16) uint32_t s_keys[];   // this CTA's positions, at most L.run
    __shared__ __align__(8) int s_hist[3][kBins];
    __shared__ Pair s_warps[kThreads / 32];
    __shared__ int s_totals[2][kThreads / 32];
    __shared__ int s_found[3][2];   // a pass's digit, and how many are to be taken of those that have it
    __shared__ __align__(8) int s_counts[2];   // heavier than the threshold, equal to it
    __shared__ int2 s_all[kMostCtas];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const CacheArgs &c = L.c;
    const int tid = threadIdx.x, ctas = L.ctas, rank = ctas > 1 ? (int)cluster_rank() : 0;
    const int head = blockIdx.y, b = blockIdx.z;
    const auto meet = [&] {
        if (ctas > 1) cluster_sync();
        else __syncthreads();
    };
    const int n = seq_len(c, b), after = min(n, L.keep);
    const int recent = min(n, L.recent), others = n - recent, take = after - recent;   // (recent <= keep)
    int *const kept = L.kept + ((size_t)b * c.kv_heads + head) * L.keep;
    if (rank == 0 && head == 0 && tid == 0) L.new_lens[b] = after;

    // This CTA's positions [p0, p0 + m), and each thread's run of them.  (Runs of odd
    // length: 32 lanes of a scan are in 32 banks.)
    const int share = (others + ctas - 1) / ctas, p0 = min(others, rank * share), m = min(others - p0, share);
    const int shift = c.page_shift, slots = 1 << shift;
    for (int i = tid; i < 3 * kBins; i += kThreads) s_hist[0][i] = 0;
    if (tid < 6) s_found[0][tid] = 0;
#pragma unroll 4
    for (int i = tid; i < m; i += kThreads) {
        const int pos = p0 + i, p = page_of(c, b, pos);
        // (A page outside the pool: reported; its positions go first.)
        s_keys[i] = p < 0 ? 0u : ordered(L.mass[(((size_t)p * c.kv_heads + head) << shift) + (pos & (slots - 1))]);
    }
    __syncthreads();
    uint32_t prefix = 0, mask = 0;   // the threshold's digits so far
    int left = take;                 // how many stay of those that share them
    // (A cluster's CTAs meet as often whatever they read: the lengths could change meanwhile.)
    if (ctas > 1 || (take > 0 && take < others)) {
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int shift_to = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digits = pass == 2 ? 1023u : 2047u;
            int *const hist = s_hist[pass];
            for (int i = tid; i < m; i += kThreads) {
                const uint32_t k = s_keys[i];
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift_to) & digits], 1);
            }
            meet();
            // Bins from the top: thread t has bins 2047 - 2t and 2046 - 2t, of all CTAs.
            const int top = kBins - 1 - 2 * tid;
            int x = 0, y = 0;
            if (ctas == 1) {
                x = hist[top], y = hist[top - 1];
            } else {
                int2 v[kMostCtas];
#pragma unroll
                for (int r = 0; r < kMostCtas; ++r)
                    if (r < ctas) v[r] = ld_cluster_pair(&hist[top - 1], r);
#pragma unroll
                for (int r = 0; r < kMostCtas; ++r)
                    if (r < ctas) x += v[r].y, y += v[r].x;
            }
            const int before = scan(x + y, s_totals[pass & 1]);
            if (before < left && left <= before + x) s_found[pass][0] = top, s_found[pass][1] = left - before;
            else if (before + x < left && left <= before + x + y) s_found[pass][0] = top - 1, s_found[pass][1] = left - before - x;
            __syncthreads();
            prefix |= (uint32_t)s_found[pass][0] << shift_to;
            mask |= digits << shift_to;
            left = s_found[pass][1];
        }
    }
    // Everything stays, or nothing but the recent ones, or those above `prefix` and
    // the first `left` that equal it.
    const bool all_stay = take >= others;
    const int run = ((m + kThreads - 1) / kThreads) | 1, i0 = min(m, tid * run), i1 = min(m, i0 + run);
    const auto heavier = [&](uint32_t k) { return all_stay || (take > 0 && k > prefix); };
    const auto equal = [&](uint32_t k) { return !all_stay && take > 0 && k == prefix; };
    Pair mine = {0, 0}, total;
    for (int i = i0; i < i1; ++i) mine.a += heavier(s_keys[i]), mine.b += equal(s_keys[i]);
    Pair before = scan(mine, total, s_warps);
    int place = 0, ties = 0;   // before this CTA: stayed, equal
    if (ctas > 1) {
        if (tid == 0) s_counts[0] = total.a, s_counts[1] = total.b;
        meet();
        if (tid < ctas) s_all[tid] = ld_cluster_pair(s_counts, tid);
        __syncthreads();
        for (int r = 0; r < rank; ++r) {
            place += s_all[r].x + max(0, min(s_all[r].y, left - ties));
            ties += s_all[r].y;
        }
    }
    int seen = ties + before.b;   // equal ones before this thread's
    place += before.a + min(max(left - ties, 0), before.b);
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = s_keys[i];
        const bool e = equal(k);
        if ((heavier(k) || (e && seen < left)) && place < L.keep) kept[place++] = p0 + i;
        seen += e;
    }
    for (int i = rank * kThreads + tid; i < L.keep - take; i += ctas * kThreads) kept[take + i] = i < recent ? others + i : -1;
    if (ctas > 1) cluster_sync();   // nobody's counts go while another CTA reads them
}

// Rows of K and V by the list, and what goes with them.  D * element bytes / 16
// threads a row, kSteps rows of each thread on their way at a time: fewer a thread and
// more CTAs hide the list's and the tables' loads better (16 sequences of 8192 to 4096
// in bf16: four rows 124 us, two 115; in 8 bits 78 and 74, 4.9 TB/s with the choice).
constexpr int kMoveThreads = 256, kSteps = 2;

template <int ROW>   // bytes of a row
__global__ void __launch_bounds__(kMoveThreads, 6) evict_move_kernel(const EvictLaunch L) {
    constexpr int kU = ROW / 16, kRows = kMoveThreads / kU;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const CacheArgs &c = L.c;
    const int u = threadIdx.x % kU, head = blockIdx.y, b = blockIdx.z;
    const int *const kept = L.kept + ((size_t)b * c.kv_heads + head) * L.keep;
    const int r0 = blockIdx.x * (kRows * kSteps) + threadIdx.x / kU, slots = 1 << c.page_shift;
    uint4 w[2][kSteps];
    size_t to[kSteps];
    float more[3][kSteps];   // weight and scales
    unsigned on = 0;
#pragma unroll
    for (int x = 0; x < kSteps; ++x) {
        const int r = r0 + x * kRows;
        const int pos = r < L.keep ? kept[r] : -1;
        if (pos < 0) continue;
        const int p = page_of(c, b, pos);
        const int slot = r >> c.page_shift, np = slot < L.new_max_pages ? L.new_table[(size_t)b * L.new_max_pages + slot] : -1;
        if ((unsigned)np >= (unsigned)c.num_pages) atomicOr(c.status, kStatusBadIndex);
        if (p < 0 || (unsigned)np >= (unsigned)c.num_pages) continue;
        on |= 1u << x;
        const size_t from = (((size_t)p * c.kv_heads + head) << c.page_shift) + (pos & (slots - 1));
        to[x] = (((size_t)np * c.kv_heads + head) << c.page_shift) + (r & (slots - 1));
        w[0][x] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const char *>(c.k) + from * ROW) + u);
        w[1][x] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const char *>(c.v) + from * ROW) + u);
        if (u == 0) {
            more[0][x] = L.mass[from];
            if (c.int8) more[1][x] = c.k_scale[from], more[2][x] = c.v_scale[from];
        }
    }
#pragma unroll
    for (int x = 0; x < kSteps; ++x) {
        if (!((on >> x) & 1)) continue;
        *(reinterpret_cast<uint4 *>(static_cast<char *>(c.k) + to[x] * ROW) + u) = w[0][x];
        *(reinterpret_cast<uint4 *>(static_cast<char *>(c.v) + to[x] * ROW) + u) = w[1][x];
        if (u == 0) {
            L.mass[to[x]] = more[0][x];
            if (c.int8) c.k_scale[to[x]] = more[1][x], c.v_scale[to[x]] = more[2][x];
        }
    }
}

template <int ROW>
cudaError_t launch_move(const EvictLaunch &L, cudaStream_t s) {
    constexpr int kRows = kMoveThreads / (ROW / 16) * kSteps;
    if (L.c.max_pages == 0) return cudaSuccess;   // nothing held, nothing moves
    const long long held = (long long)L.c.max_pages << L.c.page_shift, rows = L.keep < held ? L.keep : held;
    return launch_kernel(evict_move_kernel<ROW>, dim3((unsigned)((rows + kRows - 1) / kRows), L.c.kv_heads, L.c.batch), kMoveThreads, 0, s, L);
}

}  // namespace

cudaError_t launch_evict(EvictLaunch L, cudaStream_t s) {
    // Positions a CTA may meet: what the table can hold, in as few CTAs as hold it, or
    // more while each still has kRunLeast and every one an SM.  1, 2, 4 and 8 CTAs: 8
    // heads of 16000 39, 34, 28, 34 us; 128 heads of 8192 (16 sequences, 8 bits) 74, 84.
    const long long most = (long long)L.c.max_pages << L.c.page_shift, heads = (long long)L.c.kv_heads * L.c.batch;
    const auto each = [&](int ctas) { return (most + ctas - 1) / ctas; };
    L.ctas = 1;
    while (L.ctas < kMostCtas && (each(L.ctas) > kEvictRun || (each(2 * L.ctas) >= kRunLeast && 2 * L.ctas * heads <= current_device_sms()))) L.ctas *= 2;
    const int smem = (int)((most + L.ctas - 1) / L.ctas) * 4;
    static ContextOfDevice set;
    cudaError_t e = set_max_dyn_smem_once(evict_choose_kernel, smem, set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.ctas, L.c.kv_heads, L.c.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = (launch_options() & CBS_LAUNCH_PDL) ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = L.ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.ctas > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, evict_choose_kernel, L);
    if (e != cudaSuccess) return e;
    switch (L.c.head_dim * (L.c.int8 ? 1 : 2)) {
    case 64: return launch_move<64>(L, s);
    case 128: return launch_move<128>(L, s);
    default: return launch_move<256>(L, s);
    }
}

}  // namespace cbs
