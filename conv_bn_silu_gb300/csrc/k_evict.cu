// k_evict.cu -- eviction from a paged cache by accumulated attention weight:
// of each sequence and key head the last `recent` positions and the heaviest
// others, `keep` in all, in order, to new pages.
//
// Two kernels.  The first chooses: a cluster takes a (sequence, head), each of
// its CTAs a run of the positions, whose weights become whole numbers of the same
// order in shared memory.  A radix selection finds the lightest weight that stays
// (11, 11 and 10 bits, from the top; the CTAs' histograms meet through distributed
// shared memory, groups of 64 bins first), and one scan over (heavier, equal) counts gives
// every position that stays its place, equal weights by position.  The second
// copies rows, sixteen bytes a thread: reading and writing them once bounds it.
//
// Measured, 16 sequences of up to 8192 positions, 4096 kept, 8 heads of 128: bf16 98 us;
// 8 bits 58 us.  One of 65001, 4001 kept, 4 heads of 64: 17 us.
#include <type_traits>

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

__device__ __forceinline__ int ld_cluster_int(const int *p, uint32_t rank) {
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ int2 ld_cluster_pair(const int *p, uint32_t rank) {
    uint32_t a;
    int2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// Sum over the lanes up to this one.
__device__ __forceinline__ int inclusive(int s) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(~0u, s, o);
        if (lane >= o) s += a;
    }
    return s;
}

struct Pair { int a, b; };

__global__ void __launch_bounds__(kThreads) evict_choose_kernel(const EvictLaunch L) {
    extern __shared__ __align__(16) uint32_t s_keys[];   // this CTA's positions, at most L.run
    __shared__ __align__(8) int s_hist[3][kBins];
    __shared__ Pair s_warps[kThreads / 32];
    __shared__ int s_groups[3][kThreads / 32];   // sums of 64 bins
    __shared__ int s_found[3][2];   // a pass's digit, and how many are to be taken of those that have it
    __shared__ __align__(8) int s_counts[2];   // heavier than the threshold, equal to it
    __shared__ int2 s_all[kMostCtas];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const CacheArgs &c = L.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ctas = L.ctas, rank = ctas > 1 ? (int)cluster_rank() : 0;
    const int head = blockIdx.y, b = blockIdx.z;
    const auto meet = [&] {
        if (ctas > 1) cluster_sync();
        else __syncthreads();
    };
    const int n = seq_len(c, b), after = min(n, L.keep);
    const int recent = min(n, L.recent), others = n - recent, take = after - recent;   // (recent <= keep)
    int *const kept = L.kept + ((size_t)b * c.kv_heads + head) * L.keep;
    if (rank == 0 && head == 0 && tid == 0) L.new_lens[b] = after;

    // This CTA's positions [p0, p0 + m).
    const int share = (others + ctas - 1) / ctas, p0 = min(others, rank * share), m = min(others - p0, share);
    const int shift = c.page_shift, slots = 1 << shift;
    for (int i = tid; i < 3 * kBins; i += kThreads) s_hist[0][i] = 0;
    if (tid < 6) s_found[0][tid] = 0;
    __syncthreads();
    // Pages first, then weights, eight of each on their way at once (two where that is
    // all): what is wrong is reported behind them.  (A page outside the pool: its
    // positions go first.)  65001 positions of 4 heads 24.4 -> 16.9 us, with the groups below.
    bool bad = false;
    const auto load = [&](auto loads) {
        constexpr int kLoads = decltype(loads)::value;
        for (int i = tid; i < m; i += kLoads * kThreads) {
            int page[kLoads];
            float w[kLoads];
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
                const int at = i + x * kThreads, slot = (p0 + at) >> shift;
                page[x] = at < m && slot < c.max_pages ? c.page_table[(size_t)b * c.max_pages + slot] : -1;
            }
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
                const int pos = p0 + i + x * kThreads;
                w[x] = (unsigned)page[x] < (unsigned)c.num_pages ? L.mass[(((size_t)page[x] * c.kv_heads + head) << shift) + (pos & (slots - 1))] : 0.0f;
            }
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
                const int at = i + x * kThreads;
                if (at >= m) break;
                const bool in = (unsigned)page[x] < (unsigned)c.num_pages;
                const uint32_t key = in ? ordered(w[x]) : 0u;
                bad |= !in;
                s_keys[at] = key;
                atomicAdd(&s_hist[0][key >> 21], 1);
            }
        }
    };
    if (m <= 2 * kThreads) load(std::integral_constant<int, 2>{});
    else load(std::integral_constant<int, 8>{});
    if (bad) atomicOr(c.status, kStatusBadIndex);
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
            if (pass) {
                for (int i = tid; i < m; i += kThreads) {
                    const uint32_t k = s_keys[i];
                    if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift_to) & digits], 1);
                }
                __syncthreads();
            }
            const int2 own = *reinterpret_cast<const int2 *>(&hist[2 * tid]);
            const int sum = __reduce_add_sync(~0u, own.x + own.y);
            if (lane == 0) s_groups[pass][warp] = sum;
            meet();
            // From the top, of all CTAs: the group of 64 bins, then the bin.  (All bins of
            // all CTAs read by all threads took 4500 cycles.)  The loads have no branches
            // between them: the CTAs' answers come together.
            if (warp == 0) {
                int x = s_groups[pass][31 - lane];
                if (ctas > 1) {
                    int o[kMostCtas];
#pragma unroll
                    for (int r = 0; r < kMostCtas; ++r) o[r] = ld_cluster_int(&s_groups[pass][31 - lane], min(r, ctas - 1));
                    x = 0;
#pragma unroll
                    for (int r = 0; r < kMostCtas; ++r) x += r < ctas ? o[r] : 0;
                }
                const int before = inclusive(x) - x;
                const unsigned hit = __ballot_sync(~0u, before < left && left <= before + x);
                if (hit) {
                    const int at = __ffs(hit) - 1, rest = left - __shfl_sync(~0u, before, at), bin = (31 - at) * 64 + 62 - 2 * lane;
                    int2 v = *reinterpret_cast<const int2 *>(&hist[bin]);
                    if (ctas > 1) {
                        int2 o[kMostCtas];
#pragma unroll
                        for (int r = 0; r < kMostCtas; ++r) o[r] = ld_cluster_pair(&hist[bin], min(r, ctas - 1));
                        v = {0, 0};
#pragma unroll
                        for (int r = 0; r < kMostCtas; ++r) v.x += r < ctas ? o[r].x : 0, v.y += r < ctas ? o[r].y : 0;
                    }
                    const int above = inclusive(v.x + v.y) - (v.x + v.y);
                    if (above < rest && rest <= above + v.y) s_found[pass][0] = bin + 1, s_found[pass][1] = rest - above;
                    else if (above + v.y < rest && rest <= above + v.y + v.x) s_found[pass][0] = bin, s_found[pass][1] = rest - above - v.y;
                }
            }
            __syncthreads();
            prefix |= (uint32_t)s_found[pass][0] << shift_to;
            mask |= digits << shift_to;
            left = s_found[pass][1];
        }
    }
    // Everything stays, or nothing but the recent ones, or those above `prefix` and
    // the first `left` that equal it.
    const bool all_stay = take >= others;
    const auto heavier = [&](uint32_t k) { return all_stay || (take > 0 && k > prefix); };
    const auto equal = [&](uint32_t k) { return !all_stay && take > 0 && k == prefix; };
    // A warp takes a run of the positions, 32 at a time.
    const int run = (m + kThreads - 1) / kThreads * 32, i0 = min(m, warp * run), i1 = min(m, i0 + run);
    Pair mine = {0, 0};
    for (int i = i0; i < i1; i += 32) {
        const uint32_t k = i + lane < i1 ? s_keys[i + lane] : 0u;
        mine.a += __popc(__ballot_sync(~0u, i + lane < i1 && heavier(k)));
        mine.b += __popc(__ballot_sync(~0u, i + lane < i1 && equal(k)));
    }
    if (lane == 0) s_warps[warp] = mine;
    __syncthreads();
    const Pair upto = {inclusive(s_warps[lane].a), inclusive(s_warps[lane].b)};
    const Pair total = {__shfl_sync(~0u, upto.a, 31), __shfl_sync(~0u, upto.b, 31)};
    const Pair before = {__shfl_sync(~0u, upto.a, warp) - mine.a, __shfl_sync(~0u, upto.b, warp) - mine.b};
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
    int seen = ties + before.b;   // equal ones before this warp's
    place += before.a + min(max(left - ties, 0), before.b);
    const unsigned below = (1u << lane) - 1u;
    for (int i = i0; i < i1; i += 32) {
        const bool in = i + lane < i1;
        const uint32_t k = in ? s_keys[i + lane] : 0u;
        const bool e = in && equal(k);
        const unsigned equals = __ballot_sync(~0u, e);
        const bool stays = (in && heavier(k)) || (e && seen + __popc(equals & below) < left);
        const unsigned staying = __ballot_sync(~0u, stays);
        const int at = place + __popc(staying & below);
        if (stays && at < L.keep) kept[at] = p0 + i + lane;
        place += __popc(staying);
        seen += __popc(equals);
    }
    for (int i = rank * kThreads + tid; i < L.keep - take; i += ctas * kThreads) kept[take + i] = i < recent ? others + i : -1;
    if (ctas > 1) cluster_sync();   // nobody's counts go while another CTA reads them
}

// Rows of K and V by the list, and what goes with them.  D * element bytes / 16
// threads a row, kSteps rows of each thread on their way at a time: fewer a thread and
// more CTAs hide the list's and the tables' loads better (16 sequences of 8192 to 4096
// in bf16: four rows 105 us, two 98; in 8 bits 63 and 58).
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
    // Places, pages, rows: each step's on their way at once.  What is wrong is reported
    // behind them.
    int pos[kSteps], page[kSteps], new_page[kSteps];
    bool bad = false;
#pragma unroll
    for (int x = 0; x < kSteps; ++x) {
        const int r = r0 + x * kRows;
        pos[x] = r < L.keep ? kept[r] : -1;
    }
#pragma unroll
    for (int x = 0; x < kSteps; ++x) {
        const int slot = pos[x] >> c.page_shift, new_slot = (r0 + x * kRows) >> c.page_shift;
        page[x] = pos[x] >= 0 && slot < c.max_pages ? c.page_table[(size_t)b * c.max_pages + slot] : -1;
        new_page[x] = pos[x] >= 0 && new_slot < L.new_max_pages ? L.new_table[(size_t)b * L.new_max_pages + new_slot] : -1;
    }
#pragma unroll
    for (int x = 0; x < kSteps; ++x) {
        if (pos[x] < 0) continue;
        if ((unsigned)page[x] >= (unsigned)c.num_pages || (unsigned)new_page[x] >= (unsigned)c.num_pages) {
            bad = true;
            continue;
        }
        on |= 1u << x;
        const size_t from = (((size_t)page[x] * c.kv_heads + head) << c.page_shift) + (pos[x] & (slots - 1));
        to[x] = (((size_t)new_page[x] * c.kv_heads + head) << c.page_shift) + ((r0 + x * kRows) & (slots - 1));
        w[0][x] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const char *>(c.k) + from * ROW) + u);
        w[1][x] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const char *>(c.v) + from * ROW) + u);
        if (u == 0) {
            more[0][x] = L.mass[from];
            if (c.int8) more[1][x] = c.k_scale[from], more[2][x] = c.v_scale[from];
        }
    }
    if (bad) atomicOr(c.status, kStatusBadIndex);
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
    // heads of 16000 39, 34, 28, 34 us (the latter two 25.0 and 25.4 with the loads side by
    // side), 8 heads of 4000 2 and 4 CTAs 21.1, 22.8; 128 heads of 8192, 1 and 2, 74, 84.
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
