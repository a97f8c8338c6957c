// group_rows.cu -- rows grouped by a number (the expert or adapter of each
// row): a stable counting sort.
//
//   offsets[g]  = rows whose number is below g (numbers outside [0, groups) do
//                 not count: those rows are dropped)
//   order[p]    = the row at place p: by number, then by row; -1 past offsets[groups]
//   position[i] = the place of row i, or -1
//
// Few rows: one CTA, one launch.  More: a first kernel counts each CTA's rows
// per group, a second places them.  A CTA has 32 warps; every warp owns a run
// of rows and a row of counters, one per group, in shared memory, so places
// do not depend on timing:
//   1. each warp counts its rows, 32 at a time (__match_any_sync finds the
//      lanes of one number);
//   2. per group, the counters of the CTA's warps become running sums; the
//      counts of the CTAs before (first kernel) and a scan over the groups
//      give the CTA's first place in each group, and the offsets;
//   3. each warp walks its rows again: place = first place + rows of the group
//      in the CTA's earlier warps and steps + rank among the warp's lanes.
// More than kGroupsPass groups take one such pass per kGroupsPass of them.
//
// The traffic is 12 bytes a row; what bounds it is latency.  One cluster of 8
// CTAs that met in distributed shared memory took 37 us for 131072 rows of 128
// groups (8 SMs issue all the scattered stores).
#include "grouped.h"

namespace gemm {
namespace {

constexpr int THREADS = 1024, WARPS = 32;
constexpr int kGroupsPass = 1024;  // 32 rows of counters: 128 KiB of shared memory at most
constexpr int kUnroll = 4;         // row numbers loaded ahead per lane
constexpr int64_t kOneCta = 2048;  // rows one CTA takes alone
constexpr int kMaxCtas = 128;

struct GroupRowsArgs {
    int64_t rows, groups;
    const int32_t *ids;
    int32_t *offsets, *order, *position;
    int pass_groups;   // counters per warp
    int64_t run;       // rows per warp (a multiple of 32)
    int32_t *counts;   // [CTAs][groups] rows of each CTA (several CTAs)
};

__global__ void __launch_bounds__(THREADS) group_count_kernel(const GroupRowsArgs a) {
    __shared__ int n[kGroupsPass];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t first = blockIdx.x * (a.run * WARPS);
    const int64_t end = first + a.run * WARPS < a.rows ? first + a.run * WARPS : a.rows;
    for (int64_t gb = 0; gb < a.groups; gb += a.pass_groups) {
        const int gc = static_cast<int>(a.groups - gb < a.pass_groups ? a.groups - gb : a.pass_groups);
        for (int g = threadIdx.x; g < gc; g += THREADS) n[g] = 0;
        __syncthreads();
        for (int64_t i = first + threadIdx.x; i < end; i += THREADS) {
            const int64_t id = static_cast<int64_t>(a.ids[i]) - gb;
            if (id >= 0 && id < gc) atomicAdd(&n[id], 1);  // (a count: any order)
        }
        __syncthreads();
        for (int g = threadIdx.x; g < gc; g += THREADS)
            a.counts[blockIdx.x * a.groups + gb + g] = n[g];
        __syncthreads();
    }
}

template <bool ONE>
__global__ void __launch_bounds__(THREADS) group_place_kernel(const GroupRowsArgs a) {
    extern __shared__ int smem[];
    int *const counts = smem;                         // [WARPS][pass_groups]
    int *const base = smem + WARPS * a.pass_groups;   // [pass_groups] first place of this CTA
    int *const parts = base + a.pass_groups;          // [2][THREADS] (several CTAs)
    __shared__ int warp_sum[WARPS];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int cta = ONE ? 0 : static_cast<int>(blockIdx.x);
    const uint32_t below_me = (1u << lane) - 1u;
    const int64_t first = (static_cast<int64_t>(cta) * WARPS + warp) * a.run;
    const int64_t end = first + a.run < a.rows ? first + a.run : a.rows;
    int *const mine = counts + warp * a.pass_groups;
    int done = 0;  // rows of the groups of earlier passes

    for (int64_t gb = 0; gb < a.groups; gb += a.pass_groups) {
        const int gc = static_cast<int>(a.groups - gb < a.pass_groups ? a.groups - gb : a.pass_groups);
        for (int g = lane; g < gc; g += 32) mine[g] = 0;
        __syncwarp();
        // a step: kUnroll times 32 rows, their numbers in this pass and the
        // lanes with the same number
        int key[kUnroll];
        uint32_t same[kUnroll], dropped = 0;
        auto load = [&](int64_t i0) {
            dropped = 0;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t i = i0 + u * 32 + lane;
                const int64_t id = i < end ? static_cast<int64_t>(a.ids[i]) : -1;
                key[u] = id >= gb && id < gb + gc ? static_cast<int>(id - gb) : -1;
                if (id < 0 || id >= a.groups) dropped |= 1u << u;
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) same[u] = __match_any_sync(0xffffffffu, key[u]);
        };
        const bool one_step = a.run <= 32 * kUnroll;  // kept for the second walk
        for (int64_t i0 = first; i0 < end; i0 += 32 * kUnroll) {
            load(i0);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (key[u] >= 0 && (same[u] & below_me) == 0) mine[key[u]] += __popc(same[u]);
                __syncwarp();
            }
        }
        // rows of group gb + tid (pass_groups <= THREADS) in all CTAs and in
        // the ones before this.  The threads split the CTAs: segment tid / wide
        // takes every (THREADS / wide)-th, all its loads in flight.
        int all = 0, before = 0;
        if constexpr (!ONE) {
            int wide = 32;
            while (wide < gc) wide *= 2;
            const int g = tid % wide, segs = THREADS / wide;
            int part_all = 0, part_before = 0;
            if (g < gc) {
                const int32_t *c = a.counts + gb + g;
#pragma unroll 8
                for (int k = tid / wide; k < static_cast<int>(gridDim.x); k += segs) {
                    const int v = c[k * a.groups];
                    part_all += v;
                    if (k < cta) part_before += v;
                }
            }
            parts[tid] = part_all;
            parts[THREADS + tid] = part_before;
            __syncthreads();
            if (tid < gc)
                for (int k = 0; k < segs; ++k) {
                    all += parts[k * wide + tid];
                    before += parts[THREADS + k * wide + tid];
                }
        }
        __syncthreads();
        for (int g = tid; g < gc; g += THREADS) {
            int run = 0;
#pragma unroll 1
            for (int w0 = 0; w0 < WARPS; w0 += 8) {  // eight loads before the first store
                int c[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) c[w] = counts[(w0 + w) * a.pass_groups + g];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    counts[(w0 + w) * a.pass_groups + g] = run;
                    run += c[w];
                }
            }
            if (ONE) all = run;
        }
        int incl = all;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            int s = warp_sum[lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, s, d);
                if (lane >= d) s += v;
            }
            warp_sum[lane] = s;
        }
        __syncthreads();
        const int start = done + (warp ? warp_sum[warp - 1] : 0) + incl - all;
        if (tid < gc) {
            base[tid] = start + before;
            if (cta == 0) a.offsets[gb + tid] = start;
        }
        done += warp_sum[WARPS - 1];
        __syncthreads();
        for (int64_t i0 = first; i0 < end; i0 += 32 * kUnroll) {
            if (!one_step) load(i0);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t i = i0 + u * 32 + lane;
                int place = -1;
                if (key[u] >= 0) {
                    place = base[key[u]] + mine[key[u]] + __popc(same[u] & below_me);
                    a.order[place] = static_cast<int32_t>(i);
                }
                if (a.position != nullptr && i < end &&
                    (key[u] >= 0 || (gb == 0 && ((dropped >> u) & 1u))))
                    a.position[i] = place;
                __syncwarp();
                if (key[u] >= 0 && (same[u] & below_me) == 0) mine[key[u]] += __popc(same[u]);
                __syncwarp();
            }
        }
        __syncthreads();  // the next pass writes the counters and sums
    }
    if (cta == 0 && tid == 0) a.offsets[a.groups] = done;
    for (int64_t p = done + static_cast<int64_t>(cta) * THREADS + tid; p < a.rows;
         p += static_cast<int64_t>(gridDim.x) * THREADS)
        a.order[p] = -1;
}

template <typename... P>
cudaError_t launch_pdl(void (*kernel)(P...), int grid, size_t smem, cudaStream_t stream,
                       const GroupRowsArgs &a) {
    cudaLaunchAttribute attr;
    set_pdl_attribute(&attr);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_group_rows(int64_t rows, int64_t groups, const int32_t *group_of_row,
                              int32_t *offsets, int32_t *order, int32_t *position,
                              cudaStream_t stream, const char **name) {
    GroupRowsArgs a = {};
    a.rows = rows;
    a.groups = groups;
    a.ids = group_of_row;
    a.offsets = offsets;
    a.order = order;
    a.position = position;
    a.pass_groups = static_cast<int>(groups < kGroupsPass ? groups : kGroupsPass);
    const bool one = rows <= kOneCta;
    const size_t smem = (static_cast<size_t>(WARPS + 1) * a.pass_groups + (one ? 0 : 2 * THREADS)) * sizeof(int);
    // without the attribute a kernel has 48 KiB, its static arrays (warp_sum) included
    constexpr size_t kStatic = 1024;
    static_assert(WARPS * sizeof(int) <= kStatic, "group_place_kernel's static arrays");
    if (smem > 48 * 1024 - kStatic) {
        const int most = static_cast<int>(((WARPS + 1) * kGroupsPass + 2 * THREADS) * sizeof(int));
        const cudaError_t e =
            one ? cudaFuncSetAttribute(group_place_kernel<true>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, most)
                : cudaFuncSetAttribute(group_place_kernel<false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    if (one) {
        *name = "group_rows";
        a.run = ((rows + WARPS - 1) / WARPS + 31) / 32 * 32;
        return launch_pdl(group_place_kernel<true>, 1, smem, stream, a);
    }
    *name = "group_rows<counted>";
    int64_t ctas = (rows + THREADS - 1) / THREADS;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    const int64_t warps = ctas * WARPS;
    a.run = ((rows + warps - 1) / warps + 31) / 32 * 32;
    void *ws = nullptr;
    cudaError_t e = workspace_alloc(static_cast<size_t>(ctas * groups) * sizeof(int32_t), stream, &ws);
    if (e != cudaSuccess) return e;
    a.counts = static_cast<int32_t *>(ws);
    e = launch_pdl(group_count_kernel, static_cast<int>(ctas), 0, stream, a);
    if (e == cudaSuccess)
        e = launch_pdl(group_place_kernel<false>, static_cast<int>(ctas), smem, stream, a);
    const cudaError_t ef = workspace_free(ws, stream);
    return e != cudaSuccess ? e : ef;
}

}  // namespace gemm
