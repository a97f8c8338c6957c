// group_rows.cu -- rows grouped by a number (the expert or adapter of each
// row), in one kernel: a stable counting sort.
//
//   offsets[g]  = rows whose number is below g (numbers outside [0, groups) do
//                 not count: those rows are dropped)
//   order[p]    = the row at place p: by number, then by row; -1 past offsets[groups]
//   position[i] = the place of row i, or -1
//
// One cluster of CTAs (one CTA when there are few rows) of 32 warps.  Every
// warp owns a run of rows and a row of counters, one per group, in shared
// memory, so counting needs no atomics and places do not depend on timing:
//   1. each warp counts its rows, 32 at a time (__match_any_sync finds the
//      lanes of one number);
//   2. per group, the counters of the CTA's warps become running sums; the
//      CTAs' totals meet through distributed shared memory, and a scan over
//      the groups gives the offsets;
//   3. each warp walks its rows again: place = group's start + rows of the
//      group in earlier CTAs, warps and steps + rank among the warp's lanes.
// More than kGroupsPass groups take one such pass per kGroupsPass of them.
#include "grouped.h"

namespace gemm {
namespace {

constexpr int THREADS = 1024, WARPS = 32;
constexpr int kGroupsPass = 1024;  // 32 rows of counters: 128 KiB of shared memory at most
constexpr int kCluster = 8;        // the largest portable cluster
constexpr int kUnroll = 8;         // row numbers loaded ahead per lane

__device__ __forceinline__ uint32_t shared_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A word of the same shared-memory object in CTA `rank` of the cluster.
__device__ __forceinline__ int load_from_rank(const int *p, uint32_t rank) {
    uint32_t addr;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(shared_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

struct GroupRowsArgs {
    int64_t rows, groups;
    const int32_t *ids;
    int32_t *offsets, *order, *position;
    int pass_groups;  // counters per warp
    int64_t run;      // rows per warp (a multiple of 32)
};

template <int CL>
__global__ void __launch_bounds__(THREADS) group_rows_kernel(const GroupRowsArgs a) {
    extern __shared__ int smem[];
    int *const counts = smem;                              // [WARPS][pass_groups]
    int *const total = smem + WARPS * a.pass_groups;       // [pass_groups] this CTA's rows
    int *const base = total + a.pass_groups;               // [pass_groups] first place of this CTA
    __shared__ int warp_sum[WARPS];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t rank = CL == 1 ? 0u : blockIdx.x;  // one cluster: CTA number = cluster rank
    const uint32_t below_me = (1u << lane) - 1u;
    const int64_t first = (static_cast<int64_t>(rank) * WARPS + warp) * a.run;
    const int64_t end = first + a.run < a.rows ? first + a.run : a.rows;
    int *const mine = counts + warp * a.pass_groups;
    int done = 0;  // rows of the groups of earlier passes

    for (int64_t gb = 0; gb < a.groups; gb += a.pass_groups) {
        const int gc = static_cast<int>(a.groups - gb < a.pass_groups ? a.groups - gb : a.pass_groups);
        for (int g = lane; g < gc; g += 32) mine[g] = 0;
        __syncwarp();
        for (int64_t i0 = first; i0 < end; i0 += 32 * kUnroll) {
            int key[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t i = i0 + u * 32 + lane;
                const int64_t id = i < end ? static_cast<int64_t>(a.ids[i]) - gb : -1;
                key[u] = id >= 0 && id < gc ? static_cast<int>(id) : -1;
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const uint32_t same = __match_any_sync(0xffffffffu, key[u]);
                if (key[u] >= 0 && (same & below_me) == 0) mine[key[u]] += __popc(same);
                __syncwarp();
            }
        }
        __syncthreads();
        for (int g = tid; g < gc; g += THREADS) {
            int run = 0;
            for (int w = 0; w < WARPS; ++w) {
                const int c = counts[w * a.pass_groups + g];
                counts[w * a.pass_groups + g] = run;
                run += c;
            }
            total[g] = run;
        }
        if constexpr (CL > 1)
            cluster_sync_all();
        else
            __syncthreads();
        // (pass_groups <= THREADS: one group per thread)
        int all = 0, before = 0;
        if (tid < gc) {
            if constexpr (CL > 1) {
#pragma unroll
                for (uint32_t c = 0; c < CL; ++c) {
                    const int n = load_from_rank(total + tid, c);
                    if (c < rank) before += n;
                    all += n;
                }
            } else {
                all = total[tid];
            }
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
            if (rank == 0) a.offsets[gb + tid] = start;
        }
        done += warp_sum[WARPS - 1];
        __syncthreads();
        for (int64_t i0 = first; i0 < end; i0 += 32 * kUnroll) {
            int key[kUnroll];
            uint32_t dropped = 0;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t i = i0 + u * 32 + lane;
                const int64_t id = i < end ? static_cast<int64_t>(a.ids[i]) : -1;
                key[u] = id >= gb && id < gb + gc ? static_cast<int>(id - gb) : -1;
                if (id < 0 || id >= a.groups) dropped |= 1u << u;
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t i = i0 + u * 32 + lane;
                const uint32_t same = __match_any_sync(0xffffffffu, key[u]);
                int place = -1;
                if (key[u] >= 0) {
                    place = base[key[u]] + mine[key[u]] + __popc(same & below_me);
                    a.order[place] = static_cast<int32_t>(i);
                }
                if (a.position != nullptr && i < end &&
                    (key[u] >= 0 || (gb == 0 && ((dropped >> u) & 1u))))
                    a.position[i] = place;
                __syncwarp();
                if (key[u] >= 0 && (same & below_me) == 0) mine[key[u]] += __popc(same);
                __syncwarp();
            }
        }
        // every CTA has read the others' totals (and its own counters) before
        // the next pass writes them, or the CTA leaves
        if constexpr (CL > 1)
            cluster_sync_all();
        else
            __syncthreads();
    }
    if (rank == 0 && tid == 0) a.offsets[a.groups] = done;
    for (int64_t p = done + static_cast<int64_t>(rank) * THREADS + tid; p < a.rows;
         p += static_cast<int64_t>(CL) * THREADS)
        a.order[p] = -1;
}

template <int CL>
cudaError_t launch_cl(const GroupRowsArgs &a, size_t smem, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(group_rows_kernel<CL>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>((WARPS + 2) * kGroupsPass * sizeof(int)));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    set_pdl_attribute(&attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CL, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, group_rows_kernel<CL>, a);
}

}  // namespace

cudaError_t launch_group_rows(int64_t rows, int64_t groups, const int32_t *group_of_row,
                              int32_t *offsets, int32_t *order, int32_t *position,
                              cudaStream_t stream, const char **name) {
    GroupRowsArgs a;
    a.rows = rows;
    a.groups = groups;
    a.ids = group_of_row;
    a.offsets = offsets;
    a.order = order;
    a.position = position;
    a.pass_groups = static_cast<int>(groups < kGroupsPass ? groups : kGroupsPass);
    // one CTA while its warps have at most kUnroll steps of 32 rows each
    const int cl = rows <= WARPS * 32 * kUnroll ? 1 : kCluster;
    const int64_t warps = static_cast<int64_t>(cl) * WARPS;
    a.run = ((rows + warps - 1) / warps + 31) / 32 * 32;
    const size_t smem = static_cast<size_t>(WARPS + 2) * a.pass_groups * sizeof(int);
    *name = cl == 1 ? "group_rows" : "group_rows<cluster>";
    return cl == 1 ? launch_cl<1>(a, smem, stream) : launch_cl<kCluster>(a, smem, stream);
}

}  // namespace gemm
