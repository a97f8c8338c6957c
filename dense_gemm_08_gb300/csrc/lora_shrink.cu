// lora_shrink.cu -- the first product of gemm_lora: V = s_a X LA_a, each row
// with its own adapter, and the plan the second product follows (LoraPlan in
// grouped.h).
//
// Rows come in any order.  Every CTA that works on a tile of rows finds the
// tile's distinct adapters itself (tile_rows comparisons per row, in shared
// memory), in order of first appearance, so nothing is sorted and one launch
// makes both the plan and V.
//   few rows:  a cluster of up to 8 CTAs per row on the CUDA cores, K split
//              over them; a CTA's warps share the columns (K-major LA) or K
//              (rank-major LA), and the CTAs' sums meet in distributed shared
//              memory.  Each adapter's LA is read once per row that uses it,
//              which for a decode step is about once at all.
//   more rows: 128 rows at a time on the tensor cores; X times the adapters
//              of those rows, side by side in TMEM, up to 256 columns at a
//              time (a pass); each row keeps its own adapter's columns.  A
//              cluster of up to 8 CTAs splits K, as many passes run beside
//              each other as the SMs have room for, and the parts of a sum
//              are added in cluster order.
#include <atomic>
#include <mutex>

#include "grouped.cuh"
#include "internal.h"
#include "tcgen05.cuh"
#include "tma_maps.h"

namespace gemm {
namespace {

using namespace tc;

constexpr int kMaxTileRows = 256;
constexpr int kMaxCluster = 8;     // the largest portable cluster
constexpr int64_t kRowsMax = 128;  // rows the CUDA-core kernel takes
constexpr int kThreads = 256;

struct ShrinkArgs {
    LoraProblem p;
    LoraPlan plan;
    int ab_format;
    int la_z_step;  // 0 when all adapters share one LA
    int ks;         // CTAs of a cluster, each with a part of K
    uint64_t timeout_ns;
};

// The tile's distinct adapters: slot_of[i] for its n rows, list[s], and their
// number.  All kThreads (>= the tile's rows) call, with tile_id's result (the
// adapter of row threadIdx.x, -1: none).
struct TilePlan {
    int ids[kMaxTileRows];
    int slot_of[kMaxTileRows];
    int list[kMaxTileRows];
    int warp_first[kThreads / 32];
    int count;
};

__device__ __forceinline__ int tile_id(const LoraProblem &p, int64_t row0, int n) {
    int id = -1;
    if (static_cast<int>(threadIdx.x) < n) {
        id = p.adapter[row0 + threadIdx.x];
        if (id < 0 || id >= p.adapters) id = -1;
    }
    return id;
}

__device__ __forceinline__ void make_plan(int id, int n, TilePlan &t) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    t.ids[tid] = id;
    __syncthreads();
    int first = tid;  // the first row with this row's adapter
    for (int j = n - 4 + (4 - n % 4) % 4; j >= 0; j -= 4) {  // (rows past n hold -1)
        const int4 q = *reinterpret_cast<const int4 *>(&t.ids[j]);
        if (q.w == id) first = j + 3;
        if (q.z == id) first = j + 2;
        if (q.y == id) first = j + 1;
        if (q.x == id) first = j;
    }
    const bool leads = id >= 0 && first == tid;
    const uint32_t votes = __ballot_sync(0xffffffffu, leads);
    if (lane == 0) t.warp_first[warp] = __popc(votes);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += t.warp_first[w];
        all += t.warp_first[w];
    }
    const int mine = before + __popc(votes & ((1u << lane) - 1u));
    if (leads) {
        t.list[mine] = id;
        t.slot_of[tid] = mine;
    }
    if (tid == 0) t.count = all;
    __syncthreads();
    const int slot = id >= 0 ? t.slot_of[first] : -1;
    __syncthreads();
    t.slot_of[tid] = slot;
    __syncthreads();
}

__device__ __forceinline__ float widen_16(uint32_t bits, int ab_format) {
    return ab_format == 1 ? __uint_as_float(bits << 16)
                          : __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

__device__ __forceinline__ uint16_t round_16(float x, int ab_format) {
    return ab_format == 1 ? to_bf16_bits(x) : __half_as_ushort(__float2half_rn(x));
}

// x as a 16-bit value and the 16-bit rounding of what that leaves.
__device__ __forceinline__ void split_16(float x, int ab_format, uint16_t &hi, uint16_t &lo) {
    hi = round_16(x, ab_format);
    const float rest = x - widen_16(hi, ab_format);
    // (an infinite or NaN x: its remainder says nothing)
    lo = fabsf(rest) <= 3.4e38f ? round_16(rest, ab_format) : static_cast<uint16_t>(0);
}

// Eight 16-bit values (16 bytes) times eight, added to s.
template <int FMT>
__device__ __forceinline__ float dot8(const uint4 &a, const uint4 &b, float s) {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(widen_16(aw[i] & 0xffffu, FMT), widen_16(bw[i] & 0xffffu, FMT), s);
        s = fmaf(widen_16(aw[i] >> 16, FMT), widen_16(bw[i] >> 16, FMT), s);
    }
    return s;
}

// The row of V: own slot's columns from u (hi, and lo where kept), zeros in
// the tile's other slots.
__device__ __forceinline__ void write_v_row(const ShrinkArgs &a, int64_t row, int slot, int count,
                                            const float *u) {
    const LoraPlan &pl = a.plan;
    uint32_t *v = reinterpret_cast<uint32_t *>(pl.V + row * pl.ldv);
    const int half_cols = pl.rc / 2;  // 32-bit words per slot
    for (int c = threadIdx.x; c < count * half_cols; c += kThreads) {
        uint32_t word = 0;
        const int s = c / half_cols, in = (c - s * half_cols) * 2;
        if (s == slot) {
            uint16_t h0, l0, h1, l1;
            const int j = in < pl.r_pad ? in : in - pl.r_pad;
            split_16(j < a.p.rank ? u[j] : 0.f, a.ab_format, h0, l0);
            split_16(j + 1 < a.p.rank ? u[j + 1] : 0.f, a.ab_format, h1, l1);
            word = in < pl.r_pad ? (h0 | (static_cast<uint32_t>(h1) << 16))
                                 : (l0 | (static_cast<uint32_t>(l1) << 16));
        }
        v[c] = word;
    }
}

// -------------------------------------------------------- few rows: CUDA cores
__device__ __forceinline__ float load_from_rank(const float *p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                 : "=f"(v)
                 : "r"(map_to_rank(smem_addr(p), rank))
                 : "memory");
    return v;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) lora_shrink_rows_kernel(const ShrinkArgs a) {
    __shared__ alignas(16) TilePlan t;
    __shared__ float u[256];                     // this CTA's part of the row's sums
    __shared__ float part[kThreads / 32][256];
    pdl_wait();
    pdl_launch_dependents();
    const LoraProblem &p = a.p;
    const int64_t row = blockIdx.x / a.ks;
    const uint32_t rank = cluster_rank();
    const int64_t tile = row / a.plan.tile_rows, row0 = tile * a.plan.tile_rows;
    const int n = static_cast<int>(p.M - row0 < a.plan.tile_rows ? p.M - row0 : a.plan.tile_rows);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t id = p.adapter[row];
    const bool has = id >= 0 && id < p.adapters;
    // (loaded here, used after the sums)
    const int mine = rank == 0 ? tile_id(p, row0, n) : -1;
    const float scale = has && p.scale != nullptr ? p.scale[id] : 1.f;
    const int r_cols = static_cast<int>(p.rank);
    if (has) {
        const uint16_t *x = static_cast<const uint16_t *>(p.X) + row * p.ldx;
        const uint16_t *la = static_cast<const uint16_t *>(p.LA) + id * p.stride_a;
        // this CTA's K, in steps of 256
        const int64_t steps = (p.K + 255) / 256;
        const int64_t k_begin = steps * rank / a.ks * 256;
        const int64_t k_stop = steps * (rank + 1) / a.ks * 256;
        const int64_t k_end = k_stop < p.K ? k_stop : p.K;
        const int64_t k8 = k_end / 8 * 8;
        if (p.a_kmajor) {
            // two columns per warp at a time, lanes over K
            for (int c = warp * 2; c < r_cols; c += kThreads / 32 * 2) {
                const uint16_t *l0 = la + c * p.ld_a;
                const uint16_t *l1 = c + 1 < r_cols ? l0 + p.ld_a : l0;
                float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
                for (int64_t k = k_begin + lane * 8; k < k8; k += 256) {
                    const uint4 xv = __ldg(reinterpret_cast<const uint4 *>(x + k));
                    s0 = dot8<FMT>(xv, __ldg(reinterpret_cast<const uint4 *>(l0 + k)), s0);
                    s1 = dot8<FMT>(xv, __ldg(reinterpret_cast<const uint4 *>(l1 + k)), s1);
                }
                if (k8 >= k_begin && k8 + lane < k_end) {
                    const float xk = widen_16(x[k8 + lane], FMT);
                    s0 = fmaf(xk, widen_16(l0[k8 + lane], FMT), s0);
                    s1 = fmaf(xk, widen_16(l1[k8 + lane], FMT), s1);
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    s0 += __shfl_xor_sync(0xffffffffu, s0, d);
                    s1 += __shfl_xor_sync(0xffffffffu, s1, d);
                }
                if (lane == 0) {
                    u[c] = s0;
                    if (c + 1 < r_cols) u[c + 1] = s1;
                }
            }
        } else {
            // eight columns (16 bytes of a row of LA) per lane; the lanes of
            // one 8-column group and the warps share K; sums added in a fixed
            // order
            const int live = (r_cols + 7) / 8;  // groups of eight, at most 32
            int wide = 1;
            while (wide < live) wide *= 2;  // lanes per k
            const int g = lane % wide, per = 32 / wide;
            float s[8] = {};
            if (g < live) {
#pragma unroll 4
                for (int64_t k = k_begin + warp * per + lane / wide; k < k_end;
                     k += kThreads / 32 * per) {
                    const float xk = widen_16(x[k], FMT);
                    const uint16_t *lk = la + k * p.ld_a + g * 8;
                    uint32_t w[4] = {};
                    if (g * 8 + 8 <= r_cols) {
                        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(lk));
                        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
                    } else {  // the last columns of a rank that is no multiple of 8
                        for (int i = 0; i < r_cols - g * 8; ++i)
                            w[i / 2] |= static_cast<uint32_t>(lk[i]) << (i % 2 * 16);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[2 * i] = fmaf(xk, widen_16(w[i] & 0xffffu, FMT), s[2 * i]);
                        s[2 * i + 1] = fmaf(xk, widen_16(w[i] >> 16, FMT), s[2 * i + 1]);
                    }
                }
            }
            for (int d = 16; d >= wide; d >>= 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
            }
            if (lane < wide && g < live) {
#pragma unroll
                for (int i = 0; i < 8; ++i) part[warp][g * 8 + i] = s[i];
            }
            __syncthreads();
            if (tid < r_cols) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) sum += part[w][tid];
                u[tid] = sum;
            }
        }
    }
    // only the first CTA of the cluster goes on with the row
    if (rank == 0) make_plan(mine, n, t);
    __syncwarp();
    cluster_sync();  // every part is written
    if (rank == 0) {
        const int slot = t.slot_of[row - row0], count = t.count;
        if (tid == 0) a.plan.slot[row] = slot;
        if (row == row0) {
            if (tid == 0) a.plan.count[tile] = count;
            if (tid < count) a.plan.list[row0 + tid] = t.list[tid];
        }
        if (has && tid < r_cols) {
            float v[kMaxCluster];
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c)  // all in flight, then added in order
                v[c] = c < a.ks ? load_from_rank(&u[tid], c) : 0.f;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) sum += v[c];
            part[0][tid] = sum * scale;
            a.plan.part[row * a.plan.r_pad + tid] = sum * scale;
        }
        __syncthreads();
        write_v_row(a, row, slot, count, part[0]);
    }
    cluster_sync();  // the parts have been read
}

// ------------------------------------------------------ more rows: tensor cores
constexpr int kStages = 4;
constexpr int kStageA = BM * BK * 2, kStageB = 256 * BK * 2;
constexpr int kStageBytes = kStageA + kStageB;
constexpr int kTcSmem = kStages * kStageBytes + 1024;

// 16 columns of 32 lanes from TMEM.
__device__ __forceinline__ void tmem_load_16cols(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    lora_shrink_tc_kernel(const __grid_constant__ CUtensorMap map_x,
                          const __grid_constant__ CUtensorMap map_la, const ShrinkArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ alignas(16) TilePlan t;
    __shared__ int used[kMaxTileRows];  // slots of this CTA's rows
    __shared__ int pass_of[kMaxTileRows];  // a slot's pass
    __shared__ uint64_t full[kStages], empty[kStages], done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&full[s]), 1);
            mbar_init(smem_addr(&empty[s]), 1);
        }
        mbar_init(smem_addr(&done), 1);
        abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<1>(smem_addr(&tmem_slot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    const LoraProblem &p = a.p;
    const LoraPlan &pl = a.plan;
    // cluster x: parts of K; y: 128 rows each; z: every gridDim.z-th pass
    const uint32_t rank = cluster_rank();
    const int64_t row_first = static_cast<int64_t>(blockIdx.y) * BM;
    const bool first_z = blockIdx.z == 0;
    const int64_t tile = row_first / pl.tile_rows, row0 = tile * pl.tile_rows;
    const int n = static_cast<int>(p.M - row0 < pl.tile_rows ? p.M - row0 : pl.tile_rows);
    const int n_mine = static_cast<int>(p.M - row_first < BM ? p.M - row_first : BM);
    make_plan(tile_id(p, row0, n), n, t);
    const int off = static_cast<int>(row_first - row0);  // 0 or 128
    const int count = t.count;
    if (first_z && rank == 0) {
        if (row_first == row0) {
            if (tid == 0) pl.count[tile] = count;
            if (tid < count) pl.list[row0 + tid] = t.list[tid];
        }
        if (tid < n_mine) pl.slot[row_first + tid] = t.slot_of[off + tid];
    }
    // the slots that occur among this CTA's rows, in slot order
    int occurs = 0;
    if (tid < count)
        for (int i = 0; i < n_mine; ++i) occurs |= t.slot_of[off + i] == tid;
    const uint32_t votes = __ballot_sync(0xffffffffu, occurs != 0);
    if (lane == 0) t.warp_first[warp] = __popc(votes);
    __syncthreads();
    int at = __popc(votes & ((1u << lane) - 1u)), all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) at += t.warp_first[w];
        all += t.warp_first[w];
    }
    const int per_pass = 256 / pl.r_pad;  // slots whose columns fit the stage and TMEM
    if (occurs) {
        used[at] = tid;
        pass_of[tid] = at / per_pass;
    }
    __syncthreads();
    const int passes = (all + per_pass - 1) / per_pass;

    const int64_t blocks = (p.K + BK - 1) / BK;
    const int kb_begin = static_cast<int>(blocks * rank / a.ks);
    const int kb_end = static_cast<int>(blocks * (rank + 1) / a.ks);
    const uint32_t ring_base = smem_addr(ring);
    const uint32_t slot_bytes = static_cast<uint32_t>(pl.r_pad) * BK * 2;
    const int mn_block = pl.r_pad < 64 ? pl.r_pad : 64;  // rank-major LA: columns per TMA box
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    uint32_t parity = 0;
    for (int pass = blockIdx.z; pass < passes && ok; pass += gridDim.z) {
        const int first_used = pass * per_pass;
        const int ns = all - first_used < per_pass ? all - first_used : per_pass;
        if (warp == 0) {
            const uint32_t tx = kStageA + ns * slot_bytes;
            for (int kb = kb_begin; kb < kb_end; ++kb) {
                ok = __all_sync(0xffffffffu, wait_bounded(smem_addr(&empty[stage]), phase ^ 1,
                                                          abort_flag, a.timeout_ns));
                if (!ok) break;
                const uint32_t fb = smem_addr(&full[stage]);
                const uint32_t sa = ring_base + stage * kStageBytes, sb = sa + kStageA;
                if (elect_one()) {
                    mbar_arrive_expect_tx(fb, tx);
                    tma_load_2d<1>(sa, &map_x, kb * BK, static_cast<int32_t>(row_first), fb);
                }
                for (int s = 0; s < ns; ++s) {
                    const int32_t ad = t.list[used[first_used + s]] * a.la_z_step;
                    const uint32_t dst = sb + s * slot_bytes;
                    if (elect_one()) {
                        if (p.a_kmajor) {
                            tma_load_3d<1>(dst, &map_la, kb * BK, 0, ad, fb);
                        } else {
                            for (int j = 0; j < pl.r_pad; j += mn_block)
                                tma_load_3d<1>(dst + j * BK * 2, &map_la, j, kb * BK, ad, fb);
                        }
                    }
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok && lane == 0) raise_abort(abort_flag);
        } else if (warp == 1) {
            const uint64_t a_desc0 = desc_kmajor(ring_base, 0);
            const uint64_t a_step = (UMMA_K * 2) >> 4;
            // K-major LA: the slots' rows follow one another, one MMA for all;
            // rank-major: one MMA per slot, with the swizzle of its row length
            const uint32_t sw = mn_block == 64 ? kSwizzle128 : (mn_block == 32 ? kSwizzle64 : kSwizzle32);
            const uint32_t row_bytes = static_cast<uint32_t>(mn_block) * 2;
            const uint64_t b_desc0 =
                p.a_kmajor ? desc_kmajor(ring_base + kStageA, 0)
                           : smem_desc(ring_base + kStageA, BK * row_bytes, 8 * row_bytes, sw);
            const uint64_t b_step = p.a_kmajor ? (UMMA_K * 2) >> 4 : (UMMA_K * row_bytes) >> 4;
            const int n_mma = p.a_kmajor ? 1 : ns;
            const uint32_t idesc = make_idesc(BM, p.a_kmajor ? ns * pl.r_pad : pl.r_pad, 0,
                                              !p.a_kmajor, a.ab_format);
            for (int kb = kb_begin; kb < kb_end; ++kb) {
                ok = __all_sync(0xffffffffu, wait_bounded(smem_addr(&full[stage]), phase, abort_flag,
                                                          a.timeout_ns));
                if (!ok) break;
                tc_fence_after();
                const uint64_t st = static_cast<uint64_t>(stage) * (kStageBytes >> 4);
                if (elect_one()) {
                    for (int s = 0; s < n_mma; ++s)
#pragma unroll
                        for (int kk = 0; kk < BK / UMMA_K; ++kk)
                            tc_mma<1>(tmem_base + static_cast<uint32_t>(s * pl.r_pad),
                                      a_desc0 + st + kk * a_step,
                                      b_desc0 + st + s * (slot_bytes >> 4) + kk * b_step, idesc,
                                      kb > kb_begin || kk > 0 ? 1u : 0u);
                    tc_commit<1>(smem_addr(&empty[stage]));
                    if (kb + 1 == kb_end) tc_commit<1>(smem_addr(&done));
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok && lane == 0) raise_abort(abort_flag);
        }
        __syncwarp();
        // the sums are complete (every thread waits: TMEM is reused next pass)
        if (!wait_bounded(smem_addr(&done), parity, abort_flag, a.timeout_ns)) {
            raise_abort(abort_flag);
            ok = false;
        }
        parity ^= 1u;
        ok = __syncthreads_and(ok ? 1 : 0) != 0;
        if (!ok) break;
        tc_fence_after();
        // warps 0-3 and 4-7: the two halves of the pass's slots, a quarter of
        // the lanes each
        const int quarter = warp % 4;
        const int r = quarter * 32 + lane;
        const int my_slot = r < n_mine ? t.slot_of[off + r] : -1;
        const int64_t row = row_first + r;
        float *const mine = pl.part + (static_cast<int64_t>(rank) * p.M + row) * pl.r_pad;
        for (int s = warp / 4; s < ns; s += 2) {
            const int slot = used[first_used + s];
            for (int j = 0; j < pl.r_pad; j += 16) {
                uint32_t v[16];
                __syncwarp();
                tmem_load_16cols(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                     static_cast<uint32_t>(s * pl.r_pad + j), v);
                if (my_slot == slot) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        reinterpret_cast<uint4 *>(mine + j)[i] =
                            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
            }
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    // Each CTA of the cluster finishes a share of the rows: the parts of a sum
    // in cluster order, the scale, the rounding; zeros in the row's other
    // slots.  A row belongs to the z whose passes hold its slot (rows without
    // an adapter: the first).
    __threadfence();
    __syncwarp();
    cluster_sync();
    const int groups = pl.rc / 8;  // 16 bytes of V
    const int n_hi = pl.r_pad / 8;
    const int share = (n_mine + a.ks - 1) / a.ks;
    const int r_end = share * (static_cast<int>(rank) + 1) < n_mine ? share * (static_cast<int>(rank) + 1) : n_mine;
    const int r_begin = share * static_cast<int>(rank), n_share = r_end > r_begin ? r_end - r_begin : 0;
    // the rows' own slots: 8 columns per thread and step
    for (int i = tid; ok && i < n_share * n_hi; i += kThreads) {
        const int r = r_begin + i / n_hi, j = i % n_hi * 8;
        const int own = t.slot_of[off + r];
        if (own < 0 || pass_of[own] % gridDim.z != blockIdx.z) continue;
        float *const part = pl.part + (row_first + r) * pl.r_pad + j;
        float4 x[kMaxCluster], y[kMaxCluster];
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {  // all in flight, then added in order
            x[k] = y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < a.ks) {
                const float4 *q = reinterpret_cast<const float4 *>(
                    part + static_cast<int64_t>(k) * p.M * pl.r_pad);
                x[k] = __ldcg(q);
                y[k] = __ldcg(q + 1);
            }
        }
        float u[8] = {};
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
            u[0] += x[k].x, u[1] += x[k].y, u[2] += x[k].z, u[3] += x[k].w;
            u[4] += y[k].x, u[5] += y[k].y, u[6] += y[k].z, u[7] += y[k].w;
        }
        const float scale = p.scale != nullptr ? p.scale[t.list[own]] : 1.f;
        // (columns past the rank are zeros of LA, NaN beside an infinity of X)
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = j + k < p.rank ? u[k] * scale : 0.f;
        // (in the first part's place, which this thread alone has read)
        *reinterpret_cast<float4 *>(part) = make_float4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<float4 *>(part + 4) = make_float4(u[4], u[5], u[6], u[7]);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint16_t h0, l0, h1, l1;
            split_16(u[2 * k], a.ab_format, h0, l0);
            split_16(u[2 * k + 1], a.ab_format, h1, l1);
            hi[k] = h0 | (static_cast<uint32_t>(h1) << 16);
            lo[k] = l0 | (static_cast<uint32_t>(l1) << 16);
        }
        uint16_t *d = pl.V + (row_first + r) * pl.ldv + own * pl.rc + j;
        *reinterpret_cast<uint4 *>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (pl.rc > pl.r_pad)
            *reinterpret_cast<uint4 *>(d + pl.r_pad) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    // zeros in their other slots
    for (int r = r_begin + warp; ok && r < r_begin + n_share; r += kThreads / 32) {
        const int own = t.slot_of[off + r];
        const bool mine = own >= 0 ? pass_of[own] % gridDim.z == blockIdx.z : first_z;
        if (!mine) continue;
        uint4 *d = reinterpret_cast<uint4 *>(pl.V + (row_first + r) * pl.ldv);
        for (int c = lane; c < count * groups; c += 32)
            if (c / groups != own) d[c] = make_uint4(0, 0, 0, 0);
    }
    if (!ok) {
        // copies in flight land before the CTA exits
        const uint64_t t0 = global_timer();
        while (global_timer() - t0 < 2000000ull) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc<1>(tmem_base);
}

constexpr int kMaxDevices = 64;
std::once_flag g_once[kMaxDevices];
cudaError_t g_err[kMaxDevices];
int g_sms[kMaxDevices];
// The tensor-core kernel has been launched on the device (the other one waits
// for nothing).
std::atomic<bool> g_launched[kMaxDevices];

}  // namespace

// Tensor cores: CTAs that share K, so that few rows still fill the SMs (at
// least four K blocks each).
static int shrink_parts(const LoraProblem &p, int sms) {
    const int64_t tiles = (p.M + BM - 1) / BM, blocks = (p.K + BK - 1) / BK;
    int64_t ks = sms / tiles;
    if (ks > blocks / 4) ks = blocks / 4;
    if (ks > kMaxCluster) ks = kMaxCluster;
    return static_cast<int>(ks < 1 ? 1 : ks);
}

size_t lora_shrink_part_bytes(int64_t rows, int r_pad) {
    if (rows <= kRowsMax) return static_cast<size_t>(rows) * r_pad * sizeof(float);
    // parts x rows: at most SMs x 128 while there are several parts (256 SMs allowed for)
    const int64_t most = rows > 256 * BM ? rows : 256 * BM;
    const int64_t n = kMaxCluster * rows < most ? kMaxCluster * rows : most;
    return static_cast<size_t>(n) * r_pad * sizeof(float);
}

bool lora_shrink_eligible(const LoraProblem &p) {
    return p.rank <= 256 && tma_rows(p.X, p.ldx) &&
           tma_rows(p.LA, p.ld_a, p.adapters > 1 ? p.stride_a : 0);
}

cudaError_t launch_lora_shrink(const LoraProblem &p, const LoraPlan &plan, InType in,
                               cudaStream_t stream) {
    ShrinkArgs a = {};
    a.p = p;
    a.plan = plan;
    a.ab_format = in == InType::BF16 ? 1 : 0;
    a.timeout_ns = wait_limit_ns((p.K + BK - 1) / BK);
    cudaLaunchAttribute attr[2];
    set_pdl_attribute(&attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::call_once(g_once[dev], [dev] {
        g_err[dev] = cudaFuncSetAttribute(lora_shrink_tc_kernel,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
        // the split of the SM's memory that the second product's kernel needs: an
        // SM changes it only when it is empty, and both are to run on it at once
        if (g_err[dev] == cudaSuccess)
            g_err[dev] = cudaFuncSetAttribute(lora_shrink_rows_kernel<0>,
                                              cudaFuncAttributePreferredSharedMemoryCarveout,
                                              cudaSharedmemCarveoutMaxShared);
        if (g_err[dev] == cudaSuccess)
            g_err[dev] = cudaFuncSetAttribute(lora_shrink_rows_kernel<1>,
                                              cudaFuncAttributePreferredSharedMemoryCarveout,
                                              cudaSharedmemCarveoutMaxShared);
        if (g_err[dev] == cudaSuccess)
            g_err[dev] = cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev);
    });
    if (g_err[dev] != cudaSuccess) return g_err[dev];
    if (p.M <= kRowsMax) {
        // at least 512 of K per CTA, and no more CTAs than SMs: one leaves room
        // on its SM for a CTA of the second product's kernel, which streams W
        // meanwhile
        const int64_t ks = p.K / 512 < g_sms[dev] / p.M ? p.K / 512 : g_sms[dev] / p.M;
        a.ks = static_cast<int>(ks < 1 ? 1 : (ks > kMaxCluster ? kMaxCluster : ks));
        attr[1].val.clusterDim.x = static_cast<unsigned>(a.ks);
        cfg.gridDim = dim3(static_cast<unsigned>(p.M * a.ks), 1, 1);
        return in == InType::BF16 ? cudaLaunchKernelEx(&cfg, lora_shrink_rows_kernel<1>, a)
                                  : cudaLaunchKernelEx(&cfg, lora_shrink_rows_kernel<0>, a);
    }
    const bool bf16 = in == InType::BF16;
    const bool one = p.adapters == 1 || p.stride_a == 0;
    a.la_z_step = one ? 0 : 1;
    const int64_t count = one ? 1 : p.adapters, stride = one ? p.ld_a : p.stride_a;
    CUtensorMap map_x, map_la;
    bool ok = encode_stack(&map_x, bf16, p.X, p.K, p.M, p.ldx, 1, 0, BK, BM, 2);
    if (p.a_kmajor)
        ok = ok && encode_stack(&map_la, bf16, p.LA, p.K, p.rank, p.ld_a, count, stride, BK,
                                static_cast<uint32_t>(plan.r_pad), 3);
    else
        ok = ok && encode_stack(&map_la, bf16, p.LA, p.rank, p.K, p.ld_a, count, stride,
                                static_cast<uint32_t>(plan.r_pad < 64 ? plan.r_pad : 64), BK, 3,
                                plan.r_pad == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                                : plan.r_pad == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                   : CU_TENSOR_MAP_SWIZZLE_128B);
    if (!ok) return cudaErrorInvalidValue;
    const int64_t tiles = (p.M + BM - 1) / BM;
    a.ks = shrink_parts(p, g_sms[dev]);
    const int64_t slots = p.adapters < BM ? p.adapters : BM;
    const int64_t passes = (slots * plan.r_pad + 255) / 256;
    int64_t z = g_sms[dev] / (tiles * a.ks);
    z = z < 1 ? 1 : (z > passes ? passes : z);
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.ks);
    cfg.gridDim = dim3(static_cast<unsigned>(a.ks), static_cast<unsigned>(tiles),
                       static_cast<unsigned>(z));
    cfg.dynamicSmemBytes = kTcSmem;
    g_launched[dev].store(true);
    return cudaLaunchKernelEx(&cfg, lora_shrink_tc_kernel, map_x, map_la, a);
}

cudaError_t lora_shrink_read_and_clear_status(cudaStream_t stream, int *status) {
    *status = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !g_launched[dev].load()) return cudaSuccess;
    const int zero = 0;
    e = cudaMemcpyFromSymbolAsync(status, g_status, sizeof(int), 0,
                                              cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && *status != 0) {
        e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    return e;
}

}  // namespace gemm
