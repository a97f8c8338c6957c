// fused_tc.cu -- the fused products on the sm_103a tensor cores (BF16 or FP16
// inputs, FP32 accumulation).
//
//   forward:  Z = alpha op(A) op(B) + bias, D = act(Z) + residual, Z kept or not
//   gradient: D = alpha op(A) op(B) * act'(pre), and D's column sums
//
// One warp fills a ring of 128-byte-swizzled stages by TMA, one issues
// tcgen05.mma into one of two TMEM accumulators, eight finish the other one.
// Large problems: CTA pairs on tiles of 256 x 256.  Others: single CTAs, tiles of
// up to 128 rows and 64, 128 or 256 columns, persistent; or, when there are fewer
// tiles than SMs, K split over the CTAs of a cluster, which add each other's sums
// through distributed shared memory in the order of the pieces.
//
// The epilogue takes blocks of 32 rows and 64 columns, a row per lane.  What is
// read beside the sums (residual, pre) comes by TMA into a box of shared memory
// ahead of time -- the next block's, or the next tile's first, while a block is
// computed -- and D leaves from the same box by TMA, so that the epilogue's memory
// traffic costs the warps a few 16-byte accesses per lane.  Rows that do not start
// on 16 bytes move through the same boxes by ordinary loads and stores.
//
// Bound by the tensor cores, and by power on the largest: 8192 x 14336 x 4096 BF16
// with bias, GELU and Z kept 523 to 532 us (1810 to 1840 TFLOP/s), 590 in a long row of
// calls; the gradient with column sums 600 to 627, without 550.  Small ones by a
// tile's start, its chain of MMAs and its epilogue, one after the other: 1000 x 2049
// x 1408 FP16 20 us.
#include <atomic>
#include <mutex>
#include <type_traits>

#include "fused.cuh"
#include "internal.h"
#include "tc_epilogue.cuh"
#include "tcgen05.cuh"
#include "tma_maps.h"

namespace gemm {
namespace {

using namespace tc;

constexpr int kGroupM = 16;     // tile rows per band of the raster
constexpr int kMaxStages = 16;
constexpr int kEpiWarps = 8;
constexpr int kProducer = kEpiWarps, kIssuer = kEpiWarps + 1;
constexpr int kBox = 4096;      // 32 rows of 64 16-bit values
constexpr int kBody = 224 * 1024;  // ring and boxes
constexpr int kBiasBytes = kEpiWarps * 32 * 4;
// ring and boxes, 32 bias values per epilogue warp, barriers, alignment
constexpr int kSmemBytes = 1024 + kBody + kBiasBytes + 512;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
constexpr int kMaxSplit = 8;
constexpr int kSlot = 8192;     // 32 x 64 FP32 sums of another piece

// Column sums of a long K: sums in parts.  The tensor cores cut what an addition to
// the accumulator cannot hold (they do not round it): half a unit of its last place on the
// mean for 16 steps of K, so that a sum of random signs comes out smaller by 1e-9 of itself per
// step (of one sign 1.3e-9; FP16, whose products are cut too, 5e-9).  A D of 16 bits
// does not show it, the FP32 sums of its columns do (4.5e-6 at K = 4096, 0.6e-6 for
// FP32 products).  Where they are wanted and a tile's K is longer than a part, each part
// is summed in the other accumulator and the epilogue warps add the parts in registers:
// 0.7e-6 (BF16) to 0.95e-6 (FP16) at any K, 1.0e-6 and 3.9e-6 for products of one sign.
// The 128 registers per thread that this takes come from the
// other warps.  (Measured at 8192 x 14336 x 4096: parts of 768 602 us, of 896 588, of
// 1280 -- two of which cover a tile's epilogue -- 560 with an error of
// 1.2e-6, one part 573.  At K = 1408 two parts 19.9 us, one 18.5: an error of 1.7e-6.)
// The piece of K of a cluster's CTA is summed in parts too, side by side in TMEM: its one
// tile leaves room for them, and they are added as they are read (64 x 1000, K = 8192:
// 16.5 us, 16.2 with a piece of 1024 in one; 300 x 1024 25.9 and 24.9; 128 x 2048, K = 10000,
// whose pieces would be too long in one and were not split, 24.2 and 34).
constexpr int kPart = 768;
static_assert(kPart % (4 * BK) == 0, "a part is a number of steps");
constexpr int kEpiRegs = 216, kOtherRegs = 72, kPartsRegs = 168;
static_assert(2 * kEpiRegs + kOtherRegs <= 3 * kPartsRegs,
              "three warpgroups share the launch's registers");
template <bool PARTS>
constexpr int threads() {
    return PARTS ? 384 : 64 + 32 * kEpiWarps;
}

struct Args {
    int64_t M, N;
    uint32_t tiles_m, tiles_n;
    int num_kb, ksub, ks;  // steps of K (stages), blocks of 64 per step, pieces
    int part_steps;        // of K in a part (a piece's: as many as it has, if it is not cut)
    int bn, am;
    int stages, ring_bytes, boxes;
    uint32_t stage_bytes, a_region;
    int a_kmajor, b_kmajor, b_blocks, ab_format;
    float alpha;
    const float *bias;
    int act;
    void *D, *pre;
    const void *in;  // forward: residual; gradient: pre
    int64_t ldd, ld_pre, ld_in;
    int tma_d, tma_pre, tma_in;     // rows start on 16 bytes
    int even_d, even_pre, even_in;  // rows start on 4 bytes
    float *part;  // gradient: sums of the 32-row blocks' columns, [blocks][N], or null
    uint64_t timeout_ns;
};

struct Tile {
    int64_t m0, n0;
    int m_valid;  // its rows, 1 .. am * CG
};

template <int CG>
__device__ __forceinline__ bool get_tile(const Args &a, uint32_t w, Tile &t) {
    if (w >= a.tiles_m * a.tiles_n) return false;
    const uint32_t width = kGroupM * a.tiles_n;
    const uint32_t band = w / width, in_band = w - band * width;
    const uint32_t rest = a.tiles_m - band * kGroupM, high = rest < kGroupM ? rest : kGroupM;
    const uint32_t q = in_band / high;
    const int rows = a.am * CG;
    t.n0 = static_cast<int64_t>(q) * a.bn;
    t.m0 = static_cast<int64_t>(band * kGroupM + (in_band - q * high)) * rows;
    t.m_valid = a.M - t.m0 < rows ? static_cast<int>(a.M - t.m0) : rows;
    return true;
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                              uint32_t d) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_u32(uint32_t at, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, int32_t c0, int32_t c1,
                                             uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Eight 16-bit values as FP32.
template <int TYPE>
__device__ __forceinline__ void widen(const uint4 &q, float *v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == kOutBf16) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
template <int ACT>
__device__ __forceinline__ void activate_16(float (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = quick_activation<ACT>(v[j]);
}
template <int ACT>
__device__ __forceinline__ void slope_8(float *v, const float (&z)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= quick_slope<ACT>(z[j]);
}

// The sum of the 32 lanes' v[j] for column j = lane / 2, in a fixed order.
__device__ __forceinline__ float column_sum(float (&v)[16]) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) {
        const bool high = (lane & (2 * s)) != 0;
#pragma unroll
        for (int j = 0; j < s; ++j) {
            const float give = high ? v[j] : v[j + s], keep = high ? v[j + s] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * s);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// 32 lanes x 16 columns of 32-bit TMEM words.
__device__ __forceinline__ void tmem_load_16cols(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
}

// 32 lanes x 64 columns, one wait for two loads.
__device__ __forceinline__ void tmem_load_64cols(uint32_t taddr, float (&v)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]),
          "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
          "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]),
          "=f"(v[39]), "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]),
          "=f"(v[46]), "=f"(v[47]), "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]),
          "=f"(v[53]), "=f"(v[54]), "=f"(v[55]), "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]),
          "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
        : "r"(taddr + 32));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    // (nothing is read before the wait)
#pragma unroll
    for (int j = 0; j < 64; ++j) asm volatile("" : "+f"(v[j]));
}

// 16-byte piece p of row r of a box (128-byte swizzle).
__device__ __forceinline__ uint32_t piece_at(int r, int p) { return r * 128 + ((p ^ (r & 7)) << 4); }

// Sixteen values of this lane's row, from column h * 16 of the box on, rounded.
template <int TYPE>
__device__ __forceinline__ void narrow_16(const float (&v)[16], uint32_t box, int lane, int h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (TYPE == kOutBf16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
            const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
    st_shared_v4(box + piece_at(lane, h * 2), w[0], w[1], w[2], w[3]);
    st_shared_v4(box + piece_at(lane, h * 2 + 1), w[4], w[5], w[6], w[7]);
}

// A box's rows to memory, and back, where TMA cannot: two values per lane and row.
__device__ __forceinline__ void box_to_rows(uint32_t box, void *D, int64_t ldd, int64_t row0, int nrows,
                                            int64_t c0, int width, bool even) {
    const int lane = threadIdx.x % 32, c = lane * 2;
    uint16_t *d = static_cast<uint16_t *>(D) + row0 * ldd + c0 + c;
    if (c >= width) return;
#pragma unroll 4
    for (int r = 0; r < nrows; ++r, d += ldd) {
        const uint32_t w = ld_shared_u32(box + piece_at(r, lane / 4) + lane % 4 * 4);
        if (even && c + 1 < width) {
            *reinterpret_cast<uint32_t *>(d) = w;
        } else {
            d[0] = static_cast<uint16_t>(w);
            if (c + 1 < width) d[1] = static_cast<uint16_t>(w >> 16);
        }
    }
}
__device__ __forceinline__ void rows_to_box(uint32_t box, const void *from, int64_t ld, int64_t row0,
                                            int nrows, int64_t c0, int width, bool even) {
    const int lane = threadIdx.x % 32, c = lane * 2;
    const uint16_t *s = static_cast<const uint16_t *>(from) + row0 * ld + c0 + c;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 8) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t *at = s + (r0 + i) * ld;
            w[i] = 0;
            if (r0 + i >= nrows || c >= width) continue;
            if (even && c + 1 < width) {
                w[i] = *reinterpret_cast<const uint32_t *>(at);
            } else {
                w[i] = at[0];
                if (c + 1 < width) w[i] |= static_cast<uint32_t>(at[1]) << 16;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            st_shared_u32(box + piece_at(r0 + i, lane / 4) + lane % 4 * 4, w[i]);
    }
}

template <int CG, bool SPLIT, bool GRAD, int TYPE, bool PARTS>
__global__ void __launch_bounds__(threads<PARTS>(), 1)
    fused_tc_kernel(const __grid_constant__ CUtensorMap map_a,
                    const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ CUtensorMap map_b_edge,
                    const __grid_constant__ CUtensorMap map_in,
                    const __grid_constant__ CUtensorMap map_d,
                    const __grid_constant__ CUtensorMap map_pre,
                    const __grid_constant__ Args args) {
    static_assert(!SPLIT || CG == 1, "K is split over single CTAs");
    static_assert(!PARTS || (GRAD && !SPLIT), "parts are for column sums");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    // barriers (8 bytes each): full[kMaxStages] TMA -> MMA (the leader's count
    // both CTAs), empty[kMaxStages] MMA -> TMA, tfull[2] MMA -> epilogue,
    // tempty[2] epilogue -> MMA (the leader's count both CTAs), drain,
    // ibar[kEpiWarps] boxes of residual / pre loaded
    const uint32_t ring0 = smem_addr(ring);
    const uint32_t bias0 = ring0 + kBody;
    const uint32_t full0 = bias0 + kBiasBytes, empty0 = full0 + 8 * kMaxStages;
    const uint32_t tfull0 = empty0 + 8 * kMaxStages, tempty0 = tfull0 + 16;
    const uint32_t drain = tempty0 + 16, ibar0 = drain + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ring + (ibar0 + 8 * kEpiWarps - ring0));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = CG == 1 && !SPLIT ? 0u : cluster_rank();
    const bool leader = CG == 1 || rank == 0;
    const int group = SPLIT ? args.ks : CG;  // CTAs that share a tile
    const uint32_t first_tile = blockIdx.x / group, tile_step = gridDim.x / group;

    if (threadIdx.x == 32) {
        // (the maps are fetched while another warp sets up the barriers)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_b)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_in)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_d)) : "memory");
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < args.stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, kEpiWarps * CG);
        }
        mbar_init(drain, 1);
        for (int e = 0; e < kEpiWarps; ++e) mbar_init(ibar0 + 8 * e, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == kIssuer) tmem_alloc<CG>(smem_addr(tmem_slot));
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2 || SPLIT) cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    const int stages = args.stages, ksub = args.ksub;
    const uint32_t stage_bytes = args.stage_bytes, a_region = args.a_region;
    const int b_rows = args.bn / CG;  // columns of B this CTA loads
    // this CTA's steps of K
    const int kb_first = SPLIT ? static_cast<int>(static_cast<int64_t>(args.num_kb) * rank / args.ks) : 0;
    const int kb_end =
        SPLIT ? static_cast<int>(static_cast<int64_t>(args.num_kb) * (rank + 1) / args.ks) : args.num_kb;
    const int nkb = kb_end - kb_first;
    Tile t;
    bool aborted = false;
    // every lane waits (the warp stays converged); false: gave up
    auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
        const bool done = __all_sync(
            0xffffffffu, wait_bounded(bar, parity, abort_flag, args.timeout_ns));
        if (!done && lane == 0) raise_abort(abort_flag);
        return done;
    };

    if constexpr (PARTS) {
        if (warp >= kEpiWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    }
    if (warp == kProducer) {
        // -------------------------------------------------------- TMA producer
        const uint32_t count0 = CG == 1 ? full0 : map_to_rank(full0, 0);
        const uint32_t a_rows = args.a_kmajor ? static_cast<uint32_t>(args.am) : 128u;
        const uint32_t tx = static_cast<uint32_t>(CG) *
                            (a_rows + static_cast<uint32_t>(b_rows)) * static_cast<uint32_t>(ksub) * 128u;
        int stage = 0;
        uint32_t phase = 0, issued = 0;
        bool ok = true, reverse = false;
        for (uint32_t w = first_tile; ok && get_tile<CG>(args, w, t); w += tile_step, reverse = !reverse) {
            const int32_t b0 = static_cast<int32_t>(t.n0 + (CG == 2 ? rank : 0u) * b_rows);
            const int32_t m0 = static_cast<int32_t>(t.m0 + (CG == 2 ? rank : 0u) * BM);
            // CTA pairs: every other tile walks K backwards and starts on what the
            // tile before it read last.  Single CTAs start at different steps:
            // columns of B are a power of two apart as a rule, and CTAs in step
            // would read the same few DRAM channels at once.
            int kb = CG == 2 ? (reverse ? nkb - 1 : 0)
                             : static_cast<int>((w * 5u) % static_cast<uint32_t>(nkb));
            for (int i = 0; i < nkb; ++i) {
                ok = wait_all(empty0 + 8 * stage, phase ^ 1);
                if (!ok) break;
                const uint32_t fb = count0 + 8 * stage;
                const uint32_t sa = ring0 + stage * stage_bytes, sb = sa + a_region;
                if (elect_one()) {
                    if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, tx);
                    // several blocks of 64 at once: the maps count K in blocks
                    const int32_t block = (kb_first + kb) * ksub;
                    const int32_t k_in = ksub > 1 ? 0 : block * BK, k_block = ksub > 1 ? block : 0;
                    if (args.b_kmajor) {
                        tma_load_4d<CG>(sb, &map_b, k_in, b0, k_block, 0, fb);
                    } else if ((static_cast<int64_t>(b0) + b_rows) / 64 <= args.b_blocks) {
                        tma_load_4d<CG>(sb, &map_b, 0, block * BK, b0 / 64, 0, fb);
                    } else {
                        for (int j = 0; j < b_rows; j += 64)
                            tma_load_3d<CG>(sb + j * 128 * ksub, &map_b_edge, b0 + j, block * BK, 0, fb);
                    }
                    if (args.a_kmajor) {
                        tma_load_3d<CG>(sa, &map_a, k_in, m0, k_block, fb);
                    } else {
                        tma_load_2d<CG>(sa, &map_a, m0, block * BK, fb);
                        tma_load_2d<CG>(sa + 8192, &map_a, m0 + 64, block * BK, fb);
                    }
                }
                if (CG == 2 && reverse)
                    --kb;
                else
                    kb = kb + 1 == nkb ? 0 : kb + 1;
                issued += issued < static_cast<uint32_t>(stages) ? 1u : 0u;
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        __syncwarp();
        // the copies in flight land before the CTA exits (the leader's barriers
        // count both CTAs' bytes)
        if (lane == 0 && leader) {
            for (uint32_t i = 0; i < issued; ++i) {
                if (--stage < 0) {
                    stage = stages - 1;
                    phase ^= 1;
                }
                const volatile int never = 0;
                if (!wait_bounded(full0 + 8 * stage, phase, &never, args.timeout_ns))
                    raise_abort(abort_flag);
            }
        }
        aborted = !ok;
        __syncwarp();
    } else if (warp == kIssuer) {
        // ---------------------------------------------------------- MMA issuer
        if (leader) {
            const bool a_mn = !args.a_kmajor, b_mn = !args.b_kmajor;
            const uint64_t a_desc0 = a_mn ? desc_mnmajor(ring0, 0) : desc_kmajor(ring0, 0);
            const uint64_t b_desc0 =
                b_mn ? smem_desc(ring0 + a_region, static_cast<uint32_t>(ksub) * 8192u, 1024)
                     : desc_kmajor(ring0 + a_region, 0);
            const uint64_t a_step = (a_mn ? UMMA_K * 128 : UMMA_K * 2) >> 4;
            const uint64_t b_step = (b_mn ? UMMA_K * 128 : UMMA_K * 2) >> 4;
            // a step's blocks of 64: rows x 128 bytes apart (N-major: 64 rows of K)
            const uint64_t a_sub = static_cast<uint64_t>(args.am) * 128u >> 4;
            const uint64_t b_sub = b_mn ? 8192u >> 4 : static_cast<uint64_t>(b_rows) * 128u >> 4;
            const uint64_t stage_step = stage_bytes >> 4;
            const uint32_t idesc = make_idesc(BM * CG, args.bn, a_mn, b_mn, args.ab_format);
            int stage = 0;
            uint32_t phase = 0, acc = 0;
            bool ok = true;
            for (uint32_t w = first_tile; ok && get_tile<CG>(args, w, t); w += tile_step) {
                uint32_t d_tmem = 0;
                auto take = [&]() {  // the accumulator not filled last, once it has been read
                    ok = wait_all(tempty0 + 8 * (acc & 1), ((acc >> 1) & 1) ^ 1);
                    tc_fence_after();
                    d_tmem = tmem_base + (acc & 1) * 256;
                };
                take();
                if (!ok) break;
                int in_part = 0;
                for (int i = 0; i < nkb; ++i, ++in_part) {
                    if (PARTS && in_part == args.part_steps) {
                        if (elect_one()) tc_commit<CG>(tfull0 + 8 * (acc & 1));
                        ++acc;
                        take();
                        if (!ok) break;
                        in_part = 0;
                    }
                    if (SPLIT && in_part == args.part_steps) {  // the next columns of TMEM
                        d_tmem += static_cast<uint32_t>(args.bn);
                        in_part = 0;
                    }
                    ok = wait_all(full0 + 8 * stage, phase);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = a_desc0 + static_cast<uint64_t>(stage) * stage_step;
                    const uint64_t bd = b_desc0 + static_cast<uint64_t>(stage) * stage_step;
                    if (elect_one()) {
                        tc_mma<CG>(d_tmem, ad, bd, idesc, in_part > 0 ? 1u : 0u);
                        tc_mma<CG>(d_tmem, ad + a_step, bd + b_step, idesc, 1u);
                        tc_mma<CG>(d_tmem, ad + 2 * a_step, bd + 2 * b_step, idesc, 1u);
                        tc_mma<CG>(d_tmem, ad + 3 * a_step, bd + 3 * b_step, idesc, 1u);
                        for (int u = 1; u < ksub; ++u) {
                            const uint64_t au = ad + u * a_sub, bu = bd + u * b_sub;
                            tc_mma<CG>(d_tmem, au, bu, idesc, 1u);
                            tc_mma<CG>(d_tmem, au + a_step, bu + b_step, idesc, 1u);
                            tc_mma<CG>(d_tmem, au + 2 * a_step, bu + 2 * b_step, idesc, 1u);
                            tc_mma<CG>(d_tmem, au + 3 * a_step, bu + 3 * b_step, idesc, 1u);
                        }
                        tc_commit<CG>(empty0 + 8 * stage);  // frees the stage (both CTAs)
                    }
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                if (elect_one()) tc_commit<CG>(tfull0 + 8 * (acc & 1));
                ++acc;
            }
            __syncwarp();
            // all MMAs issued here have finished once `drain` completes
            if (elect_one()) {
                tc_commit_local<CG>(drain);
                const volatile int never = 0;
                if (!wait_bounded(drain, 0, &never, args.timeout_ns)) raise_abort(abort_flag);
            }
            aborted = !ok;
        }
        __syncwarp();
    }

    if (SPLIT || warp < kEpiWarps) {
    if constexpr (PARTS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // Epilogue warps: two per quarter of the TMEM lanes, each takes every other
    // block of 64 columns.
    const int e = warp, quarter = warp % 4, half = (e / 4) & 1;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // A block's box: residual / pre comes into it and D leaves from it.  With a residual
    // or pre there are two in turn, so that the next block's is fetched while this
    // block is computed (8192 x 8192 x 512 with a residual: 84 us with one box for it and
    // one for D, now 75).
    const uint32_t box_0 = ring0 + args.ring_bytes + (e & 7) * args.boxes * kBox;
    const uint32_t box_pre = box_0 + kBox;  // (forward with pre kept)
    const uint32_t other = args.in != nullptr ? (args.boxes - 1) * kBox : 0;
    uint32_t box = box_0, flip = 0;  // this block's; which one is the next block's
    const uint32_t bias_at = bias0 + (e & 7) * 128;
    const uint32_t ibar = ibar0 + 8 * (e & 7);
    const bool has_in = args.in != nullptr;
    const bool has_pre = !GRAD && args.pre != nullptr;
    uint32_t blocks_in = 0;  // boxes fetched by TMA and read
    bool pending = false;    // one is on its way

    int nrows = 0, n_blocks = 0;
    int64_t row0 = 0;
    // what this warp does of tile t
    auto place = [&](const Tile &tile, int64_t &r0, int &rows, int &blocks) {
        const int first = (CG == 2 ? static_cast<int>(rank) * BM : 0) + quarter * 32;
        const int left = tile.m_valid - first;
        rows = left < 0 ? 0 : (left > 32 ? 32 : left);
        r0 = tile.m0 + first;
        const int64_t cols = args.N - tile.n0;
        const int wide = cols < args.bn ? static_cast<int>(cols) : args.bn;
        blocks = rows > 0 ? (wide + 63) / 64 : 0;
    };
    auto fetch_in = [&](int64_t r0, int64_t c0) {
        // (this warp's own reads of the box are over)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (elect_one()) {
            bulk_wait_read();  // (its last D has left)
            mbar_arrive_expect_tx(ibar, kBox);
            tma_load_2d<CG>(box_0 + flip * other, &map_in, static_cast<int32_t>(c0), static_cast<int32_t>(r0),
                            CG == 1 ? ibar : map_to_rank(ibar, rank));
        }
        __syncwarp();
        pending = true;
    };

    // Before a block is written: its residual / pre is in its box, and what the boxes
    // held before has left.  False: gave up.
    auto open_block = [&](int64_t c0, int width) -> bool {
        const bool fetched = has_in && args.tma_in;
        if (fetched && !pending) fetch_in(row0, c0);
        box = box_0 + flip * other;
        flip ^= 1;
        if (!fetched || has_pre) {
            if (elect_one()) bulk_wait_read();
            __syncwarp();
        }
        if (fetched) {
            if (!wait_all(ibar, blocks_in & 1)) return false;
            ++blocks_in;
            pending = false;
        } else if (has_in) {
            rows_to_box(box, args.in, args.ld_in, row0, nrows, c0, width, args.even_in != 0);
            __syncwarp();
        }
        return true;
    };
    // After: the boxes go to memory.
    auto close_block = [&](int64_t c0, int width) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        // (TMA stores whole 16-byte pieces, and its box is 64 columns wide: a block with
        // an odd end, or cut by the tile's, goes by rows)
        const bool whole = width == 64 || (args.N % 8 == 0 && c0 + width == args.N);
        if (args.tma_d && whole) {
            if (elect_one())
                tma_store_2d(&map_d, static_cast<int32_t>(c0), static_cast<int32_t>(row0), box);
        } else {
            box_to_rows(box, args.D, args.ldd, row0, nrows, c0, width, args.even_d != 0);
        }
        if (has_pre) {
            if (args.tma_pre && whole) {
                if (elect_one())
                    tma_store_2d(&map_pre, static_cast<int32_t>(c0), static_cast<int32_t>(row0), box_pre);
            } else {
                box_to_rows(box_pre, args.pre, args.ld_pre, row0, nrows, c0, width, args.even_pre != 0);
            }
        }
        __syncwarp();
    };

    // Gradient: sixteen values times the slopes at pre's, from column h * 16 of the block.
    auto times_slopes = [&](float (&v)[16], int h) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float x[8];
            widen<TYPE>(ld_shared_u4(box + piece_at(lane, h * 2 + p)), x);
            if (args.act == kActGelu)
                slope_8<kActGelu>(v + p * 8, x);
            else if (args.act == kActSilu)
                slope_8<kActSilu>(v + p * 8, x);
            else if (args.act == kActRelu)
                slope_8<kActRelu>(v + p * 8, x);
        }
    };
    // The sums of those sixteen columns over the block's rows.
    auto add_columns = [&](float (&v)[16], int64_t c0, int h, int width) {
        if (lane >= nrows) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.f;
        }
        const float sum = column_sum(v);
        const int c = h * 16 + lane / 2;
        if (lane % 2 == 0 && c < width) args.part[row0 / 32 * args.N + c0 + c] = sum;
    };

    // One block: 64 columns from tile column b * 64 on.  sums(h, v): the product's
    // columns h * 16 .. of this lane's row; after(): all sums have been read; next():
    // fetches the next box.  False: gave up.  (Sixteen columns at a time, in a loop
    // that is not unrolled: a tile that is alone on its SM runs its epilogue once,
    // and fetching straight-line code for 64 columns took most of 3 us.)
    auto finish_block = [&](int b, auto &&sums, auto &&after, auto &&next) -> bool {
        const int64_t c0 = t.n0 + b * 64;
        const int in_tile = args.bn - b * 64 < 64 ? args.bn - b * 64 : 64;
        const int width = args.N - c0 < in_tile ? static_cast<int>(args.N - c0) : in_tile;
        float bias2[2] = {0.f, 0.f};
        if (!GRAD && args.bias != nullptr) {
            if (lane < width) bias2[0] = __ldg(args.bias + c0 + lane);
            if (lane + 32 < width) bias2[1] = __ldg(args.bias + c0 + lane + 32);
        }
        if (!open_block(c0, width)) return false;
#pragma unroll 1
        for (int h = 0; h * 16 < in_tile; ++h) {
            if (!GRAD && args.bias != nullptr && (h & 1) == 0) {
                __syncwarp();
                st_shared_f32(bias_at + lane * 4, h == 0 ? bias2[0] : bias2[1]);
                __syncwarp();
            }
            float v[16];
            sums(h, v);
            if ((h + 1) * 16 >= in_tile) after();
            if (!GRAD && args.bias != nullptr) {
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 q = ld_shared_v4(bias_at + (h & 1) * 64 + j * 4);
                    v[j] = fmaf(args.alpha, v[j], q.x), v[j + 1] = fmaf(args.alpha, v[j + 1], q.y);
                    v[j + 2] = fmaf(args.alpha, v[j + 2], q.z), v[j + 3] = fmaf(args.alpha, v[j + 3], q.w);
                }
            } else if (args.alpha != 1.f) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] *= args.alpha;
            }
            if constexpr (!GRAD) {
                if (has_pre) {
                    narrow_16<TYPE>(v, box_pre, lane, h);
                }
                if (args.act == kActGelu)
                    activate_16<kActGelu>(v);
                else if (args.act == kActSilu)
                    activate_16<kActSilu>(v);
                else if (args.act == kActRelu)
                    activate_16<kActRelu>(v);
            }
            if (has_in) {
                if constexpr (GRAD) {
                    times_slopes(v, h);
                } else {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        float x[8];
                        widen<TYPE>(ld_shared_u4(box + piece_at(lane, h * 2 + p)), x);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[p * 8 + j] += x[j];
                    }
                }
            }
            narrow_16<TYPE>(v, box, lane, h);
            if (GRAD && args.part != nullptr) add_columns(v, c0, h, width);
            if (h == 0 && has_in && args.tma_in) next();
        }
        close_block(c0, width);
        return true;
    };

    if constexpr (!SPLIT) {
        if (warp < kEpiWarps) {
            uint32_t acc = 0;
            for (uint32_t w = first_tile; get_tile<CG>(args, w, t); w += tile_step) {
                place(t, row0, nrows, n_blocks);
                const int last = n_blocks > half ? half + (n_blocks - 1 - half) / 2 * 2 : -1;
                if (has_in && args.tma_in && last >= 0 && !pending) fetch_in(row0, t.n0 + half * 64);
                uint32_t buf = 0, t_acc = 0;  // the accumulator being read
                auto next_acc = [&]() -> bool {
                    buf = acc & 1;
                    t_acc = tmem_base + lane_off + buf * 256;
                    if (!wait_all(tfull0 + 8 * buf, (acc >> 1) & 1)) return false;
                    tc_fence_after();
                    ++acc;
                    return true;
                };
                auto release_acc = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 1)
                            mbar_arrive(tempty0 + 8 * buf);
                        else
                            mbar_arrive_cluster(map_to_rank(tempty0 + 8 * buf, 0));
                    }
                };
                auto fetch_next = [&](int b) {  // the box after block b's
                    if (b != last) {
                        fetch_in(row0, t.n0 + (b + 2) * 64);
                        return;
                    }
                    Tile u;  // the next tile's first block
                    int64_t r0;
                    int rows, blocks;
                    if (!get_tile<CG>(args, w + tile_step, u)) return;
                    place(u, r0, rows, blocks);
                    if (blocks > half) fetch_in(r0, u.n0 + half * 64);
                };
                if constexpr (PARTS) {
                    // the parts' sums of this warp's four times 32 columns (indices fixed
                    // at compile time)
                    float run[4][32] = {};
                    for (int from = 0; from < nkb; from += args.part_steps) {
                        if (!next_acc()) {
                            aborted = true;
                            break;
                        }
#pragma unroll
                        for (int q = 0; q < 4; q += 2) {
                            if (half + q > last) continue;
                            float raw[64];
                            __syncwarp();
                            tmem_load_64cols(t_acc + (half + q) * 64, raw);
#pragma unroll
                            for (int j = 0; j < 64; ++j) run[q + j / 32][j % 32] += raw[j];
                        }
                        release_acc();
                    }
                    // (Four sixteens of columns in a row: 10.6 us a tile one by one, 602 us
                    // against 640 in all.  By way of shared memory, which the multiplication
                    // keeps busy, it took 18.)
#pragma unroll 4
                    for (int g = 0; g < 8 && !aborted; ++g) {
                        const int b = half + 2 * (g / 4), h = g % 4;
                        if (b > last) break;
                        const int64_t c0 = t.n0 + b * 64;
                        const int in_tile = args.bn - b * 64 < 64 ? args.bn - b * 64 : 64;
                        const int width = args.N - c0 < in_tile ? static_cast<int>(args.N - c0) : in_tile;
                        if (h == 0 && !open_block(c0, width)) {
                            aborted = true;
                            break;
                        }
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (i != g) continue;
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = args.alpha * run[i / 2][i % 2 * 16 + j];
                        }
                        if (has_in) times_slopes(v, h);
                        narrow_16<TYPE>(v, box, lane, h);
                        add_columns(v, c0, h, width);
                        if (h == 0 && has_in && args.tma_in) fetch_next(b);
                        if (h == 3) close_block(c0, width);
                    }
                    if (aborted) break;
                    continue;
                }
                if (!next_acc()) {
                    aborted = true;
                    break;
                }
                for (int b = half; b < n_blocks && !aborted; b += 2) {
                    aborted = !finish_block(
                        b,
                        [&](int h, float (&v)[16]) {
                            __syncwarp();
                            tmem_load_16cols(t_acc + b * 64 + h * 16, v);
                        },
                        [&]() {
                            if (b == last) release_acc();
                        },
                        [&]() { fetch_next(b); });
                }
                if (aborted) break;
                if (last < 0) release_acc();
            }
        }
    } else {
        // The pieces' sums: each 32 x 64 block has one owner among the cluster's
        // CTAs, which adds the others' to its own.  The blocks travel into the
        // owners' rings, which nothing uses once every piece is multiplied.
        const bool mine = get_tile<CG>(args, first_tile, t) && warp < kEpiWarps;
        int quarters = 0;
        if (mine) {
            place(t, row0, nrows, n_blocks);
            quarters = (t.m_valid + 31) / 32;
            if (!wait_all(tfull0, 0)) aborted = true;
            tc_fence_after();
        }
        const uint32_t t_acc = tmem_base + lane_off;
        // this CTA's sums of sixteen columns: its parts of K, in their order
        auto own_sums = [&](int b, int h, float (&v)[16]) {
            const uint32_t at = t_acc + b * 64 + h * 16;
            __syncwarp();
            tmem_load_16cols(at, v);
#pragma unroll 1
            for (int from = args.part_steps, q = 1; from < nkb; from += args.part_steps, ++q) {
                float more[16];
                tmem_load_16cols(at + q * args.bn, more);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += more[j];
            }
        };
        cluster_sync();
        auto owner_of = [&](int b, int &slot) -> int {
            const int u = b * quarters + quarter;
            slot = u / args.ks * (args.ks - 1);
            return u % args.ks;
        };
        if (mine) {
            for (int b = half; b < n_blocks; b += 2) {
                int slot;
                const int owner = owner_of(b, slot);
                if (owner == static_cast<int>(rank)) continue;
                // (a slot per other piece, in their order)
                slot += static_cast<int>(rank) - (static_cast<int>(rank) > owner ? 1 : 0);
                const uint32_t to = map_to_rank(ring0 + slot * kSlot + lane * 256, owner);
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    float v[16];
                    own_sums(b, h, v);
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        st_cluster_v4(to + (((h * 4 + p) ^ (lane & 15)) << 4), __float_as_uint(v[p * 4]),
                                      __float_as_uint(v[p * 4 + 1]), __float_as_uint(v[p * 4 + 2]),
                                      __float_as_uint(v[p * 4 + 3]));
                }
            }
        }
        cluster_sync();
        if (mine && !aborted) {
            for (int b = half; b < n_blocks && !aborted; b += 2) {
                int slot;
                if (owner_of(b, slot) != static_cast<int>(rank)) continue;
                aborted = !finish_block(
                    b,
                    [&](int h, float (&v)[16]) {
                        float own[16];
                        own_sums(b, h, own);
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = 0.f;
#pragma unroll 1
                        for (int q = 0; q < args.ks; ++q) {
                            if (q == static_cast<int>(rank)) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) v[j] += own[j];
                                continue;
                            }
                            const int at = slot + q - (q > static_cast<int>(rank) ? 1 : 0);
                            const uint32_t from = ring0 + at * kSlot + lane * 256;
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                const float4 f = ld_shared_v4(from + (((h * 4 + p) ^ (lane & 15)) << 4));
                                v[p * 4] += f.x, v[p * 4 + 1] += f.y;
                                v[p * 4 + 2] += f.z, v[p * 4 + 3] += f.w;
                            }
                        }
                    },
                    [] {}, [] {});
            }
        }
    }
    if (warp < kEpiWarps) {
        // a box that was fetched for nothing lands, and D is written
        if (pending) wait_all(ibar, blocks_in & 1);
        __syncwarp();
        if (elect_one()) bulk_wait_all();
        __syncwarp();
    }
    }

    if (aborted) {
        // give copies issued by a peer that gave up a short time to land
        const uint64_t t0 = global_timer();
        while (global_timer() - t0 < 2000000ull) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2 || SPLIT) cluster_sync();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc<CG>(tmem_base);
}

// ---------------------------------------------------------------- host side
constexpr int kMaxDevices = 64;
constexpr int64_t kMaxTiles = int64_t(1) << 30;  // the tile arithmetic is 32-bit

std::atomic<bool> g_launched[kMaxDevices];

template <int CG, bool SPLIT, bool GRAD, int TYPE, bool PARTS>
cudaLaunchConfig_t config(int grid, int cluster, cudaStream_t stream, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(threads<PARTS>(), 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    set_pdl_attribute(&attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

// Prepares a kernel on device `dev` before its first launch there; resident[c]:
// clusters of c CTAs the device holds at once (0: none, or not asked).
struct Prepared {
    std::once_flag once;
    cudaError_t err = cudaSuccess;
    int resident[kMaxSplit + 1] = {};
};
template <int CG, bool SPLIT, bool GRAD, int TYPE, bool PARTS>
const Prepared &prepared(int dev) {
    static Prepared all[kMaxDevices];
    Prepared &p = all[dev];
    std::call_once(p.once, [&p, dev] {
        const auto kernel = fused_tc_kernel<CG, SPLIT, GRAD, TYPE, PARTS>;
        if (PARTS) {
            // the warpgroups divide what the launch gives: without it they would wait
            cudaFuncAttributes at;
            p.err = cudaFuncGetAttributes(&at, kernel);
            if (p.err == cudaSuccess && at.numRegs != kPartsRegs) p.err = cudaErrorInvalidKernelImage;
            if (p.err != cudaSuccess) return;
        }
        p.err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (p.err != cudaSuccess) return;
        int sms = 0;
        p.err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (p.err != cudaSuccess) return;
        p.resident[1] = sms > 0 ? sms : 1;
        for (int c = 2; c <= (CG == 2 ? 2 : SPLIT ? kMaxSplit : 1); c *= 2) {
            cudaLaunchAttribute attr[2];
            cudaLaunchConfig_t cfg = config<CG, SPLIT, GRAD, TYPE, PARTS>(c, c, 0, attr);
            cfg.attrs = attr + 1;  // the occupancy query takes the cluster shape only
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&p.resident[c], kernel, &cfg) != cudaSuccess) {
                p.resident[c] = 0;
                (void)cudaGetLastError();  // that cluster size is then not used
            }
        }
    });
    return p;
}

struct Maps {
    CUtensorMap a, b, b_edge, in, d, pre;
};

template <int CG, bool SPLIT, bool GRAD, int TYPE, bool PARTS>
cudaError_t launch_as(const Maps &m, const Args &a, int dev, int grid, int cluster,
                      cudaStream_t stream) {
    g_launched[dev].store(true);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config<CG, SPLIT, GRAD, TYPE, PARTS>(grid, cluster, stream, attr);
    return cudaLaunchKernelEx(&cfg, fused_tc_kernel<CG, SPLIT, GRAD, TYPE, PARTS>, m.a, m.b, m.b_edge, m.in, m.d,
                              m.pre, a);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A way to cut the product: CTAs per tile's accumulator, rows and columns of a tile
// (per CTA and in all), pieces of K.
struct Cut {
    int cg, am, bn, ks;
};

// Blocks of 64 of K per step: a copy takes the producer about 100 ns to issue
// whatever its size, while a 128 x 128 tile multiplies a block in 130 ns.  The
// copies of K-major operands then count K in blocks of 64, which needs K to be a
// multiple of 64.
int sub_blocks(const FusedProblem &p, const Cut &c) {
    if (c.cg == 2 || p.K % BK != 0 || !p.a_kmajor) return 1;
    const int64_t piece = ceil_div(p.K, BK) / c.ks;
    int ksub = 1;
    while (ksub < 4 && c.bn * 2 * ksub <= 256 && (c.am + c.bn) * 128 * 2 * ksub <= 65536 &&
           piece >= 4 * ksub)
        ksub *= 2;
    return ksub;
}

// Steps of K that one accumulator of a cluster's CTA adds.
int piece_part_steps(const FusedProblem &p, const Cut &c) {
    const int ksub = sub_blocks(p, c);
    const int64_t piece = ceil_div(ceil_div(p.K, BK * ksub), c.ks);
    return static_cast<int>(p.grad && p.dbias != nullptr && piece > kPart / (BK * ksub) ? kPart / (BK * ksub)
                                                                                        : piece);
}
// Its parts lie side by side in TMEM (and are read 64 columns at a time).
bool parts_fit(const FusedProblem &p, const Cut &c) {
    const int64_t piece = ceil_div(ceil_div(p.K, BK * sub_blocks(p, c)), c.ks);
    const int64_t parts = ceil_div(piece, piece_part_steps(p, c));
    return parts * (c.bn > 64 ? c.bn : 64) <= kTmemCols;
}

// The cut whose slowest CTA is done first, by a model in microseconds fitted to 1022
// measured times (90 shapes from 8 x 512 x 512 to 4096 x 4096 x 14336, every cut;
// the cuts that it picks are 1.4 % slower than the best ones on the mean, 21 % at
// most; the times themselves are met within 10 %):
//   a block of 64 of K    the longest of its MMAs (0.27 for 128 x 256 or a pair's 256 x
//                         256), its bytes at 109 GB/s per SM, and its step's copies (0.16)
//   a tile's epilogue     3.0 + 1.7 per block of 64 columns of a warp, beside the next
//                         tile's sum where there is one
//   a launch              2.0, a pair 1.7 more; an exchange of pieces 2.0 and 1.5 per
//                         64 columns of 128 rows
//   all operands          once at 6.4 TB/s; tiles of 32 columns read at 0.6 of that
Cut choose_cut(const FusedProblem &p, const Prepared &pair, const Prepared &split, int sms) {
    const int64_t kb = ceil_div(p.K, BK);
    const double bytes = 2.0 * (static_cast<double>(p.M) * p.K + static_cast<double>(p.K) * p.N);
    Cut best = {1, BM, 256, 1};
    double least = 1e300;
    auto consider = [&](const Cut &c, int64_t slots) {
        if (slots <= 0) return;
        const int64_t tiles = ceil_div(p.M, c.am * c.cg) * ceil_div(p.N, c.bn);
        const double rounds = static_cast<double>(ceil_div(tiles, slots));
        double block = 0.27 * c.bn / 256;
        const double l2 = (c.am + c.bn / c.cg) * 128 / 109e3, issue = 0.16 / sub_blocks(p, c);
        block = l2 > block ? l2 : block;
        block = issue > block ? issue : block;
        const double multiply = static_cast<double>(ceil_div(kb, c.ks)) * block;
        const double epilogue = 3.0 + 1.7 * (c.bn == 32 ? 0.5 : (c.bn + 127) / 128);
        const double reads = bytes / (c.bn == 32 ? 3.8e6 : 6.4e6);
        double whole = (rounds - 1) * (multiply > epilogue ? multiply : epilogue) + multiply;
        if (reads > whole) whole = reads;
        const double cost = 2.0 + (c.cg == 2 ? 1.7 : 0.0) + whole + epilogue +
                            (c.ks > 1 ? 2.0 + 1.5 * ((c.bn + 63) / 64) * c.am / BM : 0.0);
        if (cost < least) least = cost, best = c;
    };
    if (p.M > BM) consider({2, BM, 256, 1}, pair.resident[2]);
    const int am = !p.a_kmajor || p.M > 64 ? BM : (p.M <= 16 ? 16 : (p.M <= 32 ? 32 : 64));
    for (int bn : {256, 128, 64, 32}) {
        if (bn > 64 && p.N <= bn / 2) continue;
        if (bn == 32 && !p.b_kmajor) continue;  // (N-major copies are 64 columns wide)
        consider({1, am, bn, 1}, sms);
        for (int ks = 2; ks <= kMaxSplit; ks *= 2) {
            const int64_t tiles = ceil_div(p.M, am) * ceil_div(p.N, bn);
            if (kb >= 2 * ks && tiles <= split.resident[ks] && parts_fit(p, {1, am, bn, ks}))
                consider({1, am, bn, ks}, split.resident[ks]);
        }
    }
    return best;
}

}  // namespace

bool fused_tc_eligible(const FusedProblem &p) {
    return p.K > 0 && tma_rows(p.A, p.lda) && tma_rows(p.B, p.ldb) &&
           ceil_div(p.M, 16) * ceil_div(p.N, 32) < kMaxTiles;
}

template <bool GRAD, int TYPE>
static cudaError_t launch_tc_as(const FusedProblem &p, int dev, cudaStream_t stream,
                                const char **name) {
    constexpr bool bf16 = TYPE == kOutBf16;
    const Prepared &pair = prepared<2, false, GRAD, TYPE, false>(dev);
    const Prepared &one = prepared<1, false, GRAD, TYPE, false>(dev);
    const Prepared &split = prepared<1, true, GRAD, TYPE, false>(dev);
    for (const Prepared *q : {&pair, &one, &split})
        if (q->err != cudaSuccess) return q->err;
    const Cut cut = choose_cut(p, pair, split, one.resident[1]);
    Args a = {};
    a.M = p.M;
    a.N = p.N;
    a.am = cut.am;
    a.bn = cut.bn;
    a.ks = cut.ks;
    a.ksub = sub_blocks(p, cut);
    a.num_kb = static_cast<int>(ceil_div(p.K, BK * a.ksub));
    a.part_steps = cut.ks > 1 ? piece_part_steps(p, cut) : kPart / (BK * a.ksub);
    a.tiles_m = static_cast<uint32_t>(ceil_div(p.M, cut.am * cut.cg));
    a.tiles_n = static_cast<uint32_t>(ceil_div(p.N, cut.bn));
    a.a_kmajor = p.a_kmajor;
    a.b_kmajor = p.b_kmajor;
    a.b_blocks = static_cast<int>(p.N / 64);
    a.ab_format = bf16 ? 1 : 0;
    a.alpha = p.alpha;
    a.bias = p.bias;
    a.act = p.act;
    a.D = p.D;
    a.ldd = p.ldd;
    a.in = GRAD ? p.pre : p.residual;
    a.ld_in = GRAD ? p.ld_pre : p.ld_r;
    a.pre = GRAD ? nullptr : p.pre;
    a.ld_pre = p.ld_pre;
    a.tma_d = tma_rows(a.D, a.ldd);
    a.tma_in = a.in != nullptr && tma_rows(a.in, a.ld_in);
    a.tma_pre = a.pre != nullptr && tma_rows(a.pre, a.ld_pre);
    a.even_d = reinterpret_cast<uintptr_t>(a.D) % 4 == 0 && a.ldd % 2 == 0;
    a.even_in = reinterpret_cast<uintptr_t>(a.in) % 4 == 0 && a.ld_in % 2 == 0;
    a.even_pre = reinterpret_cast<uintptr_t>(a.pre) % 4 == 0 && a.ld_pre % 2 == 0;
    // ring and boxes share the body.  With am < 128 the MMA's operand runs on past A into
    // B and the next stages, in the last stage past it: its first block of 64 stays inside
    // the ring, its second (tiles of 32 columns) may reach 4 KB into the boxes.  Whatever lies
    // there reaches only accumulator rows that are not stored.
    a.boxes = 1 + (a.pre != nullptr) + (a.in != nullptr);
    a.ring_bytes = kBody - kEpiWarps * a.boxes * kBox;
    a.a_region = static_cast<uint32_t>((p.a_kmajor ? a.am : BM) * a.ksub) * BK * 2;
    a.stage_bytes = a.a_region + static_cast<uint32_t>(a.bn / cut.cg * a.ksub) * BK * 2;
    const int over = BM * BK * 2 - static_cast<int>(a.stage_bytes);
    const int fit = (a.ring_bytes - (over > 0 ? over : 0)) / static_cast<int>(a.stage_bytes);
    a.stages = fit < kMaxStages ? fit : kMaxStages;
    a.timeout_ns = wait_limit_ns(ceil_div(p.K, BK));

    Maps m;
    bool ok = p.a_kmajor ? encode_kmajor(&m.a, bf16, p.A, p.K, p.M, p.lda, 1, p.lda, a.am, a.ksub, 3)
                         : encode_stack(&m.a, bf16, p.A, p.M, p.K, p.lda, 1, 0, 64, BK, 2);
    if (p.b_kmajor)
        ok = ok && encode_kmajor(&m.b, bf16, p.B, p.K, p.N, p.ldb, 1, p.ldb, a.bn / cut.cg, a.ksub, 4);
    else
        ok = ok && encode_nmajor(&m.b, &m.b_edge, bf16, p.B, p.N, p.K, p.ldb, 1, p.ldb,
                                 a.bn / cut.cg, a.ksub);
    if (p.b_kmajor) m.b_edge = m.b;
    m.in = m.d = m.pre = m.a;
    auto rows_map = [&](CUtensorMap *map, const void *base, int64_t ld) {
        return encode_stack(map, bf16, base, p.N, p.M, ld, 1, 0, 64, 32, 2);
    };
    if (a.tma_d) ok = ok && rows_map(&m.d, a.D, a.ldd);
    if (a.tma_in) ok = ok && rows_map(&m.in, a.in, a.ld_in);
    if (a.tma_pre) ok = ok && rows_map(&m.pre, a.pre, a.ld_pre);
    if (!ok) return cudaErrorInvalidValue;

    // the column sums of blocks of 32 rows, added by a second kernel
    const int64_t blocks = ceil_div(p.M, 32);
    void *ws = nullptr;
    cudaError_t e = cudaSuccess;
    if (GRAD && p.dbias != nullptr) {
        a.part = p.dbias;
        if (blocks > 1) {
            e = workspace_alloc(static_cast<size_t>(blocks * p.N) * sizeof(float), stream, &ws);
            if (e != cudaSuccess) return e;
            a.part = static_cast<float *>(ws);
        }
    }
    const int64_t tiles = static_cast<int64_t>(a.tiles_m) * a.tiles_n;
    static const char *const kNames[3][2] = {{"fused_tc<f16>", "fused_tc<bf16>"},
                                             {"fused_tc<f16,pair>", "fused_tc<bf16,pair>"},
                                             {"fused_tc<f16,split>", "fused_tc<bf16,split>"}};
    *name = kNames[cut.ks > 1 ? 2 : cut.cg - 1][bf16];
    // a pair, or one CTA, takes tile after tile (all variants fill an SM: as many run)
    const auto launch_tiles = [&](auto parts) -> cudaError_t {
        constexpr bool PARTS = decltype(parts)::value;
        const Prepared &q = cut.cg == 2 ? prepared<2, false, GRAD, TYPE, PARTS>(dev)
                                        : prepared<1, false, GRAD, TYPE, PARTS>(dev);
        if (q.err != cudaSuccess) return q.err;
        const int n = static_cast<int>(tiles < q.resident[cut.cg] ? tiles : q.resident[cut.cg]);
        if (n == 0) return cudaErrorInvalidConfiguration;
        return cut.cg == 2 ? launch_as<2, false, GRAD, TYPE, PARTS>(m, a, dev, 2 * n, 2, stream)
                           : launch_as<1, false, GRAD, TYPE, PARTS>(m, a, dev, n, 1, stream);
    };
    if (e == cudaSuccess) {
        if (cut.ks > 1)
            e = launch_as<1, true, GRAD, TYPE, false>(m, a, dev, static_cast<int>(tiles * cut.ks), cut.ks, stream);
        else if constexpr (GRAD)
            e = p.dbias != nullptr && p.K > kPart ? launch_tiles(std::true_type{}) : launch_tiles(std::false_type{});
        else
            e = launch_tiles(std::false_type{});
    }
    if (ws != nullptr) {
        if (e == cudaSuccess) e = launch_column_sums(a.part, blocks, p.N, p.dbias, stream);
        const cudaError_t ef = workspace_free(ws, stream);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

cudaError_t launch_fused_tc(const FusedProblem &p, InType in, cudaStream_t stream,
                            const char **name) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const bool bf16 = in == InType::BF16;
    if (!p.grad)
        return bf16 ? launch_tc_as<false, kOutBf16>(p, dev, stream, name)
                    : launch_tc_as<false, kOutF16>(p, dev, stream, name);
    return bf16 ? launch_tc_as<true, kOutBf16>(p, dev, stream, name)
                : launch_tc_as<true, kOutF16>(p, dev, stream, name);
}

cudaError_t fused_tc_read_and_clear_status(cudaStream_t stream, int *status) {
    *status = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // (no copy while none of these kernels has been launched on the device)
    if (dev < 0 || dev >= kMaxDevices || !g_launched[dev].load()) return cudaSuccess;
    const int zero = 0;
    e = cudaMemcpyFromSymbolAsync(status, g_status, sizeof(int), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && *status != 0) {
        e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    return e;
}

}  // namespace gemm
