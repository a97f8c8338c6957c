// grouped_tc.cu -- the grouped products and their weight gradients on the
// sm_103a tensor cores (BF16 or FP16 inputs, FP32 accumulation).
//
//   rows:   D(r, :) = act(alpha * A(idx(r), :) op(B_g) + bias_g), r in group g
//   wgrad:  D_g = alpha * sum_{r in g} A(idx(r), :)^T B(r, :) + beta * C_g
//
// Persistent CTAs (or CTA pairs) walk the tiles of all groups; a tile belongs
// to one group.  The sizes of the groups are on the device only: each warp
// finds a tile's group with a warp scan over the offsets (GroupWalk).  One warp
// fills a ring of 128-byte-swizzled stages by TMA, one issues tcgen05.mma into
// one of two TMEM accumulators, eight write the other to D.
//
//   rows: a row tile may end inside the next group's rows.  They only reach
//     accumulator rows that are not stored (each row of D depends on its own
//     row of A), so no zero fill is needed.  Gathered rows of small
//     groups come four at a time by TMA gather, issued by a warp of its own.
//   wgrad: both operands have their rows along K and are MN-major.  A group's
//     last K block must not read the next group's rows (not even times zero:
//     they may be infinite), so that block is fetched by TMA gather with row
//     numbers outside the tensor (zeros) past the group's end, and only its
//     16-row slices that hold rows are multiplied.
//   lora:   D(i, :) = act(X(i, :) op(W) + V(i, :) op(LB) + bias): the projection
//     of all rows, its K loop continued over the slots of the tile's adapters.
#include <atomic>
#include <cfloat>
#include <mutex>

#include "grouped.cuh"
#include "internal.h"
#include "tc_epilogue.cuh"
#include "tcgen05.cuh"
#include "tma_maps.h"

namespace gemm {
namespace {

using namespace tc;

enum : int { kRows = 0, kWgrad = 1, kLora = 2 };

constexpr int kGroupM = 16;  // row tiles per band of the raster inside a group
constexpr int kMaxStages = 24;
constexpr int kEpiWarps = 8;
constexpr int kGatherWarps = 2;  // wgrad (rows: one, their tiles have 64 rows at most)
constexpr int kRingBytes = 7 * 32768;
// lora, up to 128 rows (single CTAs): a shorter ring, and 128 registers (launch
// bounds of 512 threads), leave room on each SM for a CTA of the kernel that
// makes V, so that W streams from the start (64 rows, 4096 -> 14336: the CTAs
// otherwise start 5 us later).
constexpr int kShortRing = 5 * 32768;
constexpr int kMaxSlots = 256;         // lora: adapters of a tile
// ring + alignment + barriers + row numbers (gathers) or adapters (lora)
constexpr int smem_bytes(int ring) { return ring + 1024 + 1024 + kMaxSlots * 4; }
static_assert(smem_bytes(kRingBytes) <= 227 * 1024, "shared memory of one CTA");

// wgrad, few rows per group: the tile's epilogue, not its K loop, is the time.
// D then goes out through a box of 32 x 32 FP32 per epilogue warp in shared
// memory, and C comes in through two more: a block costs some 60 instructions
// instead of about 500.  The boxes take the end of the ring's memory, which
// keeps six stages, four with C (16 groups of 1024 rows, 4096 x 4096: BF16
// gradients 303 us, 363 from registers with seven stages; FP32 with C 455).
constexpr int kBoxes = 1, kBoxesC = 3;
__host__ __device__ constexpr int box_bytes(int boxes) { return kEpiWarps * boxes * 4096; }

// Sums in parts.  The tensor cores cut what an addition to the accumulator
// cannot hold (they do not round it): a long sum comes out too small, by 1e-9 of
// itself per step of K (2e-5 after 16384), which an FP32 D shows.  Such a D is
// summed kPart steps at a time, each part in the other accumulator, and the
// epilogue warps add the parts in registers, rounded to nearest: 7e-7 off for
// BF16 and 9e-7 for FP16 at any length.  The 128 registers per thread that this
// takes come from the other warps.  It costs 3 to 10 % (8 groups, 16384 rows,
// 4096 x 14336: 1105 us without parts, 1142 in parts of 1024, 1181 of 768, 1234
// of 640; the 16384 x 4096 x 4096 product 317 and 338), for each part is read
// in 1.4 us beside the multiplication of the next (3.4 us at 768).  (lora, up to
// 128 rows: 64 rows, 4096 -> 14336: 41 and 47 us, the SMs having no registers
// left for the kernel that makes V.)
constexpr int kPart = 768;
// The weight gradients' groups have any length, which the host does not know:
// the kernel with parts runs whenever one group could be longer than a part,
// also where all are short and the other kernel, with its free registers, would
// be 7 % faster (16 groups of 64 rows, 4096 x 4096: 215 and 201 us).
constexpr int kEpiRegs = 216, kOtherRegs = 72, kPartsRegs = 168;
static_assert(2 * kEpiRegs + kOtherRegs <= 3 * kPartsRegs,
              "three warpgroups share the launch's registers");

// Warps 0-7: epilogue, 8: TMA, 9: MMA; 10 (and 11, for the weight gradients):
// gathers, issued by warps of their own so that the producer goes on with the
// copies of whole boxes, or slices of LB (lora).
constexpr int kProducer = kEpiWarps, kIssuer = kEpiWarps + 1, kHelper = kEpiWarps + 2;
template <int MODE, bool GATHER, bool PARTS>
constexpr int threads() {
    return PARTS ? 384
                 : 64 + 32 * kEpiWarps +
                       (MODE == kWgrad ? 32 * kGatherWarps : GATHER || MODE == kLora ? 32 : 0);
}
template <int CG, int MODE, bool GATHER, bool PARTS>
constexpr int max_threads() {
    return MODE == kLora && CG == 1 && !PARTS ? 512 : threads<MODE, GATHER, PARTS>();
}

struct Args {
    int64_t groups, rows, M, N;  // M: wgrad only
    const int32_t *offsets, *row_index;
    OutArgs out;
    int64_t stride_d, stride_c;
    uint32_t tiles_m, tiles_n;  // tiles_m: wgrad only
    int num_kb;                 // rows, lora: K steps of a stage each
    int ksub;                   // rows, lora: blocks of 64 of K per stage
    int part;                   // K steps per part of a sum (see kPart)
    int a_blocks, b_blocks;     // whole 64-column blocks of A (wgrad) and B (N-major)
    int staged;                 // wgrad: D and C move as TMA boxes
    int boxes;                  // per epilogue warp, at the ring's end (see kBoxes)
    int b_kmajor;               // rows
    int bn;                     // columns per tile (of the CTA or the pair)
    int am;                     // rows of D per CTA: 128, or 16 / 32 / 64 (single CTAs)
    int stages, ring_bytes;
    uint32_t stage_bytes, a_region;  // B starts a_region bytes into a stage
    int ab_format;
    int z_step;  // rows: 0 when all groups share one B
    int lb_z_step;  // lora: likewise for LB
    int slice_warp;  // lora: at most one tile per CTA, see slice_copies
    int late_wait;  // lora: the kernel before this one wrote nothing but the plan
    LoraPlan plan;  // lora (count null: no adapters)
    LoraProblem l;  // lora: operands of the exact recomputation
    uint64_t timeout_ns;
};

struct Tile {
    int g;
    int32_t first, last;  // the group's rows
    int64_t m0, n0;       // first row (rows: of all product rows; wgrad: of D_g) and column
    int m_valid;          // rows of D in the tile, 1 .. 128 CG
    int nkb;              // K steps (stages)
    int tile_m;           // its row of tiles
};

template <int CG, int MODE>
struct TileWalk {
    const Args &a;
    GroupWalk walk;
    __device__ __forceinline__ explicit TileWalk(const Args &a)
        : a(a), walk(a.offsets, a.groups, a.rows, a.am * CG, a.tiles_n) {}

    // Tile w; the whole warp calls.  False past the last tile.
    __device__ __forceinline__ bool get(uint32_t w, Tile &t) {
        uint32_t in_group, tiles_m;
        const int tile_rows = MODE == kWgrad ? BM * CG : a.am * CG;
        if constexpr (MODE == kRows) {
            if (!walk.locate(w, t.g, t.first, t.last, in_group)) return false;
            tiles_m = static_cast<uint32_t>((static_cast<int64_t>(t.last) - t.first + tile_rows - 1) / tile_rows);
        } else if constexpr (MODE == kLora) {
            if (w >= a.tiles_m * a.tiles_n) return false;
            in_group = w;
            t.g = 0;
            t.first = 0;
            t.last = static_cast<int32_t>(a.rows);
            tiles_m = a.tiles_m;
        } else {
            const uint32_t per = a.tiles_m * a.tiles_n;
            const uint32_t g = w / per;
            if (g >= a.groups) return false;
            in_group = w - g * per;
            t.g = static_cast<int>(g);
            t.first = walk.bounded(__ldg(a.offsets + g));
            t.last = walk.bounded(__ldg(a.offsets + g + 1));
            if (t.last < t.first) t.last = t.first;
            tiles_m = a.tiles_m;
        }
        const uint32_t width = kGroupM * a.tiles_n;
        const uint32_t band = in_group / width, in_band = in_group - band * width;
        const uint32_t rest = tiles_m - band * kGroupM;
        const uint32_t high = rest < kGroupM ? rest : kGroupM;
        const uint32_t q = in_band / high;
        const int64_t tm = band * kGroupM + (in_band - q * high);
        t.n0 = static_cast<int64_t>(q) * a.bn;
        const int64_t m_first = MODE == kWgrad ? 0 : t.first;
        const int64_t m_last = MODE == kWgrad ? a.M : t.last;
        t.m0 = m_first + tm * tile_rows;
        t.m_valid = m_last - t.m0 < tile_rows ? static_cast<int>(m_last - t.m0) : tile_rows;
        t.nkb = MODE == kWgrad ? static_cast<int>((static_cast<int64_t>(t.last) - t.first + BK - 1) / BK)
                               : a.num_kb;
        t.tile_m = static_cast<int>(tm);
        return true;
    }
};

// Rows of the tile in CTA `rank` of the group (0 to 128).
__device__ __forceinline__ int cta_rows(const Tile &t, int rank) {
    const int r = t.m_valid - rank * BM;
    return r < 0 ? 0 : (r > BM ? BM : r);
}

// Bytes of A a CTA loads per stage when n of its rows hold data: one box of am
// rows (rows past the group's end come along), or whole quads of gathered rows.
template <bool GATHER>
__device__ __forceinline__ uint32_t a_bytes(const Args &a, int n) {
    if (n == 0) return 0;
    const int rows = GATHER ? (n + 3) / 4 * 4 : a.am;
    return static_cast<uint32_t>(rows * a.ksub) * 128u;
}

// The order of a tile's K blocks.  CTA pairs: every other tile walks K
// backwards, so that it starts on the blocks of B the tile before it read last.
// Single CTAs start at different blocks: columns of B are a power of two apart
// as a rule, and CTAs in step would read the same few DRAM channels, and the
// same lines of A, at once.
template <int CG>
__device__ __forceinline__ int first_block(uint32_t w, int nkb, bool reverse) {
    return CG == 1 ? static_cast<int>((w * 5u) % static_cast<uint32_t>(nkb)) : (reverse ? nkb - 1 : 0);
}
template <int CG>
__device__ __forceinline__ int next_block(int kb, int nkb, bool reverse) {
    return CG == 2 && reverse ? kb - 1 : (kb + 1 == nkb ? 0 : kb + 1);
}

// lora, second product: the adapters and first columns of LA of the (up to four)
// 16-row slices from column c0 of V on; all lanes get all of them.  (The
// rounding's remainders meet the same rows of LB again.)
__device__ __forceinline__ void slice_rows(const LoraPlan &pl, const int *numbers, int c0, int slices,
                                           int (&ads)[4], int (&j0s)[4]) {
    const int lane = threadIdx.x % 32;
    int ad = 0, j0 = 0;
    if (lane < slices) {
        const int c = c0 + lane * 16, slot = c / pl.rc;
        ad = numbers[slot];
        j0 = (c - slot * pl.rc) & (pl.r_pad - 1);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        ads[q] = __shfl_sync(0xffffffffu, ad, q);
        j0s[q] = __shfl_sync(0xffffffffu, j0, q);
    }
}

// One slice of LB: 16 rows of adapter ad, the tile's columns.
template <int CG>
__device__ __forceinline__ void slice_copies(const Args &a, const CUtensorMap *map, uint32_t dst,
                                             int b_rows, int32_t b0, int j0, int ad, uint32_t fb) {
    if (a.l.b_kmajor) {
        tma_load_3d<CG>(dst, map, j0, b0, ad, fb);
    } else {
        for (int j = 0; j < b_rows; j += 64) tma_load_3d<CG>(dst + j * 32, map, b0 + j, j0, ad, fb);
    }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// 16-bit inputs: a value, and the bits of an infinity (more: a NaN).
__device__ __forceinline__ float value_16(uint32_t bits, int ab_format) {
    return ab_format == 1 ? __uint_as_float(bits << 16)
                          : __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}
__device__ __forceinline__ uint32_t infinity_16(int ab_format) {
    return ab_format == 1 ? 0x7f80u : 0x7c00u;
}
__device__ __forceinline__ void widen_8(uint4 q, int ab_format, float (&v)[8]) {
    const uint32_t b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = value_16((b[i / 2] >> (i % 2 * 16)) & 0xffffu, ab_format);
}
// The largest magnitude among eight values, as bits.
__device__ __forceinline__ uint32_t top_of_8(uint4 q) {
    uint32_t top = 0;
    for (uint32_t w : {q.x, q.y, q.z, q.w}) top = max(top, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
    return top;
}

// lora: a slot's LB meets zeros of V in the rows of other adapters; where it
// holds infinities or NaNs those products are NaN, and the sum says nothing.
// Such values of D are computed again by their definition in FP32, from the
// row's own adapter alone, and so are the rows whose first product passed the
// inputs' type (65504 for FP16) and is infinite in V only.  Other sums that are
// not finite have it from their own row of X or column of W and stay: a request
// with a NaN costs its batch nothing.
//
// A warp's 32 x 32 block of D from row0 and n0 on, already written; bit j of
// `bad`: the sum of this lane's row and column n0 + j is not finite.  Left as
// they are:
//   - rows with a NaN in X LA, or without an adapter in X: NaN in any case;
//   - columns that are finite in the LB of all the tile's adapters, and those
//     where the row's own adapter alone is not finite and holds a NaN.
// The others take a column per lane, eight rows at a time to a value of W (64
// rows, 48 adapters, 4096 -> 14336, 40 us when all is finite: a NaN in a row of X
// 40, an infinity 71, one infinity in an adapter 1500, an adapter of NaNs 3300).
__device__ __noinline__ void lora_redo(const Args &a, int64_t row0, int64_t n0, int tile_m,
                                       uint32_t bad) {
    const LoraProblem &l = a.l;
    const LoraPlan &pl = a.plan;
    const int lane = threadIdx.x % 32;
    const uint32_t inf = infinity_16(a.ab_format);
    const uint16_t *const x0 = static_cast<const uint16_t *>(l.X) + row0 * l.ldx;
    const float *const u0 = pl.part + row0 * pl.r_pad;
    const int slot = bad != 0 ? pl.slot[row0 + lane] : -1;
    const int64_t k8 = l.K / 8 * 8;

    bool passed = false;  // X LA passed the inputs' type
    if (bad != 0 && slot >= 0) {
        const uint16_t *v = pl.V + (row0 + lane) * pl.ldv + static_cast<int64_t>(slot) * pl.rc;
        const float *u = u0 + lane * pl.r_pad;
        for (int j = 0; j < l.rank; ++j) {
            if (isnan(u[j])) bad = 0;
            passed |= (v[j] & 0x7fffu) == inf && fabsf(u[j]) <= FLT_MAX;
        }
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, bad != 0 && slot < 0); left != 0; left &= left - 1) {
        const int r = __ffs(left) - 1;
        const uint16_t *x = x0 + r * l.ldx;
        uint32_t top = 0;
        for (int64_t k = lane * 8; k < k8; k += 256)
            top = max(top, top_of_8(__ldg(reinterpret_cast<const uint4 *>(x + k))));
        if (k8 + lane < l.K) top = max(top, x[k8 + lane] & 0x7fffu);
        if (__any_sync(0xffffffffu, top > inf) && lane == r) bad = 0;
    }
    if (!__any_sync(0xffffffffu, bad != 0)) return;

    // this lane's column of the slots' LB: the first slot that is not finite
    // there, whether it holds a NaN, whether there are more
    const bool inside = n0 + lane < l.N;
    const int64_t n = inside ? n0 + lane : l.N - 1;
    const int count = pl.count[tile_m];
    const int *const list = pl.list + static_cast<int64_t>(tile_m) * pl.tile_rows;
    int first = -1;
    bool has_nan = false, more = false;
    for (int s = 0; s < count; ++s) {
        const uint16_t *lb = static_cast<const uint16_t *>(l.LB) + list[s] * l.stride_b +
                             (l.b_kmajor ? n * l.ld_b : n);
        const int64_t step = l.b_kmajor ? 1 : l.ld_b;
        const int64_t r8 = l.b_kmajor ? l.rank / 8 * 8 : 0;
        uint32_t top = 0;
        for (int64_t j = 0; j < r8; j += 8)
            top = max(top, top_of_8(__ldg(reinterpret_cast<const uint4 *>(lb + j))));
#pragma unroll 8
        for (int64_t j = r8; j < l.rank; ++j) top = max(top, __ldg(lb + j * step) & 0x7fffu);
        if (top < inf || !inside) continue;
        more = first >= 0;
        if (first < 0) first = s, has_nan = top > inf;
    }
    uint32_t redo = 0;
#pragma unroll 1
    for (int r = 0; r < 32; ++r) {
        const int own = __shfl_sync(0xffffffffu, slot, r);
        const bool all = __shfl_sync(0xffffffffu, passed, r);
        const uint32_t cols = __ballot_sync(
            0xffffffffu, inside && (all || (first >= 0 && (more || first != own || !has_nan))));
        if (lane == r) redo = cols & bad;
    }
    const uint32_t rows = __ballot_sync(0xffffffffu, redo != 0);

    const uint16_t *w = static_cast<const uint16_t *>(l.W) + (l.w_kmajor ? n * l.ldw : n);
    const int64_t w_step = l.w_kmajor ? 1 : l.ldw;
    const float bias = a.out.bias != nullptr ? a.out.bias[n] : 0.f;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 8) {
        const uint32_t some = (rows >> r0) & 0xffu;
        if (some == 0) continue;
        // (rows that are not to be replaced repeat one that is)
        const uint16_t *x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = x0 + (r0 + ((some >> i) & 1u ? i : __ffs(some) - 1)) * l.ldx;
        float sum[8] = {};
#pragma unroll 1
        for (int64_t k = 0; k < k8; k += 8) {
            float wv[8];
            if (l.w_kmajor) {
                widen_8(__ldg(reinterpret_cast<const uint4 *>(w + k)), a.ab_format, wv);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) wv[i] = value_16(__ldg(w + (k + i) * w_step), a.ab_format);
            }
            uint4 q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = __ldg(reinterpret_cast<const uint4 *>(x[i] + k));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float xv[8];
                widen_8(q[i], a.ab_format, xv);
#pragma unroll
                for (int c = 0; c < 8; ++c) sum[i] = fmaf(xv[c], wv[c], sum[i]);
            }
        }
        for (int64_t k = k8; k < l.K; ++k) {
            const float wk = value_16(w[k * w_step], a.ab_format);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = fmaf(value_16(x[i][k], a.ab_format), wk, sum[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!((some >> i) & 1u)) continue;
            const int r = r0 + i, own = __shfl_sync(0xffffffffu, slot, r);
            if (own >= 0) {
                const float *u = u0 + r * pl.r_pad;
                const uint16_t *lb = static_cast<const uint16_t *>(l.LB) + list[own] * l.stride_b +
                                     (l.b_kmajor ? n * l.ld_b : n);
                const int64_t step = l.b_kmajor ? 1 : l.ld_b;
                float own_sum = 0.f;
                for (int64_t j = 0; j < l.rank; ++j)
                    own_sum = fmaf(u[j], value_16(__ldg(lb + j * step), a.ab_format), own_sum);
                sum[i] += own_sum;
            }
            if ((__shfl_sync(0xffffffffu, redo, r) >> lane) & 1u)
                store_out(a.out.D, (row0 + r) * a.out.ldd + n, activate(sum[i] + bias, a.out.act),
                          a.out.out);
        }
    }
}

template <int CG, int MODE, bool GATHER, bool PARTS>
__global__ void __launch_bounds__(max_threads<CG, MODE, GATHER, PARTS>(), 1)
    grouped_tc_kernel(const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_a_rows,
                      const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_b_rows,
                      const __grid_constant__ CUtensorMap map_v,
                      const __grid_constant__ CUtensorMap map_c,
                      const __grid_constant__ CUtensorMap map_d,
                      const __grid_constant__ CUtensorMap map_b_edge, const Args args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    // barriers (8 bytes each): full[kMaxStages] TMA -> MMA (the leader's count
    // both CTAs), empty[kMaxStages] MMA -> TMA, tfull[2] MMA -> epilogue,
    // tempty[2] epilogue -> MMA (the leader's count both CTAs),
    // go[kGatherWarps][kMaxStages] producer -> gather warp, drain,
    // cbar[kEpiWarps][2] boxes of C loaded
    const uint32_t ring0 = smem_addr(ring);
    const uint32_t full0 = ring0 + args.ring_bytes, empty0 = full0 + 8 * kMaxStages;
    const uint32_t tfull0 = empty0 + 8 * kMaxStages, tempty0 = tfull0 + 16;
    const uint32_t go0 = tempty0 + 16, drain = go0 + 8 * kGatherWarps * kMaxStages;
    const uint32_t cbar0 = drain + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ring + (cbar0 + 16 * kEpiWarps - ring0));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *numbers = reinterpret_cast<int *>(ring + args.ring_bytes + 1024);  // [kMaxSlots]

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = CG == 1 ? 0u : cluster_rank();
    const bool leader = rank == 0;
    const uint32_t first_tile = blockIdx.x / CG, tile_step = gridDim.x / CG;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * kMaxStages; ++s) mbar_init(full0 + 8 * s, 1);
        for (int s = 0; s < kGatherWarps * kMaxStages; ++s) mbar_init(go0 + 8 * s, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, kEpiWarps * CG);
        }
        mbar_init(drain, 1);
        for (int s = 0; s < 2 * kEpiWarps; ++s) mbar_init(cbar0 + 8 * s, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        prefetch_map(&map_a);
        prefetch_map(&map_b);
        if (GATHER || MODE == kWgrad) prefetch_map(&map_a_rows);
        if (MODE != kRows) prefetch_map(&map_b_rows);
        if (MODE != kRows) prefetch_map(&map_v);
        if (MODE == kWgrad && args.staged) prefetch_map(&map_d);
        if (MODE == kWgrad && args.staged && args.out.beta != 0.f) prefetch_map(&map_c);
    }
    if (warp == kIssuer) tmem_alloc<CG>(smem_addr(tmem_slot));
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // lora: the kernel before this one only makes the plan and V, and lets this
    // one start once everything before it is complete; X and W are read at
    // once, and each role waits for that kernel when it needs the plan
    const bool late = MODE == kLora && args.late_wait;
    if (!late) pdl_wait();
    pdl_launch_dependents();

    const int stages = args.stages;
    const uint32_t stage_bytes = args.stage_bytes, a_region = args.a_region;
    const int b_rows = args.bn / CG;  // columns of B this CTA loads
    const int ksub = MODE == kWgrad ? 1 : args.ksub;
    // where the copies of a stage are counted
    const uint32_t count0 = CG == 1 ? full0 : map_to_rank(full0, 0);
    TileWalk<CG, MODE> tiles(args);
    Tile t;
    bool aborted = false;
    // every lane waits (the warp stays converged); false: gave up
    auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
        const bool done = __all_sync(
            0xffffffffu, wait_bounded(bar, parity, abort_flag, args.timeout_ns));
        if (!done && lane == 0) raise_abort(abort_flag);
        return done;
    };

    if (warp >= kEpiWarps) {
        if constexpr (PARTS)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kProducer) {
            // ---------------------------------------------------- TMA producer
            int stage = 0;
            uint32_t phase = 0;
            uint32_t issued = 0;
            bool ok = true;
            auto advance = [&]() {
                issued += issued < static_cast<uint32_t>(stages) ? 1u : 0u;
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1;
                }
            };
            bool reverse = false;
            for (uint32_t w = first_tile; ok && tiles.get(w, t); w += tile_step, reverse = !reverse) {
                const int32_t b0 = static_cast<int32_t>(t.n0 + rank * b_rows);
                const int mine = cta_rows(t, rank);
                const int32_t m0 = static_cast<int32_t>(t.m0 + rank * BM);
                if constexpr (MODE != kWgrad) {
                    const uint32_t tx = a_bytes<GATHER>(args, cta_rows(t, 0)) +
                                        (CG == 2 ? a_bytes<GATHER>(args, cta_rows(t, 1)) : 0u) +
                                        static_cast<uint32_t>(CG * b_rows * ksub) * 128u;
                    const int32_t z = t.g * args.z_step;
                    int kb = first_block<CG>(w, t.nkb, reverse);
                    for (int i = 0; i < t.nkb; ++i) {
                        ok = wait_all(empty0 + 8 * stage, phase ^ 1);
                        if (!ok) break;
                        const uint32_t fb = count0 + 8 * stage;
                        const uint32_t sa = ring0 + stage * stage_bytes, sb = sa + a_region;
                        if (elect_one()) {
                            if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, tx);
                            if constexpr (GATHER) {
                                if (mine > 0) mbar_arrive(go0 + 8 * stage);
                            }
                            // several blocks of 64 at once: the maps count K in blocks
                            const int32_t block = kb * ksub;
                            const int32_t k_in = ksub > 1 ? 0 : block * BK, k_block = ksub > 1 ? block : 0;
                            if (args.b_kmajor) {
                                tma_load_4d<CG>(sb, &map_b, k_in, b0, k_block, z, fb);
                            } else if ((b0 + b_rows) / 64 <= args.b_blocks) {
                                tma_load_4d<CG>(sb, &map_b, 0, block * BK, b0 / 64, z, fb);
                            } else {
                                for (int j = 0; j < b_rows; j += 64)
                                    tma_load_3d<CG>(sb + j * 128 * ksub, &map_b_edge, b0 + j, block * BK,
                                                    z, fb);
                            }
                            if constexpr (!GATHER) {
                                if (mine > 0) tma_load_3d<CG>(sa, &map_a, k_in, m0, k_block, fb);
                            }
                        }
                        kb = next_block<CG>(kb, t.nkb, reverse);
                        advance();
                    }
                    if (MODE == kLora && ok && args.plan.count != nullptr) {
                        // the second product: V (128-byte rows of 64 columns) times
                        // the slots' LB, fetched in 16-row slices of one adapter each
                        if (late) pdl_wait();
                        const LoraPlan &pl = args.plan;
                        const int cols = pl.count[t.tile_m] * pl.rc;
                        const int *list = pl.list + static_cast<int64_t>(t.tile_m) * pl.tile_rows;
                        __syncwarp();
                        for (int i = lane; i < cols / pl.rc; i += 32) numbers[i] = list[i] * args.lb_z_step;
                        __syncwarp();
                        const uint32_t slice_bytes = static_cast<uint32_t>(b_rows) * 32u;
                        const uint32_t v_bytes = static_cast<uint32_t>(args.am) * 128u;
                        const uint32_t v_tx = v_bytes + (CG == 2 && cta_rows(t, 1) > 0 ? v_bytes : 0u);
                        if (args.slice_warp && elect_one()) mbar_arrive(go0);
                        for (int c0 = 0; c0 < cols; c0 += BK) {
                            const int slices = cols - c0 < BK ? (cols - c0) / 16 : 4;
                            int ads[4], j0s[4];
                            slice_rows(pl, numbers, c0, slices, ads, j0s);
                            ok = wait_all(empty0 + 8 * stage, phase ^ 1);
                            if (!ok) break;
                            const uint32_t fb = count0 + 8 * stage;
                            const uint32_t sa = ring0 + stage * stage_bytes, sb = sa + a_region;
                            if (elect_one()) {
                                if (leader)
                                    mbar_arrive_expect_tx(full0 + 8 * stage, v_tx + CG * slices * slice_bytes);
                                if (mine > 0) tma_load_2d<CG>(sa, &map_v, c0, m0, fb);
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    if (q < slices && (q < 2 || !args.slice_warp))
                                        slice_copies<CG>(args, &map_b_rows, sb + q * slice_bytes, b_rows, b0,
                                                         j0s[q], ads[q], fb);
                            }
                            advance();
                        }
                    }
                } else {
                    const int b_blocks = b_rows / 64;
                    for (int i = 0; i < t.nkb; ++i) {
                        const int32_t r0 = t.first + i * BK;
                        const int rem = t.last - r0 < BK ? t.last - r0 : BK;
                        const int quads = (rem + 15) / 16 * 4;  // rows of whole 16-row slices
                        const bool part = rem < BK;
                        ok = wait_all(empty0 + 8 * stage, phase ^ 1);
                        if (!ok) break;
                        const uint32_t fb = count0 + 8 * stage;
                        const uint32_t sa = ring0 + stage * stage_bytes, sb = sa + a_region;
                        if (elect_one()) {
                            if (leader)
                                mbar_arrive_expect_tx(
                                    full0 + 8 * stage,
                                    CG * (2 + b_blocks) * static_cast<uint32_t>(quads) * 512u);
                            if (part) {
                                for (int h = 0; h < kGatherWarps; ++h)
                                    mbar_arrive(go0 + 8 * (h * kMaxStages + stage));
                            }
                            if (!part) {
                                // whole 64-column blocks in one copy; a tile that holds
                                // the columns past the last whole one, block by block
                                if (m0 / 64 + 2 <= args.a_blocks) {
                                    tma_load_3d<CG>(sa, &map_a, 0, r0, m0 / 64, fb);
                                } else {
                                    tma_load_2d<CG>(sa, &map_v, m0, r0, fb);
                                    tma_load_2d<CG>(sa + 8192, &map_v, m0 + 64, r0, fb);
                                }
                                if (b0 / 64 + b_blocks <= args.b_blocks) {
                                    tma_load_3d<CG>(sb, &map_b, 0, r0, b0 / 64, fb);
                                } else {
                                    for (int j = 0; j < b_blocks; ++j)
                                        tma_load_2d<CG>(sb + j * 8192, &map_b_edge, b0 + 64 * j, r0, fb);
                                }
                            }
                        }
                        advance();
                    }
                }
            }
            __syncwarp();
            // the copies in flight land before the CTA exits (the leader's
            // barriers count both CTAs' bytes)
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
            // ------------------------------------------------------ MMA issuer
            if (leader) {
                const bool a_mn = MODE == kWgrad, b_mn = MODE == kWgrad || !args.b_kmajor;
                // N of an MMA: the tile's columns in whole blocks of the epilogue (a
                // pair's B lies half in either CTA: always all of it)
                auto idesc_of = [&](const Tile &tile, uint32_t b_mn_major) {
                    const int64_t rest = (args.N - tile.n0 + 31) / 32 * 32;
                    const int n = CG == 1 && rest < args.bn ? static_cast<int>(rest) : args.bn;
                    return make_idesc(BM * CG, n, MODE == kWgrad, b_mn_major, args.ab_format);
                };
                const uint64_t a_desc0 = a_mn ? desc_mnmajor(ring0, 0) : desc_kmajor(ring0, 0);
                const uint64_t b_desc0 =
                    b_mn ? smem_desc(ring0 + a_region, static_cast<uint32_t>(ksub) * 8192u, 1024)
                         : desc_kmajor(ring0 + a_region, 0);
                const uint64_t a_step = a_mn ? (UMMA_K * 128) >> 4 : (UMMA_K * 2) >> 4;
                const uint64_t b_step = b_mn ? (UMMA_K * 128) >> 4 : (UMMA_K * 2) >> 4;
                // a stage's blocks of 64: rows x 128 bytes apart (N-major: 64 rows of K)
                const uint64_t a_sub = static_cast<uint64_t>(args.am) * 128u >> 4;
                const uint64_t b_sub = b_mn ? 8192u >> 4 : static_cast<uint64_t>(b_rows) * 128u >> 4;
                // lora: slices of LB -- K-major: 32-byte rows (32-byte swizzle);
                // N-major: 16 rows per 64-column block (128-byte swizzle)
                const bool lb_mn = MODE == kLora && !args.l.b_kmajor;
                const uint64_t lb_desc0 = lb_mn ? smem_desc(ring0 + a_region, 16 * 128, 1024)
                                                : smem_desc(ring0 + a_region, 16, 256, kSwizzle32);
                const uint64_t stage_step = stage_bytes >> 4;
                int stage = 0;
                uint32_t phase = 0;
                uint32_t acc = 0;  // accumulators filled so far
                bool ok = true;
                for (uint32_t w = first_tile; ok && tiles.get(w, t); w += tile_step) {
                    if (MODE == kWgrad && t.nkb == 0) continue;  // no rows: nothing to add
                    const uint32_t idesc = idesc_of(t, b_mn), lb_idesc = idesc_of(t, lb_mn);
                    uint32_t d_tmem = 0;
                    auto take = [&]() {  // the accumulator not filled last, once it has been read
                        ok = wait_all(tempty0 + 8 * (acc & 1), ((acc >> 1) & 1) ^ 1);
                        tc_fence_after();
                        d_tmem = tmem_base + (acc & 1) * 256;
                    };
                    take();
                    if (!ok) break;
                    int in_part = 0;
                    // 16-row slices of the last block that hold rows
                    const int last_slices =
                        MODE == kWgrad ? (t.last - t.first - (t.nkb - 1) * BK + 15) / 16 : 4;
                    for (int i = 0; i < t.nkb; ++i, ++in_part) {
                        if (PARTS && in_part == args.part) {
                            if (elect_one()) tc_commit<CG>(tfull0 + 8 * (acc & 1));
                            ++acc;
                            take();
                            if (!ok) break;
                            in_part = 0;
                        }
                        ok = wait_all(full0 + 8 * stage, phase);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = a_desc0 + static_cast<uint64_t>(stage) * stage_step;
                        const uint64_t bd = b_desc0 + static_cast<uint64_t>(stage) * stage_step;
                        const int slices = MODE == kWgrad && i + 1 == t.nkb ? last_slices : 4;
                        if (elect_one()) {
                            tc_mma<CG>(d_tmem, ad, bd, idesc, in_part > 0 ? 1u : 0u);
                            if (MODE != kWgrad || slices > 1)
                                tc_mma<CG>(d_tmem, ad + a_step, bd + b_step, idesc, 1u);
                            if (MODE != kWgrad || slices > 2)
                                tc_mma<CG>(d_tmem, ad + 2 * a_step, bd + 2 * b_step, idesc, 1u);
                            if (MODE != kWgrad || slices > 3)
                                tc_mma<CG>(d_tmem, ad + 3 * a_step, bd + 3 * b_step, idesc, 1u);
                            if constexpr (MODE != kWgrad) {
                                for (int u = 1; u < ksub; ++u) {
                                    const uint64_t au = ad + u * a_sub, bu = bd + u * b_sub;
                                    tc_mma<CG>(d_tmem, au, bu, idesc, 1u);
                                    tc_mma<CG>(d_tmem, au + a_step, bu + b_step, idesc, 1u);
                                    tc_mma<CG>(d_tmem, au + 2 * a_step, bu + 2 * b_step, idesc, 1u);
                                    tc_mma<CG>(d_tmem, au + 3 * a_step, bu + 3 * b_step, idesc, 1u);
                                }
                            }
                            tc_commit<CG>(empty0 + 8 * stage);  // frees the stage (both CTAs)
                        }
                        if (++stage == stages) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                    if (MODE == kLora && ok && args.plan.count != nullptr) {
                        if (late) pdl_wait();
                        const int cols = args.plan.count[t.tile_m] * args.plan.rc;
                        const uint64_t slice_step = static_cast<uint64_t>(b_rows) * 32u >> 4;
                        for (int c0 = 0; c0 < cols; c0 += BK) {
                            ok = wait_all(full0 + 8 * stage, phase);
                            if (!ok) break;
                            tc_fence_after();
                            const int slices = cols - c0 < BK ? (cols - c0) / 16 : 4;
                            const uint64_t at = static_cast<uint64_t>(stage) * stage_step;
                            if (elect_one()) {
                                for (int q = 0; q < slices; ++q)
                                    tc_mma<CG>(d_tmem, a_desc0 + at + q * a_step,
                                               lb_desc0 + at + q * slice_step, lb_idesc, 1u);
                                tc_commit<CG>(empty0 + 8 * stage);
                            }
                            if (++stage == stages) {
                                stage = 0;
                                phase ^= 1u;
                            }
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
        } else if (MODE == kLora && warp >= kHelper) {
            // --------------------------------------------------------- slice warp
            // A decode step has many slices, 100 ns each to issue: this warp issues
            // every second pair of them.  It joins the producer at the first block
            // of V (go), waits for the same stages from there on and cannot run
            // ahead of the ring: a CTA has one tile here.
            if (warp == kHelper && args.slice_warp && tiles.get(first_tile, t) &&
                __all_sync(0xffffffffu, wait_bounded(go0, 0, abort_flag, args.timeout_ns))) {
                if (late) pdl_wait();
                const LoraPlan &pl = args.plan;
                const int cols = pl.count[t.tile_m] * pl.rc;
                const int32_t b0 = static_cast<int32_t>(t.n0 + rank * b_rows);
                const uint32_t slice_bytes = static_cast<uint32_t>(b_rows) * 32u;
                // (numbers was written by the producer before it arrived on go)
                int stage = t.nkb % stages;
                uint32_t phase = static_cast<uint32_t>(t.nkb / stages) & 1u;
                for (int c0 = 0; c0 < cols; c0 += BK) {
                    const int slices = cols - c0 < BK ? (cols - c0) / 16 : 4;
                    int ads[4], j0s[4];
                    slice_rows(pl, numbers, c0, slices, ads, j0s);
                    if (!wait_all(empty0 + 8 * stage, phase ^ 1)) break;
                    const uint32_t sb = ring0 + stage * stage_bytes + a_region;
                    if (elect_one()) {
#pragma unroll
                        for (int q = 2; q < 4; ++q)
                            if (q < slices)
                                slice_copies<CG>(args, &map_b_rows, sb + q * slice_bytes, b_rows, b0, j0s[q],
                                                 ads[q], count0 + 8 * stage);
                    }
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            __syncwarp();
        } else if (MODE == kRows && warp >= kHelper + (GATHER ? 1 : 0)) {
            // (they only gave their registers)
        } else if (warp >= kHelper) {
            // -------------------------------------------------------- gather warps
            // They follow the producer's stages and issue the parts of a stage
            // that come by row number: one thread each, the numbers in shared
            // memory.  The producer, which has waited for the stage and counted
            // their bytes in its expect_tx, tells each warp through its own
            // barrier of that stage; it cannot tell it again before the bytes have
            // arrived, so one parity bit per stage is enough.
            const int half = warp - kHelper;
            int *const mine = numbers + half * 64;  // 64 row numbers
            const uint32_t go = go0 + 8 * half * kMaxStages;
            int stage = 0;
            uint32_t told = 0;  // parity of the next word on each stage
            bool ok = true;
            // 4 * quads rows (numbers from `from` on), 64 columns from c0 on, to dst
            auto gather = [&](uint32_t dst, const CUtensorMap *map, int32_t c0, const int *from,
                              int quads, uint32_t fb) {
                for (int q = 0; q < quads; ++q) {
                    const int4 r = *reinterpret_cast<const int4 *>(from + q * 4);
                    if (elect_one()) tma_gather4<CG>(dst + q * 512, map, c0, r.x, r.y, r.z, r.w, fb);
                }
            };
            bool reverse = false;
            for (uint32_t w = first_tile; ok && tiles.get(w, t); w += tile_step, reverse = !reverse) {
                const int32_t b0 = static_cast<int32_t>(t.n0 + rank * b_rows);
                const int32_t m0 = static_cast<int32_t>(t.m0 + rank * BM);
                int quads = 0;  // rows mode: the tile's
                int kb = 0;
                if constexpr (MODE != kWgrad) {
                    const int rows = cta_rows(t, rank);  // (groups of few rows: at most 64)
                    quads = (rows + 3) / 4;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = lane + i * 32;
                        mine[r] = r < rows ? __ldg(args.row_index + m0 + r) : -1;
                    }
                    __syncwarp();
                    kb = first_block<CG>(w, t.nkb, reverse);
                }
                for (int i = 0; i < t.nkb; ++i) {
                    const uint32_t fb = count0 + 8 * stage;
                    const uint32_t sa = ring0 + stage * stage_bytes, sb = sa + a_region;
                    bool work = quads > 0, part = false;
                    if constexpr (MODE == kWgrad) {
                        const int32_t r0 = t.first + i * BK;
                        const int rem = t.last - r0 < BK ? t.last - r0 : BK;
                        part = rem < BK;
                        quads = (rem + 15) / 16 * 4;  // rows of whole 16-row slices
                        work = part;
                        if (work) {
                            __syncwarp();
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int r = lane + j * 32;
                                mine[r] = r < rem ? static_cast<int>(r0 + r) : -1;
                            }
                            __syncwarp();
                        }
                    }
                    if (work) {
                        ok = wait_all(go + 8 * stage, (told >> stage) & 1u);
                        if (!ok) break;
                        told ^= 1u << stage;
                        if constexpr (MODE == kWgrad) {
                            gather(sa + half * 8192, &map_a_rows, m0 + half * 64, mine, quads, fb);
                            for (int j = half; j < b_rows / 64; j += kGatherWarps)
                                gather(sb + j * 8192, &map_b_rows, b0 + 64 * j, mine, quads, fb);
                        } else {
                            for (int u = 0; u < ksub; ++u)
                                gather(sa + u * args.am * 128, &map_a_rows, (kb * ksub + u) * BK, mine,
                                       quads, fb);
                        }
                    }
                    if constexpr (MODE != kWgrad) kb = next_block<CG>(kb, t.nkb, reverse);
                    if (++stage == stages) stage = 0;
                }
            }
            __syncwarp();
        }
    } else {
        if constexpr (PARTS)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        // -------------------------------------------------- epilogue warps
        // Two per quarter of the TMEM lanes; each takes every other block of
        // 32 columns.  C of a block is loaded while the one before it is
        // stored (the first while the tile is still summed).
        const int e = warp, quarter = warp % 4, half = e / 4;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        uint32_t acc = 0;
        // this warp's boxes; blocks that went through them so far
        const uint32_t boxes0 = ring0 + args.ring_bytes - box_bytes(args.boxes) + e * args.boxes * 4096;
        const uint32_t cbar = cbar0 + 16 * e;
        uint32_t blocks = 0;
        if (late) pdl_wait();
        for (uint32_t w = first_tile; tiles.get(w, t); w += tile_step) {
            const bool empty_sum = MODE == kWgrad && t.nkb == 0;
            int nrows = t.m_valid - static_cast<int>(rank) * BM - quarter * 32;
            nrows = nrows < 0 ? 0 : (nrows > 32 ? 32 : nrows);
            const int64_t row0 = t.m0 + rank * BM + quarter * 32;
            const int64_t rest = args.N - t.n0;
            const int ncols = rest < args.bn ? static_cast<int>(rest) : args.bn;
            const int n_chunks = nrows > 0 ? (ncols + 31) / 32 : 0;
            // this warp's last block (-1: it has none)
            const int last = n_chunks > half ? half + ((n_chunks - 1 - half) / 2) * 2 : -1;
            OutArgs o = args.out;
            if constexpr (MODE != kWgrad) {
                if (o.bias != nullptr) o.bias += t.g * args.N;
            } else {
                o.D = static_cast<uint8_t *>(o.D) + t.g * args.stride_d * (o.out == kOutF32 ? 4 : 2);
                if (o.beta != 0.f) o.C += t.g * args.stride_c;
            }
            const bool use_c = MODE == kWgrad && o.beta != 0.f;
            const bool staged = MODE == kWgrad && args.staged;
            uint32_t buf = 0, t_acc = 0;  // the accumulator being read
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
            // staged: C of block number n into its box (the block that used it last
            // has been read)
            auto fetch_c = [&](int chunk, uint32_t n) {
                if (use_c && elect_one()) {
                    const uint32_t bar = cbar + 8 * (n & 1);
                    mbar_arrive_expect_tx(bar, 4096);
                    tma_load_3d<CG>(boxes0 + (1 + (n & 1)) * 4096, &map_c,
                                    static_cast<int32_t>(t.n0) + chunk * 32,
                                    static_cast<int32_t>(row0), t.g,
                                    CG == 1 ? bar : map_to_rank(bar, rank));
                }
            };
            // staged: C of the next block is on its way, and this block's is there
            // (false: it did not come)
            auto c_ready = [&](int chunk) -> bool {
                if (chunk + 2 < n_chunks) fetch_c(chunk + 2, blocks + 1);
                return !use_c || wait_all(cbar + 8 * (blocks & 1), (blocks >> 1) & 1);
            };
            // staged: quad q of this lane's row of the block
            auto finished = [&](int q, float4 v) -> float4 {
                v.x *= o.alpha, v.y *= o.alpha, v.z *= o.alpha, v.w *= o.alpha;
                if (use_c) {
                    const float4 c = ld_shared_v4(boxes0 + (1 + (blocks & 1)) * 4096 + box_quad(lane, q));
                    v.x = fmaf(o.beta, c.x, v.x), v.y = fmaf(o.beta, c.y, v.y);
                    v.z = fmaf(o.beta, c.z, v.z), v.w = fmaf(o.beta, c.w, v.w);
                }
                return v;
            };
            // staged: the last store has read the box / the box goes to D
            auto open_box = [&]() {
                if (elect_one()) bulk_wait_read();
                __syncwarp();
            };
            auto close_box = [&](int chunk) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (elect_one())
                    tma_store_3d(&map_d, static_cast<int32_t>(t.n0) + chunk * 32,
                                 static_cast<int32_t>(row0), t.g, boxes0);
                ++blocks;
            };
            auto put_quad = [&](int q, float4 v) {
                st_shared_v4(boxes0 + box_quad(lane, q), __float_as_uint(v.x), __float_as_uint(v.y),
                             __float_as_uint(v.z), __float_as_uint(v.w));
            };
            // The next accumulator, when it is complete.
            auto next_acc = [&]() -> bool {
                buf = acc & 1;
                t_acc = tmem_base + lane_off + buf * 256;
                if (!wait_all(tfull0 + 8 * buf, (acc >> 1) & 1)) return false;
                tc_fence_after();
                ++acc;
                return true;
            };
            auto take_block = [&](int chunk, uint32_t (&raw)[32]) {
                __syncwarp();
                tmem_load_32cols(t_acc + chunk * 32, raw);
                if (chunk == last) release_acc();
            };
            // lora: which of this lane's sums are not finite, and what to do about
            // them once the block is written (lora_redo)
            auto bad_sum = [](float x) -> uint32_t { return fabsf(x) <= FLT_MAX ? 0u : 1u; };
            auto bad_quad = [&](float4 x) -> uint32_t {
                return bad_sum(x.x) | bad_sum(x.y) << 1 | bad_sum(x.z) << 2 | bad_sum(x.w) << 3;
            };
            auto in_rows = [&](uint32_t bad) -> uint32_t {
                return args.plan.count != nullptr && lane < nrows ? bad : 0u;
            };
            auto redo_block = [&](int chunk, uint32_t bad) {
                if (__any_sync(0xffffffffu, bad != 0))
                    lora_redo(args, row0, t.n0 + chunk * 32, t.tile_m, bad);
            };
            if constexpr (PARTS) {
                // run: the sums of this warp's blocks, where they have several parts
                const bool parts = t.nkb > args.part;
                uint32_t run[4][32] = {};  // (FP32)
                if (staged && last >= 0) fetch_c(half, blocks);
                for (int from = 0; from < t.nkb && !aborted; from += args.part) {
                    if (!next_acc()) {
                        aborted = true;
                        break;
                    }
                    if (!parts) break;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (half + 2 * b > last) continue;
                        uint32_t raw[32];
                        __syncwarp();
                        tmem_load_32cols(t_acc + (half + 2 * b) * 32, raw);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            run[b][j] =
                                __float_as_uint(__uint_as_float(run[b][j]) + __uint_as_float(raw[j]));
                    }
                    release_acc();
                }
                if (aborted) break;
                uint32_t bad[4] = {};  // (lora, of this warp's blocks)
#pragma unroll 1
                for (int chunk = half; chunk < n_chunks; chunk += 2) {
                    if (staged) open_box();
                    auto put = [&](const uint32_t (&x)[32]) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            st_shared_v4(boxes0 + box_quad(lane, q), x[q * 4], x[q * 4 + 1],
                                         x[q * 4 + 2], x[q * 4 + 3]);
                    };
                    if (parts) {
                        // (indices into run are fixed at compile time)
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (chunk == half + 2 * b) put(run[b]);
                    } else {
                        uint32_t raw[32];
                        if (empty_sum) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) raw[j] = 0;
                        } else {
                            take_block(chunk, raw);
                        }
                        put(raw);
                    }
                    if (!staged) {
                        if constexpr (MODE == kLora) {
                            uint32_t b = 0;
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                b |= bad_quad(ld_shared_v4(boxes0 + box_quad(lane, q))) << (q * 4);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (chunk == half + 2 * i) bad[i] = in_rows(b);
                        }
                        __syncwarp();
                        store_from_box<MODE == kWgrad>(boxes0, o, row0, nrows, t.n0 + chunk * 32,
                                                       ncols - chunk * 32);
                        __syncwarp();
                        continue;
                    }
                    if (!c_ready(chunk)) {
                        aborted = true;
                        break;
                    }
                    if (use_c || o.alpha != 1.f) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            put_quad(q, finished(q, ld_shared_v4(boxes0 + box_quad(lane, q))));
                    }
                    close_box(chunk);
                }
                if (aborted) break;
                if constexpr (MODE == kLora) {
                    // (after the loop: the parts' sums need no registers any more)
#pragma unroll
                    for (int i = 0; i < 4; ++i) redo_block(half + 2 * i, bad[i]);
                }
                if (!parts && last < 0 && !empty_sum) release_acc();
                continue;
            }
            if (staged) {
                if (last >= 0) fetch_c(half, blocks);
                if (!empty_sum && !next_acc()) {
                    aborted = true;
                    break;
                }
#pragma unroll 1
                for (int chunk = half; chunk < n_chunks; chunk += 2) {
                    uint32_t raw[32];
                    if (empty_sum) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) raw[j] = 0;
                    } else {
                        take_block(chunk, raw);
                    }
                    if (!c_ready(chunk)) {
                        aborted = true;
                        break;
                    }
                    float4 v[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        v[q] = finished(q, make_float4(__uint_as_float(raw[q * 4]),
                                                       __uint_as_float(raw[q * 4 + 1]),
                                                       __uint_as_float(raw[q * 4 + 2]),
                                                       __uint_as_float(raw[q * 4 + 3])));
                    open_box();
                    if (o.out == kOutF32) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) put_quad(q, v[q]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)  // 64-byte rows
                            st_shared_v4(boxes0 + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4),
                                         pack_16(v[2 * q].x, v[2 * q].y, o.out),
                                         pack_16(v[2 * q].z, v[2 * q].w, o.out),
                                         pack_16(v[2 * q + 1].x, v[2 * q + 1].y, o.out),
                                         pack_16(v[2 * q + 1].z, v[2 * q + 1].w, o.out));
                    }
                    close_box(chunk);
                }
                if (aborted) break;
                if (last < 0 && !empty_sum) release_acc();
                continue;
            }
            float c[32];
            const bool quads = in_quads(o);
            auto load_c = [&](int chunk) {
                if (!use_c) return;
                if (quads)
                    load_c_quads(o, row0, nrows, t.n0 + chunk * 32, ncols - chunk * 32, c);
                else
                    load_c_columns(o, row0, nrows, t.n0 + chunk * 32, ncols - chunk * 32, c);
            };
            if (last >= 0) load_c(half);
            uint32_t bads[4] = {};
            if (!empty_sum && !next_acc()) {
                aborted = true;
                break;
            }
#pragma unroll 1
            for (int chunk = half; chunk < n_chunks; chunk += 2) {
                float v[32];
                uint32_t bad = 0;
                if (empty_sum) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.f;
                } else {
                    uint32_t raw[32];
                    take_block(chunk, raw);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]);
                    if constexpr (MODE == kLora) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) bad |= bad_sum(v[j]) << j;
                        bad = in_rows(bad);
                    }
                }
                const int left = ncols - chunk * 32;
                const int width = left < 32 ? left : 32;
                const int64_t c0 = t.n0 + chunk * 32;
                if (quads) {
                    transpose_quads(v);
                    finish_quads<MODE == kWgrad>(v, c, o, c0, width);
                    if (chunk + 2 < n_chunks) load_c(chunk + 2);
                    store_quads(v, o, row0, nrows, c0, width);
                } else {
                    transpose_32x32(v);
                    finish_columns<MODE == kWgrad>(v, c, o, c0, width);
                    if (chunk + 2 < n_chunks) load_c(chunk + 2);
                    store_columns(v, o, row0, nrows, c0, width);
                }
                __syncwarp();
                if constexpr (MODE == kLora) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (chunk == half + 2 * i) bads[i] = bad;
                }
            }
            if constexpr (MODE == kLora) {
#pragma unroll
                for (int i = 0; i < 4; ++i) redo_block(half + 2 * i, bads[i]);
            }
            if (last < 0 && !empty_sum) release_acc();
        }
        __syncwarp();
        if (MODE == kWgrad && args.staged && elect_one()) bulk_wait_all();  // D is written
        __syncwarp();
    }

    if (aborted) {
        // give copies issued by a peer that gave up a short time to land
        const uint64_t t0 = global_timer();
        while (global_timer() - t0 < 2000000ull) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc<CG>(tmem_base);
}

// Rows of A in product order: out(r, :) = A(index[r], :), zeros for an index
// outside A.  TMA fetches gathered rows one 128-byte line per 8 ns and SM, a
// third of what the MMAs of a CTA pair take (8 experts, 16384 rows, 4096 ->
// 14336: 3.1 ms gathered by TMA, 1.06 ms with the rows in order).  So only
// groups of a few rows (kGatherRows on average) are gathered by TMA, which
// saves a launch; others, and the weight gradients' rows, are put in order
// first (16384 rows of 4096: 41 us at 6.5 TB/s).
// (Tiles have 32 or 64 rows at such means.)
constexpr int64_t kGatherRows = 16;
__global__ void __launch_bounds__(256) order_rows_kernel(const uint16_t *A, int64_t lda,
                                                         int64_t rows_a, const int32_t *index,
                                                         int64_t rows, int64_t cols, uint16_t *out,
                                                         int64_t ldo) {
    pdl_wait();
    pdl_launch_dependents();
    // 16-byte pieces of all rows in order, four per thread and step
    const int64_t per_row = (cols + 7) / 8, all = rows * per_row;
    for (int64_t q0 = blockIdx.x * 1024ll + threadIdx.x; q0 < all; q0 += gridDim.x * 1024ll) {
        uint4 v[4];
        int64_t r[4], c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t q = q0 + i * 256;
            r[i] = q < all ? q / per_row : -1;
            c[i] = q - r[i] * per_row;
            v[i] = make_uint4(0, 0, 0, 0);
            if (r[i] < 0) continue;
            const int64_t from = index[r[i]];
            if (from < 0 || from >= rows_a) continue;
            const uint16_t *src = A + from * lda + c[i] * 8;
            if (c[i] * 8 + 8 <= cols) {
                v[i] = __ldg(reinterpret_cast<const uint4 *>(src));
            } else {  // the end of a row
                uint32_t w[4] = {};
                for (int k = 0; k < cols - c[i] * 8; ++k)
                    w[k / 2] |= static_cast<uint32_t>(src[k]) << (k % 2 * 16);
                v[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r[i] >= 0) *reinterpret_cast<uint4 *>(out + r[i] * ldo + c[i] * 8) = v[i];
    }
}

// ---------------------------------------------------------------- host side
constexpr int kMaxDevices = 64;

struct DeviceInfo {
    std::once_flag once;
    cudaError_t err = cudaSuccess;
    int dev = 0;
    int sms = 1;
    int pairs = 0;  // CTA pairs resident at once
};
DeviceInfo g_dev[kMaxDevices];
// A kernel of this file has been launched on the device (and stays so: it may
// set its status word at any time until it ends).
std::atomic<bool> g_launched[kMaxDevices];

template <int CG, int MODE, bool GATHER, bool PARTS>
cudaLaunchConfig_t config(int grid, int ring, cudaStream_t stream, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(threads<MODE, GATHER, PARTS>(), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes(ring));
    cfg.stream = stream;
    cfg.attrs = attr;
    set_pdl_attribute(&attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = CG > 1 ? 2 : 1;
    return cfg;
}

// Prepares a kernel on device `dev` before its first launch there.  Each kernel
// has its own answer: one that cannot run does not take the others with it.
template <int CG, int MODE, bool GATHER, bool PARTS>
cudaError_t prepared(int dev) {
    static std::once_flag once[kMaxDevices];
    static cudaError_t err[kMaxDevices];
    std::call_once(once[dev], [dev] {
        const auto kernel = grouped_tc_kernel<CG, MODE, GATHER, PARTS>;
        if (PARTS) {
            // the warpgroups divide what the launch gives: without it they would wait
            cudaFuncAttributes at;
            err[dev] = cudaFuncGetAttributes(&at, kernel);
            if (err[dev] == cudaSuccess && at.numRegs != kPartsRegs) err[dev] = cudaErrorInvalidKernelImage;
            if (err[dev] != cudaSuccess) return;
        }
        err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        smem_bytes(kRingBytes));
    });
    return err[dev];
}

DeviceInfo *device_info() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    DeviceInfo *d = &g_dev[dev];
    std::call_once(d->once, [d, dev] {
        d->dev = dev;
        int n = 0;
        d->err = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (d->err != cudaSuccess) return;
        d->sms = n > 0 ? n : 1;
        d->err = prepared<2, kRows, false, false>(dev);
        if (d->err != cudaSuccess) return;
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = config<2, kRows, false, false>(2 * (d->sms / 2), kRingBytes, 0, attr);
        cfg.attrs = attr + 1;  // the occupancy query takes the cluster shape only
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&d->pairs, grouped_tc_kernel<2, kRows, false, false>, &cfg) !=
            cudaSuccess) {
            d->pairs = 0;
            (void)cudaGetLastError();  // the pair variants are then not used
        }
    });
    return d;
}

template <int CG, int MODE, bool GATHER, bool PARTS>
cudaError_t launch_as(const CUtensorMap (&maps)[8], const Args &a, int grid, const DeviceInfo *d,
                      cudaStream_t stream) {
    const cudaError_t e = prepared<CG, MODE, GATHER, PARTS>(d->dev);
    if (e != cudaSuccess) return e;
    g_launched[d->dev].store(true);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config<CG, MODE, GATHER, PARTS>(grid, a.ring_bytes, stream, attr);
    return cudaLaunchKernelEx(&cfg, grouped_tc_kernel<CG, MODE, GATHER, PARTS>, maps[0], maps[1],
                              maps[2], maps[3], maps[4], maps[5], maps[6], maps[7], a);
}

// Boxes at the ring's end, for fewer stages.
void take_boxes(Args &a, int boxes) {
    a.boxes = boxes;
    const int over = BM * BK * 2 - static_cast<int>(a.stage_bytes);
    const int fit = (a.ring_bytes - box_bytes(boxes) - (over > 0 ? over : 0)) / static_cast<int>(a.stage_bytes);
    if (a.stages > fit) a.stages = fit;
}

// `parts`: sums longer than kPart are made in parts.
template <int CG, int MODE>
cudaError_t launch(const CUtensorMap (&maps)[8], Args &a, bool gather, int64_t max_tiles,
                   bool parts, const DeviceInfo *d, cudaStream_t stream) {
    const int64_t resident = CG == 2 ? d->pairs : d->sms;
    const int grid = static_cast<int>((max_tiles < resident ? max_tiles : resident) * CG);
    a.part = kPart / (BK * a.ksub);
    if (parts) {
        if (a.boxes == 0) take_boxes(a, kBoxes);
        if constexpr (MODE == kRows && CG == 1) {
            if (gather) return launch_as<CG, MODE, true, true>(maps, a, grid, d, stream);
        }
        return launch_as<CG, MODE, false, true>(maps, a, grid, d, stream);
    }
    if constexpr (MODE == kRows && CG == 1) {
        if (gather) return launch_as<CG, MODE, true, false>(maps, a, grid, d, stream);
    }
    return launch_as<CG, MODE, false, false>(maps, a, grid, d, stream);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tile of am rows per CTA and bn columns, and the ring to match: stages of am
// rows of A and the CTA's rows of B, as many as fit.  With am < 128 the MMA's
// 128-row A operand runs on into B and the next stages: stale rows, which
// reach only accumulator rows that are not stored.  The last stage keeps 128
// rows inside the ring.  ksub blocks of 64 of K share a stage (see sub_blocks).
void set_tile(Args &a, int cg, int am, int bn, int ksub = 1, int ring = kRingBytes) {
    a.ring_bytes = ring;
    a.am = am;
    a.bn = bn;
    a.ksub = ksub;
    a.a_region = static_cast<uint32_t>(am * ksub) * BK * 2;
    a.stage_bytes = a.a_region + static_cast<uint32_t>(bn / cg * ksub) * BK * 2;
    const int over = BM * BK * 2 - static_cast<int>(a.stage_bytes);
    const int fit = (ring - (over > 0 ? over : 0)) / static_cast<int>(a.stage_bytes);
    a.stages = fit < kMaxStages ? fit : kMaxStages;
}

// Blocks of 64 of K per stage: a copy takes the producer about 100 ns to issue
// whatever its size, while 128 x 128 tiles multiply a block in 130 ns, so tiles
// that small put two or four blocks into one stage.  The copies of K-major
// operands then count K in blocks of 64, which needs K to be a multiple of 64.
int sub_blocks(int64_t K, int am, int bn) {
    int ksub = 1;
    while (ksub < 4 && bn * 2 * ksub <= 256 && (am + bn) * 128 * 2 * ksub <= 65536) ksub *= 2;
    return K % BK == 0 ? ksub : 1;
}

constexpr int64_t kMaxTiles = int64_t(1) << 30;  // the tile arithmetic is 32-bit

}  // namespace

// A launch's error, after the workspace (or null) is given back in stream order.
static cudaError_t free_after(void *ws, cudaStream_t stream, cudaError_t e) {
    if (ws == nullptr) return e;
    const cudaError_t ef = workspace_free(ws, stream);
    return e != cudaSuccess ? e : ef;
}

// Rows in product order in a workspace (order_rows_kernel); *ws to be freed.
static cudaError_t order_rows(const void *A, int64_t lda, int64_t rows_a, const int32_t *index,
                              int64_t rows, int64_t cols, int sms, cudaStream_t stream, void **ws,
                              int64_t *ldo) {
    *ldo = ceil_div(cols, 8) * 8;
    cudaError_t e = workspace_alloc(static_cast<size_t>(rows * *ldo) * 2, stream, ws);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    set_pdl_attribute(&attr);
    cudaLaunchConfig_t cfg = {};
    const int64_t steps = ceil_div(rows * (*ldo / 8), 1024);
    const int64_t grid = steps < 8 * sms ? steps : 8 * sms;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, order_rows_kernel, static_cast<const uint16_t *>(A), lda, rows_a,
                              index, rows, cols, static_cast<uint16_t *>(*ws), *ldo);
}

bool grouped_tc_eligible(const GroupedProblem &p) {
    return p.K > 0 && p.rows_a > 0 && tma_rows(p.A, p.lda) &&
           tma_rows(p.B, p.ldb, p.groups > 1 ? p.stride_b : 0) &&
           (ceil_div(p.rows, 16) + (p.groups < p.rows ? p.groups : p.rows)) * ceil_div(p.N, 64) <
               kMaxTiles;
}

cudaError_t launch_grouped_tc(const GroupedProblem &whole, InType in, cudaStream_t stream,
                              const char **name) {
    GroupedProblem p = whole;
    const bool bf16 = in == InType::BF16;
    DeviceInfo *d = device_info();
    if (d == nullptr) return cudaErrorInvalidDevice;
    if (d->err != cudaSuccess) return d->err;
    Args a = {};
    a.groups = p.groups;
    a.rows = p.rows;
    a.N = p.N;
    a.offsets = p.offsets;
    a.row_index = p.row_index;
    a.out.D = p.D;
    a.out.ldd = p.ldd;
    a.out.bias = p.bias;
    a.out.alpha = p.alpha;
    a.out.act = p.act;
    a.out.out = p.out;
    a.out.row_vec = row_alignment(p.D, p.ldd, 0, p.out == kOutF32 ? 4 : 2);
    a.b_kmajor = p.b_kmajor ? 1 : 0;
    a.ab_format = bf16 ? 1 : 0;
    a.timeout_ns = wait_limit_ns(ceil_div(p.K, BK), p.groups);
    const bool one_b = p.groups == 1 || p.stride_b == 0;
    a.z_step = one_b ? 0 : 1;
    // Groups that may hold rows, and row tiles if the rows spread evenly.
    const int64_t live = p.groups < p.rows ? p.groups : p.rows;
    const int64_t pair_tiles = live * ceil_div(ceil_div(p.rows, live), 2 * BM) * ceil_div(p.N, 256);
    const bool pair = d->pairs > 0 && p.rows / live > BM && pair_tiles >= d->pairs;
    if (pair) {
        set_tile(a, 2, BM, 256);
    } else {
        // Few rows per group: the weights are the time; narrow tiles and few
        // rows per tile (32 groups of 32 rows, 4096 x 2048: 90 us with 32, 101
        // with 128).  A group's further rows read the weights again, from L2:
        // 16 rows gain 2 % for groups of two rows and lose 6 % when they are
        // uneven (64 groups, 128 rows).
        const int64_t mean = ceil_div(p.rows, live);
        const int am = mean <= 12 ? 32 : (mean <= 32 ? 64 : BM);
        const int64_t row_tiles = live * ceil_div(mean, am);
        int bn = 256;
        if (am < BM) {
            while (bn > 64 && row_tiles * ceil_div(p.N, bn) < 4 * d->sms) bn /= 2;
        } else {
            // rounds of tiles, each as long as its columns and a fixed part (17
            // groups, 672 rows, 173 x 10416: 37 us at 256 columns, 45 at 64)
            int64_t best = INT64_MAX;
            for (int w : {256, 128, 64}) {
                const int64_t cost = ceil_div(row_tiles * ceil_div(p.N, w), d->sms) * (w + 64);
                if (cost < best) best = cost, bn = w;
            }
        }
        set_tile(a, 1, am, bn, sub_blocks(p.K, am, bn));
    }
    a.num_kb = static_cast<int>(ceil_div(p.K, BK * a.ksub));
    a.tiles_n = static_cast<uint32_t>(ceil_div(p.N, a.bn));
    const int cg = pair ? 2 : 1;
    void *ws = nullptr;
    cudaError_t e = cudaSuccess;
    if (p.row_index != nullptr && p.rows / live > kGatherRows) {
        int64_t ldo = 0;
        e = order_rows(p.A, p.lda, p.rows_a, p.row_index, p.rows, p.K, d->sms, stream, &ws, &ldo);
        p.A = ws;
        p.lda = ldo;
        p.rows_a = p.rows;
        p.row_index = nullptr;
    }
    const bool gather = p.row_index != nullptr;
    CUtensorMap maps[8];
    bool ok = e == cudaSuccess && encode_kmajor(&maps[0], bf16, p.A, p.K, p.rows_a, p.lda, 1, p.lda, a.am, a.ksub, 3) &&
              encode_stack(&maps[1], bf16, p.A, p.K, p.rows_a, p.lda, 1, 0, BK, 1, 2);
    const int64_t count = one_b ? 1 : p.groups, stride = one_b ? p.ldb : p.stride_b;
    if (p.b_kmajor)
        ok = ok && encode_kmajor(&maps[2], bf16, p.B, p.K, p.N, p.ldb, count, stride, a.bn / cg,
                                 a.ksub, 4);
    else
        ok = ok && encode_nmajor(&maps[2], &maps[7], bf16, p.B, p.N, p.K, p.ldb, count, stride,
                                 a.bn / cg, a.ksub);
    a.b_blocks = static_cast<int>(p.N / 64);
    if (p.b_kmajor) maps[7] = maps[2];
    maps[3] = maps[4] = maps[5] = maps[6] = maps[2];
    const int64_t max_tiles = (p.rows / (a.am * cg) + live) * a.tiles_n;
    const bool parts = p.out == kOutF32 && p.K > kPart;
    static const char *const kNames[2][2] = {{"grouped_tc<f16>", "grouped_tc<f16,pair>"},
                                             {"grouped_tc<bf16>", "grouped_tc<bf16,pair>"}};
    *name = kNames[bf16][pair];
    if (e == cudaSuccess && !ok) e = cudaErrorInvalidValue;
    if (e == cudaSuccess)
        e = pair ? launch<2, kRows>(maps, a, gather, max_tiles, parts, d, stream)
                 : launch<1, kRows>(maps, a, gather, max_tiles, parts, d, stream);
    return free_after(ws, stream, e);
}

bool wgrad_tc_eligible(const WgradProblem &p) {
    return p.rows > 0 && p.rows_a > 0 && tma_rows(p.A, p.lda) && tma_rows(p.B, p.ldb) &&
           ceil_div(p.M, BM) * ceil_div(p.N, 64) < kMaxTiles / p.groups;
}

cudaError_t launch_wgrad_tc(const WgradProblem &whole, InType in, cudaStream_t stream,
                            const char **name) {
    WgradProblem p = whole;
    const bool bf16 = in == InType::BF16;
    DeviceInfo *d = device_info();
    if (d == nullptr) return cudaErrorInvalidDevice;
    if (d->err != cudaSuccess) return d->err;
    Args a = {};
    a.groups = p.groups;
    a.rows = p.rows;
    a.M = p.M;
    a.N = p.N;
    a.offsets = p.offsets;
    a.row_index = p.row_index;
    const int64_t elt = p.out == kOutF32 ? 4 : 2;
    a.out.D = p.D;
    a.out.ldd = p.ldd;
    a.out.C = p.C;
    a.out.ldc = p.ldc;
    a.out.alpha = p.alpha;
    a.out.beta = p.beta;
    a.out.out = p.out;
    a.out.row_vec = row_alignment(p.D, p.ldd, p.groups > 1 ? p.stride_d : 0, elt);
    if (p.beta != 0.f) {
        // (quads of C are 16 bytes)
        if (row_alignment(p.C, p.ldc, p.groups > 1 ? p.stride_c : 0, 4) < 16) a.out.row_vec = 0;
    }
    a.stride_d = p.stride_d;
    a.stride_c = p.stride_c;
    a.ab_format = bf16 ? 1 : 0;
    const int64_t pair_tiles = p.groups * ceil_div(p.M, 2 * BM) * ceil_div(p.N, 256);
    const bool pair = d->pairs > 0 && p.M > BM && pair_tiles >= d->pairs;
    const int cg = pair ? 2 : 1;
    if (pair) {
        set_tile(a, 2, BM, 256);
    } else {
        int bn = 256;
        while (bn > 64 && p.groups * ceil_div(p.M, BM) * ceil_div(p.N, bn) < 2 * d->sms) bn /= 2;
        set_tile(a, 1, BM, bn);
    }
    a.tiles_m = static_cast<uint32_t>(ceil_div(p.M, BM * cg));
    a.tiles_n = static_cast<uint32_t>(ceil_div(p.N, a.bn));
    CUtensorMap maps[8];
    void *ws = nullptr;
    cudaError_t e = cudaSuccess;
    if (p.row_index != nullptr) {
        int64_t ldo = 0;
        e = order_rows(p.A, p.lda, p.rows_a, p.row_index, p.rows, p.M, d->sms, stream, &ws, &ldo);
        p.A = ws;
        p.lda = ldo;
        p.rows_a = p.rows;
        p.row_index = nullptr;
    }
    const uint32_t boxes_b = static_cast<uint32_t>(a.bn / cg / 64);
    a.a_blocks = static_cast<int>(p.M / 64);
    a.b_blocks = static_cast<int>(p.N / 64);
    bool ok = e == cudaSuccess &&
              encode_stack(&maps[4], bf16, p.A, p.M, p.rows_a, p.lda, 1, 0, 64, BK, 2) &&
              encode_stack(&maps[1], bf16, p.A, p.M, p.rows_a, p.lda, 1, 0, 64, 1, 2) &&
              encode_stack(&maps[7], bf16, p.B, p.N, p.rows, p.ldb, 1, 0, 64, BK, 2) &&
              encode_stack(&maps[3], bf16, p.B, p.N, p.rows, p.ldb, 1, 0, 64, 1, 2);
    maps[0] = maps[4];
    maps[2] = maps[7];
    if (a.a_blocks > 0)
        ok = ok && encode_blocks(&maps[0], bf16, p.A, p.M / 64 * 64, p.rows_a, p.lda, 1, p.lda, BK, 2, 3);
    if (a.b_blocks > 0)
        ok = ok && encode_blocks(&maps[2], bf16, p.B, p.N / 64 * 64, p.rows, p.ldb, 1, p.ldb, BK,
                                 boxes_b, 3);
    maps[5] = maps[6] = maps[3];
    // D and C as TMA boxes: whole 16-byte pieces everywhere
    const int64_t per_16 = 16 / elt;
    auto boxes = [&](const void *q, int64_t ld, int64_t stride, int64_t per) {
        return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld % per == 0 && p.N % per == 0 &&
               (p.groups == 1 || (stride % per == 0 && stride > 0)) && ld < (int64_t(1) << 37) &&
               stride < (int64_t(1) << 37);
    };
    a.staged = ok && boxes(p.D, p.ldd, p.stride_d, per_16) &&
               (p.beta == 0.f || boxes(p.C, p.ldc, p.stride_c, 4));
    if (a.staged) {
        const int64_t sd = p.groups > 1 ? p.stride_d : p.ldd, sc = p.groups > 1 ? p.stride_c : p.ldc;
        if (!encode_box32(&maps[6], static_cast<int>(elt), bf16, p.D, p.N, p.M, p.ldd, p.groups, sd) ||
            (p.beta != 0.f &&
             !encode_box32(&maps[5], 4, false, p.C, p.N, p.M, p.ldc, p.groups, sc)))
            a.staged = 0;
    }
    if (a.staged) take_boxes(a, p.beta != 0.f ? kBoxesC : kBoxes);
    const int64_t max_tiles = p.groups * a.tiles_m * a.tiles_n;
    a.timeout_ns = wait_limit_ns(ceil_div(p.rows, BK), 0, ceil_div(max_tiles * cg, d->sms));
    const bool parts = p.out == kOutF32 && p.rows > kPart;
    static const char *const kNames[2][2] = {{"wgrad_tc<f16>", "wgrad_tc<f16,pair>"},
                                             {"wgrad_tc<bf16>", "wgrad_tc<bf16,pair>"}};
    *name = kNames[bf16][pair];
    if (e == cudaSuccess && !ok) e = cudaErrorInvalidValue;
    if (e == cudaSuccess)
        e = pair ? launch<2, kWgrad>(maps, a, false, max_tiles, parts, d, stream)
                 : launch<1, kWgrad>(maps, a, false, max_tiles, parts, d, stream);
    return free_after(ws, stream, e);
}

bool lora_tc_eligible(const LoraProblem &p) {
    if (p.K == 0 || !tma_rows(p.X, p.ldx) || !tma_rows(p.W, p.ldw) ||
        ceil_div(p.M, 16) * ceil_div(p.N, 32) >= kMaxTiles)
        return false;
    return p.adapters == 0 ||
           (lora_shrink_eligible(p) && tma_rows(p.LB, p.ld_b, p.adapters > 1 ? p.stride_b : 0));
}

cudaError_t launch_lora_tc(const LoraProblem &p, InType in, cudaStream_t stream,
                           const char **name) {
    const bool bf16 = in == InType::BF16;
    DeviceInfo *d = device_info();
    if (d == nullptr) return cudaErrorInvalidDevice;
    if (d->err != cudaSuccess) return d->err;
    Args a = {};
    a.groups = 1;
    a.N = p.N;
    a.out.ldd = p.ldd;
    a.out.bias = p.bias;
    a.out.alpha = 1.f;
    a.out.act = p.act;
    a.out.out = p.out;
    const int64_t elt = p.out == kOutF32 ? 4 : 2;
    a.out.row_vec = row_alignment(p.D, p.ldd, 0, elt);
    a.b_kmajor = p.w_kmajor ? 1 : 0;
    a.ab_format = bf16 ? 1 : 0;
    a.timeout_ns = wait_limit_ns(ceil_div(p.K, BK));
    // and what lora_redo may take meanwhile: up to four blocks a warp, 1 us per
    // step of K in all (16 are allowed)
    if (p.adapters > 0) a.timeout_ns += static_cast<uint64_t>(p.K) * 16000ull;
    const bool parts = p.out == kOutF32 && p.K > kPart;
    const int64_t pair_tiles = ceil_div(p.M, 2 * BM) * ceil_div(p.N, 256);
    const bool pair = d->pairs > 0 && p.M > BM && pair_tiles >= d->pairs;
    const int cg = pair ? 2 : 1;
    if (pair) {
        set_tile(a, 2, BM, 256);
    } else {
        const int am = p.M <= 16 ? 16 : (p.M <= 32 ? 32 : (p.M <= 64 ? 64 : BM));
        // the narrowest tiles that still fill the SMs once (all K-major: in
        // steps of 32 columns; an N-major operand comes in blocks of 64)
        const int step = p.w_kmajor && (p.adapters == 0 || p.b_kmajor) ? 32 : 64;
        const int64_t per_row = d->sms / ceil_div(p.M, am) > 0 ? d->sms / ceil_div(p.M, am) : 1;
        int64_t bn = ceil_div(ceil_div(p.N, per_row), step) * step;
        if (bn > 256) bn = 256;
        set_tile(a, 1, am, static_cast<int>(bn), sub_blocks(p.K, am, static_cast<int>(bn)),
                 p.M <= BM && !parts ? kShortRing : kRingBytes);
    }
    a.num_kb = static_cast<int>(ceil_div(p.K, BK * a.ksub));
    a.tiles_n = static_cast<uint32_t>(ceil_div(p.N, a.bn));
    static const char *const kNames[2][2] = {{"lora_tc<f16>", "lora_tc<f16,pair>"},
                                             {"lora_tc<bf16>", "lora_tc<bf16,pair>"}};
    *name = kNames[bf16][pair];

    LoraPlan plan = {};
    plan.tile_rows = a.am * cg;
    int64_t chunk = p.M;  // rows per launch
    void *ws = nullptr;
    size_t v_bytes = 0, count_bytes = 0, list_bytes = 0;
    if (p.adapters > 0) {
        plan.r_pad = 16;
        while (plan.r_pad < p.rank) plan.r_pad *= 2;
        // a 16-bit D is rounded to the inputs' type itself: one rounding of
        // the first product is of the same size; an FP32 D takes two parts
        plan.rc = p.out == kOutF32 ? 2 * plan.r_pad : plan.r_pad;
        const int64_t slots = p.adapters < plan.tile_rows ? p.adapters : plan.tile_rows;
        plan.ldv = ceil_div(slots * plan.rc, BK) * BK;
        // V is at most 128 MiB: more rows go in several launches
        const int64_t fit = (int64_t(128) << 20) / (plan.ldv * 2) / plan.tile_rows * plan.tile_rows;
        const int64_t most = fit > plan.tile_rows ? fit : plan.tile_rows;
        if (chunk > most) chunk = most;
        const int64_t tiles = ceil_div(chunk, plan.tile_rows);
        v_bytes = static_cast<size_t>(tiles * plan.tile_rows * plan.ldv * 2);
        count_bytes = static_cast<size_t>(ceil_div(tiles * 4, 256) * 256);
        list_bytes = static_cast<size_t>(tiles * plan.tile_rows * 4);
        list_bytes = static_cast<size_t>(ceil_div(static_cast<int64_t>(list_bytes), 256) * 256);
        const size_t part_bytes = lora_shrink_part_bytes(chunk, plan.r_pad);
        cudaError_t e =
            workspace_alloc(v_bytes + count_bytes + 2 * list_bytes + part_bytes, stream, &ws);
        if (e != cudaSuccess) return e;
        uint8_t *at = static_cast<uint8_t *>(ws);
        plan.V = reinterpret_cast<uint16_t *>(at);
        plan.count = reinterpret_cast<int *>(at + v_bytes);
        plan.list = reinterpret_cast<int *>(at + v_bytes + count_bytes);
        plan.slot = reinterpret_cast<int *>(at + v_bytes + count_bytes + list_bytes);
        plan.part = reinterpret_cast<float *>(at + v_bytes + count_bytes + 2 * list_bytes);
    }
    cudaError_t e = cudaSuccess;
    for (int64_t row = 0; row < p.M && e == cudaSuccess; row += chunk) {
        const int64_t rows = p.M - row < chunk ? p.M - row : chunk;
        LoraProblem l = p;
        l.M = rows;
        l.X = static_cast<const uint16_t *>(p.X) + row * p.ldx;
        l.adapter = p.adapters > 0 ? p.adapter + row : nullptr;
        a.rows = rows;
        a.tiles_m = static_cast<uint32_t>(ceil_div(rows, plan.tile_rows));
        a.out.D = static_cast<uint8_t *>(p.D) + row * p.ldd * elt;
        a.l = l;
        a.plan = plan;
        if (p.adapters > 0) {
            e = launch_lora_shrink(l, plan, in, stream);
            if (e != cudaSuccess) break;
            a.late_wait = 1;
        }
        CUtensorMap maps[8];
        bool ok = encode_kmajor(&maps[0], bf16, l.X, p.K, rows, p.ldx, 1, p.ldx, a.am, a.ksub, 3);
        if (p.w_kmajor)
            ok = ok && encode_kmajor(&maps[2], bf16, p.W, p.K, p.N, p.ldw, 1, p.ldw, a.bn / cg,
                                     a.ksub, 4);
        else
            ok = ok && encode_nmajor(&maps[2], &maps[7], bf16, p.W, p.N, p.K, p.ldw, 1, p.ldw,
                                     a.bn / cg, a.ksub);
        a.b_blocks = static_cast<int>(p.N / 64);
        if (p.w_kmajor) maps[7] = maps[2];
        maps[1] = maps[3] = maps[4] = maps[5] = maps[6] = maps[2];
        if (p.adapters > 0) {
            const bool one_lb = p.adapters == 1 || p.stride_b == 0;
            const int64_t stride = one_lb ? p.ld_b : p.stride_b;
            const int64_t count = one_lb ? 1 : p.adapters;
            a.lb_z_step = one_lb ? 0 : 1;
            if (p.b_kmajor)
                ok = ok && encode_stack(&maps[3], bf16, p.LB, p.rank, p.N, p.ld_b, count, stride,
                                        16, static_cast<uint32_t>(a.bn / cg), 3,
                                        CU_TENSOR_MAP_SWIZZLE_32B);
            else
                ok = ok && encode_stack(&maps[3], bf16, p.LB, p.N, p.rank, p.ld_b, count, stride,
                                        64, 16, 3);
            ok = ok && encode_stack(&maps[4], bf16, plan.V, plan.ldv,
                                    static_cast<int64_t>(a.tiles_m) * plan.tile_rows, plan.ldv, 1,
                                    0, BK, static_cast<uint32_t>(a.am), 2);
        }
        if (!ok) {
            e = cudaErrorInvalidValue;
            break;
        }
        const int64_t tiles = static_cast<int64_t>(a.tiles_m) * a.tiles_n;
        a.slice_warp = !pair && p.adapters > 0 && tiles <= d->sms;
        e = pair ? launch<2, kLora>(maps, a, false, tiles, parts, d, stream)
                 : launch<1, kLora>(maps, a, false, tiles, parts, d, stream);
    }
    return free_after(ws, stream, e);
}

cudaError_t grouped_tc_read_and_clear_status(cudaStream_t stream, int *status) {
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
