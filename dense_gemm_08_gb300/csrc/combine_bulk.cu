// combine_bulk.cu -- the combination and its gradients (combine.cu) for large
// batches of long rows: rows of Y come by asynchronous bulk copies.
//
// A CTA takes tokens one after another, a token in steps of up to eight rows and a
// run of columns.  One warp has each row's run (and the residual's, or dD's) copied
// into a stage of shared memory, as many stages ahead as fit; the number and weight
// of each row go with it.  Two groups of four warps (or four of two) take a token
// each.  So some 70 to 100 KB per CTA, two per SM, are under way at any time, whatever
// the rows' number and without registers: 6.8 TB/s, where loads into registers
// (combine.cu) reached 5.1 with 8 rows and less with fewer.
#include <atomic>
#include <type_traits>

#include "combine.h"
#include "internal.h"
#include "tcgen05.cuh"

namespace gemm {
namespace {

using namespace tc;

constexpr int kRows = 8;         // of a stage at most
constexpr int kWarps = 8;        // that sum, in groups of 2 or 4 that take a token
constexpr int kMaxGroups = 4;
constexpr int kThreads = 32 * kWarps + 32;
constexpr int kMaxStages = 16;
constexpr int kRing = 104 * 1024;
// what goes with a stage: the rows' numbers (-1: none) and weights
struct __align__(16) Meta {
    int32_t at[kRows];
    float w[kRows];
};
// ring, meta, dot products of the warps (two sets of them), barriers, alignment
constexpr int kSmemBytes = 128 + kRing + kMaxStages * static_cast<int>(sizeof(Meta)) +
                           2 * kWarps * kRows * 4 + (kMaxGroups + 1) * kMaxStages * 8 + 16;
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");

struct BulkArgs {
    CombineProblem p;
    int rows, j_steps;      // rows per step, steps of rows per token
    int cols, chunks;       // columns per step, runs of columns per row
    int stages;
    uint32_t row_bytes, stage_bytes;
    bool extra;             // the residual's, or dD's, run comes by bulk copy too
    bool dvec;              // rows of D and the residual start on 16 bytes
    uint64_t timeout_ns;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar)
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

template <int YT, int DT, bool GRAD, int WARPS>
__global__ void __launch_bounds__(kThreads, 2)
    combine_bulk_kernel(const __grid_constant__ BulkArgs a) {
    using Y = Value<YT>;
    using D = Value<DT>;
    constexpr int WIDE = Y::PER_16, GROUPS = kWarps / WARPS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                                      ~static_cast<uintptr_t>(127));
    Meta *const meta = reinterpret_cast<Meta *>(ring + kRing);
    float *const parts = reinterpret_cast<float *>(meta + kMaxStages);  // [GROUPS][2][WARPS][kRows]
    constexpr int kParts = 2 * kWarps * kRows;
    const uint32_t ring0 = smem_addr(ring);
    // barriers: full[GROUPS][kMaxStages] copies -> the group the stage is for,
    // empty[kMaxStages] sums -> copies.  (A full barrier per group: a group waits for
    // each of its own stages in turn, so one parity bit per stage tells them apart;
    // with one for both it could take a stage that the other has not seen yet for
    // its own.)
    const uint32_t full0 = smem_addr(parts + kParts), empty0 = full0 + 8 * GROUPS * kMaxStages;
    volatile int *const abort_flag =
        reinterpret_cast<volatile int *>(parts + kParts + 2 * (GROUPS + 1) * kMaxStages);
    const CombineProblem &p = a.p;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            for (int g = 0; g < GROUPS; ++g) mbar_init(full0 + 8 * (g * kMaxStages + s), 1);
            mbar_init(empty0 + 8 * s, WARPS);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
        const bool done = __all_sync(
            0xffffffffu, wait_bounded(bar, parity, abort_flag, a.timeout_ns));
        if (!done && lane == 0) raise_abort(abort_flag);
        return done;
    };
    // A token's steps: forward all rows of a run of columns (their sum stays in
    // registers), gradient all columns of a set of rows (so do its dot products).
    const uint32_t steps = a.j_steps * a.chunks;
    auto set_of = [&](int s) { return GRAD ? s / a.chunks : s % a.j_steps; };
    auto run_of = [&](int s) { return GRAD ? s % a.chunks : s / a.j_steps; };
    auto cols_of = [&](int c) {
        const int64_t left = p.N - static_cast<int64_t>(c) * a.cols;
        return left < a.cols ? static_cast<int>(left) : a.cols;
    };
    const bool with_y = !GRAD || p.dweights != nullptr;
    int stage = 0;

    if (warp == kWarps) {
        // ------------------------------------------------------- copies
        // The rows' numbers and weights are loaded for 32 rows at a time, some steps
        // ahead: with those of the next step alone under way, every step waited for
        // their latency (8190 tokens, 2 rows of 2048 FP16, gradient: 40 us, now 33).
        const uint32_t per = 32 / a.rows;  // steps
        auto advance = [&](int64_t &t, uint32_t &s, uint32_t by) {
            s += by;
            t += static_cast<int64_t>(s / steps) * gridDim.x;
            s %= steps;
        };
        auto choices = [&](int64_t t, uint32_t s, int32_t &at, float &w) {
            advance(t, s, lane / a.rows);
            const int64_t j = static_cast<int64_t>(set_of(s)) * a.rows + lane % a.rows;
            at = -1;
            w = 1.f;
            if (t < p.tokens && j < p.k) {
                at = __ldg(p.position + t * p.k + j);
                if (p.weights != nullptr) w = __ldg(p.weights + t * p.k + j);
            }
            if (at >= p.rows_y) at = -1;
        };
        int32_t ats, next_ats;
        float ws, next_ws;
        int64_t t = blockIdx.x;
        uint32_t s = 0;
        choices(t, s, ats, ws);
        uint32_t phase = 0;           // of the empty barriers
        uint32_t told[GROUPS] = {};  // bit s: parity of the next copies on the group's full[s]
        uint32_t group = 0, used[GROUPS] = {};  // bit s: stage s was filled last for the group
        bool ok = true;
        for (; ok && t < p.tokens; ats = next_ats, ws = next_ws) {
            {
                int64_t t_next = t;
                uint32_t s_next = s;
                advance(t_next, s_next, per);
                choices(t_next, s_next, next_ats, next_ws);
            }
            for (uint32_t b = 0; b < per && t < p.tokens; ++b) {
                int32_t at = __shfl_sync(0xffffffffu, ats, (b * a.rows + lane) % 32);
                const float w = __shfl_sync(0xffffffffu, ws, (b * a.rows + lane) % 32);
                if (lane >= a.rows) at = -1;
                ok = wait_all(empty0 + 8 * stage, phase ^ 1);
                if (!ok) break;
                const int c = run_of(s), cols = cols_of(c);
                // whole 16 bytes: up to those that hold the row's end (the rest of them is
                // the pitch before the next row), of the last row up to its end
                const uint32_t y_most = with_y ? static_cast<uint32_t>(cols * Y::BYTES + 15) & ~15u : 0u;
                const uint32_t y_least = with_y ? static_cast<uint32_t>(cols * Y::BYTES) & ~15u : 0u;
                const uint32_t y_bytes = at + 1 < p.rows_y ? y_most : y_least;
                const uint32_t d_bytes =
                    !a.extra ? 0u : static_cast<uint32_t>(cols * D::BYTES + (t + 1 < p.tokens ? 15 : 0)) & ~15u;
                const uint32_t have = __ballot_sync(0xffffffffu, at >= 0);
                const uint32_t lasts = __ballot_sync(0xffffffffu, at >= 0 && at + 1 == p.rows_y);
                if (lane < kRows) {
                    meta[stage].at[lane] = at;
                    meta[stage].w[lane] = w;
                }
                __syncwarp();
                const uint32_t bar = full0 + 8 * (group * kMaxStages + stage), to = ring0 + stage * a.stage_bytes;
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, __popc(have & ~lasts) * y_most + __popc(lasts) * y_least + d_bytes);
                __syncwarp();
                const int64_t c0 = static_cast<int64_t>(c) * a.cols;
                if (at >= 0 && y_bytes != 0)
                    bulk_load(to + lane * a.row_bytes,
                              static_cast<const uint8_t *>(p.Y) + (at * p.ldy + c0) * Y::BYTES, y_bytes, bar);
                if (lane == 31 && d_bytes != 0) {
                    const uint8_t *from =
                        GRAD ? static_cast<const uint8_t *>(p.D) + (t * p.ldd + c0) * D::BYTES
                             : static_cast<const uint8_t *>(p.residual) + (t * p.ld_r + c0) * D::BYTES;
                    bulk_load(to + a.rows * a.row_bytes, from, d_bytes, bar);
                }
                const uint32_t bit = 1u << stage;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    told[g] ^= group == g ? bit : 0u;
                    used[g] = group == g ? used[g] | bit : used[g] & ~bit;
                }
                if (++stage == a.stages) {
                    stage = 0;
                    phase ^= 1;
                }
                if (++s == steps) {
                    s = 0;
                    t += gridDim.x;
                    group = (group + 1) % GROUPS;
                }
            }
        }
        __syncwarp();
        // the copies in flight land before the CTA exits
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
            for (int i = 0; i < a.stages; ++i) {
                if (!((used[g] >> i) & 1u)) continue;
                const volatile int never = 0;
                if (!wait_bounded(full0 + 8 * (g * kMaxStages + i), ((told[g] >> i) & 1u) ^ 1u, &never,
                                  a.timeout_ns))
                    raise_abort(abort_flag);
            }
        return;
    }

    // ------------------------------------------------------------- sums
    const int group = warp / WARPS, tid = threadIdx.x - group * 32 * WARPS;
    uint32_t flip = 0;  // which of the two sets of parts
    bool ok = true;     // (after a wait that ran out the warps still meet at their barrier)
    uint32_t seen = 0;  // bit s: parity of the next copies on this group's full[s]
    auto skip_tokens = [&](uint32_t n) { stage = (stage + n * steps) % a.stages; };  // other groups' stages
    skip_tokens(group);
    for (int64_t t = blockIdx.x + static_cast<int64_t>(group) * gridDim.x; t < p.tokens;
         t += static_cast<int64_t>(GROUPS) * gridDim.x, skip_tokens(GROUPS - 1)) {
        float sum[WIDE] = {};    // forward, several sets of rows: one piece per thread
        float dot[kRows] = {};   // gradient
        for (uint32_t s = 0; s < steps; ++s) {
            ok = ok && wait_all(full0 + 8 * (group * kMaxStages + stage), (seen >> stage) & 1u);
            seen ^= 1u << stage;
            const int c = run_of(s), set = set_of(s), cols = cols_of(c);
            const uint32_t from = ring0 + stage * a.stage_bytes, extra = from + a.rows * a.row_bytes;
            int32_t at[kRows];
            float w[kRows];
            int lowest = 0;
#pragma unroll
            for (int j = 0; j < kRows; j += 4) {
                const int4 q = *reinterpret_cast<const int4 *>(meta[stage].at + j);
                const float4 u = *reinterpret_cast<const float4 *>(meta[stage].w + j);
                at[j] = q.x, at[j + 1] = q.y, at[j + 2] = q.z, at[j + 3] = q.w;
                w[j] = u.x, w[j + 1] = u.y, w[j + 2] = u.z, w[j + 3] = u.w;
            }
#pragma unroll
            for (int j = 0; j < kRows; ++j)
                if (j < a.rows) lowest = min(lowest, at[j]);
            // One piece.  ALL: every row of the step is there and the piece is whole.
            auto take = [&](int piece, int n, auto all_rows) {
                constexpr bool ALL = decltype(all_rows)::value;
                const int64_t c0 = static_cast<int64_t>(c) * a.cols + piece * WIDE;
                float d[WIDE] = {};  // the residual's or dD's piece
                if (a.extra && (ALL || n == WIDE || t + 1 < p.tokens)) {
#pragma unroll
                    for (int i = 0; i < WIDE / D::PER_16; ++i) {
                        float v[D::PER_16];
                        // (past a row's end: what the pitch holds, below not used)
                        D::unpack(ld_shared_u4(extra + (piece * (WIDE / D::PER_16) + i) * 16), v);
#pragma unroll
                        for (int u = 0; u < D::PER_16; ++u) d[i * D::PER_16 + u] = v[u];
                    }
                } else if (GRAD) {
                    load_values<DT, kSome, WIDE>(p.D, t * p.ldd, c0, n, false, d);
                } else if (p.residual != nullptr && set == a.j_steps - 1) {
                    load_values<DT, kSome, WIDE>(p.residual, t * p.ld_r, c0, n, false, d);
                }
#pragma unroll
                for (int j = 0; j < kRows; ++j) {
                    if (ALL ? j >= a.rows : at[j] < 0) continue;
                    if (GRAD && p.dY != nullptr) {
                        float g[WIDE];
#pragma unroll
                        for (int i = 0; i < WIDE; ++i) g[i] = w[j] * d[i];
                        if (ALL || n == WIDE)
                            store_values<YT, kAll, WIDE>(p.dY, at[j] * p.ld_dy, c0, n, true, g);
                        else
                            store_values<YT, kSome, WIDE>(p.dY, at[j] * p.ld_dy, c0, n, true, g);
                    }
                    if (!with_y) continue;
                    float y[WIDE];
                    // (of the last row the end that is no whole 16 bytes was not copied)
                    Y::unpack(ALL || n == WIDE || at[j] + 1 < p.rows_y
                                  ? ld_shared_u4(from + j * a.row_bytes + piece * 16)
                                  : load_piece<YT, false, kSome>(p.Y, at[j] * p.ldy, c0, n),
                              y);
#pragma unroll
                    for (int i = 0; i < WIDE; ++i) {
                        if constexpr (GRAD) {
                            if (ALL || i < n) dot[j] = fmaf(d[i], y[i], dot[j]);
                        } else {
                            sum[i] = fmaf(w[j], y[i], sum[i]);
                        }
                    }
                }
                if (!GRAD && set == a.j_steps - 1) {
#pragma unroll
                    for (int i = 0; i < WIDE; ++i) sum[i] += d[i];
                    if (ALL || n == WIDE)
                        store_values<DT, kAll, WIDE>(p.D, t * p.ldd, c0, n, a.dvec, sum);
                    else
                        store_values<DT, kSome, WIDE>(p.D, t * p.ldd, c0, n, a.dvec, sum);
#pragma unroll
                    for (int i = 0; i < WIDE; ++i) sum[i] = 0.f;
                }
            };
            for (int piece = tid; ok && piece * WIDE < cols; piece += 32 * WARPS) {
                const int n = cols - piece * WIDE < WIDE ? cols - piece * WIDE : WIDE;
                if (lowest == 0 && n == WIDE)
                    take(piece, WIDE, std::true_type());
                else
                    take(piece, n, std::false_type());
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * stage);
            if (++stage == a.stages) stage = 0;
            if (GRAD && with_y && c == a.chunks - 1) {
                float *const mine = parts + ((group * 2 + flip) * WARPS + warp % WARPS) * kRows;
                float all = 0.f;
#pragma unroll
                for (int j = 0; j < kRows; ++j) {
#pragma unroll
                    for (int i = 16; i > 0; i >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], i);
                    all = lane == j ? dot[j] : all;
                    dot[j] = 0.f;
                }
                if (lane < kRows) mine[lane] = all;
                asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * WARPS) : "memory");
                const int64_t j = static_cast<int64_t>(set) * a.rows + lane;
                if (ok && warp % WARPS == 0 && lane < a.rows && j < p.k) {
                    for (int i = 1; i < WARPS; ++i) all += mine[i * kRows + lane];
                    int32_t mine_at = -1;
#pragma unroll
                    for (int i = 0; i < kRows; ++i) mine_at = lane == i ? at[i] : mine_at;
                    p.dweights[t * p.k + j] = mine_at >= 0 ? all : 0.f;
                }
                flip ^= 1;
            }
        }
    }
}

constexpr int kMaxDevices = 64;
std::atomic<bool> g_launched[kMaxDevices];

template <int YT, int DT, bool GRAD, int WARPS>
cudaError_t launch_groups(const BulkArgs &a, cudaStream_t stream) {
    const auto kernel = combine_bulk_kernel<YT, DT, GRAD, WARPS>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    set_pdl_attribute(&attr);
    cudaLaunchConfig_t cfg = {};
    const int64_t most = 2 * int64_t(sm_count());
    cfg.gridDim = dim3(static_cast<unsigned>(a.p.tokens < most ? a.p.tokens : most), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int YT, int DT, bool GRAD>
cudaError_t launch_as(const CombineProblem &p, cudaStream_t stream) {
    using Y = Value<YT>;
    using D = Value<DT>;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    BulkArgs a = {};
    a.p = p;
    a.rows = 1;
    while (a.rows < p.k && a.rows < kRows) a.rows *= 2;
    a.j_steps = static_cast<int>((p.k + a.rows - 1) / a.rows);
    // 32 KB of Y per step, up to 8 KB of a row: a copy takes the producer some 100 ns
    // to issue (8 rows of 4096 BF16, 16384 tokens: 229 us with 2 KB of a row per copy,
    // 197 with 4).  With several sets of rows a thread keeps one piece's sum: 2 KB.
    int bytes = (a.j_steps > 1 ? 16384 : 32768) / a.rows;
    if (bytes > 8192) bytes = 8192;
    const int64_t row_bytes = (p.N * Y::BYTES + 15) / 16 * 16;
    if (row_bytes < bytes) bytes = static_cast<int>(row_bytes);
    a.row_bytes = static_cast<uint32_t>(bytes);
    a.cols = bytes / Y::BYTES;
    a.chunks = static_cast<int>((p.N + a.cols - 1) / a.cols);
    a.dvec = rows_on_16(p.D, p.ldd, D::BYTES) &&
             (GRAD || p.residual == nullptr || rows_on_16(p.residual, p.ld_r, D::BYTES));
    a.extra = a.dvec && (GRAD || p.residual != nullptr);
    a.stage_bytes = static_cast<uint32_t>(a.rows) * a.row_bytes +
                    (a.extra ? static_cast<uint32_t>(a.cols * D::BYTES) : 0u);
    a.stage_bytes = (a.stage_bytes + 127) / 128 * 128;
    const int fit = kRing / static_cast<int>(a.stage_bytes);
    a.stages = fit < kMaxStages ? fit : kMaxStages;
    a.timeout_ns = 1000000000ull;  // (a stage's copies, or the sums of one)
    g_launched[dev].store(true);
    // A token whose step is short is mostly latency: four groups of two warps (us, two
    // groups of four / four of two, BF16, gradient: 16384 tokens, 2 rows of 1024 52 / 44,
    // 1 of 4096 78 / 64, 8 of 1024 102 / 100, 8 of 2048 186 / 196; forward: 2 rows of
    // 2048 46 / 44, 4 of 2048 63.6 / 62.9, 8 of 2048 103 / 116).
    if (a.j_steps == 1 && a.rows * bytes <= 16384) return launch_groups<YT, DT, GRAD, 2>(a, stream);
    return launch_groups<YT, DT, GRAD, 4>(a, stream);
}

template <bool GRAD>
cudaError_t launch_types(const CombineProblem &p, cudaStream_t stream) {
    if (p.y_type == kOutF32) return launch_as<kOutF32, kOutF32, GRAD>(p, stream);
    if (p.y_type == kOutBf16)
        return p.d_type == kOutF32 ? launch_as<kOutBf16, kOutF32, GRAD>(p, stream)
                                   : launch_as<kOutBf16, kOutBf16, GRAD>(p, stream);
    return p.d_type == kOutF32 ? launch_as<kOutF16, kOutF32, GRAD>(p, stream)
                               : launch_as<kOutF16, kOutF16, GRAD>(p, stream);
}

}  // namespace

bool combine_bulk_eligible(const CombineProblem &p, bool grad) {
    const int64_t bytes = value_bytes(p.y_type);
    if (p.k == 0 || p.N == 0 || p.rows_y == 0) return false;
    // A step costs some time whatever its bytes, so rows must be long; and the
    // pipeline must run for a while.  Both ways measured in BF16, loads / bulk, us:
    //   forward   16384 tokens, 8 rows: 2048 columns 132 / 103, 1024 columns 68 / 62,
    //             768 columns 53 / 56, 512 columns 36 / 55; 4 rows of 1024 46 / 45;
    //             2 rows: 4096 columns 110 / 83, 2048 columns 56 / 44, 1024 30 / 40;
    //             4096 tokens, 2 rows of 2048: 15.2 / 13.8; 512, 8 of 4096: 10.9 / 11.1
    //   gradient  16384 tokens, 8 rows: 1024 columns 110 / 100, 512 columns 58 / 61;
    //             4 rows of 640 75 / 49, 512 42 / 47; 2 rows: 2048 columns 114 / 64,
    //             1024 58 / 44;
    //             1 row: 4096 columns 73 / 64, 2048 38 / 44; 2048 tokens, 2 rows of
    //             2048 17.8 / 12.0, 1 row of 4096 12.4 / 13.8
    // (a token's steps are counted in 31 bits; no step has less than 4 KB)
    if (p.k > (int64_t(1) << 20) || p.N > (int64_t(1) << 28) || p.k * p.N > (int64_t(1) << 40))
        return false;
    const int64_t row = p.N * bytes;
    auto all_mb = [&](int64_t mb) { return p.tokens * p.k >= ((mb << 20) + row - 1) / row; };
    if (grad) {
        if (row < 1280 || row * p.k < 4096 || !all_mb(16)) return false;
        if (p.k == 1 && (row < 8192 || !all_mb(64))) return false;
    } else {
        if (row < 2048 || row * p.k < 8192 || !all_mb(32)) return false;
    }
    if (grad)
        return (p.dweights == nullptr || rows_on_16(p.Y, p.ldy, bytes)) &&
               (p.dY == nullptr || rows_on_16(p.dY, p.ld_dy, bytes));
    return rows_on_16(p.Y, p.ldy, bytes);
}

cudaError_t launch_combine_bulk(const CombineProblem &p, bool grad, cudaStream_t stream) {
    return grad ? launch_types<true>(p, stream) : launch_types<false>(p, stream);
}

cudaError_t combine_read_and_clear_status(cudaStream_t stream, int *status) {
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
