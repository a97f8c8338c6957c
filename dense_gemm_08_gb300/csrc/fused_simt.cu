// fused_simt.cu -- the fused products on the CUDA cores.
//
// Large FP32 products (no TF32): the library's FP32 product (launch_f32) into D --
// into the value before the activation where that is kept -- and one pass over it
// (fused_finish_kernel: bias, activation, residual, slopes, column sums).
//
// Small FP32 products, and 16-bit inputs that TMA cannot describe: tiles of 64 x 64
// (4 x 4 sums per thread); slices of 16 of K come through registers into two
// shared-memory buffers, sums are paired FMAs.  Few tiles: K is split over a cluster,
// whose CTAs add each other's sums through distributed shared memory, each for its
// share of the tile's rows and in the order of the pieces.  The tile then lies in
// shared memory, and a thread finishes one of its columns.
//
// A row or two of A (up to four in FP32, or where B is small) and a K-contiguous B:
// warps stream B's columns once (fused_rows_kernel).
#include <atomic>
#include <type_traits>

#include "fused.cuh"
#include "mixture.h"
#include "values.cuh"

namespace gemm {
namespace {

constexpr int BK = 16;
constexpr int THREADS = 256;

// What follows the sum of one value; D's value before rounding.
template <int TYPE>
__device__ __forceinline__ float finish(const FusedProblem &p, float sum, int64_t r, int64_t c,
                                        float bias) {
    using V = Value<TYPE>;
    float d;
    if (p.grad) {
        d = p.alpha * sum;
        if (p.act != kActNone) d *= fused_slope(V::load(p.pre, r * p.ld_pre + c), p.act);
    } else {
        const float z = fmaf(p.alpha, sum, bias);
        if (p.pre != nullptr) V::store(p.pre, r * p.ld_pre + c, z);
        d = fused_activation(z, p.act);
        if (p.residual != nullptr) d += V::load(p.residual, r * p.ld_r + c);
    }
    V::store(p.D, r * p.ldd + c, d);
    return d;
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_of_rank(uint32_t addr, int rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// Two products added to two sums, each rounded as fmaf.
__device__ __forceinline__ void fma_pair(float2 &acc, float2 a, float2 b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<uint64_t &>(acc))
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
}

constexpr int kTile = 64;             // rows and columns of a tile
constexpr int kPitch = kTile + 4;     // of a slice's rows
constexpr int kOutPitch = kTile + 1;  // of the finished tile's
constexpr int kLoads = kTile * BK / THREADS;
constexpr int kSliceFloats = 4 * BK * kPitch;  // two buffers of A's and B's
constexpr int kTileFloats =
    kSliceFloats > kTile * kOutPitch ? kSliceFloats : kTile * kOutPitch;

// ks pieces of K per tile (cluster), blockIdx.x = tile * ks + piece.
template <int TYPE>
__global__ void __launch_bounds__(THREADS)
    fused_tile_kernel(const __grid_constant__ FusedProblem p, int64_t tiles_n, int ks, float *part) {
    using V = Value<TYPE>;
    constexpr int T = kTile;
    extern __shared__ __align__(16) float smem[];
    float *const sa = smem, *const sb = smem + 2 * BK * kPitch;
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int64_t tile = blockIdx.x / ks;
    const int piece = static_cast<int>(blockIdx.x % ks);
    const int64_t m0 = tile / tiles_n * T, n0 = tile % tiles_n * T;
    const int64_t slices = (p.K + BK - 1) / BK;
    const int64_t first = slices * piece / ks, end = slices * (piece + 1) / ks;
    pdl_wait();
    pdl_launch_dependents();

    // the values of a slice that this thread brings: K fastest where K is contiguous
    float ra[kLoads], rb[kLoads];
    auto where = [&](bool kmajor, int i, int &k, int &x) {
        const int v = tid + i * THREADS;
        k = kmajor ? v % BK : v / T;
        x = kmajor ? v / BK : v % T;
    };
    auto fetch = [&](int64_t slice) {
        const int64_t k0 = slice * BK;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            int k, x;
            where(p.a_kmajor, i, k, x);
            ra[i] = m0 + x < p.M && k0 + k < p.K
                        ? V::load(p.A, p.a_kmajor ? (m0 + x) * p.lda + k0 + k : (k0 + k) * p.lda + m0 + x)
                        : 0.f;
            where(p.b_kmajor, i, k, x);
            rb[i] = n0 + x < p.N && k0 + k < p.K
                        ? V::load(p.B, p.b_kmajor ? (n0 + x) * p.ldb + k0 + k : (k0 + k) * p.ldb + n0 + x)
                        : 0.f;
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            int k, x;
            where(p.a_kmajor, i, k, x);
            sa[(buf * BK + k) * kPitch + x] = ra[i];
            where(p.b_kmajor, i, k, x);
            sb[(buf * BK + k) * kPitch + x] = rb[i];
        }
    };
    float2 acc[4][2] = {};
    if (first < end) {
        fetch(first);
        put(0);
    }
    __syncthreads();
    for (int64_t s = first; s < end; ++s) {
        const int buf = static_cast<int>(s - first) & 1;
        if (s + 1 < end) fetch(s + 1);
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            const float *a = sa + (buf * BK + k) * kPitch, *b = sb + (buf * BK + k) * kPitch;
            const float4 av = *reinterpret_cast<const float4 *>(a + ty * 4);
            const float4 bv = *reinterpret_cast<const float4 *>(b + tx * 4);
            const float ai[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fma_pair(acc[i][0], make_float2(ai[i], ai[i]), make_float2(bv.x, bv.y));
                fma_pair(acc[i][1], make_float2(ai[i], ai[i]), make_float2(bv.z, bv.w));
            }
        }
        if (s + 1 < end) put(buf ^ 1);
        __syncthreads();
    }

    // the sums into shared memory, in place of the slices
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float *to = smem + (ty * 4 + i) * kOutPitch + tx * 4;
        to[0] = acc[i][0].x, to[1] = acc[i][0].y, to[2] = acc[i][1].x, to[3] = acc[i][1].y;
    }
    if (ks > 1)
        cluster_sync_all();
    else
        __syncthreads();
    // this CTA's rows of the tile
    const int rows = T / ks, row0 = piece * rows;
    const int col = tid % T, lanes = THREADS / T;
    const bool inside = n0 + col < p.N;
    const float bias = !p.grad && p.bias != nullptr && inside ? p.bias[n0 + col] : 0.f;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    float column = 0.f;
    for (int r = row0 + tid / T; r < row0 + rows; r += lanes) {
        float sum = 0.f;
        if (ks > 1) {
            for (int q = 0; q < ks; ++q)
                sum += ld_of_rank(base + static_cast<uint32_t>(r * kOutPitch + col) * 4u, q);
        } else {
            sum = smem[r * kOutPitch + col];
        }
        if (inside && m0 + r < p.M) column += finish<TYPE>(p, sum, m0 + r, n0 + col, bias);
    }
    if (ks > 1)
        cluster_sync_all();  // the others have read this CTA's sums
    else
        __syncthreads();
    if (p.grad && p.dbias != nullptr) {
        smem[tid] = column;
        __syncthreads();
        if (tid < T && inside) {
            for (int i = 1; i < lanes; ++i) column += smem[i * T + tid];
            part[((m0 / T) * ks + piece) * p.N + n0 + col] = column;
        }
    }
}

// ------------------------------------------------------------- few rows of A
// D for up to ROWS rows of A and a K-contiguous B: `split` warps of a CTA share a
// column's K, 16 bytes a lane and eight loads of B in flight; their sums are added
// in order.  B is read once, A comes from L1.
constexpr int kRowsWarps = 8;
template <int TYPE, int ROWS>
__global__ void __launch_bounds__(32 * kRowsWarps)
    fused_rows_kernel(const __grid_constant__ FusedProblem p, int split) {
    using V = Value<TYPE>;
    constexpr int W = V::PER_16, AHEAD = 8;
    __shared__ float sums[kRowsWarps][ROWS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per_cta = kRowsWarps / split;
    const int64_t n = blockIdx.x * int64_t(per_cta) + warp / split;
    const int piece = warp % split;
    const bool inside = n < p.N;
    // K in steps of 32 * W, the steps dealt out to the warps in runs
    const int64_t steps = (p.K + 32 * W - 1) / (32 * W);
    const int64_t first = steps * piece / split, end = steps * (piece + 1) / split;
    const uint8_t *const b = static_cast<const uint8_t *>(p.B) + (inside ? n : 0) * p.ldb * V::BYTES;
    pdl_wait();
    pdl_launch_dependents();
    float sum[ROWS] = {};
    // N whole steps from s on: all loads of B first, then A from L1
    auto whole_steps = [&](int64_t s, auto count) {
        constexpr int n = decltype(count)::value;
        uint4 q[n];
#pragma unroll
        for (int u = 0; u < n; ++u)
            q[u] = __ldcs(reinterpret_cast<const uint4 *>(b + ((s + u) * 32 + lane) * W * V::BYTES));
#pragma unroll
        for (int u = 0; u < n; ++u) {
            float bv[W];
            V::unpack(q[u], bv);
#pragma unroll
            for (int m = 0; m < ROWS; ++m) {
                if (ROWS > 2 && m >= p.M) continue;  // (ROWS up to 2 is M)
                float av[W];
                V::unpack(__ldg(reinterpret_cast<const uint4 *>(
                              static_cast<const uint8_t *>(p.A) +
                              (m * p.lda + ((s + u) * 32 + lane) * W) * V::BYTES)),
                          av);
#pragma unroll
                for (int i = 0; i < W; ++i) sum[m] = fmaf(av[i], bv[i], sum[m]);
            }
        }
    };
    const int64_t whole = p.K / (32 * W), last = end < whole ? end : whole;
    int64_t s = first;
    if (inside) {
        for (; s + AHEAD <= last; s += AHEAD) whole_steps(s, std::integral_constant<int, AHEAD>());
        for (; s < last; ++s) whole_steps(s, std::integral_constant<int, 1>());
    }
    if (inside && end > whole) {  // K's end
        for (int i = 0; i < W; ++i) {
            const int64_t k = (whole * 32 + lane) * W + i;
            if (k >= p.K) break;
            const float bv = V::load(b, k);
#pragma unroll
            for (int m = 0; m < ROWS; ++m)
                if (m < p.M) sum[m] = fmaf(V::load(p.A, m * p.lda + k), bv, sum[m]);
        }
    }
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], d);
    }
    if (split > 1) {
        if (lane == 0) {
#pragma unroll
            for (int m = 0; m < ROWS; ++m) sums[warp][m] = sum[m];
        }
        __syncthreads();
        if (piece != 0) return;
        for (int i = 1; i < split; ++i) {
#pragma unroll
            for (int m = 0; m < ROWS; ++m) sum[m] += sums[warp + i][m];
        }
    }
    if (!inside) return;
    // lane m finishes row m
    float mine = 0.f;
#pragma unroll
    for (int m = 0; m < ROWS; ++m) mine = lane == m ? sum[m] : mine;
    float d = 0.f;
    if (lane < p.M)
        d = finish<TYPE>(p, mine, lane, n, !p.grad && p.bias != nullptr ? p.bias[n] : 0.f);
    if (p.grad && p.dbias != nullptr) {
#pragma unroll
        for (int s = ROWS / 2; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
        if (lane == 0) p.dbias[n] = d;
    }
}

// ------------------------------------------------------------- FP32: second pass
// D from the product in T (null: a product of nothing).  A CTA takes 64 times four
// columns of 32 rows, a thread four columns of eight of them; T may be D or the value
// kept.  With part the block's column sums go there.
constexpr int kPassRows = 32, kPassCols = 256;
template <bool VEC>
__global__ void __launch_bounds__(256) fused_finish_kernel(const __grid_constant__ FusedProblem p,
                                                           const float *T, int64_t ldt, float *part) {
    __shared__ float sums[4][kPassCols];
    const int64_t wide = (p.N + kPassCols - 1) / kPassCols;
    const int64_t blocks = (p.M + kPassRows - 1) / kPassRows * wide;
    const int quad = threadIdx.x % 64, group = threadIdx.x / 64;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t block = b / wide, c0 = (b - block * wide) * kPassCols + quad * 4;
        const int64_t r0 = block * kPassRows + group;  // and every fourth row on
        const int n = p.N - c0 < 4 ? static_cast<int>(p.N - c0 < 0 ? 0 : p.N - c0) : 4;
        auto load = [&](const void *m, int64_t ld, int64_t r, float (&v)[4]) {
            const float *from = static_cast<const float *>(m) + r * ld + c0;
            if (VEC && n == 4) {
                const float4 q = *reinterpret_cast<const float4 *>(from);
                v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = i < n ? from[i] : 0.f;
            }
        };
        auto store = [&](void *m, int64_t ld, int64_t r, const float (&v)[4]) {
            float *to = static_cast<float *>(m) + r * ld + c0;
            if (VEC && n == 4) {
                *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < n) to[i] = v[i];
            }
        };
        float bias[4] = {}, column[4] = {};
        if (!p.grad && p.bias != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) bias[i] = p.bias[c0 + i];
        }
        const void *const other = p.grad ? (p.act != kActNone ? p.pre : nullptr) : p.residual;
        const int64_t ld_other = p.grad ? p.ld_pre : p.ld_r;
#pragma unroll
        for (int h = 0; h < kPassRows / 4; h += 4) {  // four rows' loads at once
            float z[4][4] = {}, x[4][4] = {};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t r = r0 + (h + u) * 4;
                if (r >= p.M || n == 0) continue;
                if (T != nullptr) load(T, ldt, r, z[u]);
                if (other != nullptr) load(other, ld_other, r, x[u]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t r = r0 + (h + u) * 4;
                if (r >= p.M || n == 0) continue;
                float d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (p.grad) {
                        d[i] = p.act != kActNone ? z[u][i] * fused_slope(x[u][i], p.act) : z[u][i];
                        column[i] += d[i];
                    } else {
                        z[u][i] += bias[i];
                        d[i] = fused_activation(z[u][i], p.act) + x[u][i];
                    }
                }
                if (!p.grad && p.pre != nullptr) store(p.pre, p.ld_pre, r, z[u]);
                store(p.D, p.ldd, r, d);
            }
        }
        if (part != nullptr) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[group][quad * 4 + i] = column[i];
            __syncthreads();
            const int64_t c = (b - block * wide) * kPassCols + threadIdx.x;
            if (c < p.N)
                part[block * p.N + c] = (sums[0][threadIdx.x] + sums[1][threadIdx.x]) +
                                        (sums[2][threadIdx.x] + sums[3][threadIdx.x]);
        }
    }
}

// dbias from the row blocks' partial sums: 32 columns per CTA, its eight warps
// take every eighth block each.
__global__ void __launch_bounds__(256) column_sums_kernel(const float *part, int64_t blocks,
                                                          int64_t N, float *dbias) {
    __shared__ float sums[8][32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t n = blockIdx.x * 32ll + lane;
    pdl_wait();
    pdl_launch_dependents();
    float s = 0.f;
    if (n < N) {
        int64_t b = warp;
        for (; b + 24 < blocks; b += 32) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = part[(b + 8 * i) * N + n];
            s += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; b < blocks; b += 8) s += part[b * N + n];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && n < N) {
        for (int i = 1; i < 8; ++i) s += sums[i][lane];
        dbias[n] = s;
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename K, typename... A>
cudaError_t launch(K kernel, int64_t ctas, int threads, size_t smem, int cluster,
                   cudaStream_t stream, A... args) {
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[2];
    set_pdl_attribute(&attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The rows kernel's operands: K contiguous and on 16 bytes, few rows.  Past two rows
// of 16 bits its arithmetic is the time, and the tensor cores are faster where B is
// large (4096 x 4096: 1 row 7.8 us, 2 rows 8.1, 4 rows 14.9 and 14.4; 4096 x 14336,
// 4 rows 43 and 26; 4096 x 1024, 4 rows 7.3 and 11).
bool rows_fit(const FusedProblem &p, int64_t bytes) {
    const int most = bytes == 4 || p.N * p.K <= (int64_t(8) << 20) ? 4 : 2;
    if (p.M > most || p.K == 0 || !p.b_kmajor || !rows_on_16(p.B, p.ldb, bytes)) return false;
    if (p.M == 1)
        return reinterpret_cast<uintptr_t>(p.A) % 16 == 0 && (p.a_kmajor || p.lda == 1);
    return p.a_kmajor && rows_on_16(p.A, p.lda, bytes);
}

// Column sums of `blocks` blocks of rows: where the kernel puts them (*part), dbias
// itself if there is one block, and the sum of several.
cudaError_t sums_begin(const FusedProblem &p, int64_t blocks, cudaStream_t stream, float **part,
                       void **ws) {
    *part = p.dbias;
    *ws = nullptr;
    if (!p.grad || p.dbias == nullptr || blocks <= 1) return cudaSuccess;
    const cudaError_t e = workspace_alloc(static_cast<size_t>(blocks * p.N) * sizeof(float), stream, ws);
    if (e == cudaSuccess) *part = static_cast<float *>(*ws);
    return e;
}
cudaError_t sums_end(const FusedProblem &p, int64_t blocks, cudaStream_t stream, float *part, void *ws,
                     cudaError_t e) {
    if (ws == nullptr) return e;
    if (e == cudaSuccess) e = launch_column_sums(part, blocks, p.N, p.dbias, stream);
    const cudaError_t ef = workspace_free(ws, stream);
    return e == cudaSuccess ? ef : e;
}

template <int TYPE>
cudaError_t tiles_of(const FusedProblem &p, cudaStream_t stream) {
    const int64_t tiles_m = ceil_div(p.M, kTile), tiles_n = ceil_div(p.N, kTile);
    int ks = 1;
    while (ks < 8 && tiles_m * tiles_n * ks * 2 <= 2 * sm_count() && p.K >= 128 * ks) ks *= 2;
    float *part;
    void *ws;
    cudaError_t e = sums_begin(p, tiles_m * ks, stream, &part, &ws);
    if (e == cudaSuccess)
        e = launch(fused_tile_kernel<TYPE>, tiles_m * tiles_n * ks, THREADS, kTileFloats * sizeof(float), ks,
                   stream, p, tiles_n, ks, part);
    return sums_end(p, tiles_m * ks, stream, part, ws, e);
}

template <int TYPE>
cudaError_t rows_of(const FusedProblem &p, cudaStream_t stream) {
    FusedProblem q = p;
    q.a_kmajor = true;  // (one row whose K lies one apart may be column-major)
    // warps for about 24 per SM, each with a few steps of K
    int split = 1;
    while (split < kRowsWarps && p.N * split < 24 * sm_count() &&
           ceil_div(p.K, 32 * Value<TYPE>::PER_16) >= 4 * split)
        split *= 2;
    const int64_t ctas = ceil_div(p.N, kRowsWarps / split);
    const int n = 32 * kRowsWarps;
    if (p.M == 1) return launch(fused_rows_kernel<TYPE, 1>, ctas, n, 0, 1, stream, q, split);
    if (p.M == 2) return launch(fused_rows_kernel<TYPE, 2>, ctas, n, 0, 1, stream, q, split);
    return launch(fused_rows_kernel<TYPE, 4>, ctas, n, 0, 1, stream, q, split);
}

// FP32: the product, then what follows it.
cudaError_t f32_of(const FusedProblem &p, cudaStream_t stream, const char **name) {
    Problem g = {};
    g.M = p.M, g.N = p.N, g.K = p.K;
    g.alpha = p.alpha;
    g.A = p.A, g.lda = p.lda, g.a_kmajor = p.a_kmajor;
    g.B = p.B, g.ldb = p.ldb, g.b_kmajor = p.b_kmajor;
    g.D = static_cast<float *>(p.D), g.ldd = p.ldd;
    const bool alone = p.act == kActNone && p.bias == nullptr && (p.grad || p.pre == nullptr) &&
                       p.dbias == nullptr;
    if (alone && p.K > 0) {  // nothing follows that the product's own epilogue cannot do
        if (!p.grad && p.residual != nullptr) {
            g.beta = 1.f;
            g.C = static_cast<const float *>(p.residual), g.ldc = p.ld_r;
        }
        return launch_f32(g, stream, name);
    }
    // the product goes where nothing that is still needed lies
    void *product = nullptr;
    if (!p.grad && p.pre != nullptr) {
        g.D = static_cast<float *>(p.pre), g.ldd = p.ld_pre;
    } else if (p.D == p.residual || p.D == p.pre) {
        if (p.K > 0) {
            const cudaError_t e =
                workspace_alloc(static_cast<size_t>(p.M) * p.N * sizeof(float), stream, &product);
            if (e != cudaSuccess) return e;
        }
        g.D = static_cast<float *>(product), g.ldd = p.N;
    }
    cudaError_t e = p.K > 0 ? launch_f32(g, stream, name) : cudaSuccess;
    FusedProblem q = p;
    q.alpha = 1.f;  // (in the product)
    const int64_t blocks = ceil_div(p.M, kPassRows);
    float *part = nullptr;
    void *ws = nullptr;
    if (e == cudaSuccess) e = sums_begin(q, blocks, stream, &part, &ws);
    if (e == cudaSuccess) {
        const int64_t ctas = blocks * ceil_div(p.N, kPassCols), most = 32 * int64_t(sm_count());
        const bool vec = rows_on_16(p.D, p.ldd, 4) && rows_on_16(g.D, g.ldd, 4) &&
                         (p.pre == nullptr || rows_on_16(p.pre, p.ld_pre, 4)) &&
                         (p.residual == nullptr || rows_on_16(p.residual, p.ld_r, 4));
        e = launch(vec ? fused_finish_kernel<true> : fused_finish_kernel<false>, ctas < most ? ctas : most,
                   256, 0, 1, stream, q, static_cast<const float *>(p.K > 0 ? g.D : nullptr), g.ldd,
                   p.grad && p.dbias != nullptr ? part : nullptr);
    }
    e = sums_end(q, blocks, stream, part, ws, e);
    if (product != nullptr) {
        const cudaError_t ef = workspace_free(product, stream);
        if (e == cudaSuccess) e = ef;
    }
    *name = "fused_f32";
    return e;
}

}  // namespace

int sm_count() {
    static std::atomic<int> counts[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    int n = counts[dev].load();
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 1;
        counts[dev].store(n);
    }
    return n;
}

cudaError_t launch_column_sums(const float *part, int64_t blocks, int64_t N, float *dbias,
                               cudaStream_t stream) {
    return launch(column_sums_kernel, ceil_div(N, 32), 256, 0, 1, stream, part, blocks, N, dbias);
}

bool fused_rows_eligible(const FusedProblem &p, InType in) {
    return rows_fit(p, in == InType::F32 ? 4 : 2);
}

cudaError_t launch_fused_simt(const FusedProblem &p, InType in, cudaStream_t stream,
                              const char **name) {
    if (fused_rows_eligible(p, in)) {
        *name = "fused_rows";
        if (in == InType::F32) return rows_of<kOutF32>(p, stream);
        return in == InType::BF16 ? rows_of<kOutBf16>(p, stream) : rows_of<kOutF16>(p, stream);
    }
    *name = "fused_simt";
    if (in == InType::F32) {
        // few tiles: one kernel with K split over clusters (64 x 1024, K = 1000: 16 us,
        // product and pass 21; 512 x 512 x 512: 22 and 24; 2000 x 200, K = 1000: 69 and 48)
        const bool few = ceil_div(p.M, kTile) * ceil_div(p.N, kTile) * 2 <= sm_count();
        return few ? tiles_of<kOutF32>(p, stream) : f32_of(p, stream, name);
    }
    return in == InType::BF16 ? tiles_of<kOutBf16>(p, stream) : tiles_of<kOutF16>(p, stream);
}

}  // namespace gemm
