// fused_simt.cu -- the fused products on the CUDA cores: FP32 inputs (no TF32),
// and 16-bit inputs that TMA cannot describe.
//
// Tiles of 128 x 128 (8 x 8 sums per thread) or, where those would not fill the
// SMs, 64 x 64 (4 x 4); slices of 16 of K come through registers into two
// shared-memory buffers, sums are paired FMAs.  Few 64 x 64 tiles: K is split
// over a cluster, whose CTAs add each other's sums through distributed shared
// memory, each for its share of the tile's rows and in the order of the pieces.
// The tile then lies in shared memory, and a thread finishes one of its columns:
// bias, activation, residual, the value before the activation, column sums.
//
// Up to four rows of A and a K-contiguous B: warps stream B's columns once
// (fused_rows_kernel).
#include <atomic>

#include "fused.cuh"
#include "mixture.h"
#include "values.cuh"

namespace gemm {
namespace {

constexpr int BK = 16;
constexpr int THREADS = 256;

template <int TYPE>
__device__ __forceinline__ float finish(const FusedProblem &p, float sum, int64_t r, int64_t c,
                                        float bias) {
    constexpr bool FAST = TYPE != kOutF32;
    using V = Value<TYPE>;
    float d;
    if (p.grad) {
        d = p.alpha * sum;
        if (p.act != kActNone) d *= fused_slope<FAST>(V::load(p.pre, r * p.ld_pre + c), p.act);
    } else {
        const float z = fmaf(p.alpha, sum, bias);
        if (p.pre != nullptr) V::store(p.pre, r * p.ld_pre + c, z);
        d = fused_activation<FAST>(z, p.act);
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

template <int T>
struct Tile {
    static constexpr int T_ = T;            // rows and columns of a tile
    static constexpr int S = T / 16;        // and of a thread's block, 4 at a time
    static constexpr int PITCH = T + 4;     // of a slice's rows
    static constexpr int OUT = T + 1;       // of the finished tile's
    static constexpr int LOADS = T * BK / THREADS;
    static constexpr int SLICES = 4 * BK * PITCH;  // two buffers of A's and B's
    static constexpr int FLOATS = SLICES > T * OUT ? SLICES : T * OUT;
};

// ks pieces of K per tile (cluster), blockIdx.x = tile * ks + piece.
template <int TYPE, int T>
__global__ void __launch_bounds__(THREADS)
    fused_tile_kernel(const __grid_constant__ FusedProblem p, int64_t tiles_n, int ks, float *part) {
    using V = Value<TYPE>;
    using C = Tile<T>;
    extern __shared__ __align__(16) float smem[];
    float *const sa = smem, *const sb = smem + 2 * BK * C::PITCH;
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int64_t tile = blockIdx.x / ks;
    const int piece = static_cast<int>(blockIdx.x % ks);
    const int64_t m0 = tile / tiles_n * T, n0 = tile % tiles_n * T;
    const int64_t slices = (p.K + BK - 1) / BK;
    const int64_t first = slices * piece / ks, end = slices * (piece + 1) / ks;
    pdl_wait();
    pdl_launch_dependents();

    // the values of a slice that this thread brings: K fastest where K is contiguous
    float ra[C::LOADS], rb[C::LOADS];
    auto where = [&](bool kmajor, int i, int &k, int &x) {
        const int v = tid + i * THREADS;
        k = kmajor ? v % BK : v / T;
        x = kmajor ? v / BK : v % T;
    };
    auto fetch = [&](int64_t slice) {
        const int64_t k0 = slice * BK;
#pragma unroll
        for (int i = 0; i < C::LOADS; ++i) {
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
        for (int i = 0; i < C::LOADS; ++i) {
            int k, x;
            where(p.a_kmajor, i, k, x);
            sa[(buf * BK + k) * C::PITCH + x] = ra[i];
            where(p.b_kmajor, i, k, x);
            sb[(buf * BK + k) * C::PITCH + x] = rb[i];
        }
    };
    float2 acc[C::S][C::S / 2] = {};
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
            const float *a = sa + (buf * BK + k) * C::PITCH, *b = sb + (buf * BK + k) * C::PITCH;
            float av[C::S];
            float2 bv[C::S / 2];
#pragma unroll
            for (int h = 0; h < C::S / 4; ++h) {
                const float4 q = *reinterpret_cast<const float4 *>(a + h * (T / 2) + ty * 4);
                av[h * 4] = q.x, av[h * 4 + 1] = q.y, av[h * 4 + 2] = q.z, av[h * 4 + 3] = q.w;
                const float4 u = *reinterpret_cast<const float4 *>(b + h * (T / 2) + tx * 4);
                bv[h * 2] = make_float2(u.x, u.y), bv[h * 2 + 1] = make_float2(u.z, u.w);
            }
#pragma unroll
            for (int i = 0; i < C::S; ++i)
#pragma unroll
                for (int j = 0; j < C::S / 2; ++j) fma_pair(acc[i][j], make_float2(av[i], av[i]), bv[j]);
        }
        if (s + 1 < end) put(buf ^ 1);
        __syncthreads();
    }

    // the sums into shared memory, in place of the slices
#pragma unroll
    for (int i = 0; i < C::S; ++i)
#pragma unroll
        for (int j = 0; j < C::S / 2; ++j) {
            float *to = smem + (i / 4 * (T / 2) + ty * 4 + i % 4) * C::OUT + j / 2 * (T / 2) + tx * 4 +
                        j % 2 * 2;
            to[0] = acc[i][j].x;
            to[1] = acc[i][j].y;
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
                sum += ld_of_rank(base + static_cast<uint32_t>(r * C::OUT + col) * 4u, q);
        } else {
            sum = smem[r * C::OUT + col];
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
// column's K, 16 bytes a lane and four loads of B in flight; their sums are added
// in order.  B is read once, A comes from L1.
constexpr int kRowsWarps = 8;
template <int TYPE, int ROWS>
__global__ void __launch_bounds__(32 * kRowsWarps)
    fused_rows_kernel(const __grid_constant__ FusedProblem p, int split) {
    using V = Value<TYPE>;
    constexpr int W = V::PER_16, AHEAD = 4;
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
    for (int64_t s = first; inside && s < end; s += AHEAD) {
        uint4 q[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int64_t k = ((s + u) * 32 + lane) * W;
            q[u] = make_uint4(0, 0, 0, 0);
            if (s + u < end && k + W <= p.K) q[u] = __ldcs(reinterpret_cast<const uint4 *>(b + k * V::BYTES));
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int64_t k = ((s + u) * 32 + lane) * W;
            if (s + u >= end || k >= p.K) continue;
            float bv[W];
            if (k + W <= p.K) {
                V::unpack(q[u], bv);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) bv[i] = k + i < p.K ? V::load(b, k + i) : 0.f;
            }
#pragma unroll
            for (int m = 0; m < ROWS; ++m) {
                if (m >= p.M) continue;
                const uint8_t *a = static_cast<const uint8_t *>(p.A) + (m * p.lda + k) * V::BYTES;
                float av[W];
                if (k + W <= p.K) {
                    V::unpack(__ldg(reinterpret_cast<const uint4 *>(a)), av);
                } else {
#pragma unroll
                    for (int i = 0; i < W; ++i) av[i] = k + i < p.K ? V::load(a, i) : 0.f;
                }
#pragma unroll
                for (int i = 0; i < W; ++i) sum[m] = fmaf(av[i], bv[i], sum[m]);
            }
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

template <int TYPE, int T>
cudaError_t tiles_as(const FusedProblem &p, int ks, cudaStream_t stream) {
    const int64_t tiles_m = ceil_div(p.M, T), tiles_n = ceil_div(p.N, T);
    constexpr size_t smem = Tile<T>::FLOATS * sizeof(float);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            fused_tile_kernel<TYPE, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    const int64_t blocks = tiles_m * ks;
    float *part = p.dbias;
    void *ws = nullptr;
    cudaError_t e = cudaSuccess;
    if (p.grad && p.dbias != nullptr && blocks > 1) {
        e = workspace_alloc(static_cast<size_t>(blocks * p.N) * sizeof(float), stream, &ws);
        if (e != cudaSuccess) return e;
        part = static_cast<float *>(ws);
    }
    e = launch(fused_tile_kernel<TYPE, T>, tiles_m * tiles_n * ks, THREADS, smem, ks, stream, p,
               tiles_n, ks, part);
    if (ws != nullptr) {
        if (e == cudaSuccess) e = launch_column_sums(part, blocks, p.N, p.dbias, stream);
        const cudaError_t ef = workspace_free(ws, stream);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

// The rows kernel's operands: K contiguous and on 16 bytes, M at most 4.
bool rows_fit(const FusedProblem &p, int64_t bytes) {
    if (p.M > 4 || p.K == 0 || !p.b_kmajor || !rows_on_16(p.B, p.ldb, bytes)) return false;
    if (p.M == 1)
        return reinterpret_cast<uintptr_t>(p.A) % 16 == 0 && (p.a_kmajor || p.lda == 1);
    return p.a_kmajor && rows_on_16(p.A, p.lda, bytes);
}

template <int TYPE>
cudaError_t fused_of(const FusedProblem &p, cudaStream_t stream, const char **name) {
    using V = Value<TYPE>;
    const int64_t sms = sm_count();
    if (rows_fit(p, V::BYTES)) {
        FusedProblem q = p;
        q.a_kmajor = true;  // (one row whose K lies one apart may be column-major)
        *name = "fused_rows";
        // warps for about 24 per SM, each with a few steps of K
        int split = 1;
        while (split < kRowsWarps && p.N * split < 24 * sms && ceil_div(p.K, 32 * V::PER_16) >= 4 * split)
            split *= 2;
        const int64_t ctas = ceil_div(p.N, kRowsWarps / split);
        if (p.M == 1)
            return launch(fused_rows_kernel<TYPE, 1>, ctas, 32 * kRowsWarps, 0, 1, stream, q, split);
        if (p.M == 2)
            return launch(fused_rows_kernel<TYPE, 2>, ctas, 32 * kRowsWarps, 0, 1, stream, q, split);
        return launch(fused_rows_kernel<TYPE, 4>, ctas, 32 * kRowsWarps, 0, 1, stream, q, split);
    }
    *name = "fused_simt";
    if (ceil_div(p.M, 128) * ceil_div(p.N, 128) >= sms) return tiles_as<TYPE, 128>(p, 1, stream);
    const int64_t tiles = ceil_div(p.M, 64) * ceil_div(p.N, 64);
    int ks = 1;
    while (ks < 8 && tiles * ks * 2 <= 2 * sms && p.K >= 128 * ks) ks *= 2;
    return tiles_as<TYPE, 64>(p, ks, stream);
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
    if (in == InType::F32) return fused_of<kOutF32>(p, stream, name);
    return in == InType::BF16 ? fused_of<kOutBf16>(p, stream, name)
                              : fused_of<kOutF16>(p, stream, name);
}

}  // namespace gemm
