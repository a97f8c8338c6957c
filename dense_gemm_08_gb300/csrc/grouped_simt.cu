// grouped_simt.cu -- the grouped operators on the CUDA cores: FP32 inputs, and
// 16-bit inputs whose rows TMA cannot describe.
//
// One kernel body for the three products; a CTA of 256 threads makes one 64 x
// 64 tile of D from 16-deep slices staged in shared memory as FP32, each
// thread a 4 x 4 block with FP32 FMAs (products of 16-bit values are exact):
//   rows:   D(r, j) = act(alpha * sum_k A(idx(r), k) B_g(k, j) + bias_g(j)),
//           r in group g; a tile never holds rows of two groups;
//   wgrad:  D_g(i, j) = alpha * sum_{r in g} A(idx(r), i) B(r, j) + beta C_g(i, j);
//           a group without rows gives beta C_g (zeros when beta = 0);
//   lora:   one group of M rows; the epilogue adds s_a * sum_c U(r, c) LB_a(c, j),
//           with U = X LA (FP32, from lora_shrink_simt) and each row's own
//           adapter, so no row ever reads another row's adapter.
#include "grouped.cuh"

namespace gemm {
namespace {

constexpr int TM = 64, TN = 64, TK = 16, THREADS = 256;

template <typename T>
__device__ __forceinline__ float widened(const T *p);
template <>
__device__ __forceinline__ float widened<float>(const float *p) {
    return __ldg(p);
}
template <>
__device__ __forceinline__ float widened<uint16_t>(const uint16_t *p) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}
template <>
__device__ __forceinline__ float widened<__half>(const __half *p) {
    return __half2float(*p);
}

enum : int { kRows = 0, kWgrad = 1, kLora = 2 };

struct SimtGroupedArgs {
    GroupedProblem g;  // kRows; kLora (groups = 1, A = X, B = W)
    WgradProblem w;    // kWgrad
    LoraProblem l;     // kLora
    const float *U;    // kLora: M x rank
    uint32_t tiles_n, tiles_m;
};

template <typename T, int MODE>
__global__ void __launch_bounds__(THREADS) grouped_simt_kernel(const SimtGroupedArgs a) {
    __shared__ float As[TK][TM + 4], Bs[TK][TN + 4];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    int g = 0;
    int32_t first = 0, last = 0;  // the group's rows
    uint32_t in_group = 0;
    if constexpr (MODE == kWgrad) {
        const uint32_t per = a.tiles_m * a.tiles_n;
        g = static_cast<int>(blockIdx.x / per);
        in_group = blockIdx.x % per;
        const int32_t lo = __ldg(a.w.offsets + g), hi = __ldg(a.w.offsets + g + 1);
        const int32_t rows = static_cast<int32_t>(a.w.rows);
        first = lo < 0 ? 0 : (lo > rows ? rows : lo);
        last = hi < first ? first : (hi > rows ? rows : hi);
    } else if constexpr (MODE == kRows) {
        GroupWalk walk(a.g.offsets, a.g.groups, a.g.rows, TM, a.tiles_n);
        if (!walk.locate(blockIdx.x, g, first, last, in_group)) return;
    } else {
        last = static_cast<int32_t>(a.l.M);
        in_group = blockIdx.x;
    }
    const int64_t tm = in_group / a.tiles_n, tn = in_group % a.tiles_n;
    const int64_t m0 = (MODE == kWgrad ? 0 : first) + tm * TM;  // first row of D in the tile
    const int64_t m_end = MODE == kWgrad ? a.w.M : last;
    const int64_t n0 = tn * TN, n_end = MODE == kWgrad ? a.w.N : a.g.N;
    const int64_t k_begin = MODE == kWgrad ? first : 0;
    const int64_t k_end = MODE == kWgrad ? last : a.g.K;

    const T *A = static_cast<const T *>(MODE == kWgrad ? a.w.A : a.g.A);
    const T *B = static_cast<const T *>(MODE == kWgrad ? a.w.B : a.g.B) +
                 (MODE == kRows ? g * a.g.stride_b : 0);
    const int64_t lda = MODE == kWgrad ? a.w.lda : a.g.lda;
    const int64_t ldb = MODE == kWgrad ? a.w.ldb : a.g.ldb;
    const int32_t *row_index = MODE == kWgrad ? a.w.row_index : a.g.row_index;
    const int64_t rows_a = MODE == kWgrad ? a.w.rows_a : a.g.rows_a;

    // rows / lora: this thread stages A(row0 + tid / 4, 4 (tid % 4) ..)
    int64_t my_row = -1;
    if constexpr (MODE != kWgrad) {
        const int64_t r = m0 + tid / 4;
        if (r < m_end) {
            my_row = row_index != nullptr ? row_index[r] : r;
            if (my_row < 0 || my_row >= rows_a) my_row = -1;
        }
    }
    float acc[4][4] = {};
    const int tx = tid % 16, ty = tid / 16;
    for (int64_t k0 = k_begin; k0 < k_end; k0 += TK) {
        if constexpr (MODE == kWgrad) {
            const int64_t r = k0 + tid / 16;
            int64_t ar = -1;
            if (r < k_end) {
                ar = row_index != nullptr ? row_index[r] : r;
                if (ar < 0 || ar >= rows_a) ar = -1;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + (tid % 16) * 4 + i, n = n0 + (tid % 16) * 4 + i;
                As[tid / 16][(tid % 16) * 4 + i] =
                    ar >= 0 && m < m_end ? widened<T>(A + ar * lda + m) : 0.f;
                Bs[tid / 16][(tid % 16) * 4 + i] =
                    r < k_end && n < n_end ? widened<T>(B + r * ldb + n) : 0.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t k = k0 + (tid % 4) * 4 + i;
                As[(tid % 4) * 4 + i][tid / 4] =
                    my_row >= 0 && k < k_end ? widened<T>(A + my_row * lda + k) : 0.f;
            }
            if (a.g.b_kmajor) {
                const int64_t n = n0 + tid / 4;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t k = k0 + (tid % 4) * 4 + i;
                    Bs[(tid % 4) * 4 + i][tid / 4] =
                        n < n_end && k < k_end ? widened<T>(B + n * ldb + k) : 0.f;
                }
            } else {
                const int64_t k = k0 + tid / 16;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t n = n0 + (tid % 16) * 4 + i;
                    Bs[tid / 16][(tid % 16) * 4 + i] =
                        n < n_end && k < k_end ? widened<T>(B + k * ldb + n) : 0.f;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < TK; ++k) {
            float av[4], bv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) av[i] = As[k][ty * 4 + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) bv[j] = Bs[k][tx * 4 + j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = m0 + ty * 4 + i;
        if (r >= m_end) continue;
        int64_t adapter = -1;
        if constexpr (MODE == kLora) {
            adapter = a.l.adapter[r];
            if (adapter >= a.l.adapters) adapter = -1;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx * 4 + j;
            if (n >= n_end) continue;
            float v = acc[i][j];
            if constexpr (MODE == kWgrad) {
                v *= a.w.alpha;
                if (a.w.beta != 0.f)
                    v = fmaf(a.w.beta, a.w.C[g * a.w.stride_c + r * a.w.ldc + n], v);
                store_out(a.w.D, g * a.w.stride_d + r * a.w.ldd + n, v, a.w.out);
            } else {
                if constexpr (MODE == kLora) {
                    if (adapter >= 0) {
                        const T *lb = static_cast<const T *>(a.l.LB) + adapter * a.l.stride_b;
                        const float *u = a.U + r * a.l.rank;
                        float s = 0.f;
                        for (int64_t c = 0; c < a.l.rank; ++c)
                            s = fmaf(u[c], widened<T>(lb + (a.l.b_kmajor ? c + n * a.l.ld_b
                                                                         : c * a.l.ld_b + n)), s);
                        v += s;
                    }
                }
                v *= a.g.alpha;
                if (a.g.bias != nullptr) v += a.g.bias[g * a.g.N + n];
                store_out(a.g.D, r * a.g.ldd + n, apply_activation(v, a.g.act), a.g.out);
            }
        }
    }
}

// U(i, c) = s_a * sum_k X(i, k) LA_a(k, c), a = adapter[i]: one CTA per row,
// one warp per column c, the lanes over k and a fixed shuffle tree.
template <typename T>
__global__ void __launch_bounds__(THREADS) lora_shrink_simt_kernel(const LoraProblem p, float *U) {
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int64_t i = blockIdx.x; i < p.M; i += gridDim.x) {
        const int64_t ad = p.adapter[i];
        if (ad < 0 || ad >= p.adapters) continue;
        const T *x = static_cast<const T *>(p.X) + i * p.ldx;
        const T *la = static_cast<const T *>(p.LA) + ad * p.stride_a;
        const float scale = p.scale != nullptr ? p.scale[ad] : 1.f;
        for (int64_t c = warp; c < p.rank; c += THREADS / 32) {
            float s = 0.f;
            for (int64_t k = lane; k < p.K; k += 32)
                s = fmaf(widened<T>(x + k),
                         widened<T>(la + (p.a_kmajor ? k + c * p.ld_a : k * p.ld_a + c)), s);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (lane == 0) U[i * p.rank + c] = s * scale;
        }
    }
}

template <int MODE, typename T>
cudaError_t launch_as(const SimtGroupedArgs &a, int64_t grid, cudaStream_t stream) {
    if (grid <= 0) return cudaSuccess;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr;
    set_pdl_attribute(&attr);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, grouped_simt_kernel<T, MODE>, a);
}

template <int MODE>
cudaError_t launch_typed(const SimtGroupedArgs &a, InType in, int64_t grid, cudaStream_t stream) {
    switch (in) {
        case InType::F32: return launch_as<MODE, float>(a, grid, stream);
        case InType::BF16: return launch_as<MODE, uint16_t>(a, grid, stream);
        case InType::F16: return launch_as<MODE, __half>(a, grid, stream);
    }
    return cudaErrorInvalidValue;
}

uint32_t tiles(int64_t n, int t) { return static_cast<uint32_t>((n + t - 1) / t); }

const char *kNames[3][3] = {
    {"grouped_simt<f32>", "grouped_simt<bf16>", "grouped_simt<f16>"},
    {"wgrad_simt<f32>", "wgrad_simt<bf16>", "wgrad_simt<f16>"},
    {"lora_simt<f32>", "lora_simt<bf16>", "lora_simt<f16>"}};

}  // namespace

cudaError_t launch_grouped_simt(const GroupedProblem &p, InType in, cudaStream_t stream,
                                const char **name) {
    *name = kNames[kRows][static_cast<int>(in)];
    SimtGroupedArgs a = {};
    a.g = p;
    a.tiles_n = tiles(p.N, TN);
    // at most one partly filled row tile per group
    const int64_t row_tiles = p.rows / TM + (p.groups < p.rows ? p.groups : p.rows);
    return launch_typed<kRows>(a, in, row_tiles * a.tiles_n, stream);
}

cudaError_t launch_wgrad_simt(const WgradProblem &p, InType in, cudaStream_t stream,
                              const char **name) {
    *name = kNames[kWgrad][static_cast<int>(in)];
    SimtGroupedArgs a = {};
    a.w = p;
    a.tiles_m = tiles(p.M, TM);
    a.tiles_n = tiles(p.N, TN);
    return launch_typed<kWgrad>(a, in, p.groups * a.tiles_m * a.tiles_n, stream);
}

cudaError_t launch_lora_simt(const LoraProblem &p, InType in, cudaStream_t stream,
                             const char **name) {
    *name = kNames[kLora][static_cast<int>(in)];
    if (in == InType::F32) return cudaErrorInvalidValue;
    SimtGroupedArgs a = {};
    a.l = p;
    GroupedProblem &g = a.g;
    g.groups = 1;
    g.rows = g.rows_a = p.M;
    g.N = p.N;
    g.K = p.K;
    g.alpha = 1.f;
    g.A = p.X;
    g.lda = p.ldx;
    g.B = p.W;
    g.ldb = p.ldw;
    g.b_kmajor = p.w_kmajor;
    g.D = p.D;
    g.ldd = p.ldd;
    g.bias = p.bias;
    g.act = p.act;
    g.out = p.out;
    a.tiles_n = tiles(p.N, TN);
    void *u = nullptr;
    const bool any = p.adapters > 0 && p.rank > 0 && p.K > 0;
    cudaError_t e;
    if (any) {
        e = workspace_alloc(static_cast<size_t>(p.M) * p.rank * sizeof(float), stream, &u);
        if (e != cudaSuccess) return e;
        a.U = static_cast<float *>(u);
        const unsigned grid = static_cast<unsigned>(p.M < 65536 ? p.M : 65536);
        if (in == InType::BF16)
            lora_shrink_simt_kernel<uint16_t><<<grid, THREADS, 0, stream>>>(p, static_cast<float *>(u));
        else
            lora_shrink_simt_kernel<__half><<<grid, THREADS, 0, stream>>>(p, static_cast<float *>(u));
        e = cudaGetLastError();
    } else {
        a.l.adapters = 0;
        e = cudaSuccess;
    }
    if (e == cudaSuccess)
        e = launch_typed<kLora>(a, in, static_cast<int64_t>(tiles(p.M, TM)) * a.tiles_n, stream);
    if (u != nullptr) {
        const cudaError_t ef = workspace_free(u, stream);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

}  // namespace gemm
