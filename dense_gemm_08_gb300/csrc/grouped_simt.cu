// grouped_simt.cu -- the grouped operators on the CUDA cores: FP32 inputs, and
// 16-bit inputs whose rows TMA cannot describe.
//
// One kernel body for the three products; a CTA makes one 64 x 128 tile of D,
// each thread an 8 x 8 or 8 x 4 block:
//   rows:   D(r, j) = act(alpha * sum_k A(idx(r), k) B_g(k, j) + bias_g(j)),
//           r in group g; a tile never holds rows of two groups;
//   wgrad:  D_g(i, j) = alpha * sum_{r in g} A(idx(r), i) B(r, j) + beta C_g(i, j);
//           a group without rows gives beta C_g (zeros when beta = 0);
//   lora:   one group of M rows; the epilogue adds s_a * sum_c U(r, c) LB_a(c, j),
//           with U = X LA (FP32, from lora_shrink_simt) and each row's own
//           adapter, so no row ever reads another row's adapter.
// Slices 32 deep in K go through shared memory as FP32, the next one loaded
// into registers while the current one is multiplied.  The arithmetic is FP32
// FMAs two rows at a time (fma.rn.f32x2, each half rounded as fmaf; products
// of 16-bit values are exact), so the FMA pipe is the bound (80.5 TFLOP/s);
// measured 46, the rest shared-memory reads and the waits at a slice's end.
// 64 rows per tile rather than 128: groups are small where FP32 is used, and a
// tile's rows past the group's end are lost work.
//
// 8 x 8 per thread (128 threads, three CTAs per SM) for the row products: four
// 16-byte reads of shared memory per 32 FMAs (8 groups, 4096 rows, 2048 x 2048:
// 741 us, 8 x 4 779).  8 x 4 (256 threads, two CTAs) for the weight gradients,
// whose sums are often short: twice the warps hide more of a tile's start and
// end (4 groups of 300 rows, 600 x 600: 39 us, 8 x 8 41; 16 groups, 2000 rows,
// 1000 x 1024: 109 and 119).
#include "grouped.cuh"

namespace gemm {
namespace {

constexpr int TM = 64, TN = 128, TK = 32;
constexpr int kSmemBytes = 2 * TK * (TM + TN) * 4;

enum : int { kRows = 0, kWgrad = 1, kLora = 2 };

template <int MODE>
struct Shape {
    static constexpr int RN = MODE == kWgrad ? 4 : 8;  // columns per thread, in quads TN / 2 apart
    static constexpr int THREADS = TM / 8 * (TN / RN);
    static constexpr int RESIDENT = MODE == kWgrad ? 2 : 3;
    static constexpr int QA = TM * TK / 4 / THREADS, QB = TN * TK / 4 / THREADS;  // quads per slice
};

// Where four values from column q (a multiple of 4) of step k of a slice are:
// the quads of a row change places with k / 4, so that a warp that stores
// quads along K as columns meets every bank once.
__device__ __forceinline__ int spot(int k, int q) { return q ^ (k / 4 % 8 * 4); }

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

__device__ __forceinline__ float to_float(uint16_t b) {
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
}
__device__ __forceinline__ float to_float(__half h) { return __half2float(h); }

// Four consecutive values, of which the first `n` (<= 4) are read; zeros for
// the rest.  `vec`: the address is aligned to all four.
template <typename T>
__device__ __forceinline__ float4 load4(const T *p, int64_t n, bool vec) {
    if (n >= 4 && vec) {
        if constexpr (sizeof(T) == 4) {
            return __ldg(reinterpret_cast<const float4 *>(p));
        } else {
            alignas(8) T v[4];
            *reinterpret_cast<uint2 *>(v) = __ldg(reinterpret_cast<const uint2 *>(p));
            return make_float4(to_float(v[0]), to_float(v[1]), to_float(v[2]), to_float(v[3]));
        }
    }
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n > 0) f.x = widened<T>(p);
    if (n > 1) f.y = widened<T>(p + 1);
    if (n > 2) f.z = widened<T>(p + 2);
    if (n > 3) f.w = widened<T>(p + 3);
    return f;
}

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ void fma2(uint64_t &c, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

struct SimtGroupedArgs {
    GroupedProblem g;  // kRows; kLora (groups = 1, A = X, B = W)
    WgradProblem w;    // kWgrad
    LoraProblem l;     // kLora
    const float *U;    // kLora: M x rank
    uint32_t tiles_n, tiles_m;
    bool vec_a, vec_b;  // rows of A and B start on four values
    bool vec_d;         // rows of an FP32 D (and C) start on 16 bytes
    int ks;             // CTAs of a cluster, which share a tile's K
};

// 16 bytes of the same shared-memory object in CTA `rank` of the cluster.
__device__ __forceinline__ float4 load_from_rank(const float *p, uint32_t rank) {
    uint32_t at;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

__device__ __forceinline__ void sync_cluster() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Four columns of row r of D from n4 on: the sums o, then the epilogue.
template <typename T, int MODE>
__device__ __forceinline__ void finish_quad(const SimtGroupedArgs &a, int g, int64_t r, int64_t n4,
                                            int64_t n_end, float4 sum) {
    float o[4] = {sum.x, sum.y, sum.z, sum.w};
    const bool whole = a.vec_d && n4 + 4 <= n_end;
    if constexpr (MODE == kWgrad) {
        const int64_t at = g * a.w.stride_d + r * a.w.ldd + n4;
        const float *c = a.w.beta != 0.f ? a.w.C + g * a.w.stride_c + r * a.w.ldc + n4 : nullptr;
        if (whole) {
            float4 v = make_float4(o[0] * a.w.alpha, o[1] * a.w.alpha, o[2] * a.w.alpha,
                                   o[3] * a.w.alpha);
            if (c != nullptr) {
                const float4 cv = *reinterpret_cast<const float4 *>(c);
                v.x = fmaf(a.w.beta, cv.x, v.x), v.y = fmaf(a.w.beta, cv.y, v.y);
                v.z = fmaf(a.w.beta, cv.z, v.z), v.w = fmaf(a.w.beta, cv.w, v.w);
            }
            *reinterpret_cast<float4 *>(static_cast<float *>(a.w.D) + at) = v;
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n4 + j >= n_end) continue;
            float v = o[j] * a.w.alpha;
            if (c != nullptr) v = fmaf(a.w.beta, c[j], v);
            store_out(a.w.D, at + j, v, a.w.out);
        }
    } else {
        int64_t adapter = -1;
        if constexpr (MODE == kLora) {
            if (a.l.adapters > 0) adapter = a.l.adapter[r];
            if (adapter >= a.l.adapters) adapter = -1;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n4 + j;
            if (n >= n_end) continue;
            float v = o[j];
            if constexpr (MODE == kLora) {
                if (adapter >= 0) {
                    const T *lb = static_cast<const T *>(a.l.LB) + adapter * a.l.stride_b;
                    const float *u = a.U + r * a.l.rank;
                    float s = 0.f;
                    for (int64_t c = 0; c < a.l.rank; ++c)
                        s = fmaf(u[c],
                                 widened<T>(lb + (a.l.b_kmajor ? c + n * a.l.ld_b : c * a.l.ld_b + n)),
                                 s);
                    v += s;
                }
            }
            v *= a.g.alpha;
            if (a.g.bias != nullptr) v += a.g.bias[g * a.g.N + n];
            o[j] = grouped_activation(v, a.g.act);
        }
        const int64_t at = r * a.g.ldd + n4;
        if (whole) {
            *reinterpret_cast<float4 *>(static_cast<float *>(a.g.D) + at) =
                make_float4(o[0], o[1], o[2], o[3]);
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n4 + j < n_end) store_out(a.g.D, at + j, o[j], a.g.out);
    }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(Shape<MODE>::THREADS, Shape<MODE>::RESIDENT)
    grouped_simt_kernel(const SimtGroupedArgs a) {
    constexpr int THREADS = Shape<MODE>::THREADS, RN = Shape<MODE>::RN, QA = Shape<MODE>::QA,
                  QB = Shape<MODE>::QB;
    extern __shared__ float4 smem4[];
    float(*As)[TK][TM] = reinterpret_cast<float(*)[TK][TM]>(smem4);
    float(*Bs)[TK][TN] = reinterpret_cast<float(*)[TK][TN]>(reinterpret_cast<float *>(smem4) + 2 * TK * TM);
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    // the CTAs of a cluster share a tile
    const uint32_t tile = blockIdx.x / static_cast<uint32_t>(a.ks);
    const uint32_t rank = blockIdx.x % static_cast<uint32_t>(a.ks);
    int g = 0;
    int32_t first = 0, last = 0;  // the group's rows
    uint32_t in_group = 0;
    if constexpr (MODE == kWgrad) {
        const uint32_t per = a.tiles_m * a.tiles_n;
        g = static_cast<int>(tile / per);
        in_group = tile % per;
        const int32_t lo = __ldg(a.w.offsets + g), hi = __ldg(a.w.offsets + g + 1);
        const int32_t rows = static_cast<int32_t>(a.w.rows);
        first = lo < 0 ? 0 : (lo > rows ? rows : lo);
        last = hi < first ? first : (hi > rows ? rows : hi);
    } else if constexpr (MODE == kRows) {
        GroupWalk walk(a.g.offsets, a.g.groups, a.g.rows, TM, a.tiles_n);
        if (!walk.locate(tile, g, first, last, in_group)) return;
    } else {
        last = static_cast<int32_t>(a.l.M);
        in_group = tile;
    }
    const int64_t tm = in_group / a.tiles_n, tn = in_group % a.tiles_n;
    const int64_t m0 = (MODE == kWgrad ? 0 : first) + tm * TM;  // first row of D in the tile
    const int64_t m_end = MODE == kWgrad ? a.w.M : last;
    const int64_t n0 = tn * TN, n_end = MODE == kWgrad ? a.w.N : a.g.N;
    const int64_t k_first = MODE == kWgrad ? first : 0;
    const int64_t k_last = MODE == kWgrad ? last : a.g.K;
    const int64_t slices = (k_last - k_first + TK - 1) / TK;
    const int64_t k_begin = k_first + slices * rank / a.ks * TK;
    const int64_t k_stop = k_first + slices * (rank + 1) / a.ks * TK;
    const int64_t k_end = k_stop < k_last ? k_stop : k_last;

    const T *A = static_cast<const T *>(MODE == kWgrad ? a.w.A : a.g.A);
    const T *B = static_cast<const T *>(MODE == kWgrad ? a.w.B : a.g.B) +
                 (MODE == kRows ? g * a.g.stride_b : 0);
    const int64_t lda = MODE == kWgrad ? a.w.lda : a.g.lda;
    const int64_t ldb = MODE == kWgrad ? a.w.ldb : a.g.ldb;
    const int32_t *row_index = MODE == kWgrad ? a.w.row_index : a.g.row_index;
    const int64_t rows_a = MODE == kWgrad ? a.w.rows_a : a.g.rows_a;
    const bool b_kmajor = MODE != kWgrad && a.g.b_kmajor;

    // Quads of four values:
    //   K-contiguous: quad i is row i / 8, values 4 (i % 8) of the slice's 32
    //   else:         quad i is step i / (width / 4) of K, columns 4 (i % ..)
    int64_t a_row[QA];
    if constexpr (MODE != kWgrad) {
#pragma unroll
        for (int q = 0; q < QA; ++q) {
            const int64_t r = m0 + (tid + q * THREADS) / 8;
            a_row[q] = -1;
            if (r < m_end) {
                a_row[q] = row_index != nullptr ? row_index[r] : r;
                if (a_row[q] < 0 || a_row[q] >= rows_a) a_row[q] = -1;
            }
        }
    }
    float4 a_next[QA], b_next[QB];
    auto fetch = [&](int64_t k0) {
        if constexpr (MODE == kWgrad) {
#pragma unroll
            for (int q = 0; q < QA; ++q) {
                const int i = tid + q * THREADS;
                const int64_t r = k0 + i / 16, m = m0 + (i % 16) * 4;
                int64_t from = -1;
                if (r < k_end) {
                    from = row_index != nullptr ? row_index[r] : r;
                    if (from < 0 || from >= rows_a) from = -1;
                }
                a_next[q] = load4(A + (from >= 0 ? from * lda + m : 0), from >= 0 ? m_end - m : 0, a.vec_a);
            }
        } else {
#pragma unroll
            for (int q = 0; q < QA; ++q) {
                const int64_t k = k0 + (tid % 8) * 4;
                a_next[q] = load4(A + (a_row[q] >= 0 ? a_row[q] * lda + k : 0),
                                  a_row[q] >= 0 ? k_end - k : 0, a.vec_a);
            }
        }
        if (b_kmajor) {
#pragma unroll
            for (int q = 0; q < QB; ++q) {
                const int64_t n = n0 + (tid + q * THREADS) / 8, k = k0 + (tid % 8) * 4;
                b_next[q] = load4(B + (n < n_end ? n * ldb + k : 0), n < n_end ? k_end - k : 0, a.vec_b);
            }
        } else {
#pragma unroll
            for (int q = 0; q < QB; ++q) {
                const int i = tid + q * THREADS;
                const int64_t k = k0 + i / 32, n = n0 + (i % 32) * 4;
                b_next[q] = load4(B + (k < k_end ? k * ldb + n : 0), k < k_end ? n_end - n : 0, a.vec_b);
            }
        }
    };
    auto put = [&](int s) {
#pragma unroll
        for (int q = 0; q < QA; ++q) {
            const int i = tid + q * THREADS;
            if constexpr (MODE == kWgrad) {
                *reinterpret_cast<float4 *>(&As[s][i / 16][spot(i / 16, (i % 16) * 4)]) = a_next[q];
            } else {
                const int k = (i % 8) * 4, r = spot(k, i / 8);
                As[s][k + 0][r] = a_next[q].x;
                As[s][k + 1][r] = a_next[q].y;
                As[s][k + 2][r] = a_next[q].z;
                As[s][k + 3][r] = a_next[q].w;
            }
        }
#pragma unroll
        for (int q = 0; q < QB; ++q) {
            const int i = tid + q * THREADS;
            if (b_kmajor) {
                const int k = (i % 8) * 4, n = spot(k, i / 8);
                Bs[s][k + 0][n] = b_next[q].x;
                Bs[s][k + 1][n] = b_next[q].y;
                Bs[s][k + 2][n] = b_next[q].z;
                Bs[s][k + 3][n] = b_next[q].w;
            } else {
                *reinterpret_cast<float4 *>(&Bs[s][i / 32][spot(i / 32, (i % 32) * 4)]) = b_next[q];
            }
        }
    };

    // rows ty * 8 .. + 7 in pairs; columns tx * 4 .. + 3, and as many TN / 2 on
    // (RN = 8); a warp's block is 16 rows of 64 columns, or twice 64
    const int tx = (RN == 8 ? 0 : tid / 32 % 2 * 16) + tid % 16;
    const int ty = tid / (RN == 8 ? 32 : 64) * 2 + tid / 16 % 2;
    uint64_t acc[4][RN];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < RN; ++j) acc[i][j] = 0;
    if (k_begin < k_end) {
        fetch(k_begin);
        put(0);
    }
    __syncthreads();
    int s = 0;
    for (int64_t k0 = k_begin; k0 < k_end; k0 += TK) {
        const bool more = k0 + TK < k_end;
        if (more) fetch(k0 + TK);
#pragma unroll
        for (int k = 0; k < TK; ++k) {
            uint64_t av[4];
            const ulonglong2 a0 = *reinterpret_cast<const ulonglong2 *>(&As[s][k][spot(k, ty * 8)]);
            const ulonglong2 a1 = *reinterpret_cast<const ulonglong2 *>(&As[s][k][spot(k, ty * 8 + 4)]);
            av[0] = a0.x, av[1] = a0.y, av[2] = a1.x, av[3] = a1.y;
#pragma unroll
            for (int h = 0; h < RN / 4; ++h) {
                const float4 b =
                    *reinterpret_cast<const float4 *>(&Bs[s][k][spot(k, h * (TN / 2) + tx * 4)]);
                const uint64_t bv[4] = {pair(b.x, b.x), pair(b.y, b.y), pair(b.z, b.z), pair(b.w, b.w)};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) fma2(acc[i][h * 4 + j], av[i], bv[j]);
            }
        }
        if (more) put(s ^ 1);  // the other buffer was last read before the previous barrier
        __syncthreads();
        s ^= 1;
    }
    auto sums = [&](int i, int h) {  // row ty * 8 + i of the tile, columns from h TN / 2 + tx * 4 on
        float o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            unpair(acc[i / 2][h * 4 + j], lo, hi);
            o[j] = i % 2 ? hi : lo;
        }
        return make_float4(o[0], o[1], o[2], o[3]);
    };
    if (a.ks == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < RN / 4; ++h)
                if (m0 + ty * 8 + i < m_end)
                    finish_quad<T, MODE>(a, g, m0 + ty * 8 + i, n0 + h * (TN / 2) + tx * 4, n_end,
                                         sums(i, h));
        return;
    }
    // the parts meet in the cluster's shared memory, each CTA adding a share of
    // the rows in rank order (the slices are no longer needed)
    float(*part)[TN] = reinterpret_cast<float(*)[TN]>(smem4);
    static_assert(TM * TN * 4 <= kSmemBytes, "a tile of sums replaces the slices");
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < RN / 4; ++h)
            *reinterpret_cast<float4 *>(&part[ty * 8 + i][h * (TN / 2) + tx * 4]) = sums(i, h);
    sync_cluster();
    const int col = tid % 32 * 4;
    for (int i = static_cast<int>(rank) * (TM / a.ks) + tid / 32;
         i < (static_cast<int>(rank) + 1) * (TM / a.ks); i += THREADS / 32) {
        if (m0 + i >= m_end) break;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t c = 0; c < static_cast<uint32_t>(a.ks); ++c) {
            const float4 v = load_from_rank(&part[i][col], c);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
        finish_quad<T, MODE>(a, g, m0 + i, n0 + col, n_end, sum);
    }
    sync_cluster();  // no CTA leaves while another reads its sums
}

// U(i, c) = s_a * sum_k X(i, k) LA_a(k, c), a = adapter[i]: one CTA per row,
// one warp per column c, the lanes over k and a fixed shuffle tree.
constexpr int kShrinkThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_simt_kernel(const LoraProblem p, float *U) {
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int64_t i = blockIdx.x; i < p.M; i += gridDim.x) {
        const int64_t ad = p.adapter[i];
        if (ad < 0 || ad >= p.adapters) continue;
        const T *x = static_cast<const T *>(p.X) + i * p.ldx;
        const T *la = static_cast<const T *>(p.LA) + ad * p.stride_a;
        const float scale = p.scale != nullptr ? p.scale[ad] : 1.f;
        for (int64_t c = warp; c < p.rank; c += kShrinkThreads / 32) {
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
    cudaLaunchAttribute attr[2];
    set_pdl_attribute(&attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.ks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(Shape<MODE>::THREADS, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = a.ks > 1 ? 2 : 1;
    const cudaError_t e = cudaFuncSetAttribute(grouped_simt_kernel<T, MODE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
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

// Rows of a matrix (and the matrices of a stack) start on `bytes`.
bool rows_on(const void *p, int64_t ld, int64_t stride, int64_t elt, int64_t bytes) {
    return (static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) % 16) | (ld * elt) | (stride * elt)) %
               bytes == 0;
}

// CTAs that share a tile's K: few are resident per SM, so a few tiles more than
// fit would take twice as long; up to 8 parts (each at least 128 of K) while
// there are fewer than 12 per SM.  (16 groups, 2000 rows, 1000 x 1024, 320
// tiles: 164 us in one part, 129 split, both with 8 x 4 per thread.)
int k_parts(int64_t tiles, int64_t k) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 1;
    int ks = 1;
    while (ks < 8 && tiles * ks < 6 * static_cast<int64_t>(sms) && k / (2 * ks) >= 128) ks *= 2;
    return ks;
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
    const int64_t elt = in == InType::F32 ? 4 : 2;
    a.vec_a = rows_on(p.A, p.lda, 0, elt, 4 * elt);
    a.vec_b = rows_on(p.B, p.ldb, p.groups > 1 ? p.stride_b : 0, elt, 4 * elt);
    a.vec_d = p.out == kOutF32 && rows_on(p.D, p.ldd, 0, 4, 16);
    // at most one partly filled row tile per group
    const int64_t live = p.groups < p.rows ? p.groups : p.rows;
    const int64_t row_tiles = p.rows / TM + live;
    // (the last tile of a group is half full on average)
    a.ks = k_parts((p.rows / TM + live / 2) * a.tiles_n, p.K);
    return launch_typed<kRows>(a, in, row_tiles * a.tiles_n * a.ks, stream);
}

cudaError_t launch_wgrad_simt(const WgradProblem &p, InType in, cudaStream_t stream,
                              const char **name) {
    *name = kNames[kWgrad][static_cast<int>(in)];
    SimtGroupedArgs a = {};
    a.w = p;
    a.tiles_m = tiles(p.M, TM);
    a.tiles_n = tiles(p.N, TN);
    const int64_t elt = in == InType::F32 ? 4 : 2;
    a.vec_a = rows_on(p.A, p.lda, 0, elt, 4 * elt);
    a.vec_b = rows_on(p.B, p.ldb, 0, elt, 4 * elt);
    a.vec_d = p.out == kOutF32 && rows_on(p.D, p.ldd, p.groups > 1 ? p.stride_d : 0, 4, 16) &&
              (p.beta == 0.f || rows_on(p.C, p.ldc, p.groups > 1 ? p.stride_c : 0, 4, 16));
    const int64_t all = p.groups * a.tiles_m * a.tiles_n;
    a.ks = k_parts(all, p.rows / p.groups);
    return launch_typed<kWgrad>(a, in, all * a.ks, stream);
}

cudaError_t launch_lora_simt(const LoraProblem &p, InType in, cudaStream_t stream,
                             const char **name) {
    *name = kNames[kLora][static_cast<int>(in)];
    if (in == InType::F32) return cudaErrorInvalidValue;
    SimtGroupedArgs a = {};
    a.l = p;
    GroupedProblem &g = a.g;
    g.groups = 1;
    g.N = p.N;
    g.K = p.K;
    g.alpha = 1.f;
    g.lda = p.ldx;
    g.B = p.W;
    g.ldb = p.ldw;
    g.b_kmajor = p.w_kmajor;
    g.ldd = p.ldd;
    g.bias = p.bias;
    g.act = p.act;
    g.out = p.out;
    a.tiles_n = tiles(p.N, TN);
    a.vec_a = rows_on(p.X, p.ldx, 0, 2, 8);
    a.vec_b = rows_on(p.W, p.ldw, 0, 2, 8);
    a.vec_d = p.out == kOutF32 && rows_on(p.D, p.ldd, 0, 4, 16);
    // U is at most 128 MiB (64 rows at least): more rows go in several launches
    int64_t chunk = p.M;
    void *u = nullptr;
    const bool any = p.adapters > 0 && p.rank > 0 && p.K > 0;
    cudaError_t e = cudaSuccess;
    if (any) {
        const int64_t fit = (int64_t(128) << 20) / (p.rank * static_cast<int64_t>(sizeof(float))) / TM * TM;
        const int64_t most = fit > TM ? fit : TM;
        if (chunk > most) chunk = most;
        e = workspace_alloc(static_cast<size_t>(chunk * p.rank) * sizeof(float), stream, &u);
        if (e != cudaSuccess) return e;
        a.U = static_cast<float *>(u);
    } else {
        a.l.adapters = 0;
    }
    for (int64_t row = 0; row < p.M && e == cudaSuccess; row += chunk) {
        a.l.M = g.rows = g.rows_a = p.M - row < chunk ? p.M - row : chunk;
        a.l.X = g.A = static_cast<const uint16_t *>(p.X) + row * p.ldx;
        g.D = static_cast<uint8_t *>(p.D) + row * p.ldd * (p.out == kOutF32 ? 4 : 2);
        if (any) {
            a.l.adapter = p.adapter + row;
            const unsigned grid = static_cast<unsigned>(a.l.M < 65536 ? a.l.M : 65536);
            if (in == InType::BF16)
                lora_shrink_simt_kernel<uint16_t><<<grid, kShrinkThreads, 0, stream>>>(a.l, static_cast<float *>(u));
            else
                lora_shrink_simt_kernel<__half><<<grid, kShrinkThreads, 0, stream>>>(a.l, static_cast<float *>(u));
            e = cudaGetLastError();
            if (e != cudaSuccess) break;
        }
        const int64_t all = static_cast<int64_t>(tiles(a.l.M, TM)) * a.tiles_n;
        a.ks = k_parts(all, p.K);
        e = launch_typed<kLora>(a, in, all * a.ks, stream);
    }
    if (u != nullptr) {
        const cudaError_t ef = workspace_free(u, stream);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

}  // namespace gemm
