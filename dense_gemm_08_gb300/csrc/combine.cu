// combine.cu -- the experts' rows back to the tokens, and its gradients:
//
//   D(t, :) = residual(t, :) + sum_j w(t, j) Y(position(t, j), :)
//   dY(position(t, j), :) = w(t, j) dD(t, :),  dw(t, j) = <dD(t, :), Y(position(t, j), :)>
//
// Both are bound by memory: every row of Y is used once.  A thread takes 16
// bytes of a token's columns and has the loads of eight of its rows in flight.
// Going by position (tokens in order, rows gathered) instead of by row needs no
// atomics, fixes the order of each sum, and reads a token's dD once for all its
// experts.
#include <type_traits>

#include "combine.h"
#include "internal.h"

namespace gemm {
namespace {

// Loads of Y in flight per thread: R rows (the power of two that k fills, at most
// 8) times the pieces of each.  (k = 2 with one piece of two rows: 369 us for 16384
// tokens of 8192 BF16 columns.)
__host__ __device__ constexpr int pieces_of(int rows) { return rows == 8 ? 1 : rows == 1 ? 4 : 2; }
constexpr int kGradThreads = 256;

// Row numbers and weights of R of a token's choices from j0 on (-1: none).
template <int R>
struct Choices {
    int32_t at[R];
    float w[R];
    __device__ __forceinline__ Choices(const CombineProblem &p, int64_t t, int64_t j0) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const bool there = t < p.tokens && j0 + j < p.k;
            at[j] = there ? __ldg(p.position + t * p.k + j0 + j) : -1;
            w[j] = there && p.weights != nullptr ? __ldg(p.weights + t * p.k + j0 + j) : 1.f;
        }
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (at[j] < 0 || at[j] >= p.rows_y) at[j] = -1;
    }
};

// A thread's C pieces of D, `apart` columns apart from column c0 on.  HELD: what of
// them is inside the row.  (With loads of single values for all pieces of a run that
// is not all inside, the gradient of 16384 tokens, 4 rows of 640 BF16, took 126 us, now
// 78; with whole pieces that are there or not as the only other way, 8 rows of 512
// took 89, now 58.)
template <int YT, int DT, bool YVEC, int HELD, int R, int C>
__device__ __forceinline__ void combine_pieces(const CombineProblem &p, int64_t t, int64_t c0,
                                               int64_t apart, bool dvec) {
    using Y = Value<YT>;
    constexpr int WIDE = Y::PER_16;
    float sum[C][WIDE] = {}, r[C][WIDE] = {};
    int n[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t left = p.N - (c0 + c * apart);
        n[c] = HELD == kAll || left >= WIDE ? WIDE : (left > 0 ? static_cast<int>(left) : 0);
        // (the residual is under way with the rows)
        if (p.residual != nullptr)
            load_values<DT, HELD, WIDE>(p.residual, t * p.ld_r, c0 + c * apart, n[c], dvec, r[c]);
    }
    for (int64_t j0 = 0; j0 < p.k; j0 += R) {
        const Choices<R> ch(p, t, j0);
        uint4 q[R][C];
#pragma unroll
        for (int j = 0; j < R; ++j) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                q[j][c] = make_uint4(0, 0, 0, 0);
                if (ch.at[j] >= 0)
                    q[j][c] = load_piece<YT, YVEC, HELD>(p.Y, ch.at[j] * p.ldy, c0 + c * apart, n[c]);
            }
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (ch.at[j] < 0) continue;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float y[WIDE];
                Y::unpack(q[j][c], y);
#pragma unroll
                for (int i = 0; i < WIDE; ++i) sum[c][i] = fmaf(ch.w[j], y[i], sum[c][i]);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < WIDE; ++i) sum[c][i] += r[c][i];
        store_values<DT, HELD, WIDE>(p.D, t * p.ldd, c0 + c * apart, n[c], dvec, sum[c]);
    }
}

// `lanes` threads (a power of two, at most 32) take lanes * C pieces of a token:
// piece (chunk * C + c) * lanes + lane; `chunks` such runs make a row.
template <int YT, int DT, bool YVEC, int R>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ CombineProblem p,
                                                      int lanes, uint32_t chunks, bool dvec) {
    constexpr int WIDE = Value<YT>::PER_16, C = pieces_of(R);
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t all = p.tokens * chunks, step = static_cast<int64_t>(gridDim.x) * (blockDim.x / lanes);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes; u < all;
         u += step) {
        const int64_t t = all <= UINT32_MAX ? static_cast<uint32_t>(u) / chunks : u / chunks;
        const int64_t apart = lanes * WIDE, run = (u - t * chunks) * C * apart, c0 = run + lane * WIDE;
        // (several pieces: the same way for all threads of a run)
        if ((C == 1 ? c0 + WIDE : run + C * apart) <= p.N)
            combine_pieces<YT, DT, YVEC, kAll, R, C>(p, t, c0, apart, dvec);
        else if (c0 >= p.N)
            continue;
        else if (C > 1 && !has_end<WIDE, C>(p.N, c0, apart))
            combine_pieces<YT, DT, YVEC, (C > 1 ? kAllOrNone : kSome), R, C>(p, t, c0, apart, dvec);
        else
            combine_pieces<YT, DT, YVEC, kSome, R, C>(p, t, c0, apart, dvec);
    }
}

// A thread's C pieces of the gradients: its part of the dot products, and dY.
template <int YT, int DT, bool YVEC, int HELD, int R, int C>
__device__ __forceinline__ void grad_pieces(const CombineProblem &p, const Choices<R> &ch, int64_t t,
                                            int64_t c0, int64_t apart, bool dvec,
                                            float (&dot)[R]) {
    using Y = Value<YT>;
    constexpr int WIDE = Y::PER_16;
    uint4 q[R][C];
    int n[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t left = p.N - (c0 + c * apart);
        n[c] = HELD == kAll || left >= WIDE ? WIDE : (left > 0 ? static_cast<int>(left) : 0);
    }
    if (p.dweights != nullptr) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                q[j][c] = make_uint4(0, 0, 0, 0);
                if (ch.at[j] >= 0)
                    q[j][c] = load_piece<YT, YVEC, HELD>(p.Y, ch.at[j] * p.ldy, c0 + c * apart, n[c]);
            }
        }
    }
    float d[C][WIDE];
#pragma unroll
    for (int c = 0; c < C; ++c)
        load_values<DT, HELD, WIDE>(p.D, t * p.ldd, c0 + c * apart, n[c], dvec, d[c]);
    if (p.dY != nullptr) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (ch.at[j] < 0) continue;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float g[WIDE];
#pragma unroll
                for (int i = 0; i < WIDE; ++i) g[i] = ch.w[j] * d[c][i];
                store_values<YT, HELD, WIDE>(p.dY, ch.at[j] * p.ld_dy, c0 + c * apart, n[c], YVEC, g);
            }
        }
    }
    if (p.dweights != nullptr) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (ch.at[j] < 0) continue;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float y[WIDE];
                Y::unpack(q[j][c], y);
#pragma unroll
                for (int i = 0; i < WIDE; ++i) dot[j] = fmaf(d[c][i], y[i], dot[j]);
            }
        }
    }
}

// `lanes` threads per token (a power of two, at most the CTA's).  A thread keeps
// its share of R dot products; they are added in a fixed order.
template <int YT, int DT, bool YVEC, int R>
__global__ void __launch_bounds__(kGradThreads) combine_grad_kernel(const __grid_constant__ CombineProblem p,
                                                           int lanes, bool dvec) {
    constexpr int WIDE = Value<YT>::PER_16, C = pieces_of(R);
    __shared__ float parts[kGradThreads / 32][R];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & (lanes - 1), per_cta = kGradThreads / lanes;
    const int warp = threadIdx.x / 32, warps = lanes / 32;  // warps of a token (0: part of one)
    const int64_t ctas = (p.tokens + per_cta - 1) / per_cta, apart = lanes * WIDE;
    for (int64_t b = blockIdx.x; b < ctas; b += gridDim.x) {
        const int64_t t = b * per_cta + threadIdx.x / lanes;
        for (int64_t j0 = 0; j0 < p.k; j0 += R) {
            const Choices<R> ch(p, t, j0);
            float dot[R] = {};
            if (t < p.tokens) {
                for (int64_t c0 = lane * WIDE; c0 < p.N; c0 += C * apart) {
                    if ((C == 1 ? c0 + WIDE : c0 - lane * WIDE + C * apart) <= p.N)
                        grad_pieces<YT, DT, YVEC, kAll, R, C>(p, ch, t, c0, apart, dvec, dot);
                    else if (C > 1 && !has_end<WIDE, C>(p.N, c0, apart))
                        grad_pieces<YT, DT, YVEC, (C > 1 ? kAllOrNone : kSome), R, C>(p, ch, t, c0, apart, dvec,
                                                                                      dot);
                    else
                        grad_pieces<YT, DT, YVEC, kSome, R, C>(p, ch, t, c0, apart, dvec, dot);
                }
            }
            if (p.dweights == nullptr) continue;
            for (int s = (lanes < 32 ? lanes : 32) / 2; s > 0; s >>= 1) {
#pragma unroll
                for (int j = 0; j < R; ++j) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
            }
            if (warps > 1) {
                __syncthreads();  // (the parts of the step before have been read)
                if (lane % 32 == 0) {
#pragma unroll
                    for (int j = 0; j < R; ++j) parts[warp][j] = dot[j];
                }
                __syncthreads();
                if (lane == 0) {
                    for (int s = 1; s < warps; ++s) {
#pragma unroll
                        for (int j = 0; j < R; ++j) dot[j] += parts[warp + s][j];
                    }
                }
            }
            if (lane == 0 && t < p.tokens) {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (j0 + j < p.k) p.dweights[t * p.k + j0 + j] = ch.at[j] >= 0 ? dot[j] : 0.f;
            }
        }
    }
}

template <typename K, typename... A>
cudaError_t launch(K kernel, int64_t ctas, int threads, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr;
    set_pdl_attribute(&attr);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas < (1 << 20) ? ctas : (1 << 20)), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The power of two at or above n, at most `most`.
int power_of_2(int64_t n, int most) {
    int v = 1;
    while (v < n && v < most) v *= 2;
    return v;
}

template <int YT, int DT, int R>
cudaError_t combine_as(const CombineProblem &p, cudaStream_t stream) {
    using Y = Value<YT>;
    using D = Value<DT>;
    const int64_t pieces = (p.N + Y::PER_16 - 1) / Y::PER_16, per_thread = pieces_of(R);
    const int lanes = power_of_2((pieces + per_thread - 1) / per_thread, 32);
    const int64_t chunks = (pieces + lanes * per_thread - 1) / (lanes * per_thread);
    const int64_t threads = p.tokens * chunks * lanes;
    // few rows: small CTAs, so that every SM has one
    const int cta = threads < int64_t(sm_count()) * 256 ? 64 : 256;
    const int64_t ctas = (threads + cta - 1) / cta;
    const bool yv = rows_on_16(p.Y, p.ldy, Y::BYTES);
    const bool dv = rows_on_16(p.D, p.ldd, D::BYTES) &&
                    (p.residual == nullptr || rows_on_16(p.residual, p.ld_r, D::BYTES));
    const uint32_t n = static_cast<uint32_t>(chunks);
    return yv ? launch(combine_kernel<YT, DT, true, R>, ctas, cta, stream, p, lanes, n, dv)
              : launch(combine_kernel<YT, DT, false, R>, ctas, cta, stream, p, lanes, n, dv);
}

template <int YT, int DT, int R>
cudaError_t combine_grad_as(const CombineProblem &p, cudaStream_t stream) {
    using Y = Value<YT>;
    using D = Value<DT>;
    const int64_t pieces = (p.N + Y::PER_16 - 1) / Y::PER_16, per_thread = pieces_of(R);
    // two steps per thread, up to a CTA per token
    const int lanes = power_of_2((pieces + 2 * per_thread - 1) / (2 * per_thread), kGradThreads);
    const int64_t ctas = (p.tokens + kGradThreads / lanes - 1) / (kGradThreads / lanes);
    const bool yv = (p.dweights == nullptr || rows_on_16(p.Y, p.ldy, Y::BYTES)) &&
                    (p.dY == nullptr || rows_on_16(p.dY, p.ld_dy, Y::BYTES));
    const bool dv = rows_on_16(p.D, p.ldd, D::BYTES);
    const int n = kGradThreads;
    return yv ? launch(combine_grad_kernel<YT, DT, true, R>, ctas, n, stream, p, lanes, dv)
              : launch(combine_grad_kernel<YT, DT, false, R>, ctas, n, stream, p, lanes, dv);
}

template <int YT, int DT>
cudaError_t combine_rows(const CombineProblem &p, cudaStream_t stream) {
    if (p.k <= 1) return combine_as<YT, DT, 1>(p, stream);
    if (p.k == 2) return combine_as<YT, DT, 2>(p, stream);
    return p.k <= 4 ? combine_as<YT, DT, 4>(p, stream) : combine_as<YT, DT, 8>(p, stream);
}
template <int YT, int DT>
cudaError_t combine_grad_rows(const CombineProblem &p, cudaStream_t stream) {
    if (p.k <= 1) return combine_grad_as<YT, DT, 1>(p, stream);
    if (p.k == 2) return combine_grad_as<YT, DT, 2>(p, stream);
    return p.k <= 4 ? combine_grad_as<YT, DT, 4>(p, stream) : combine_grad_as<YT, DT, 8>(p, stream);
}

}  // namespace

cudaError_t launch_combine(const CombineProblem &p, cudaStream_t stream, const char **name) {
    if (combine_bulk_eligible(p, false)) {
        *name = "combine<bulk>";
        return launch_combine_bulk(p, false, stream);
    }
    *name = "combine";
    if (p.y_type == kOutF32) return combine_rows<kOutF32, kOutF32>(p, stream);
    if (p.y_type == kOutBf16)
        return p.d_type == kOutF32 ? combine_rows<kOutBf16, kOutF32>(p, stream)
                                   : combine_rows<kOutBf16, kOutBf16>(p, stream);
    return p.d_type == kOutF32 ? combine_rows<kOutF16, kOutF32>(p, stream)
                               : combine_rows<kOutF16, kOutF16>(p, stream);
}

cudaError_t launch_combine_grad(const CombineProblem &p, cudaStream_t stream, const char **name) {
    if (combine_bulk_eligible(p, true)) {
        *name = "combine_grad<bulk>";
        return launch_combine_bulk(p, true, stream);
    }
    *name = "combine_grad";
    if (p.y_type == kOutF32) return combine_grad_rows<kOutF32, kOutF32>(p, stream);
    if (p.y_type == kOutBf16)
        return p.d_type == kOutF32 ? combine_grad_rows<kOutBf16, kOutF32>(p, stream)
                                   : combine_grad_rows<kOutBf16, kOutBf16>(p, stream);
    return p.d_type == kOutF32 ? combine_grad_rows<kOutF16, kOutF32>(p, stream)
                               : combine_grad_rows<kOutF16, kOutF16>(p, stream);
}

}  // namespace gemm
