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

#include "mixture.h"
#include "values.cuh"

namespace gemm {
namespace {

constexpr int kRowsAhead = 8;  // rows of Y in flight per thread

// `n` values of a row from column c on: 16 bytes at once, or one by one where
// the row does not start on 16 bytes or ends inside (n < PER_16).
template <int TYPE, bool VEC>
__device__ __forceinline__ void load_piece(const void *row, int64_t c, int n,
                                           float (&v)[Value<TYPE>::PER_16]) {
    using V = Value<TYPE>;
    if (VEC && n == V::PER_16) {
        V::unpack(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(row) + c * V::BYTES)), v);
    } else {
#pragma unroll
        for (int i = 0; i < V::PER_16; ++i) v[i] = i < n ? V::load(row, c + i) : 0.f;
    }
}

// `n` of WIDE values to a row of another type; and from one (the residual, dD).
template <int TYPE, bool VEC, int WIDE>
__device__ __forceinline__ void store_values(void *row, int64_t c, int n, const float (&v)[WIDE]) {
    using V = Value<TYPE>;
    if (VEC && n == WIDE) {
        uint8_t *to = static_cast<uint8_t *>(row) + c * V::BYTES;
#pragma unroll
        for (int i = 0; i < WIDE / V::PER_16; ++i)
            reinterpret_cast<uint4 *>(to)[i] = V::pack(v + i * V::PER_16);
    } else {
#pragma unroll
        for (int i = 0; i < WIDE; ++i)
            if (i < n) V::store(row, c + i, v[i]);
    }
}
template <int TYPE, bool VEC, int WIDE>
__device__ __forceinline__ void load_values(const void *row, int64_t c, int n, float (&v)[WIDE]) {
    using V = Value<TYPE>;
    if (VEC && n == WIDE) {
        const uint8_t *from = static_cast<const uint8_t *>(row) + c * V::BYTES;
#pragma unroll
        for (int i = 0; i < WIDE / V::PER_16; ++i) {
            float part[V::PER_16];
            V::unpack(reinterpret_cast<const uint4 *>(from)[i], part);
#pragma unroll
            for (int j = 0; j < V::PER_16; ++j) v[i * V::PER_16 + j] = part[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < WIDE; ++i) v[i] = i < n ? V::load(row, c + i) : 0.f;
    }
}

// A thread per 16 bytes of Y's columns and token; `pieces` of them in a row.
template <int YT, int DT, bool YVEC, bool DVEC>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ CombineProblem p,
                                                      int64_t pieces) {
    using Y = Value<YT>;
    constexpr int WIDE = Y::PER_16;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t all = p.tokens * pieces, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; q < all; q += step) {
        const int64_t t = all <= UINT32_MAX
                              ? static_cast<uint32_t>(q) / static_cast<uint32_t>(pieces)
                              : q / pieces;
        const int64_t c = (q - t * pieces) * WIDE;
        const int n = p.N - c < WIDE ? static_cast<int>(p.N - c) : WIDE;
        float sum[WIDE] = {};
        for (int64_t j0 = 0; j0 < p.k; j0 += kRowsAhead) {
            int32_t at[kRowsAhead];
            float w[kRowsAhead], y[kRowsAhead][WIDE];
#pragma unroll
            for (int j = 0; j < kRowsAhead; ++j) {
                const int64_t r = t * p.k + j0 + j;
                at[j] = j0 + j < p.k ? __ldg(p.position + r) : -1;
                w[j] = j0 + j < p.k && p.weights != nullptr ? __ldg(p.weights + r) : 1.f;
                if (at[j] < 0 || at[j] >= p.rows_y) at[j] = -1;
            }
#pragma unroll
            for (int j = 0; j < kRowsAhead; ++j)
                if (at[j] >= 0)
                    load_piece<YT, YVEC>(static_cast<const uint8_t *>(p.Y) + at[j] * p.ldy * Y::BYTES, c, n, y[j]);
#pragma unroll
            for (int j = 0; j < kRowsAhead; ++j) {
                if (at[j] < 0) continue;
#pragma unroll
                for (int i = 0; i < WIDE; ++i) sum[i] = fmaf(w[j], y[j][i], sum[i]);
            }
        }
        if (p.residual != nullptr) {
            float r[WIDE];
            load_values<DT, DVEC, WIDE>(
                static_cast<const uint8_t *>(p.residual) + t * p.ld_r * Value<DT>::BYTES, c, n, r);
#pragma unroll
            for (int i = 0; i < WIDE; ++i) sum[i] += r[i];
        }
        store_values<DT, DVEC, WIDE>(static_cast<uint8_t *>(p.D) + t * p.ldd * Value<DT>::BYTES, c,
                                     n, sum);
    }
}

// `warps` warps per token (1, 2, 4 or 8 of the CTA's eight).  A thread keeps its
// share of eight dot products; the token's warps add theirs in a fixed order.
template <int YT, int DT, bool YVEC, bool DVEC>
__global__ void __launch_bounds__(256) combine_grad_kernel(const __grid_constant__ CombineProblem p,
                                                           int64_t pieces, int warps) {
    using Y = Value<YT>;
    constexpr int WIDE = Y::PER_16;
    __shared__ float parts[8][kRowsAhead];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int in_token = warp % warps, per_cta = 8 / warps;
    const int64_t ctas = (p.tokens + per_cta - 1) / per_cta;
    for (int64_t b = blockIdx.x; b < ctas; b += gridDim.x) {
        const int64_t t = b * per_cta + warp / warps;
        for (int64_t j0 = 0; j0 < p.k; j0 += kRowsAhead) {
            int32_t at[kRowsAhead];
            float w[kRowsAhead], dot[kRowsAhead] = {};
#pragma unroll
            for (int j = 0; j < kRowsAhead; ++j) {
                const bool there = t < p.tokens && j0 + j < p.k;
                const int64_t r = t * p.k + j0 + j;
                at[j] = there ? __ldg(p.position + r) : -1;
                w[j] = there && p.weights != nullptr ? __ldg(p.weights + r) : 1.f;
                if (at[j] < 0 || at[j] >= p.rows_y) at[j] = -1;
            }
            for (int64_t v = in_token * 32 + lane; t < p.tokens && v < pieces; v += warps * 32) {
                const int64_t c = v * WIDE;
                const int n = p.N - c < WIDE ? static_cast<int>(p.N - c) : WIDE;
                float d[WIDE];
                load_values<DT, DVEC, WIDE>(
                    static_cast<const uint8_t *>(p.D) + t * p.ldd * Value<DT>::BYTES, c, n, d);
                if (p.dweights != nullptr) {
                    float y[kRowsAhead][WIDE];
#pragma unroll
                    for (int j = 0; j < kRowsAhead; ++j)
                        if (at[j] >= 0)
                            load_piece<YT, YVEC>(
                                static_cast<const uint8_t *>(p.Y) + at[j] * p.ldy * Y::BYTES, c, n, y[j]);
#pragma unroll
                    for (int j = 0; j < kRowsAhead; ++j) {
                        if (at[j] < 0) continue;
#pragma unroll
                        for (int i = 0; i < WIDE; ++i) dot[j] = fmaf(d[i], y[j][i], dot[j]);
                    }
                }
                if (p.dY != nullptr) {
#pragma unroll
                    for (int j = 0; j < kRowsAhead; ++j) {
                        if (at[j] < 0) continue;
                        float g[WIDE];
#pragma unroll
                        for (int i = 0; i < WIDE; ++i) g[i] = w[j] * d[i];
                        store_values<YT, YVEC, WIDE>(
                            static_cast<uint8_t *>(p.dY) + at[j] * p.ld_dy * Y::BYTES, c, n, g);
                    }
                }
            }
            if (p.dweights == nullptr) continue;
#pragma unroll
            for (int j = 0; j < kRowsAhead; ++j) {
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
            }
            if (warps > 1) {
                __syncthreads();  // (the parts of the step before have been read)
                if (lane == 0) {
#pragma unroll
                    for (int j = 0; j < kRowsAhead; ++j) parts[warp][j] = dot[j];
                }
                __syncthreads();
                if (in_token == 0) {
                    for (int s = 1; s < warps; ++s) {
#pragma unroll
                        for (int j = 0; j < kRowsAhead; ++j) dot[j] += parts[warp + s][j];
                    }
                }
            }
            if (in_token == 0 && t < p.tokens) {
#pragma unroll
                for (int j = 0; j < kRowsAhead; ++j)
                    if (lane == j && j0 + j < p.k)
                        p.dweights[t * p.k + j0 + j] = at[j] >= 0 ? dot[j] : 0.f;
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

template <int YT, int DT>
cudaError_t combine_as(const CombineProblem &p, cudaStream_t stream) {
    using Y = Value<YT>;
    using D = Value<DT>;
    const int64_t pieces = (p.N + Y::PER_16 - 1) / Y::PER_16;
    const int64_t threads = p.tokens * pieces;
    // few rows: small CTAs, so that every SM has one
    const int cta = threads < 152 * 256 ? 64 : 256;
    const int64_t ctas = (threads + cta - 1) / cta;
    const bool yv = rows_on_16(p.Y, p.ldy, Y::BYTES);
    const bool dv = rows_on_16(p.D, p.ldd, D::BYTES) &&
                    (p.residual == nullptr || rows_on_16(p.residual, p.ld_r, D::BYTES));
    if (yv)
        return dv ? launch(combine_kernel<YT, DT, true, true>, ctas, cta, stream, p, pieces)
                  : launch(combine_kernel<YT, DT, true, false>, ctas, cta, stream, p, pieces);
    return dv ? launch(combine_kernel<YT, DT, false, true>, ctas, cta, stream, p, pieces)
              : launch(combine_kernel<YT, DT, false, false>, ctas, cta, stream, p, pieces);
}

template <int YT, int DT>
cudaError_t combine_grad_as(const CombineProblem &p, cudaStream_t stream) {
    using Y = Value<YT>;
    using D = Value<DT>;
    const int64_t pieces = (p.N + Y::PER_16 - 1) / Y::PER_16;
    // two steps per thread at most, up to eight warps
    int warps = 1;
    while (warps < 8 && warps * 64 < pieces) warps *= 2;
    const int64_t ctas = (p.tokens + 8 / warps - 1) / (8 / warps);
    const bool yv = (p.dweights == nullptr || rows_on_16(p.Y, p.ldy, Y::BYTES)) &&
                    (p.dY == nullptr || rows_on_16(p.dY, p.ld_dy, Y::BYTES));
    const bool dv = rows_on_16(p.D, p.ldd, D::BYTES);
    if (yv)
        return dv ? launch(combine_grad_kernel<YT, DT, true, true>, ctas, 256, stream, p, pieces, warps)
                  : launch(combine_grad_kernel<YT, DT, true, false>, ctas, 256, stream, p, pieces, warps);
    return dv ? launch(combine_grad_kernel<YT, DT, false, true>, ctas, 256, stream, p, pieces, warps)
              : launch(combine_grad_kernel<YT, DT, false, false>, ctas, 256, stream, p, pieces, warps);
}

}  // namespace

cudaError_t launch_combine(const CombineProblem &p, cudaStream_t stream, const char **name) {
    *name = "combine";
    if (p.y_type == kOutF32) return combine_as<kOutF32, kOutF32>(p, stream);
    if (p.y_type == kOutBf16)
        return p.d_type == kOutF32 ? combine_as<kOutBf16, kOutF32>(p, stream)
                                   : combine_as<kOutBf16, kOutBf16>(p, stream);
    return p.d_type == kOutF32 ? combine_as<kOutF16, kOutF32>(p, stream)
                               : combine_as<kOutF16, kOutF16>(p, stream);
}

cudaError_t launch_combine_grad(const CombineProblem &p, cudaStream_t stream, const char **name) {
    *name = "combine_grad";
    if (p.y_type == kOutF32) return combine_grad_as<kOutF32, kOutF32>(p, stream);
    if (p.y_type == kOutBf16)
        return p.d_type == kOutF32 ? combine_grad_as<kOutBf16, kOutF32>(p, stream)
                                   : combine_grad_as<kOutBf16, kOutBf16>(p, stream);
    return p.d_type == kOutF32 ? combine_grad_as<kOutF16, kOutF32>(p, stream)
                               : combine_grad_as<kOutF16, kOutF16>(p, stream);
}

}  // namespace gemm
