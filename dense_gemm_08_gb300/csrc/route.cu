// route.cu -- the experts of each token and their weights, and the gradient of
// the weights with respect to the logits (the formulas stand in include/gemm.h).
//
// A warp per token; lane l holds the experts l * ept .. l * ept + ept - 1, so
// that among equal values the lowest lane, and in it the lowest register, is
// the lowest index.  The k largest come one after another: each lane keeps its
// best value as an integer of the same order, one redux finds the warp's
// largest and one ballot the lane; that lane drops it and looks for its next.
//
// The choice must not depend on how FP32 rounds.  Without a bias the order is
// the logits' own and nothing is rounded.  With one (and for group scores of two
// terms), c is computed in FP32 together with a bound of its error; wherever two
// values that a decision compares are closer than that, the token is chosen
// again in 64 bits.  That is 0.3 % of the tokens for 256 experts with sigmoid
// scores of N(0, 1.5^2) logits (FP64 runs at 1/64 of the FP32 rate: all tokens in
// FP64 would take some hundred times the kernel's time).
#include <type_traits>

#include "mixture.h"
#include "values.cuh"

namespace gemm {
namespace {

constexpr int kWarps = 4;  // tokens per CTA
constexpr uint32_t kAll = 0xffffffffu;

// Integers in the order of the values, 0 for "not there" (no value maps to it
// but -infinity, which is not there either); a NaN is the largest.
template <typename F>
struct Order;
template <>
struct Order<float> {
    using Key = uint32_t;
    static __device__ __forceinline__ Key of(float v) {
        if (isnan(v)) return 0xffffffffu;
        const uint32_t b = __float_as_uint(v + 0.f);  // -0 becomes 0
        const Key k = b >> 31 ? ~b : b | 0x80000000u;
        return v == -INFINITY ? 0u : k;
    }
    static __device__ __forceinline__ float value(Key k) {  // (NaN: some NaN)
        return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
    }
    static __device__ __forceinline__ Key warp_max(Key k) { return __reduce_max_sync(kAll, k); }
};
template <>
struct Order<double> {
    using Key = unsigned long long;
    static __device__ __forceinline__ Key of(double v) {
        if (isnan(v)) return ~0ull;
        const Key b = static_cast<Key>(__double_as_longlong(v + 0.0));
        const Key k = b >> 63 ? ~b : b | (1ull << 63);
        return v == -INFINITY ? 0ull : k;
    }
    static __device__ __forceinline__ double value(Key k) {
        return __longlong_as_double(static_cast<long long>(k >> 63 ? k & ~(1ull << 63) : ~k));
    }
    static __device__ __forceinline__ Key warp_max(Key k) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const Key o = __shfl_xor_sync(kAll, k, d);
            k = o > k ? o : k;
        }
        return k;
    }
};

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
template <typename F>
__device__ __forceinline__ F warp_max(F v) {  // (NaNs do not count)
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const F o = __shfl_xor_sync(kAll, v, d);
        v = o > v || isnan(v) ? o : v;
    }
    return v;
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// The two largest of both pairs (first >= second).
template <typename Key>
__device__ __forceinline__ void merge_top(Key &a1, Key &a2, Key b1, Key b2) {
    const Key low = a1 < b1 ? a1 : b1, second = a2 > b2 ? a2 : b2;
    a1 = a1 > b1 ? a1 : b1;
    a2 = low > second ? low : second;
}

// This lane's logits; -infinity past the last expert.
template <int TYPE, int VPT, bool VEC>
__device__ __forceinline__ void load_row(const RouteProblem &p, const void *row, int ept,
                                         float (&x)[VPT]) {
    using V = Value<TYPE>;
    const int lane = threadIdx.x % 32;
    if constexpr (VEC) {  // (experts = 32 * VPT)
        constexpr int BYTES = VPT * V::BYTES;
        const uint8_t *from = static_cast<const uint8_t *>(row) + lane * BYTES;
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                float v[V::PER_16];
                V::unpack(__ldg(reinterpret_cast<const uint4 *>(from) + i), v);
#pragma unroll
                for (int j = 0; j < V::PER_16; ++j) x[i * V::PER_16 + j] = v[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) x[i] = V::load(from, i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int e = lane * ept + i;
            x[i] = i < ept && e < p.experts ? V::load(row, e) : -INFINITY;
        }
    }
}

// The largest logit and the sum of exp(x - max) over the row.
template <typename F, int VPT>
__device__ __forceinline__ void softmax_stats(const float (&x)[VPT], F &m, F &z) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPT; ++i) top = fmaxf(top, x[i]);
    top = warp_max(top);
    m = top;
    z = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        z += x[i] == -INFINITY ? F(0) : exp_of(static_cast<F>(x[i]) - m);
    z = warp_sum(z);
}

// The token's choice: `mine` = lane j's expert (j < k), or -1.  In FP32 false
// where a decision is too close to call.
template <typename F, int VPT>
__device__ __forceinline__ bool choose(const RouteProblem &p, const float (&x)[VPT], int ept, F m,
                                       F z, int &mine) {
    using Key = typename Order<F>::Key;
    constexpr bool FAST = std::is_same<F, float>::value;
    const int lane = threadIdx.x % 32;
    const bool biased = p.bias != nullptr;
    const bool group_sums = p.groups > 1 && p.top == 2;
    bool safe = true;
    F most = 0;  // FP32: the largest s + |b|, which the error of c is in proportion to

    // scores, and c as an ordered integer
    Key key[VPT];
    F s[VPT];
    const F inv = z > 0 ? F(1) / z : F(0);  // (0: every expert is masked; NaN stays NaN below)
    float b[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int e = lane * ept + i;
        b[i] = biased && i < ept && e < p.experts ? __ldg(p.bias + e) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const bool masked = x[i] == -INFINITY;
        s[i] = 0;
        if ((biased || group_sums) && !masked) {
            if (p.score == kSigmoid)
                s[i] = F(1) / (F(1) + exp_of(-static_cast<F>(x[i])));
            else
                s[i] = isnan(z) ? z : exp_of(static_cast<F>(x[i]) - m) * inv;
        }
        if (biased) {
            const F c = s[i] + static_cast<F>(b[i]);
            key[i] = masked ? Key(0) : Order<F>::of(c);
            if (FAST && !masked && key[i] != 0) {
                const F size = s[i] + fabsf(b[i]);
                most = size > most ? size : most;
            }
        } else {
            key[i] = masked ? Key(0) : Order<F>::of(static_cast<F>(x[i]));
        }
    }
    // Errors in FP32.  A score: expf and the division a few units of 2^-24, the
    // sum z of a softmax at most 37 roundings, the rounding of x - m (it moves
    // exp(x - m) by 2^-24 |x - m| of itself, at most 0.37 * 2^-24 of the largest
    // score); altogether below 2^-18.7 of s + |b| for a softmax, 2^-21 for a
    // sigmoid.  Two values differ for certain when they are twice that apart,
    // sums of two of them four times.
    F tol = 0;
    if (FAST && biased) tol = warp_max(most) * (p.score == kSigmoid ? 0x1p-19f : 0x1p-17f);

    uint32_t out = 0;  // bit i: expert i of this lane is out of the choice
    if (p.groups > 1 && p.kept < p.groups) {
        const int size = p.experts / p.groups;
        Key g1 = 0, g2 = 0;  // lane g: group g's two largest
        // what the groups are compared by: c, or s where a sum is wanted
        auto by = [&](int i) -> Key {
            if (biased || !group_sums) return key[i];
            return x[i] == -INFINITY ? Key(0) : Order<F>::of(s[i]);
        };
        const int lanes = 32 / p.groups;  // of a group, when groups end with lanes
        if (32 % p.groups == 0 && p.experts == 32 * ept) {
            Key a1 = 0, a2 = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (i < ept) merge_top(a1, a2, by(i), Key(0));
            for (int d = lanes / 2; d > 0; d /= 2) {
                const Key o1 = __shfl_xor_sync(kAll, a1, d), o2 = __shfl_xor_sync(kAll, a2, d);
                merge_top(a1, a2, o1, o2);
            }
            g1 = __shfl_sync(kAll, a1, (lane * lanes) & 31);
            g2 = __shfl_sync(kAll, a2, (lane * lanes) & 31);
        } else {
            for (int g = 0; g < p.groups; ++g) {
                Key a1 = 0, a2 = 0;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int e = lane * ept + i;
                    if (i < ept && e >= g * size && e < (g + 1) * size) merge_top(a1, a2, by(i), Key(0));
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    const Key o1 = __shfl_xor_sync(kAll, a1, d), o2 = __shfl_xor_sync(kAll, a2, d);
                    merge_top(a1, a2, o1, o2);
                }
                if (lane == g) g1 = a1, g2 = a2;
            }
        }
        Key score = g1;
        if (p.top == 2 && g2 != 0) {
            score = Order<F>::of(Order<F>::value(g1) + Order<F>::value(g2));
            if (g1 == ~Key(0) || g2 == ~Key(0)) score = ~Key(0);  // (a NaN among them)
        }
        if (lane >= p.groups) score = 0;
        uint32_t kept = 0;
        Key last = 0;
        for (int r = 0; r < p.kept; ++r) {
            const Key left = (kept >> lane) & 1u ? Key(0) : score;
            const Key best = Order<F>::warp_max(left);
            if (best == 0) break;
            last = best;
            kept |= 1u << (__ffs(__ballot_sync(kAll, left == best)) - 1);
        }
        if (FAST && (biased || group_sums)) {
            const Key next = Order<F>::warp_max((kept >> lane) & 1u ? Key(0) : score);
            if (next != 0) {
                const F a = Order<F>::value(last), c = Order<F>::value(next);
                // (without a bias scores are positive, and their errors relative:
                // 2^-24 |x - m| <= 100 * 2^-24 more for a softmax)
                const F near = biased ? 2 * tol
                                      : a * (p.score == kSigmoid ? F(0x1p-18) : F(0x1p-15));
                if (!(a - c > near) || (!biased && !(a > F(1e-30)))) safe = false;
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i < ept && !((kept >> ((lane * ept + i) / size & 31)) & 1u)) out |= 1u << i;
    }
    if (!safe) return false;

    Key best = 0;
    int at = 0;
    auto look = [&]() {
        best = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (key[i] > best && !((out >> i) & 1u)) best = key[i], at = i;
        }
    };
    look();
    mine = -1;
    Key before = 0;
    int e_before = 0;
    // (with a bias one more round: the first that is not chosen must not be too close)
    const int rounds = FAST && biased ? p.k + 1 : p.k;
    for (int r = 0; r < rounds; ++r) {
        const Key top = Order<F>::warp_max(best);
        if (top == 0) break;
        const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;
        const int e = __shfl_sync(kAll, lane * ept + at, owner);
        if (FAST && biased && r > 0) {
            if (!(Order<F>::value(before) - Order<F>::value(top) > tol)) {
                // the same logit and the same bias are equal for certain
                float xa = 0.f, xb = 0.f;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    if (lane * ept + i == e_before) xa = x[i];
                    if (lane * ept + i == e) xb = x[i];
                }
                xa = __shfl_sync(kAll, xa, e_before / ept);
                xb = __shfl_sync(kAll, xb, owner);
                if (!(xa == xb && __ldg(p.bias + e_before) == __ldg(p.bias + e))) return false;
            }
        }
        before = top;
        e_before = e;
        if (r < p.k && lane == r) mine = e;
        if (lane == owner) {
            out |= 1u << at;
            look();
        }
    }
    return true;
}

// Rarely called, and much larger than the FP32 form: a function of its own.
template <int TYPE, int VPT, bool VEC>
__device__ __noinline__ int choose_exactly(const RouteProblem &p, const void *row, int ept) {
    float x[VPT];
    load_row<TYPE, VPT, VEC>(p, row, ept, x);
    double m = 0, z = 0;
    if (p.score == kSoftmax) softmax_stats<double>(x, m, z);
    int mine;
    choose<double>(p, x, ept, m, z, mine);
    return mine;
}

// log of the logistic function, for scores that FP32 cannot hold
__device__ __forceinline__ float log_sigmoid(float x) {
    return fminf(x, 0.f) - log1pf(expf(-fabsf(x)));
}

// The lane's share of the chosen experts' scores (lanes with `has`): s_j / sum s.
// Scores too small for FP32 keep their ratios.
__device__ __forceinline__ float share(const RouteProblem &p, bool has, float x) {
    if (p.score == kSoftmax) {
        const float m = warp_max(has ? x : -INFINITY);
        const float e = has ? expf(x - m) : 0.f;
        return e / warp_sum(e);
    }
    const float s = has ? 1.f / (1.f + expf(-x)) : 0.f;
    const float sum = warp_sum(s);
    if (sum < 1e-30f) {
        const float l = has ? log_sigmoid(x) : -INFINITY;
        const float m = warp_max(l);
        const float e = has ? expf(l - m) : 0.f;
        return e / warp_sum(e);
    }
    return s / sum;
}

template <int TYPE, int VPT, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const __grid_constant__ RouteProblem p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x % 32;
    const int ept = VEC ? VPT : (p.experts + 31) / 32;
    for (int64_t t = blockIdx.x * int64_t(kWarps) + threadIdx.x / 32; t < p.tokens;
         t += gridDim.x * int64_t(kWarps)) {
        const void *row = static_cast<const uint8_t *>(p.logits) + t * p.ld * Value<TYPE>::BYTES;
        float x[VPT];
        load_row<TYPE, VPT, VEC>(p, row, ept, x);
        const bool sums = p.bias != nullptr || (p.groups > 1 && p.top == 2);
        float m = 0.f, z = 0.f;
        if (p.score == kSoftmax && (sums || !p.renorm)) softmax_stats<float>(x, m, z);
        int mine;
        if (!choose<float>(p, x, ept, m, z, mine))
            mine = choose_exactly<TYPE, VPT, VEC>(p, row, ept);
        const bool has = lane < p.k && mine >= 0;
        const float mx = has ? Value<TYPE>::load(row, mine) : 0.f;
        float w;
        if (p.renorm) {
            w = share(p, has, mx);
            if (isnan(z)) w = z;  // (with a bias, other experts than the NaN may be chosen)
        } else if (p.score == kSigmoid) {
            w = 1.f / (1.f + expf(-mx));
        } else {
            w = expf(mx - m) / z;
        }
        if (lane < p.k) {
            p.chosen[t * p.k + lane] = mine;
            p.weights[t * p.k + lane] = has ? w * p.scale : 0.f;
        }
    }
}

// ------------------------------------------------------------------ gradient
// A warp per token, the row in shared memory: the chosen experts' terms are
// added to it (an expert named twice gets both), then it is written once.
// Renormalised weights depend on the chosen logits alone, and so do sigmoid
// scores: the row is then not read.
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) route_grad_kernel(const __grid_constant__ RouteProblem p) {
    using V = Value<TYPE>;
    extern __shared__ __align__(16) float rows[];
    const int lane = threadIdx.x % 32;
    const int pitch = (p.experts + 7) / 8 * 8;
    float *const mine = rows + threadIdx.x / 32 * pitch;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t t = blockIdx.x * int64_t(kWarps) + threadIdx.x / 32; t < p.tokens;
         t += gridDim.x * int64_t(kWarps)) {
        const void *row = static_cast<const uint8_t *>(p.logits) + t * p.ld * V::BYTES;
        int e = -1;
        if (lane < p.k) e = p.chosen[t * p.k + lane];
        const bool has = e >= 0 && e < p.experts;
        const float x = has ? V::load(row, e) : 0.f;
        const float dw = has ? p.dweights[t * p.k + lane] * p.scale : 0.f;
        float dx;
        if (p.renorm) {
            const float q = share(p, has, x);
            dx = q * (dw - warp_sum(has ? q * dw : 0.f));
            if (p.score == kSigmoid) dx *= 1.f / (1.f + expf(x));
            for (int i = lane; i < p.experts; i += 32) mine[i] = 0.f;
        } else if (p.score == kSigmoid) {
            dx = dw / (1.f + expf(-x)) / (1.f + expf(x));
            for (int i = lane; i < p.experts; i += 32) mine[i] = 0.f;
        } else {
            float m = -INFINITY;
            for (int i = lane; i < p.experts; i += 32) {
                const float v = V::load(row, i);
                mine[i] = v;
                m = fmaxf(m, v);
            }
            m = warp_max(m);
            float z = 0.f;
            for (int i = lane; i < p.experts; i += 32) {
                const float s = mine[i] == -INFINITY ? 0.f : expf(mine[i] - m);
                mine[i] = s;
                z += s;
            }
            z = warp_sum(z);
            const float inv = z == 0.f ? 0.f : 1.f / z;
            const float s = !has || x == -INFINITY ? 0.f : expf(x - m) * inv;
            dx = s * dw;
            const float dot = warp_sum(has ? dx : 0.f) * inv;
            for (int i = lane; i < p.experts; i += 32) mine[i] *= -dot;
        }
        __syncwarp();
        if (has) atomicAdd(mine + e, dx);
        __syncwarp();
        uint8_t *out = static_cast<uint8_t *>(p.dlogits) + t * p.ld_d * V::BYTES;
        if constexpr (VEC) {
            for (int i = lane; i < p.experts / V::PER_16; i += 32)
                reinterpret_cast<uint4 *>(out)[i] = V::pack(mine + i * V::PER_16);
        } else {
            for (int i = lane; i < p.experts; i += 32) V::store(out, i, mine[i]);
        }
        __syncwarp();
    }
}

template <typename K>
cudaError_t launch(K kernel, const RouteProblem &p, size_t smem, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    set_pdl_attribute(&attr);
    cudaLaunchConfig_t cfg = {};
    const int64_t ctas = (p.tokens + kWarps - 1) / kWarps;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas < (1 << 20) ? ctas : (1 << 20)), 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int TYPE, int VPT>
cudaError_t route_as(const RouteProblem &p, cudaStream_t stream) {
    // whole lanes of 16-byte (or smaller, whole) pieces
    const bool vec = p.experts == 32 * VPT && rows_on_16(p.logits, p.ld, Value<TYPE>::BYTES);
    return vec ? launch(route_kernel<TYPE, VPT, true>, p, 0, stream)
               : launch(route_kernel<TYPE, VPT, false>, p, 0, stream);
}

template <int TYPE>
cudaError_t route_of(const RouteProblem &p, cudaStream_t stream) {
    const int ept = (p.experts + 31) / 32;
    if (ept <= 2) return route_as<TYPE, 2>(p, stream);
    if (ept <= 4) return route_as<TYPE, 4>(p, stream);
    if (ept <= 8) return route_as<TYPE, 8>(p, stream);
    if (ept <= 16) return route_as<TYPE, 16>(p, stream);
    return route_as<TYPE, 32>(p, stream);
}

template <int TYPE>
cudaError_t route_grad_of(const RouteProblem &p, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>((p.experts + 7) / 8 * 8) * kWarps * sizeof(float);
    const bool vec = p.experts % Value<TYPE>::PER_16 == 0 &&
                     rows_on_16(p.dlogits, p.ld_d, Value<TYPE>::BYTES);
    return vec ? launch(route_grad_kernel<TYPE, true>, p, smem, stream)
               : launch(route_grad_kernel<TYPE, false>, p, smem, stream);
}

}  // namespace

cudaError_t launch_route(const RouteProblem &p, cudaStream_t stream, const char **name) {
    *name = "route";
    if (p.type == kOutF32) return route_of<kOutF32>(p, stream);
    return p.type == kOutBf16 ? route_of<kOutBf16>(p, stream) : route_of<kOutF16>(p, stream);
}

cudaError_t launch_route_grad(const RouteProblem &p, cudaStream_t stream, const char **name) {
    *name = "route_grad";
    if (p.type == kOutF32) return route_grad_of<kOutF32>(p, stream);
    return p.type == kOutBf16 ? route_grad_of<kOutBf16>(p, stream)
                              : route_grad_of<kOutF16>(p, stream);
}

}  // namespace gemm
