// route.cu -- the experts of each token and their weights, and the gradient of
// the weights with respect to the logits (the formulas stand in include/gemm.h).
//
// A warp per token; lane l holds the experts l * ept .. l * ept + ept - 1, and
// values are compared as integers of the same order.  The k largest:
//   1. a lower bound of the k-th largest: the k-th largest of the lanes' own
//      largest values (each lane counts, from shared memory, how many lanes have at
//      least its own);
//   2. the values that reach it, some k + 1 to k + 3 of them, are dealt out to the
//      lanes, one each; a lane counts those that come before its own: its place.
// No step waits on a chain of shuffles (two sorts across the lanes, or k rounds of
// one maximum each, took twice the time).  Where more than 32 values reach the
// bound (a row of equal logits) they are taken one after another.
//
// The choice must not depend on how FP32 rounds.  Without a bias the order is
// the logits' own and nothing is rounded.  With one, c is computed in FP32 together
// with a bound of its error; the candidates are all that could be among the k
// largest, and where two that are next to each other are closer than that, the
// candidates (one per lane) are compared again in 64 bits: 0.3 % of the tokens for
// 256 experts with sigmoid scores of N(0, 1.5^2) logits.  Group scores of two rounded
// terms that are too close are rarer; those groups' largest experts are then computed
// in 64 bits, or, where they are too many, the whole token is chosen again.  (FP64 runs
// at 1/64 of the FP32 rate.)
#include <type_traits>

#include "mixture.h"
#include "values.cuh"

namespace gemm {
namespace {

constexpr int kWarps = 4;  // tokens per CTA
constexpr uint32_t kAll = 0xffffffffu;

// Integers in the order of the values, 0 for -infinity ("not there"); a NaN is the
// largest.  Adding 0 makes -0 a 0 and every NaN the one with all bits but the sign.
template <typename F>
struct Order;
template <>
struct Order<float> {
    using Key = uint32_t;
    static __device__ __forceinline__ Key of(float v) {
        const int b = __float_as_int(v + 0.f);
        return static_cast<Key>(b ^ ((b >> 31) | INT32_MIN)) - 0x007fffffu;
    }
    static __device__ __forceinline__ float value(Key k) {
        const uint32_t b = k + 0x007fffffu;
        return __uint_as_float(b >> 31 ? b & 0x7fffffffu : ~b);
    }
    static __device__ __forceinline__ Key warp_max(Key k) { return __reduce_max_sync(kAll, k); }
    static constexpr Key NAN_KEY = 0xff800000u;
};
template <>
struct Order<double> {
    using Key = unsigned long long;
    static __device__ __forceinline__ Key of(double v) {
        if (isnan(v)) return NAN_KEY;
        const Key b = static_cast<Key>(__double_as_longlong(v + 0.0));
        const Key k = b >> 63 ? ~b : b | (1ull << 63);
        return v == -INFINITY ? 0ull : k;
    }
    static __device__ __forceinline__ double value(Key k) {  // (not of a NaN's)
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
    static constexpr Key NAN_KEY = ~0ull;
};

// The lanes that n values take, as a power of two.
__device__ __forceinline__ int lanes_of(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }

// Sums and maxima over the warp (NaNs do not count), or its first `width` lanes.
template <typename F>
__device__ __forceinline__ F warp_sum(F v, int width = 32) {
    for (int d = width / 2; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v, int width = 32) {
    for (int d = width / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
// For the choice: the hardware's exponential (off by 2 + 1.2 |x| units of 2^-23) and
// reciprocal (2 units; 0 past 2^126) in FP32.
__device__ __forceinline__ float rough_exp(float x) { return __expf(x); }
__device__ __forceinline__ double rough_exp(double x) { return exp(x); }
__device__ __forceinline__ float rough_inverse(float x) { return __fdividef(1.f, x); }
__device__ __forceinline__ double rough_inverse(double x) { return 1.0 / x; }

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
    m = warp_max(top);
    z = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        z += x[i] == -INFINITY ? F(0) : exp_of(static_cast<F>(x[i]) - m);
    z = warp_sum(z);
}

// A score for the choice, from the row's statistics (1 / z, or z itself if that is a NaN).
template <typename F>
__device__ __forceinline__ F score_of(const RouteProblem &p, float x, F m, F inv) {
    if (p.score == kSigmoid) return rough_inverse(F(1) + rough_exp(-static_cast<F>(x)));
    return isnan(inv) ? inv : rough_exp(static_cast<F>(x) - m) * inv;
}

// The k largest keys one after another: each time the warp's largest, and among
// its equals the lowest number.  Lane r gets the r-th one's number (or -1).
template <typename F, int VPT>
__device__ __forceinline__ int in_rounds(const RouteProblem &p, int ept,
                                         const typename Order<F>::Key (&key)[VPT]) {
    using Key = typename Order<F>::Key;
    const int lane = threadIdx.x % 32;
    int mine = -1, at = 0;
    uint32_t out = 0;  // bit i: taken
    Key best;
    auto look = [&]() {
        best = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (key[i] > best && !((out >> i) & 1u)) best = key[i], at = i;
    };
    look();
    for (int r = 0; r < p.k; ++r) {
        const Key top = Order<F>::warp_max(best);
        if (top == 0) break;
        const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;
        const int e = __shfl_sync(kAll, lane * ept + at, owner);
        if (lane == r) mine = e;
        if (lane == owner) {
            out |= 1u << at;
            look();
        }
    }
    return mine;
}

// Shared memory of a warp.
template <int VPT>
struct Slots {
    __align__(16) uint32_t key[32 * VPT];  // of register i of lane l at l * VPT + i
    __align__(16) unsigned long long candidate[32];
    __align__(16) uint32_t best[32];
    uint16_t at[32];
    int number[32];
    float logit[32];
};

// The groups that stay, where FP32 cannot tell: `score`, the lane's group's, lies near
// the border between `last` (stays) and `next` (does not).  Groups further off than
// `near` are certain; of the others the experts that may be among a group's two
// largest (at least its second, g2, less `tol`, or a relative bound without a bias) are
// dealt out to the lanes and computed in 64 bits.  False: more than 32 of them, or NaNs.
// (Choosing the whole token again in 64 bits takes 8 us, at the end of a launch more
// often than not: 16384 tokens of 256 experts in 8 groups 30 us, now 25.)
template <int TYPE, int VPT, bool VEC>
__device__ __noinline__ bool kept_exactly(const RouteProblem &p, const void *row, int ept,
                                          Slots<VPT> &s, float m, float z, uint32_t g2, uint32_t score,
                                          uint32_t last, uint32_t next, float near, float tol,
                                          uint32_t &kept) {
    using V = Value<TYPE>;
    const int lane = threadIdx.x % 32, size = p.experts / p.groups;
    const bool biased = p.bias != nullptr;
    const float high = Order<float>::value(last) + near, low = Order<float>::value(next) - near;
    if (!(high >= low) || (!biased && !(low > 1e-30f))) return false;
    const float mine = Order<float>::value(score);
    const bool open = score != 0 && mine <= high && mine >= low;
    const uint32_t in = __ballot_sync(kAll, score != 0 && !open && score > last);
    // what an expert of the lane's group must reach
    float least = -INFINITY;
    if (g2 != 0 && p.top == 2)
        least = biased ? Order<float>::value(g2) - tol : Order<float>::value(g2) * (1.f - 0x1p-14f);
    else if (p.top == 1)
        least = mine - tol;
    if (__any_sync(kAll, open && isnan(least))) return false;
    const uint32_t opened = __ballot_sync(kAll, open);
    float x[VPT];
    load_row<TYPE, VPT, VEC>(p, row, ept, x);
    const float inv = z > 0 ? 1.f / z : 0.f;
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int e = lane * ept + i;
        const bool there = i < ept && e < p.experts;
        const int g = there ? e / size : 0;
        const float from = __shfl_sync(kAll, least, g);
        if (!there || x[i] == -INFINITY || !((opened >> g) & 1u)) continue;
        const float b = biased ? __ldg(p.bias + e) : 0.f;
        const float c = score_of<float>(p, x[i], m, inv) + b;
        if (!(c < from) && b != -INFINITY) mask |= 1u << i;
    }
    int total = 0;
    for (uint32_t who; (who = __ballot_sync(kAll, mask != 0)) != 0; mask &= mask - 1) {
        const int slot = total + __popc(who & ((1u << lane) - 1u));
        if (mask != 0 && slot < 32) s.at[slot] = static_cast<uint16_t>(lane * ept + __ffs(mask) - 1);
        total += __popc(who);
        if (total > 32) break;
    }
    __syncwarp();
    if (total > 32) return false;
    double md = 0, zd = 0;
    if (p.score == kSoftmax) softmax_stats<double>(x, md, zd);
    using Key = Order<double>::Key;
    Key key = 0;
    int of = -1;
    if (lane < total) {
        const int e = s.at[lane];
        double c = score_of<double>(p, V::load(row, e), md, 1.0 / zd);
        if (biased) c += __ldg(p.bias + e);
        key = Order<double>::of(c);
        of = e / size;
    }
    Key a1 = 0, a2 = 0;
    for (int i = 0; i < total; ++i) {
        const Key o = __shfl_sync(kAll, key, i);
        if (__shfl_sync(kAll, of, i) == lane) merge_top(a1, a2, o, Key(0));
    }
    Key sum = a1;
    if (p.top == 2 && a2 != 0)
        sum = a1 == Order<double>::NAN_KEY ? a1
                                           : Order<double>::of(Order<double>::value(a1) + Order<double>::value(a2));
    int before = 0;
    for (int g = 0; g < p.groups; ++g) {
        const Key o = __shfl_sync(kAll, sum, g);
        if ((opened >> g) & 1u) before += o > sum || (o == sum && g < lane) ? 1 : 0;
    }
    kept = in | __ballot_sync(kAll, open && before < p.kept - __popc(in));
    __syncwarp();
    return true;
}

// Keys of the lane's experts, 0 where they or their groups are out of the choice.
// tol: how far apart two c must be to differ for certain.  FP32: false where two
// groups are too close.
template <typename F, int TYPE, int VPT, bool VEC>
__device__ __forceinline__ bool keys_of(const RouteProblem &p, const void *row, Slots<VPT> *slots,
                                        const float (&x)[VPT], int ept, F m, F z,
                                        typename Order<F>::Key (&key)[VPT], float &tol) {
    using Key = typename Order<F>::Key;
    constexpr bool FAST = std::is_same<F, float>::value;
    const int lane = threadIdx.x % 32;
    const bool biased = p.bias != nullptr;
    const bool group_sums = p.groups > 1 && p.top == 2;
    Key by[VPT];  // what groups are compared by: c, or s for a sum without a bias
    tol = 0.f;
    if (biased || group_sums) {
        const F inv = z > 0 ? F(1) / z : (isnan(z) ? z : F(0));  // (0: every expert is masked)
        float most = 0.f, b[VPT] = {};
        if (biased) {
            const float *from = p.bias + lane * ept;
            if (VEC && VPT % 4 == 0 && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0) {
#pragma unroll
                for (int i = 0; i < VPT / 4; ++i) {
                    const float4 q = __ldg(reinterpret_cast<const float4 *>(from) + i);
                    b[i * 4] = q.x, b[i * 4 + 1] = q.y, b[i * 4 + 2] = q.z, b[i * 4 + 3] = q.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (i < ept && lane * ept + i < p.experts) b[i] = __ldg(from + i);
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            // (a bias of -infinity is a mask too, also of a NaN)
            const bool masked = x[i] == -INFINITY || (biased && b[i] == -INFINITY);
            const F s = masked ? F(0) : score_of<F>(p, x[i], m, inv);
            if (biased) {
                key[i] = masked ? Key(0) : Order<F>::of(s + static_cast<F>(b[i]));
                by[i] = key[i];
                if (FAST && key[i] != 0) most = fmaxf(most, static_cast<float>(s) + fabsf(b[i]));
            } else {
                key[i] = Order<F>::of(static_cast<F>(x[i]));
                by[i] = masked ? Key(0) : Order<F>::of(s);
            }
        }
        // Errors in FP32, in units of 2^-23; top is the largest s + |b|.  A score's
        // exponential is off by 2 + 1.2 d units of itself, with d = |x| for a sigmoid (past
        // x = 0 it is the smaller term, and d exp(-d) < 0.4) and d = m - x for a softmax, whose
        // x - m is rounded: 0.5 d more.  The sum and the reciprocal add 3 units, of a softmax
        // 25 (z is a sum of 37 roundings), c itself half a unit of s + |b|: 5 or 28 units of
        // top, and 1.2 or 1.7 d s.  As d <= log(1 / s), and s log(1 / s) grows up to s = 1 / e,
        // the latter is 1.2 or 1.7 log(1 / top) units of top at most: 3 or 4 from top = 1 / 8
        // on, and the largest part where all scores are small (a sigmoid's logits far below 0,
        // a softmax whose largest logits the bias masks; with 8 units for all, groups at -60
        // were chosen wrong).  Results below 2^-126 may be 0 instead.  So 8 or 32 units, times the
        // logarithm's share, and 2^-125; two values differ for certain when they are twice
        // that apart, sums of two of them four times.
        if (FAST && biased) {
            const float top = warp_max(most);
            tol = top * (p.score == kSigmoid ? 0x1p-19f : 0x1p-17f);
            if (top < 0.125f)
                tol *= 1.f - (p.score == kSigmoid ? 0.15f : 0.06f) * __logf(fmaxf(top, 0x1p-126f));
            tol += 0x1p-124f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) by[i] = key[i] = Order<F>::of(static_cast<F>(x[i]));
    }
    if (p.groups == 1 || p.kept == p.groups) return true;

    // lane g: group g's largest two
    Key g1 = 0, g2 = 0;
    const int size = p.experts / p.groups;
    const int lanes = 32 / p.groups;  // of a group, when groups end with lanes
    const bool aligned = 32 % p.groups == 0 && p.experts == 32 * ept;
    if (aligned) {
        Key a1 = 0, a2 = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i < ept) merge_top(a1, a2, by[i], Key(0));
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
                if (i < ept && e >= g * size && e < (g + 1) * size) merge_top(a1, a2, by[i], Key(0));
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
    if (p.top == 2 && g2 != 0)
        score = g1 == Order<F>::NAN_KEY ? g1
                                        : Order<F>::of(Order<F>::value(g1) + Order<F>::value(g2));
    if (lane >= p.groups) score = 0;
    // a group stays when fewer than groups_kept come before it
    int before = 0;
#pragma unroll 4
    for (int g = 0; g < p.groups; ++g) {
        const Key o = __shfl_sync(kAll, score, g);
        before += o > score || (o == score && g < lane) ? 1 : 0;
    }
    uint32_t kept = __ballot_sync(kAll, score != 0 && before < p.kept);
    if constexpr (FAST) {
        if (biased || group_sums) {
            const bool stays = (kept >> lane) & 1u;
            const Key next = Order<F>::warp_max(stays ? Key(0) : score);
            const Key last = ~Order<F>::warp_max(stays ? ~score : Key(0));
            if (next != 0) {
                const float a = Order<F>::value(last), c = Order<F>::value(next);
                // (without a bias scores are positive and their errors relative, 1.2 |x|
                // units of 2^-23 with |x| below 80 among them: below 2^-16)
                const float near = biased ? 2 * tol : a * 0x1p-14f;
                if ((!(a - c > near) || (!biased && !(a > 1e-30f))) &&
                    !kept_exactly<TYPE, VPT, VEC>(p, row, ept, *slots, m, z, g2, score, last, next, near,
                                                  tol, kept))
                    return false;
            }
        }
    }
    if (aligned) {
        const bool mine = (kept >> (lane / lanes)) & 1u;
#pragma unroll
        for (int i = 0; i < VPT; ++i) key[i] = mine ? key[i] : Key(0);
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i < ept && !((kept >> ((lane * ept + i) / size & 31)) & 1u)) key[i] = 0;
    }
    return true;
}

// The whole choice in 64 bits: rarely called, and much larger than the FP32 form.
template <int TYPE, int VPT, bool VEC>
__device__ __noinline__ int choose_exactly(const RouteProblem &p, const void *row, int ept) {
    float x[VPT], tol;
    load_row<TYPE, VPT, VEC>(p, row, ept, x);
    double m = 0, z = 0;
    if (p.score == kSoftmax) softmax_stats<double>(x, m, z);
    Order<double>::Key key[VPT];
    keys_of<double, TYPE, VPT, VEC>(p, row, static_cast<Slots<VPT> *>(nullptr), x, ept, m, z, key, tol);
    return in_rounds<double>(p, ept, key);
}

// The lane's candidate again in 64 bits: how many of the `total` come before it.
template <int TYPE, int VPT, bool VEC>
__device__ __noinline__ int place_exactly(const RouteProblem &p, const void *row, int ept, int total,
                                          int e, float x) {
    double m = 0, z = 0;
    if (p.score == kSoftmax) {
        float all[VPT];
        load_row<TYPE, VPT, VEC>(p, row, ept, all);
        softmax_stats<double>(all, m, z);
    }
    Order<double>::Key key = 0;
    if (e >= 0) key = Order<double>::of(score_of<double>(p, x, m, 1.0 / z) + __ldg(p.bias + e));
    int before = 0;
    for (int i = 0; i < total; ++i) {
        const Order<double>::Key o = __shfl_sync(kAll, key, i);
        const int n = __shfl_sync(kAll, e, i);
        before += o > key || (o == key && n < e) ? 1 : 0;
    }
    return before;
}

// What a lane knows of the choice: an expert (or -1), its logit and its place.
struct Choice {
    int expert, place;
    float logit;
};

// The token's choice in FP32; lanes below `width` may have one.  False where a
// decision is too close to call and not among 32 candidates.
template <int TYPE, int VPT, bool VEC>
__device__ __forceinline__ bool choose(const RouteProblem &p, const void *row, const float (&x)[VPT],
                                       int ept, float m, float z, Slots<VPT> &s, Choice &mine,
                                       int &width) {
    const int lane = threadIdx.x % 32;
    const bool biased = p.bias != nullptr;
    uint32_t key[VPT];
    float tol;
    if (!keys_of<float, TYPE, VPT, VEC>(p, row, &s, x, ept, m, z, key, tol)) return false;
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) best = max(best, key[i]);
#pragma unroll
    for (int i = 0; i < VPT; i += 4) {
        if constexpr (VPT >= 4)
            *reinterpret_cast<uint4 *>(s.key + lane * VPT + i) =
                make_uint4(key[i], key[i + 1], key[i + 2], key[i + 3]);
        else
            *reinterpret_cast<uint2 *>(s.key + lane * VPT) = make_uint2(key[0], key[1]);
    }
    uint32_t bound;
    if (p.k == 1) {
        bound = __reduce_max_sync(kAll, best);
    } else {
        s.best[lane] = best;
        __syncwarp();
        int as_large = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint4 o = reinterpret_cast<const uint4 *>(s.best)[q];
            as_large += (o.x >= best) + (o.y >= best) + (o.z >= best) + (o.w >= best);
        }
        bound = __reduce_max_sync(kAll, as_large >= p.k ? best : 0u);
    }
    // (a value that only seems smaller than the bound may be larger)
    if (biased && bound != 0) {
        const float low = Order<float>::value(bound) - tol;
        if (isnan(low)) return false;
        bound = Order<float>::of(low);
    }
    if (bound == 0) bound = 1;
    uint32_t mask = 0;  // this lane's candidates
#pragma unroll
    for (int i = 0; i < VPT; ++i) mask |= key[i] >= bound ? 1u << i : 0u;
    int total = 0;
    for (uint32_t who; (who = __ballot_sync(kAll, mask != 0)) != 0; mask &= mask - 1) {
        const int slot = total + __popc(who & ((1u << lane) - 1u));
        if (mask != 0 && slot < 32) s.at[slot] = static_cast<uint16_t>(lane * VPT + __ffs(mask) - 1);
        total += __popc(who);
        if (total > 32) break;
    }
    if (total > 32) {
        if (biased) return false;
        mine.expert = in_rounds<float>(p, ept, key);
        mine.place = lane;
        mine.logit = mine.expert >= 0 ? Value<TYPE>::load(row, mine.expert) : 0.f;
        width = 32;
        return true;
    }
    __syncwarp();
    // lane i: candidate i, and how many of the others come before it
    uint32_t k32 = 0, at = 0;
    if (lane < total) at = s.at[lane], k32 = s.key[at];
    const unsigned long long cand =
        lane < total ? static_cast<unsigned long long>(k32) << 32 | static_cast<uint32_t>(~at) : 0ull;
    s.candidate[lane] = cand;
    __syncwarp();
    int place = 0;
    for (int q = 0; q < total; q += 4) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(s.candidate + q);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(s.candidate + q + 2);
        place += (a.x > cand) + (a.y > cand) + (b.x > cand) + (b.y > cand);
    }
    const int e = lane < total ? static_cast<int>(at / VPT * ept + at % VPT) : -1;
    float l = Order<float>::value(k32);  // (without a bias a key is a logit)
    if (biased) {
        l = e >= 0 ? Value<TYPE>::load(row, e) : 0.f;
        if (e >= 0) s.best[place] = k32, s.number[place] = e, s.logit[place] = l;
        __syncwarp();
        // the candidates in order: too close to the next one, unless that has the
        // same logit and the same bias (equal for certain)?  (Also past the k-th: equal
        // ones may stand between it and one that is close.)
        bool close = false;
        if (lane + 1 < total &&
            !(Order<float>::value(s.best[lane]) - Order<float>::value(s.best[lane + 1]) > tol))
            close = !(s.logit[lane] == s.logit[lane + 1] &&
                      __ldg(p.bias + s.number[lane]) == __ldg(p.bias + s.number[lane + 1]));
        if (__any_sync(kAll, close)) place = place_exactly<TYPE, VPT, VEC>(p, row, ept, total, e, l);
    }
    mine.expert = e;
    mine.place = place;
    mine.logit = l;
    width = lanes_of(total);
    __syncwarp();
    return true;
}

// log of the logistic function, for scores that FP32 cannot hold
__device__ __forceinline__ float log_sigmoid(float x) {
    return fminf(x, 0.f) - log1pf(expf(-fabsf(x)));
}

// (of equal numbers 1, exactly: a single expert's share; the gradient through it is 0)
__device__ __forceinline__ float ratio(float a, float b) { return a == b ? 1.f : __fdividef(a, b); }

// The lane's share of the chosen experts' scores (lanes with `has`, all below
// `width`): s_j / sum s.  Scores too small for FP32 keep their ratios.
__device__ __forceinline__ float share(const RouteProblem &p, bool has, float x, int width) {
    if (p.score == kSoftmax) {
        const float m = warp_max(has ? x : -INFINITY, width);
        const float e = has ? expf(x - m) : 0.f;
        return ratio(e, warp_sum(e, width));
    }
    const float s = has ? __fdividef(1.f, 1.f + expf(-x)) : 0.f;
    const float sum = __shfl_sync(kAll, warp_sum(s, width), 0);
    if (sum < 1e-30f) {
        const float l = has ? log_sigmoid(x) : -INFINITY;
        const float m = warp_max(l, width);
        const float e = has ? expf(l - m) : 0.f;
        return ratio(e, warp_sum(e, width));
    }
    return ratio(s, sum);
}

// (Register limits: many warps per SM hide the latency of each; the spills are in the
// parts that run rarely.  Up to 256 experts 12 CTAs per SM: 16384 x 256 without a bias
// 11.7 us, with 8 CTAs 0.8 more; CTAs that stay and load the next token ahead 14.4.)
template <int TYPE, int VPT, bool VEC>
__global__ void __launch_bounds__(32 * kWarps, VPT <= 8 ? 12 : VPT <= 16 ? 5 : 3)
    route_kernel(const __grid_constant__ RouteProblem p) {
    __shared__ Slots<VPT> slots[kWarps];
    const int lane = threadIdx.x % 32;
    const int ept = VEC ? VPT : (p.experts + 31) / 32;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t t = blockIdx.x * int64_t(kWarps) + threadIdx.x / 32; t < p.tokens;
         t += gridDim.x * int64_t(kWarps)) {
        const void *row = static_cast<const uint8_t *>(p.logits) + t * p.ld * Value<TYPE>::BYTES;
        float x[VPT];
        load_row<TYPE, VPT, VEC>(p, row, ept, x);
        const bool sums = p.bias != nullptr || (p.groups > 1 && p.top == 2);
        float m = 0.f, z = 0.f;
        if (p.score == kSoftmax && (sums || !p.renorm)) softmax_stats<float>(x, m, z);
        Choice mine;
        int width;
        if (!choose<TYPE, VPT, VEC>(p, row, x, ept, m, z, slots[threadIdx.x / 32], mine, width)) {
            mine.expert = choose_exactly<TYPE, VPT, VEC>(p, row, ept);
            mine.place = lane;
            mine.logit = mine.expert >= 0 ? Value<TYPE>::load(row, mine.expert) : 0.f;
            width = 32;
        }
        const bool has = mine.expert >= 0 && mine.place < p.k;
        float w;
        if (p.renorm) {
            w = share(p, has, mine.logit, width);
            if (isnan(z)) w = z;  // (with a bias, other experts than the NaN may be chosen)
        } else if (p.score == kSigmoid) {
            w = __fdividef(1.f, 1.f + expf(-mine.logit));
        } else {
            w = __fdividef(expf(mine.logit - m), z);
        }
        int32_t *chosen = p.chosen + t * p.k;
        float *weights = p.weights + t * p.k;
        if (has) {
            chosen[mine.place] = mine.expert;
            weights[mine.place] = w * p.scale;
        }
        const int count = __popc(__ballot_sync(kAll, has));
        if (lane >= count && lane < p.k) {  // fewer than k can be chosen
            chosen[lane] = -1;
            weights[lane] = 0.f;
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
        // an expert named twice: its terms are added in the order of the names
        if (has) mine[e] = __int_as_float(lane);
        __syncwarp();
        const bool twice = __any_sync(kAll, has && __float_as_int(mine[e]) != lane);
        __syncwarp();
        const float dw = has ? p.dweights[t * p.k + lane] * p.scale : 0.f;
        float dx;
        if (p.renorm) {
            const float q = share(p, has, x, lanes_of(p.k));
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
        if (!twice) {
            if (has) mine[e] += dx;
        } else {
            for (int j = 0; j < p.k; ++j) {
                if (has && lane == j) mine[e] += dx;
                __syncwarp();
            }
        }
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
