// mixture_api.cu -- the C ABI of the router and the combination (include/gemm.h):
// argument checks and dispatch.  Every rule is checked before any CUDA call.
#include <cuda_runtime.h>

#include <cstdint>

#include "call.h"
#include "gemm.h"
#include "mixture.h"

#define GEMM_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t kMaxDim = 0x7fffffff;
constexpr int64_t kMaxPairs = int64_t(1) << 40;  // tokens * k
// Pitches are at most 2^40 elements, more than any device holds.
constexpr int64_t kMaxPitch = int64_t(1) << 40;

bool dim_ok(int64_t v) { return v >= 0 && v <= kMaxDim; }
bool is_type(gemm_d_type_t t) {
    return t == GEMM_D_F32 || t == GEMM_D_BF16 || t == GEMM_D_F16;
}
uintptr_t type_bytes(gemm_d_type_t t) { return t == GEMM_D_F32 ? 4 : 2; }

bool usable(const void *p, uintptr_t bytes) {
    return p != nullptr && reinterpret_cast<uintptr_t>(p) % bytes == 0;
}
bool matrix_ok(const void *p, int64_t cols, int64_t ld, gemm_d_type_t t) {
    return usable(p, type_bytes(t)) && ld >= cols && ld <= kMaxPitch;
}

// The parts of a rule that both directions read.
bool rule_ok(const gemm_route_rule_t *r, gemm::RouteProblem *p) {
    p->score = gemm::kSoftmax;
    p->renorm = 1;
    p->scale = 1.f;
    p->groups = p->kept = p->top = 1;
    if (r == nullptr) return true;
    if ((r->score != GEMM_SCORE_SOFTMAX && r->score != GEMM_SCORE_SIGMOID) ||
        (r->renormalize != 0 && r->renormalize != 1))
        return false;
    p->score = r->score == GEMM_SCORE_SIGMOID ? gemm::kSigmoid : gemm::kSoftmax;
    p->renorm = r->renormalize;
    p->scale = r->scale;
    return true;
}

bool route_sizes_ok(int64_t tokens, int64_t experts, int64_t k) {
    return dim_ok(tokens) && experts >= 1 && experts <= gemm::kMaxExperts && k >= 1 && k <= experts &&
           k <= gemm::kMaxChoices;
}

}  // namespace

GEMM_API gemm_status_t gemm_route(int64_t tokens, int64_t experts, int64_t k, const void *logits,
                                  int64_t ld, gemm_d_type_t type, const gemm_route_rule_t *rule,
                                  int32_t *chosen, float *weights, cudaStream_t stream) {
    gemm::set_last_kernel("");
    gemm::RouteProblem p = {};
    if (!route_sizes_ok(tokens, experts, k) || !is_type(type) || !rule_ok(rule, &p))
        return GEMM_ERR_INVALID_VALUE;
    if (rule != nullptr) {
        if (rule->bias != nullptr && !usable(rule->bias, 4)) return GEMM_ERR_INVALID_VALUE;
        p.bias = rule->bias;
        if (rule->groups < 1 || rule->groups > gemm::kMaxExpertGroups || experts % rule->groups != 0)
            return GEMM_ERR_INVALID_VALUE;
        if (rule->groups > 1) {
            if (rule->groups_kept < 1 || rule->groups_kept > rule->groups ||
                (rule->group_top != 1 && rule->group_top != 2))
                return GEMM_ERR_INVALID_VALUE;
            p.groups = rule->groups;
            p.kept = rule->groups_kept;
            p.top = rule->group_top;
        }
    }
    if (tokens == 0) return GEMM_OK;
    if (!matrix_ok(logits, experts, ld, type) || !usable(chosen, 4) || !usable(weights, 4))
        return GEMM_ERR_INVALID_VALUE;
    const gemm_status_t dev = gemm::check_device_status();
    if (dev != GEMM_OK) return dev;
    p.tokens = tokens;
    p.experts = static_cast<int>(experts);
    p.k = static_cast<int>(k);
    p.logits = logits;
    p.ld = ld;
    p.type = static_cast<int>(type);
    p.chosen = chosen;
    p.weights = weights;
    const char *name = "";
    return gemm::finish_call(gemm::launch_route(p, stream, &name), name);
}

GEMM_API gemm_status_t gemm_route_grad(int64_t tokens, int64_t experts, int64_t k,
                                       const void *logits, int64_t ld, gemm_d_type_t type,
                                       const gemm_route_rule_t *rule, const int32_t *chosen,
                                       const float *dweights, void *dlogits, int64_t ld_d,
                                       cudaStream_t stream) {
    gemm::set_last_kernel("");
    gemm::RouteProblem p = {};
    if (!route_sizes_ok(tokens, experts, k) || !is_type(type) || !rule_ok(rule, &p))
        return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0) return GEMM_OK;
    if (!matrix_ok(logits, experts, ld, type) || !matrix_ok(dlogits, experts, ld_d, type) ||
        !usable(chosen, 4) || !usable(dweights, 4) || (logits == dlogits && ld != ld_d))
        return GEMM_ERR_INVALID_VALUE;
    const gemm_status_t dev = gemm::check_device_status();
    if (dev != GEMM_OK) return dev;
    p.tokens = tokens;
    p.experts = static_cast<int>(experts);
    p.k = static_cast<int>(k);
    p.logits = logits;
    p.ld = ld;
    p.type = static_cast<int>(type);
    p.chosen = const_cast<int32_t *>(chosen);
    p.dweights = dweights;
    p.dlogits = dlogits;
    p.ld_d = ld_d;
    const char *name = "";
    return gemm::finish_call(gemm::launch_route_grad(p, stream, &name), name);
}

namespace {

// What both directions share; false: refused.
bool combine_sizes_ok(int64_t tokens, int64_t k, int64_t N, int64_t rows_y, gemm_d_type_t y_type,
                      gemm_d_type_t d_type) {
    return dim_ok(tokens) && dim_ok(k) && dim_ok(N) && dim_ok(rows_y) && is_type(y_type) &&
           (d_type == GEMM_D_F32 || d_type == y_type) && tokens * k <= kMaxPairs;
}

}  // namespace

GEMM_API gemm_status_t gemm_combine(int64_t tokens, int64_t k, int64_t N, const void *Y,
                                    int64_t ldy, int64_t rows_y, gemm_d_type_t y_type,
                                    const int32_t *position, const float *weights,
                                    const void *residual, int64_t ld_r, void *D, int64_t ldd,
                                    gemm_d_type_t d_type, cudaStream_t stream) {
    gemm::set_last_kernel("");
    if (!combine_sizes_ok(tokens, k, N, rows_y, y_type, d_type)) return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0 || N == 0) return GEMM_OK;
    if (!matrix_ok(D, N, ldd, d_type) ||
        (residual != nullptr && !matrix_ok(residual, N, ld_r, d_type)) ||
        (k > 0 && !usable(position, 4)) ||
        (weights != nullptr && !usable(weights, 4)) ||
        (k > 0 && rows_y > 0 && (!matrix_ok(Y, N, ldy, y_type) || Y == D)) ||
        (residual == D && ld_r != ldd))
        return GEMM_ERR_INVALID_VALUE;
    const gemm_status_t dev = gemm::check_device_status();
    if (dev != GEMM_OK) return dev;
    gemm::CombineProblem p = {};
    p.tokens = tokens;
    p.k = k;
    p.N = N;
    p.Y = Y;
    p.ldy = ldy;
    p.rows_y = rows_y;
    p.y_type = static_cast<int>(y_type);
    p.position = position;
    p.weights = weights;
    p.residual = residual;
    p.ld_r = ld_r;
    p.D = D;
    p.ldd = ldd;
    p.d_type = static_cast<int>(d_type);
    const char *name = "";
    return gemm::finish_call(gemm::launch_combine(p, stream, &name), name);
}

GEMM_API gemm_status_t gemm_combine_grad(int64_t tokens, int64_t k, int64_t N, const void *dD,
                                         int64_t ld_d, gemm_d_type_t d_type, const void *Y,
                                         int64_t ldy, int64_t rows_y, gemm_d_type_t y_type,
                                         const int32_t *position, const float *weights, void *dY,
                                         int64_t ld_dy, float *dweights, cudaStream_t stream) {
    gemm::set_last_kernel("");
    if (!combine_sizes_ok(tokens, k, N, rows_y, y_type, d_type) || k < 1)
        return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0 || (dY == nullptr && dweights == nullptr)) return GEMM_OK;
    if (N == 0 && dweights == nullptr) return GEMM_OK;
    if ((N > 0 && !matrix_ok(dD, N, ld_d, d_type)) || !usable(position, 4) ||
        (weights != nullptr && !usable(weights, 4)) ||
        (dweights != nullptr && !usable(dweights, 4)) ||
        (N > 0 && rows_y > 0 && dweights != nullptr && !matrix_ok(Y, N, ldy, y_type)) ||
        (N > 0 && rows_y > 0 && dY != nullptr && (!matrix_ok(dY, N, ld_dy, y_type) || dY == dD)) ||
        (dY != nullptr && dY == Y) || (dweights != nullptr && dweights == weights))
        return GEMM_ERR_INVALID_VALUE;
    const gemm_status_t dev = gemm::check_device_status();
    if (dev != GEMM_OK) return dev;
    gemm::CombineProblem p = {};
    p.tokens = tokens;
    p.k = k;
    p.N = N;
    p.Y = Y;
    p.ldy = ldy;
    p.rows_y = rows_y;
    p.y_type = static_cast<int>(y_type);
    p.position = position;
    p.weights = weights;
    p.D = const_cast<void *>(dD);
    p.ldd = ld_d;
    p.d_type = static_cast<int>(d_type);
    p.dY = dY;
    p.ld_dy = ld_dy;
    p.dweights = dweights;
    const char *name = "";
    return gemm::finish_call(gemm::launch_combine_grad(p, stream, &name), name);
}
