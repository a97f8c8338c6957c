// fused_api.cu -- the C ABI of the fused products (include/gemm.h): argument
// checks and dispatch.  Every rule is checked before any CUDA call.
#include <cuda_runtime.h>

#include <cstdint>

#include "call.h"
#include "fused.h"
#include "gemm.h"

#define GEMM_API extern "C" __attribute__((visibility("default")))

using gemm::InType;

namespace {

constexpr int64_t kMaxDim = 0x7fffffff;
// Pitches are at most 2^40 elements, more than any device holds.
constexpr int64_t kMaxPitch = int64_t(1) << 40;

bool dim_ok(int64_t v) { return v >= 0 && v <= kMaxDim; }
bool is_order(gemm_order_t o) { return o == GEMM_ROW_MAJOR || o == GEMM_COL_MAJOR; }
bool usable(const void *p, uintptr_t bytes) {
    return p != nullptr && reinterpret_cast<uintptr_t>(p) % bytes == 0;
}
uintptr_t in_bytes(InType in) { return in == InType::F32 ? 4 : 2; }

bool operand_ok(const void *p, InType in, int64_t rows, int64_t cols, int64_t ld, gemm_order_t o) {
    const int64_t need = o == GEMM_ROW_MAJOR ? cols : rows;
    return usable(p, in_bytes(in)) && ld >= need && ld <= kMaxPitch;
}
bool rows_ok(const void *p, InType in, int64_t N, int64_t ld) {
    return usable(p, in_bytes(in)) && ld >= N && ld <= kMaxPitch;
}
bool act_ok(gemm_activation_t a) {
    return a == GEMM_ACT_NONE || a == GEMM_ACT_RELU || a == GEMM_ACT_GELU || a == GEMM_ACT_SILU;
}

// The problem but for what follows the product; GEMM_OK with p->N == 0: nothing to do.
gemm_status_t product(InType in, int64_t M, int64_t N, int64_t K, float alpha, const void *A,
                      int64_t lda, gemm_order_t order_a, const void *B, int64_t ldb,
                      gemm_order_t order_b, void *D, int64_t ldd, gemm::FusedProblem *p) {
    if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K) || !is_order(order_a) || !is_order(order_b))
        return GEMM_ERR_INVALID_VALUE;
    // (no device holds a larger D; tile numbers are 32-bit on that assumption)
    if (M > 0 && N > (int64_t(1) << 43) / M) return GEMM_ERR_INVALID_VALUE;
    *p = {};
    if (M == 0 || N == 0) return GEMM_OK;
    if (!rows_ok(D, in, N, ldd)) return GEMM_ERR_INVALID_VALUE;
    const bool sums = K > 0 && alpha != 0.f;
    if (sums && (!operand_ok(A, in, M, K, lda, order_a) || !operand_ok(B, in, K, N, ldb, order_b) ||
                 D == A || D == B))
        return GEMM_ERR_INVALID_VALUE;
    p->M = M;
    p->N = N;
    p->K = sums ? K : 0;
    p->alpha = sums ? alpha : 1.f;
    p->A = A;
    p->lda = lda;
    p->a_kmajor = order_a == GEMM_ROW_MAJOR;
    p->B = B;
    p->ldb = ldb;
    p->b_kmajor = order_b == GEMM_COL_MAJOR;
    p->D = D;
    p->ldd = ldd;
    return GEMM_OK;
}

gemm_status_t run(const gemm::FusedProblem &p, InType in, cudaStream_t stream) {
    const char *name = "";
    // up to four rows: the CUDA cores stream B (fused_rows) where its columns are contiguous
    const bool tc = in != InType::F32 && gemm::fused_tc_eligible(p) && !gemm::fused_rows_eligible(p, in);
    return gemm::finish_call(tc ? gemm::launch_fused_tc(p, in, stream, &name)
                                : gemm::launch_fused_simt(p, in, stream, &name),
                             name);
}

gemm_status_t fused(InType in, int64_t M, int64_t N, int64_t K, float alpha, const void *A,
                    int64_t lda, gemm_order_t order_a, const void *B, int64_t ldb,
                    gemm_order_t order_b, void *D, int64_t ldd, const gemm_fusion_t *fusion,
                    cudaStream_t stream) {
    gemm::set_last_kernel("");
    const gemm_fusion_t f = fusion != nullptr ? *fusion : gemm_fusion_t{};
    if (!act_ok(f.activation)) return GEMM_ERR_INVALID_VALUE;
    gemm::FusedProblem p;
    const gemm_status_t st =
        product(in, M, N, K, alpha, A, lda, order_a, B, ldb, order_b, D, ldd, &p);
    if (st != GEMM_OK || p.N == 0) return st;
    if ((f.bias != nullptr && !usable(f.bias, 4)) ||
        (f.residual != nullptr && (!rows_ok(f.residual, in, N, f.ld_residual) ||
                                   (f.residual == D && f.ld_residual != ldd))) ||
        (f.pre != nullptr && (!rows_ok(f.pre, in, N, f.ld_pre) || f.pre == D || f.pre == f.residual ||
                              (p.K > 0 && (f.pre == A || f.pre == B)))))
        return GEMM_ERR_INVALID_VALUE;
    const gemm_status_t dev = gemm::check_device_status();
    if (dev != GEMM_OK) return dev;
    p.bias = f.bias;
    p.act = static_cast<int>(f.activation);
    p.residual = f.residual;
    p.ld_r = f.ld_residual;
    p.pre = f.pre;
    p.ld_pre = f.ld_pre;
    return run(p, in, stream);
}

gemm_status_t fused_grad(InType in, int64_t M, int64_t N, int64_t K, float alpha, const void *A,
                         int64_t lda, gemm_order_t order_a, const void *B, int64_t ldb,
                         gemm_order_t order_b, gemm_activation_t activation, const void *pre,
                         int64_t ld_pre, void *D, int64_t ldd, float *dbias, cudaStream_t stream) {
    gemm::set_last_kernel("");
    if (!act_ok(activation) || (dbias != nullptr && !usable(dbias, 4)))
        return GEMM_ERR_INVALID_VALUE;
    gemm::FusedProblem p;
    const gemm_status_t st =
        product(in, M, N, K, alpha, A, lda, order_a, B, ldb, order_b, D, ldd, &p);
    if (st != GEMM_OK || N == 0) return st;
    if (M == 0 && dbias == nullptr) return GEMM_OK;
    if (M > 0 && activation != GEMM_ACT_NONE && (!rows_ok(pre, in, N, ld_pre) || (pre == D && ld_pre != ldd)))
        return GEMM_ERR_INVALID_VALUE;
    if (dbias != nullptr && (dbias == D || dbias == pre || dbias == A || dbias == B))
        return GEMM_ERR_INVALID_VALUE;
    const gemm_status_t dev = gemm::check_device_status();
    if (dev != GEMM_OK) return dev;
    if (M == 0)  // no rows: the sums are empty
        return gemm::finish_call(cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * 4, stream), "");
    p.act = static_cast<int>(activation);
    p.pre = activation != GEMM_ACT_NONE ? const_cast<void *>(pre) : nullptr;
    p.ld_pre = ld_pre;
    p.grad = true;
    p.dbias = dbias;
    return run(p, in, stream);
}

}  // namespace

#define FUSED(name, T, in)                                                                      \
    GEMM_API gemm_status_t gemm_fused_##name(                                                   \
        int64_t M, int64_t N, int64_t K, float alpha, const T *A, int64_t lda,                  \
        gemm_order_t order_a, const T *B, int64_t ldb, gemm_order_t order_b, T *D, int64_t ldd, \
        const gemm_fusion_t *fusion, cudaStream_t stream) {                                     \
        return fused(in, M, N, K, alpha, A, lda, order_a, B, ldb, order_b, D, ldd, fusion,      \
                     stream);                                                                   \
    }                                                                                           \
    GEMM_API gemm_status_t gemm_fused_grad_##name(                                              \
        int64_t M, int64_t N, int64_t K, float alpha, const T *A, int64_t lda,                  \
        gemm_order_t order_a, const T *B, int64_t ldb, gemm_order_t order_b,                    \
        gemm_activation_t activation, const T *pre, int64_t ld_pre, T *D, int64_t ldd,          \
        float *dbias, cudaStream_t stream) {                                                    \
        return fused_grad(in, M, N, K, alpha, A, lda, order_a, B, ldb, order_b, activation,     \
                          pre, ld_pre, D, ldd, dbias, stream);                                  \
    }

FUSED(f32, float, InType::F32)
FUSED(bf16_f32acc, gemm_bf16_t, InType::BF16)
FUSED(f16_f32acc, gemm_f16_t, InType::F16)
