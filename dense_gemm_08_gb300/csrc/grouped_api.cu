// grouped_api.cu -- the C ABI of the grouped operators (include/gemm.h):
// argument checks and dispatch.  Every rule is checked before any CUDA call.
#include <cuda_runtime.h>

#include <cstdint>

#include "call.h"
#include "gemm.h"
#include "grouped.h"
#include "internal.h"

#define GEMM_API extern "C" __attribute__((visibility("default")))

using gemm::InType;

namespace {

constexpr int64_t kMaxDim = 0x7fffffff;
// Strides are at most 2^40 elements, more than any device holds.
constexpr int64_t kMaxStride = int64_t(1) << 40;

// The row products walk the groups 32 at a time to find a tile's (GroupWalk): 2^24
// of them take 0.3 s, and 32-bit group numbers keep room for a step past the last.
constexpr int64_t kMaxGroups = int64_t(1) << 24;

bool dim_ok(int64_t v) { return v >= 0 && v <= kMaxDim; }
bool is_order(gemm_order_t o) { return o == GEMM_ROW_MAJOR || o == GEMM_COL_MAJOR; }
int64_t at_least_1(int64_t v) { return v > 1 ? v : 1; }

template <typename T>
bool usable(const T *p, size_t bytes) {
    return p != nullptr && reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

size_t in_bytes(InType in) { return in == InType::F32 ? 4 : 2; }

bool out_ok(InType in, gemm_d_type_t d) {
    return d == GEMM_D_F32 || (d == GEMM_D_BF16 && in == InType::BF16) ||
           (d == GEMM_D_F16 && in == InType::F16);
}

size_t out_bytes(gemm_d_type_t d) { return d == GEMM_D_F32 ? 4 : 2; }

// A stack of `count` rows x cols matrices in `order` is addressable.
bool stack_ok(const void *p, InType in, int64_t rows, int64_t cols, int64_t ld, gemm_order_t order,
              int64_t stride, int64_t count) {
    if (!usable(p, in_bytes(in))) return false;
    if (ld < at_least_1(order == GEMM_ROW_MAJOR ? cols : rows)) return false;
    return stride >= 0 && (count <= 1 || stride <= kMaxStride);
}

// The epilogue of the row products; NULL: FP32 D and nothing else.
bool epilogue_ok(const gemm_epilogue_t *e, InType in, gemm_epilogue_t *out) {
    *out = gemm_epilogue_t{nullptr, GEMM_ACT_NONE, GEMM_D_F32};
    if (e != nullptr) *out = *e;
    if (out->activation != GEMM_ACT_NONE && out->activation != GEMM_ACT_RELU &&
        out->activation != GEMM_ACT_GELU)
        return false;
    if (out->bias != nullptr && !usable(out->bias, sizeof(float))) return false;
    return out_ok(in, out->d_type);
}

gemm_status_t grouped(InType in, int64_t groups, int64_t rows, int64_t N, int64_t K, float alpha,
                      const void *A, int64_t lda, int64_t rows_a, const int32_t *row_index,
                      const int32_t *offsets, const void *B, int64_t ldb, int64_t stride_b,
                      gemm_order_t order_b, void *D, int64_t ldd, const gemm_epilogue_t *epilogue,
                      cudaStream_t stream) {
    gemm::set_last_kernel("");
    gemm_epilogue_t ep;
    if (!dim_ok(groups) || groups > kMaxGroups || !dim_ok(rows) || !dim_ok(N) || !dim_ok(K) ||
        !is_order(order_b) || !epilogue_ok(epilogue, in, &ep))
        return GEMM_ERR_INVALID_VALUE;
    if (groups == 0 || rows == 0 || N == 0) return GEMM_OK;
    if (!usable(offsets, 4) || !usable(D, out_bytes(ep.d_type)) || ldd < N)
        return GEMM_ERR_INVALID_VALUE;
    if (K > 0 && alpha != 0.f) {
        if ((!usable(A, in_bytes(in)) && rows_a != 0) || lda < K || !dim_ok(rows_a) ||
            (row_index == nullptr ? rows_a < rows : !usable(row_index, 4)) ||
            !stack_ok(B, in, K, N, ldb, order_b, stride_b, groups))
            return GEMM_ERR_INVALID_VALUE;
    }
    const gemm_status_t dev = gemm::check_device_status();
    if (dev != GEMM_OK) return dev;
    gemm::GroupedProblem p;
    p.groups = groups;
    p.rows = rows;
    p.N = N;
    p.K = alpha == 0.f ? 0 : K;  // nothing of A and B is read
    p.alpha = alpha;
    p.A = A;
    p.lda = lda;
    p.rows_a = rows_a;
    p.row_index = p.K > 0 ? row_index : nullptr;
    p.offsets = offsets;
    p.B = B;
    p.ldb = ldb;
    p.stride_b = stride_b;
    p.b_kmajor = order_b == GEMM_COL_MAJOR;
    p.D = D;
    p.ldd = ldd;
    p.bias = ep.bias;
    p.act = static_cast<int>(ep.activation);
    p.out = static_cast<int>(ep.d_type);
    const char *name = "";
    const bool tc = in != InType::F32 && gemm::grouped_tc_eligible(p);
    return gemm::finish_call(tc ? gemm::launch_grouped_tc(p, in, stream, &name)
                                : gemm::launch_grouped_simt(p, in, stream, &name),
                             name);
}

gemm_status_t wgrad(InType in, int64_t groups, int64_t rows, int64_t M, int64_t N, float alpha,
                    const void *A, int64_t lda, int64_t rows_a, const int32_t *row_index,
                    const int32_t *offsets, const void *B, int64_t ldb, float beta, const float *C,
                    int64_t ldc, int64_t stride_c, void *D, int64_t ldd, int64_t stride_d,
                    gemm_d_type_t d_type, cudaStream_t stream) {
    gemm::set_last_kernel("");
    if (!dim_ok(groups) || !dim_ok(rows) || !dim_ok(M) || !dim_ok(N) || !out_ok(in, d_type))
        return GEMM_ERR_INVALID_VALUE;
    if (groups == 0 || M == 0 || N == 0) return GEMM_OK;
    if (!usable(offsets, 4) || !usable(D, out_bytes(d_type)) || ldd < N ||
        (groups > 1 && (stride_d < 1 || stride_d > kMaxStride)))
        return GEMM_ERR_INVALID_VALUE;
    if (beta != 0.f && (!usable(C, 4) || ldc < N || stride_c < 0 || stride_c > kMaxStride))
        return GEMM_ERR_INVALID_VALUE;
    if (rows > 0 && alpha != 0.f) {
        if ((!usable(A, in_bytes(in)) && rows_a != 0) || !usable(B, in_bytes(in)) || lda < M ||
            ldb < N || !dim_ok(rows_a) || (row_index == nullptr ? rows_a < rows : !usable(row_index, 4)))
            return GEMM_ERR_INVALID_VALUE;
    }
    const gemm_status_t dev = gemm::check_device_status();
    if (dev != GEMM_OK) return dev;
    gemm::WgradProblem p;
    p.groups = groups;
    p.rows = alpha == 0.f ? 0 : rows;  // every group without rows: beta * C
    p.M = M;
    p.N = N;
    p.alpha = alpha;
    p.beta = beta;
    p.A = A;
    p.lda = lda;
    p.rows_a = rows_a;
    p.row_index = row_index;
    p.offsets = offsets;
    p.B = B;
    p.ldb = ldb;
    p.C = C;
    p.ldc = ldc;
    p.stride_c = stride_c;
    p.D = D;
    p.ldd = ldd;
    p.stride_d = stride_d;
    p.out = static_cast<int>(d_type);
    const char *name = "";
    const bool tc = in != InType::F32 && gemm::wgrad_tc_eligible(p);
    return gemm::finish_call(tc ? gemm::launch_wgrad_tc(p, in, stream, &name)
                                : gemm::launch_wgrad_simt(p, in, stream, &name),
                             name);
}

gemm_status_t lora(InType in, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                   const void *W, int64_t ldw, gemm_order_t order_w, int64_t adapters,
                   int64_t rank, const int32_t *adapter_of_row, const float *scale, const void *LA,
                   int64_t ld_a, int64_t stride_a, gemm_order_t order_a, const void *LB,
                   int64_t ld_b, int64_t stride_b, gemm_order_t order_b, void *D, int64_t ldd,
                   const gemm_epilogue_t *epilogue, cudaStream_t stream) {
    gemm::set_last_kernel("");
    gemm_epilogue_t ep;
    if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K) || !dim_ok(adapters) || !dim_ok(rank) ||
        !is_order(order_w) || !is_order(order_a) || !is_order(order_b) ||
        !epilogue_ok(epilogue, in, &ep))
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return GEMM_OK;
    if (!usable(D, out_bytes(ep.d_type)) || ldd < N) return GEMM_ERR_INVALID_VALUE;
    const bool any = adapters > 0 && rank > 0 && K > 0;
    if (K > 0) {
        if (!usable(X, in_bytes(in)) || ldx < K || !stack_ok(W, in, K, N, ldw, order_w, 0, 1))
            return GEMM_ERR_INVALID_VALUE;
    }
    if (any) {
        if (!usable(adapter_of_row, 4) || (scale != nullptr && !usable(scale, 4)) ||
            !stack_ok(LA, in, K, rank, ld_a, order_a, stride_a, adapters) ||
            !stack_ok(LB, in, rank, N, ld_b, order_b, stride_b, adapters))
            return GEMM_ERR_INVALID_VALUE;
    }
    const gemm_status_t dev = gemm::check_device_status();
    if (dev != GEMM_OK) return dev;
    gemm::LoraProblem p;
    p.M = M;
    p.N = N;
    p.K = K;
    p.adapters = any ? adapters : 0;
    p.rank = any ? rank : 0;
    p.X = X;
    p.ldx = ldx;
    p.W = W;
    p.ldw = ldw;
    p.w_kmajor = order_w == GEMM_COL_MAJOR;
    p.adapter = adapter_of_row;
    p.scale = scale;
    p.LA = LA;
    p.ld_a = ld_a;
    p.stride_a = stride_a;
    p.a_kmajor = order_a == GEMM_COL_MAJOR;
    p.LB = LB;
    p.ld_b = ld_b;
    p.stride_b = stride_b;
    p.b_kmajor = order_b == GEMM_COL_MAJOR;
    p.D = D;
    p.ldd = ldd;
    p.bias = ep.bias;
    p.act = static_cast<int>(ep.activation);
    p.out = static_cast<int>(ep.d_type);
    const char *name = "";
    return gemm::finish_call(gemm::lora_tc_eligible(p) ? gemm::launch_lora_tc(p, in, stream, &name)
                                                       : gemm::launch_lora_simt(p, in, stream, &name),
                             name);
}

}  // namespace

GEMM_API gemm_status_t gemm_group_rows(int64_t rows, int64_t groups, const int32_t *group_of_row,
                                       int32_t *offsets, int32_t *order, int32_t *position,
                                       cudaStream_t stream) {
    gemm::set_last_kernel("");
    if (!dim_ok(rows) || !dim_ok(groups) || groups < 1 || !usable(offsets, 4))
        return GEMM_ERR_INVALID_VALUE;
    if (rows > 0 && (!usable(group_of_row, 4) || !usable(order, 4) ||
                     (position != nullptr && !usable(position, 4))))
        return GEMM_ERR_INVALID_VALUE;
    const gemm_status_t dev = gemm::check_device_status();
    if (dev != GEMM_OK) return dev;
    const char *name = "";
    return gemm::finish_call(gemm::launch_group_rows(rows, groups, group_of_row, offsets, order,
                                                     position, stream, &name),
                             name);
}

#define GROUPED_ENTRY(suffix, type, in)                                                            \
    GEMM_API gemm_status_t gemm_grouped_##suffix(                                                  \
        int64_t groups, int64_t rows, int64_t N, int64_t K, float alpha, const type *A,            \
        int64_t lda, int64_t rows_a, const int32_t *row_index, const int32_t *offsets,             \
        const type *B, int64_t ldb, int64_t stride_b, gemm_order_t order_b, void *D, int64_t ldd,  \
        const gemm_epilogue_t *epilogue, cudaStream_t stream) {                                    \
        return grouped(in, groups, rows, N, K, alpha, A, lda, rows_a, row_index, offsets, B, ldb,  \
                       stride_b, order_b, D, ldd, epilogue, stream);                               \
    }                                                                                              \
    GEMM_API gemm_status_t gemm_grouped_wgrad_##suffix(                                            \
        int64_t groups, int64_t rows, int64_t M, int64_t N, float alpha, const type *A,            \
        int64_t lda, int64_t rows_a, const int32_t *row_index, const int32_t *offsets,             \
        const type *B, int64_t ldb, float beta, const float *C, int64_t ldc, int64_t stride_c,     \
        void *D, int64_t ldd, int64_t stride_d, gemm_d_type_t d_type, cudaStream_t stream) {       \
        return wgrad(in, groups, rows, M, N, alpha, A, lda, rows_a, row_index, offsets, B, ldb,    \
                     beta, C, ldc, stride_c, D, ldd, stride_d, d_type, stream);                    \
    }

GROUPED_ENTRY(f32, float, InType::F32)
GROUPED_ENTRY(bf16_f32acc, gemm_bf16_t, InType::BF16)
GROUPED_ENTRY(f16_f32acc, gemm_f16_t, InType::F16)

#define LORA_ENTRY(suffix, type, in)                                                               \
    GEMM_API gemm_status_t gemm_lora_##suffix(                                                     \
        int64_t M, int64_t N, int64_t K, const type *X, int64_t ldx, const type *W, int64_t ldw,   \
        gemm_order_t order_w, int64_t adapters, int64_t rank, const int32_t *adapter_of_row,       \
        const float *scale, const type *LA, int64_t ld_a, int64_t stride_a, gemm_order_t order_a,  \
        const type *LB, int64_t ld_b, int64_t stride_b, gemm_order_t order_b, void *D,             \
        int64_t ldd, const gemm_epilogue_t *epilogue, cudaStream_t stream) {                       \
        return lora(in, M, N, K, X, ldx, W, ldw, order_w, adapters, rank, adapter_of_row, scale,   \
                    LA, ld_a, stride_a, order_a, LB, ld_b, stride_b, order_b, D, ldd, epilogue,    \
                    stream);                                                                       \
    }

LORA_ENTRY(bf16_f32acc, gemm_bf16_t, InType::BF16)
LORA_ENTRY(f16_f32acc, gemm_f16_t, InType::F16)
