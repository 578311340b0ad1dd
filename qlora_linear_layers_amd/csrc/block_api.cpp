// extern "C" entry points declared in include/qlora_block.h: host-side
// validation and kernel sequencing.
#include <cmath>
#include <initializer_list>

#include "qlora_block.h"
#include "int8.hpp"
#include "rows.hpp"

static_assert(QLORA_ROWS8_PITCH(1) == ql::kRows8Pitch, "pitch of the header and the kernels");

namespace {

int dev(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_DEVICE; }

int check_aligned(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return QLORA_ERR_ALIGN;
    return QLORA_OK;
}

int check_rows(int64_t R, int64_t K, int64_t longest) {
    return R < 1 || R > QLORA_ROWS_MAX || K < 1 || K > longest ? QLORA_ERR_SHAPE : QLORA_OK;
}

int quantize_impl(const uint16_t* x, int64_t R, int64_t K, int8_t* codes, float* scale, void* stream, bool f16) {
    if (!x || !codes || !scale) return QLORA_ERR_NULL;
    if (int st = check_rows(R, K, QLORA_ROWS8_MAX)) return st;
    if (int st = check_aligned({x, codes, scale})) return st;
    return dev(ql::launch_rows8_quantize(x, R, K, codes, scale, static_cast<hipStream_t>(stream), f16));
}

int dequantize_impl(const int8_t* codes, const float* scale, int64_t R, int64_t K, uint16_t* out, void* stream,
                    bool f16) {
    if (!codes || !scale || !out) return QLORA_ERR_NULL;
    if (int st = check_rows(R, K, QLORA_ROWS8_MAX)) return st;
    if (int st = check_aligned({codes, scale, out})) return st;
    return dev(ql::launch_rows8_dequantize(codes, scale, R, K, out, static_cast<hipStream_t>(stream), f16));
}

int check_norm(const void* weight, int weight_f32, float eps) {
    if (!std::isfinite(eps) || !(eps > 0.0f)) return QLORA_ERR_VALUE;
    return weight_f32 != 0 && (weight_f32 != 1 || !weight) ? QLORA_ERR_VALUE : QLORA_OK;
}

int norm_impl(const uint16_t* x, const uint16_t* residual, int64_t T, int64_t D, const void* weight, int weight_f32,
              float eps, uint16_t* h, uint16_t* y, int8_t* y_codes, float* y_scale, void* stream, bool f16) {
    if (!x || !y_codes != !y_scale || (!y && !y_codes)) return QLORA_ERR_NULL;
    if (int st = check_rows(T, D, QLORA_NORM_MAX)) return st;
    if (int st = check_aligned({x, residual, weight, h, y, y_codes, y_scale})) return st;
    if (int st = check_norm(weight, weight_f32, eps)) return st;
    const ql::NormArgs a{x, residual, weight, h, y, y_codes, y_scale, T, (int)D, weight_f32, eps};
    return dev(ql::launch_rmsnorm(a, static_cast<hipStream_t>(stream), f16));
}

int norm_bwd_impl(const uint16_t* dy, const uint16_t* h, int64_t T, int64_t D, const void* weight, int weight_f32,
                  float eps, const uint16_t* dx_add, uint16_t* dx, void* d_weight, void* workspace,
                  size_t workspace_bytes, void* stream, bool f16) {
    if (!dy || !h || !dx || (d_weight && !weight)) return QLORA_ERR_NULL;
    if (int st = check_rows(T, D, QLORA_NORM_MAX)) return st;
    if (int st = check_aligned({dy, h, weight, dx_add, dx, d_weight, workspace})) return st;
    if (int st = check_norm(weight, weight_f32, eps)) return st;
    if (d_weight && (!workspace || workspace_bytes < rmsnorm_workspace_bytes_bwd(T, D))) return QLORA_ERR_WORKSPACE;
    const ql::NormBwd a{dy, h, weight, dx_add, dx, d_weight, static_cast<float*>(workspace), T, (int)D, weight_f32, eps};
    return dev(ql::launch_rmsnorm_bwd(a, static_cast<hipStream_t>(stream), f16));
}

int check_int8_shape(int64_t T, int64_t K, int64_t N) {
    if (T < 1 || K < 1 || N < 1 || T > QLORA_ROWS_MAX || N > (int64_t(1) << 20) || K > QLORA_ROWS8_MAX)
        return QLORA_ERR_SHAPE;
    return T * K > (int64_t(1) << 30) || T * N > (int64_t(1) << 30) ? QLORA_ERR_SHAPE : QLORA_OK;
}

int int8_impl(const int8_t* x_codes, const float* x_scale, int64_t T, int64_t K, int64_t N, const int8_t* w_codes,
              const float* w_scale, const qlora_epilogue* e, uint16_t* y, void* workspace, size_t workspace_bytes,
              void* stream, bool f16) {
    if (!x_codes || !x_scale || !w_codes || !w_scale || !e || !y) return QLORA_ERR_NULL;
    if (int st = check_int8_shape(T, K, N)) return st;
    if (int st = check_aligned({x_codes, x_scale, w_codes, w_scale, e->bias, e->mul, e->residual, y, workspace}))
        return st;
    if (e->act < 0 || e->act >= ql::kActs || e->z || e->z_codes || e->z_scale) return QLORA_ERR_VALUE;
    const size_t need = ql::int8_workspace(T, K, N);
    if (need && (!workspace || workspace_bytes < need)) return QLORA_ERR_WORKSPACE;
    const ql::Int8Args a{x_codes, x_scale, w_codes, w_scale, y,
                         ql::Epilogue{e->act, e->bias, e->mul, e->residual, nullptr, nullptr, nullptr}, T, N,
                         (int)ql::rows8_pitch(K), 1, nullptr};
    return dev(ql::launch_int8(a, K, workspace, static_cast<hipStream_t>(stream), f16));
}

}  // namespace

extern "C" {

int rows8_quantize(const uint16_t* x, int64_t R, int64_t K, int8_t* codes, float* scale, void* stream) {
    return quantize_impl(x, R, K, codes, scale, stream, false);
}

int rows8_quantize_f16(const uint16_t* x, int64_t R, int64_t K, int8_t* codes, float* scale, void* stream) {
    return quantize_impl(x, R, K, codes, scale, stream, true);
}

int rows8_dequantize(const int8_t* codes, const float* scale, int64_t R, int64_t K, uint16_t* x_out, void* stream) {
    return dequantize_impl(codes, scale, R, K, x_out, stream, false);
}

int rows8_dequantize_f16(const int8_t* codes, const float* scale, int64_t R, int64_t K, uint16_t* x_out,
                         void* stream) {
    return dequantize_impl(codes, scale, R, K, x_out, stream, true);
}

int rmsnorm_fwd(const uint16_t* x, const uint16_t* residual, int64_t T, int64_t D, const void* weight,
                int weight_f32, float eps, uint16_t* h, uint16_t* y, int8_t* y_codes, float* y_scale, void* stream) {
    return norm_impl(x, residual, T, D, weight, weight_f32, eps, h, y, y_codes, y_scale, stream, false);
}

int rmsnorm_fwd_f16(const uint16_t* x, const uint16_t* residual, int64_t T, int64_t D, const void* weight,
                    int weight_f32, float eps, uint16_t* h, uint16_t* y, int8_t* y_codes, float* y_scale,
                    void* stream) {
    return norm_impl(x, residual, T, D, weight, weight_f32, eps, h, y, y_codes, y_scale, stream, true);
}

int rmsnorm_bwd(const uint16_t* dy, const uint16_t* h, int64_t T, int64_t D, const void* weight, int weight_f32,
                float eps, const uint16_t* dx_add, uint16_t* dx, void* d_weight, void* workspace,
                size_t workspace_bytes, void* stream) {
    return norm_bwd_impl(dy, h, T, D, weight, weight_f32, eps, dx_add, dx, d_weight, workspace, workspace_bytes,
                         stream, false);
}

int rmsnorm_bwd_f16(const uint16_t* dy, const uint16_t* h, int64_t T, int64_t D, const void* weight, int weight_f32,
                    float eps, const uint16_t* dx_add, uint16_t* dx, void* d_weight, void* workspace,
                    size_t workspace_bytes, void* stream) {
    return norm_bwd_impl(dy, h, T, D, weight, weight_f32, eps, dx_add, dx, d_weight, workspace, workspace_bytes,
                         stream, true);
}

size_t rmsnorm_workspace_bytes_bwd(int64_t T, int64_t D) {
    if (check_rows(T, D, QLORA_NORM_MAX) != QLORA_OK) return 0;
    return ql::align256((size_t)ql::rmsnorm_bwd_partials(T, D) * D * 4);
}

int int8_linear_fwd(const int8_t* x_codes, const float* x_scale, int64_t T, int64_t K, int64_t N,
                    const int8_t* w_codes, const float* w_scale, const qlora_epilogue* epilogue, uint16_t* y,
                    void* workspace, size_t workspace_bytes, void* stream) {
    return int8_impl(x_codes, x_scale, T, K, N, w_codes, w_scale, epilogue, y, workspace, workspace_bytes, stream,
                     false);
}

int int8_linear_fwd_f16(const int8_t* x_codes, const float* x_scale, int64_t T, int64_t K, int64_t N,
                        const int8_t* w_codes, const float* w_scale, const qlora_epilogue* epilogue, uint16_t* y,
                        void* workspace, size_t workspace_bytes, void* stream) {
    return int8_impl(x_codes, x_scale, T, K, N, w_codes, w_scale, epilogue, y, workspace, workspace_bytes, stream,
                     true);
}

size_t int8_linear_workspace_bytes(int64_t T, int64_t K, int64_t N) {
    if (check_int8_shape(T, K, N) != QLORA_OK) return 0;
    return ql::int8_workspace(T, K, N);
}

}  // extern "C"
