// layers.cpp -- host side of layer norm and dropout: validation and launches.
#include <cmath>

#include "host_checks.h"
#include "kernels.h"

using namespace miconv;

extern "C" {

mic_status mic_layer_norm(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, int rows, int cols, double eps,
                          const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                          const void* bias, void* y, int64_t ldy, void* sum, int64_t lds, float* mean, float* rstd,
                          float* scale)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    if (!plain_type(dtype) || (out_dtype != dtype && out_dtype != MIC_DTYPE_F8_E4M3)) return MIC_STATUS_NOT_SUPPORTED;
    MIC_TRY(check_sizes(rows, cols, 0));
    if (!(eps >= 0.0)) return MIC_STATUS_BAD_PARAM;
    if (rows == 0) return MIC_STATUS_SUCCESS;
    if (cols == 0) return MIC_STATUS_BAD_PARAM;                // the mean of nothing
    const size_t e = size_of(dtype);
    const bool e4m3 = out_dtype == MIC_DTYPE_F8_E4M3;
    MIC_TRY(check_matrix(x, ldx, rows, cols, e));
    if (residual) MIC_TRY(check_matrix(residual, ldr, rows, cols, e));
    if (sum) MIC_TRY(check_matrix(sum, lds, rows, cols, e));
    MIC_TRY(check_matrix(y, ldy, rows, cols, size_of(out_dtype)));
    if (!weight || !aligned(weight, e) || !aligned(bias, e)) return MIC_STATUS_BAD_PARAM;
    if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(scale, 4)) return MIC_STATUS_BAD_PARAM;
    if (e4m3 && !scale) return MIC_STATUS_BAD_PARAM;
    const LayerNormArgs p = {rows, cols, (float)eps, x, ldx, residual, ldr, weight, bias, y, ldy, sum, lds, mean, rstd, scale,
                             handle->num_cu};
    return launched(launch_layer_norm(device_type(dtype), e4m3, p, handle->stream));
}

mic_status mic_layer_norm_backward_workspace(mic_handle handle, int rows, int cols, size_t* bytes)
{
    if (!bytes) return MIC_STATUS_BAD_PARAM;
    MIC_TRY(check_sizes(rows, cols, 0));
    *bytes = most_bytes(handle, [&](int cus) { return (size_t)layer_norm_grad_groups(rows, cols, cus) * cols * 8; });
    return MIC_STATUS_SUCCESS;
}

mic_status mic_layer_norm_backward(mic_handle handle, mic_dtype dtype, int rows, int cols, const void* dy, int64_t lddy,
                                   const void* sum, int64_t lds, const void* weight, const float* mean,
                                   const float* rstd, const void* dsum, int64_t ldd, void* dx, int64_t lddx,
                                   void* dweight, void* dbias, void* workspace, size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    if (!plain_type(dtype)) return MIC_STATUS_NOT_SUPPORTED;
    size_t need;
    MIC_TRY(mic_layer_norm_backward_workspace(handle, rows, cols, &need));
    if (cols == 0) return rows == 0 ? MIC_STATUS_SUCCESS : MIC_STATUS_BAD_PARAM;
    // a vector of 2^30 columns has no rows to be checked
    if (cols >= kMaxPitchBytes / (int64_t)size_of(dtype)) return MIC_STATUS_NOT_SUPPORTED;
    const size_t e = size_of(dtype);
    MIC_TRY(check_matrix(dy, lddy, rows, cols, e));
    MIC_TRY(check_matrix(sum, lds, rows, cols, e));
    if (dsum) MIC_TRY(check_matrix(dsum, ldd, rows, cols, e));
    MIC_TRY(check_matrix(dx, lddx, rows, cols, e));
    if (!weight || !aligned(weight, e) || !aligned(dweight, e) || !aligned(dbias, e)) return MIC_STATUS_BAD_PARAM;
    if (rows && (!mean || !aligned(mean, 4) || !rstd || !aligned(rstd, 4))) return MIC_STATUS_BAD_PARAM;
    const bool sums = dweight || dbias;
    if (rows == 0 && !sums) return MIC_STATUS_SUCCESS;
    if (sums && need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return MIC_STATUS_BAD_PARAM;
    const LayerNormGradArgs p = {rows, cols, dy, lddy, sum, lds, weight, mean, rstd, dsum, ldd, dx, lddx, dweight, dbias,
                                 static_cast<float*>(workspace), layer_norm_grad_groups(rows, cols, handle->num_cu), handle->num_cu};
    return launched(launch_layer_norm_grad(device_type(dtype), p, handle->stream));
}

mic_status mic_dropout(mic_handle handle, mic_dtype dtype, int64_t rows, int64_t cols, double p, uint64_t seed,
                       uint64_t offset, const uint64_t* state, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                       void* y, int64_t ldy)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    if (!plain_type(dtype)) return MIC_STATUS_NOT_SUPPORTED;
    if (rows < 0 || cols < 0 || !(p >= 0.0 && p <= 1.0)) return MIC_STATUS_BAD_PARAM;
    if (rows == 0 || cols == 0) return MIC_STATUS_SUCCESS;
    constexpr int64_t most = int64_t(1) << 40;
    if (rows >= most || cols >= most || rows > most / cols) return MIC_STATUS_NOT_SUPPORTED;
    const size_t e = size_of(dtype);
    auto matrix = [&](const void* m, int64_t ld) {
        return m && aligned(m, e) && ld >= cols ? ld >= most / rows && rows > 1 ? MIC_STATUS_NOT_SUPPORTED : MIC_STATUS_SUCCESS
                                                : MIC_STATUS_BAD_PARAM;
    };
    MIC_TRY(matrix(x, ldx));
    if (residual) MIC_TRY(matrix(residual, ldr));
    MIC_TRY(matrix(y, ldy));
    if (!aligned(state, 8)) return MIC_STATUS_BAD_PARAM;
    const uint32_t least = (uint32_t)std::nearbyint(p * 65536.0);
    DropoutArgs a = {rows, cols, seed, offset, state, least, least < 65536 ? (float)(65536.0 / (65536.0 - least)) : 0.0f,
                     x, ldx, residual, ldr, y, ldy};
    if (ldx == cols && ldy == cols && (!residual || ldr == cols)) a.rows = 1, a.cols = rows * cols;
    return launched(launch_dropout(device_type(dtype), a, handle->stream));
}

}  // extern "C"
