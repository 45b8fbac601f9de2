// linear.cpp -- host side of the feed-forward operators: validation, the
// choice of kernel and tile, workspaces and launches.
#include <stdint.h>

#include <algorithm>

#include <hip/hip_runtime.h>

#include "miconv.h"
#include "handle.h"
#include "linear_common.h"
#include "kernels.h"

namespace {

using miconv::DType;
using miconv::Product;
using miconv::ProductArgs;
using miconv::ProductType;

constexpr int kMaxSize = 1 << 30;
constexpr int64_t kMaxPitchBytes = int64_t(1) << 23;   // 256 rows of a tile stay inside a 32-bit offset

size_t size_of(mic_dtype d) { return d == MIC_DTYPE_F32 ? 4 : d == MIC_DTYPE_BF16 ? 2 : 1; }
bool plain_type(mic_dtype d) { return d == MIC_DTYPE_F32 || d == MIC_DTYPE_BF16; }
DType device_type(mic_dtype d) { return d == MIC_DTYPE_F32 ? DType::F32 : DType::BF16; }
bool valid_act(mic_activation a) { return (int)a >= 0 && (int)a <= (int)MIC_ACT_SILU; }

// Host-only calls need no device: without a handle they plan for the MI355X.
int num_cus(mic_handle h) { return h ? h->num_cu : 256; }

int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mic_status check_sizes(int m, int n, int k)
{
    if (m < 0 || n < 0 || k < 0) return MIC_STATUS_BAD_PARAM;
    return m >= kMaxSize || n >= kMaxSize || k >= kMaxSize ? MIC_STATUS_NOT_SUPPORTED : MIC_STATUS_SUCCESS;
}

// One matrix of rows x cols elements of `size` bytes.
mic_status check_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, size_t size)
{
    if (rows == 0 || cols == 0) return MIC_STATUS_SUCCESS;
    if (!p || !aligned(p, size) || ld < cols) return MIC_STATUS_BAD_PARAM;
    return ld >= kMaxPitchBytes / (int64_t)size ? MIC_STATUS_NOT_SUPPORTED : MIC_STATUS_SUCCESS;
}

#define MIC_TRY(expr)                                            \
    do {                                                         \
        const mic_status status_ = (expr);                       \
        if (status_ != MIC_STATUS_SUCCESS) return status_;       \
    } while (0)

mic_status launched(hipError_t e) { return e == hipSuccess ? MIC_STATUS_SUCCESS : MIC_STATUS_LAUNCH_FAILED; }

// How a product runs.
struct Plan {
    int tile;
    int splits;
    int64_t part_ld;
    size_t bytes;            // workspace
};

Plan plan_product(int num_cu, Product kind, ProductType type, int m, int n, int k, int k_segments)
{
    Plan pl = {};
    const int raw_n = kind == Product::GATED ? miconv::gated_raw_columns(n) : n;
    auto tiles = [&](int t) { return (int64_t)((m + t - 1) / t) * ((raw_n + t - 1) / t); };
    pl.tile = tiles(128) >= num_cu / 2 ? 128 : 64;
    const int line = type == ProductType::F32 ? 32 : type == ProductType::BF16 ? 64 : 128;
    const int64_t steps = (int64_t)((k + line - 1) / line) * k_segments;
    const int64_t t = tiles(pl.tile);
    // a second wave of workgroups per CU hides the first one's loads; a part has at least eight steps
    pl.splits = (int)std::max<int64_t>(1, std::min<int64_t>(2 * num_cu / std::max<int64_t>(t, 1), steps / 8));
    pl.part_ld = align_up(raw_n, pl.tile);
    pl.bytes = pl.splits > 1 ? (size_t)pl.splits * m * pl.part_ld * 4 : 0;
    return pl;
}

mic_status run_product(mic_handle h, Product kind, ProductType type, ProductArgs& p, void* workspace, size_t bytes)
{
    if (p.M == 0 || p.N == 0) return MIC_STATUS_SUCCESS;
    const Plan pl = plan_product(num_cus(h), kind, type, p.M, p.N, p.K, p.k_segments);
    if (pl.bytes > bytes || (pl.bytes && (!workspace || !aligned(workspace, 16)))) return MIC_STATUS_BAD_PARAM;
    p.splits = pl.splits;
    p.part = static_cast<float*>(workspace);
    p.part_ld = pl.part_ld;
    hipError_t e = miconv::launch_product_any(kind, type, p, pl.tile, h->stream);
    if (e == hipSuccess && pl.splits > 1) e = miconv::launch_product_join(kind, type, p, h->stream);
    return launched(e);
}

mic_status product_type(mic_dtype in, mic_dtype out, ProductType* type, bool fast = false)
{
    if (in == MIC_DTYPE_F32 && out == MIC_DTYPE_F32) *type = ProductType::F32;
    else if (in == MIC_DTYPE_BF16 && out == MIC_DTYPE_BF16) *type = ProductType::BF16;
    else if (in == MIC_DTYPE_F8_E4M3 && out == MIC_DTYPE_BF16) *type = fast ? ProductType::E4M3_BF16_SHORT : ProductType::E4M3_BF16;
    else if (in == MIC_DTYPE_F8_E4M3 && out == MIC_DTYPE_F32) *type = fast ? ProductType::E4M3_F32_SHORT : ProductType::E4M3_F32;
    else return MIC_STATUS_NOT_SUPPORTED;
    return MIC_STATUS_SUCCESS;
}

mic_status forward_workspace(mic_handle h, Product kind, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    if (!bytes) return MIC_STATUS_BAD_PARAM;
    MIC_TRY(check_sizes(m, n, k));
    ProductType type;
    MIC_TRY(product_type(dtype, plain_type(dtype) ? dtype : MIC_DTYPE_BF16, &type));
    *bytes = m && n ? plan_product(num_cus(h), kind, type, m, n, k, 1).bytes : 0;
    return MIC_STATUS_SUCCESS;
}

// The backward workspace: dz, dbias's partial sums, the products' own.
struct GradLayout {
    int64_t pitch;           // of one layer's dz columns
    size_t dz, sums, product, total;
};

GradLayout grad_layout(mic_handle h, ProductType type, int m, int n, int k, bool gated, bool bias)
{
    GradLayout g = {};
    const int two = gated ? 2 : 1;
    g.pitch = align_up(n, 64);
    g.dz = (size_t)align_up((int64_t)m * g.pitch * two * (type == ProductType::F32 ? 4 : 2), 256);
    g.sums = bias ? (size_t)align_up((int64_t)miconv::slope_row_groups(m, n) * n * 4, 256) : 0;
    const size_t a = m && k ? plan_product(num_cus(h), Product::INPUT_GRAD, type, m, k, n, two).bytes : 0;
    const size_t b = n && k ? plan_product(num_cus(h), Product::WEIGHT_GRAD, type, (int)(gated ? 2 * g.pitch : n), k, m, 1).bytes : 0;
    g.product = std::max(a, b);
    g.total = g.dz + g.sums + g.product;
    return g;
}

mic_status backward_workspace(mic_handle h, mic_dtype dtype, int m, int n, int k, bool gated, size_t* bytes)
{
    if (!bytes) return MIC_STATUS_BAD_PARAM;
    MIC_TRY(check_sizes(m, n, k));
    if (!plain_type(dtype)) return MIC_STATUS_NOT_SUPPORTED;
    if (n >= kMaxSize / 2) return MIC_STATUS_NOT_SUPPORTED;
    ProductType type;
    MIC_TRY(product_type(dtype, dtype, &type));
    *bytes = grad_layout(h, type, m, n, k, gated, !gated).total;
    return MIC_STATUS_SUCCESS;
}

// dx = dz w (+ dz2 w2) and dw = dz^T x (dw2 = dz2^T x)
mic_status grad_products(mic_handle h, ProductType type, int m, int n, int k, const void* dz, int64_t dz_pitch,
                         int64_t up_at, const void* x, int64_t ldx, const void* w, int64_t ldw, const void* w2,
                         int64_t ldw2, void* dx, int64_t lddx, void* dw, int64_t lddw, void* dw2, int64_t lddw2,
                         void* workspace, size_t bytes)
{
    const int64_t e = type == ProductType::F32 ? 4 : 2;
    const bool gated = w2 != nullptr || dw2 != nullptr;
    if (dx) {
        ProductArgs p = {};
        p.a = static_cast<const uint8_t*>(dz), p.lda = dz_pitch * e;
        p.b = static_cast<const uint8_t*>(w), p.ldb = ldw * e;
        p.b2 = static_cast<const uint8_t*>(w2), p.ldb2 = ldw2 * e;
        p.M = m, p.N = k, p.K = n;
        p.k_segments = gated ? 2 : 1, p.k_pitch = (int)up_at;
        p.m_pitch = INT32_MAX, p.m_valid = m;
        p.y = dx, p.ldy = lddx;
        MIC_TRY(run_product(h, Product::INPUT_GRAD, type, p, workspace, bytes));
    }
    if (dw) {
        ProductArgs p = {};
        p.a = static_cast<const uint8_t*>(dz), p.lda = dz_pitch * e;
        p.b = static_cast<const uint8_t*>(x), p.ldb = ldx * e;
        p.M = gated ? (int)(2 * up_at) : n, p.N = k, p.K = m;
        p.k_segments = 1;
        p.m_pitch = gated ? (int)up_at : INT32_MAX, p.m_valid = n;
        p.y = dw, p.ldy = lddw;
        p.y2 = dw2, p.ldy2 = lddw2;
        MIC_TRY(run_product(h, Product::WEIGHT_GRAD, type, p, workspace, bytes));
    }
    return MIC_STATUS_SUCCESS;
}

}  // namespace

extern "C" {

mic_status mic_rms_norm(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, int rows, int cols, double eps,
                        const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                        void* y, int64_t ldy, void* sum, int64_t lds, float* rstd, float* scale)
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
    if (!weight || !aligned(weight, e) || !aligned(rstd, 4) || !aligned(scale, 4)) return MIC_STATUS_BAD_PARAM;
    if (e4m3 && !scale) return MIC_STATUS_BAD_PARAM;
    miconv::NormArgs p = {rows, cols, (float)eps, x, ldx, residual, ldr, weight, y, ldy, sum, lds, rstd, scale};
    return launched(miconv::launch_rms_norm(device_type(dtype), e4m3, p, handle->stream));
}

mic_status mic_rms_norm_backward_workspace(mic_handle handle, int rows, int cols, size_t* bytes)
{
    if (!bytes) return MIC_STATUS_BAD_PARAM;
    MIC_TRY(check_sizes(rows, cols, 0));
    *bytes = (size_t)miconv::rms_norm_grad_groups(rows, cols, num_cus(handle)) * cols * 4;
    return MIC_STATUS_SUCCESS;
}

mic_status mic_rms_norm_backward(mic_handle handle, mic_dtype dtype, int rows, int cols, const void* dy, int64_t lddy,
                                 const void* sum, int64_t lds, const void* weight, const float* rstd,
                                 const void* dsum, int64_t ldd, void* dx, int64_t lddx, void* dweight,
                                 void* workspace, size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    if (!plain_type(dtype)) return MIC_STATUS_NOT_SUPPORTED;
    size_t need;
    MIC_TRY(mic_rms_norm_backward_workspace(handle, rows, cols, &need));
    if (cols == 0) return rows == 0 ? MIC_STATUS_SUCCESS : MIC_STATUS_BAD_PARAM;
    const size_t e = size_of(dtype);
    MIC_TRY(check_matrix(dy, lddy, rows, cols, e));
    MIC_TRY(check_matrix(sum, lds, rows, cols, e));
    if (dsum) MIC_TRY(check_matrix(dsum, ldd, rows, cols, e));
    MIC_TRY(check_matrix(dx, lddx, rows, cols, e));
    if (!weight || !aligned(weight, e) || !aligned(dweight, e)) return MIC_STATUS_BAD_PARAM;
    if (rows && (!rstd || !aligned(rstd, 4))) return MIC_STATUS_BAD_PARAM;
    if (rows == 0 && !dweight) return MIC_STATUS_SUCCESS;
    if (dweight && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return MIC_STATUS_BAD_PARAM;
    miconv::NormGradArgs p = {rows, cols, dy, lddy, sum, lds, weight, rstd, dsum, ldd, dx, lddx, dweight,
                              static_cast<float*>(workspace),
                              miconv::rms_norm_grad_groups(rows, cols, num_cus(handle))};
    return launched(miconv::launch_rms_norm_grad(device_type(dtype), p, handle->stream));
}

mic_status mic_linear_forward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return forward_workspace(handle, Product::FORWARD, dtype, m, n, k, bytes);
}

mic_status mic_linear_forward(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, mic_activation act,
                              int fast_sums, int m, int n, int k, const void* x, int64_t ldx, const void* w, int64_t ldw,
                              const float* x_scale, const float* w_scale, const void* bias, const void* residual,
                              int64_t ldr, void* y, int64_t ldy, void* preact, int64_t ldp, void* workspace,
                              size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    ProductType type;
    MIC_TRY(product_type(dtype, out_dtype, &type, fast_sums != 0));
    if (!valid_act(act)) return MIC_STATUS_NOT_SUPPORTED;
    MIC_TRY(check_sizes(m, n, k));
    if (m == 0 || n == 0) return MIC_STATUS_SUCCESS;
    const size_t e = size_of(dtype), o = size_of(out_dtype);
    MIC_TRY(check_matrix(x, ldx, m, k, e));
    MIC_TRY(check_matrix(w, ldw, n, k, e));
    MIC_TRY(check_matrix(y, ldy, m, n, o));
    if (residual) MIC_TRY(check_matrix(residual, ldr, m, n, o));
    if (preact) MIC_TRY(check_matrix(preact, ldp, m, n, o));
    if (!aligned(bias, o) || !aligned(x_scale, 4) || !aligned(w_scale, 4)) return MIC_STATUS_BAD_PARAM;
    const bool scaled = dtype == MIC_DTYPE_F8_E4M3;
    if (scaled != (x_scale != nullptr) || scaled != (w_scale != nullptr)) return MIC_STATUS_BAD_PARAM;
    ProductArgs p = {};
    p.a = static_cast<const uint8_t*>(x), p.lda = ldx * (int64_t)e;
    p.b = static_cast<const uint8_t*>(w), p.ldb = ldw * (int64_t)e;
    p.M = m, p.N = n, p.K = k, p.k_segments = 1;
    p.act = act;
    p.y = y, p.ldy = ldy;
    p.bias = bias, p.residual = residual, p.ldr = ldr;
    p.x_scale = x_scale, p.w_scale = w_scale;
    p.pre = preact, p.ldp = ldp;
    return run_product(handle, Product::FORWARD, type, p, workspace, workspace_bytes);
}

mic_status mic_linear_backward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return backward_workspace(handle, dtype, m, n, k, false, bytes);
}

mic_status mic_linear_backward(mic_handle handle, mic_dtype dtype, mic_activation act, int m, int n, int k,
                               const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                               const void* preact, int64_t ldp, void* dx, int64_t lddx, void* dw, int64_t lddw,
                               void* dbias, void* workspace, size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    size_t need;
    MIC_TRY(backward_workspace(handle, dtype, m, n, k, false, &need));
    if (!valid_act(act)) return MIC_STATUS_NOT_SUPPORTED;
    const size_t e = size_of(dtype);
    const bool slope = act != MIC_ACT_NONE;
    MIC_TRY(check_matrix(dy, lddy, m, n, e));
    if (slope) MIC_TRY(check_matrix(preact, ldp, m, n, e));
    if (dw) MIC_TRY(check_matrix(x, ldx, m, k, e));
    if (dx) MIC_TRY(check_matrix(w, ldw, n, k, e));
    if (dx) MIC_TRY(check_matrix(dx, lddx, m, k, e));
    if (dw) MIC_TRY(check_matrix(dw, lddw, n, k, e));
    if (!aligned(dbias, e)) return MIC_STATUS_BAD_PARAM;
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return MIC_STATUS_BAD_PARAM;
    if (n == 0 && (!dx || k == 0)) return MIC_STATUS_SUCCESS;
    ProductType type;
    MIC_TRY(product_type(dtype, dtype, &type));
    const GradLayout g = grad_layout(handle, type, m, n, k, false, true);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    // without an activation dz is dy, read where it is
    const bool own = slope && (dx || dw);
    if (n && (own || dbias)) {
        miconv::SlopeArgs s = {};
        s.rows = m, s.cols = n, s.act = act;
        s.dy = dy, s.lddy = lddy;
        s.pre = slope ? preact : nullptr, s.ldp = ldp;
        s.dz = own && m ? ws : nullptr, s.dz_pitch = g.pitch, s.up_at = g.pitch;
        s.sums = dbias ? reinterpret_cast<float*>(ws + g.dz) : nullptr;
        s.dbias = dbias;
        MIC_TRY(launched(miconv::launch_slope(device_type(dtype), s, handle->stream)));
    }
    return grad_products(handle, type, m, n, k, own ? ws : dy, own ? g.pitch : lddy, 0, x, ldx, w, ldw, nullptr, 0,
                         dx, lddx, dw, lddw, nullptr, 0, ws + g.dz + g.sums, g.product);
}

mic_status mic_gated_linear_forward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes)
{
    return forward_workspace(handle, Product::GATED, dtype, m, n, k, bytes);
}

mic_status mic_gated_linear_forward(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, mic_activation act,
                                    int fast_sums, int m, int n, int k, const void* x, int64_t ldx, const void* w_gate,
                                    int64_t ldg, const void* w_up, int64_t ldu, const float* x_scale,
                                    const float* w_gate_scale, const float* w_up_scale, void* y, int64_t ldy,
                                    void* gate, int64_t ldgate, void* up, int64_t ldup, void* workspace,
                                    size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    ProductType type;
    MIC_TRY(product_type(dtype, out_dtype, &type, fast_sums != 0));
    if (!valid_act(act)) return MIC_STATUS_NOT_SUPPORTED;
    MIC_TRY(check_sizes(m, n, k));
    if (n >= kMaxSize / 2) return MIC_STATUS_NOT_SUPPORTED;
    if (m == 0 || n == 0) return MIC_STATUS_SUCCESS;
    const size_t e = size_of(dtype), o = size_of(out_dtype);
    MIC_TRY(check_matrix(x, ldx, m, k, e));
    MIC_TRY(check_matrix(w_gate, ldg, n, k, e));
    MIC_TRY(check_matrix(w_up, ldu, n, k, e));
    MIC_TRY(check_matrix(y, ldy, m, n, o));
    if ((gate == nullptr) != (up == nullptr)) return MIC_STATUS_BAD_PARAM;
    if (gate) {
        MIC_TRY(check_matrix(gate, ldgate, m, n, o));
        MIC_TRY(check_matrix(up, ldup, m, n, o));
    }
    const bool scaled = dtype == MIC_DTYPE_F8_E4M3;
    if (scaled != (x_scale != nullptr) || scaled != (w_gate_scale != nullptr) || scaled != (w_up_scale != nullptr))
        return MIC_STATUS_BAD_PARAM;
    if (!aligned(x_scale, 4) || !aligned(w_gate_scale, 4) || !aligned(w_up_scale, 4)) return MIC_STATUS_BAD_PARAM;
    ProductArgs p = {};
    p.a = static_cast<const uint8_t*>(x), p.lda = ldx * (int64_t)e;
    p.b = static_cast<const uint8_t*>(w_gate), p.ldb = ldg * (int64_t)e;
    p.b2 = static_cast<const uint8_t*>(w_up), p.ldb2 = ldu * (int64_t)e;
    p.M = m, p.N = n, p.K = k, p.k_segments = 1;
    p.act = act;
    p.y = y, p.ldy = ldy;
    p.x_scale = x_scale, p.w_scale = w_gate_scale, p.w2_scale = w_up_scale;
    p.pre = gate, p.ldp = ldgate;
    p.pre2 = up, p.ldp2 = ldup;
    return run_product(handle, Product::GATED, type, p, workspace, workspace_bytes);
}

mic_status mic_gated_linear_backward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k,
                                               size_t* bytes)
{
    return backward_workspace(handle, dtype, m, n, k, true, bytes);
}

mic_status mic_gated_linear_backward(mic_handle handle, mic_dtype dtype, mic_activation act, int m, int n, int k,
                                     const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w_gate,
                                     int64_t ldg, const void* w_up, int64_t ldu, const void* gate, int64_t ldgate,
                                     const void* up, int64_t ldup, void* dx, int64_t lddx, void* dw_gate,
                                     int64_t lddg, void* dw_up, int64_t lddu, void* workspace,
                                     size_t workspace_bytes)
{
    if (!handle) return MIC_STATUS_BAD_PARAM;
    size_t need;
    MIC_TRY(backward_workspace(handle, dtype, m, n, k, true, &need));
    if (!valid_act(act)) return MIC_STATUS_NOT_SUPPORTED;
    const size_t e = size_of(dtype);
    MIC_TRY(check_matrix(dy, lddy, m, n, e));
    MIC_TRY(check_matrix(gate, ldgate, m, n, e));
    MIC_TRY(check_matrix(up, ldup, m, n, e));
    if ((dw_gate == nullptr) != (dw_up == nullptr)) return MIC_STATUS_BAD_PARAM;
    if (dw_gate) {
        MIC_TRY(check_matrix(x, ldx, m, k, e));
        MIC_TRY(check_matrix(dw_gate, lddg, n, k, e));
        MIC_TRY(check_matrix(dw_up, lddu, n, k, e));
    }
    if (dx) {
        MIC_TRY(check_matrix(w_gate, ldg, n, k, e));
        MIC_TRY(check_matrix(w_up, ldu, n, k, e));
        MIC_TRY(check_matrix(dx, lddx, m, k, e));
    }
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return MIC_STATUS_BAD_PARAM;
    if ((!dx && !dw_gate) || k == 0) return MIC_STATUS_SUCCESS;
    ProductType type;
    MIC_TRY(product_type(dtype, dtype, &type));
    const GradLayout g = grad_layout(handle, type, m, n, k, true, false);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (m && n) {
        miconv::SlopeArgs s = {};
        s.rows = m, s.cols = n, s.act = act;
        s.dy = dy, s.lddy = lddy;
        s.pre = gate, s.ldp = ldgate;
        s.up = up, s.ldu = ldup;
        s.dz = ws, s.dz_pitch = 2 * g.pitch, s.up_at = g.pitch;
        MIC_TRY(launched(miconv::launch_slope(device_type(dtype), s, handle->stream)));
    }
    // n == 0: dx is a sum of nothing, and the weights are never read
    const void* w2 = w_up ? w_up : ws;
    return grad_products(handle, type, m, n, k, ws, 2 * g.pitch, g.pitch, x, ldx, w_gate, ldg, w2, ldu, dx, lddx,
                         dw_gate, lddg, dw_up, lddu, ws + g.dz + g.sums, g.product);
}

}  // extern "C"
