// rms_norm.hip -- root-mean-square norm with the residual's addition, and its
// gradient:
//
//   s = x + residual      rstd = 1 / sqrt(mean(s^2) + eps)      y = s rstd weight
//   g = dy weight         dx = rstd (g - s rstd^2 mean(g s)) + dsum
//   dweight = sum over rows of dy s rstd
//
// y in x's type, or in e4m3 with a scale per row: scale = max|y| / 448, and
// y / scale rounded to the nearest e4m3.  Both passes are bound by memory:
// each tensor is read and written once, a row stays in registers between its
// sum and its output, and all sums are fp32.
//
// The gradient of 8192 x 4096 bf16 takes 50 us, a copy's rate, and joining the
// weight's partial sums 6 more.  2047 x 4096 with e4m3 outputs takes 16.8 us,
// 3.5 TB/s: a row's loads, its two sums over the workgroup and its stores follow
// one another, and all rows are on the chip at once.  Four waves a row are best
// there (one 18.7, two 18.3, eight 18.5).
#include <type_traits>

#include "norm_common.h"
#include "kernels.h"

namespace miconv {

namespace {

// One row per workgroup, NV vectors of eight columns per thread; past them
// (LOOP) the rest of a longer row is read a second time.
template <class T, bool E4M3, int WAVES, int NV, bool LOOP>
__global__ __launch_bounds__(64 * WAVES) void rms_norm_kernel(const NormArgs p)
{
    constexpr int THREADS = 64 * WAVES, SPAN = THREADS * 8;
    __shared__ float part[2][WAVES];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
    const T* weight = static_cast<const T*>(p.weight);
    const int c0 = threadIdx.x * 8;

    float s[NV][8], w[NV][8];
    float total = 0.0f;
    auto fetch = [&](int c, float (&v)[8]) {
        const int nv = p.cols - c;
        load8(x + c, nv, v);
        if (res) {
            float r[8];
            load8(res + c, nv, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r[i];
        }
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * SPAN;
        if (c < p.cols) {
            fetch(c, s[j]);
            load8(weight + c, p.cols - c, w[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[j][i] = w[j][i] = 0.0f;
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * SPAN;
        if (p.sum && c < p.cols) store8(static_cast<T*>(p.sum) + row * p.lds + c, p.cols - c, s[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) total += s[j][i] * s[j][i];
    }
    if constexpr (LOOP) {
        for (int c = c0 + NV * SPAN; c < p.cols; c += SPAN) {
            float v[8];
            fetch(c, v);
            if (p.sum) store8(static_cast<T*>(p.sum) + row * p.lds + c, p.cols - c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) total += v[i] * v[i];
        }
    }
    total = block_sum<WAVES>(total, part[0]);
    const float rstd = 1.0f / sqrtf(total / (float)p.cols + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;

    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[j][i] = s[j][i] * rstd * w[j][i];
            if constexpr (E4M3) most = fmaxf(most, fabsf(s[j][i]));
        }
    auto again = [&](int c, float (&v)[8]) {
        float g[8];
        fetch(c, v);
        load8(weight + c, p.cols - c, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * rstd * g[i];
    };
    float inv = 1.0f, shift = 1.0f;
    if constexpr (E4M3) {
        if constexpr (LOOP)
            for (int c = c0 + NV * SPAN; c < p.cols; c += SPAN) {
                float v[8];
                again(c, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i]));
            }
        most = block_max<WAVES>(most, part[1]);
        // a row of zeros (or one too small for a scale) keeps the scale 1
        const float scale = most / E4M3_MAX > 0.0f ? most / E4M3_MAX : 1.0f;
        shift = scale < 0x1p-100f ? 0x1p+64f : 1.0f;
        inv = 1.0f / (scale * shift);
        if (threadIdx.x == 0) p.scale[row] = scale;
    }
    auto put = [&](int c, const float (&v)[8]) {
        if constexpr (E4M3)
            store8_e4m3(static_cast<uint8_t*>(p.y) + row * p.ldy + c, p.cols - c, v, inv, shift);
        else
            store8(static_cast<T*>(p.y) + row * p.ldy + c, p.cols - c, v);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * SPAN;
        if (c < p.cols) put(c, s[j]);
    }
    if constexpr (LOOP)
        for (int c = c0 + NV * SPAN; c < p.cols; c += SPAN) {
            float v[8];
            again(c, v);
            put(c, v);
        }
}

// dx, and this workgroup's share of dweight, for rows blockIdx.x, + gridDim.x,
// ...  The share stays in registers until the last row (LOOP: rows too long
// for that get dweight from norm_weight_kernel).
template <class T, int WAVES, int NV, bool LOOP>
__global__ __launch_bounds__(64 * WAVES) void rms_norm_grad_kernel(const NormGradArgs p)
{
    constexpr int THREADS = 64 * WAVES, SPAN = THREADS * 8;
    __shared__ float part[2][WAVES];
    const T* weight = static_cast<const T*>(p.weight);
    const int c0 = threadIdx.x * 8;
    float w[NV][8], dw[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        load8(weight + c0 + j * SPAN, p.cols - c0 - j * SPAN, w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
        const T* sum = static_cast<const T*>(p.sum) + row * p.lds;
        const T* dsum = p.dsum ? static_cast<const T*>(p.dsum) + row * p.ldd : nullptr;
        T* dx = static_cast<T*>(p.dx) + row * p.lddx;
        const float rstd = p.rstd[row];
        float s[NV][8], g[NV][8], d[NV][8];
        float along = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN, nv = p.cols - c;
            load8(dy + c, nv, g[j]);
            load8(sum + c, nv, s[j]);
            if (dsum) load8(dsum + c, nv, d[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[j][i] += g[j][i] * s[j][i] * rstd;
                g[j][i] *= w[j][i];
                along += g[j][i] * s[j][i];
            }
        if constexpr (LOOP)
            for (int c = c0 + NV * SPAN; c < p.cols; c += SPAN) {
                float a[8], b[8], e[8];
                load8(dy + c, p.cols - c, a);
                load8(sum + c, p.cols - c, b);
                load8(weight + c, p.cols - c, e);
#pragma unroll
                for (int i = 0; i < 8; ++i) along += a[i] * e[i] * b[i];
            }
        // two parts in turn: a wave may start the next row's sum while another still reads this one's
        along = block_sum<WAVES>(along, part[turn]);
        const float k = along / (float)p.cols * rstd * rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g[j][i] = rstd * (g[j][i] - s[j][i] * k);
                if (dsum) g[j][i] += d[j][i];
            }
            if (c < p.cols) store8(dx + c, p.cols - c, g[j]);
        }
        if constexpr (LOOP)
            for (int c = c0 + NV * SPAN; c < p.cols; c += SPAN) {
                float a[8], b[8], e[8];
                load8(dy + c, p.cols - c, a);
                load8(sum + c, p.cols - c, b);
                load8(weight + c, p.cols - c, e);
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] = rstd * (a[i] * e[i] - b[i] * k);
                if (dsum) {
                    load8(dsum + c, p.cols - c, e);
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] += e[i];
                }
                store8(dx + c, p.cols - c, a);
            }
    }
    if constexpr (!LOOP) {
        if (!p.dweight) return;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN;
            if (c < p.cols) store8(p.partial + (int64_t)blockIdx.x * p.cols + c, p.cols - c, dw[j]);
        }
    }
}

// dweight's partial column sums on their own, for rows past the registers:
// a group walks its rows with one vector of eight columns a thread.
template <class T> __global__ __launch_bounds__(64) void norm_weight_kernel(const NormGradArgs p)
{
    const int c = (blockIdx.y * 64 + threadIdx.x) * 8, nv = p.cols - c;
    if (nv <= 0) return;
    float dw[8] = {};
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float a[8], b[8];
        load8(static_cast<const T*>(p.dy) + row * p.lddy + c, nv, a);
        load8(static_cast<const T*>(p.sum) + row * p.lds + c, nv, b);
        const float rstd = p.rstd[row];
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] += a[i] * b[i] * rstd;
    }
    store8(p.partial + (int64_t)blockIdx.x * p.cols + c, nv, dw);
}

// HIP takes grids of fewer than 2^32 threads; a workgroup per row of at most 512 threads reaches that at 2^23 rows.
constexpr int GRID_ROWS = 1 << 22;

template <class T, bool E4M3> hipError_t launch_rows(const NormArgs& p, hipStream_t stream)
{
    const int v = (p.cols + 7) / 8;                            // vectors in a row
    if (v <= 64) rms_norm_kernel<T, E4M3, 1, 1, false><<<p.rows, 64, 0, stream>>>(p);
    else if (v <= 256) rms_norm_kernel<T, E4M3, 4, 1, false><<<p.rows, 256, 0, stream>>>(p);
    else if (v <= 512) rms_norm_kernel<T, E4M3, 4, 2, false><<<p.rows, 256, 0, stream>>>(p);
    else if (v <= 1024) rms_norm_kernel<T, E4M3, 4, 4, false><<<p.rows, 256, 0, stream>>>(p);
    else rms_norm_kernel<T, E4M3, 8, 4, true><<<p.rows, 512, 0, stream>>>(p);
    return hipGetLastError();
}

template <class T, bool E4M3> hipError_t launch_type(const NormArgs& all, hipStream_t stream)
{
    using Out = typename std::conditional<E4M3, uint8_t, T>::type;
    for (int64_t first = 0; first < all.rows; first += GRID_ROWS) {
        NormArgs p = all;
        p.rows = (int)(all.rows - first < GRID_ROWS ? all.rows - first : GRID_ROWS);
        p.x = static_cast<const T*>(all.x) + first * all.ldx;
        if (p.residual) p.residual = static_cast<const T*>(all.residual) + first * all.ldr;
        p.y = static_cast<Out*>(all.y) + first * all.ldy;
        if (p.sum) p.sum = static_cast<T*>(all.sum) + first * all.lds;
        if (p.rstd) p.rstd = all.rstd + first;
        if (p.scale) p.scale = all.scale + first;
        const hipError_t err = launch_rows<T, E4M3>(p, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

constexpr int GRAD_MOST = 8192;    // columns whose dweight share a workgroup keeps in registers

template <class T> hipError_t launch_grad_type(const NormGradArgs& p, hipStream_t stream)
{
    const int v = (p.cols + 7) / 8;
    if (v <= 64) rms_norm_grad_kernel<T, 1, 1, false><<<p.groups, 64, 0, stream>>>(p);
    else if (v <= 256) rms_norm_grad_kernel<T, 4, 1, false><<<p.groups, 256, 0, stream>>>(p);
    else if (v <= 512) rms_norm_grad_kernel<T, 4, 2, false><<<p.groups, 256, 0, stream>>>(p);
    else if (p.cols <= GRAD_MOST) rms_norm_grad_kernel<T, 8, 2, false><<<p.groups, 512, 0, stream>>>(p);
    else {
        rms_norm_grad_kernel<T, 8, 2, true><<<p.groups, 512, 0, stream>>>(p);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess || !p.dweight) return err;
        norm_weight_kernel<T><<<dim3(p.groups, (v + 63) / 64), 64, 0, stream>>>(p);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(DType dt, bool e4m3, const NormArgs& p, hipStream_t stream)
{
    if (dt == DType::F32) return e4m3 ? launch_type<float, true>(p, stream) : launch_type<float, false>(p, stream);
    return e4m3 ? launch_type<Bf16, true>(p, stream) : launch_type<Bf16, false>(p, stream);
}

int rms_norm_grad_groups(int rows, int cols, int num_cu)
{
    const int per_cu = cols <= 512 ? 16 : cols <= 4096 ? 4 : 2;
    return rows < num_cu * per_cu ? (rows > 1 ? rows : 1) : num_cu * per_cu;
}

hipError_t launch_rms_norm_grad(DType dt, const NormGradArgs& p, hipStream_t stream)
{
    const hipError_t err = dt == DType::F32 ? launch_grad_type<float>(p, stream) : launch_grad_type<Bf16>(p, stream);
    if (err != hipSuccess || !p.dweight) return err;
    return launch_column_join(dt, p.partial, p.groups, p.cols, p.dweight, stream);
}

}  // namespace miconv
