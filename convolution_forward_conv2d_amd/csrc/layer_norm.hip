// layer_norm.hip -- layer norm with the residual's addition, and its gradient:
//
//   s = x + residual    mean = sum(s) / n    rstd = 1 / sqrt(sum((s - mean)^2) / n + eps)
//   y = (s - mean) rstd weight + bias
//   u = (s - mean) rstd    g = dy weight
//   dx = rstd (g - mean(g) - u mean(g u)) + dsum
//   dweight = sum over rows of dy u    dbias = sum over rows of dy
//
// y in x's type, or in e4m3 with a scale per row as the root-mean-square norm's.
// Both passes are bound by memory: each tensor is read and written once, a row
// stays in registers between its sums and its output, and all sums are fp32.
//
// The variance is a sum of squared distances, never a difference of sums: each
// wave takes its own values' mean and their squared distances from it, and the
// waves' means and squares are put together by
//   sum (s - mean)^2 = sum over waves of (squares_w + n_w (mean_w - mean)^2),
// so one exchange through LDS gives both, and a row far from zero keeps its
// variance.
#include <type_traits>

#include "norm_common.h"
#include "kernels.h"

namespace miconv {

namespace {

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Two sums over a workgroup in one exchange.
template <int WAVES> __device__ __forceinline__ void block_sums(float& a, float& b, float (*part)[2])
{
    a = wave_sum(a), b = wave_sum(b);
    if constexpr (WAVES == 1) return;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave][0] = a, part[wave][1] = b;
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) a += part[w][0], b += part[w][1];
}

// One row per workgroup, NV vectors of eight columns per thread; past them
// (LOOP) the rest of a longer row is read again in every pass.
template <class T, bool E4M3, int WAVES, int NV, bool LOOP>
__global__ __launch_bounds__(64 * WAVES) void layer_norm_kernel(const LayerNormArgs p)
{
    constexpr int THREADS = 64 * WAVES, SPAN = THREADS * 8;
    __shared__ float part[3][WAVES][2];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
    const T* weight = static_cast<const T*>(p.weight);
    const T* bias = static_cast<const T*>(p.bias);
    const int c0 = threadIdx.x * 8;

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
    auto factors = [&](int c, float (&w)[8], float (&b)[8]) {
        load8(weight + c, p.cols - c, w);
        if (bias) load8(bias + c, p.cols - c, b);
        else {
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = 0.0f;
        }
    };
    float s[NV][8], w[NV][8], b[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * SPAN;
        if (c < p.cols) {
            fetch(c, s[j]);
            factors(c, w[j], b[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[j][i] = w[j][i] = b[j][i] = 0.0f;
        }
    }
    float total = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * SPAN;
        if (p.sum && c < p.cols) store8(static_cast<T*>(p.sum) + row * p.lds + c, p.cols - c, s[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) total += s[j][i];
    }
    auto squares = [&](float from) {
        float q = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float apart = c0 + j * SPAN + i < p.cols ? s[j][i] - from : 0.0f;
                q += apart * apart;
            }
        return q;
    };
    float mean, spread;
    if constexpr (LOOP) {
        for (int c = c0 + NV * SPAN; c < p.cols; c += SPAN) {
            float v[8];
            fetch(c, v);
            if (p.sum) store8(static_cast<T*>(p.sum) + row * p.lds + c, p.cols - c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) total += v[i];
        }
        float unused = 0.0f;
        block_sums<WAVES>(total, unused, part[0]);
        mean = total / (float)p.cols;
        spread = squares(mean);
        for (int c = c0 + NV * SPAN; c < p.cols; c += SPAN) {
            float v[8];
            fetch(c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float apart = c + i < p.cols ? v[i] - mean : 0.0f;
                spread += apart * apart;
            }
        }
        block_sums<WAVES>(spread, unused, part[1]);
    } else {
        // columns of a wave: 512 at each of its NV places
        auto columns = [&](int wave) {
            int n = 0;
#pragma unroll
            for (int j = 0; j < NV; ++j) n += min(max(p.cols - wave * 512 - j * SPAN, 0), 512);
            return (float)n;
        };
        total = wave_sum(total);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const float own = columns(wave);
        const float near = own > 0.0f ? total / own : 0.0f;
        spread = wave_sum(squares(near));
        if constexpr (WAVES == 1) {
            mean = near;
        } else {
            if ((threadIdx.x & 63) == 0) part[0][wave][0] = total, part[0][wave][1] = spread;
            __syncthreads();
            mean = spread = 0.0f;
#pragma unroll
            for (int v = 0; v < WAVES; ++v) mean += part[0][v][0];
            mean /= (float)p.cols;
#pragma unroll
            for (int v = 0; v < WAVES; ++v) {
                const float n = columns(v), apart = n > 0.0f ? part[0][v][0] / n - mean : 0.0f;
                spread += part[0][v][1] + n * apart * apart;
            }
        }
    }
    const float rstd = 1.0f / sqrtf(spread / (float)p.cols + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }

    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[j][i] = (s[j][i] - mean) * rstd * w[j][i] + b[j][i];
            if constexpr (E4M3) most = fmaxf(most, fabsf(s[j][i]));
        }
    auto again = [&](int c, float (&v)[8]) {
        float g[8], h[8];
        fetch(c, v);
        factors(c, g, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (v[i] - mean) * rstd * g[i] + h[i];
    };
    float inv = 1.0f, shift = 1.0f;
    if constexpr (E4M3) {
        // columns past the row's end have weight and bias 0, so their y is 0 (or no number, as the row's own are)
        if constexpr (LOOP)
            for (int c = c0 + NV * SPAN; c < p.cols; c += SPAN) {
                float v[8];
                again(c, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i]));
            }
        most = block_max<WAVES>(most, &part[2][0][0]);
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

// dx, and this workgroup's share of dweight and dbias, for rows blockIdx.x,
// + gridDim.x, ...  The shares stay in registers until the last row (LOOP:
// rows too long for that get them from layer_norm_weight_kernel).
template <class T, int WAVES, int NV, bool LOOP>
__global__ __launch_bounds__(64 * WAVES) void layer_norm_grad_kernel(const LayerNormGradArgs p)
{
    constexpr int THREADS = 64 * WAVES, SPAN = THREADS * 8;
    __shared__ float part[2][WAVES][2];
    const T* weight = static_cast<const T*>(p.weight);
    const int c0 = threadIdx.x * 8;
    float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        load8(weight + c0 + j * SPAN, p.cols - c0 - j * SPAN, w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = db[j][i] = 0.0f;
    }
    const float per = 1.0f / (float)p.cols;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
        const T* sum = static_cast<const T*>(p.sum) + row * p.lds;
        const T* dsum = p.dsum ? static_cast<const T*>(p.dsum) + row * p.ldd : nullptr;
        T* dx = static_cast<T*>(p.dx) + row * p.lddx;
        const float mean = p.mean[row], rstd = p.rstd[row];
        float u[NV][8], g[NV][8], d[NV][8];
        float level = 0.0f, along = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN, nv = p.cols - c;
            load8(dy + c, nv, g[j]);
            load8(sum + c, nv, u[j]);
            if (dsum) load8(dsum + c, nv, d[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                u[j][i] = (u[j][i] - mean) * rstd;             // past the row's end g is 0
                dw[j][i] += g[j][i] * u[j][i];
                db[j][i] += g[j][i];
                g[j][i] *= w[j][i];
                level += g[j][i];
                along += g[j][i] * u[j][i];
            }
        if constexpr (LOOP)
            for (int c = c0 + NV * SPAN; c < p.cols; c += SPAN) {
                float a[8], b[8], e[8];
                load8(dy + c, p.cols - c, a);
                load8(sum + c, p.cols - c, b);
                load8(weight + c, p.cols - c, e);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] *= e[i];
                    level += a[i];
                    along += a[i] * ((b[i] - mean) * rstd);
                }
            }
        // two parts in turn: a wave may start the next row's sums while another still reads this one's
        block_sums<WAVES>(level, along, part[turn]);
        level *= per, along *= per;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g[j][i] = rstd * (g[j][i] - level - u[j][i] * along);
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
                for (int i = 0; i < 8; ++i) a[i] = rstd * (a[i] * e[i] - level - (b[i] - mean) * rstd * along);
                if (dsum) {
                    load8(dsum + c, p.cols - c, e);
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] += e[i];
                }
                store8(dx + c, p.cols - c, a);
            }
    }
    if constexpr (!LOOP) {
        float* out = p.partial + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN;
            if (c >= p.cols) continue;
            if (p.dweight) store8(out + c, p.cols - c, dw[j]);
            if (p.dbias) store8(out + p.cols + c, p.cols - c, db[j]);
        }
    }
}

// dweight's and dbias's partial column sums on their own, for rows past the
// registers: a group walks its rows with one vector of eight columns a thread.
template <class T> __global__ __launch_bounds__(64) void layer_norm_weight_kernel(const LayerNormGradArgs p)
{
    const int c = (blockIdx.y * 64 + threadIdx.x) * 8, nv = p.cols - c;
    if (nv <= 0) return;
    float dw[8] = {}, db[8] = {};
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float a[8], b[8];
        load8(static_cast<const T*>(p.dy) + row * p.lddy + c, nv, a);
        load8(static_cast<const T*>(p.sum) + row * p.lds + c, nv, b);
        const float mean = p.mean[row], rstd = p.rstd[row];
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] += a[i] * ((b[i] - mean) * rstd), db[i] += a[i];
    }
    float* out = p.partial + (int64_t)blockIdx.x * 2 * p.cols + c;
    if (p.dweight) store8(out, nv, dw);
    if (p.dbias) store8(out + p.cols, nv, db);
}

// Sixteen columns a block, 64 lanes of groups; blockIdx.y: dweight's sums, dbias's.
template <class T> __global__ __launch_bounds__(1024) void layer_norm_join_kernel(const LayerNormGradArgs p)
{
    T* out = static_cast<T*>(blockIdx.y ? p.dbias : p.dweight);
    if (!out) return;
    __shared__ float part[64][17];
    const float* from = p.partial + blockIdx.y * p.cols;
    const int c = blockIdx.x * 16 + threadIdx.x;
    float s = 0.0f;
    if (c < p.cols) {
#pragma unroll 4
        for (int g = threadIdx.y; g < p.groups; g += 64) s += from[(int64_t)g * 2 * p.cols + c];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y >= 4) return;
    s = 0.0f;
#pragma unroll
    for (int y = 0; y < 16; ++y) s += part[16 * threadIdx.y + y][threadIdx.x];
    // the first wave holds four sums a column, in lanes 16 apart
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (threadIdx.y == 0 && c < p.cols) out[c] = from_f32<T>(s);
}

// HIP takes grids of fewer than 2^32 threads; a workgroup per row of at most 512 threads reaches that at 2^23 rows.
constexpr int GRID_ROWS = 1 << 22;

template <class T, bool E4M3> hipError_t launch_rows(const LayerNormArgs& p, hipStream_t stream)
{
    const int v = (p.cols + 7) / 8;                            // vectors in a row
    if (v <= 64) layer_norm_kernel<T, E4M3, 1, 1, false><<<p.rows, 64, 0, stream>>>(p);
    else if (v <= 256) layer_norm_kernel<T, E4M3, 4, 1, false><<<p.rows, 256, 0, stream>>>(p);
    else if (v <= 512) layer_norm_kernel<T, E4M3, 4, 2, false><<<p.rows, 256, 0, stream>>>(p);
    else if (v <= 1024) layer_norm_kernel<T, E4M3, 4, 4, false><<<p.rows, 256, 0, stream>>>(p);
    else if (v <= 2048) layer_norm_kernel<T, E4M3, 8, 4, false><<<p.rows, 512, 0, stream>>>(p);
    else layer_norm_kernel<T, E4M3, 8, 4, true><<<p.rows, 512, 0, stream>>>(p);
    return hipGetLastError();
}

template <class T, bool E4M3> hipError_t launch_type(const LayerNormArgs& all, hipStream_t stream)
{
    using Out = typename std::conditional<E4M3, uint8_t, T>::type;
    for (int64_t first = 0; first < all.rows; first += GRID_ROWS) {
        LayerNormArgs p = all;
        p.rows = (int)(all.rows - first < GRID_ROWS ? all.rows - first : GRID_ROWS);
        p.x = static_cast<const T*>(all.x) + first * all.ldx;
        if (p.residual) p.residual = static_cast<const T*>(all.residual) + first * all.ldr;
        p.y = static_cast<Out*>(all.y) + first * all.ldy;
        if (p.sum) p.sum = static_cast<T*>(all.sum) + first * all.lds;
        if (p.mean) p.mean = all.mean + first;
        if (p.rstd) p.rstd = all.rstd + first;
        if (p.scale) p.scale = all.scale + first;
        const hipError_t err = launch_rows<T, E4M3>(p, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

constexpr int GRAD_MOST = 16384;   // columns whose shares of dweight and dbias a workgroup keeps in registers

template <class T> hipError_t launch_grad_type(const LayerNormGradArgs& p, hipStream_t stream)
{
    const int v = (p.cols + 7) / 8;
    if (v <= 64) layer_norm_grad_kernel<T, 1, 1, false><<<p.groups, 64, 0, stream>>>(p);
    else if (v <= 256) layer_norm_grad_kernel<T, 4, 1, false><<<p.groups, 256, 0, stream>>>(p);
    else if (v <= 512) layer_norm_grad_kernel<T, 4, 2, false><<<p.groups, 256, 0, stream>>>(p);
    else if (v <= 1024) layer_norm_grad_kernel<T, 8, 2, false><<<p.groups, 512, 0, stream>>>(p);
    else if (p.cols <= GRAD_MOST) layer_norm_grad_kernel<T, 16, 2, false><<<p.groups, 1024, 0, stream>>>(p);
    else {
        layer_norm_grad_kernel<T, 8, 2, true><<<p.groups, 512, 0, stream>>>(p);
        if (p.dweight || p.dbias)
            layer_norm_weight_kernel<T><<<dim3(p.groups, (v + 63) / 64), 64, 0, stream>>>(p);
    }
    if (p.dweight || p.dbias)
        layer_norm_join_kernel<T><<<dim3((p.cols + 15) / 16, 2), dim3(16, 64), 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(DType dt, bool e4m3, const LayerNormArgs& p, hipStream_t stream)
{
    if (dt == DType::F32) return e4m3 ? launch_type<float, true>(p, stream) : launch_type<float, false>(p, stream);
    return e4m3 ? launch_type<Bf16, true>(p, stream) : launch_type<Bf16, false>(p, stream);
}

int layer_norm_grad_groups(int rows, int cols, int num_cu)
{
    const int per_cu = cols <= 512 ? 16 : cols <= 4096 ? 4 : cols <= 8192 ? 2 : 1;
    return rows < num_cu * per_cu ? (rows > 1 ? rows : 1) : num_cu * per_cu;
}

hipError_t launch_layer_norm_grad(DType dt, const LayerNormGradArgs& p, hipStream_t stream)
{
    return dt == DType::F32 ? launch_grad_type<float>(p, stream) : launch_grad_type<Bf16>(p, stream);
}

}  // namespace miconv
