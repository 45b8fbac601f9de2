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
// Resident workgroups walk the rows, so that weight and bias are loaded once and
// the next row is on its way while this one is summed: 4095 x 4096 to e4m3 with a
// residual takes 23.4 us, 5.0 TB/s (a workgroup per row: 40), the gradient of
// 8192 x 4096 bf16 45 us and 4 more to join the weight's and bias's partial sums,
// a copy's rate (104 before); few rows' gradients are a launch, 64 x 4096 4.5.
//
// The variance is a sum of squared distances, never a difference of sums: each
// wave takes its own values' mean and their squared distances from it, and the
// waves' means and squares are put together by
//   sum (s - mean)^2 = sum over waves of (squares_w + n_w (mean_w - mean)^2),
// so one exchange through LDS gives both, and a row far from zero keeps its
// variance.
#include <algorithm>
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

// How a row's columns end: with a whole vector of eight, or inside one.  A cut
// vector is loaded as the row's last eight elements and shifted into place where
// it is used: element by element its loads would wait for each other, and for the
// next row's on their way (8192 x 4095 bf16 then takes 110 us instead of 54).  Rows of
// fewer than eight columns have no such eight.
enum RowEnd : int { END_WHOLE, END_CUT, END_SHORT };

// Eight columns as they lie in memory, so that a row on its way takes half the registers of its values in bf16.
template <class T, int END> struct Vec {
    static constexpr int E = sizeof(T), WORDS = 2 * E;
    uint32_t word[WORDS];
    // the first nv exist
    __device__ __forceinline__ void load(const T* p, int nv)
    {
        if constexpr (END == END_SHORT) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const u32x4 t = load_piece<E>(reinterpret_cast<const uint8_t*>(p) + 16 * i, nv - i * (16 / E));
#pragma unroll
                for (int k = 0; k < 4; ++k) word[4 * i + k] = t[k];
            }
        } else if (nv > 0) {
            __builtin_memcpy(word, END == END_CUT && nv < 8 ? p + (nv - 8) : p, sizeof(word));
        } else {
            clear();
        }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) word[i] = 0;
    }
    // after load, before value: a cut vector's elements to their places, zeros behind them
    __device__ __forceinline__ void settle(int nv)
    {
        if (END != END_CUT || nv <= 0 || nv >= 8) return;
        const int by = 8 - nv;
#pragma unroll
        for (int step = 4; step > 0; step >>= 1) {
            if (!(by & step)) continue;
            if constexpr (E == 2)
                if (step == 1) {
#pragma unroll
                    for (int i = 0; i < WORDS; ++i) word[i] = word[i] >> 16 | (i + 1 < WORDS ? word[i + 1] << 16 : 0);
                    continue;
                }
            const int words = step * E / 4;
#pragma unroll
            for (int i = 0; i < WORDS; ++i) word[i] = i + words < WORDS ? word[i + words] : 0;
        }
    }
    // what was made of these before is made again from here on
    __device__ __forceinline__ void forget()
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) asm volatile("" : "+v"(word[i]));
    }
    __device__ __forceinline__ float value(int i) const
    {
        if constexpr (E == 4) return __uint_as_float(word[i & (WORDS - 1)]);
        return __uint_as_float(i & 1 ? word[(i >> 1) & 3] & 0xffff0000u : word[(i >> 1) & 3] << 16);
    }
};

// The same number, no longer known to be: what follows from it is not kept in registers from row to row (the masks of a
// cut vector's elements, two scalars each).
__device__ __forceinline__ int anew(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// The scale of a row whose largest |y| is `most` (1 for a row of zeros, or one too small for a scale): stored at `to`,
// its inverse as inv * shift.
__device__ __forceinline__ float e4m3_scale(float most, float& shift, float* to)
{
    const float scale = most / E4M3_MAX > 0.0f ? most / E4M3_MAX : 1.0f;
    shift = scale < 0x1p-100f ? 0x1p+64f : 1.0f;
    if (to) *to = scale;
    return 1.0f / (scale * shift);
}

// Rows blockIdx.x, + gridDim.x, ..., NV vectors of eight columns per thread;
// weight and bias stay in registers, the next row is on its way while this one
// is summed.
template <class T, bool E4M3, int WAVES, int NV, int END>
__global__ __launch_bounds__(64 * WAVES) void layer_norm_kernel(const LayerNormArgs p)
{
    constexpr int SPAN = 64 * WAVES * 8;
    __shared__ float part[2][WAVES][3], top[2][WAVES];
    const int c0 = threadIdx.x * 8;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // columns of a wave: 512 at each of its NV places
    auto columns = [&](int of) {
        int n = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) n += min(max(p.cols - of * 512 - j * SPAN, 0), 512);
        return (float)n;
    };
    Vec<T, END> w[NV], b[NV], x[NV], res[NV];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN, nv = p.cols - c;
            x[j].load(static_cast<const T*>(p.x) + row * p.ldx + c, nv);
            if (p.residual) res[j].load(static_cast<const T*>(p.residual) + row * p.ldr + c, nv);
        }
    };
    load(blockIdx.x);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * SPAN;
        w[j].load(static_cast<const T*>(p.weight) + c, p.cols - c);
        if (p.bias) b[j].load(static_cast<const T*>(p.bias) + c, p.cols - c);
        else b[j].clear();
        w[j].settle(p.cols - c);
        if (p.bias) b[j].settle(p.cols - c);
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        float s[NV][8];
        float total = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int nv = anew(p.cols - c0 - j * SPAN);
            x[j].settle(nv);
            if (p.residual) res[j].settle(nv);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[j][i] = x[j].value(i);
                if (p.residual) s[j][i] += res[j].value(i);
                total += s[j][i];
            }
        }
        if (row + gridDim.x < p.rows) load(row + gridDim.x);
        total = wave_sum(total);
        const float own = columns(wave);
        const float near = own > 0.0f ? total / own : 0.0f;
        float spread = 0.0f, mean = near;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN;
            const int nv = anew(p.cols - c);
            if (END == END_WHOLE ? nv > 0 : nv >= 8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) spread += (s[j][i] - near) * (s[j][i] - near);
            } else if (END != END_WHOLE && nv > 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float apart = i < nv ? s[j][i] - near : 0.0f;
                    spread += apart * apart;
                }
            }
            if (p.sum && nv > 0)
                store8(static_cast<T*>(p.sum) + row * p.lds + c, END == END_WHOLE ? 8 : nv, s[j]);
        }
        spread = wave_sum(spread);
        if constexpr (WAVES > 1) {
            // two parts in turn: a wave may be at the next row while another still reads this one's
            if ((threadIdx.x & 63) == 0)
                part[turn][wave][0] = total, part[turn][wave][1] = near, part[turn][wave][2] = spread;
            __syncthreads();
            mean = spread = 0.0f;
#pragma unroll
            for (int v = 0; v < WAVES; ++v) mean += part[turn][v][0];
            mean /= (float)p.cols;
#pragma unroll
            for (int v = 0; v < WAVES; ++v) {
                const float apart = part[turn][v][1] - mean;
                spread += part[turn][v][2] + columns(v) * apart * apart;
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
                // past the row's end weight and bias are 0, and so is y (or no number, as the row's own are)
                s[j][i] = (s[j][i] - mean) * rstd * w[j].value(i) + b[j].value(i);
                if constexpr (E4M3) most = fmaxf(most, fabsf(s[j][i]));
            }
        float inv = 1.0f, shift = 1.0f;
        if constexpr (E4M3) {
            most = block_max<WAVES>(most, top[turn]);
            inv = e4m3_scale(most, shift, threadIdx.x == 0 ? p.scale + row : nullptr);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN;
            const int nv = anew(p.cols - c);
            if (nv <= 0) continue;
            if constexpr (E4M3)
                store8_e4m3(static_cast<uint8_t*>(p.y) + row * p.ldy + c, END == END_WHOLE ? 8 : nv, s[j], inv, shift);
            else
                store8(static_cast<T*>(p.y) + row * p.ldy + c, END == END_WHOLE ? 8 : nv, s[j]);
        }
    }
}

// A long row per workgroup: NV vectors of eight columns per thread stay in
// registers, weight and bias do not; the rest of a row past them is read again in
// every pass.
template <class T, bool E4M3, int WAVES, int NV>
__global__ __launch_bounds__(64 * WAVES) void layer_norm_long_kernel(const LayerNormArgs p)
{
    constexpr int SPAN = 64 * WAVES * 8;
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
    // over all of this thread's columns: the kept ones, then those read again
    float s[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) fetch(c0 + j * SPAN, s[j]);
    auto each = [&](auto&& f) {
#pragma unroll
        for (int j = 0; j < NV; ++j) f(c0 + j * SPAN, s[j]);
        for (int c = c0 + NV * SPAN; c < p.cols; c += SPAN) {
            float v[8];
            fetch(c, v);
            f(c, v);
        }
    };
    float total = 0.0f, spread = 0.0f, unused = 0.0f;
    each([&](int c, const float (&v)[8]) {
        if (p.sum && c < p.cols) store8(static_cast<T*>(p.sum) + row * p.lds + c, p.cols - c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) total += v[i];
    });
    block_sums<WAVES>(total, unused, part[0]);
    const float mean = total / (float)p.cols;
    each([&](int c, const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float apart = c + i < p.cols ? v[i] - mean : 0.0f;
            spread += apart * apart;
        }
    });
    block_sums<WAVES>(spread, unused, part[1]);
    const float rstd = 1.0f / sqrtf(spread / (float)p.cols + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    auto result = [&](int c, const float (&v)[8], float (&y)[8]) {
        float w[8], b[8] = {};
        load8(weight + c, p.cols - c, w);
        if (bias) load8(bias + c, p.cols - c, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (v[i] - mean) * rstd * w[i] + b[i];
    };
    float inv = 1.0f, shift = 1.0f;
    if constexpr (E4M3) {
        float most = 0.0f;
        each([&](int c, const float (&v)[8]) {
            float y[8];
            result(c, v, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(y[i]));
        });
        most = block_max<WAVES>(most, &part[2][0][0]);
        inv = e4m3_scale(most, shift, threadIdx.x == 0 ? p.scale + row : nullptr);
    }
    each([&](int c, const float (&v)[8]) {
        if (c >= p.cols) return;
        float y[8];
        result(c, v, y);
        if constexpr (E4M3)
            store8_e4m3(static_cast<uint8_t*>(p.y) + row * p.ldy + c, p.cols - c, y, inv, shift);
        else
            store8(static_cast<T*>(p.y) + row * p.ldy + c, p.cols - c, y);
    });
}

// dx, and this workgroup's share of dweight and dbias, for rows blockIdx.x,
// + gridDim.x, ...: the shares and the weight stay in registers until the last
// row, the next row is on its way while this one is summed (NEXT, where the
// registers hold both).  ROWS > 1: short rows, one to each wave at a time.
template <class T, int WAVES, int ROWS, int NV, bool NEXT, int END>
__global__ __launch_bounds__(64 * WAVES * ROWS) void layer_norm_grad_kernel(const LayerNormGradArgs p)
{
    static_assert(ROWS == 1 || (WAVES == 1 && NV == 1), "a wave to a row");
    constexpr int SPAN = 64 * WAVES * 8;
    __shared__ float part[2][WAVES][2];
    const int c0 = (ROWS > 1 ? threadIdx.x & 63 : threadIdx.x) * 8;
    const int64_t start = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x >> 6 : 0);
    const int64_t hop = (int64_t)gridDim.x * ROWS;
    Vec<T, END> w[NV], dy[NV], sum[NV], dsum[NV];
    float dw[NV][8], db[NV][8], mean, rstd;
    auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN, nv = p.cols - c;
            dy[j].load(static_cast<const T*>(p.dy) + row * p.lddy + c, nv);
            sum[j].load(static_cast<const T*>(p.sum) + row * p.lds + c, nv);
            if (p.dsum) dsum[j].load(static_cast<const T*>(p.dsum) + row * p.ldd + c, nv);
        }
        mean = p.mean[row], rstd = p.rstd[row];
    };
    if (start < p.rows) load(start);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int nv = p.cols - c0 - j * SPAN;
        w[j].load(static_cast<const T*>(p.weight) + c0 + j * SPAN, nv);
        w[j].settle(nv);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = db[j][i] = 0.0f;
    }
    const float per = 1.0f / (float)p.cols;
    int turn = 0;
    for (int64_t row = start; row < p.rows; row += hop, turn ^= 1) {
        float u[NV][8], g[NV][8];
        const float scale = rstd;
        float level = 0.0f, along = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int nv = anew(p.cols - c0 - j * SPAN);
            dy[j].settle(nv);
            sum[j].settle(nv);
            if (p.dsum) dsum[j].settle(nv);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = dy[j].value(i);                // past the row's end 0
                u[j][i] = (sum[j].value(i) - mean) * scale;
                dw[j][i] += v * u[j][i];
                db[j][i] += v;
                g[j][i] = v * w[j].value(i);
                level += g[j][i];
                along += g[j][i] * u[j][i];
            }
        }
        Vec<T, END> add[NV];
        if constexpr (NEXT) {
#pragma unroll
            for (int j = 0; j < NV; ++j) add[j] = dsum[j];
            if (row + hop < p.rows) load(row + hop);
        }
        // two parts in turn: a wave may start the next row's sums while another still reads this one's
        block_sums<WAVES>(level, along, part[turn]);
        level *= per, along *= per;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * SPAN, nv = anew(p.cols - c);
            float v[8];
            if constexpr (!NEXT) {
                // from the row as it came: its products do not stay in registers over the exchange
                dy[j].forget();
                sum[j].forget();
                add[j] = dsum[j];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float gi = NEXT ? g[j][i] : dy[j].value(i) * w[j].value(i);
                const float ui = NEXT ? u[j][i] : (sum[j].value(i) - mean) * scale;
                v[i] = scale * (gi - level - ui * along);
                if (p.dsum) v[i] += add[j].value(i);
            }
            if (nv > 0) store8(static_cast<T*>(p.dx) + row * p.lddx + c, END == END_WHOLE ? 8 : nv, v);
        }
        if (!NEXT && row + hop < p.rows) load(row + hop);
    }
    float* out = p.partial + (int64_t)blockIdx.x * 2 * p.cols;
    if constexpr (ROWS > 1) {
        __shared__ float shares[ROWS][2][512 + 8];
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < 8; ++i) shares[wave][0][c0 + i] = dw[0][i], shares[wave][1][c0 + i] = db[0][i];
        __syncthreads();
        for (int c = threadIdx.x; c < p.cols; c += 64 * ROWS) {
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) a += shares[r][0][c], b += shares[r][1][c];
            if (p.dweight) out[c] = a;
            if (p.dbias) out[p.cols + c] = b;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * SPAN;
        if (c >= p.cols) continue;
        if (p.dweight) store8(out + c, p.cols - c, dw[j]);
        if (p.dbias) store8(out + p.cols + c, p.cols - c, db[j]);
    }
}

// All of it in one launch, without partial sums, for few rows or rows past the registers: a workgroup per 64 columns walks
// all rows for dweight and dbias, the others have dx, a row at a time.  dy and sum are read twice, by both, mostly from
// cache; rows of more than 8192 columns again past those.
template <class T, int END> __global__ __launch_bounds__(512) void layer_norm_grad_few_kernel(const LayerNormGradArgs p, int column_blocks)
{
    constexpr int WAVES = 8, SPAN = 64 * WAVES * 8, KEPT = 2;
    const T* weight = static_cast<const T*>(p.weight);
    auto fetch = [&](const void* from, int64_t at, int nv, float (&v)[8]) {
        Vec<T, END> t;
        t.load(static_cast<const T*>(from) + at, nv);
        t.settle(nv);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = t.value(i);
    };
    if ((int)blockIdx.x < column_blocks) {
        // eight threads across, 64 rows at a time
        __shared__ float part[WAVES][2][64];
        const int x = threadIdx.x & 7, c = (int)blockIdx.x * 64 + x * 8, nv = p.cols - c;
        float dw[8] = {}, db[8] = {};
        if (nv > 0) {
#pragma unroll 2
            for (int row = threadIdx.x >> 3; row < p.rows; row += 64) {
                float a[8], b[8];
                fetch(p.dy, row * p.lddy + c, nv, a);
                fetch(p.sum, row * p.lds + c, nv, b);
                const float mean = p.mean[row], rstd = p.rstd[row];
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[i] += a[i] * ((b[i] - mean) * rstd), db[i] += a[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int o = 8; o < 64; o <<= 1) dw[i] += __shfl_xor(dw[i], o), db[i] += __shfl_xor(db[i], o);
            if ((threadIdx.x & 63) < 8) part[threadIdx.x >> 6][0][x * 8 + i] = dw[i], part[threadIdx.x >> 6][1][x * 8 + i] = db[i];
        }
        __syncthreads();
        if (threadIdx.x >= 128) return;
        const int of = threadIdx.x >> 6, column = (int)blockIdx.x * 64 + (threadIdx.x & 63);
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += part[w][of][threadIdx.x & 63];
        T* out = static_cast<T*>(of ? p.dbias : p.dweight);
        if (out && column < p.cols) out[column] = from_f32<T>(s);
        return;
    }
    __shared__ float part[2][WAVES][2];
    const float per = 1.0f / (float)p.cols;
    int turn = 0;
    for (int64_t row = (int)blockIdx.x - column_blocks; row < p.rows; row += (int)gridDim.x - column_blocks, turn ^= 1) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        float g[KEPT][8], u[KEPT][8];
        auto both = [&](int c, float (&gc)[8], float (&uc)[8]) {
            float w[8];
            fetch(p.dy, row * p.lddy + c, p.cols - c, gc);
            fetch(p.sum, row * p.lds + c, p.cols - c, uc);
            fetch(weight, c, p.cols - c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) gc[i] *= w[i], uc[i] = (uc[i] - mean) * rstd;
        };
        // over all of this thread's columns: the kept ones, then those read again
#pragma unroll
        for (int j = 0; j < KEPT; ++j) both(threadIdx.x * 8 + j * SPAN, g[j], u[j]);
        auto each = [&](auto&& f) {
#pragma unroll
            for (int j = 0; j < KEPT; ++j) f(threadIdx.x * 8 + j * SPAN, g[j], u[j]);
            for (int c = threadIdx.x * 8 + KEPT * SPAN; c < p.cols; c += SPAN) {
                float gc[8], uc[8];
                both(c, gc, uc);
                f(c, gc, uc);
            }
        };
        float level = 0.0f, along = 0.0f;
        each([&](int, const float (&gc)[8], const float (&uc)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) level += gc[i], along += gc[i] * uc[i];
        });
        block_sums<WAVES>(level, along, part[turn]);
        level *= per, along *= per;
        each([&](int c, const float (&gc)[8], const float (&uc)[8]) {
            const int nv = p.cols - c;
            if (nv <= 0) return;
            float d[8] = {}, v[8];
            if (p.dsum) fetch(p.dsum, row * p.ldd + c, nv, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = rstd * (gc[i] - level - uc[i] * along) + d[i];
            store8(static_cast<T*>(p.dx) + row * p.lddx + c, END == END_WHOLE ? 8 : nv, v);
        });
    }
}

// 32 columns a block, 32 lanes of groups: lines of 128 bytes (of 64, 512 groups of 4096 columns took 7 us instead of 4.8);
// blockIdx.y: dweight's sums, dbias's.
template <class T> __global__ __launch_bounds__(1024) void layer_norm_join_kernel(const LayerNormGradArgs p)
{
    T* out = static_cast<T*>(blockIdx.y ? p.dbias : p.dweight);
    if (!out) return;
    __shared__ float part[32][33];
    const float* from = p.partial + blockIdx.y * p.cols;
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < p.cols) {
#pragma unroll 8
        for (int g = threadIdx.y; g < p.groups; g += 32) s += from[(int64_t)g * 2 * p.cols + c];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    // a column's 32 sums across half a wave
    s = part[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor(s, o);
    const int column = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && column < p.cols) out[column] = from_f32<T>(s);
}

// Workgroups that walk `rows` rows, at most `most`, all with as many rows but the last one's.
int even_groups(int rows, int most)
{
    const int per = (rows + most - 1) / most;
    return per > 1 ? (rows + per - 1) / per : rows;
}

template <class T, bool E4M3, int WAVES, int NV> void launch_waves(const LayerNormArgs& p, int per_cu, hipStream_t stream)
{
    const int grid = even_groups(p.rows, per_cu * p.num_cu);
    if (p.cols % 8 == 0) layer_norm_kernel<T, E4M3, WAVES, NV, END_WHOLE><<<grid, 64 * WAVES, 0, stream>>>(p);
    else layer_norm_kernel<T, E4M3, WAVES, NV, END_CUT><<<grid, 64 * WAVES, 0, stream>>>(p);
}

// Rows of a workgroup each go 2^16 to a launch, a millisecond of rows past the registers: HIP takes grids of fewer than 2^32
// threads, which a workgroup of 512 per row reaches at 2^23 rows, and tests can reach the next launch's rows.  (Resident
// workgroups that walk these rows, weight and bias read again for each, are 2 to 13 percent slower: 8192 x 20000 fp32
// 358 us instead of 318, bf16 239 instead of 231.)
constexpr int GRID_ROWS = 1 << 16;

template <class T, bool E4M3> hipError_t launch_type(const LayerNormArgs& p, hipStream_t stream)
{
    const int v = (p.cols + 7) / 8;                            // vectors in a row
    if (p.cols < 8) layer_norm_kernel<T, E4M3, 1, 1, END_SHORT><<<even_groups(p.rows, 24 * p.num_cu), 64, 0, stream>>>(p);
    else if (v <= 64) launch_waves<T, E4M3, 1, 1>(p, 24, stream);
    else if (v <= 128) launch_waves<T, E4M3, 2, 1>(p, 12, stream);
    else if (v <= 256) launch_waves<T, E4M3, 4, 1>(p, 6, stream);
    else if (v <= 512) launch_waves<T, E4M3, 4, 2>(p, 4, stream);
    else if (v <= 1024) launch_waves<T, E4M3, 8, 2>(p, 2, stream);
    else if (v <= 1536) launch_waves<T, E4M3, 12, 2>(p, 1, stream);
    else {
        using Out = typename std::conditional<E4M3, uint8_t, T>::type;
        for (int64_t first = 0; first < p.rows; first += GRID_ROWS) {
            LayerNormArgs part = p;
            part.rows = (int)(p.rows - first < GRID_ROWS ? p.rows - first : GRID_ROWS);
            part.x = static_cast<const T*>(p.x) + first * p.ldx;
            if (p.residual) part.residual = static_cast<const T*>(p.residual) + first * p.ldr;
            part.y = static_cast<Out*>(p.y) + first * p.ldy;
            if (p.sum) part.sum = static_cast<T*>(p.sum) + first * p.lds;
            if (p.mean) part.mean = p.mean + first;
            if (p.rstd) part.rstd = p.rstd + first;
            if (p.scale) part.scale = p.scale + first;
            layer_norm_long_kernel<T, E4M3, 8, 4><<<part.rows, 512, 0, stream>>>(part);
            const hipError_t err = hipGetLastError();
            if (err != hipSuccess) return err;
        }
    }
    return hipGetLastError();
}

template <class T, int WAVES, int ROWS, int NV, bool NEXT> void launch_grad_waves(const LayerNormGradArgs& p, hipStream_t stream)
{
    constexpr int THREADS = 64 * WAVES * ROWS;
    if (p.cols % 8 == 0) layer_norm_grad_kernel<T, WAVES, ROWS, NV, NEXT, END_WHOLE><<<p.groups, THREADS, 0, stream>>>(p);
    else layer_norm_grad_kernel<T, WAVES, ROWS, NV, NEXT, END_CUT><<<p.groups, THREADS, 0, stream>>>(p);
}

constexpr int ROWS_AT_ONCE = 768, LONG_WALKS = 16;
constexpr int SHORT_ROWS = 4;      // rows of up to 512 columns that a workgroup walks side by side

template <class T> hipError_t launch_grad_type(const LayerNormGradArgs& p, hipStream_t stream)
{
    const int v = (p.cols + 7) / 8;
    if (!p.groups) {
        const int columns = p.dweight || p.dbias ? (p.cols + 63) / 64 : 0;
        const uint32_t grid = (uint32_t)(columns + std::min(p.rows, GRID_ROWS));
        if (p.cols < 8) layer_norm_grad_few_kernel<T, END_SHORT><<<grid, 512, 0, stream>>>(p, columns);
        else if (p.cols % 8) layer_norm_grad_few_kernel<T, END_CUT><<<grid, 512, 0, stream>>>(p, columns);
        else layer_norm_grad_few_kernel<T, END_WHOLE><<<grid, 512, 0, stream>>>(p, columns);
        return hipGetLastError();
    }
    if (p.cols < 8)
        layer_norm_grad_kernel<T, 1, SHORT_ROWS, 1, true, END_SHORT><<<p.groups, 64 * SHORT_ROWS, 0, stream>>>(p);
    else if (v <= 64) launch_grad_waves<T, 1, SHORT_ROWS, 1, true>(p, stream);
    else if (v <= 128 && p.rows > LONG_WALKS * p.num_cu) launch_grad_waves<T, 2, 1, 1, true>(p, stream);
    else if (v <= 256) launch_grad_waves<T, 4, 1, 1, true>(p, stream);
    else if (v <= 512) launch_grad_waves<T, 8, 1, 1, true>(p, stream);
    else if (v <= 1024) launch_grad_waves<T, 16, 1, 1, true>(p, stream);
    else if (v <= 1536) launch_grad_waves<T, 12, 1, 2, sizeof(T) == 2>(p, stream);
    else launch_grad_waves<T, 16, 1, 2, false>(p, stream);
    if (p.dweight || p.dbias)
        layer_norm_join_kernel<T><<<dim3((p.cols + 31) / 32, 2), dim3(32, 32), 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(DType dt, bool e4m3, const LayerNormArgs& p, hipStream_t stream)
{
    if (dt == DType::F32) return e4m3 ? launch_type<float, true>(p, stream) : launch_type<float, false>(p, stream);
    return e4m3 ? launch_type<Bf16, true>(p, stream) : launch_type<Bf16, false>(p, stream);
}

// 0: one launch.  Of few rows it saves the second launch and the walk: 64 x 4096 bf16 5.2 us (9.1), 300 x 4096 5.2 (10.9),
// 768 x 4096 7.3 (14.3); 1024 x 4095 19.8 (17.9).  Rows past 16384 columns do not stay in the registers of a walk's sixteen
// waves, and are then read as often: 8192 x 20000 bf16 385 us (863 with a walk of their own for dweight and dbias).
// Otherwise a group's shares of dweight and dbias are written and read again, so as few groups as keep memory busy: one of
// eight waves a CU (8192 x 4096 bf16 takes 49 us, 56 with two), two of four waves (8192 x 2048 30, 35 with four), each
// walking three rows at least.  Rows that fill a quarter to a half of four waves go to two where walks stay long: 8192 x
// 768 bf16 16.6 us (21.2), 32768 x 1000 49 (70), fp32 105 (100); 2048 x 768 would take 11.9 (10.5).
int layer_norm_grad_groups(int rows, int cols, int num_cu)
{
    if (rows <= ROWS_AT_ONCE || cols > 16384) return 0;
    const int walks = cols <= 512 ? (rows + SHORT_ROWS - 1) / SHORT_ROWS : rows;
    const int most = std::min((cols > 512 && cols <= 1024 && rows > LONG_WALKS * num_cu ? 4 : cols <= 2048 ? 2 : 1) * num_cu, (walks + 2) / 3);
    return even_groups(walks, most);
}

hipError_t launch_layer_norm_grad(DType dt, const LayerNormGradArgs& p, hipStream_t stream)
{
    return dt == DType::F32 ? launch_grad_type<float>(p, stream) : launch_grad_type<Bf16>(p, stream);
}

}  // namespace miconv
