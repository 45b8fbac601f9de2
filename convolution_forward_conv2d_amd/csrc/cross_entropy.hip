// cross_entropy.hip -- cross entropy around the products that make the logits:
// logits that are in memory, for the products too small for the fused epilogues
// (loss_tile.h), and what follows the pieces of a row:
//
//   largest = max over runs,  sum = sum over runs of sum_run e^(largest_run - largest)
//   lse = largest + log(sum)
//   loss = log(sum) + (1 - a) (largest - z_t) + a (largest - mean(z))
//
// so a confident row's loss is not the difference of two large numbers.  All
// fp32, joined in a fixed order.  Logits in memory are read once, partial sums of a
// split product added on the way: 128 x 1000 in sixteen parts take 7 us, the gradient
// of 256 x 1000 in eight 6, both the latency of loads; the join of 4096 rows of 782
// runs 9, the losses' sum, one workgroup's, 2 to 5 (19 of 65536 rows, 300 of 2^20, a
// thousand of them to a thread).
#include "linear_common.h"
#include "kernels.h"

namespace miconv {

namespace {

// e^(most - top), what a sum taken from `most` is worth at `top`, at least as large: 0 of nothing (-infinity).
__device__ __forceinline__ float above(float most, float top)
{
    return exponential<true>(most - (top == -__builtin_inff() ? 0.0f : top));
}

constexpr int THREADS = 256;

__device__ __forceinline__ void finish_row(const LossArgs& p, int64_t row, float most, float sum, float total, float* lse, float* loss)
{
    const int64_t target = p.target[row];
    const float log_sum = logf(sum);
    lse[row] = most + log_sum;
    float v = 0.0f;
    if (target != p.ignore) {
        if (loss_column(p, target) < 0) {
            v = __builtin_nanf("");
        } else if (most == -__builtin_inff() && sum == 0.0f) {
            v = __builtin_inff();                              // no class left: the target's share is nothing
        } else {
            v = log_sum + (1.0f - p.smooth) * (most - p.hit[row]);
            if (p.smooth > 0.0f) v += p.smooth * (most - total / (float)p.classes);
        }
    }
    loss[row] = v;
}

// A workgroup per row and run of its columns, four columns a thread at a time; rows of one run are finished here.
template <class T> __global__ __launch_bounds__(THREADS) void loss_rows_kernel(const LossRowsArgs p)
{
    __shared__ float part[THREADS / 64][3];
    const int runs = (p.cols + p.run - 1) / p.run;
    const int64_t hop = p.rows * p.ld;
    for (int64_t item = blockIdx.x; item < (int64_t)p.rows * runs; item += gridDim.x) {
        const int64_t row = item / runs;
        const int run = (int)(item - row * runs), first = run * p.run, last = min(first + p.run, p.cols);
        const int at = loss_column(p.loss, p.loss.target[row]);
        float most = -__builtin_inff(), sum = 0.0f, total = 0.0f;
        for (int c = first + 4 * threadIdx.x; c < last; c += 4 * THREADS) {
            // rows start at multiples of four, so four columns from c on are there whether they exist or not
            const float* at_c = p.z + row * p.ld + c;
            f32x4 z = *reinterpret_cast<const f32x4*>(at_c);
#pragma unroll 8                                               // loads of eight parts in flight together
            for (int s = 1; s < p.splits; ++s) z += *reinterpret_cast<const f32x4*>(at_c + s * hop);
            float top = most;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (c + u < last) {
                    if (p.bias) z[u] += to_f32(static_cast<const T*>(p.bias)[c + u]);
                    total += z[u];
                    if (c + u == at) p.loss.hit[row] = z[u];
                } else {
                    z[u] = -__builtin_inff();
                }
                top = fmaxf(top, z[u]);
            }
            const float from = top == -__builtin_inff() ? 0.0f : top;
            sum *= exponential<true>(most - from);             // nothing before: 0 e^-infinity
#pragma unroll
            for (int u = 0; u < 4; ++u) sum += exponential<true>(z[u] - from);
            most = top;
        }
        // the largest first, so that each lane, and wave, brings its sum there once
        float top = most;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        sum *= above(most, top);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o), total += __shfl_xor(total, o);
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) part[wave][0] = top, part[wave][1] = sum, part[wave][2] = total;
        __syncthreads();                                       // hit[row] is another thread's, too
        if (threadIdx.x == 0) {
            most = -__builtin_inff(), sum = total = 0.0f;
#pragma unroll
            for (int w = 0; w < THREADS / 64; ++w) most = fmaxf(most, part[w][0]);
#pragma unroll
            for (int w = 0; w < THREADS / 64; ++w) sum += part[w][1] * above(part[w][0], most), total += part[w][2];
            if (p.lse) {
                finish_row(p.loss, row, most, sum, total, p.lse, p.row_loss);
            } else {
                const int64_t to = (int64_t)(p.loss.part_first + run) * p.rows + row;
                reinterpret_cast<float2*>(p.loss.part)[to] = float2{most, sum};
                if (p.loss.part_z) p.loss.part_z[to] = total;
            }
        }
        __syncthreads();
    }
}

constexpr int COLS = 32;           // groups of eight columns per block
constexpr int LANES = 8;           // rows a block walks side by side

// dz of logits in memory, and its column sums.
template <class T> __global__ __launch_bounds__(COLS * LANES) void loss_gradient_kernel(const LossRowsArgs p)
{
    constexpr bool EXACT = sizeof(T) == 4;
    const int c = (blockIdx.x * COLS + threadIdx.x) * 8, nv = p.cols - c;
    const float every = p.loss.smooth / (float)p.loss.classes, goal = 1.0f - p.loss.smooth + every;
    const float unit = loss_unit<EXACT>(p.loss);
    float total[8] = {};
    if (c < p.dz_pitch) {
        float bias[8] = {};
        if (p.bias) load8(static_cast<const T*>(p.bias) + c, nv, bias);
        for (int r = blockIdx.y * LANES + threadIdx.y; r < p.rows; r += gridDim.y * LANES) {
            const float* z = p.z + (int64_t)r * p.ld + c;
            float v[8];
            load8(z, nv, v);
#pragma unroll 4                                               // loads of four parts in flight together
            for (int s = 1; s < p.splits; ++s) {
                float more[8];
                load8(z + (int64_t)s * p.rows * p.ld, nv, more);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += more[i];
            }
            const LossRow row = loss_row(p.loss, r, unit);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = i < nv ? loss_gradient<EXACT>(row, v[i] + bias[i], c + i == row.at, goal, every) : 0.0f;
                total[i] += v[i];
            }
            store8(static_cast<T*>(p.dz) + (int64_t)r * p.dz_pitch + c, 8, v);
        }
    }
    if (!p.sums) return;
    __shared__ float part[LANES][COLS * 8 + 4];
#pragma unroll
    for (int i = 0; i < 8; ++i) part[threadIdx.y][threadIdx.x * 8 + i] = total[i];
    __syncthreads();
    const int k = threadIdx.y * COLS + threadIdx.x;
    float s = 0.0f;
#pragma unroll
    for (int y = 0; y < LANES; ++y) s += part[y][k];
    const int col = blockIdx.x * COLS * 8 + k;
    if (col < p.cols) p.sums[(int64_t)blockIdx.y * p.cols + col] = s * unit;
}

// 16 rows a block, 64 lanes of runs: 4096 rows of 782 runs in 256 blocks (32 rows a block took 16.6 us).
// A row a block (ROWS = 1) where rows are few and their runs many: one row of 8192 runs takes 5 us.
template <int ROWS>
__global__ __launch_bounds__(1024) void loss_join_kernel(const LossArgs p, int rows, int runs, float* lse, float* loss)
{
    constexpr int LANES = 1024 / ROWS;
    __shared__ float part[16][ROWS][3];
    for (int64_t first = (int64_t)blockIdx.x * ROWS; first < rows; first += (int64_t)gridDim.x * ROWS) {
        const int64_t row = first + threadIdx.x;
        float most = -__builtin_inff(), sum = 0.0f, total = 0.0f;
        if (row < rows) {
            for (int r0 = threadIdx.y; r0 < runs; r0 += 8 * LANES) {
                float2 v[8];
                float top = most;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int64_t at = (int64_t)(r0 + u * LANES) * rows + row;
                    const bool some = r0 + u * LANES < runs;
                    v[u] = some ? reinterpret_cast<const float2*>(p.part)[at] : float2{-__builtin_inff(), 0.0f};
                    if (some && p.part_z) total += p.part_z[at];
                    top = fmaxf(top, v[u].x);
                }
                sum *= above(most, top);
#pragma unroll
                for (int u = 0; u < 8; ++u) sum += v[u].y * above(v[u].x, top);
                most = top;
            }
        }
        // lanes ROWS apart are a row's: their largest first, so that each brings its sum there once
        float top = most;
#pragma unroll
        for (int o = ROWS; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
        sum *= above(most, top);
#pragma unroll
        for (int o = ROWS; o < 64; o <<= 1) sum += __shfl_xor(sum, o), total += __shfl_xor(total, o);
        constexpr int PER = 64 / ROWS;                         // a wave's lanes of a row
        if (threadIdx.y % PER == 0) {
            float* to = part[threadIdx.y / PER][threadIdx.x];
            to[0] = top, to[1] = sum, to[2] = total;
        }
        __syncthreads();
        if (threadIdx.y == 0 && row < rows) {
            top = -__builtin_inff(), sum = total = 0.0f;
#pragma unroll
            for (int w = 0; w < 16; ++w) top = fmaxf(top, part[w][threadIdx.x][0]);
#pragma unroll
            for (int w = 0; w < 16; ++w) {
                sum += part[w][threadIdx.x][1] * above(part[w][threadIdx.x][0], top);
                total += part[w][threadIdx.x][2];
            }
            finish_row(p, row, top, sum, total, lse, loss);
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(1024) void loss_reduce_kernel(const LossArgs p, int rows, const float* loss, bool mean, float* total,
                                                           float* count)
{
    __shared__ float part[16];
    __shared__ int many[16];
    float sum = 0.0f;
    int n = 0;
    for (int64_t r = threadIdx.x; r < rows; r += 1024) {
        sum += loss[r];
        n += p.target[r] != p.ignore;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o), n += __shfl_xor(n, o);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave] = sum, many[wave] = n;
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < 16; ++w) sum += part[w], n += many[w];
    *total = !mean ? sum : n ? sum / (float)n : 0.0f;
    *count = (float)n;
}

}  // namespace

hipError_t launch_loss_rows(DType dt, const LossRowsArgs& p, hipStream_t stream)
{
    const int64_t items = (int64_t)p.rows * ((p.cols + p.run - 1) / p.run);
    const uint32_t grid = (uint32_t)(items < 1 << 20 ? items : 1 << 20);
    if (dt == DType::F32) loss_rows_kernel<float><<<grid, THREADS, 0, stream>>>(p);
    else loss_rows_kernel<Bf16><<<grid, THREADS, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_loss_gradient(DType dt, const LossRowsArgs& p, hipStream_t stream)
{
    const int groups = slope_row_groups(p.rows, p.cols);
    const dim3 grid((uint32_t)((p.dz_pitch + COLS * 8 - 1) / (COLS * 8)), groups), block(COLS, LANES);
    if (dt == DType::F32) loss_gradient_kernel<float><<<grid, block, 0, stream>>>(p);
    else loss_gradient_kernel<Bf16><<<grid, block, 0, stream>>>(p);
    hipError_t err = hipGetLastError();
    if (err == hipSuccess && p.sums) err = launch_column_join(dt, p.sums, groups, p.cols, p.dbias, stream);
    return err;
}

hipError_t launch_loss_join(const LossArgs& p, int rows, int runs, float* lse, float* loss, hipStream_t stream)
{
    if (rows <= FEW_ROWS) {
        loss_join_kernel<1><<<rows, dim3(1, 1024), 0, stream>>>(p, rows, runs, lse, loss);
        return hipGetLastError();
    }
    const int64_t grid = ((int64_t)rows + 15) / 16;
    loss_join_kernel<16><<<(uint32_t)(grid < 1 << 20 ? grid : 1 << 20), dim3(16, 64), 0, stream>>>(p, rows, runs, lse, loss);
    return hipGetLastError();
}

hipError_t launch_loss_reduce(const LossArgs& p, int rows, const float* loss, bool mean, float* total, float* count,
                              hipStream_t stream)
{
    loss_reduce_kernel<<<1, 1024, 0, stream>>>(p, rows, loss, mean, total, count);
    return hipGetLastError();
}

}  // namespace miconv
