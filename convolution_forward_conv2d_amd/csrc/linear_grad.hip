// linear_grad.hip -- between the gradient of a layer's output and its two
// products:
//
//   linear   dz = dy act'(z)                      dbias = sum over rows of dz
//   gated    dgate = dy up act'(gate)             dup = dy act(gate)
//
// One pass, bound by memory: each input read once, dz written once.  dz is
// rounded to the tensors' type, since the matrix instructions that take it
// multiply nothing wider; dbias sums it in fp32 before that rounding.  A gated
// layer's 4096 x 9216 take 72 us, 5.2 TB/s, a copy's rate.
#include "linear_common.h"
#include "kernels.h"

namespace miconv {

namespace {

constexpr int COLS = 32;           // groups of eight columns per block: lines of 512 bytes in bf16
constexpr int LANES = 8;           // rows a block walks side by side

template <class T, bool GATED>
__global__ __launch_bounds__(COLS * LANES) void slope_kernel(const SlopeArgs p)
{
    constexpr bool EXACT = sizeof(T) == 4;
    const int c = (blockIdx.x * COLS + threadIdx.x) * 8;
    const int padded = (int)(GATED ? p.up_at : p.dz_pitch);
    const int nv = p.cols - c;
    float total[8] = {};
    if (c < (p.dz ? padded : p.cols)) {
        for (int r = blockIdx.y * LANES + threadIdx.y; r < p.rows; r += gridDim.y * LANES) {
            float d[8], z[8], u[8];
            load8(static_cast<const T*>(p.dy) + (int64_t)r * p.lddy + c, nv, d);
            if (p.pre) load8(static_cast<const T*>(p.pre) + (int64_t)r * p.ldp + c, nv, z);
            if constexpr (GATED) load8(static_cast<const T*>(p.up) + (int64_t)r * p.ldu + c, nv, u);
            if (p.pre) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float value, slope;
                    act_both<EXACT>(p.act, z[i], value, slope);
                    if constexpr (GATED) {
                        z[i] = d[i] * value;               // dup
                        d[i] *= u[i] * slope;              // dgate
                    } else {
                        d[i] *= slope;
                    }
                    if (i >= nv) d[i] = z[i] = 0.0f;
                }
            }
            if (p.dz) {
                T* out = static_cast<T*>(p.dz) + (int64_t)r * p.dz_pitch + c;
                store8(out, 8, d);
                if constexpr (GATED) store8(out + p.up_at, 8, z);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) total[i] += d[i];
        }
    }
    if constexpr (!GATED) {
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
        if (col < p.cols) p.sums[(int64_t)blockIdx.y * p.cols + col] = s;
    }
}

// Sixteen columns a block, 64 lanes of rows: blocks enough to fill the chip from 4096 columns on (with 64 columns a
// block, 1024 rows of 4096 partial sums took 16.9 us).
template <class T>
__global__ __launch_bounds__(1024) void column_join_kernel(const float* partial, int groups, int cols, T* out)
{
    __shared__ float part[64][17];
    const int c = blockIdx.x * 16 + threadIdx.x;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 4
        for (int g = threadIdx.y; g < groups; g += 64) s += partial[(int64_t)g * cols + c];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y < 4) {
        s = 0.0f;
#pragma unroll
        for (int y = 0; y < 16; ++y) s += part[16 * threadIdx.y + y][threadIdx.x];
    }
    // the first wave holds four sums a column, in lanes 16 apart
    if (threadIdx.y >= 4) return;
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (threadIdx.y == 0 && c < cols) out[c] = from_f32<T>(s);
}

}  // namespace

int slope_row_groups(int rows, int cols)
{
    // enough blocks for eight to a CU, down to one row a lane: rows one after another wait for memory each
    const int wide = cols > 0 ? (cols + COLS * 8 - 1) / (COLS * 8) : 1;
    const int want = (2048 + wide - 1) / wide;
    const int most = (rows + LANES - 1) / LANES;
    return want < most ? want : (most > 1 ? most : 1);
}

hipError_t launch_column_join(DType dt, const float* partial, int groups, int cols, void* out, hipStream_t stream)
{
    const dim3 grid((cols + 15) / 16), block(16, 64);
    if (dt == DType::F32)
        column_join_kernel<<<grid, block, 0, stream>>>(partial, groups, cols, static_cast<float*>(out));
    else
        column_join_kernel<<<grid, block, 0, stream>>>(partial, groups, cols, static_cast<Bf16*>(out));
    return hipGetLastError();
}

hipError_t launch_slope(DType dt, const SlopeArgs& p, hipStream_t stream)
{
    const int64_t wide = p.dz ? (p.up ? p.up_at : p.dz_pitch) : p.cols;
    const int groups = slope_row_groups(p.rows, p.cols);
    const dim3 grid((uint32_t)((wide + COLS * 8 - 1) / (COLS * 8)), groups), block(COLS, LANES);
    if (dt == DType::F32) {
        if (p.up) slope_kernel<float, true><<<grid, block, 0, stream>>>(p);
        else slope_kernel<float, false><<<grid, block, 0, stream>>>(p);
    } else {
        if (p.up) slope_kernel<Bf16, true><<<grid, block, 0, stream>>>(p);
        else slope_kernel<Bf16, false><<<grid, block, 0, stream>>>(p);
    }
    hipError_t err = hipGetLastError();
    if (err == hipSuccess && p.sums) err = launch_column_join(dt, p.sums, groups, p.cols, p.dbias, stream);
    return err;
}

}  // namespace miconv
