// dropout.hip -- dropout whose mask is computed, never stored:
//
//   y[i] = lot(i) >= least ? x[i] * scale : 0, + residual[i]
//
// lot(i) is a 16-bit number of the element's position i in row-major order: the
// Philox4x32 generator with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011) with the seed as key and the
// counter (i / 8, offset), 64 bits each, whose four words are eight lots, low
// halves first.  So the gradient is the same call on dy, whatever the launch.
//
// Eight lots from one block keep the generator's twenty wide products, a quarter
// of the vector rate each, below memory's time: with four lots of 32 bits a bf16
// row would wait for them.  p is then a multiple of 2^-16.  Bound by memory: 8192 x
// 4096 bf16 with a residual takes 41.7 us, 4.8 TB/s, the gradient of 4095 x 9216
// 29.3, 5.1 TB/s, two vectors of eight a thread and no loop; a call on 128 x 4096 is
// its launch, 4.2.
#include "linear_common.h"
#include "kernels.h"

namespace miconv {

namespace {

struct Lots {
    uint32_t word[4];
    __device__ __forceinline__ uint32_t lot(int i) const { return i & 1 ? word[i >> 1] >> 16 : word[i >> 1] & 0xffffu; }
};

__device__ __forceinline__ Lots philox(uint64_t block, uint64_t seed, uint64_t offset)
{
    uint32_t a = (uint32_t)block, b = (uint32_t)(block >> 32), c = (uint32_t)offset, d = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)a * 0xd2511f53u, q = (uint64_t)c * 0xcd9e8d57u;
        a = (uint32_t)(q >> 32) ^ b ^ k0, b = (uint32_t)q;
        c = (uint32_t)(p >> 32) ^ d ^ k1, d = (uint32_t)p;
        k0 += 0x9e3779b9u, k1 += 0xbb67ae85u;
    }
    return Lots{{a, b, c, d}};
}

// The call's seed and offset: its own, or with those that the caller keeps in device memory.
__device__ __forceinline__ void stream_of(const DropoutArgs& p, uint64_t& seed, uint64_t& offset)
{
    seed = p.seed, offset = p.offset;
    if (p.state) seed = p.state[0], offset += p.state[1];
}

__device__ __forceinline__ void drop8(const DropoutArgs& p, const Lots& lots, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = lots.lot(i) >= p.least ? v[i] * p.scale : 0.0f;
}

constexpr int THREADS = 256, UNROLL = 2;

// Everything packed: one row of p.cols elements, eight a thread and turn.
template <class T> __global__ __launch_bounds__(THREADS) void dropout_kernel(const DropoutArgs p)
{
    uint64_t seed, offset;
    stream_of(p, seed, offset);
    const T* x = static_cast<const T*>(p.x);
    const T* res = static_cast<const T*>(p.residual);
    T* y = static_cast<T*>(p.y);
    const int64_t blocks = (p.cols + 7) / 8;
    for (int64_t at = (int64_t)blockIdx.x * THREADS * UNROLL + threadIdx.x; at < blocks;
         at += (int64_t)gridDim.x * THREADS * UNROLL) {
        float v[UNROLL][8], r[UNROLL][8];
        int nv[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int64_t i = (at + u * THREADS) * 8, left = p.cols - i;
            nv[u] = left > 8 ? 8 : (int)left;                  // <= 0 past the end
            if (left <= 0) continue;
            load8(x + i, nv[u], v[u]);
            if (res) load8(res + i, nv[u], r[u]);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (nv[u] <= 0) continue;
            drop8(p, philox(at + u * THREADS, seed, offset), v[u]);
            if (res) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] += r[u][i];
            }
            store8(y + (at + u * THREADS) * 8, nv[u], v[u]);
        }
    }
}

// Rows apart: a thread still takes the eight positions of one block, which may lie in two or more rows.
template <class T> __global__ __launch_bounds__(THREADS) void dropout_rows_kernel(const DropoutArgs p)
{
    uint64_t seed, offset;
    stream_of(p, seed, offset);
    const T* x = static_cast<const T*>(p.x);
    const T* res = static_cast<const T*>(p.residual);
    T* y = static_cast<T*>(p.y);
    const int64_t count = p.rows * p.cols, blocks = (count + 7) / 8;
    for (int64_t at = (int64_t)blockIdx.x * THREADS + threadIdx.x; at < blocks; at += (int64_t)gridDim.x * THREADS) {
        const Lots lots = philox(at, seed, offset);
        const int64_t first = at * 8;
        int64_t row = first / p.cols, col = first - row * p.cols;
        if (col + 8 <= p.cols) {
            float v[8], r[8];
            load8(x + row * p.ldx + col, 8, v);
            if (res) load8(res + row * p.ldr + col, 8, r);
            drop8(p, lots, v);
            if (res) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += r[i];
            }
            store8(y + row * p.ldy + col, 8, v);
            continue;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (first + i >= count) break;
            float v = to_f32(x[row * p.ldx + col]);
            v = lots.lot(i) >= p.least ? v * p.scale : 0.0f;
            if (res) v += to_f32(res[row * p.ldr + col]);
            y[row * p.ldy + col] = from_f32<T>(v);
            if (++col == p.cols) col = 0, ++row;
        }
    }
}

constexpr int64_t GRID_MOST = 1 << 22;                         // HIP takes grids of fewer than 2^32 threads

template <class T> hipError_t launch_type(const DropoutArgs& p, hipStream_t stream)
{
    const int64_t blocks = (p.rows * p.cols + 7) / 8;
    if (p.rows == 1) {
        const int64_t grid = (blocks + THREADS * UNROLL - 1) / (THREADS * UNROLL);
        dropout_kernel<T><<<(uint32_t)(grid < GRID_MOST ? grid : GRID_MOST), THREADS, 0, stream>>>(p);
    } else {
        const int64_t grid = (blocks + THREADS - 1) / THREADS;
        dropout_rows_kernel<T><<<(uint32_t)(grid < GRID_MOST ? grid : GRID_MOST), THREADS, 0, stream>>>(p);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(DType dt, const DropoutArgs& p, hipStream_t stream)
{
    return dt == DType::F32 ? launch_type<float>(p, stream) : launch_type<Bf16>(p, stream);
}

}  // namespace miconv
