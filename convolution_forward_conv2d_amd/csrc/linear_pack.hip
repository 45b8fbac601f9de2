// linear_pack.hip -- rows at any pitch and alignment into 16-byte aligned rows
// with zeros behind them, for the kernels that load straight into LDS.
#include "linear_common.h"
#include "kernels.h"

namespace miconv {

namespace {

__global__ __launch_bounds__(256) void pack_kernel(const uint8_t* from, int64_t from_pitch, int rows, int64_t bytes,
                                                   uint8_t* to, int64_t pitch)
{
    const int64_t per = pitch / 16;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < rows * per; i += gridDim.x * 256ll) {
        const int64_t r = i / per, c = i % per * 16;
        const uint8_t* p = from + r * from_pitch + c;
        u32x4 v = {0, 0, 0, 0};
        if (c + 16 <= bytes) {
            __builtin_memcpy(&v, p, 16);
        } else {
            const int n = (int)(bytes - c);
#pragma unroll
            for (int b = 0; b < 16; ++b)
                if (b < n) v[b >> 2] |= (uint32_t)p[b] << (8 * (b & 3));
        }
        *reinterpret_cast<u32x4*>(to + r * pitch + c) = v;
    }
}

}  // namespace

hipError_t launch_pack(const void* from, int64_t from_pitch, int rows, int64_t bytes, void* to, int64_t pitch,
                       hipStream_t stream)
{
    const int64_t work = rows * (pitch / 16);
    const int blocks = (int)(work / 256 + 1 < 8192 ? work / 256 + 1 : 8192);
    pack_kernel<<<blocks, 256, 0, stream>>>(static_cast<const uint8_t*>(from), from_pitch, rows, bytes,
                                            static_cast<uint8_t*>(to), pitch);
    return hipGetLastError();
}

}  // namespace miconv
