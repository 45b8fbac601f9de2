// linear_pack.hip -- rows at any pitch and alignment into 16-byte aligned rows
// with zeros behind them, for the kernels that load straight into LDS.  All of
// a product's operands that need it in one launch: a launch costs as much as
// copying 16 MB.
#include "linear_common.h"
#include "kernels.h"

namespace miconv {

namespace {

struct PackArgs {
    PackJob job[PACK_JOBS];
};

template <class Index> __device__ __forceinline__ void pack(const PackJob& j)
{
    const Index per = (Index)(j.to_pitch / 16), work = (Index)j.rows * per;
    for (Index i = blockIdx.x * (Index)256 + threadIdx.x; i < work; i += gridDim.x * (Index)256) {
        const Index r = i / per;
        const int64_t c = (int64_t)(i - r * per) * 16;
        const uint8_t* p = j.from + (int64_t)r * j.from_pitch + c;
        u32x4 v = {0, 0, 0, 0};
        if (c + 16 <= j.bytes) {
            __builtin_memcpy(&v, p, 16);
        } else {
            const int n = (int)(j.bytes - c);
#pragma unroll
            for (int b = 0; b < 16; ++b)
                if (b < n) v[b >> 2] |= (uint32_t)p[b] << (8 * (b & 3));
        }
        *reinterpret_cast<u32x4*>(j.to + (int64_t)r * j.to_pitch + c) = v;
    }
}

__global__ __launch_bounds__(256) void pack_kernel(const PackArgs a)
{
    const PackJob& j = a.job[blockIdx.y];
    if (j.rows * (j.to_pitch / 16) < (1 << 30)) pack<uint32_t>(j);     // a 64-bit division takes longer than its 16 bytes
    else pack<int64_t>(j);
}

}  // namespace

hipError_t launch_pack(const PackJob* jobs, int count, hipStream_t stream)
{
    PackArgs a = {};
    int64_t most = 0;
    for (int i = 0; i < count; ++i) {
        a.job[i] = jobs[i];
        const int64_t work = jobs[i].rows * (jobs[i].to_pitch / 16);
        most = work > most ? work : most;
    }
    const int blocks = (int)(most / 256 + 1 < 4096 ? most / 256 + 1 : 4096);
    pack_kernel<<<dim3(blocks, count), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace miconv
