// host_checks.h -- what the C entries of the feed-forward operators check and answer with.
#pragma once

#include <stdint.h>

#include <algorithm>

#include <hip/hip_runtime.h>

#include "miconv.h"
#include "handle.h"
#include "kernels.h"

namespace miconv {

constexpr int kMaxSize = 1 << 30;
constexpr int64_t kMaxPitchBytes = int64_t(1) << 23;   // 256 rows of a tile stay inside a 32-bit offset

inline size_t size_of(mic_dtype d) { return d == MIC_DTYPE_F32 ? 4 : d == MIC_DTYPE_BF16 ? 2 : 1; }
inline bool plain_type(mic_dtype d) { return d == MIC_DTYPE_F32 || d == MIC_DTYPE_BF16; }
inline DType device_type(mic_dtype d) { return d == MIC_DTYPE_F32 ? DType::F32 : DType::BF16; }

// The compute units a handle may have: an MI355X whole and in its two, four and eight partitions.  Host-only calls
// need no device: without a handle they answer for every one of these.
constexpr int kCuCounts[] = {256, 128, 64, 32};

template <class Bytes> size_t most_bytes(mic_handle h, Bytes bytes)
{
    if (h) return bytes(h->num_cu);
    size_t most = 0;
    for (int cus : kCuCounts) most = std::max(most, bytes(cus));
    return most;
}

inline int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline mic_status check_sizes(int m, int n, int k)
{
    if (m < 0 || n < 0 || k < 0) return MIC_STATUS_BAD_PARAM;
    return m >= kMaxSize || n >= kMaxSize || k >= kMaxSize ? MIC_STATUS_NOT_SUPPORTED : MIC_STATUS_SUCCESS;
}

// One matrix of rows x cols elements of `size` bytes.
inline mic_status check_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, size_t size)
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

inline mic_status launched(hipError_t e) { return e == hipSuccess ? MIC_STATUS_SUCCESS : MIC_STATUS_LAUNCH_FAILED; }

}  // namespace miconv
