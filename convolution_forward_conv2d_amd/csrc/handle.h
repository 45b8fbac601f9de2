// handle.h -- what a library handle holds on the host.
#pragma once

#include <hip/hip_runtime.h>

struct mic_handle_st {
    int device;
    int num_cu;
    hipStream_t stream;
};
