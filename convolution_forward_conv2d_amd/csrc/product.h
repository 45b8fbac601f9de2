// product.h -- how the feed-forward operators' products are priced, chosen and run (linear.cpp), for the files that put
// calls together from them.
#pragma once

#include <string.h>

#include "host_checks.h"
#include "kernels.h"
#include "linear_common.h"

namespace miconv {

// How a product runs.
struct Plan {
    bool few;                // linear_few.hip
    bool fast;               // linear_fast.h, else linear_any.hip
    FastTile fast_tile;
    int tile;                // linear_any.hip's
    int splits;
    int64_t part_ld;
    int64_t pack_a, pack_b;  // bytes of a packed operand's row, 0: read where it is
    size_t a_bytes, b_bytes; // of the packed copies (b_bytes: each of a gated layer's two)
    size_t bytes;            // workspace: the copies, then the partial sums
    double us;
};

constexpr double kLaunchUs = 4.0, kBytesPerUs = 4.0e6;       // a launch; memory's rate for copies and partial sums

inline int element_bytes(ProductType t)
{
    return t == ProductType::F32 ? 4 : t == ProductType::BF16 || t == ProductType::BF16_F32 ? 2 : 1;
}

// The cheapest way through a product of m x n outputs and k_segments * k terms.
// `aligned_a` / `aligned_b`: the operand's rows can be read 16 bytes at a time.
// `least_splits`: the parts the reduction has at least.
Plan plan_product(int num_cu, Product kind, ProductType type, int m, int n, int k, int k_segments, bool aligned_a,
                  bool aligned_b, int least_splits = 1);

// Whether any kernel's grid holds the product.
inline bool planned(const Plan& pl) { return pl.us < 1e30; }

// "fast 256x192 split 2 pack a", for the calls that say how a product runs.
void describe(const Plan& pl, char* text, size_t size);

// Where a product's sums are if they are not joined: `splits` matrices of rows of `ld`, one after the other.
struct Sums {
    const float* data;
    int64_t ld;
    int splits;
};

// Runs p in the workspace, in p.splits parts at least.  sums: the outputs are fp32 in p.y, or left there in parts.
mic_status run_product(mic_handle h, Product kind, ProductType type, ProductArgs& p, void* workspace, size_t bytes,
                       Sums* sums = nullptr);

// Runs a cross entropy's dx and dw in one launch, on operands that are aligned.
mic_status run_pair(mic_handle h, ProductType type, ProductArgs& dx, ProductArgs& dw);

inline mic_status give_name(const char* text, char* buf, size_t buflen)
{
    const size_t len = strlen(text);
    if (!buf || len + 1 > buflen) return MIC_STATUS_BAD_PARAM;
    memcpy(buf, text, len + 1);
    return MIC_STATUS_SUCCESS;
}

inline int cus_of(mic_handle h) { return h ? h->num_cu : kCuCounts[0]; }

// A matrix that counts as aligned (its rows' length is looked at where it matters).
inline bool aligned_matrix(const void* p, int64_t ld_bytes)
{
    return aligned(p, 16) && ld_bytes % 16 == 0 && ld_bytes < kMaxPitchBytes / 2;
}

}  // namespace miconv
