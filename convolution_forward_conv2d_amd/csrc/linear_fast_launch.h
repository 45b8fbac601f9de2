// linear_fast_launch.h -- the tiles of linear_fast.h, for the files that instantiate them.
#pragma once

#include "linear_fast.h"

namespace miconv {

namespace {

template <class Mul, bool AACROSS, bool BACROSS, int EPI, int BM, int BN, int WM, int WN>
hipError_t launch_tile(const ProductArgs& p, hipStream_t stream)
{
    const int raw_n = EPI == EPI_GATED ? gated_raw_columns(p.N) : p.N;
    const int64_t tiles = (int64_t)((p.M + BM - 1) / BM) * ((raw_n + BN - 1) / BN);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    linear_fast_kernel<Mul, AACROSS, BACROSS, EPI, BM, BN, WM, WN>
        <<<dim3((uint32_t)tiles, 1, (uint32_t)p.splits), FAST_THREADS, 0, stream>>>(static_cast<const ArgsOf<EPI>&>(p));
    return hipGetLastError();
}

template <class Mul, bool AACROSS, bool BACROSS, int EPI>
hipError_t launch_one(const ProductArgs& p, FastTile tile, hipStream_t stream)
{
    // fp32's matrix instructions take sixteen times bf16's time: already small tiles wait for nothing else
    if constexpr (Mul::E == 4) switch (tile) {
    case FastTile::T128x128: return launch_tile<Mul, AACROSS, BACROSS, EPI, 128, 128, 2, 4>(p, stream);
    case FastTile::T128x64: return launch_tile<Mul, AACROSS, BACROSS, EPI, 128, 64, 4, 2>(p, stream);
    case FastTile::T64x128: return launch_tile<Mul, AACROSS, BACROSS, EPI, 64, 128, 2, 4>(p, stream);
    default: return hipErrorInvalidValue;
    } else switch (tile) {
    case FastTile::T256x256: return launch_tile<Mul, AACROSS, BACROSS, EPI, 256, 256, 2, 4>(p, stream);
    case FastTile::T256x192: return launch_tile<Mul, AACROSS, BACROSS, EPI, 256, 192, 4, 2>(p, stream);
    case FastTile::T192x256: return launch_tile<Mul, AACROSS, BACROSS, EPI, 192, 256, 2, 4>(p, stream);
    case FastTile::T256x128: return launch_tile<Mul, AACROSS, BACROSS, EPI, 256, 128, 4, 2>(p, stream);
    case FastTile::T128x256: return launch_tile<Mul, AACROSS, BACROSS, EPI, 128, 256, 2, 4>(p, stream);
    case FastTile::T128x128: return launch_tile<Mul, AACROSS, BACROSS, EPI, 128, 128, 2, 4>(p, stream);
    default: break;
    }
    return hipErrorInvalidValue;
}

}  // namespace

}  // namespace miconv
