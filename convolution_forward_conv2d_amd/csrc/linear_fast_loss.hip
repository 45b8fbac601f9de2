// linear_fast_loss.hip -- a classifier's logits on large tiles: reduced to its rows' softmax statistics, turned into the
// loss's gradient, or as they are in fp32; and dz W of one piece of the classes, added to the others'.
//
// Bound by power on large products: 4096 x 50021 of 4096 terms 1192 us, 1.41 PFLOP/s, matrix units 76 percent busy at 1.7
// GHz; its dz 1270, dx 1140, dw 1260.
#include "linear_chain.h"
#include "linear_fast_launch.h"

namespace miconv {

namespace {

template <class Mul, bool AACROSS, bool BACROSS, int EPI, int BM, int BN, int WM, int WN>
hipError_t launch_chain(const LossProductArgs& p, hipStream_t stream)
{
    const int64_t tiles = (int64_t)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    // as many workgroups as the CUs hold: two of up to 80 KB of LDS
    const int64_t grid = (int64_t)p.cus * (3 * BM + 2 * BN <= 640 ? 2 : 1);
    linear_chain_kernel<Mul, AACROSS, BACROSS, EPI, BM, BN, WM, WN>
        <<<(uint32_t)(tiles < grid ? tiles : grid), FAST_THREADS, 0, stream>>>(p);
    return hipGetLastError();
}

template <class Mul, bool AACROSS, bool BACROSS, int EPI>
hipError_t launch_chains(const ProductArgs& args, FastTile tile, hipStream_t stream)
{
    const auto& p = static_cast<const LossProductArgs&>(args);
    if constexpr (Mul::E == 4) switch (tile) {
    case FastTile::T128x128: return launch_chain<Mul, AACROSS, BACROSS, EPI, 128, 128, 2, 4>(p, stream);
    case FastTile::T128x64: return launch_chain<Mul, AACROSS, BACROSS, EPI, 128, 64, 4, 2>(p, stream);
    case FastTile::T64x128: return launch_chain<Mul, AACROSS, BACROSS, EPI, 64, 128, 2, 4>(p, stream);
    default: return hipErrorInvalidValue;
    } else switch (tile) {
    case FastTile::T256x256: return launch_chain<Mul, AACROSS, BACROSS, EPI, 256, 256, 2, 4>(p, stream);
    case FastTile::T256x192: return launch_chain<Mul, AACROSS, BACROSS, EPI, 256, 192, 4, 2>(p, stream);
    case FastTile::T192x256: return launch_chain<Mul, AACROSS, BACROSS, EPI, 192, 256, 2, 4>(p, stream);
    case FastTile::T256x128: return launch_chain<Mul, AACROSS, BACROSS, EPI, 256, 128, 4, 2>(p, stream);
    case FastTile::T128x256: return launch_chain<Mul, AACROSS, BACROSS, EPI, 128, 256, 2, 4>(p, stream);
    case FastTile::T128x128: return launch_chain<Mul, AACROSS, BACROSS, EPI, 128, 128, 2, 4>(p, stream);
    default: break;
    }
    return hipErrorInvalidValue;
}

template <class Mul> hipError_t launch_kind(Product kind, const ProductArgs& p, FastTile tile, hipStream_t stream)
{
    switch (kind) {
    case Product::LOSS: return launch_chains<Mul, false, false, EPI_LOSS>(p, tile, stream);
    case Product::LOGITS_GRAD: return launch_chains<Mul, false, false, EPI_LOGITS_GRAD>(p, tile, stream);
    case Product::CLASS_GRAD: return launch_chains<Mul, true, true, EPI_STORE>(p, tile, stream);
    case Product::INPUT_SUM: return launch_one<Mul, false, true, EPI_SUM>(p, tile, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_product_fast_loss(Product kind, ProductType type, const ProductArgs& p, FastTile tile, hipStream_t stream)
{
    // a split reduction leaves partial sums as any weights' gradient
    if (kind == Product::CLASS_GRAD && p.splits > 1) return launch_product_fast_grad(Product::WEIGHT_GRAD, type, p, tile, stream);
    if (type == ProductType::BF16_F32)
        return kind == Product::FORWARD ? launch_one<MulBf16F32, false, false, EPI_LINEAR>(p, tile, stream) : hipErrorInvalidValue;
    if (type == ProductType::BF16) return launch_kind<MulBf16>(kind, p, tile, stream);
    if (type == ProductType::F32) return launch_kind<MulF32>(kind, p, tile, stream);
    return hipErrorInvalidValue;
}

hipError_t launch_product_pair(ProductType type, const ProductArgs& dx, const ProductArgs& dw, hipStream_t stream)
{
    const auto& a = static_cast<const LossProductArgs&>(dx);
    const auto& b = static_cast<const LossProductArgs&>(dw);
    auto tiles = [](const ProductArgs& p) { return (uint32_t)((p.M + 127) / 128) * ((p.N + 127) / 128); };
    const uint32_t first = tiles(a), grid = first + tiles(b);
    if (type == ProductType::BF16)
        linear_pair_kernel<MulBf16, 128, 128, 2, 4><<<grid, FAST_THREADS, 0, stream>>>(a, b, (int)first);
    else if (type == ProductType::F32)
        linear_pair_kernel<MulF32, 128, 128, 2, 4><<<grid, FAST_THREADS, 0, stream>>>(a, b, (int)first);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

// BN / WN of launch_one's tiles
int loss_columns(ProductType type, FastTile tile)
{
    if (type == ProductType::F32) return 32;
    return tile == FastTile::T256x192 ? 96 : tile == FastTile::T128x128 ? 32 : 64;
}

// BM / WM
int loss_rows(ProductType type, FastTile tile)
{
    if (type == ProductType::F32) return tile == FastTile::T128x128 ? 64 : 32;
    return tile == FastTile::T256x256 ? 128 : tile == FastTile::T192x256 ? 96 : 64;
}

}  // namespace miconv
