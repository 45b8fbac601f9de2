// linear_fast_loss.hip -- a classifier's logits on large tiles: reduced to its rows' softmax statistics, turned into the
// loss's gradient, or as they are in fp32; and dz W of one piece of the classes, added to the others'.
//
// Bound by power on large products: 4096 x 50021 of 4096 terms 1192 us, 1.41 PFLOP/s, matrix units 76 percent busy at 1.7
// GHz; its dz 1270, dx 1140, dw 1260.
#include "linear_chain.h"
#include "linear_fast_launch.h"

namespace miconv {

namespace {

// A tile and how its eight waves share it: rows and columns of waves.  The kernels' arguments and what the host counts
// by (loss_columns, loss_rows) both come from here.
struct LossTile {
    int bm, bn, wm, wn;
};
constexpr LossTile loss_tile(FastTile tile)
{
    switch (tile) {
    case FastTile::T256x256: return {256, 256, 2, 4};
    case FastTile::T256x192: return {256, 192, 4, 2};
    case FastTile::T192x256: return {192, 256, 2, 4};
    case FastTile::T256x128: return {256, 128, 4, 2};
    case FastTile::T128x256: return {128, 256, 2, 4};
    case FastTile::T128x128: return {128, 128, 2, 4};
    case FastTile::T128x64: return {128, 64, 4, 2};
    case FastTile::T64x128: return {64, 128, 2, 4};
    default: return {1, 1, 1, 1};
    }
}
constexpr bool has_tile(bool f32, FastTile tile)
{
    const bool small = tile == FastTile::T128x64 || tile == FastTile::T64x128;
    return tile == FastTile::T128x128 || small == f32;
}

template <class Mul, bool AACROSS, bool BACROSS, int EPI, FastTile TILE>
hipError_t launch_chain(const LossProductArgs& p, hipStream_t stream)
{
    if constexpr (!has_tile(Mul::E == 4, TILE)) {
        return hipErrorInvalidValue;
    } else {
        constexpr LossTile t = loss_tile(TILE);
        const int64_t tiles = (int64_t)((p.M + t.bm - 1) / t.bm) * ((p.N + t.bn - 1) / t.bn);
        if (tiles > INT32_MAX) return hipErrorInvalidValue;
        // as many workgroups as the CUs hold: two of up to 80 KB of LDS
        const int64_t grid = (int64_t)p.cus * (3 * t.bm + 2 * t.bn <= 640 ? 2 : 1);
        linear_chain_kernel<Mul, AACROSS, BACROSS, EPI, t.bm, t.bn, t.wm, t.wn>
            <<<(uint32_t)(tiles < grid ? tiles : grid), FAST_THREADS, 0, stream>>>(p);
        return hipGetLastError();
    }
}

template <class Mul, bool AACROSS, bool BACROSS, int EPI>
hipError_t launch_chains(const ProductArgs& args, FastTile tile, hipStream_t stream)
{
    const auto& p = static_cast<const LossProductArgs&>(args);
    switch (tile) {
    case FastTile::T256x256: return launch_chain<Mul, AACROSS, BACROSS, EPI, FastTile::T256x256>(p, stream);
    case FastTile::T256x192: return launch_chain<Mul, AACROSS, BACROSS, EPI, FastTile::T256x192>(p, stream);
    case FastTile::T192x256: return launch_chain<Mul, AACROSS, BACROSS, EPI, FastTile::T192x256>(p, stream);
    case FastTile::T256x128: return launch_chain<Mul, AACROSS, BACROSS, EPI, FastTile::T256x128>(p, stream);
    case FastTile::T128x256: return launch_chain<Mul, AACROSS, BACROSS, EPI, FastTile::T128x256>(p, stream);
    case FastTile::T128x128: return launch_chain<Mul, AACROSS, BACROSS, EPI, FastTile::T128x128>(p, stream);
    case FastTile::T128x64: return launch_chain<Mul, AACROSS, BACROSS, EPI, FastTile::T128x64>(p, stream);
    case FastTile::T64x128: return launch_chain<Mul, AACROSS, BACROSS, EPI, FastTile::T64x128>(p, stream);
    default: return hipErrorInvalidValue;
    }
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
    constexpr LossTile t = loss_tile(FastTile::T128x128);
    auto tiles = [](const ProductArgs& p) { return (uint32_t)((p.M + t.bm - 1) / t.bm) * ((p.N + t.bn - 1) / t.bn); };
    const uint32_t first = tiles(a), grid = first + tiles(b);
    if (type == ProductType::BF16)
        linear_pair_kernel<MulBf16, t.bm, t.bn, t.wm, t.wn><<<grid, FAST_THREADS, 0, stream>>>(a, b, (int)first);
    else if (type == ProductType::F32)
        linear_pair_kernel<MulF32, t.bm, t.bn, t.wm, t.wn><<<grid, FAST_THREADS, 0, stream>>>(a, b, (int)first);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

int loss_columns(FastTile tile) { return loss_tile(tile).bn / loss_tile(tile).wn; }
int loss_rows(FastTile tile) { return loss_tile(tile).bm / loss_tile(tile).wm; }

}  // namespace miconv
