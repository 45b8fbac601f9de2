// linear_fast_loss.hip -- a classifier's logits on large tiles: reduced to its rows' softmax statistics, turned into the
// loss's gradient, or as they are in fp32; and dz W of one piece of the classes, added to the others'.
#include "linear_fast_launch.h"

namespace miconv {

template <class Mul> static hipError_t launch_kind(Product kind, const ProductArgs& p, FastTile tile, hipStream_t stream)
{
    switch (kind) {
    case Product::LOSS: return launch_one<Mul, false, false, EPI_LOSS>(p, tile, stream);
    case Product::LOGITS_GRAD: return launch_one<Mul, false, false, EPI_LOGITS_GRAD>(p, tile, stream);
    case Product::INPUT_SUM: return launch_one<Mul, false, true, EPI_SUM>(p, tile, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_product_fast_loss(Product kind, ProductType type, const ProductArgs& p, FastTile tile, hipStream_t stream)
{
    if (type == ProductType::BF16_F32)
        return kind == Product::FORWARD ? launch_one<MulBf16F32, false, false, EPI_LINEAR>(p, tile, stream) : hipErrorInvalidValue;
    if (type == ProductType::BF16) return launch_kind<MulBf16>(kind, p, tile, stream);
    if (type == ProductType::F32) return launch_kind<MulF32>(kind, p, tile, stream);
    return hipErrorInvalidValue;
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
