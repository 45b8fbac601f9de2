// linear_fast_loss.hip -- a classifier's logits on large tiles: reduced to its rows' softmax statistics, turned into the
// loss's gradient, or as they are in fp32.
#include "linear_fast_launch.h"

namespace miconv {

hipError_t launch_product_fast_loss(Product kind, ProductType type, const ProductArgs& p, FastTile tile, hipStream_t stream)
{
    if (type == ProductType::BF16_F32)
        return kind == Product::FORWARD ? launch_one<MulBf16F32, false, false, EPI_LINEAR>(p, tile, stream) : hipErrorInvalidValue;
    if (type == ProductType::BF16)
        return kind == Product::LOSS ? launch_one<MulBf16, false, false, EPI_LOSS>(p, tile, stream)
                                     : launch_one<MulBf16, false, false, EPI_LOGITS_GRAD>(p, tile, stream);
    if (type == ProductType::F32)
        return kind == Product::LOSS ? launch_one<MulF32, false, false, EPI_LOSS>(p, tile, stream)
                                     : launch_one<MulF32, false, false, EPI_LOGITS_GRAD>(p, tile, stream);
    return hipErrorInvalidValue;
}

// BN / WN of launch_one's tiles
int loss_columns(ProductType type, FastTile tile)
{
    if (type == ProductType::F32) return 32;
    return tile == FastTile::T256x192 ? 96 : tile == FastTile::T128x128 ? 32 : 64;
}

}  // namespace miconv
