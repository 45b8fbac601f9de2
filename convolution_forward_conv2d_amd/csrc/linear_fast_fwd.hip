// linear_fast_fwd.hip -- x W^T of linear and gated layers on large tiles.
#include "linear_fast_launch.h"

namespace miconv {

hipError_t launch_product_fast(Product kind, ProductType type, const ProductArgs& p, FastTile tile, hipStream_t stream)
{
    if (kind == Product::INPUT_GRAD || kind == Product::WEIGHT_GRAD)
        return launch_product_fast_grad(kind, type, p, tile, stream);
    if ((kind != Product::FORWARD && kind != Product::GATED) || type == ProductType::BF16_F32)
        return launch_product_fast_loss(kind, type, p, tile, stream);
    const bool gated = kind == Product::GATED;
    switch (type) {
    case ProductType::BF16:
        return gated ? launch_one<MulBf16, false, false, EPI_GATED>(p, tile, stream)
                     : launch_one<MulBf16, false, false, EPI_LINEAR>(p, tile, stream);
    case ProductType::F32:
        return gated ? launch_one<MulF32, false, false, EPI_GATED>(p, tile, stream)
                     : launch_one<MulF32, false, false, EPI_LINEAR>(p, tile, stream);
    case ProductType::E4M3_BF16:
        return gated ? launch_one<MulE4m3<Bf16, false>, false, false, EPI_GATED>(p, tile, stream)
                     : launch_one<MulE4m3<Bf16, false>, false, false, EPI_LINEAR>(p, tile, stream);
    case ProductType::E4M3_F32:
        return gated ? launch_one<MulE4m3<float, false>, false, false, EPI_GATED>(p, tile, stream)
                     : launch_one<MulE4m3<float, false>, false, false, EPI_LINEAR>(p, tile, stream);
    case ProductType::E4M3_BF16_SHORT:
        return gated ? launch_one<MulE4m3<Bf16, true>, false, false, EPI_GATED>(p, tile, stream)
                     : launch_one<MulE4m3<Bf16, true>, false, false, EPI_LINEAR>(p, tile, stream);
    case ProductType::E4M3_F32_SHORT:
        return gated ? launch_one<MulE4m3<float, true>, false, false, EPI_GATED>(p, tile, stream)
                     : launch_one<MulE4m3<float, true>, false, false, EPI_LINEAR>(p, tile, stream);
    default: break;
    }
    return hipErrorInvalidValue;
}

}  // namespace miconv
