// linear_fast_grad.hip -- dz W and dz^T x on large tiles.
#include "linear_fast_launch.h"

namespace miconv {

template <class Mul> static hipError_t launch_kind(Product kind, const ProductArgs& p, FastTile tile, hipStream_t stream)
{
    return kind == Product::INPUT_GRAD ? launch_one<Mul, false, true, EPI_PLAIN>(p, tile, stream)
                                       : launch_one<Mul, true, true, EPI_PLAIN>(p, tile, stream);
}

hipError_t launch_product_fast_grad(Product kind, ProductType type, const ProductArgs& p, FastTile tile, hipStream_t stream)
{
    if (type == ProductType::BF16) return launch_kind<MulBf16>(kind, p, tile, stream);
    if (type == ProductType::F32) return launch_kind<MulF32>(kind, p, tile, stream);
    return hipErrorInvalidValue;                               // no gradients in e4m3
}

}  // namespace miconv
