// linear_fast_grad.hip -- dz W and dz^T x on large tiles.
#include "linear_fast_launch.h"

namespace miconv {

hipError_t launch_product_fast_grad(Product kind, const ProductArgs& p, FastTile tile, hipStream_t stream)
{
    return kind == Product::INPUT_GRAD ? launch_one<MulBf16, false, true, EPI_PLAIN>(p, tile, stream)
                                       : launch_one<MulBf16, true, true, EPI_PLAIN>(p, tile, stream);
}

}  // namespace miconv
