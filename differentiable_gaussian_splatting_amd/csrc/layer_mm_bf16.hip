// layer_mm_bf16.hip -- the layers' matrix products over bf16 values.
#include "layer_mm.h"

namespace gsm {

gs_status launch_layer_mm_bf16(gs_ctx* ctx, const LayerMm& g)
{
    return launch_layer_mm<bf16, 1, Tile<128, 128, 64, 2, 2, 2>, Tile<64, 64, 64, 2, 2, 2>>(ctx, g);
}

}  // namespace gsm
