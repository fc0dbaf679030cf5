// layer_mm_f32.hip -- the layers' matrix products over f32 values.
#include "layer_mm.h"

namespace gsm {

gs_status launch_layer_mm_f32(gs_ctx* ctx, const LayerMm& g)
{
    return launch_layer_mm<float, 3, Tile<128, 128, 32, 2, 2, 2>, Tile<64, 64, 32, 2, 2, 2>>(ctx, g);
}

}  // namespace gsm
