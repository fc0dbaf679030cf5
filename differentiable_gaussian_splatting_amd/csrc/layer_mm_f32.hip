// layer_mm_f32.hip -- the layers' matrix products over f32 values.
#include "layer_mm.h"

namespace gsm {

gs_status launch_layer_mm_f32(gs_ctx* ctx, const LayerMm& g)
{
    return launch_layer_mm<float, 3, Large32, Medium32, Small32, Tiny32>(ctx, g);
}

gs_status launch_layer_pair_f32(gs_ctx* ctx, const LayerMm& x, const LayerMm& w)
{
    return launch_layer_pair<float, 3, Small32>(ctx, x, w);
}

}  // namespace gsm
