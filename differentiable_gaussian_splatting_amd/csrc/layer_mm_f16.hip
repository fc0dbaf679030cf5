// layer_mm_f16.hip -- the layers' matrix products over f16 values.
#include "layer_mm.h"

namespace gsm {

gs_status launch_layer_mm_f16(gs_ctx* ctx, const LayerMm& g)
{
    return launch_layer_mm<f16, 1, Large16, Medium16, Small16, Tiny16>(ctx, g);
}

gs_status launch_layer_pair_f16(gs_ctx* ctx, const LayerMm& x, const LayerMm& w)
{
    return launch_layer_pair<f16, 1, Small16>(ctx, x, w);
}

}  // namespace gsm
