// layer_mm_bf16.hip -- the layers' matrix products over bf16 values.
#include "layer_mm.h"

namespace gsm {

gs_status launch_layer_mm_bf16(gs_ctx* ctx, const LayerMm& g)
{
    return launch_layer_mm<bf16, 1, Large16, Medium16, Small16, Tiny16>(ctx, g);
}

gs_status launch_layer_pair_bf16(gs_ctx* ctx, const LayerMm& x, const LayerMm& w)
{
    return launch_layer_pair<bf16, 1, Small16>(ctx, x, w);
}

}  // namespace gsm
