// layer_narrow_f32.hip -- narrow linear layers over f32 values.
#include "layer_narrow.h"

namespace gsm {

void launch_narrow_fwd_f32(gs_ctx* ctx, const LayerMm& g) { launch_narrow_fwd<float>(ctx, g); }
void launch_narrow_bwd_f32(gs_ctx* ctx, const NarrowBwd& g, int64_t blocks) { launch_narrow_bwd<float>(ctx, g, blocks); }

}  // namespace gsm
