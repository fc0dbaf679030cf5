// layer_narrow_f32.hip -- narrow linear layers over f32 values.
#include "layer_narrow.h"

namespace gsm {

bool launch_narrow_fwd_f32(gs_ctx* ctx, const LayerMm& g) { return launch_narrow_fwd<float>(ctx, g); }
bool launch_narrow_bwd_f32(gs_ctx* ctx, const NarrowBwd& g, int64_t blocks) { return launch_narrow_bwd<float>(ctx, g, blocks); }

}  // namespace gsm
