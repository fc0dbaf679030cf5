// layer_narrow_f16.hip -- narrow linear layers over f16 values.
#include "layer_narrow.h"

namespace gsm {

void launch_narrow_fwd_f16(gs_ctx* ctx, const LayerMm& g) { launch_narrow_fwd<f16>(ctx, g); }
void launch_narrow_bwd_f16(gs_ctx* ctx, const NarrowBwd& g, int64_t blocks) { launch_narrow_bwd<f16>(ctx, g, blocks); }

}  // namespace gsm
