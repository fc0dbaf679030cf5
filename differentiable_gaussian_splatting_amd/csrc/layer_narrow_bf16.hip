// layer_narrow_bf16.hip -- narrow linear layers over bf16 values.
#include "layer_narrow.h"

namespace gsm {

void launch_narrow_fwd_bf16(gs_ctx* ctx, const LayerMm& g) { launch_narrow_fwd<bf16>(ctx, g); }
void launch_narrow_bwd_bf16(gs_ctx* ctx, const NarrowBwd& g, int64_t blocks) { launch_narrow_bwd<bf16>(ctx, g, blocks); }

}  // namespace gsm
