// The attention on the matrix cores in bf16, over a cache of bf16.
#include "attn_tile_impl.h"

namespace tpl {

hipError_t launch_attention_bf16(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s) {
    return launch_by_size<2, 2>(a, p, dma, s);
}

}  // namespace tpl
