// The attention on the matrix cores in bf16, over a cache in 8 bits.
#include "attn_tile_impl.h"

namespace tpl {

hipError_t launch_attention_bf16_int8(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s) {
    return launch_by_size<2, 1>(a, p, dma, s);
}

}  // namespace tpl
