// The attention on the matrix cores in fp32, over a cache in 8 bits.
#include "attn_tile_impl.h"

namespace tpl {

hipError_t launch_attention_f32_int8(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s) {
    return launch_by_size<4, 1>(a, p, dma, s);
}

}  // namespace tpl
