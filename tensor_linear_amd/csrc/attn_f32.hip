// The attention on the matrix cores in fp32, over a cache of fp32.
#include "attn_tile_impl.h"

namespace tpl {

hipError_t launch_attention_f32(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s) {
    return launch_by_size<4, 4>(a, p, dma, s);
}

}  // namespace tpl
