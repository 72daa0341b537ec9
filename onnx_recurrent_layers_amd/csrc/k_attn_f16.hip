// k_attn_f16.hip -- linear attention over chunks, f16 tensors (attn_chunk.h).
#include "attn_chunk.h"

namespace rnnhip {

hipError_t launch_attn_chunks_f16(const AttnArgs& a, bool local, hipStream_t s) { return attn_chunks<f16_t>(a, local, s); }
hipError_t launch_attn_walks_f16(const AttnArgs* w, int n, int K, hipStream_t s) { return attn_walks<f16_t>(w, n, K, s); }

}  // namespace rnnhip
