// k_attn_f32.hip -- linear attention over chunks, f32 tensors (attn_chunk.h).
#include "attn_chunk.h"

namespace rnnhip {

hipError_t launch_attn_chunks_f32(const AttnArgs& a, bool local, hipStream_t s) { return attn_chunks<float>(a, local, s); }
hipError_t launch_attn_walks_f32(const AttnArgs* w, int n, int K, hipStream_t s) { return attn_walks<float>(w, n, K, s); }

}  // namespace rnnhip
