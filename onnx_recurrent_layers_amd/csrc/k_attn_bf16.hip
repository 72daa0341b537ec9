// k_attn_bf16.hip -- linear attention over chunks, bf16 tensors (attn_chunk.h).
#include "attn_chunk.h"

namespace rnnhip {

hipError_t launch_attn_chunks_bf16(const AttnArgs& a, bool local, hipStream_t s) { return attn_chunks<bf16_t>(a, local, s); }
hipError_t launch_attn_walks_bf16(const AttnArgs* w, int n, int K, hipStream_t s) { return attn_walks<bf16_t>(w, n, K, s); }

}  // namespace rnnhip
