// Shared-prefix decode attention over bf16 pools (see prefix_attn.cuh).
#include "prefix_attn.cuh"

namespace qkv {

cudaError_t launch_prefix_mma_bf16(const PrefixArgs& a, bool overlaps, cudaStream_t stream) {
  return prefix::launch_mma<QKV_BF16>(a, overlaps, stream);
}

}  // namespace qkv
