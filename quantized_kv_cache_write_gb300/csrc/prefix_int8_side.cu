// Shared-prefix decode attention over int8_side pools (see prefix_attn.cuh).
#include "prefix_attn.cuh"

namespace qkv {

cudaError_t launch_prefix_mma_int8_side(const PrefixArgs& a, bool overlaps, cudaStream_t stream) {
  return prefix::launch_mma<QKV_INT8_SIDE>(a, overlaps, stream);
}

}  // namespace qkv
