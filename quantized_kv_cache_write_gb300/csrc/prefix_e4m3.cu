// Shared-prefix decode attention over e4m3 pools (see prefix_attn.cuh).
#include "prefix_attn.cuh"

namespace qkv {

cudaError_t launch_prefix_mma_e4m3(const PrefixArgs& a, bool overlaps, cudaStream_t stream) {
  return prefix::launch_mma<QKV_E4M3>(a, overlaps, stream);
}

}  // namespace qkv
