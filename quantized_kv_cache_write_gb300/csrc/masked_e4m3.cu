// Masked attention over e4m3 pools (see prefix_attn.cuh).
#include "prefix_attn.cuh"

namespace qkv {

cudaError_t launch_masked_mma_e4m3(const PrefixArgs& a, cudaStream_t stream) { return prefix::launch_mma<QKV_E4M3, true>(a, false, stream); }

}  // namespace qkv
