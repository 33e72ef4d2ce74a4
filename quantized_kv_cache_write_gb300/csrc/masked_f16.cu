// Masked attention over f16 pools (see prefix_attn.cuh).
#include "prefix_attn.cuh"

namespace qkv {

cudaError_t launch_masked_mma_f16(const PrefixArgs& a, cudaStream_t stream) { return prefix::launch_mma<QKV_F16, true>(a, false, stream); }

}  // namespace qkv
