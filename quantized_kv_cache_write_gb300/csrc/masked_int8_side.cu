// Masked attention over int8_side pools (see prefix_attn.cuh).
#include "prefix_attn.cuh"

namespace qkv {

cudaError_t launch_masked_mma_int8_side(const PrefixArgs& a, cudaStream_t stream) { return prefix::launch_mma<QKV_INT8_SIDE, true>(a, false, stream); }

}  // namespace qkv
