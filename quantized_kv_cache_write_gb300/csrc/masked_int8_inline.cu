// Masked attention over int8_inline pools (see prefix_attn.cuh).
#include "prefix_attn.cuh"

namespace qkv {

cudaError_t launch_masked_mma_int8_inline(const PrefixArgs& a, cudaStream_t stream) { return prefix::launch_mma<QKV_INT8_INLINE, true>(a, false, stream); }

}  // namespace qkv
