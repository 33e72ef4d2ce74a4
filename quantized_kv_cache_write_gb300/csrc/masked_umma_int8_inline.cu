// Masked attention on tcgen05 over int8_inline pools (see prefix_umma.cuh).
#include "prefix_umma.cuh"

namespace qkv {

cudaError_t launch_masked_umma_int8_inline(const PrefixArgs& a, cudaStream_t stream) { return prefix::launch_masked_umma<QKV_INT8_INLINE>(a, stream); }

}  // namespace qkv
