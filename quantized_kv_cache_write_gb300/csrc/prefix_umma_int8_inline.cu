// The shared prefix on tcgen05 over int8_inline pools (see prefix_umma.cuh).
#include "prefix_umma.cuh"

namespace qkv {

cudaError_t launch_prefix_umma_int8_inline(const PrefixArgs& a, cudaStream_t stream) { return prefix::launch_umma<QKV_INT8_INLINE>(a, stream); }

}  // namespace qkv
