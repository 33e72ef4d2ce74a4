// Masked attention on tcgen05 over int8_side pools (see prefix_umma.cuh).
#include "prefix_umma.cuh"

namespace qkv {

cudaError_t launch_masked_umma_int8_side(const PrefixArgs& a, cudaStream_t stream) { return prefix::launch_masked_umma<QKV_INT8_SIDE>(a, stream); }

}  // namespace qkv
