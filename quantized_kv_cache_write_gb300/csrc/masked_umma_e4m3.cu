// Masked attention on tcgen05 over e4m3 pools (see prefix_umma.cuh).
#include "prefix_umma.cuh"

namespace qkv {

cudaError_t launch_masked_umma_e4m3(const PrefixArgs& a, cudaStream_t stream) { return prefix::launch_masked_umma<QKV_E4M3>(a, stream); }

}  // namespace qkv
