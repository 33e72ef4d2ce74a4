// The shared prefix on tcgen05 over f16 pools (see prefix_umma.cuh).
#include "prefix_umma.cuh"

namespace qkv {

cudaError_t launch_prefix_umma_f16(const PrefixArgs& a, cudaStream_t stream) { return prefix::launch_umma<QKV_F16>(a, stream); }

}  // namespace qkv
