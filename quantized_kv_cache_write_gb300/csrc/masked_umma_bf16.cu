// Masked attention on tcgen05 over bf16 pools (see prefix_umma.cuh).
#include "prefix_umma.cuh"

namespace qkv {

cudaError_t launch_masked_umma_bf16(const PrefixArgs& a, cudaStream_t stream) { return prefix::launch_masked_umma<QKV_BF16>(a, stream); }

}  // namespace qkv
