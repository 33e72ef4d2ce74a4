// Append with rotation by one position per token (see append.cuh).
#include "append.cuh"

namespace qkv {

cudaError_t launch_append_rope(const AppendArgs& a, qkv_format fmt, bool f16, cudaStream_t stream) {
  return launch<false>(a, fmt, f16, stream);
}

}  // namespace qkv
