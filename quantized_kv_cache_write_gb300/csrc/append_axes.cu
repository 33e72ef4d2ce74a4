// Append with rotation by several positions per token, a pair's by its axis (see append.cuh).
#include "append.cuh"

namespace qkv {

cudaError_t launch_append_axes(const AppendArgs& a, qkv_format fmt, bool f16, cudaStream_t stream) {
  return launch<true>(a, fmt, f16, stream);
}

}  // namespace qkv
