// The decode kernels for fp32 caches with d = 64 (a file each, to compile side by side).
#include "decode.cuh"

namespace ea {
cudaError_t launch_decode_fp32_64(const DecodeProblem& P, cudaStream_t s) {
  return launch_decode_t<float, 64>(P, s);
}
}  // namespace ea
