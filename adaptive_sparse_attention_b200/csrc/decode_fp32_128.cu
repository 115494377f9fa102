// The decode kernels for fp32 caches with d = 128 (a file each, to compile side by side).
#include "decode.cuh"

namespace ea {
cudaError_t launch_decode_fp32_128(const DecodeProblem& P, cudaStream_t s) {
  return launch_decode_t<float, 128>(P, s);
}
}  // namespace ea
