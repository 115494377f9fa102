// The decode kernels for bf16 caches with d = 64 (a file each, to compile side by side).
#include "decode.cuh"

namespace ea {
cudaError_t launch_decode_bf16_64(const DecodeProblem& P, cudaStream_t s) {
  return launch_decode_t<__nv_bfloat16, 64>(P, s);
}
}  // namespace ea
