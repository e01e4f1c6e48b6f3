// Decode attention, heads of 64 values.
#include "decode.cuh"

namespace pkv {
cudaError_t launch_decode_d64(const DecodeArgs& a, int dtype, bool fused, cudaStream_t stream) {
  return launch_decode_dim<64>(a, dtype, fused, stream);
}
}  // namespace pkv
