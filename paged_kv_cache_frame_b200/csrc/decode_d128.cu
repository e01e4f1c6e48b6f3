// Decode attention, heads of 128 values.
#include "decode.cuh"

namespace pkv {
cudaError_t launch_decode_d128(const DecodeArgs& a, int dtype, bool fused, cudaStream_t stream) {
  return launch_decode_dim<128>(a, dtype, fused, stream);
}
}  // namespace pkv
