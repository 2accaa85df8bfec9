// Decode over the bf16 cache with block weights (the kernel is in decode_list.cuh).
#include "decode_list.cuh"

namespace minipic {

using decode_list::launch_d;

cudaError_t launch_decode_weights(const DecodeArgs& a, cudaStream_t s) {
  return a.D == 128 ? launch_d<false, 128, true>(a, s) : launch_d<false, 64, true>(a, s);
}

}  // namespace minipic
