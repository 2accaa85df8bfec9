// Decode over the 8-bit cache (the kernel is in decode_list.cuh).
#include "decode_list.cuh"

namespace minipic {

using decode_list::launch_d;

cudaError_t launch_decode_q8(const DecodeArgs& a, cudaStream_t s) {
  if (a.D == 128) return a.weights ? launch_d<true, 128, true>(a, s) : launch_d<true, 128, false>(a, s);
  return a.weights ? launch_d<true, 64, true>(a, s) : launch_d<true, 64, false>(a, s);
}

}  // namespace minipic
