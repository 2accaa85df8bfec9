// Decode over the selected blocks of the 8-bit cache (the kernel is in decode_list.cuh).
#include "decode_list.cuh"

namespace minipic {

using namespace decode_list;

cudaError_t launch_decode_selected_q8(const DecodeArgs& a, cudaStream_t s) {
  return a.D == 128 ? launch_d<true, 128, false, kSelected>(a, s) : launch_d<true, 64, false, kSelected>(a, s);
}

}  // namespace minipic
