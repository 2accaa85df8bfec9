// Decode of a batch whose requests share prefixes: first form, every request reads all its keys
// (the kernel is in decode_list.cuh).
#include "decode_list.cuh"

namespace minipic {

using namespace decode_list;

cudaError_t launch_decode_prefix(const DecodeArgs& a, cudaStream_t s) {
  return a.D == 128 ? launch_d<false, 128, false>(a, s) : launch_d<false, 64, false>(a, s);
}

}  // namespace minipic
