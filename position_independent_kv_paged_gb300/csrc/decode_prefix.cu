// Decode of a batch whose requests share prefixes: the keys behind the prefixes, joined with the attention to those
// (the kernel is in decode_list.cuh; the shared part in prefill_pair.cu and prefill_tc.cu).
#include "decode_list.cuh"

namespace minipic {

using namespace decode_list;

cudaError_t launch_decode_prefix(const DecodeArgs& a, cudaStream_t s) {
  return a.D == 128 ? launch_d<false, 128, false, kPrefix>(a, s) : launch_d<false, 64, false, kPrefix>(a, s);
}

}  // namespace minipic
