// Decode of a batch whose requests share prefixes, in three kernels: the shared part (prefill_pair.cu, prefill_tc.cu);
// meanwhile, on the SMs that it leaves free, the keys behind the prefixes (decode_list.cuh); and here the join of both,
//   out = sum_i 2^(lse_i - M) O_i / sum_i 2^(lse_i - M)
// over the request's own part and the parts of its prefix.  Memory-bound: 4 d bytes read a part and head, 2 d written.
#include "decode_list.cuh"

namespace minipic {

using namespace decode_list;

namespace {

template <int D>
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ DecodeArgs a) {
  const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;  // (request, query head, four dims)
  const long long row = idx / (D / 4);
  const int dim = 4 * (int)(idx % (D / 4)), i = (int)(row / a.Hq), h = (int)(row % a.Hq);
  if (i >= a.batch) return;
  const int L = __ldg(a.seq_lens + i);
  const Shared sh = shared_of(a, a.cu_requests, a.prefix_blocks, i, L);
  if (L <= 0 || sh.blocks == 0) return;  // written by the kernel before
  const int2 gi = prefix::items_of(a, sh.p, sh.q0, i);
  const size_t at = prefix::row_of(a, gi, sh.q0, i, h / a.G, h % a.G);
  const float own = a.own_lse[row];
  float M = own;
  for (int s = 0; s < gi.y; ++s) M = fmaxf(M, a.prefix_lse[at + (size_t)s * prefix::kRows]);
  const float ref = M == -CUDART_INF_F ? 0.f : M;  // no key at all: every weight is 0
  float sum = exp2f(own - ref);
  float4 O = *reinterpret_cast<const float4*>(a.own_o + row * D + dim);
  O = make_float4(O.x * sum, O.y * sum, O.z * sum, O.w * sum);
#pragma unroll 4
  for (int s = 0; s < gi.y; ++s) {
    const float w = exp2f(a.prefix_lse[at + (size_t)s * prefix::kRows] - ref);
    const float4 p = *reinterpret_cast<const float4*>(a.prefix_o + (at + (size_t)s * prefix::kRows) * D + dim);
    sum += w;
    O = make_float4(fmaf(p.x, w, O.x), fmaf(p.y, w, O.y), fmaf(p.z, w, O.z), fmaf(p.w, w, O.w));
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * D + dim) =
      make_uint2(ptx::pack_bf16(O.x * inv, O.y * inv), ptx::pack_bf16(O.z * inv, O.w * inv));
  if (dim == 0 && a.lse) a.lse[row] = sum == 0.f ? -CUDART_INF_F : (ref + log2f(sum)) * kLn2;
}

}  // namespace

cudaError_t launch_decode_apart(const DecodeArgs& a, cudaStream_t s) {
  const cudaError_t e = a.D == 128 ? launch_d<false, 128, false, kApart>(a, s) : launch_d<false, 64, false, kApart>(a, s);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(((long long)a.batch * a.Hq * (a.D / 4) + 255) / 256);
  if (a.D == 128) prefix_join_kernel<128><<<grid, 256, 0, s>>>(a);
  else prefix_join_kernel<64><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace minipic
