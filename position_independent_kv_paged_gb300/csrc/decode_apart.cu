// Decode of a batch whose requests share prefixes, in three kernels: the shared part (prefill_pair.cu, prefill_tc.cu);
// meanwhile, on the SMs that it leaves free, the keys behind the prefixes (decode_list.cuh); and here the join of both,
//   out = sum_i 2^(lse_i - M) O_i / sum_i 2^(lse_i - M)
// over the request's own part and the parts of its prefix.  4 d bytes read a part and head, 2 d written: 21 MB for 256
// requests of 64 heads and one part, 11.6 us from cold caches (ncu), where latency bounds it: the chain of lengths,
// groups, items and partial results is walked once for four rows a thread.
#include "decode_list.cuh"

namespace minipic {

using namespace decode_list;

namespace {

// CTA = (request, part of its heads); a thread takes four dims of a head, four such at a time.
template <int D>
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ DecodeArgs a, const int heads_per) {
  constexpr int U = 4, T = 256;
  const int i = blockIdx.x, h0 = blockIdx.y * heads_per, n = min(heads_per, a.Hq - h0) * (D / 4);
  const int L = __ldg(a.seq_lens + i);
  const Shared sh = shared_of(a, a.cu_requests, a.prefix_blocks, *a.n_groups, i, L);
  if (L <= 0 || sh.blocks == 0) return;  // written by the kernel before
  const int2 gi = prefix::items_of(a, sh.p, sh.q0, i);
  for (int base = threadIdx.x; base < n; base += U * T) {
    float4 O[U];
    float ref[U], sum[U];
    size_t row[U], at[U];
    int dim[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = min(base + u * T, n - 1), h = h0 + e / (D / 4);
      dim[u] = 4 * (e % (D / 4));
      row[u] = (size_t)i * a.Hq + h;
      at[u] = prefix::row_of(a, gi, sh.q0, i, h / a.G, h % a.G);
      O[u] = *reinterpret_cast<const float4*>(a.own_o + row[u] * D + dim[u]);
      sum[u] = ref[u] = a.own_lse[row[u]];
    }
    for (int s = 0; s < gi.y; ++s)
#pragma unroll
      for (int u = 0; u < U; ++u) ref[u] = fmaxf(ref[u], a.prefix_lse[at[u] + (size_t)s * prefix::kRows]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ref[u] == -CUDART_INF_F) ref[u] = 0.f;  // no key at all: every weight is 0
      sum[u] = exp2f(sum[u] - ref[u]);
      O[u] = make_float4(O[u].x * sum[u], O[u].y * sum[u], O[u].z * sum[u], O[u].w * sum[u]);
    }
    for (int s = 0; s < gi.y; ++s) {
      float4 p[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        p[u] = *reinterpret_cast<const float4*>(a.prefix_o + (at[u] + (size_t)s * prefix::kRows) * D + dim[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = exp2f(a.prefix_lse[at[u] + (size_t)s * prefix::kRows] - ref[u]);
        sum[u] += w;
        O[u] = make_float4(fmaf(p[u].x, w, O[u].x), fmaf(p[u].y, w, O[u].y), fmaf(p[u].z, w, O[u].z),
                           fmaf(p[u].w, w, O[u].w));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u * T >= n) break;
      const float inv = sum[u] == 0.f ? 0.f : 1.f / sum[u];
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row[u] * D + dim[u]) =
          make_uint2(ptx::pack_bf16(O[u].x * inv, O[u].y * inv), ptx::pack_bf16(O[u].z * inv, O[u].w * inv));
      if (dim[u] == 0 && a.lse) a.lse[row[u]] = sum[u] == 0.f ? -CUDART_INF_F : (ref[u] + log2f(sum[u])) * kLn2;
    }
  }
}

}  // namespace

cudaError_t launch_decode_apart(const DecodeArgs& a, cudaStream_t s) {
  const cudaError_t e = a.D == 128 ? launch_d<false, 128, false, kApart>(a, s) : launch_d<false, 64, false, kApart>(a, s);
  if (e != cudaSuccess) return e;
  const int heads_per = 4096 / a.D;  // one pass of a CTA
  const dim3 grid((unsigned)a.batch, (unsigned)((a.Hq + heads_per - 1) / heads_per));
  if (a.D == 128) prefix_join_kernel<128><<<grid, 256, 0, s>>>(a, heads_per);
  else prefix_join_kernel<64><<<grid, 256, 0, s>>>(a, heads_per);
  return cudaGetLastError();
}

}  // namespace minipic
