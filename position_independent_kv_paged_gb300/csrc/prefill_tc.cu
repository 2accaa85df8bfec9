// Prefill kernel wrapper and launcher for head dim 64 (the CTA body is in
// prefill2_body.cuh; head dim 128 goes to the CTA-pair kernel).
#include "prefill2_body.cuh"
#include "tmap.cuh"

namespace minipic {
namespace {

using namespace prefill2_impl;

// One CTA per (query-tile pair, kv head, request); each CTA loads its own K~/V
// tiles.
template <int D, bool ROPE, bool KROT>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const PrefillLaunch2 L) {
  extern __shared__ uint8_t smem_raw[];
  // heaviest (latest) query-tile pairs first
  const int n = gridDim.x;
  prefill2_cta<D, ROPE, kNB, kNSK, kNSV, KROT>(&kmap, &vmap, L, n - 1 - (int)blockIdx.x, n, blockIdx.y, blockIdx.z, smem_raw);
}

template <int D, bool ROPE, bool KROT = ROPE>
cudaError_t launch_t(const PrefillArgs& a, cudaStream_t s) {
  const int smem = PG2<D>::TOTAL + 1024;
  static bool done[64] = {false};
  cudaError_t e = set_smem_once(prefill_tc_kernel<D, ROPE, KROT>, smem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  const long long rows = (long long)a.num_blocks * a.Hkv * 16;
  if (!make_pool_map(&km, a.k_pool, rows, D) || !make_pool_block_map(&vm, a.v_pool, rows, D))
    return cudaErrorInvalidValue;
  PrefillLaunch2 L{a, 128 / a.G};
  const int n_pairs = (a.max_q_len + 2 * L.tq - 1) / (2 * L.tq);
  if (n_pairs <= 0) return cudaSuccess;
  prefill_tc_kernel<D, ROPE, KROT>
      <<<dim3((unsigned)n_pairs, (unsigned)a.Hkv, (unsigned)a.batch), kThreads, smem, s>>>(km, vm, L);
  return cudaGetLastError();
}

// Grid: one CTA an item.
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ PrefillLaunch2 L) {
  extern __shared__ uint8_t smem_raw[];
  ptx::launch_dependents();
  prefix::Item it;
  if (!prefix::find_item<64>(L.a, L.tq, blockIdx.x, it)) return;
  prefill2_cta<64, true, kNB, kNSK, kNSV, true, true>(&kmap, &vmap, L, it.pair, it.pair + 1, it.head, it.p, smem_raw, &it);
}

}  // namespace

cudaError_t launch_prefix(const PrefillArgs& a, long long items, cudaStream_t s) {
  if (a.D == 128) return launch_prefix_pair(a, items, s);
  if (a.D != 64 || items > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int smem = PG2<64>::TOTAL + 1024;
  static bool done[64] = {false};
  cudaError_t e = set_smem_once(prefix_tc_kernel, smem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  const long long rows = (long long)a.num_blocks * a.Hkv * 16;
  if (!make_pool_map(&km, a.k_pool, rows, 64) || !make_pool_block_map(&vm, a.v_pool, rows, 64))
    return cudaErrorInvalidValue;
  prefix_tc_kernel<<<(unsigned)items, kThreads, smem, s>>>(km, vm, PrefillLaunch2{a, 128 / a.G});
  return cudaGetLastError();
}

// Head dim 128 runs the CTA-pair kernel; head dim 64 this single-CTA kernel.
cudaError_t launch_prefill_tc(const PrefillArgs& a, bool rotate, cudaStream_t s) {
  if (a.D == 128) return launch_prefill_pair(a, rotate, s);
  if (a.D != 64) return cudaErrorInvalidValue;
  return rotate ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
}

// The same over a pool whose keys are rotated already (fp16 bit patterns).
cudaError_t launch_prefill_rotated(const PrefillArgs& a, cudaStream_t s) {
  if (a.D == 128) return launch_prefill_pair_rotated(a, s);
  return a.D == 64 ? launch_t<64, true, false>(a, s) : cudaErrorInvalidValue;
}

}  // namespace minipic
