// Decode attention over one list of blocks, tensor-core form (bf16 query and
// output; the f32 form is in decode_simt.cu).  The position-free cache it reads is
//   e4m3  bytes with one scale per (block, kv head), or
//   bf16  (for the call that records block weights);
// keys are unrotated and rotated here at pi(j) = start[r][block] + slot (MiniPIC
// summary, gist.science 2606.13126, section 2.1).
//
// Work: the blocks of all (request, kv head) pairs form one list, request by
// request; a resident grid cuts it into equal ranges, one per CTA, whatever the
// lengths are (they are on the device).  A CTA walks its range pair by pair: a pair
// that lies inside one range is written at once, one that is cut leaves a partial
// result per CTA, and the last of them to arrive merges them in order.  Against a
// grid of (split, kv head, request) this has no partly filled last wave, and pays
// a start (table entries, scales, queries, first tiles) once or twice per
// CTA instead of per split.  Within a pair each warp owns every NW-th 16-key
// block and runs its own ring of stages, each of two e4m3 blocks or one bf16 block.
// A (block, head) tile is contiguous in the pool; its 16-byte chunks are stored
// permuted in shared memory (mix below), so that the key-row reads and the
// transposing reads of V are free of bank conflicts.  The fp16 cos | sin row of the
// block's query rotation comes with them.  The copies are cp.async of the whole
// warp (17 instructions a stage at d 128): in place of one thread's tensor copies,
// and with the references made finite in the same step, they brought 431 warp
// instructions per block to 375, and the kernel is bound by issue.
//
// Per block, with t the query's position, b the block's start, s the slot:
//   score = (R_{t-b} q) . (R_s k) * (k scale) * softmax scale
// e4m3 widens to fp16 exactly, bf16 within fp16's range, with rows outside it scaled
// by a power of two where that matters (kFactor below; the test costs 2.7 %).  bf16
// operands would show: three roundings of 2^-8 each, an output error of 5.4e-3 of its
// norm at d 64 where this has 2.2e-3.  R_s is constant per lane, R_{t-b} q is formed
// once per block, both in packed fp16, and S^T = K' Q'^T, O^T += V^T P^T run as
// mma.sync m16n8k16 with fp32 accumulation (keys, then head dims, as M; up to 8
// query heads as N, so a group of 8 wastes nothing and the operands come from
// registers).  For one request at a time: the tcgen05 form needs M >= 64 and would
// take the widened, rotated keys through shared memory again.  Several requests that
// read one block could share both, in a list ordered by physical block; not built.
//  - The query is scaled by a power of two per head to a largest element in
//    [1, 2) first, so that fp16 holds it whatever its size.
//  - bf16: P is 2^(s - ms) in bf16 and V enters as it is.
//  - e4m3: V bytes stay unscaled in the product; the block's scale rides on P.  P is
//    2^(s + log2 vscale - mt + 7) in fp16 with a running reference mt of its own
//    (so blocks whose scales differ by any factor keep fp16's full precision
//    where they matter, and a weight 2^-31 of the largest is still above zero; a
//    block whose scale is zero does not count in mt),
//    the denominator 2^(s - ms) in fp32.  Both references move only when a value
//    exceeds them by more than 2^8 (P then is below 2^15).
//  - V fragments come from transposing byte reads: a register holds a head dim of
//    four consecutive keys, whose pairs widen straight into the operand; the
//    fragment rows of the scores are numbered to match.
// Slots past the request's length, blocks with a bad id, keys past the table and
// zero-scale values are masked in the scores and cleared in V (P = 0 must not
// meet a NaN byte); a pair of blocks with none of these takes a path without masks.
//
// What bounds it and what it measured (GB300; 3 CTAs of 4 warps per SM, held there
// by registers: 168 a thread):
//  - 64 requests x 8192 keys, 32 / 8 heads, spans shared: 119 us, 1.07 GB read of
//    which 0.30 GB from HBM.  Issue: 282 instructions a block and warp (81 of
//    them fp16 rotation, 66 conversions, 16 matrix products), 53 % of the issue slots used.
//  - 8 x 131072 keys, 64 / 8 heads, with block weights: 330 us, the same bound.
//  - the first batch over the bf16 cache, with block weights: 190 us, 2.15 GB read
//    (a grid of splits with tensor copies took 257 us and 669 instructions a block);
//    317 us with queries so large that every row is looked at, 604 us with keys
//    beyond fp16, whose pairs are gone through twice.
//  - 128 ragged contexts to 32768 keys, 28 / 4 heads, nothing shared: HBM, 2.29 GB at
//    6.40 TB/s (0.94 of the measured copy bandwidth).
#pragma once

#include <cuda_fp16.h>
#include <math_constants.h>

#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "tmap.cuh"

namespace minipic {
namespace decode_list {

using ptx::U4;

constexpr int kWarps = kListWarps;
constexpr int kChunk = 256;                   // blocks whose metadata is staged at a time
constexpr int kMinRange = 64;                 // blocks of a CTA, unless there are fewer in all (16, 32 and 128: slower)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;               // a reference moves when exceeded by 2^8
constexpr float kHeadQ8 = 7.f;                // e4m3: P of a key at its reference is 2^7
constexpr float kNone = -3e38f;               // a reference before the first key
constexpr float kKeyMin = 0x1p-10f, kKeyMax = 0x1p15f;  // largest element of a bf16 key row that fp16 holds well
constexpr uint32_t kWide = 0x40000u;          // mask bit: the key rows may need scaling
constexpr float kNoValue = -3e38f;            // log2 of a value scale of zero: finite, and no score brings it near a reference

// Shared-memory plan; Q8: e4m3 cache (else bf16).
template <int D, int NS, bool Q8>
struct Lay {
  static constexpr int BPS = Q8 ? 2 : 1;           // blocks of a stage
  static constexpr int TILE = 16 * D * (Q8 ? 1 : 2);  // bytes of one (block, head) tile of K or V
  static constexpr int STAGE = 2 * BPS * TILE;     // K and V of its blocks
  static constexpr int ROWB = 2 * D;               // one fp16 cos | sin row
  static constexpr int MT = D / 16;                // M tiles of O^T
  static constexpr int STAGES = kWarps * NS * STAGE;
  static constexpr int ROWS = STAGES;                               // [warp][stage][BPS] table rows
  static constexpr int META = ROWS + kWarps * NS * BPS * ROWB;      // [chunk block, padded to stages] int4
  static constexpr int MASK = META + (kChunk + 2 * kWarps) * 16;    // [same] uint32
  static constexpr int OST = D + 4;                             // padded row stride of the merge
  static constexpr int MERGE_W = (48 + 16 * OST) * 4;           // ms[16], l[16], mt[16], O[16][OST] of one warp
  static constexpr int MERGE = kWarps * MERGE_W;                // overlays stages, rows and meta
  static constexpr int TOTAL = MASK + (kChunk + 2 * kWarps) * 4;
  static_assert(MERGE <= TOTAL, "the merge overlays what the loop no longer reads");
  static_assert(kListMaxCtas * 8 * 4 <= STAGES, "so do the weights of the parts (half the CTAs for groups above 8)");
};

// Slot held by MMA fragment row g < 8 (row g + 8 holds slot + 2): rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9 are four
// consecutive keys, those that lane t's transposing byte read of V brings.
__device__ __forceinline__ int frag_slot(int g) { return (g >> 1) * 4 + (g & 1); }

// A tile's lines: e4m3 128 bytes (one key at d 128, two at d 64), bf16 one key.  Chunk c (16 bytes) of a line is
// stored at chunk c ^ mix(line); mix is linear, mix(a ^ b) = mix(a) ^ mix(b).  The chunks that one shared access
// reads then lie in different banks: for K two rows 2 t, 2 t + 1 times four lanes, for V equal chunks of eight keys
// (consecutive ones for the byte reads, the fragment's rows for the 16-bit ones).
template <int D, bool Q8>
struct Lines {
  static constexpr int BYTES = Q8 ? 128 : 2 * D;
  static constexpr int CHUNKS = BYTES / 16;
  static constexpr int PER = 512 / BYTES;  // lines of one copy of a warp
  __host__ __device__ static constexpr int mix(int line) {
    if (Q8) return D == 128 ? ((line & 1) << 2) | ((line >> 1) & 3) : line & 7;
    const int b0 = line & 1, b2 = (line >> 2) & 1, b3 = (line >> 3) & 1;
    return D == 128 ? b0 | (b2 << 1) | (b3 << 2) : (b0 << 2) | b2 | (b3 << 1);
  }
};
// Byte offset of 16-byte chunk c of key `key`.
template <int D, bool Q8>
__device__ __forceinline__ uint32_t at(int key, int c) {
  using LN = Lines<D, Q8>;
  const int line = Q8 && D == 64 ? key >> 1 : key;
  const int ch = Q8 && D == 64 ? (key & 1) * 4 + c : c;
  return (uint32_t)(line * LN::BYTES + ((ch ^ LN::mix(line)) << 4));
}

// bf16 keys: a row whose largest element is outside [kKeyMin, kKeyMax] would lose bits in fp16 or leave it (rotated, an
// element grows by up to sqrt(2)).  A block with such a row has its rows scaled, where they lie in shared memory, to a
// largest element in [1, 2); returned are the powers of two that the scores of this lane's rows then lack.  Rare, and a
// function of its own, so that its registers are not the loop's.
template <int D>
__device__ __noinline__ float2 rescale_rows(uint32_t kbase, int ks0, int tig) {
  constexpr unsigned FULL = 0xffffffffu;
  auto chunk = [&](int row, int u) {  // this lane's chunks of its rows: no other lane reads them
    return kbase + at<D, false>(ks0 + 2 * row, (D == 128 ? 2 * tig + (u & 1) : tig) + (u >= D / 64 ? D / 16 : 0));
  };
  float m[2] = {0.f, 0.f};
  bool off = false;
#pragma unroll
  for (int row = 0; row < 2; ++row) {
#pragma unroll 1
    for (int u = 0; u < D / 32; ++u) {
      const U4 x = ptx::lds128(chunk(row, u));
      auto larger = [&](uint32_t w) { m[row] = fmaxf(m[row], fmaxf(fabsf(ptx::bf_lo(w)), fabsf(ptx::bf_hi(w)))); };
      larger(x.x);
      larger(x.y);
      larger(x.z);
      larger(x.w);
    }
    m[row] = fmaxf(m[row], __shfl_xor_sync(FULL, m[row], 1));
    m[row] = fmaxf(m[row], __shfl_xor_sync(FULL, m[row], 2));
    off |= m[row] != 0.f && !(m[row] >= kKeyMin && m[row] <= kKeyMax);
  }
  if (!__any_sync(FULL, off)) return make_float2(1.f, 1.f);
  float up[2];
#pragma unroll
  for (int row = 0; row < 2; ++row) {
    const int ex = max(-126, min(126, (__float_as_int(m[row]) >> 23) - 127));
    const float down = __int_as_float((127 - ex) << 23);
    up[row] = __int_as_float((ex + 127) << 23);
#pragma unroll 1
    for (int u = 0; u < D / 32; ++u) {
      const U4 x = ptx::lds128(chunk(row, u));
      auto scaled = [&](uint32_t w) { return ptx::pack_bf16(ptx::bf_lo(w) * down, ptx::bf_hi(w) * down); };
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(chunk(row, u)), "r"(scaled(x.x)), "r"(scaled(x.y)),
                   "r"(scaled(x.z)), "r"(scaled(x.w)) : "memory");
    }
  }
  return make_float2(up[0], up[1]);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ __half2 h2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t u32(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// (x, y) rotated by the angle with cos c and sin s, two pairs at a time
__device__ __forceinline__ void rotate(uint32_t x, uint32_t y, uint32_t c, uint32_t s, uint32_t& xo, uint32_t& yo) {
  xo = u32(__hfma2(__hneg2(h2(y)), h2(s), __hmul2(h2(x), h2(c))));
  yo = u32(__hfma2(h2(x), h2(s), __hmul2(h2(y), h2(c))));
}

// Blocks of a request's length (clamped to its table).
__device__ __forceinline__ int blocks_of(int L, int mb) {
  return L <= 0 ? 0 : min((L >> 4) + ((L & 15) != 0), mb);
}

// |t - b| for any two 32-bit integers
__device__ __forceinline__ uint32_t distance(int t, int b) {
  return b > t ? (uint32_t)b - (uint32_t)t : (uint32_t)t - (uint32_t)b;
}

// DUAL (groups of up to 4 heads): the 8 columns of a product hold the group's heads twice, columns 0-3 with the
// query rotated for the first block of a pair and 4-7 for the second, so the query rotation and the softmax run
// once for two blocks; each block's products use their half of the columns, and the two halves are states of
// their own until the merge.
template <bool Q8, int D, int NT, bool DUAL, bool WTS, int NS, int CPS>
__global__ void __launch_bounds__(kWarps * 32, CPS) decode_list_kernel(const __grid_constant__ DecodeArgs a) {
  static_assert(!DUAL || (NT == 1 && Q8), "two half groups fill one column tile");
  using LY = Lay<D, NS, Q8>;
  using LN = Lines<D, Q8>;
  constexpr int BPS = LY::BPS;
  constexpr float kHead = Q8 ? kHeadQ8 : 0.f;
  constexpr int NW = kWarps;
  constexpr int NH = D / 32;  // 4-dim words of x (and of y) a thread holds per key: 4 at d 128, 2 at d 64
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t sgen[];
  const uint32_t sbase = ptx::smem_addr(sgen);
  int4* meta = reinterpret_cast<int4*>(sgen + LY::META);
  uint32_t* vmask = reinterpret_cast<uint32_t*>(sgen + LY::MASK);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, tig = lane & 3;
  const int G = a.G, mb = a.max_blocks;

  // this thread's key rows (slots ks0, ks0 + 2) and rotary pairs (f0 .. f0 + 4 NH - 1 with + d/2)
  const int ks0 = frag_slot(g8);
  const int f0 = 4 * NH * tig;
  // R_slot of both rows, fp16 (a slot past a table of fewer rows is masked)
  uint32_t rc[2][2 * NH], rs[2][2 * NH];
#pragma unroll
  for (int row = 0; row < 2; ++row) {
    const uint16_t* t = a.cs_f16 + (size_t)min(ks0 + 2 * row, a.max_pos - 1) * D + f0;
#pragma unroll
    for (int u = 0; u < NH / 2; ++u) {
      const uint4 c = __ldg(reinterpret_cast<const uint4*>(t) + u), sn = __ldg(reinterpret_cast<const uint4*>(t + D / 2) + u);
      rc[row][4 * u] = c.x; rc[row][4 * u + 1] = c.y; rc[row][4 * u + 2] = c.z; rc[row][4 * u + 3] = c.w;
      rs[row][4 * u] = sn.x; rs[row][4 * u + 1] = sn.y; rs[row][4 * u + 2] = sn.z; rs[row][4 * u + 3] = sn.w;
    }
  }
  // ---- this CTA's range [x0, x1) of the list, and the pair it is at.  In shared memory: registers that live
  // through the main loop are what bounds the CTAs per SM.
  __shared__ long long s_part[NW];
  __shared__ struct {
    long long x0, x1, total, n_cta;
    int r, hk, nblk, L;   // the pair: request, kv head, blocks, length
    int b_begin, left;    // its first block in this range, blocks of the range from there on
    int whole, last;      // one part of a pair per CTA; last to finish its pair
    int large, wide;      // the pair's key rows may need scaling: its queries are large; it was seen to need it
    int redo;             // the pair has to be gone through again, wide
  } sg;
  auto cta_total = [&](int v, int& before) {  // sum of v over the CTA, and over the threads before this one
    int pre = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULL, pre, o);
      if (lane >= o) pre += y;
    }
    __syncthreads();
    if (lane == 31) s_part[warp] = pre;
    __syncthreads();
    long long sum = 0;
    before = pre - v;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before += (int)s_part[w];
      sum += s_part[w];
    }
    return sum;
  };
  // No owner until a thread below finds the pair.  Stored before the barriers of the first pass, which order it before
  // that thread's store: a batch of up to one pass in equal ranges meets no other barrier in between.
  if (threadIdx.x == 0) {
    sg.r = -1;
    sg.large = sg.wide = sg.redo = 0;
  }
  long long total = 0, sum = 0;
  int pairs = 0, zero = 0, Li = 0, n = 0, before = 0;
  for (int base = 0; base < a.batch; base += NW * 32) {
    const int i = base + threadIdx.x;
    Li = i < a.batch ? __ldg(a.seq_lens + i) : 0;
    n = blocks_of(Li, mb);
    if ((Li < 0 || (long long)Li > 16LL * mb) && blockIdx.x == 0) atomicOr(a.err, kErrSeqLen);
    total += sum = cta_total(n, before);
    pairs += __syncthreads_count(n > 0);
    zero |= i < a.batch && n == 0 && i % gridDim.x == blockIdx.x;
  }
  if (__syncthreads_or(zero)) {  // requests with no key, shared out over the grid
    for (int i = blockIdx.x; i < a.batch; i += gridDim.x) {
      if (blocks_of(__ldg(a.seq_lens + i), mb)) continue;
      for (int e = threadIdx.x; e < a.Hq * D; e += NW * 32)
        static_cast<__nv_bfloat16*>(a.out)[(size_t)i * a.Hq * D + e] = __float2bfloat16_rn(0.f);
      if (a.lse)
        for (int e = threadIdx.x; e < a.Hq; e += NW * 32) a.lse[(size_t)i * a.Hq + e] = -CUDART_INF_F;
    }
  }
  total *= a.Hkv;
  {
    // A batch that does not fill the grid is cut into parts of pairs instead, one per CTA, so that no CTA walks two
    // pairs one after the other.  A part costs about 0.12 us a block, joining the parts of a pair about 5 us and more
    // with their number and the group's heads.  So pairs of up to 64 blocks are cut to 8 or 16 where that fits (1024
    // keys, 8 heads: 11 us, against 12 to 13 in parts of 32 or whole) and else left whole (128 pairs of 64 blocks: 15 us
    // against 16 in halves), longer ones to 32 (8192 keys: 15.4 us against 16.3 in 16) or, above 8 heads, 64.
    const long long all_pairs = (long long)pairs * a.Hkv;
    int part = total <= 64 * all_pairs ? 8 : (NT == 1 ? 32 : 64);
    while (part <= kMinRange && total / part + all_pairs > (long long)gridDim.x) part = part == 16 ? 64 : part * 2;
    const bool whole = part <= kMinRange;
    // else equal ranges of the list, of at least kMinRange blocks, but no fewer of them than pairs
    const long long want = max((total + kMinRange - 1) / kMinRange, all_pairs);
    const long long n_cta = max(1LL, min((long long)gridDim.x, want));  // 1: no request has a key
    if (blockIdx.x >= n_cta && !whole) return;
    const long long x0 = whole ? blockIdx.x : blockIdx.x * total / n_cta;
    const long long x1 = (blockIdx.x + 1) * total / n_cta;
    long long first = 0;  // blocks or parts (of one kv head) of the requests before `base`
    for (int base = 0; base < a.batch; base += NW * 32) {
      const int i = base + threadIdx.x;
      if (a.batch > NW * 32) {  // else the one pass above still holds them
        Li = i < a.batch ? __ldg(a.seq_lens + i) : 0;
        n = blocks_of(Li, mb);
      }
      const int units = whole ? (n + part - 1) / part : n;
      if (a.batch > NW * 32 || whole) sum = cta_total(units, before);
      const long long at = (first + before) * a.Hkv;
      if (x0 >= at && x0 < at + (long long)units * a.Hkv) {
        const int k = (int)((x0 - at) % units);
        sg.r = i;
        sg.hk = (int)((x0 - at) / units);
        sg.nblk = n;
        sg.L = min(Li, (int)min(16LL * mb, 2147483632LL));
        sg.whole = whole;
        if (whole) {
          sg.b_begin = (int)((long long)k * n / units);
          sg.left = (int)((long long)(k + 1) * n / units) - sg.b_begin;
          sg.x0 = x0 - k;           // the pair's first CTA
          sg.x1 = sg.x0 + units - 1;  // ... and its last
        } else {
          sg.b_begin = k;
          sg.left = (int)(x1 - x0);
          sg.x0 = x0;
          sg.x1 = x1;
          sg.total = total;
          sg.n_cta = n_cta;
        }
      }
      first += sum;
      if (first * a.Hkv > x0) break;
    }
    __syncthreads();
    if (sg.r < 0) return;  // more CTAs than parts
  }
  constexpr float kFactor = 8192.f / D;
  int b0 = 0, span = 0, n_stage = 0;             // the chunk's first block, blocks, stages of this warp
  uint32_t qx[NT][2 * NH], qy[NT][2 * NH];       // queries of this thread's heads (column g8 + 8 nt), fp16
  __shared__ float2 s_qf[NT][4];                 // the power of two taken out of those of columns 2 tig + j + 8 nt

  // What a block needs: x = its (block, head) tile (-1: nothing usable), y = table row of |t - start|.
  auto place = [&](int phys, int start, int tq, int hk) {
    const uint32_t ad = distance(tq, start);
    const bool ok = phys >= 0 && phys < a.num_blocks && ad < (uint32_t)a.max_pos;
    return make_int2(ok ? phys * a.Hkv + hk : -1, ok ? (int)ad : 0);
  };
  // The warp copies a stage's blocks: lane -> 16 bytes of each tile's next 512, swizzled, and of the
  // two table rows.  A block with nothing usable copies tile 0 and row 0, which its mask keeps out.
  const uint32_t wbase = sbase + warp * NS * LY::STAGE, wrow = sbase + LY::ROWS + warp * NS * BPS * LY::ROWB;
  const uint32_t sw0 =
      (uint32_t)((lane / LN::CHUNKS) * LN::BYTES + (((lane % LN::CHUNKS) ^ LN::mix(lane / LN::CHUNKS)) << 4));
  const uint8_t* kg = static_cast<const uint8_t*>(a.k_pool) + 16 * lane;
  const uint8_t* vg = static_cast<const uint8_t*>(a.v_pool) + 16 * lane;
  constexpr int RL = LY::ROWB / 16;  // lanes of a table row
  auto issue = [&](const int stg, int2 p0, int2 p1) {
    const uint32_t dst = wbase + stg * LY::STAGE;
#pragma unroll
    for (int u = 0; u < BPS; ++u) {
      const size_t tile = (size_t)max(u ? p1.x : p0.x, 0) * LY::TILE;
#pragma unroll
      for (int i = 0; i < LY::TILE / 512; ++i) {
        const uint32_t to = dst + 2 * u * LY::TILE + 512 * i + (sw0 ^ (uint32_t)(LN::mix(LN::PER * i) << 4));
        ptx::cp_async16(to, kg + tile + 512 * i);
        ptx::cp_async16(to + LY::TILE, vg + tile + 512 * i);
      }
    }
    const int2 pr = lane < RL ? p0 : p1;
    if (lane < BPS * RL)
      ptx::cp_async16(wrow + stg * BPS * LY::ROWB + 16 * lane,
                      reinterpret_cast<const uint8_t*>(a.cs_f16) + 16 * (lane % RL) + (size_t)pr.y * LY::ROWB);
  };
  // Start of a chunk: the first copies, and per block, once for the CTA: place, score factor (softmax scale *
  // log2 e * key scale), log2 of the value scale (finite), and the mask of its usable slots (bit 16: the values are
  // zero, bit 17: the angle is negative).  With FIRST (of a pair) also its query.  Every load that depends on
  // nothing else comes first, so that a start costs about two round trips to memory (ids, then scales).
  auto start_chunk = [&](bool first) {
    const int r = sg.r, hk = sg.hk;
    int tq = __ldg(a.q_pos + r);
    const int* bt = a.block_tables + (size_t)r * mb + b0;
    const int* bs = a.block_starts + (size_t)r * mb + b0;
    int e_phys = -1, e_start = 0;  // lane BPS p + u: block u of this warp's stage p
    if (lane < BPS * NS && warp + NW * lane < span) {
      e_phys = __ldg(bt + warp + NW * lane);
      e_start = __ldg(bs + warp + NW * lane);
    }
    constexpr int kPer = kChunk / (NW * 32);  // staged entries of a thread
    int t_phys[kPer], t_start[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = threadIdx.x + u * NW * 32;
      t_phys[u] = i < span ? __ldg(bt + i) : -1;
      t_start[u] = i < span ? __ldg(bs + i) : 0;
    }
    if (first) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int head = DUAL ? (g8 & 3) : 8 * nt + g8;
        const __nv_bfloat16* p =
            static_cast<const __nv_bfloat16*>(a.q) + ((size_t)r * a.Hq + (size_t)hk * G + head) * D + f0;
#pragma unroll
        for (int u = 0; u < NH / 2; ++u) {
          const uint4 z = make_uint4(0u, 0u, 0u, 0u);
          const uint4 x = head < G ? __ldg(reinterpret_cast<const uint4*>(p) + u) : z;
          const uint4 y = head < G ? __ldg(reinterpret_cast<const uint4*>(p + D / 2) + u) : z;
          qx[nt][4 * u] = x.x; qx[nt][4 * u + 1] = x.y; qx[nt][4 * u + 2] = x.z; qx[nt][4 * u + 3] = x.w;
          qy[nt][4 * u] = y.x; qy[nt][4 * u + 1] = y.y; qy[nt][4 * u + 2] = y.z; qy[nt][4 * u + 3] = y.w;
        }
      }
    }
    if (tq < 0 || tq >= a.max_pos) {
      if (threadIdx.x == 0) atomicOr(a.err, kErrPosition);
      tq = 0;
    }
    __syncthreads();  // the metadata and the merge of what came before have been read
#pragma unroll
    for (int p = 0; p < NS; ++p) {
      const int2 p0 = place(__shfl_sync(FULL, e_phys, BPS * p), __shfl_sync(FULL, e_start, BPS * p), tq, hk);
      int2 p1 = make_int2(-1, 0);
      if constexpr (BPS == 2) {
        const int2 q = place(__shfl_sync(FULL, e_phys, 2 * p + 1), __shfl_sync(FULL, e_start, 2 * p + 1), tq, hk);
        if (warp + NW * (2 * p + 1) < span) p1 = q;
      }
      if (p < n_stage) issue(p, p0, p1);
      ptx::cp_async_commit();
    }
    auto scale_queries = [&] {  // to fp16
      bool large = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 2 * NH; ++e)
          amax = fmaxf(amax, fmaxf(fmaxf(fabsf(ptx::bf_lo(qx[nt][e])), fabsf(ptx::bf_hi(qx[nt][e]))),
                                   fmaxf(fabsf(ptx::bf_lo(qy[nt][e])), fabsf(ptx::bf_hi(qy[nt][e])))));
        amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 2));
        // exponent of the largest element (at most 127, an infinity's; a row of zeros or subnormals takes -126)
        int ex = (__float_as_int(amax) >> 23) - 127;
        ex = ex < -126 ? -126 : (ex > 126 ? 126 : ex);
        const float down = __int_as_float((127 - ex) << 23);
#pragma unroll
        for (int e = 0; e < 2 * NH; ++e) {
          qx[nt][e] = ptx::pack_f16(ptx::bf_lo(qx[nt][e]) * down, ptx::bf_hi(qx[nt][e]) * down);
          qy[nt][e] = ptx::pack_f16(ptx::bf_lo(qy[nt][e]) * down, ptx::bf_hi(qy[nt][e]) * down);
        }
        const float up = __int_as_float((ex + 127) << 23);
        if (warp == 0 && tig == 0) reinterpret_cast<float*>(s_qf[nt])[g8] = up;
        large |= up * (a.scale * kLog2e) > kFactor;
      }
      return large;
    };
    [[maybe_unused]] bool wide = false;
    if constexpr (!Q8) {
      if (first) {
        const bool large = __any_sync(FULL, scale_queries());  // every warp holds every head of the pair
        if (threadIdx.x == 0) sg.large = large;
        wide = large || sg.wide;
      } else {
        wide = sg.large || sg.wide;
      }
    }
    float t_ks[kPer], t_vs[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const bool in = Q8 && t_phys[u] >= 0 && t_phys[u] < a.num_blocks;
      t_ks[u] = in ? __ldg(a.k_scale + (size_t)t_phys[u] * a.Hkv + hk) : 0.f;
      t_vs[u] = in ? __ldg(a.v_scale + (size_t)t_phys[u] * a.Hkv + hk) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = threadIdx.x + u * NW * 32;
      int2 pl = make_int2(-1, 0);
      float ks = 0.f, lv = 0.f;
      uint32_t m = 0u;
      if (i < span) {
        const int phys = t_phys[u], start = t_start[u];
        pl = place(phys, start, tq, hk);
        const int nk = min(16, sg.L - (b0 + i) * 16);
        if (phys < 0 || phys >= a.num_blocks) {
          atomicOr(a.err, kErrBlockId);
        } else {
          const uint32_t all = (1u << nk) - 1u;
          m = all;
          // keys whose position falls outside the table are masked
          if (pl.x < 0 || start <= -16 || start >= a.max_pos) m = 0u;
          else if (start < 0) m &= 0xffffu << -start;
          else if (start > a.max_pos - nk) m &= (1u << (a.max_pos - start)) - 1u;
          if (a.max_pos < 16) m &= (1u << a.max_pos) - 1u;  // R_slot reaches as far as the table
          if (m != all) atomicOr(a.err, kErrPosition);
          ks = (Q8 ? t_ks[u] : 1.f) * (a.scale * kLog2e);
          lv = Q8 ? log2f(t_vs[u]) : 0.f;
          if (Q8 && t_vs[u] == 0.f) {  // it must not raise mt for the others
            lv = kNoValue;
            m |= 0x10000u;
          }
          if (start > tq) m |= 0x20000u;
          if (wide) m |= kWide;
        }
      }
      meta[i] = make_int4(pl.x, pl.y, __float_as_int(ks), __float_as_int(lv));
      vmask[i] = m;
    }
    if (threadIdx.x < 2 * NW) {  // the stages of a full chunk reach past its last entry
      meta[kChunk + threadIdx.x] = make_int4(-1, 0, 0, 0);
      vmask[kChunk + threadIdx.x] = 0u;
    }
    if constexpr (Q8)
      if (first) scale_queries();
    __syncthreads();  // metadata visible
  };

  // bf16 keys.  A key beyond fp16 makes its row's every product infinite or NaN: the softmax sees that, and the pair
  // is gone through again with every row looked at.  A small key loses bits, at most 3.4 * 2^-25 of a rotated element,
  // 2^-9 of a score's binary logarithm (the rounding of P) while the scores' factor is up to kFactor (queries up to
  // 500 at the default scale); beyond, the rows are looked at from the start.  So a batch of usual sizes pays only a
  // sum and a comparison a block.
  // references: ms of the scores (denominator l), mt of the scores plus log2 of the value scale (O)
  // (before the first key a finite value far below any score, so that no difference of two is undefined)
  float ms[NT][2], mt[NT][2], l[NT][2];
  float oacc[LY::MT][NT][4];
  // the rotated query words of column tile nt, R_{t - start} q, from a staged cos | sin row
  auto rotate_q = [&](auto plain, uint32_t row, uint32_t m, uint32_t (&bx)[NT][2 * NH], uint32_t (&by)[NT][2 * NH]) {
    uint32_t cw[2 * NH], sw[2 * NH];
#pragma unroll
    for (int u = 0; u < NH / 2; ++u) {
      const U4 c = ptx::lds128(row + 2 * f0 + 16 * u);
      const U4 s = ptx::lds128(row + D + 2 * f0 + 16 * u);
      cw[4 * u] = c.x; cw[4 * u + 1] = c.y; cw[4 * u + 2] = c.z; cw[4 * u + 3] = c.w;
      sw[4 * u] = s.x; sw[4 * u + 1] = s.y; sw[4 * u + 2] = s.z; sw[4 * u + 3] = s.w;
    }
    if constexpr (!decltype(plain)::value) {  // a key ahead of the query: the sine takes the angle's sign
      const uint32_t sgn = m & 0x20000u ? 0x80008000u : 0u;
#pragma unroll
      for (int e = 0; e < 2 * NH; ++e) sw[e] ^= sgn;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2 * NH; ++e) rotate(qx[nt][e], qy[nt][e], cw[e], sw[e], bx[nt][e], by[nt][e]);
  };
  // S^T = K' Q'^T of one block
  auto scores = [&](uint32_t kbase, const uint32_t (&bx)[NT][2 * NH], const uint32_t (&by)[NT][2 * NH],
                    float (&sc)[NT][4]) {
    // words of this thread's pairs: e4m3 4 dims a word, all at once; bf16 2 dims, 8 words (of both rows, x and y:
    // 4 each) at a time
    constexpr int NWORD = Q8 ? NH : 4;
    uint32_t kx[2][NWORD], ky[2][NWORD];
    auto load = [&](int part) {
#pragma unroll
      for (int row = 0; row < 2; ++row) {
        if constexpr (Q8 && D == 64) {
          const uint2 x = ptx::lds64(kbase + at<D, Q8>(ks0 + 2 * row, tig >> 1) + 8 * (tig & 1));
          const uint2 y = ptx::lds64(kbase + at<D, Q8>(ks0 + 2 * row, 2 + (tig >> 1)) + 8 * (tig & 1));
          kx[row][0] = x.x; kx[row][1] = x.y;
          ky[row][0] = y.x; ky[row][1] = y.y;
        } else {
          // chunks of 16 (e4m3) or 8 (bf16) dims; y is half a row further
          const int c = Q8 ? tig : (D == 128 ? 2 * tig + part : tig);
          const U4 x = ptx::lds128(kbase + at<D, Q8>(ks0 + 2 * row, c));
          const U4 y = ptx::lds128(kbase + at<D, Q8>(ks0 + 2 * row, c + (Q8 ? D / 32 : D / 16)));
          kx[row][0] = x.x; kx[row][1] = x.y; kx[row][2] = x.z; kx[row][3] = x.w;
          ky[row][0] = y.x; ky[row][1] = y.y; ky[row][2] = y.z; ky[row][3] = y.w;
        }
      }
    };
    // two accumulation chains (the x and the y halves of the pairs)
    float sy[NT][4];
#pragma unroll
    for (int w = 0; w < NH; ++w) {  // 4 pairs of each key row
      if (w == 0 || (!Q8 && w == 2)) load(w >> 1);
      uint32_t x[2][2], y[2][2];    // [row][dims 0-1, 2-3]
#pragma unroll
      for (int row = 0; row < 2; ++row) {
        uint32_t hx[2], hy[2];
        if constexpr (Q8) {
          ptx::e4m3x4_to_h2(kx[row][w], hx[0], hx[1]);
          ptx::e4m3x4_to_h2(ky[row][w], hy[0], hy[1]);
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t u = kx[row][2 * (w & 1) + e], v = ky[row][2 * (w & 1) + e];
            hx[e] = ptx::pack_f16(ptx::bf_lo(u), ptx::bf_hi(u));
            hy[e] = ptx::pack_f16(ptx::bf_lo(v), ptx::bf_hi(v));
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          rotate(hx[e], hy[e], rc[row][2 * w + e], rs[row][2 * w + e], x[row][e], y[row][e]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (w == 0) {
          ptx::mma_f16_16816_set(sc[nt], x[0][0], x[1][0], x[0][1], x[1][1], bx[nt][0], bx[nt][1]);
          ptx::mma_f16_16816_set(sy[nt], y[0][0], y[1][0], y[0][1], y[1][1], by[nt][0], by[nt][1]);
        } else {
          ptx::mma_f16_16816(sc[nt], x[0][0], x[1][0], x[0][1], x[1][1], bx[nt][2 * w], bx[nt][2 * w + 1]);
          ptx::mma_f16_16816(sy[nt], y[0][0], y[1][0], y[0][1], y[1][1], by[nt][2 * w], by[nt][2 * w + 1]);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[nt][e] += sy[nt][e];
  };
  float* w_base = nullptr;  // raw sums of the pair
  // one step of the online softmax over 16 keys; m, ks and lv are those of the columns' block, wb the block
  // whose sum is recorded
  auto softmax = [&](auto plain, float (&sc)[NT][4], [[maybe_unused]] const float (&kf)[2], uint32_t m, float ks, float lv,
                     int wb, uint32_t (&pb0)[NT], uint32_t (&pb1)[NT]) {
    const bool v0 = decltype(plain)::value || ((m >> ks0) & 1u), v1 = decltype(plain)::value || ((m >> (ks0 + 2)) & 1u);
    bool over = false;
    [[maybe_unused]] bool beyond = false;
    if constexpr (!Q8) {
      if constexpr (decltype(plain)::value) beyond = !(fabsf(sc[0][0]) + fabsf(sc[0][2]) < 3e38f);
      else beyond = !(m & kWide) && ((v0 && !(fabsf(sc[0][0]) < 3e38f)) || (v1 && !(fabsf(sc[0][2]) < 3e38f)));
      over = beyond;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 qf = s_qf[nt][tig];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // finite: a product of 0 stays 0
        constexpr bool one = Q8 || decltype(plain)::value;
        const float q = j ? qf.y : qf.x;
        const float f0 = fminf(ks * (one ? q : q * kf[0]), 3.4e38f), f1 = one ? f0 : fminf(ks * (q * kf[1]), 3.4e38f);
        sc[nt][j] = v0 ? sc[nt][j] * f0 : -CUDART_INF_F;
        sc[nt][2 + j] = v1 ? sc[nt][2 + j] * f1 : -CUDART_INF_F;
        over |= fmaxf(sc[nt][j], sc[nt][2 + j]) > (Q8 ? fminf(ms[nt][j], mt[nt][j] - lv) : ms[nt][j]) + kRescale;
      }
    }
    if (__any_sync(FULL, over)) {  // rare: move the references, rescale what was summed
      if constexpr (!Q8)
        if (beyond) sg.redo = 1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float bm = fmaxf(sc[nt][j], sc[nt][2 + j]);
          bm = fmaxf(bm, __shfl_xor_sync(FULL, bm, 4));
          bm = fmaxf(bm, __shfl_xor_sync(FULL, bm, 8));
          bm = fmaxf(bm, __shfl_xor_sync(FULL, bm, 16));
          const float msn = fmaxf(ms[nt][j], bm), mtn = fmaxf(mt[nt][j], bm + lv);
          const float cs = ex2(ms[nt][j] - msn), ct = Q8 ? ex2(mt[nt][j] - mtn) : cs;
          ms[nt][j] = msn;
          mt[nt][j] = mtn;
          l[nt][j] *= cs;
#pragma unroll
          for (int mm = 0; mm < LY::MT; ++mm) {
            oacc[mm][nt][j] *= ct;
            oacc[mm][nt][2 + j] *= ct;
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pv[4], es[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // P = e * 2^(ms - mt + lv + 7); the cap only meets scores whose e is 0
        const float w = Q8 ? ex2(fminf(ms[nt][j] - mt[nt][j] + (lv + kHead), 126.f)) : 1.f;
        const float ea = ex2(sc[nt][j] - ms[nt][j]), eb = ex2(sc[nt][2 + j] - ms[nt][j]);
        pv[j] = ea * w;
        pv[2 + j] = eb * w;
        es[j] = ea + eb;
        l[nt][j] += es[j];
      }
      if constexpr (WTS) {
        // the block's sum of each column over the fragment rows: the first step leaves even rows with column 0 and
        // odd rows with column 1, so two columns take three shuffles
        const bool odd = g8 & 1;
        float e = (odd ? es[1] : es[0]) + __shfl_xor_sync(FULL, odd ? es[0] : es[1], 4);
        e += __shfl_xor_sync(FULL, e, 8);
        e += __shfl_xor_sync(FULL, e, 16);
        const int head = DUAL ? (2 * tig + g8) & 3 : 8 * nt + 2 * tig + g8;
        if (g8 < 2 && head < G && wb < b0 + span)
          w_base[(size_t)wb * G + head] = e == 0.f ? -CUDART_INF_F : (odd ? ms[nt][1] : ms[nt][0]) + log2f(e);
      }
      pb0[nt] = ptx::movmatrix_trans(Q8 ? ptx::pack_f16(pv[0], pv[1]) : ptx::pack_bf16(pv[0], pv[1]));  // rows 0 .. 7
      pb1[nt] = ptx::movmatrix_trans(Q8 ? ptx::pack_f16(pv[2], pv[3]) : ptx::pack_bf16(pv[2], pv[3]));  // 8 .. 15
    }
  };
  // O^T += V^T P^T of one block
  const int v_key = Q8 ? lane & 15 : frag_slot(lane & 7) + 2 * (lane >> 4);
  const int v_chunk = Q8 ? lane >> 4 : (lane >> 3) & 1;
  auto values = [&](auto plain, uint32_t vbase, uint32_t m, const uint32_t (&pb0)[NT], const uint32_t (&pb1)[NT]) {
    constexpr bool part = !decltype(plain)::value;
    // which of this lane's four keys (slots 4 tig .. 4 tig + 3) count: as bytes (e4m3), or as halves (bf16: the
    // first two keys, the last two)
    [[maybe_unused]] uint32_t use = FULL, use2 = FULL;
    if constexpr (part) {
      const uint32_t u = m & 0x10000u ? 0u : m >> (4 * tig);
      if constexpr (Q8) {
        use = (u & 1u ? 0xffu : 0u) | (u & 2u ? 0xff00u : 0u) | (u & 4u ? 0xff0000u : 0u) | (u & 8u ? 0xff000000u : 0u);
      } else {
        use = (u & 1u ? 0xffffu : 0u) | (u & 2u ? 0xffff0000u : 0u);
        use2 = (u & 4u ? 0xffffu : 0u) | (u & 8u ? 0xffff0000u : 0u);
      }
    }
    if constexpr (Q8) {
#pragma unroll
      for (int mm = 0; mm < LY::MT; mm += 2) {
        uint32_t w[4];
        ptx::ldsm_b8_trans_x2(vbase + at<D, Q8>(v_key, mm + v_chunk), w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // head dims 16 (mm + u) + g8 and + 8
          uint32_t a0, a1, a2, a3;
          ptx::e4m3x4_to_h2(part ? w[2 * u] & use : w[2 * u], a0, a2);
          ptx::e4m3x4_to_h2(part ? w[2 * u + 1] & use : w[2 * u + 1], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) ptx::mma_f16_16816(oacc[mm + u][nt], a0, a1, a2, a3, pb0[nt], pb1[nt]);
        }
      }
    } else {
#pragma unroll
      for (int mm = 0; mm < LY::MT; ++mm) {  // head dims 16 mm + g8 and + 8
        uint32_t a0, a1, a2, a3;
        ptx::ldsm_x4_trans(vbase + at<D, Q8>(v_key, 2 * mm + v_chunk), a0, a1, a2, a3);
        if constexpr (part) {
          a0 &= use;
          a1 &= use;
          a2 &= use2;
          a3 &= use2;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) ptx::mma_bf16_16816(oacc[mm][nt], a0, a1, a2, a3, pb0[nt], pb1[nt]);
      }
    }
  };

  auto pair = [&](auto plain, uint32_t kbase, uint32_t rowb, int i0, uint32_t m0, uint32_t m1) {
    uint32_t bx[NT][2 * NH], by[NT][2 * NH], pb0[NT], pb1[NT];
    float sc[NT][4], kf[2] = {1.f, 1.f};
    if constexpr (DUAL) {
      const int4 mc = meta[i0 + (tig >= 2 ? NW : 0)];  // of these score columns' block
      rotate_q(plain, rowb + (g8 >= 4 ? LY::ROWB : 0), g8 >= 4 ? m1 : m0, bx, by);
      float s1[NT][4];
      scores(kbase, bx, by, sc);
      scores(kbase + 2 * LY::TILE, bx, by, s1);
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[0][e] = tig >= 2 ? s1[0][e] : sc[0][e];
      softmax(plain, sc, kf, tig >= 2 ? m1 : m0, __int_as_float(mc.z), __int_as_float(mc.w),
              b0 + i0 + (tig >= 2 ? NW : 0), pb0, pb1);
      const uint32_t z0[1] = {g8 < 4 ? pb0[0] : 0u}, z1[1] = {g8 < 4 ? pb1[0] : 0u};
      const uint32_t y0[1] = {g8 < 4 ? 0u : pb0[0]}, y1[1] = {g8 < 4 ? 0u : pb1[0]};
      values(plain, kbase + LY::TILE, m0, z0, z1);
      values(plain, kbase + 3 * LY::TILE, m1, y0, y1);
    } else {
#pragma unroll 1
      for (int u = 0; u < BPS; ++u) {
        const int4 md = meta[i0 + u * NW];
        const uint32_t m = u ? m1 : m0;
        if constexpr (!Q8 && !decltype(plain)::value)
          if (m & kWide) {
            const float2 up = rescale_rows<D>(kbase, ks0, tig);
            kf[0] = up.x;
            kf[1] = up.y;
          }
        rotate_q(plain, rowb + u * LY::ROWB, m, bx, by);
        scores(kbase + 2 * u * LY::TILE, bx, by, sc);
        softmax(plain, sc, kf, m, __int_as_float(md.z), __int_as_float(md.w), b0 + i0 + u * NW, pb0, pb1);
        values(plain, kbase + (2 * u + 1) * LY::TILE, m, pb0, pb1);
      }
    }
  };
  // one stage `stg` (a compile-time constant: every shared address is a per-thread base and an immediate)
  auto step = [&](const int stg, const int p) {
    const int i0 = warp + BPS * NW * p;  // blocks i0 and, in a stage of two, i0 + NW of the chunk
    const uint32_t kbase = wbase + stg * LY::STAGE, rowb = wrow + stg * BPS * LY::ROWB;
    const uint32_t m0 = vmask[i0], m1 = BPS == 2 ? vmask[i0 + NW] : 0xffffu;
    ptx::cp_async_wait<NS - 1>();
    __syncwarp();  // every lane's part of the stage has landed
    // blocks whole and behind the query: no masks, no signs
    if (m0 == 0xffffu && m1 == 0xffffu) pair(std::true_type{}, kbase, rowb, i0, m0, m1);
    else pair(std::false_type{}, kbase, rowb, i0, m0, m1);
    __syncwarp();  // every lane has read the stage
    if (p + NS < n_stage) {
      const int n0 = i0 + BPS * NW * NS;
      issue(stg, *reinterpret_cast<const int2*>(meta + n0),
            BPS == 2 ? *reinterpret_cast<const int2*>(meta + n0 + NW) : make_int2(-1, 0));
    }
    ptx::cp_async_commit();
  };
#pragma unroll 1
  while (true) {
    if (WTS) w_base = a.w_raw + ((size_t)sg.r * a.Hkv + sg.hk) * mb * G;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ms[nt][0] = ms[nt][1] = mt[nt][0] = mt[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int m = 0; m < LY::MT; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k) oacc[m][nt][k] = 0.f;
    }
#pragma unroll 1
    for (b0 = sg.b_begin;;) {
      span = min(kChunk, min(sg.nblk, sg.b_begin + sg.left) - b0);
      n_stage = span > warp ? (span - warp + BPS * NW - 1) / (BPS * NW) : 0;
      start_chunk(b0 == sg.b_begin);
#pragma unroll 1
      for (int p = 0; p < n_stage; p += NS) {
#pragma unroll
        for (int stg = 0; stg < NS; ++stg)
          if (p + stg < n_stage) step(stg, p + stg);
      }
      ptx::cp_async_wait<0>();
      b0 += span;
      if (b0 >= sg.nblk || b0 >= sg.b_begin + sg.left) break;
    }
    __syncthreads();  // every stage has been read: the merge overlays them
    if constexpr (!Q8)
      if (sg.redo) {
        __syncthreads();
        if (threadIdx.x == 0) {
          sg.redo = 0;
          sg.wide = 1;
        }
        __syncthreads();
        continue;
      }
    const int r = sg.r, hk = sg.hk, b_begin = sg.b_begin, nblk = sg.nblk, b_end = b0;

    // per-warp state: ms[16], l[16], mt[16], O[16][OST], by column
    {
      float* w = reinterpret_cast<float*>(sgen + warp * LY::MERGE_W);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float s = l[nt][j];
          s += __shfl_xor_sync(FULL, s, 4);
          s += __shfl_xor_sync(FULL, s, 8);
          s += __shfl_xor_sync(FULL, s, 16);
          const int head = 8 * nt + 2 * tig + j;
          if (g8 == 0) {
            w[head] = ms[nt][j];
            w[16 + head] = s;
            w[32 + head] = Q8 ? mt[nt][j] : ms[nt][j];
          }
#pragma unroll
          for (int m = 0; m < LY::MT; ++m) {
            w[48 + head * LY::OST + 16 * m + g8] = oacc[m][nt][j];
            w[48 + head * LY::OST + 16 * m + g8 + 8] = oacc[m][nt][2 + j];
          }
        }
    }
    __syncthreads();

    // the CTA's output of each head, already divided by its denominator: values no larger than V's
    const bool direct = b_begin == 0 && b_end == nblk;
    for (int idx = threadIdx.x; idx < G * D; idx += NW * 32) {
      const int head = idx / D, dim = idx - head * D;
      constexpr int NST = DUAL ? 2 * NW : NW;  // states of a head: warps, and half columns 4 apart
      auto state = [&](int w) {
        return reinterpret_cast<const float*>(sgen + (w % NW) * LY::MERGE_W);
      };
      auto column = [&](int w) { return head + (w / NW) * 4; };
      float M = kNone, T = kNone;
#pragma unroll
      for (int w = 0; w < NST; ++w) {
        M = fmaxf(M, state(w)[column(w)]);
        T = fmaxf(T, state(w)[32 + column(w)]);
      }
      float Ls = 0.f, O = 0.f;
#pragma unroll
      for (int w = 0; w < NST; ++w) {
        const float* p = state(w);
        const int c = column(w);
        Ls = fmaf(p[16 + c], exp2f(p[c] - M), Ls);
        O = fmaf(p[48 + c * LY::OST + dim], exp2f(p[32 + c] - T), O);
      }
      // the power in two factors: value scales down to fp32's least are 2^-149, past one factor's range with kHead
      const float e = T - M - kHead, e1 = fmaxf(e, -80.f);
      O = Ls == 0.f ? 0.f : O / Ls * exp2f(e1) * exp2f(e - e1);
      const float lse2 = Ls == 0.f ? -CUDART_INF_F : M + log2f(Ls);
      const size_t hq = (size_t)r * a.Hq + (size_t)hk * G + head;
      if (direct) {
        static_cast<__nv_bfloat16*>(a.out)[hq * D + dim] = __float2bfloat16_rn(O);
        if (dim == 0 && a.lse) a.lse[hq] = lse2 * kLn2;
        if (WTS && dim == 0) a.w_lse[hq] = lse2;
      } else {
        // a pair cut in front is this CTA's first (slot 0), one cut behind its last (slot 1)
        const size_t pi = (size_t)(2 * blockIdx.x + (b_begin == 0)) * G + head;
        a.part_o[pi * D + dim] = O;
        if (dim == 0) a.part_ml[pi] = lse2;
      }
    }
  if (!direct) {
      // CTAs c1 .. c2 hold parts of this pair; the last of them to arrive merges them in order
      int c1 = (int)sg.x0, c2 = (int)sg.x1;
      if (!sg.whole) {
        const long long ps = b_begin ? sg.x0 - b_begin : sg.x1 - (b_end - b_begin);  // the pair's place in the list
        auto owner = [&](long long x) { return ((x + 1) * sg.n_cta - 1) / sg.total; };
        c1 = (int)owner(ps);
        c2 = (int)owner(ps + nblk - 1);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        __threadfence();
        sg.last = atomicAdd(a.counters + (size_t)r * a.Hkv + hk, 1) == c2 - c1;
      }
      __syncthreads();
      if (sg.last) {
        __threadfence();
        // weights of the parts first (one read of their log sums), then the weighted sum, four dims a thread
        const int n_part = c2 - c1 + 1;
        float* wt = reinterpret_cast<float*>(sgen);  // [part][G], over what the stages held
        auto slot = [&](int c) { return (size_t)(2 * (c1 + c) + (c == 0)) * G; };
        for (int i = threadIdx.x; i < n_part * G; i += NW * 32) wt[i] = __ldcg(a.part_ml + slot(i / G) + i % G);
        __syncthreads();
        for (int head = warp; head < G; head += NW) {
          float M = -CUDART_INF_F, Ls = 0.f;
          for (int c = lane; c < n_part; c += 32) M = fmaxf(M, wt[c * G + head]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
          for (int c = lane; c < n_part; c += 32) {
            const float m = wt[c * G + head];
            Ls += m == -CUDART_INF_F ? 0.f : exp2f(m - M);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) Ls += __shfl_xor_sync(FULL, Ls, o);
          for (int c = lane; c < n_part; c += 32) {
            const float m = wt[c * G + head];
            wt[c * G + head] = m == -CUDART_INF_F ? 0.f : exp2f(m - M) / Ls;
          }
          if (lane == 0) {
            const float lse2 = Ls == 0.f ? -CUDART_INF_F : M + log2f(Ls);
            const size_t hq = (size_t)r * a.Hq + (size_t)hk * G + head;
            if (a.lse) a.lse[hq] = lse2 * kLn2;
            if (WTS) a.w_lse[hq] = lse2;
          }
        }
        __syncthreads();
        for (int idx = threadIdx.x; idx < G * D / 4; idx += NW * 32) {
          const int head = idx / (D / 4), dim = (idx % (D / 4)) * 4;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int c = 0; c < n_part; ++c) {
            const float4 p = __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot(c) + head) * D + dim));
            const float w = wt[c * G + head];
            o.x = fmaf(p.x, w, o.x);
            o.y = fmaf(p.y, w, o.y);
            o.z = fmaf(p.z, w, o.z);
            o.w = fmaf(p.w, w, o.w);
          }
          const size_t hq = (size_t)r * a.Hq + (size_t)hk * G + head;
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + hq * D + dim) =
              make_uint2(ptx::pack_bf16(o.x, o.y), ptx::pack_bf16(o.z, o.w));
        }
        if (threadIdx.x == 0) a.counters[(size_t)r * a.Hkv + hk] = 0;
      }
    }
    const int left = sg.left - (b_end - b_begin);
    if (left <= 0) break;
    __syncthreads();  // the pair has been read
    if (threadIdx.x == 0) {
      sg.left = left;
      sg.wide = 0;
      sg.b_begin = 0;
      sg.hk = hk + 1;
      if (hk + 1 == a.Hkv) {
        sg.hk = 0;
        int i = r, n = 0, Li = 0;
        while (n == 0 && ++i < a.batch) {  // a later request has blocks, as the range goes on
          Li = a.seq_lens[i];
          n = blocks_of(Li, mb);
        }
        if (n == 0) sg.left = 0;  // not reached
        sg.r = min(i, a.batch - 1);
        sg.nblk = n;
        sg.L = min(Li, (int)min(16LL * mb, 2147483632LL));
      }
    }
    __syncthreads();
    if (sg.left <= 0) break;
  }
}

// kernel<<<...>>> with its shared memory; a.n_split CTAs.
template <bool Q8, int D, int NT, bool DUAL, bool WTS, int NS, int CPS>
cudaError_t launch_t(const DecodeArgs& a, cudaStream_t s) {
  const auto kernel = decode_list_kernel<Q8, D, NT, DUAL, WTS, NS, CPS>;
  const int smem = Lay<D, NS, Q8>::TOTAL;
  static bool done[64] = {false};
  cudaError_t e = set_smem_once(kernel, smem, done);
  if (e != cudaSuccess) return e;
  kernel<<<a.n_split, kWarps * 32, smem, s>>>(a);
  return cudaGetLastError();
}

// Groups of up to 4 heads take two e4m3 blocks at once, of more than 8 two column tiles.
template <bool Q8, int D, bool WTS>
cudaError_t launch_d(const DecodeArgs& a, cudaStream_t s) {
  if (a.G > 8) return launch_t<Q8, D, 2, false, WTS, 2, 2>(a, s);
  constexpr int CPS = D == 64 ? 4 : 3;
  if constexpr (Q8)
    if (a.G <= 4) return launch_t<Q8, D, 1, true, WTS, 2, CPS>(a, s);
  return launch_t<Q8, D, 1, false, WTS, 2, CPS>(a, s);
}

}  // namespace decode_list
}  // namespace minipic
