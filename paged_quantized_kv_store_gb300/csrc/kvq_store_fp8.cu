// kvq_store_fp8: write new K/V rows into an FP8 pool (kvq_fp8.cuh), one
// power-of-two scale for each block of 16 tokens and kv head.
//
// LMDeploy article (devpress.csdn.net) §2.2: blocks of 16 tokens; §2.4: the
// cache is quantized online as rows are stored. The pages' scales belong to a
// token; here a block fills token by token under one scale, so a row that
// does not fit raises the scale and rounds the codes already there to it.
//
// A run is a maximal stretch of adjacent tokens of one block with rising
// offsets: what a request's new tokens are. With amax the largest finite |x|
// of the run's rows (of one kv head, of K or of V) and e the block's scale:
//   e' = max(e, fp8_scale_for(amax)), with e = 0 where the run writes the
//        block's first row (it starts the block anew),
//   code = rne_e4m3(x 2^-(e' - 127)),
//   and, where e' > e, every row that the run does not write:
//   code' = rne_e4m3(code 2^(e - e')), and 0 where e is 0.
//
// Work decomposition: a CTA takes the runs that begin in 48 consecutive
// tokens, for one kv head of K and V; a half-warp has two of the 64 rows those
// runs can reach (16 bytes a lane and row), so a run's largest value meets in
// shared memory, nothing is read twice, and every lane has four loads in
// flight. Bound by the latency of those loads and of the launch.
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_fp8.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kSpan = 48;           // tokens whose runs a CTA takes
constexpr int kRows = 64;           // rows those runs can reach (a run has at most 16)
constexpr int kStoreThreads = 512;  // a half-warp per two rows, 32 apart
static_assert(kSpan + kBlock <= kRows && kRows == 4 * kStoreThreads / 32, "rows of a span");
constexpr unsigned kFullMask = 0xFFFFFFFFu;

// Largest finite |x| of the 8 elements of v, as 16-bit float bits.
template <bool BF>
__device__ __forceinline__ uint32_t amax8(const uint4& v) {
  constexpr uint32_t kInf = BF ? 0x7F80u : 0x7C00u;
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  const uint32_t w[4] = {v.x & kAbs, v.y & kAbs, v.z & kAbs, v.w & kAbs};
  const uint32_t m2 = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  if (m >= kInf) {  // infinities and NaN do not set a scale
    m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0xFFFFu, hi = w[i] >> 16;
      if (lo < kInf) m = max(m, lo);
      if (hi < kInf) m = max(m, hi);
    }
  }
  return m;
}

__device__ __forceinline__ uint32_t half_max(uint32_t m) {
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, off));
  return m;
}

// Four codes at a new scale: each times `ratio`, rounded to nearest even.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  const uint32_t a = e4m3_lo_to_f16(w), b = e4m3_hi_to_f16(w);
  return f32_to_e4m3(lo_to_float<false>(a) * ratio, hi_to_float<false>(a) * ratio) |
         f32_to_e4m3(lo_to_float<false>(b) * ratio, hi_to_float<false>(b) * ratio) << 16;
}

// Moves the rows of `keep` of one (block, head) tile that fall to worker `me`
// of `n` to a new scale: code * ratio, or zeros. Four rows at a time, loads
// before stores.
__device__ __forceinline__ void rescale_rows(uint8_t* tile, int64_t stride, uint32_t keep, int n,
                                             int me, float ratio, bool zero) {
  int seen = 0;
#pragma unroll 1
  for (int o0 = 0; o0 < kBlock; o0 += 4) {
    uint2 v[4];
    uint32_t mine = 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if ((keep >> (o0 + u)) & 1u) {
        if (seen == me) {
          mine |= 1u << u;
          v[u] = *reinterpret_cast<const uint2*>(tile + (o0 + u) * stride);
        }
        seen = seen + 1 == n ? 0 : seen + 1;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if ((mine >> u) & 1u)
        *reinterpret_cast<uint2*>(tile + (o0 + u) * stride) =
            zero ? make_uint2(0u, 0u)
                 : make_uint2(rescale4(v[u].x, ratio), rescale4(v[u].y, ratio));
  }
}

template <bool BF>
__global__ void __launch_bounds__(kStoreThreads) store_fp8_kernel(const StoreArgs a) {
  __shared__ uint32_t smax[2][kRows];  // [K or V][row]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l16 = lane & 15;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * kSpan;
  const int64_t nslots = a.num_blocks * kBlock;

  // lane r of every warp looks at rows r and r + 32: the runs are the same
  // for all warps
  int64_t slot[2];
  uint64_t firsts = 0u, live = 0u;
  int64_t before = tok0 > 0 ? a.slot_mapping[tok0 - 1] : -1;  // the slot before lane 0's
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t i = tok0 + 32 * q + lane;
    slot[q] = i < a.num_tokens ? a.slot_mapping[i] : -1;
    int64_t prev = __shfl_up_sync(kFullMask, slot[q], 1);
    if (lane == 0) prev = before;
    before = __shfl_sync(kFullMask, slot[q], 31);
    const bool in_pool = slot[q] >= 0 && slot[q] < nslots;
    if (slot[q] >= nslots && 32 * q + lane < kSpan && warp == 0 && blockIdx.y == 0)
      report(a.dev_err, KVQ_DEV_ERR_SLOT);
    const bool first = in_pool && !(prev >= 0 && prev < nslots &&
                                    prev / kBlock == slot[q] / kBlock && prev < slot[q]);
    firsts |= static_cast<uint64_t>(__ballot_sync(kFullMask, first)) << (32 * q);
    live |= static_cast<uint64_t>(__ballot_sync(kFullMask, in_pool)) << (32 * q);
  }
  if ((firsts & ((1ull << kSpan) - 1ull)) == 0ull) return;  // (the same in every warp)

  const int h = blockIdx.y;
  const int64_t stride = static_cast<int64_t>(a.kv_heads) * kHeadDim;
  int lead[2], end[2];        // the run of this half-warp's row is rows [lead, end)
  uint32_t written[2], old[2][2];
  int64_t my_slot[2];
  bool active[2];
  uint4 x[2][2];              // [row][K or V]
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = 32 * q + 2 * warp + (lane >> 4);
    const uint64_t upto = firsts & ((2ull << row) - 1ull);
    lead[q] = upto != 0ull ? 63 - __clzll(upto) : kRows;
    active[q] = ((live >> row) & 1ull) != 0ull && lead[q] < kSpan;
    const uint64_t stops = (firsts | ~live) & ~((2ull << (lead[q] & 63)) - 1ull);
    end[q] = stops != 0ull ? __ffsll(stops) - 1 : kRows;
    my_slot[q] = __shfl_sync(kFullMask, slot[q], row & 31);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      x[q][side] = make_uint4(0u, 0u, 0u, 0u);
      old[q][side] = 0u;
      if (active[q]) {
        x[q][side] = ldg_stream16(static_cast<const uint16_t*>(side ? a.v_new : a.k_new) +
                                  ((tok0 + row) * a.kv_heads + h) * kHeadDim + 8 * l16);
        old[q][side] = static_cast<const uint8_t*>(
            side ? a.v_sz : a.k_sz)[my_slot[q] / kBlock * a.kv_heads + h];
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {  // the block offsets that each half's run writes
    written[q] = 0u;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int lo = __shfl_sync(kFullMask, lead[q], 16 * hf);
      const int hi = __shfl_sync(kFullMask, end[q], 16 * hf);
      uint32_t bit = lane >= lo && lane < hi ? 1u << (slot[0] % kBlock) : 0u;
      if (lane + 32 >= lo && lane + 32 < hi) bit |= 1u << (slot[1] % kBlock);
      const uint32_t all = __reduce_or_sync(kFullMask, bit);
      if ((lane >> 4) == hf) written[q] = all;
    }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint32_t m = half_max(amax8<BF>(x[q][side]));
      if (l16 == 0) smax[side][32 * q + 2 * warp + (lane >> 4)] = active[q] ? m : 0u;
    }
  __syncthreads();  // also: every row of a run has read the block's scales

#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = 32 * q + 2 * warp + (lane >> 4);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint32_t run_max =
          half_max(active[q] && lead[q] + l16 < end[q] ? smax[side][lead[q] + l16] : 0u);
      if (!active[q]) continue;  // (whole half-warps)
      const uint32_t bits =
          BF ? run_max << 16 : __float_as_uint(__half2float(__ushort_as_half(run_max)));
      const bool fresh = (written[q] & 1u) != 0u;
      const uint32_t was = old[q][side], now = max(fresh ? 0u : was, fp8_scale_for(bits));
      const int64_t blk = my_slot[q] / kBlock;
      if (row == lead[q] && l16 == 0)
        static_cast<uint8_t*>(side ? a.v_sz : a.k_sz)[blk * a.kv_heads + h] =
            static_cast<uint8_t>(now);
      // 2^-(now - 127); any finite factor serves a block of zeros
      const float inv = now == 0u    ? 1.f
                        : now < 254u ? __uint_as_float((254u - now) << 23)
                                     : __uint_as_float(now == 254u ? 0x00400000u : 0u);
      uint8_t* tile = static_cast<uint8_t*>(side ? a.v_pool : a.k_pool) +
                      (blk * kBlock * a.kv_heads + h) * kHeadDim + 8 * l16;
      const uint32_t w[4] = {x[q][side].x, x[q][side].y, x[q][side].z, x[q][side].w};
      uint32_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c[e] = f32_to_e4m3(lo_to_float<BF>(w[e]) * inv, hi_to_float<BF>(w[e]) * inv);
      *reinterpret_cast<uint2*>(tile + (my_slot[q] % kBlock) * stride) =
          make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
      if (!fresh && now > was) {  // the block's other rows, shared out over the run's half-warps
        const uint32_t by = now - was;
        rescale_rows(tile, stride, ~written[q] & 0xFFFFu, end[q] - lead[q], row - lead[q],
                     by > 30u ? 0.f : __uint_as_float((127u - by) << 23), was == 0u);
      }
    }
  }
}

}  // namespace

cudaError_t launch_store_fp8(const StoreArgs& a, cudaStream_t s) {
  if (a.num_tokens == 0) return cudaSuccess;
  const int64_t spans = (a.num_tokens + kSpan - 1) / kSpan;
  if (spans > 0x7FFFFFFFll || a.kv_heads > kMaxFp8Heads) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(spans), static_cast<unsigned>(a.kv_heads));
  if (a.in_dtype == kBF16)
    store_fp8_kernel<true><<<grid, kStoreThreads, 0, s>>>(a);
  else
    store_fp8_kernel<false><<<grid, kStoreThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
