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
// Work decomposition: a CTA takes the runs that begin in 16 consecutive
// tokens, for one kv head of K or of V; a half-warp has one of the 32 rows
// those runs can reach (16 bytes a lane), so a run's largest value meets in
// shared memory and nothing is read twice. Bound by HBM for a prefill chunk
// and by the launch for a decode step's rows.
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_fp8.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kSpan = 16;                   // tokens whose runs a CTA takes
constexpr int kRows = 2 * kSpan;            // rows those runs can reach
constexpr int kStoreThreads = 16 * kRows;   // a half-warp per row
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

template <bool BF>
__global__ void __launch_bounds__(kStoreThreads) store_fp8_kernel(const StoreArgs a) {
  __shared__ uint32_t smax[kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l16 = lane & 15;
  const int row = 2 * warp + (lane >> 4);
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * kSpan;
  const int64_t nslots = a.num_blocks * kBlock;

  // lane r of every warp looks at row r: the runs are the same for all warps
  const int64_t i = tok0 + lane;
  const int64_t slot = i < a.num_tokens ? a.slot_mapping[i] : -1;
  int64_t prev = __shfl_up_sync(kFullMask, slot, 1);
  if (lane == 0) prev = tok0 > 0 ? a.slot_mapping[tok0 - 1] : -1;
  const bool in_pool = slot >= 0 && slot < nslots;
  if (slot >= nslots && lane < kSpan && warp == 0 && blockIdx.y == 0)
    report(a.dev_err, KVQ_DEV_ERR_SLOT);
  const bool first = in_pool && !(prev >= 0 && prev < nslots && prev / kBlock == slot / kBlock &&
                                  prev < slot);
  const uint32_t firsts = __ballot_sync(kFullMask, first);
  const uint32_t live = __ballot_sync(kFullMask, in_pool);
  if ((firsts & ((1u << kSpan) - 1u)) == 0u) return;  // (the same in every warp)

  // this half-warp's row: its run is rows [lead, end)
  const uint32_t upto = firsts & ((2u << row) - 1u);
  const int lead = upto != 0u ? 31 - __clz(upto) : kRows;
  const bool active = ((live >> row) & 1u) != 0u && lead < kSpan;
  const uint32_t stops = (firsts | ~live) & ~((2u << (lead & 31)) - 1u);
  const int end = stops != 0u ? __ffs(stops) - 1 : kRows;
  // the block offsets that each half's run writes
  uint32_t written = 0u;
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const int lo = __shfl_sync(kFullMask, lead, 16 * hf), hi = __shfl_sync(kFullMask, end, 16 * hf);
    const uint32_t bit = lane >= lo && lane < hi ? 1u << (slot % kBlock) : 0u;
    const uint32_t all = __reduce_or_sync(kFullMask, bit);
    if ((lane >> 4) == hf) written = all;
  }
  const int64_t my_slot = __shfl_sync(kFullMask, slot, row);

  const int h = blockIdx.y >> 1;
  const bool is_v = (blockIdx.y & 1) != 0;
  const int64_t blk = active ? my_slot / kBlock : 0;
  uint8_t* scale = static_cast<uint8_t*>(is_v ? a.v_sz : a.k_sz) + blk * a.kv_heads + h;
  uint4 x = make_uint4(0u, 0u, 0u, 0u);
  uint32_t old = 0u;
  if (active) {
    x = ldg_stream16(static_cast<const uint16_t*>(is_v ? a.v_new : a.k_new) +
                     ((tok0 + row) * a.kv_heads + h) * kHeadDim + 8 * l16);
    old = *scale;
  }
  const uint32_t m = half_max(amax8<BF>(x));
  if (l16 == 0) smax[row] = active ? m : 0u;
  __syncthreads();  // also: every row of a run has read the block's scale

  const uint32_t run_max =
      half_max(active && lead + l16 < end ? smax[lead + l16] : 0u);
  if (!active) return;  // (whole half-warps; no full-warp operation follows)
  const uint32_t bits =
      BF ? run_max << 16 : __float_as_uint(__half2float(__ushort_as_half(run_max)));
  const bool fresh = (written & 1u) != 0u;
  const uint32_t now = max(fresh ? 0u : old, fp8_scale_for(bits));
  if (row == lead && l16 == 0) *scale = static_cast<uint8_t>(now);

  // 2^-(now - 127); any finite factor serves a block of zeros
  const float inv = now == 0u    ? 1.f
                    : now < 254u ? __uint_as_float((254u - now) << 23)
                                 : __uint_as_float(now == 254u ? 0x00400000u : 0u);
  uint8_t* tile = static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool) +
                  (blk * kBlock * a.kv_heads + h) * kHeadDim + 8 * l16;
  const int64_t stride = static_cast<int64_t>(a.kv_heads) * kHeadDim;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    c[e] = f32_to_e4m3(lo_to_float<BF>(w[e]) * inv, hi_to_float<BF>(w[e]) * inv);
  *reinterpret_cast<uint2*>(tile + (my_slot % kBlock) * stride) =
      make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);

  if (!fresh && now > old) {
    // the block's other rows move to the new scale, shared out over the run's
    // half-warps; all loads before the first store
    const uint32_t by = now - old;
    const float ratio = by > 30u ? 0.f : __uint_as_float((127u - by) << 23);
    const uint32_t keep = ~written & 0xFFFFu;
    const int n = end - lead;
    uint2 v[kBlock];
    uint32_t mine = 0u;
    int seen = 0;
#pragma unroll
    for (int o = 0; o < kBlock; ++o) {
      if ((keep >> o) & 1u) {
        if (seen == row - lead) {
          mine |= 1u << o;
          v[o] = *reinterpret_cast<const uint2*>(tile + o * stride);
        }
        seen = seen + 1 == n ? 0 : seen + 1;
      }
    }
#pragma unroll
    for (int o = 0; o < kBlock; ++o)
      if ((mine >> o) & 1u)
        *reinterpret_cast<uint2*>(tile + o * stride) =
            old == 0u ? make_uint2(0u, 0u)
                      : make_uint2(rescale4(v[o].x, ratio), rescale4(v[o].y, ratio));
  }
}

}  // namespace

cudaError_t launch_store_fp8(const StoreArgs& a, cudaStream_t s) {
  if (a.num_tokens == 0) return cudaSuccess;
  const int64_t spans = (a.num_tokens + kSpan - 1) / kSpan;
  if (spans > 0x7FFFFFFFll || a.kv_heads > kMaxFp8Heads) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(spans), static_cast<unsigned>(2 * a.kv_heads));
  if (a.in_dtype == kBF16)
    store_fp8_kernel<true><<<grid, kStoreThreads, 0, s>>>(a);
  else
    store_fp8_kernel<false><<<grid, kStoreThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
