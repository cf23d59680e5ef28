// kvq_extend_tc: extend (chunked prefill) attention on the 5th-generation
// tensor cores (tcgen05, accumulators in tensor memory), warp-specialised.
//
// Same computation as kvq_extend.cu ("pymllm Runtime Design", forward stage:
// extend / prefill; LMDeploy article §2.3: prefills split into chunks; §2.4:
// per-token, per-head INT8/INT4 scale and zero). A work unit is 256 rows
// (query, q head) of one kv head; the request's context is walked in tiles
// of 64 tokens (4 blocks). One CTA per SM, fourteen working warps (fifteen
// for INT8 pools) in five roles:
//   * raw-ring producer (warp 14, INT8 pools): hands out the work units (an
//     atomic counter, longest tiles first) and copies each tile's raw codes
//     and scale/zero words by TMA into a two-stage raw ring, one box per
//     (block, K or V), two tiles ahead of the staging warpgroup;
//   * staging warpgroup (warps 8-11): takes each tile's codes from the raw
//     ring (INT8) or straight from the pool (other kinds: per-thread
//     addresses fixed for the unit, the tile's four block ids fetched a tile
//     ahead; these pools' units are handed out here) and writes K in a
//     K-major 128-byte-swizzled tile and V transposed (dims as rows) into a
//     three-stage ring;
//   * two MMA warps (warps 12 and 13, one per softmax warpgroup g, on
//     different sub-partitions; one elected lane issues): S_g = Q_g K^T
//     (M 128, N 64, K 128) into the warpgroup's own TMEM columns, the next
//     tile's S_g as soon as warpgroup g has read the current one out of TMEM
//     (so it runs during that warpgroup's exponentials), and O_g += P_g V
//     (M 128, K 64, A read from TMEM) as soon as warpgroup g's P is ready;
//   * two softmax warpgroups (warps 0-3, 4-7), one thread per row: read the
//     row of S (tcgen05.ld), mask (causal, missing blocks), apply the online
//     softmax with a lazily moved maximum (a stale maximum only scales every
//     term alike; O is rescaled in TMEM when it moves), and write P to their
//     own TMEM columns (tcgen05.st).
// Numerics by query type:
//   * fp16 queries: K and V are staged dequantized, (c - mid) S + (Z + mid S)
//     in fp16 with one rounding; P = 2^(s - m) is computed as fp16 pairs, and
//     V's tile carries a row of ones, so the P V product also gives the row
//     sum over the same fp16 P. Output: O / l.
//   * bf16 queries: the codes stay exact (K as c - mid in bf16, V as c - mid
//     in fp16); s = S_k (q.(c - mid)) + (Z_k + mid S_k) sum(q) from per-token
//     arrays, P' = p S_v in fp16, and sum p and sum p (Z_v + mid S_v) in fp32
//     registers. Output: (O + z) / l.
// Roles meet only at mbarriers (no CTA-wide barrier inside the work loop);
// every wait is bounded (2 s, then KVQ_DEV_ERR_TIMEOUT and every role leaves
// its loop), and the MMA warps wait for their products in flight before the
// CTA frees its TMEM.
#include <cuda_runtime.h>

#include "kvq_extend_tc_body.cuh"
#include "kvq_internal.h"

namespace kvq {

int extend_tc_max_batch() { return kTcMaxBatch; }

bool extend_tc_supported(int kv_dtype, int q_dtype) {
  return kv_dtype == kI8 || kv_dtype == kI4 || kv_dtype == kF8 ||
         (kv_dtype == kF16 && q_dtype == kF16);
}

cudaError_t launch_extend_tc(const ExtendArgs& a, int kv_dtype, int q_dtype, int grid,
                             cudaStream_t s) {
  const bool qbf = q_dtype == kBF16;
  switch (kv_dtype) {
    case kF16:
      return launch_tc_t<kF16, false>(a, grid, s);
    case kI8:
      return qbf ? launch_tc_t<kI8, true>(a, grid, s) : launch_tc_t<kI8, false>(a, grid, s);
    case kI4:
      return qbf ? launch_tc_t<kI4, true>(a, grid, s) : launch_tc_t<kI4, false>(a, grid, s);
    default:
      return cudaErrorInvalidValue;
  }
}

int extend_tc_ctas_per_sm(int kv_dtype, int q_dtype, int batch) {
  const bool qbf = q_dtype == kBF16;
  switch (kv_dtype) {
    case kF16: return tc_occupancy_t<kF16, false>(batch);
    case kI8: return qbf ? tc_occupancy_t<kI8, true>(batch) : tc_occupancy_t<kI8, false>(batch);
    case kI4: return qbf ? tc_occupancy_t<kI4, true>(batch) : tc_occupancy_t<kI4, false>(batch);
    default: return 0;
  }
}

}  // namespace kvq
