// kvq_extend: extend (chunked prefill) attention over the paged, quantized pool.
//
// "pymllm Runtime Design", forward stage: an extend / prefill batch writes its
// prompt tokens into the KV cache and attends over them. LMDeploy article
// §2.3 "动态拆分与融合": a prefill longer than the 4096-token threshold is
// split into chunks prefilled in turn, so a chunk's queries attend the
// request's cached prefix and, causally, the chunk itself; §2.2 / §3.2 item 3:
// the KV is read through the block table.
//
// Request b holds kv_lens[b] tokens; its last C_b = qo_indptr[b+1] -
// qo_indptr[b] are the chunk, whose query i sits at position kv_lens[b] - C_b
// + i and attends positions 0 .. that position. The rows of the computation
// are (query, q head) pairs of one kv head, row = i * group + head, so all q
// heads of a kv head share every K/V block read. A work unit is (request, kv
// head, tile of 16 rows, part of the context); the per-block arithmetic is the
// shared-prefix kernel's (kvq_prefix.cu): S = Q K^T and O += P' V on
// mma.m16n8k16 with the 16 rows as M, the decode kernel's K/V fragments as B
// operands, scale/zero applied outside the products. Scores past a row's
// position are masked. Units are handed out by an atomic counter, longest
// tiles first. When the batch has too few tiles to fill the device, the
// context is cut into parts (pchunk blocks each) whose partial records a
// combine kernel merges; otherwise every unit writes its rows' outputs.
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_extend_body.cuh"
#include "kvq_internal.h"

namespace kvq {

cudaError_t launch_extend(const ExtendArgs& a, int kv_dtype, int q_dtype, int grid,
                          cudaStream_t s) {
  const bool qbf = q_dtype == kBF16;
  switch (kv_dtype) {
    case kF16:
      return launch_t<kF16, false>(a, grid, s);
    case kBF16:
      return launch_t<kBF16, true>(a, grid, s);
    case kI8:
      return qbf ? launch_t<kI8, true>(a, grid, s) : launch_t<kI8, false>(a, grid, s);
    case kI4:
      return qbf ? launch_t<kI4, true>(a, grid, s) : launch_t<kI4, false>(a, grid, s);
    default:
      return cudaErrorInvalidValue;
  }
}

int extend_ctas_per_sm(int kv_dtype, int q_dtype, int batch) {
  const bool qbf = q_dtype == kBF16;
  switch (kv_dtype) {
    case kF16: return occupancy_t<kF16, false>(batch);
    case kBF16: return occupancy_t<kBF16, true>(batch);
    case kI8: return qbf ? occupancy_t<kI8, true>(batch) : occupancy_t<kI8, false>(batch);
    case kI4: return qbf ? occupancy_t<kI4, true>(batch) : occupancy_t<kI4, false>(batch);
    default: return 0;
  }
}

}  // namespace kvq
