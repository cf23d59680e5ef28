// kvq_extend_scored: the extend attention over FP8 pools, and over pools of any
// kind with scores that are capped, biased by distance, or masked by a window
// and a prefix (kvq_extend_body.cuh), on mma.sync.
//
// "pymllm Runtime Design", forward stage: an extend batch attends over the
// cached prefix and its own tokens; LMDeploy article §2.2: through block
// tables. The pages have no scales for a block and no score forms.
#include <cuda_runtime.h>

#include "kvq_extend_body.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

struct Launch {
  const ExtendArgs& a;
  int grid;
  cudaStream_t s;
  template <int KV, bool QBF, bool SC>
  cudaError_t run() const { return launch_t<KV, QBF, SC>(a, grid, s); }
  cudaError_t fail() const { return cudaErrorInvalidValue; }
};

struct Occupancy {
  int batch;
  template <int KV, bool QBF, bool SC>
  int run() const { return occupancy_t<KV, QBF, SC>(batch); }
  int fail() const { return 0; }
};

// f.run<KV, QBF, SC>() for the runtime kinds; only FP8 pools have a kernel
// without scores here.
template <typename F>
auto with_kinds(int kv_dtype, int q_dtype, bool scored, const F& f) -> decltype(f.fail()) {
  const bool qbf = q_dtype == kBF16;
  if (kv_dtype == kF8 && !scored)
    return qbf ? f.template run<kF8, true, false>() : f.template run<kF8, false, false>();
  if (!scored) return f.fail();
  switch (kv_dtype) {
    case kF16: return f.template run<kF16, false, true>();
    case kBF16: return f.template run<kBF16, true, true>();
    case kF8: return qbf ? f.template run<kF8, true, true>() : f.template run<kF8, false, true>();
    case kI8: return qbf ? f.template run<kI8, true, true>() : f.template run<kI8, false, true>();
    case kI4: return qbf ? f.template run<kI4, true, true>() : f.template run<kI4, false, true>();
    default: return f.fail();
  }
}

}  // namespace

cudaError_t launch_extend_scored(const ExtendArgs& a, int kv_dtype, int q_dtype, bool scored,
                                 int grid, cudaStream_t s) {
  return with_kinds(kv_dtype, q_dtype, scored, Launch{a, grid, s});
}

cudaError_t launch_extend_combine(const ExtendArgs& a, bool out_bf16, cudaStream_t s) {
  return out_bf16 ? launch_combine_t<true>(a, s) : launch_combine_t<false>(a, s);
}

int extend_scored_ctas_per_sm(int kv_dtype, int q_dtype, bool scored, int batch) {
  return with_kinds(kv_dtype, q_dtype, scored, Occupancy{batch});
}

}  // namespace kvq
