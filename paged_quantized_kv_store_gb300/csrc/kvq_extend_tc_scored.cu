// kvq_extend_tc_scored: the tcgen05 extend attention over FP8 pools, and over
// INT8, INT4 and fp16 pools with scores that are capped, biased by distance, or
// masked by a window and a prefix. The roles are kvq_extend_tc.cu's.
//
// FP8 pools: the staging warpgroup writes K's codes as exact fp16 values, and
// the softmax multiplies a block's 16 scores by its scale (in the exponent's
// FMA, so this costs nothing: only the maximum is taken block by block). V's
// codes are staged as code * 2^(scale - reference), exact in fp16 while the
// block's scale lies within [-8, 7] powers of two of the unit's reference; when
// a tile's largest scale leaves that range the reference moves to it and O is
// rescaled in TMEM like for a moved maximum. The row sum's column is not. bf16
// queries enter as fp16 times a power of two for each row. The producer warp
// turns a tile's scales into these factors. A 64-token tile of 256 rows takes
// 1.13 us; left out in turn, the exponentials are 18 of a 4096-token prompt's
// 154 us (32/8 heads: 893 TFLOP/s), the staging 10, the wait for the last
// product 9, the maxima 6 and the products 3: the roles are balanced, and the
// softmax warpgroups' instructions come first.
//
// INT8 and INT4 pools with scores keep their codes exact in the products for
// queries of either type (an fp16 K dequantized once would put an error of
// 2^-11 sum |q k| into scores that a cap then spreads).
//
// Scores: the whole tile of a row goes through the cap and the bias in
// registers; a tile whose scores are all below 1.25 of the cap takes tanh by a
// polynomial on the FMA pipe (packed pairs), the others two special-function
// operations a score. A unit's tiles begin at its first query's window.
#include <cuda_runtime.h>

#include "kvq_extend_tc_body.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

struct Launch {
  const ExtendArgs& a;
  int grid;
  cudaStream_t s;
  template <int KV, bool QBF, bool OBF, bool SC, bool EX = false>
  cudaError_t run() const { return launch_tc_t<KV, QBF, OBF, SC, EX>(a, grid, s); }
  cudaError_t fail() const { return cudaErrorInvalidValue; }
};

struct Occupancy {
  int batch;
  template <int KV, bool QBF, bool OBF, bool SC, bool EX = false>
  int run() const { return tc_occupancy_t<KV, QBF, OBF, SC, EX>(batch); }
  int fail() const { return 0; }
};

template <bool SC, typename F>
auto with_kinds(int kv_dtype, int q_dtype, const F& f) -> decltype(f.fail()) {
  const bool qbf = q_dtype == kBF16;
  switch (kv_dtype) {
    case kF8:
      return qbf ? f.template run<kF8, false, true, SC>() : f.template run<kF8, false, false, SC>();
    case kF16:
      if constexpr (SC) return f.template run<kF16, false, false, true>();
      return f.fail();
    case kI8:
      if constexpr (SC)
        return qbf ? f.template run<kI8, true, true, true, true>()
                   : f.template run<kI8, false, false, true, true>();
      return f.fail();
    case kI4:
      if constexpr (SC)
        return qbf ? f.template run<kI4, true, true, true, true>()
                   : f.template run<kI4, false, false, true, true>();
      return f.fail();
    default:
      return f.fail();
  }
}

}  // namespace

cudaError_t launch_extend_tc_scored(const ExtendArgs& a, int kv_dtype, int q_dtype, bool scored,
                                    int grid, cudaStream_t s) {
  const Launch f{a, grid, s};
  return scored ? with_kinds<true>(kv_dtype, q_dtype, f) : with_kinds<false>(kv_dtype, q_dtype, f);
}

int extend_tc_scored_ctas_per_sm(int kv_dtype, int q_dtype, bool scored, int batch) {
  const Occupancy f{batch};
  return scored ? with_kinds<true>(kv_dtype, q_dtype, f) : with_kinds<false>(kv_dtype, q_dtype, f);
}

}  // namespace kvq
