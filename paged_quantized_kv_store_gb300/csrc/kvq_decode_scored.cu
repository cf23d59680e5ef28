// kvq_decode_scored: the decode attention over FP8 pools, and over pools of any
// kind with scores that are capped, biased by distance or windowed. Both are
// the general decode (kvq_decode.cu has the work decomposition and the
// arithmetic, kvq_decode_body.cuh what FP8 blocks and scores add), with the
// same stream, workspace and combine.
//
// LMDeploy article (devpress.csdn.net) §2.2: 16-token blocks reached through
// block tables; §3.2 item 3 and §4.2: generation attention reads the paged KV
// through indirect block pointers in its own kernel. The pages have no scales
// for a block and no score forms: models that cap, bias or window their scores
// read the same cache.
#include <cuda_runtime.h>

#include "kvq_decode_body.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

template <int KV, bool QBF, bool SC>
__global__ void __launch_bounds__(kDecodeThreads, KV == kI4 ? 1 : 3)
    decode_scored_kernel(const __grid_constant__ DecodeArgs a) {
  extern __shared__ __align__(128) unsigned char dsmem[];
  __shared__ int32_t warp_sum[kWarps];
  // the combine kernel may be scheduled now; it waits for this grid to finish
  asm volatile("griddepcontrol.launch_dependents;");
  if constexpr (Stage<KV>::kTma) {
    if (threadIdx.x == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.k_map)));
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.v_map)));
    }
  }
  decode_body<KV, QBF, true, SC>(a, dsmem, warp_sum, blockIdx.x, gridDim.x);
}

// The opt-in to the largest dynamic shared memory, once per host thread and
// device.
template <int KV, bool QBF, bool SC>
cudaError_t opt_in(int dev) {
  thread_local int opted_in_device = -1;
  if (opted_in_device == dev) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(decode_scored_kernel<KV, QBF, SC>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem_bytes_for<KV>(kMaxBatch)));
  if (e == cudaSuccess) opted_in_device = dev;
  return e;
}

struct Launch {
  const DecodeArgs& a;
  int grid;
  cudaStream_t s;
  template <int KV, bool QBF, bool SC>
  cudaError_t run() const {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = opt_in<KV, QBF, SC>(dev);
    if (e != cudaSuccess) return e;
    decode_scored_kernel<KV, QBF, SC>
        <<<grid, kDecodeThreads, smem_bytes_for<KV>(a.batch), s>>>(a);
    return cudaGetLastError();
  }
  cudaError_t fail() const { return cudaErrorInvalidValue; }
};

struct Occupancy {
  int batch;
  template <int KV, bool QBF, bool SC>
  int run() const {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || opt_in<KV, QBF, SC>(dev) != cudaSuccess) return 0;
    thread_local int cached_dev = -1, cached_batch = -1, cached_n = 0;
    if (dev == cached_dev && batch == cached_batch) return cached_n;
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, decode_scored_kernel<KV, QBF, SC>,
                                                      kDecodeThreads,
                                                      smem_bytes_for<KV>(batch)) != cudaSuccess)
      return 0;
    cached_dev = dev;
    cached_batch = batch;
    cached_n = n;
    return n;
  }
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

cudaError_t launch_decode_scored(const DecodeArgs& a, int kv_dtype, int q_dtype, bool scored,
                                 int grid, cudaStream_t s) {
  return with_kinds(kv_dtype, q_dtype, scored, Launch{a, grid, s});
}

int decode_scored_ctas_per_sm(int kv_dtype, int q_dtype, bool scored, int batch) {
  return with_kinds(kv_dtype, q_dtype, scored, Occupancy{batch});
}

}  // namespace kvq
