// kvq_decode: single-token decode attention over the paged, quantized pool.
//
// LMDeploy article (devpress.csdn.net) §3.2 item 3: generation attention reads
// a non-contiguous KV layout through indirect block pointers; §4.2: decoding
// has its own hand-written kernel; §2.2: per-sequence block tables of 16-token
// blocks; §2.4: INT8/INT4 KV with per-token, per-head scale and zero.
//
// Work decomposition
//   All the work is one stream of blocks ordered by (q-head group, request,
//   block), where a q-head group is a kv head with up to 8 of its q heads.
//   A persistent grid (as many CTAs as fit on the device) gives every warp
//   one contiguous range of the stream of equal length, so the split between
//   warps is exact whatever the mix of request lengths. Each CTA first scans
//   the request lengths into per-request block offsets in shared memory.
//   A warp streams its range through its own ring of shared-memory stages
//   (several blocks in flight: TMA tensor copies completing on an mbarrier
//   for INT8 tiles, per-lane cp.async otherwise), crossing request boundaries without
//   a pause: it writes the output of every request it covers entirely and,
//   for the request holding the first and the one holding the last block of
//   its range, a partial record (running max, sum, unnormalised output) that
//   the combine kernel merges with a log-sum-exp. All q heads of a kv head's
//   group are handled by the same warp, so every KV byte is read once.
//   Long shares (RangeMap) keep about nine tenths of the stream in such
//   static ranges and hand the rest out in short chunks from a counter, each
//   chunk a range of its own, so that warps that ran slower are not waited
//   for.
//
// Per-block arithmetic of one warp (16 tokens of one kv head):
//   S^T = K Q^T  with mma.m16n8k16: M = 16 tokens, N = 8 q heads (padded),
//                K = 128 dims in 8 steps (two independent accumulators).
//   O^T += V^T P'^T with M = 16 dims (8 steps over 128), N = 8 heads,
//                K = 16 tokens.
//   Quantized codes go into the tensor cores as exact 16-bit floats a + c,
//   made by writing the code into the mantissa of a constant (INT4: a shift
//   and a lop3 per two codes, a = 16, or a = 128 on the K side of bf16
//   queries; INT8 K side: one prmt per two codes, a = 1024, or a = -128
//   through fp32 for bf16 queries; INT8 V side: a
//   prmt and a packed subtract, centred, a = -128); the offset is removed
//   outside the products together with the per-token zero:
//   c S + Z = (a + c) S + Z - a S.
//     q.k = S (q.(a + c)) + (Z - a S) sum(q)
//     sum_t p_t v_t = sum_t P'_t (a + c_t) + sum_t p_t (Z_t + mid S_t)
//                     - (a + mid) sum_t P'_t,   P'_t = fp16(p_t S_t)
//   where the last sum runs over the rounded P' fed to the product, so their
//   rounding error only multiplies c - mid (mid = 2^(b-1)); for centred INT8
//   codes (a = -mid) that term vanishes. The INT4 offset of 16 keeps the P.V
//   accumulator within a few times its centred size, so its fp32
//   accumulation error stays negligible over long contexts. The P.V product is fp16 for quantized
//   pools whatever Q's type (P' = p S <= S fits fp16); bf16 pools carry P as a
//   bf16 hi + lo pair. The score fragment is transposed in registers
//   (movmatrix) to become the B operand of the second product.
//   Each lane's K and V reads are 8-64 contiguous bytes of a token row; the
//   dims are assigned to mma k-columns so that these stay contiguous (the dot
//   product does not depend on the order of the dims, and Q is permuted the
//   same way once per request).
#include <cuda_runtime.h>

#include "kvq_decode_body.cuh"
#include "kvq_decode_common.cuh"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_store_row.cuh"
#include "kvq_tables_item.cuh"
#include "kvq_tile.cuh"

namespace kvq {
namespace {

template <int KV, bool QBF, bool TAIL>
__global__ void __launch_bounds__(kDecodeThreads, TAIL && KV != kI4 ? 3 : 1)
    decode_kernel(const __grid_constant__ DecodeArgs a) {
  extern __shared__ __align__(128) unsigned char dsmem[];
  __shared__ int32_t warp_sum[kWarps];
  // the combine kernel may be scheduled now; it waits for this grid to finish
  asm volatile("griddepcontrol.launch_dependents;");
  decode_body<KV, QBF, TAIL>(a, dsmem, warp_sum, blockIdx.x, gridDim.x);
}

// The merge of one (request, q head) row that the decode did not finish
// itself, by one warp: the split-K records of the ranges its blocks were
// split between (slot 1 for the first when the request starts inside that
// range), then its shared-prefix records, if any (a request made of shared
// blocks only has nothing else). Log-sum-exp in the exp2 domain, 8 pieces
// per round of loads.
// The pieces a row has: records of ranges r_first .. r_first + nd - 1 of the
// decode, then npc shared-prefix records; nd + npc = 0 for a row that needs no
// merge.
struct Pieces {
  int64_t r_first, nd, seg_start;
  int hh, npc;
  RangeMap rm;
};

// W = 1: by one warp. W > 1: by the W warps of a CTA, each every W-th batch of
// pieces, joined in shared memory (sh) at the end.
template <bool QBF, int W = 1>
__device__ __forceinline__ void merge_pieces(const DecodeArgs& a, int64_t bh, int hh, int lane,
                                             int64_t r_first, int64_t nd, int64_t seg_start,
                                             const RangeMap& rm, int npc, int warp = 0,
                                             float (*sh)[kPartStride] = nullptr) {
  auto rec_of = [&](int64_t i) -> const float* {
    if (i < nd) {
      const int slot = (i == 0 && seg_start != range_start(rm, r_first)) ? 1 : 0;
      return a.part + (((r_first + i) * 2 + slot) * a.hpg + hh) * kPartStride;
    }
    return a.ppart + (bh * a.pmax_chunks + (i - nd)) * kPartStride;
  };
  const int64_t npieces = nd + npc;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float lsum = 0.f, M = -INFINITY;
  constexpr int kBatch = 8;  // pieces whose loads are in flight together
  for (int64_t base = kBatch * warp; base < npieces; base += W * kBatch) {
    // every lane reads each piece's maximum and sum (one address: broadcast)
    // and its own 4 columns, all loads of the batch issued before any use;
    // through L2, as other SMs wrote the records
    float mm[kBatch], ll[kBatch];
    float4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      mm[i] = -INFINITY;
      ll[i] = 0.f;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (base + i < npieces) {
        const float* rec = rec_of(base + i);
        mm[i] = __ldcg(rec + kHeadDim);
        ll[i] = __ldcg(rec + kHeadDim + 1);
        x[i] = __ldcg(reinterpret_cast<const float4*>(rec) + lane);
      }
    }
    float Mb = mm[0];
#pragma unroll
    for (int i = 1; i < kBatch; ++i) Mb = fmaxf(Mb, mm[i]);
    const float Mn = fmaxf(M, Mb);
    if (Mn == -INFINITY) continue;
    if (M != Mn && M != -INFINITY) {  // this batch raised the maximum
      const float al = exp2f(M - Mn);
      lsum *= al;
      acc.x *= al; acc.y *= al; acc.z *= al; acc.w *= al;
    }
    M = Mn;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float e = mm[i] == -INFINITY ? 0.f : exp2f(mm[i] - M);
      lsum += e * ll[i];
      acc.x += e * x[i].x; acc.y += e * x[i].y; acc.z += e * x[i].z; acc.w += e * x[i].w;
    }
  }
  if constexpr (W > 1) {
    reinterpret_cast<float4*>(sh[warp])[lane] = acc;
    if (lane == 0) {
      sh[warp][kHeadDim] = M;
      sh[warp][kHeadDim + 1] = lsum;
    }
    __syncthreads();
    if (warp != 0) return;
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < W; ++i) M = fmaxf(M, sh[i][kHeadDim]);
    lsum = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float m = sh[i][kHeadDim], e = m == -INFINITY ? 0.f : exp2f(m - M);
      const float4 x = reinterpret_cast<const float4*>(sh[i])[lane];
      lsum += e * sh[i][kHeadDim + 1];
      acc.x += e * x.x; acc.y += e * x.y; acc.z += e * x.z; acc.w += e * x.w;
    }
  }
  const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
  uint2 w;
  w.x = pack2<QBF>(acc.x * inv, acc.y * inv);
  w.y = pack2<QBF>(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + bh * kHeadDim)[lane] = w;
}

__device__ __forceinline__ Pieces pieces_of(const DecodeArgs& a, int64_t bh) {
  Pieces p;
  p.r_first = p.nd = p.seg_start = 0;
  p.hh = p.npc = 0;
  if (bh >= static_cast<int64_t>(a.batch) * a.q_heads) return p;
  const int b = static_cast<int>(bh / a.q_heads);
  const int hq = static_cast<int>(bh - static_cast<int64_t>(b) * a.q_heads);
  const int tb = a.hdr[0];
  RangeMap& rm = p.rm;
  rm.Pst = a.hdr[1];
  rm.C = a.hdr[2];
  rm.nwarps = a.hdr[3];
  rm.ntail = 0;  // not needed to map blocks to ranges
  rm.k = a.hdr[4];
  rm.tb = tb;
  const int32_t* cum = a.hdr + kHdrCum;
  const int nblk = cum[b + 1] - cum[b];
  const int skip = a.skip != nullptr ? a.skip[b] : 0;
  const int npc = skip > 0 ? (skip + a.pchunk - 1) / a.pchunk : 0;
  if (nblk == 0 && npc == 0) return p;  // zeroed by the decode kernel
  int hgi, hh;  // the row's q-head group in the stream, and its record row in the group
  if (a.cta_heads > 0) {  // grouped-query kernel: groups of cta_heads kv heads
    const int qpg = a.cta_heads * a.group;
    hgi = hq / qpg;
    hh = hq - hgi * qpg;
  } else {
    const int h = hq / a.group, within = hq - h * a.group;
    hgi = h * a.head_groups + within / kHeadsPerGroup;
    hh = within % kHeadsPerGroup;
  }
  const int64_t seg_start = static_cast<int64_t>(hgi) * tb + cum[b];
  p.hh = hh;
  p.seg_start = seg_start;
  if (nblk > 0) {
    p.r_first = range_of(rm, seg_start);
    const int64_t r_last = range_of(rm, seg_start + nblk - 1);
    if (p.r_first == r_last) return p;  // one range: written by the decode kernel
    p.nd = r_last - p.r_first + 1;
  }
  p.npc = npc;
  return p;
}

template <bool QBF>
__device__ __forceinline__ void combine_row(const DecodeArgs& a, int64_t bh, int lane) {
  const Pieces p = pieces_of(a, bh);
  if (p.nd + p.npc > 0)
    merge_pieces<QBF>(a, bh, p.hh, lane, p.r_first, p.nd, p.seg_start, p.rm, p.npc);
}

// One CTA of kWideWarps warps for each row. A row of a 100K-token request has
// over a hundred pieces, and with few rows one warp's rounds of loads were
// most of the merge: the call's 128 rows of about 150 pieces took 109 us with a
// warp each and 94.5 us so.
constexpr int kWideWarps = 8;

template <bool QBF>
__global__ void __launch_bounds__(32 * kWideWarps)
    combine_wide_kernel(const __grid_constant__ DecodeArgs a) {
  __shared__ __align__(16) float sh[kWideWarps][kPartStride];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Pieces p = pieces_of(a, blockIdx.x);
  if (p.nd + p.npc > 0)  // (the same for the whole CTA)
    merge_pieces<QBF, kWideWarps>(a, blockIdx.x, p.hh, threadIdx.x & 31, p.r_first, p.nd,
                                  p.seg_start, p.rm, p.npc, threadIdx.x >> 5, sh);
}

// Launched as a programmatic dependent of the decode kernel: its CTAs may
// start while the decode runs and wait here until the decode grid has
// finished and its records are visible.
template <bool QBF>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ DecodeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  combine_row<QBF>(a, static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5),
                   threadIdx.x & 31);
}

// ---- the fused step ------------------------------------------------------------

constexpr int kStepUnroll = 4;  // table entries / pool rows a half-warp has in flight

// Grid-wide barrier of a cooperative launch: thread 0 of every CTA counts in
// and waits, with acquire loads, until `target` CTAs have; the wait gives up
// after limit_ns (2 s in the step; KVQ_DEV_ERR_TIMEOUT, false: the caller
// stops).
__device__ __forceinline__ bool grid_sync(unsigned int* ctr, unsigned int target,
                                          int32_t* dev_err,
                                          uint64_t limit_ns = 2000000000ull) {
  __shared__ int ok_s;
  asm volatile("fence.proxy.async.global;" ::: "memory");  // global writes before TMA reads
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(ctr, 1u);
    int ok = 1;
    const uint64_t t0 = global_ns();
    for (;;) {
      unsigned int v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
      if (v >= target) break;
      if (global_ns() - t0 > limit_ns) {
        ok = 0;
        report(dev_err, KVQ_DEV_ERR_TIMEOUT);
        break;
      }
      __nanosleep(128);
    }
    __threadfence();
    ok_s = ok;
  }
  __syncthreads();
  asm volatile("fence.proxy.async.global;" ::: "memory");
  return ok_s != 0;
}

// One decode step: (1) block tables and the quantizing store of the new
// tokens, spread over the whole grid; (2) the decode, as decode_kernel; (3)
// the combine, one warp per (request, q head). The phases are separated by
// grid barriers, so the step is one launch instead of four.
template <int KV, bool QBF, bool TAIL>
__global__ void __launch_bounds__(kDecodeThreads, KV == kI4 && !TAIL ? kMaxCtasPerSm : 3)
    step_kernel(const __grid_constant__ StepArgs s) {
  extern __shared__ __align__(128) unsigned char dsmem[];
  __shared__ int32_t warp_sum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t gwarp = static_cast<int64_t>(blockIdx.x) * kWarps + (tid >> 5);
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  // (1) block tables, then the store: a half-warp per table entry and per pool
  // row, kStepUnroll of them with their loads in flight together
  const int lane16 = lane & 15;
  const int64_t hw = 2 * gwarp + (lane >> 4), nhw = 2 * nwarps;
  const int64_t entries = static_cast<int64_t>(s.t.batch) * s.t.max_blocks_per_seq;
  for (int64_t i = hw; i < entries; i += kStepUnroll * nhw)
    tables_blocks<kStepUnroll>(s.t, i, nhw, lane16);
  const int64_t rows = s.st.num_tokens * 2 * s.st.kv_heads;
  for (int64_t r = hw; r < rows; r += kStepUnroll * nhw) {
    RowIn in[kStepUnroll];
#pragma unroll
    for (int u = 0; u < kStepUnroll; ++u) in[u] = load_row<KV, QBF>(s.st, r + u * nhw, lane16);
#pragma unroll
    for (int u = 0; u < kStepUnroll; ++u) write_row<KV, QBF>(s.st, in[u], lane16);
  }
  if (!grid_sync(s.barrier, gridDim.x, s.d.dev_err)) return;
  // (2) decode
  decode_body<KV, QBF, TAIL>(s.d, dsmem, warp_sum, blockIdx.x, gridDim.x);
  if (!grid_sync(s.barrier, 2 * gridDim.x, s.d.dev_err)) return;
  // (3) combine
  for (int64_t bh = gwarp; bh < static_cast<int64_t>(s.d.batch) * s.d.q_heads; bh += nwarps)
    combine_row<QBF>(s.d, bh, lane);
}

// Self-test of the step's barrier: the grid's CTAs meet at one barrier that
// waits for one CTA more than the grid has, with a limit of limit_ns, so the
// wait runs out, reports KVQ_DEV_ERR_TIMEOUT and every CTA returns.
__global__ void __launch_bounds__(kDecodeThreads) barrier_selftest_kernel(unsigned int* ctr,
                                                                         int32_t* dev_err,
                                                                         uint64_t limit_ns) {
  grid_sync(ctr, gridDim.x + 1, dev_err, limit_ns);
}

template <int KV, bool QBF, bool TAIL>
cudaError_t launch_step_t(const StepArgs& a, int grid, cudaStream_t s) {
  thread_local int opted_in_device = -1;  // per host thread: no shared state
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (opted_in_device != dev) {
    e = cudaFuncSetAttribute(step_kernel<KV, QBF, TAIL>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem_bytes_for<KV>(kMaxBatch)));
    if (e != cudaSuccess) return e;
    opted_in_device = dev;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kDecodeThreads);
  cfg.dynamicSmemBytes = smem_bytes_for<KV>(a.d.batch);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeCooperative;  // every CTA resident: the barriers need it
  attr.val.cooperative = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, step_kernel<KV, QBF, TAIL>, a);
}

template <int KV, bool QBF, bool TAIL>
int step_occupancy_t(int batch) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  thread_local int cached_dev = -1, cached_batch = -1, cached_n = 0;
  if (dev == cached_dev && batch == cached_batch) return cached_n;
  if (cudaFuncSetAttribute(step_kernel<KV, QBF, TAIL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem_bytes_for<KV>(kMaxBatch))) != cudaSuccess)
    return 0;
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, step_kernel<KV, QBF, TAIL>, kDecodeThreads,
                                                    smem_bytes_for<KV>(batch)) != cudaSuccess)
    return 0;
  cached_dev = dev;
  cached_batch = batch;
  cached_n = n;
  return n;
}

template <int KV, bool QBF, bool TAIL>
cudaError_t launch_t(const DecodeArgs& a, int grid, cudaStream_t s) {
  // allow the largest dynamic shared memory the kernel can ask for, once
  // per device
  thread_local int opted_in_device = -1;  // per host thread: no shared state
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (opted_in_device != dev) {
    e = cudaFuncSetAttribute(decode_kernel<KV, QBF, TAIL>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem_bytes_for<KV>(kMaxBatch)));
    if (e != cudaSuccess) return e;
    opted_in_device = dev;
  }
  decode_kernel<KV, QBF, TAIL><<<grid, kDecodeThreads, smem_bytes_for<KV>(a.batch), s>>>(a);
  return cudaGetLastError();
}

template <int KV, bool QBF, bool TAIL>
int occupancy_t(int batch) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  thread_local int cached_dev = -1, cached_batch = -1, cached_n = 0;
  if (dev == cached_dev && batch == cached_batch) return cached_n;
  if (cudaFuncSetAttribute(decode_kernel<KV, QBF, TAIL>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem_bytes_for<KV>(kMaxBatch))) != cudaSuccess)
    return 0;
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, decode_kernel<KV, QBF, TAIL>,
                                                    kDecodeThreads,
                                                    smem_bytes_for<KV>(batch)) != cudaSuccess)
    return 0;
  cached_dev = dev;
  cached_batch = batch;
  cached_n = n;
  return n;
}

}  // namespace

namespace {

// f.run<KV, QBF, TAIL>() for the runtime pool kind, Q type and tail flag;
// f.fail() for a kind without a kernel.
template <typename F>
auto with_kinds(int kv_dtype, int q_dtype, bool tail, const F& f) -> decltype(f.fail()) {
  const bool qbf = q_dtype == kBF16;
  switch (kv_dtype) {
    case kF16:
      return tail ? f.template run<kF16, false, true>() : f.template run<kF16, false, false>();
    case kBF16:
      return tail ? f.template run<kBF16, true, true>() : f.template run<kBF16, true, false>();
    case kI8:
      if (qbf)
        return tail ? f.template run<kI8, true, true>() : f.template run<kI8, true, false>();
      return tail ? f.template run<kI8, false, true>() : f.template run<kI8, false, false>();
    case kI4:
      if (qbf)
        return tail ? f.template run<kI4, true, true>() : f.template run<kI4, true, false>();
      return tail ? f.template run<kI4, false, true>() : f.template run<kI4, false, false>();
    default:
      return f.fail();
  }
}

struct LaunchDecode {
  const DecodeArgs& a;
  int grid;
  cudaStream_t s;
  template <int KV, bool QBF, bool TAIL>
  cudaError_t run() const { return launch_t<KV, QBF, TAIL>(a, grid, s); }
  cudaError_t fail() const { return cudaErrorInvalidValue; }
};

struct LaunchStep {
  const StepArgs& a;
  int grid;
  cudaStream_t s;
  template <int KV, bool QBF, bool TAIL>
  cudaError_t run() const { return launch_step_t<KV, QBF, TAIL>(a, grid, s); }
  cudaError_t fail() const { return cudaErrorInvalidValue; }
};

struct DecodeOccupancy {
  int batch;
  template <int KV, bool QBF, bool TAIL>
  int run() const { return occupancy_t<KV, QBF, TAIL>(batch); }
  int fail() const { return 0; }
};

struct StepOccupancy {
  int batch;
  template <int KV, bool QBF, bool TAIL>
  int run() const { return step_occupancy_t<KV, QBF, TAIL>(batch); }
  int fail() const { return 0; }
};

}  // namespace

cudaError_t launch_decode(const DecodeArgs& a, int kv_dtype, int q_dtype, int grid,
                          cudaStream_t s) {
  return with_kinds(kv_dtype, q_dtype, a.tail_ctr != nullptr, LaunchDecode{a, grid, s});
}

cudaError_t launch_combine(const DecodeArgs& a, int q_dtype, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.batch) * a.q_heads;
  if (rows == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // overlap the decode's tail
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return q_dtype == kBF16 ? cudaLaunchKernelEx(&cfg, combine_kernel<true>, a)
                          : cudaLaunchKernelEx(&cfg, combine_kernel<false>, a);
}

cudaError_t launch_combine_wide(const DecodeArgs& a, int q_dtype, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.batch) * a.q_heads;
  if (rows == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows));
  cfg.blockDim = dim3(32 * kWideWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as launch_combine
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return q_dtype == kBF16 ? cudaLaunchKernelEx(&cfg, combine_wide_kernel<true>, a)
                          : cudaLaunchKernelEx(&cfg, combine_wide_kernel<false>, a);
}

cudaError_t launch_step(const StepArgs& a, int kv_dtype, int q_dtype, int grid,
                        cudaStream_t s) {
  return with_kinds(kv_dtype, q_dtype, a.d.tail_ctr != nullptr, LaunchStep{a, grid, s});
}

cudaError_t launch_barrier_selftest(unsigned int* ctr, int32_t* dev_err, int grid,
                                    uint64_t limit_ns, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kDecodeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeCooperative;  // as the step: every CTA resident
  attr.val.cooperative = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, barrier_selftest_kernel, ctr, dev_err, limit_ns);
}

int step_ctas_per_sm(int kv_dtype, int q_dtype, int batch, bool tail) {
  return with_kinds(kv_dtype, q_dtype, tail, StepOccupancy{batch});
}

int decode_ctas_per_sm(int kv_dtype, int q_dtype, int batch, bool tail) {
  return with_kinds(kv_dtype, q_dtype, tail, DecodeOccupancy{batch});
}

}  // namespace kvq
