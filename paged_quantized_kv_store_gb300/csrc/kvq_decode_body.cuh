// kvq_decode_body.cuh: the general decode of one CTA (see kvq_decode.cu for the
// work decomposition and the arithmetic), instantiated by the plain kernels
// (kvq_decode.cu), and by the FP8 and scored kernels (kvq_decode_scored.cu).
#pragma once

#include <cuda_runtime.h>

#include "kvq_decode_common.cuh"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_tile.cuh"

namespace kvq {

// One block of the stream for each lane: its pool block, q-head group and (FP8
// pools) scale bytes.
struct Window {
  int32_t phys;
  int hgi;
  uint32_t ke, ve;
};

// The decode of CTA `cta` out of `ncta` (the persistent grid); dsmem is the
// CTA's dynamic shared memory, warp_sum 4 ints of static shared memory.
// TAIL: the instantiation that can hand out tail chunks (make_range_map);
// without it a warp has one range, as the tail-free sizes want.
// SC: scores go through a.score (a cap, a distance bias, a window) before the
// softmax; the token positions below count from the first block read, which
// leaves distances to the query, the request's last token, as they are.
// FP8 pools (kvq_fp8.cuh): the codes enter both products as exact fp16. A
// block's K scale multiplies its scores. Its V scale goes into the weights as
// a power of two relative to the request's reference exponent (vref): while
// the block's lies within [-2, 10] of it the weights stay normal fp16 numbers,
// else the output so far is rescaled to the block's; the output takes the
// reference once, at the end.
template <int KV, bool QBF, bool TAIL, bool SC = false>
__device__ __forceinline__ void decode_body(const DecodeArgs& a, unsigned char* dsmem,
                                            int32_t* warp_sum, int cta, int ncta) {
  using S = Stage<KV>;
  constexpr bool kQuant = KvTraits<KV>::kQuant;
  constexpr bool kPvBf = KV == kBF16;  // P.V product type: bf16 only for bf16 pools
  constexpr bool kF8Pool = KV == kF8;
  constexpr bool kAhead = kF8Pool || SC;  // block ids and scales loaded windows ahead
  constexpr bool kQkBf = QBF && !kF8Pool;  // Q.K product type: FP8 pools take fp16 always
  constexpr float kAk = CodeOffset<KV, QBF>::kK;
  constexpr float kAv = CodeOffset<KV, QBF>::kV;
  constexpr float kMid = CodeOffset<KV, QBF>::kMid;
  constexpr bool kPCorr = CodeOffset<KV, QBF>::kPCorr;
  constexpr int D = S::kDepth;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;

  // ---- blocks per request, prefix-summed (every CTA); the cut into ranges ------
  constexpr bool kLockstep = KV != kI4;
  const StreamPlan sp = plan_stream<QBF, TAIL, SC>(a, dsmem, warp_sum, cta, ncta, kLockstep);
  const int32_t* cum = sp.cum;
  unsigned char* stages = sp.stages;
  const int tb = sp.tb;

  // ---- this warp's ranges: its static range, then tail chunks ----------------------
  // (no block barrier follows: warps are independent from here)
  const int64_t gw = static_cast<int64_t>(cta) * kWarps + warp;
  // this warp's stage region, 1024-byte aligned (the 128-byte swizzle repeats
  // every 1024 bytes)
  const uint32_t region0 =
      (static_cast<uint32_t>(__cvta_generic_to_shared(stages)) + 1023u) & ~1023u;
  const uint32_t wr = region0 + static_cast<uint32_t>(warp * S::kWarpBytes);
  LaneMap<KV> lm;
  lm.init(lane, g, t, static_cast<uint32_t>(a.kv_heads * S::kRow));
  if constexpr (S::kTma) {
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < D; ++i) mbar_init(wr + S::kBarOff + 8 * i);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
  }

  uint32_t phase = 0;  // parity to wait for, per stage (TMA path), across ranges
  // the range [x0, x0 + n), its records filed under range id rid; false when a
  // copy timed out (the warp stops)
  auto run_range = [&](const int64_t x0, const int n, const int64_t rid) -> bool {
    // issue side: cursor, a 32-entry window of the block table, validity bits
    Cursor ic;
    locate(ic, x0, cum, a.batch, tb);
    Cursor cc = ic;  // compute side
    int win_b = -1, win_j0 = 0;
    int32_t win = -1;
    // FP8 and scored kernels: windows of 32 blocks of the range (whatever
    // requests they belong to), a block a lane, loaded ahead: while one is
    // issued the next has its ids and its scale bytes are on the way, and so
    // are the ids of the one after it. Waiting for each window's ids and then
    // its scales once per 32 blocks cost 4 % on long contexts; loading a
    // block's scales as it was issued cost 20 % (the next use of the register
    // waits for the load of the newest block).
    Window w0, w1, w2;
    uint32_t ring_se = 0u;  // FP8 pools: scale bytes of the blocks in flight, stage s in lane s
    auto load_ids = [&](int first) -> Window {
      Window w;
      w.phys = -1;
      w.hgi = 0;
      w.ke = w.ve = 0u;
      if (first + lane < n) {
        Cursor c;
        locate(c, x0 + first + lane, cum, a.batch, tb);
        w.hgi = c.hgi;
        w.phys = __ldg(a.block_tables + static_cast<int64_t>(c.b) * a.max_blocks +
                       lead_of<SC>(a, c.b) + c.j);
      }
      return w;
    };
    auto load_scales = [&](Window& w) {
      if constexpr (kF8Pool) {
        if (w.phys >= 0 && w.phys < a.num_blocks) {
          const int64_t e = static_cast<int64_t>(w.phys) * a.kv_heads + w.hgi / a.head_groups;
          w.ke = __ldg(a.k_se + e);
          w.ve = __ldg(a.v_se + e);
        }
      }
    };
    if constexpr (kAhead) {
      w0 = load_ids(0);
      w1 = load_ids(32);
      w2 = w1;
      load_scales(w0);
    }
    uint32_t ok_mask = 0;  // stages holding a valid block in flight
    int k_issue = 0;   // next block of the range to issue
    int st_issue = 0;  // its stage
    auto issue_next = [&]() {
      if (k_issue < n) {
        int32_t phys;
        int h;
        if constexpr (kAhead) {
          const int kk = k_issue & 31;
          if (kk == 0) {
            if (k_issue > 0) {
              w0 = w1;
              w1 = w2;
            }
            load_scales(w1);
            w2 = load_ids(k_issue + 64);
          }
          phys = __shfl_sync(kFull, w0.phys, kk);
          h = __shfl_sync(kFull, w0.hgi, kk) / a.head_groups;
        } else {
        // (a range that crosses into the next q-head group of a lone request
        // starts over at its first block)
        if (ic.b != win_b || ic.j < win_j0 || ic.j >= win_j0 + 32) {
          win_b = ic.b;
          win_j0 = ic.j;
          const int jj = win_j0 + lane;
          win = jj < ic.nblk ? a.block_tables[static_cast<int64_t>(ic.b) * a.max_blocks +
                                              lead_of<SC>(a, ic.b) + jj]
                             : -1;
        }
        phys = __shfl_sync(kFull, win, ic.j - win_j0);
        h = ic.hgi / a.head_groups;
        }
        const bool ok = phys >= 0 && phys < a.num_blocks;
        const uint32_t bit = 1u << st_issue;
        if (ok) {
          issue_block<KV>(wr, st_issue, a, lm, phys, h, lane);
          ok_mask |= bit;
        } else {
          ok_mask &= ~bit;
          if (lane == 0) report(a.dev_err, KVQ_DEV_ERR_BLOCK_ID);
        }
        if constexpr (kF8Pool) {
          const uint32_t se = __shfl_sync(kFull, w0.ke | w0.ve << 8, k_issue & 31);
          if (lane == st_issue) ring_se = se;
        }
        if constexpr (!kAhead) {
          if (k_issue + 1 < n) advance(ic, cum, a.batch);
        }
      }
      if constexpr (!S::kTma) cp_async_commit();
      ++k_issue;
      st_issue = st_issue == D - 1 ? 0 : st_issue + 1;
    };
  #pragma unroll
    for (int k = 0; k < D - 1; ++k) issue_next();

    // ---- per-request state ---------------------------------------------------------
    int seg_b = -1, seg_hgi = -1, hq0 = 0, nh = 0, L = 0, seg_nblk = 0, seg_skip = 0;
    int64_t seg_start = 0;
    uint32_t qb[8][2];
    float qs0 = 0.f, qs1 = 0.f;  // sum(q) of heads 2t and 2t+1
    bool hv0 = false, hv1 = false;
    uint32_t vref = 0u;           // FP8 pools: scale byte o is counted in (0: none yet)
    float qd0 = 1.f, qd1 = 1.f;   // FP8 pools, bf16 queries: factors of heads 2t, 2t + 1
    float sl0 = 0.f, sl1 = 0.f;   // distance bias of those heads, times log2(e)
    int wlo = 0;                  // first token inside the window
    float o[8][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, z0 = 0.f, z1 = 0.f;
    float r0 = 0.f, r1 = 0.f;  // sums of the 16-bit P' values fed to the P.V product

    // writes the finished state of request seg_b: the output if this warp
    // covered all of its blocks, else a partial record
    auto flush = [&]() {
  #pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(kFull, l0, off);
        l1 += __shfl_xor_sync(kFull, l1, off);
        if constexpr (kQuant) {
          z0 += __shfl_xor_sync(kFull, z0, off);
          z1 += __shfl_xor_sync(kFull, z1, off);
          if constexpr (kPCorr) {
            r0 += __shfl_xor_sync(kFull, r0, off);
            r1 += __shfl_xor_sync(kFull, r1, off);
          }
        }
      }
      if constexpr (kPCorr) {
        // o = sum P'(a + c) + sum p (Z + mid S) - (a + mid) sum P'
        z0 -= (kAv + kMid) * r0;
        z1 -= (kAv + kMid) * r1;
      }
      if constexpr (kF8Pool) {
        const float unit = fp8_scale(vref);
  #pragma unroll
        for (int i = 0; i < 8; ++i)
  #pragma unroll
          for (int c = 0; c < 4; ++c) o[i][c] *= unit;
      }
      const bool contained = seg_start >= x0 && seg_start + seg_nblk <= x0 + n;
      const int64_t row0 = static_cast<int64_t>(seg_b) * a.q_heads + hq0;
  #pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int hh = 2 * t + u;
        if (hh >= nh) continue;
        const float z = u ? z1 : z0, l = u ? l1 : l0, m = u ? m1 : m0;
        if (contained) {
          float acc[16];
  #pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[2 * i] = o[i][u] + z;
            acc[2 * i + 1] = o[i][2 + u] + z;
          }
          float mm = m, ll = l;
          if (seg_skip > 0) merge_prefix(a, row0 + hh, seg_skip, g, mm, ll, acc);
          const float inv = ll > 0.f ? 1.f / ll : 0.f;
          uint32_t w[8];
  #pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = pack2<QBF>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                                (row0 + hh) * kHeadDim + 16 * g);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          const int slot = seg_start <= x0 ? 0 : 1;  // the request holding x0, else the last one
          float* rec = a.part + ((rid * 2 + slot) * a.hpg + hh) * kPartStride;
          float4* ov = reinterpret_cast<float4*>(rec + 16 * g);
  #pragma unroll
          for (int i = 0; i < 8; i += 2)
            ov[i / 2] =
                make_float4(o[i][u] + z, o[i][2 + u] + z, o[i + 1][u] + z, o[i + 1][2 + u] + z);
          if (g == 0) {
            rec[kHeadDim] = m;
            rec[kHeadDim + 1] = l;
          }
        }
      }
    };

    int st = 0;  // stage of block k
    for (int k = 0; k < n; ++k) {
      issue_next();  // refills the stage block k - 1 used
      const bool blk_ok = (ok_mask >> st) & 1u;
      if constexpr (S::kTma) {
        if (blk_ok) {
          if (!mbar_wait(wr + S::kBarOff + 8 * st, (phase >> st) & 1u)) {
            // a copy did not land: report, wait (bounded) for the other copies
            // this warp started, and stop
            if (lane == 0) report(a.dev_err, KVQ_DEV_ERR_TIMEOUT);
            const uint32_t rest = ok_mask & ~(1u << st);
            for (int i = 0; i < D; ++i)
              if ((rest >> i) & 1u) mbar_wait(wr + S::kBarOff + 8 * i, (phase >> i) & 1u);
            return false;
          }
          phase ^= 1u << st;
        }
      } else {
        cp_async_wait<D - 1>();  // this lane's copies of block k have landed
        __syncwarp();            // ... and every other lane's
      }

      if (cc.b != seg_b || cc.hgi != seg_hgi) {
        if (seg_b >= 0) flush();
        // start request cc.b for q-head group cc.hgi
        seg_b = cc.b;
        seg_hgi = cc.hgi;
        seg_nblk = cc.nblk;
        seg_start = static_cast<int64_t>(cc.hgi) * tb + cum[cc.b];
        const int h = cc.hgi / a.head_groups;
        const int hg = cc.hgi - h * a.head_groups;
        hq0 = h * a.group + hg * kHeadsPerGroup;
        nh = min(kHeadsPerGroup, a.group - hg * kHeadsPerGroup);
        seg_skip = SC ? 0 : skip_of(a, cc.b);
        // tokens of this request's own blocks
        L = clamped_len(a, cc.b) - kBlock * lead_of<SC>(a, cc.b);
        // Q fragments (B operand of S^T = K Q^T), permuted like the K dims
        uint32_t qw[16];
        if (g < nh) {
          const uint4* qp = reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(a.q) +
              (static_cast<int64_t>(cc.b) * a.q_heads + hq0 + g) * kHeadDim + 32 * t);
  #pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = qp[i];
            qw[4 * i] = v.x; qw[4 * i + 1] = v.y; qw[4 * i + 2] = v.z; qw[4 * i + 3] = v.w;
          }
        } else {
  #pragma unroll
          for (int i = 0; i < 16; ++i) qw[i] = 0u;
        }
        if constexpr (kF8Pool && QBF) {
          const float down = q_to_f16(qw);  // lanes 4h hold head h
          qd0 = __shfl_sync(kFull, down, (2 * t) * 4);
          qd1 = __shfl_sync(kFull, down, (2 * t + 1) * 4);
        }
        if constexpr (KV == kI4) {
  #pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const int j = kk >> 1, u = kk & 1;
            qb[kk][0] = prmt(qw[4 * j + u], qw[4 * j + u + 2], 0x5410u);
            qb[kk][1] = prmt(qw[4 * j + u], qw[4 * j + u + 2], 0x7632u);
          }
        } else {
  #pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            qb[kk][0] = qw[2 * kk];
            qb[kk][1] = qw[2 * kk + 1];
          }
        }
        if constexpr (kQuant) {
          float part = 0.f;
  #pragma unroll
          for (int i = 0; i < 16; ++i) part += lo_to_float<QBF>(qw[i]) + hi_to_float<QBF>(qw[i]);
          part += __shfl_xor_sync(kFull, part, 1);
          part += __shfl_xor_sync(kFull, part, 2);
          qs0 = __shfl_sync(kFull, part, (2 * t) * 4);  // lanes 4h hold sum(q) of head h
          qs1 = __shfl_sync(kFull, part, (2 * t + 1) * 4);
        }
        hv0 = 2 * t < nh;
        hv1 = 2 * t + 1 < nh;
        if constexpr (SC) {
          wlo = a.score.window > 0 ? max(L - a.score.window, 0) : 0;
          if (a.score.slopes != nullptr) {
            sl0 = hv0 ? a.score.slopes[hq0 + 2 * t] * 1.4426950408889634f : 0.f;
            sl1 = hv1 ? a.score.slopes[hq0 + 2 * t + 1] * 1.4426950408889634f : 0.f;
          }
        }
        vref = 0u;
  #pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = z0 = z1 = r0 = r1 = 0.f;
      }

      if (blk_ok) {
        ok_mask &= ~(1u << st);
        Frag<KV> cur;
        read_frag<KV>(cur, wr, st, lm, g);
        uint32_t ke = 0u, ve = 0u;  // FP8 pools: the block's scale bytes
        if constexpr (kF8Pool) {
          const uint32_t se = __shfl_sync(kFull, ring_se, st);
          ke = se & 0xFFu;
          ve = se >> 8;
          if (ve == 0u) clear_v_rows<KV>(cur, t, 0, 0);
        }
        if constexpr (kF8Pool || SC) {
          const int left = L - cc.j * kBlock, skip = wlo - cc.j * kBlock;
          if (left < kBlock || skip > 0) clear_v_rows<KV>(cur, t, skip, left);
          if constexpr (kQuant) {  // ... and the scale/zero words of those tokens
            if (g >= left || g < skip) cur.vsz[0] = 0u;
            if (g + 8 >= left || g + 8 < skip) cur.vsz[1] = 0u;
          }
        }
        // S^T = K Q^T, even and odd k-steps in two accumulators
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
  #pragma unroll
        for (int kk = 0; kk < 8; kk += 2) {
          uint32_t ak[4];
          k_operand<KV, QBF>(cur, kk, ak);
          mma16816<kQkBf>(sa, ak, qb[kk]);
          k_operand<KV, QBF>(cur, kk + 1, ak);
          mma16816<kQkBf>(sb, ak, qb[kk + 1]);
        }
        const float sc0 = sa[0] + sb[0], sc1 = sa[1] + sb[1];
        const float sc2 = sa[2] + sb[2], sc3 = sa[3] + sb[3];
        // scores of tokens g, g+8 for heads 2t, 2t+1, in the exp2 domain
        const int tok0 = cc.j * kBlock + g, tok1 = tok0 + 8;
        float s00, s01, s10, s11;
        if constexpr (kQuant) {
          // q.k = S (q.(a + c)) + (Z - a S) sum(q)
          const float S0 = half_lo(cur.ksz[0]), Z0 = half_hi(cur.ksz[0]) - kAk * S0;
          const float S1 = half_lo(cur.ksz[1]), Z1 = half_hi(cur.ksz[1]) - kAk * S1;
          s00 = (S0 * sc0 + Z0 * qs0) * a.sm_scale_log2;
          s01 = (S0 * sc1 + Z0 * qs1) * a.sm_scale_log2;
          s10 = (S1 * sc2 + Z1 * qs0) * a.sm_scale_log2;
          s11 = (S1 * sc3 + Z1 * qs1) * a.sm_scale_log2;
        } else if constexpr (kF8Pool) {
          const float f = fp8_scale(ke) * a.sm_scale_log2;
          const float f0 = QBF ? f * qd0 : f, f1 = QBF ? f * qd1 : f;
          s00 = ke != 0u ? sc0 * f0 : 0.f;
          s01 = ke != 0u ? sc1 * f1 : 0.f;
          s10 = ke != 0u ? sc2 * f0 : 0.f;
          s11 = ke != 0u ? sc3 * f1 : 0.f;
        } else {
          s00 = sc0 * a.sm_scale_log2;
          s01 = sc1 * a.sm_scale_log2;
          s10 = sc2 * a.sm_scale_log2;
          s11 = sc3 * a.sm_scale_log2;
        }
        if constexpr (SC) {
          if (a.score.cap > 0.f) {
            s00 = softcap(a.score, s00);
            s01 = softcap(a.score, s01);
            s10 = softcap(a.score, s10);
            s11 = softcap(a.score, s11);
          }
          if (a.score.slopes != nullptr) {
            const float d0 = static_cast<float>(L - 1 - tok0), d1 = d0 - 8.f;
            s00 -= sl0 * d0;
            s01 -= sl1 * d0;
            s10 -= sl0 * d1;
            s11 -= sl1 * d1;
          }
          if (tok0 < wlo) s00 = s01 = -INFINITY;
          if (tok1 < wlo) s10 = s11 = -INFINITY;
        }
        if (tok0 >= L) s00 = s01 = -INFINITY;
        if (tok1 >= L) s10 = s11 = -INFINITY;
        if (!hv0) s00 = s10 = 0.f;  // padded heads: finite, never written
        if (!hv1) s01 = s11 = 0.f;
        // the running maximum moves only when some lane holds a larger score:
        // then reduce the block maximum over the 16 tokens (lanes with equal t)
        // and rescale the running state
        float bm0 = fmaxf(s00, s10), bm1 = fmaxf(s01, s11);
        float mn0 = m0, mn1 = m1;
        if (__any_sync(kFull, bm0 > m0 || bm1 > m1)) {
  #pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            bm0 = fmaxf(bm0, __shfl_xor_sync(kFull, bm0, off));
            bm1 = fmaxf(bm1, __shfl_xor_sync(kFull, bm1, off));
          }
          mn0 = fmaxf(m0, bm0);
          mn1 = fmaxf(m1, bm1);
          const float al0 = ex2(m0 - mn0), al1 = ex2(m1 - mn1);
          l0 *= al0;
          l1 *= al1;
          z0 *= al0;
          z1 *= al1;
          r0 *= al0;
          r1 *= al1;
  #pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i][0] *= al0; o[i][2] *= al0;
            o[i][1] *= al1; o[i][3] *= al1;
          }
        }
        m0 = mn0;
        m1 = mn1;
        const float p00 = ex2(s00 - mn0), p10 = ex2(s10 - mn0);
        const float p01 = ex2(s01 - mn1), p11 = ex2(s11 - mn1);
        l0 += p00 + p10;
        l1 += p01 + p11;
        float q00 = p00, q01 = p01, q10 = p10, q11 = p11;
        if constexpr (kQuant) {
          // sum_t p_t v_t = sum_t P'_t (a + c_t) + sum_t p_t (Z_t + mid S_t)
          //                 - (a + mid) sum_t P'_t,  with P'_t = p_t S_t in fp16:
          // subtracting the rounded P' actually used leaves their rounding
          // error multiplied by c - mid only, as if the codes were centred
          const float S0 = half_lo(cur.vsz[0]), Z0 = half_hi(cur.vsz[0]) + kMid * S0;
          const float S1 = half_lo(cur.vsz[1]), Z1 = half_hi(cur.vsz[1]) + kMid * S1;
          z0 += p00 * Z0 + p10 * Z1;
          z1 += p01 * Z0 + p11 * Z1;
          q00 *= S0; q01 *= S0; q10 *= S1; q11 *= S1;
        }
        if constexpr (kF8Pool) {
          if (ve != 0u) {
            int d = static_cast<int>(ve) - static_cast<int>(vref);
            if (vref == 0u) {  // nothing but blocks of zeros so far
              vref = ve;
              d = 0;
            } else if (d > 10 || (d < -2 && d >= -90)) {
              // 2^-d; blocks 2^90 below the reference only lose what is lost
              // in the output's own rounding
              const float by = d > 126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - d) << 23);
  #pragma unroll
              for (int i = 0; i < 8; ++i)
  #pragma unroll
                for (int c = 0; c < 4; ++c) o[i][c] *= by;
              vref = ve;
              d = 0;
            }
            const float f = d < -90 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + d) << 23);
            q00 *= f; q01 *= f; q10 *= f; q11 *= f;
          }
        }
        // P'^T as the B operand: transpose the (token x head) fragments
        uint32_t bp[2], bp_lo[2];
        const uint32_t h0 = pack2<kPvBf>(q00, q01), h1 = pack2<kPvBf>(q10, q11);
        if constexpr (kPCorr) {
          r0 += lo_to_float<false>(h0) + lo_to_float<false>(h1);
          r1 += hi_to_float<false>(h0) + hi_to_float<false>(h1);
        }
        bp[0] = movmatrix_trans(h0);
        bp[1] = movmatrix_trans(h1);
        if constexpr (kPvBf) {
          // bf16 keeps 8 bits of P: add the rounding residual in a second
          // product so P carries ~16 bits (P = hi + lo)
          bp_lo[0] = movmatrix_trans(pack2<true>(q00 - lo_to_float<true>(h0),
                                                 q01 - hi_to_float<true>(h0)));
          bp_lo[1] = movmatrix_trans(pack2<true>(q10 - lo_to_float<true>(h1),
                                                 q11 - hi_to_float<true>(h1)));
        }
        // O^T += V^T P'^T
  #pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t av[4];
          v_operand<KV>(cur, i, av);
          mma16816<kPvBf>(o[i], av, bp);
          if constexpr (kPvBf) mma16816<true>(o[i], av, bp_lo);
        }
      }
      __syncwarp();  // all lanes are done with this stage before it is refilled
      st = st == D - 1 ? 0 : st + 1;
      if (k + 1 < n) advance(cc, cum, a.batch);
    }
    if constexpr (!S::kTma) cp_async_wait<0>();
    flush();
    return true;
  };  // run_range

  if constexpr (kF8Pool || SC) {
    if (a.whole) {  // a warp for each (q-head group, request): nothing to merge
      if (gw < static_cast<int64_t>(sp.groups) * a.batch) {
        const int hgi = static_cast<int>(gw / a.batch);
        const int b = static_cast<int>(gw - static_cast<int64_t>(hgi) * a.batch);
        const int nblk = cum[b + 1] - cum[b];
        if (nblk > 0) run_range(static_cast<int64_t>(hgi) * tb + cum[b], nblk, 0);
      }
      return;
    }
  }
  for_each_range<TAIL>(a, sp, gw, lane, run_range);
}

}  // namespace kvq
