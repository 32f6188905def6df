// eb_lmscore.cuh -- token log-probabilities and entropies from hidden states
// and the LM head: z = h W^T (h [rows, d], W [V, d], bf16) is formed tile by
// tile on the tensor cores and reduced on chip, so the logits never reach
// HBM.
//
// A CTA owns one 128-row tile and a contiguous range of the 256-wide
// vocabulary tiles.  Warp 0 loads (TMA), warp 1 issues tcgen05.mma into one
// of two TMEM accumulators, warps 2-5 hold one row per thread and fold each
// accumulator into the row's sums (row_sums of eb_score.cuh).  Columns past V
// and hidden elements past d read as zeros and the columns are left out.  The
// ranges' sums are joined in vocabulary order by lmscore_finish_kernel.
#pragma once

#include "eb_score.cuh"
#include "eb_tc.cuh"

namespace ebk {

constexpr int kLsBM = 128, kLsBN = 256, kLsBK = 64;
constexpr int kLsStages = 4;
constexpr int kLsThreads = 6 * 32;
constexpr uint32_t kLsABytes = kLsBM * kLsBK * 2, kLsBBytes = kLsBN * kLsBK * 2;
constexpr uint32_t kLsTmemCols = 2 * kLsBN;

using LmSums = RowSums;

struct LmScoreArgs {
  const int32_t* tokens;
  const float* temps;
  float temp;
  LmSums* sums;  // [n_split][rows]
  float* za;     // [rows] the tokens' logits
  int rows, V, d, n_split;
  uint64_t wait_ns;
  uint32_t* status;
  float* logprobs;
  float* entropies;
};

// Vocabulary ranges per row tile: one CTA per SM over all tiles.
inline int lm_score_split(int sms, int64_t rows, int64_t V) {
  const int64_t n_mt = (rows + kLsBM - 1) / kLsBM, n_nt = (V + kLsBN - 1) / kLsBN;
  const int64_t s = n_nt < sms / n_mt ? n_nt : sms / n_mt;
  return s < 1 ? 1 : (int)s;
}

// Most (range, row) records of any call of up to max_rows rows.
inline size_t lm_score_slots(int sms, int64_t max_rows) {
  const size_t wide = (size_t)sms * (size_t)kLsBM;
  return (size_t)max_rows > wide ? (size_t)max_rows : wide;
}

struct LmScoreLayout {
  uint32_t a, b, bars, total;
};
__host__ __device__ inline LmScoreLayout lm_score_layout() {
  LmScoreLayout y;
  y.a = 0;
  y.b = kLsStages * kLsABytes;
  y.bars = y.b + kLsStages * kLsBBytes;
  y.total = y.bars + 8u * (2 * kLsStages + 5) + 16u + 1024u;
  return y;
}

__device__ __forceinline__ float lm_temp(const LmScoreArgs& p, int row) {
  const float T = p.temps ? p.temps[row] : p.temp;
  return row_temp_ok(T) ? T : __int_as_float(0x7fc00000);
}

__global__ void __launch_bounds__(kLsThreads, 1)
    lmscore_kernel(const __grid_constant__ CUtensorMap tm_h,
                   const __grid_constant__ CUtensorMap tm_w, const LmScoreArgs p) {
  extern __shared__ unsigned char ls_smem_raw[];
  const LmScoreLayout lay = lm_score_layout();
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(ls_smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* sa = smem + lay.a;
  unsigned char* sb = smem + lay.b;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + lay.bars);
  uint64_t* empty = full + kLsStages;
  uint64_t* acc_full = empty + kLsStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_nt = (p.V + kLsBN - 1) / kLsBN;
  const int mt = blockIdx.x / p.n_split, ns = blockIdx.x % p.n_split;
  const int nt_lo = (int)((long long)ns * n_nt / p.n_split);
  const int nt_hi = (int)((long long)(ns + 1) * n_nt / p.n_split);
  const int n_tiles = nt_hi - nt_lo;
  const int KB = (p.d + kLsBK - 1) / kLsBK;

  if (tid == 0) {
    for (int s = 0; s < kLsStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) tc_alloc(tmem_slot, kLsTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&]() {
    atomicOr(p.status, kScoreTimeout);
    *(volatile int*)abort_flag = 1;
  };

  int issued = 0, consumed = 0;
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t keep = evict_last_policy(), once = evict_first_policy();
      for (int t = 0; t < n_tiles && !*(volatile int*)abort_flag; ++t) {
        for (int kb = 0; kb < KB; ++kb, ++issued) {
          const int s = issued % kLsStages;
          if (issued >= kLsStages && !mbar_wait(&empty[s], (uint32_t)(issued / kLsStages - 1) & 1u,
                                                p.wait_ns, abort_flag)) {
            fail();
            break;
          }
          mbar_arrive_expect_tx(&full[s], kLsABytes + kLsBBytes);
          tma_load_2d(sa + s * kLsABytes, &tm_h, kb * kLsBK, mt * kLsBM, &full[s], keep);
          tma_load_2d(sb + s * kLsBBytes, &tm_w, kb * kLsBK, (nt_lo + t) * kLsBN, &full[s], once);
        }
      }
      for (int i = max(0, issued - kLsStages); i < issued; ++i)
        mbar_wait(&full[i % kLsStages], (uint32_t)(i / kLsStages) & 1u, kDrainLimitNs);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = lm_idesc(kLsBM, kLsBN);
      const uint32_t a0 = smem_u32(sa), b0 = smem_u32(sb);
      for (int t = 0; t < n_tiles && !*(volatile int*)abort_flag; ++t) {
        const int buf = t & 1;
        if (t >= 2 && !mbar_wait(&acc_empty[buf], (uint32_t)(t / 2 - 1) & 1u, p.wait_ns,
                                 abort_flag)) {
          fail();
          break;
        }
        tc_fence_after();
        bool ok = true;
        for (int kb = 0; kb < KB; ++kb, ++consumed) {
          const int s = consumed % kLsStages;
          if (!mbar_wait(&full[s], (uint32_t)(consumed / kLsStages) & 1u, p.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kLsBK / 16; ++k)
            tc_mma(tmem + (uint32_t)(buf * kLsBN),
                   sw128_desc(a0 + (uint32_t)(s * kLsABytes + k * 32)),
                   sw128_desc(b0 + (uint32_t)(s * kLsBBytes + k * 32)), idesc,
                   (kb | k) != 0 ? 1u : 0u);
          tc_commit(&empty[s]);
        }
        if (!ok) {
          fail();
          break;
        }
        tc_commit(&acc_full[buf]);
      }
      tc_commit(drain);
      mbar_wait(drain, 0u, kDrainLimitNs);
    }
  } else {
    const int q = warp & 3;  // TMEM lanes 32 q .. 32 q + 31
    const int row = mt * kLsBM + 32 * q + lane;
    const bool valid = row < p.rows;
    const int token = valid ? p.tokens[row] : -1;
    const float c2 = valid ? kLog2e / lm_temp(p, row) : 1.f;
    RowSums s = row_sums_empty();
    for (int t = 0; t < n_tiles; ++t) {
      const int buf = t & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (uint32_t)(t / 2) & 1u, p.wait_ns,
                                             abort_flag))) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * kLsBN);
#pragma unroll 1
      for (int g = 0; g < kLsBN / 32; ++g) {
        float z[32];
        __syncwarp();  // tcgen05.ld is warp-wide: every lane, converged
        tc_ld32(taddr + (uint32_t)(g * 32), z);
        tc_wait_ld();
        const int v0 = (nt_lo + t) * kLsBN + g * 32;
        const int n = min(32, p.V - v0);
        if (n <= 0) continue;
        const int at = token - v0;
        if (at >= 0 && at < n) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i == at) {
              p.za[row] = z[i];
              z[i] = -INFINITY;
            }
        }
        if (n < 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i >= n) z[i] = -INFINITY;
        }
        float m = z[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) m = fmaxf(m, z[i]);
        if (m > s.m) s = row_sums_join(s, RowSums{m, 0.f, 0.f}, c2);
        float r4[4] = {}, q4[4] = {};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float d = (z[i] - s.m) * c2;
          d = d < -kDeep ? -kDeep : d;
          const float e = ex2(d);
          r4[i & 3] += e;
          q4[i & 3] = fmaf(e, d, q4[i & 3]);
        }
        s.R += (r4[0] + r4[1]) + (r4[2] + r4[3]);
        s.Q += (q4[0] + q4[1]) + (q4[2] + q4[3]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
    }
    // a cut-short pass leaves NaN, not stale sums
    if (*(volatile int*)abort_flag) s.R = __int_as_float(0x7fc00000);
    if (valid) p.sums[(size_t)ns * (size_t)p.rows + (size_t)row] = s;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    __syncwarp();
    tc_dealloc(tmem, kLsTmemCols);
    tc_relinquish();
  }
}

// One thread per row: the ranges' sums in vocabulary order, then the row's
// results.
__global__ void lmscore_finish_kernel(const LmScoreArgs p) {
  const int row = blockIdx.x * blockDim.x + threadIdx.x;
  if (row >= p.rows) return;
  const int token = p.tokens[row];
  if (token < 0) {
    p.logprobs[row] = 0.f;
    if (p.entropies) p.entropies[row] = 0.f;
    return;
  }
  const float c2 = kLog2e / lm_temp(p, row);
  RowSums s = p.sums[row];
  for (int k = 1; k < p.n_split; ++k)
    s = row_sums_join(s, p.sums[(size_t)k * (size_t)p.rows + (size_t)row], c2);
  const bool bad = token >= p.V;
  const RowResult r = row_result(s, bad ? __int_as_float(0x7fc00000) : p.za[row], c2);
  p.logprobs[row] = r.lp;
  if (p.entropies) p.entropies[row] = r.H;
  const uint32_t bits = (bad ? kScoreBadToken : 0u) | (r.finite ? 0u : kScoreNonFinite);
  if (bits) atomicOr(p.status, bits);
}

}  // namespace ebk
