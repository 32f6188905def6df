// eb_lmscore.cuh -- token log-probabilities and entropies from hidden states
// and the LM head: z = h W^T (h [rows, d], W [V, d], bf16) is formed tile by
// tile on the tensor cores and reduced on chip, so the logits never reach
// HBM.
//
// A pair of CTAs (a cluster of two, one per SM) owns 256 rows and a contiguous
// range of the 256-wide vocabulary tiles; each CTA loads its own 128 rows of h
// and half of each W tile, and one tcgen05.mma.cta_group::2 works on both
// SMs' shared memory, so a W tile crosses the L2 once per pair.  Roles:
//   warp 0     loads (TMA, 128-byte swizzle) into a ring of 32 KB stages; both
//              CTAs' copies are counted by the first CTA's barriers;
//   warp 1     of the first CTA issues the MMAs (M = 256, N = 256, K = 16) into
//              one of two accumulators (2 x 256 TMEM columns in each CTA);
//   warps 2-9  read the accumulators: a thread holds one row and 128 columns.
//
// The tensor cores add each K = 16 step's products to the accumulator with
// truncation: about 2^-26 of the sum lost per step, always toward zero (1.6e-8
// measured; over the 160 steps of d = 2560 a logit of 10 was 2.6e-5 low, five
// times what fp32 summation loses).  So an accumulator takes 512 elements of
// K at most, and the pieces are added in registers, rounded to nearest (2048
// rows: 3 % of the time against 1024 elements, for half the error; 256 elements
// would take 15 % more).
//
// Where a pair's product would be half padding (65 to 128 rows, and small odd
// numbers of 128-row tiles) each CTA works alone, with M = 128.
//
// Up to 64 rows that product would be mostly padding too: lmfew_kernel turns it
// around (W's rows on the 128 TMEM lanes, h's as 32 or 64 columns), so that
// only the reading of W is left.
//
// Vocabulary ids past V and hidden elements past d read as zeros; the ids are
// left out of the sums.  The ranges' sums are joined in vocabulary order by
// lmscore_finish_kernel.
//
// What bounds them, at 262144 ids and d = 2560: up to 64 rows the reading of W
// (24 rows 208 us, 6.5 TB/s, 0.98 of the measured copy rate).  Above that the
// tensor cores (84 % busy at 512 rows), and under a steady load the chip's
// power: 256 rows 356 us (273 in a short burst, at 1.26 PFLOP/s; 234 of zeros,
// close to the reading of W), 2048 rows 2.11 ms (1.30 PFLOP/s, 0.93 of what a
// library product sustains; a library product of the same sizes, which writes
// the logits, 2.10).  W asked for in L2 some stages ahead: 5 to 15 % slower.
#pragma once

#include "eb_score.cuh"
#include "eb_tc.cuh"

namespace ebk {

constexpr int kLsRows = 128;          // rows per CTA
constexpr int kLsBN = 256, kLsBK = 64;
constexpr int kLsHalf = kLsBN / 2;    // rows of W in one copy, columns a thread holds
constexpr int kLsChunk = 8;           // stages of one accumulator: 512 elements of K
constexpr int kLsEpiWarps = 8;
constexpr int kLsThreads = (2 + kLsEpiWarps) * 32;
constexpr uint32_t kLsABytes = kLsRows * kLsBK * 2, kLsBBytes = kLsHalf * kLsBK * 2;
template <bool PAIR>
struct LsShape {
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kBM = kCtas * kLsRows;     // rows of a tile
  static constexpr int kCopies = PAIR ? 1 : 2;    // of W's tile, by this CTA
  static constexpr int kStages = PAIR ? 6 : 4;
  static constexpr uint32_t kStage = kLsABytes + kCopies * kLsBBytes;
  static constexpr uint32_t kBars = kStages * kStage,
                            kSmem = kBars + 8 * (2 * kStages + 5) + 16 + 1024;
};
constexpr uint32_t kLsTmemCols = 2 * kLsBN;

using LmSums = RowSums;

struct LmScoreArgs {
  const int32_t* tokens;
  const float* temps;
  float temp;
  LmSums* sums;  // [n_rec][rows]
  float* za;     // [rows] the tokens' logits
  int rows, V, d;
  int n_split;  // vocabulary ranges (per row tile)
  int n_rec;    // records per row
  uint64_t wait_ns;
  uint32_t* status;
  float* logprobs;
  float* entropies;
};

// Vocabulary ranges per row tile: one CTA per SM over all tiles.
template <bool PAIR>
inline int lm_score_split(int sms, int64_t rows, int64_t V) {
  using S = LsShape<PAIR>;
  const int64_t n_mt = (rows + S::kBM - 1) / S::kBM, n_nt = (V + kLsBN - 1) / kLsBN;
  const int64_t fit = sms / S::kCtas / n_mt;
  const int64_t s = n_nt < fit ? n_nt : fit;
  return s < 1 ? 1 : (int)s;
}

// Most (half range, row) records of any call of up to max_rows rows: ranges x
// tile rows is at most sms x 128, two halves each; or one range.
inline size_t lm_score_slots(int sms, int64_t max_rows) {
  const size_t wide = 2 * (size_t)sms * (size_t)kLsRows, tall = 2 * (size_t)max_rows;
  return tall > wide ? tall : wide;
}

// -- the cta_group::2 forms ------------------------------------------------------
// This CTA's part of a stage, counted by the barrier at `bar` (a cluster
// address: the pair's first CTA).  Reads this GPU's own memory.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y,
                                              uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;"
      :
      : "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tc2_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
               :
               : "r"(smem_u32(dst)), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tc2_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" : : "r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tc2_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
// Arrives on the barrier at this offset in both CTAs once every MMA issued so
// far has completed.
__device__ __forceinline__ void tc2_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], m;\n\t}"
      :
      : "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tc2_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :
      : "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A bounded wait: one test (which may suspend the thread for a while, so only
// where the limit is longer), then the timed form.
__device__ __forceinline__ bool lm_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                        const int* abort) {
  return (limit_ns >= kSuspendHintNs && mbar_try_wait(bar, parity)) ||
         mbar_wait_timed(bar, parity, limit_ns, abort);
}

__device__ __forceinline__ float lm_temp(const LmScoreArgs& p, int row) {
  const float T = p.temps ? p.temps[row] : p.temp;
  return row_temp_ok(T) ? T : __int_as_float(0x7fc00000);
}

// Folds 128 columns (pairs) into a row's sums.  CLAMP: some of them were set
// to -inf.
template <bool CLAMP>
__device__ __forceinline__ void lm_fold(RowSums& s, const uint64_t (&z)[kLsHalf / 2], float c2) {
  float hi = -INFINITY;
#pragma unroll
  for (int i = 0; i < kLsHalf / 2; ++i) {
    float a, b;
    unpack2(z[i], a, b);
    hi = fmaxf(hi, fmaxf(a, b));
  }
  // moved only by 2^2: see kMuch on what that costs
  if ((hi - s.m) * c2 > 2.f) s = row_sums_join(s, RowSums{hi, 0.f, 0.f}, c2);
  const uint64_t nm = pack2(-s.m, -s.m), cc = pack2(c2, c2);
  uint64_t R[2] = {}, Q[2] = {};
#pragma unroll
  for (int i = 0; i < kLsHalf / 2; ++i) {
    uint64_t d = mul2(add2(z[i], nm), cc);
    float d0, d1;
    unpack2(d, d0, d1);
    if (CLAMP) {
      d0 = d0 < -kDeep ? -kDeep : d0;
      d1 = d1 < -kDeep ? -kDeep : d1;
      d = pack2(d0, d1);
    }
    const uint64_t e = pack2(ex2(d0), ex2(d1));
    R[i & 1] = add2(R[i & 1], e);
    Q[i & 1] = fma2(e, d, Q[i & 1]);
  }
  s.R += pair_sum(R);
  s.Q += pair_sum(Q);
}

template <bool PAIR>
__global__ void __cluster_dims__(PAIR ? 2 : 1, 1, 1) __launch_bounds__(kLsThreads, 1)
    lmscore_kernel(const __grid_constant__ CUtensorMap tm_h,
                   const __grid_constant__ CUtensorMap tm_w, const LmScoreArgs p) {
  using S = LsShape<PAIR>;
  extern __shared__ unsigned char ls_smem_raw[];
  // the same offset in both CTAs: the MMA's descriptors and the commits name it
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(ls_smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* empty = full + S::kStages;
  uint64_t* acc_full = empty + S::kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  uint32_t* copied = reinterpret_cast<uint32_t*>(abort_flag + 1);  // stages this CTA has asked for

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int pair = blockIdx.x / S::kCtas;
  const int n_nt = (p.V + kLsBN - 1) / kLsBN;
  const int mt = pair / p.n_split, ns = pair % p.n_split;
  const int nt_lo = (int)((long long)ns * n_nt / p.n_split);
  const int nt_hi = (int)((long long)(ns + 1) * n_nt / p.n_split);
  const int n_tiles = nt_hi - nt_lo;
  const int KB = (p.d + kLsBK - 1) / kLsBK;
  const int row0 = mt * S::kBM + rank * kLsRows;

  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], S::kCtas * kLsEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    if (PAIR)
      tc2_alloc(tmem_slot, kLsTmemCols);
    else
      tc_alloc(tmem_slot, kLsTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // A wait that gave up cuts the pair short.
  auto fail = [&]() {
    atomicOr(p.status, kScoreTimeout);
    *(volatile int*)abort_flag = 1;
    if (PAIR) st_cluster(map_rank(smem_u32(abort_flag), rank ^ 1), 1u);
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {  // the whole warp, one outcome
    return (bool)__all_sync(0xffffffffu, lm_wait(bar, parity, p.wait_ns, abort_flag));
  };
  // This CTA's copies of stage `kb` of tile `t`, into slot `s`.
  auto copy_stage = [&](int t, int kb, int s, uint64_t keep, uint64_t wpol) {
    const int y = (nt_lo + t) * kLsBN + rank * kLsHalf;
    unsigned char* dst = smem + s * S::kStage;
    if (PAIR) {
      // the first CTA's barrier counts both CTAs' bytes
      const uint32_t bar = map_rank(smem_u32(&full[s]), 0);
      if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * S::kStage);
      tma_load_pair(dst, &tm_h, kb * kLsBK, row0, bar, keep);
      tma_load_pair(dst + kLsABytes, &tm_w, kb * kLsBK, y, bar, wpol);
    } else {
      mbar_arrive_expect_tx(&full[s], S::kStage);
      tma_load_2d(dst, &tm_h, kb * kLsBK, row0, &full[s], keep);
      tma_load_2d(dst + kLsABytes, &tm_w, kb * kLsBK, y, &full[s], wpol);
      tma_load_2d(dst + kLsABytes + kLsBBytes, &tm_w, kb * kLsBK, y + kLsHalf, &full[s], wpol);
    }
  };

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      const uint64_t keep = evict_last_policy();  // h: every vocabulary tile reads it again
      // W: read once, or by every row tile at about the same time
      const uint64_t wpol = p.rows > S::kBM ? keep : evict_first_policy();
      int s = 0;
      uint32_t phase = 1u, n = 0;  // an empty stage's first wait passes at once
      bool ok = true;
      for (int t = 0; t < n_tiles && ok; ++t) {
        for (int kb = 0; kb < KB; ++kb, ++n) {
          if (!lm_wait(&empty[s], phase, p.wait_ns, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          copy_stage(t, kb, s, keep, wpol);
          if (++s == S::kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      *copied = n;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer
    // The warp runs the loop together and one elected lane issues: what the MMAs
    // name is then uniform for the compiler too (2048 rows of zeros, where power
    // does not bound: 1.39 ms against 1.65 with the loop in one lane; of random
    // values 2.08 against 2.24).
    if (rank == 0) {
      const bool lead = elect_one();
      constexpr uint32_t idesc = lm_idesc(S::kBM, kLsBN);
      const uint32_t base = smem_u32(smem);
      auto mma = [](uint32_t d, uint64_t a, uint64_t b, uint32_t i, uint32_t acc) {
        if (PAIR)
          tc2_mma(d, a, b, i, acc);
        else
          tc_mma(d, a, b, i, acc);
      };
      auto commit = [](uint64_t* bar) {
        if (PAIR)
          tc2_commit(bar);
        else
          tc_commit(bar);
      };
      int s = 0, used = 0;  // stage; accumulators filled
      uint32_t phase = 0u;
      bool ok = true;
      for (int t = 0; t < n_tiles && ok; ++t) {
        for (int kb = 0; kb < KB && ok; ++kb) {
          const int buf = used & 1, in_chunk = kb % kLsChunk;
          if (in_chunk == 0 && used >= 2) {
            if (!warp_wait(&acc_empty[buf], (uint32_t)(used / 2 - 1) & 1u)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          if (!warp_wait(&full[s], phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = base + (uint32_t)s * S::kStage, b = a + kLsABytes;
          // 16 elements of K on: 32 bytes, 2 in the descriptor
          const uint64_t da = sw128_desc(a), db = sw128_desc(b);
          if (lead) {
#pragma unroll
            for (int k = 0; k < kLsBK / 16; ++k)
              mma(tmem + (uint32_t)(buf * kLsBN), da + 2u * k, db + 2u * k, idesc,
                  (in_chunk | k) != 0 ? 1u : 0u);
            commit(&empty[s]);  // in both CTAs: the stage has been read
          }
          __syncwarp();
          if (++s == S::kStages) {
            s = 0;
            phase ^= 1u;
          }
          if (in_chunk == kLsChunk - 1 || kb == KB - 1) {
            if (lead) commit(&acc_full[buf]);
            __syncwarp();
            ++used;
          }
        }
      }
      if (!ok && lead) fail();
      if (lead) commit(drain);
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------- epilogue
    const int q = warp & 3;              // TMEM lanes 32 q .. 32 q + 31
    const int half = (warp - 2) >> 2;    // columns 128 half ..
    const int row = row0 + 32 * q + lane;
    const bool valid = row < p.rows;
    const int token = valid ? p.tokens[row] : -1;
    const float c2 = valid ? log2e_over(lm_temp(p, row)) : 1.f;
    const uint32_t free_bar[2] = {map_rank(smem_u32(&acc_empty[0]), 0),
                                  map_rank(smem_u32(&acc_empty[1]), 0)};
    const int chunks = (KB + kLsChunk - 1) / kLsChunk;
    RowSums s = row_sums_empty();
    int used = 0;
    bool ok = true;
    for (int t = 0; t < n_tiles && ok; ++t) {
      uint64_t z[kLsHalf / 2];
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++used) {
        const int buf = used & 1;
        // a warp-uniform outcome: the TMEM loads below need the whole warp
        if (!__all_sync(0xffffffffu, lm_wait(&acc_full[buf], (uint32_t)(used / 2) & 1u,
                                               p.wait_ns, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t taddr =
            tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * kLsBN + half * kLsHalf);
        if (c == 0) {
#pragma unroll
          for (int i = 0; i < kLsHalf / 2; ++i) z[i] = 0ull;
        }
#pragma unroll
        for (int g = 0; g < kLsHalf / 16; ++g) {
          float v[16];
          __syncwarp();  // tcgen05.ld is warp-wide: every lane, converged
          tc_ld16(taddr + (uint32_t)(g * 16), v);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) z[8 * g + i] = add2(z[8 * g + i], pack2(v[2 * i], v[2 * i + 1]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_remote(free_bar[buf]);
      }
      if (!ok) break;
      const int v0 = (nt_lo + t) * kLsBN + half * kLsHalf;
      const int n = p.V - v0;  // columns of this half inside the vocabulary
      const int at = token - v0;
      const bool here = at >= 0 && at < min(n, kLsHalf);
      if (n < kLsHalf || __any_sync(0xffffffffu, here)) {
#pragma unroll
        for (int i = 0; i < kLsHalf / 2; ++i) {
          float a, b;
          unpack2(z[i], a, b);
          if (here && i == at >> 1) {
            p.za[row] = at & 1 ? b : a;
            if (at & 1)
              b = -INFINITY;
            else
              a = -INFINITY;
          }
          z[i] = pack2(2 * i < n ? a : -INFINITY, 2 * i + 1 < n ? b : -INFINITY);
        }
        lm_fold<true>(s, z, c2);
      } else {
        lm_fold<false>(s, z, c2);
      }
    }
    if (!ok) {
      if (lane == 0) fail();
      s.R = __int_as_float(0x7fc00000);  // a cut-short pass leaves NaN, not a part of the sums
    }
    if (valid) p.sums[(size_t)(2 * ns + half) * (size_t)p.rows + (size_t)row] = s;
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // Every MMA issued has completed before TMEM is released, and the commits'
  // arrivals, which go to both CTAs, have come before either leaves.
  if (warp == 1) mbar_wait(drain, 0u, kDrainLimitNs);
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  // After a pass cut short copies may still be on their way into either CTA's
  // memory.  Nobody copies or reads stages any more, so each CTA asks for those
  // that only the other one has asked for (at most a ring of them); then every
  // phase of the barriers has both CTAs' bytes to come, and is waited for.
  if (*(volatile int*)abort_flag) {
    if (warp == 0 && lane == 0) {
      const uint32_t mine = *copied;
      const uint32_t other = PAIR ? ld_cluster(map_rank(smem_u32(copied), rank ^ 1)) : mine;
      const uint32_t n = max(mine, other);
      const uint64_t once = evict_first_policy();
      for (uint32_t i = mine; i < n; ++i)
        copy_stage(i / KB, i % KB, i % S::kStages, once, once);
      if (rank == 0)
        for (uint32_t i = n > S::kStages ? n - S::kStages : 0; i < n; ++i)
          mbar_wait(&full[i % S::kStages], (i / S::kStages) & 1u, kDrainLimitNs);
    }
    __syncwarp();
    __syncthreads();
    cluster_sync_all();
  }
  if (warp == 0) {
    __syncwarp();
    if (PAIR) {
      tc2_dealloc(tmem, kLsTmemCols);
      tc2_relinquish();
    } else {
      tc_dealloc(tmem, kLsTmemCols);
      tc_relinquish();
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows
//
// A CTA owns a contiguous range of 128-wide vocabulary tiles and every row:
// W's 128 rows are the MMA's M, the hidden states its N = 32 NH.  A thread of
// the epilogue holds one vocabulary id and 16 rows, and keeps a running
// (reference, sum e, sum e d) for each of them over all its tiles; lanes and
// warps meet once, at the end.
// ---------------------------------------------------------------------------
constexpr int kLfRows = 64;
// Stages of one accumulator: 256 elements of K, for half the truncation of 512
// (24 rows of 262144 x 2560: 212 us; 128 elements 219).
constexpr int kLfChunk = 4;
constexpr int kLfPer = 16;  // rows per epilogue thread
// Within +-kDeep; NaN stays NaN.
__device__ __forceinline__ float clamp_deep(float d) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(d) : "f"(-kDeep));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(d) : "f"(kDeep));
  return d;
}

template <int NH>
struct FewShape {
  static constexpr int kN = 32 * NH;
  static constexpr int kStages = NH == 1 ? 10 : 8;
  static constexpr uint32_t kWBytes = 128 * kLsBK * 2, kHBytes = kN * kLsBK * 2;
  static constexpr uint32_t kStage = kWBytes + kHBytes;
  static constexpr int kGroups = kN / kLfPer;  // of four warps each
  static constexpr int kThreads = (2 + 4 * kGroups) * 32;
  static constexpr uint32_t kCols = 2 * kN < 32 ? 32 : 2 * kN;
  // stages, each row's log2(e) / T and token, the warps' sums, barriers
  static constexpr uint32_t kC2 = kStages * kStage, kToken = kC2 + kN * 4,
                            kJoin = kToken + kN * 4,
                            kBars = kJoin + 4 * kN * 16, kSmem = kBars + 8 * (2 * kStages + 5) +
                                                                16 + 1024;
};

template <int NH>
__global__ void __launch_bounds__(FewShape<NH>::kThreads, 1)
    lmfew_kernel(const __grid_constant__ CUtensorMap tm_h, const __grid_constant__ CUtensorMap tm_w,
                 const LmScoreArgs p) {
  using S = FewShape<NH>;
  extern __shared__ unsigned char ls_smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(ls_smem_raw) + 1023) & ~(uintptr_t)1023);
  float* row_c2 = reinterpret_cast<float*>(smem + S::kC2);
  int* row_token = reinterpret_cast<int*>(smem + S::kToken);
  float4* join = reinterpret_cast<float4*>(smem + S::kJoin);  // [4][kN]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* empty = full + S::kStages;
  uint64_t* acc_full = empty + S::kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;       // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_nt = (p.V + 127) / 128;
  const int nt_lo = (int)((long long)blockIdx.x * n_nt / p.n_split);
  const int nt_hi = (int)((long long)(blockIdx.x + 1) * n_nt / p.n_split);
  const int n_tiles = nt_hi - nt_lo;
  const int KB = (p.d + kLsBK - 1) / kLsBK;

  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4 * S::kGroups);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  for (int r = tid; r < S::kN; r += S::kThreads) {
    row_token[r] = r < p.rows ? p.tokens[r] : -1;
    row_c2[r] = r < p.rows ? log2e_over(lm_temp(p, r)) : 1.f;
  }
  if (warp == 0) tc_alloc(tmem_slot, S::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&]() {
    atomicOr(p.status, kScoreTimeout);
    *(volatile int*)abort_flag = 1;
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {  // the whole warp, one outcome
    return (bool)__all_sync(0xffffffffu, lm_wait(bar, parity, p.wait_ns, abort_flag));
  };

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      const uint64_t keep = evict_last_policy(), once = evict_first_policy();
      int s = 0, issued = 0;
      uint32_t phase = 1u;
      bool ok = true;
      for (int t = 0; t < n_tiles && ok; ++t) {
        for (int kb = 0; kb < KB; ++kb, ++issued) {
          if (!lm_wait(&empty[s], phase, p.wait_ns, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], S::kStage);
          unsigned char* dst = smem + (uint32_t)s * S::kStage;
          tma_load_2d(dst, &tm_w, kb * kLsBK, (nt_lo + t) * 128, &full[s], once);
          tma_load_2d(dst + S::kWBytes, &tm_h, kb * kLsBK, 0, &full[s], keep);
          if (++s == S::kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      // every copy issued has landed before the CTA may leave
      for (int i = max(0, issued - S::kStages); i < issued; ++i)
        mbar_wait(&full[i % S::kStages], (uint32_t)(i / S::kStages) & 1u, kDrainLimitNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer
    {
      const bool lead = elect_one();
      constexpr uint32_t idesc = lm_idesc(128, S::kN);
      const uint32_t base = smem_u32(smem);
      int s = 0, used = 0;
      uint32_t phase = 0u;
      bool ok = true;
      for (int t = 0; t < n_tiles && ok; ++t) {
        for (int kb = 0; kb < KB && ok; ++kb) {
          const int buf = used & 1, in_chunk = kb % kLfChunk;
          if (in_chunk == 0 && used >= 2) {
            if (!warp_wait(&acc_empty[buf], (uint32_t)(used / 2 - 1) & 1u)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          if (!warp_wait(&full[s], phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = base + (uint32_t)s * S::kStage, b = a + S::kWBytes;
          const uint64_t da = sw128_desc(a), db = sw128_desc(b);
          if (lead) {
#pragma unroll
            for (int k = 0; k < kLsBK / 16; ++k)
              tc_mma(tmem + (uint32_t)(buf * S::kN), da + 2u * k, db + 2u * k, idesc,
                     (in_chunk | k) != 0 ? 1u : 0u);
            tc_commit(&empty[s]);
          }
          __syncwarp();
          if (++s == S::kStages) {
            s = 0;
            phase ^= 1u;
          }
          if (in_chunk == kLfChunk - 1 || kb == KB - 1) {
            if (lead) tc_commit(&acc_full[buf]);
            __syncwarp();
            ++used;
          }
        }
      }
      if (!ok && lead) fail();
      if (lead) tc_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0u, kDrainLimitNs);
    }
  } else {
    // --------------------------------------------------------- epilogue
    const int q = warp & 3;            // TMEM lanes 32 q .. 32 q + 31
    const int r0 = ((warp - 2) >> 2) * kLfPer;  // rows r0 ..
    const int chunks = (KB + kLfChunk - 1) / kLfChunk;
    const int n_rows = min(kLfPer, p.rows - r0);
    float m[kLfPer], R[kLfPer], Q[kLfPer];
#pragma unroll
    for (int r = 0; r < kLfPer; ++r) {
      m[r] = -FLT_MAX;
      R[r] = Q[r] = 0.f;
    }
    int used = 0;
    bool ok = true;
    for (int t = 0; t < n_tiles && ok; ++t) {
      float z[kLfPer];
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++used) {
        const int buf = used & 1;
        if (!__all_sync(0xffffffffu, lm_wait(&acc_full[buf], (uint32_t)(used / 2) & 1u,
                                               p.wait_ns, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        float v[kLfPer];
        __syncwarp();  // tcgen05.ld is warp-wide: every lane, converged
        tc_ld16(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * S::kN + r0), v);
        tc_wait_ld();
#pragma unroll
        for (int r = 0; r < kLfPer; ++r) z[r] = c == 0 ? v[r] : z[r] + v[r];
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
      }
      if (!ok) break;
      const int id0 = (nt_lo + t) * 128 + 32 * q, id = id0 + lane;
      const float4* c4 = reinterpret_cast<const float4*>(row_c2 + r0);
      // rare: a row's token among this warp's ids, ids past the vocabulary
      const int tok = row_token[r0 + (lane & (kLfPer - 1))] - id0;
      if (id0 + 32 > p.V || __any_sync(0xffffffffu, tok >= 0 && tok < 32)) {
#pragma unroll
        for (int r = 0; r < kLfPer; ++r) {
          if (row_token[r0 + r] == id && id < p.V) {
            p.za[r0 + r] = z[r];
            z[r] = -INFINITY;
          }
          if (id >= p.V) z[r] = -INFINITY;
        }
      }
      // every id is its own reference's next candidate, so new maxima are
      // common: without a branch, one of the two factors being 1
#pragma unroll
      for (int r = 0; r < kLfPer; r += 4) {
        const float4 c = c4[r / 4];
        const float cr[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = z[r + k];
          const float d = clamp_deep((x - m[r + k]) * cr[k]);
          const bool up = d > 0.f;
          const float f = ex2(-fabsf(d));
          const float Qup = f * fmaf(-d, R[r + k], Q[r + k]);
          Q[r + k] = up ? Qup : fmaf(f, d, Q[r + k]);
          R[r + k] = up ? fmaf(R[r + k], f, 1.f) : R[r + k] + f;
          m[r + k] = up ? x : m[r + k];
        }
      }
    }
    if (!ok && lane == 0) fail();
#pragma unroll
    for (int r = 0; r < kLfPer; ++r) {
      if (r >= n_rows) break;
      const RowSums w =
          warp_join(RowSums{m[r], R[r], Q[r]}, row_c2[r0 + r]);
      if (lane == 0) join[q * S::kN + r0 + r] = make_float4(w.m, w.R, w.Q, 0.f);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  for (int r = tid; r < p.rows; r += S::kThreads) {
    const float c2 = row_c2[r];
    RowSums s = row_sums_empty();
    for (int q = 0; q < 4; ++q) {
      const float4 v = join[q * S::kN + r];
      s = row_sums_join(s, RowSums{v.x, v.y, v.z}, c2);
    }
    // a cut-short pass leaves NaN, not a part of the sums
    if (*(volatile int*)abort_flag) s.R = __int_as_float(0x7fc00000);
    p.sums[(size_t)blockIdx.x * (size_t)p.rows + (size_t)r] = s;
  }
  if (warp == 0) {
    __syncwarp();
    tc_dealloc(tmem, S::kCols);
    tc_relinquish();
  }
}

// A warp per row: the ranges' sums, then the row's results.  Launched as a
// programmatic dependent: it waits for the product's kernel to complete.
__global__ void __launch_bounds__(128) lmscore_finish_kernel(const LmScoreArgs p) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= p.rows) return;
  const int token = p.tokens[row];
  const Scale sc = row_scale(lm_temp(p, row));
  const float c2 = sc.c2;
  griddep_wait();
  if (token < 0) {
    if (lane == 0) {
      p.logprobs[row] = 0.f;
      if (p.entropies) p.entropies[row] = 0.f;
    }
    return;
  }
  const bool bad = token >= p.V;
  const float za = bad ? __int_as_float(0x7fc00000) : __ldcg(p.za + row);
  RowSums s = row_sums_empty();
  for (int k0 = lane; k0 < p.n_rec; k0 += 5 * 32) {
    RowSums v[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      const int k = k0 + 32 * j;
      v[j] = row_sums_empty();
      if (k < p.n_rec) {
        const float* r = reinterpret_cast<const float*>(p.sums + (size_t)k * (size_t)p.rows + row);
        v[j] = RowSums{__ldcg(r), __ldcg(r + 1), __ldcg(r + 2)};
      }
    }
#pragma unroll
    for (int j = 0; j < 5; ++j) s = row_sums_join(s, v[j], c2);
  }
  s = warp_join(s, c2);
  const RowResult r = row_result<true>(s, za, sc);
  if (lane != 0) return;
  p.logprobs[row] = r.lp;
  if (p.entropies) p.entropies[row] = r.H;
  const uint32_t bits = (bad ? kScoreBadToken : 0u) | (r.finite ? 0u : kScoreNonFinite);
  if (bits) atomicOr(p.status, bits);
}

}  // namespace ebk
