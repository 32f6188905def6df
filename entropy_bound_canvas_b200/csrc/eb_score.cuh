// eb_score.cuh -- scoring of sampled tokens and the losses that learn from
// them: log p[a] and the entropy of softmax(z / T) for every row of logits,
// the clipped policy loss, the preference loss, and their gradients for the
// logits.
//
// With M the row's maximum, d_v = (z_v - M) log2(e) / T, e_v = 2^d_v and the
// sums over every v but the row's token a
//     R = sum e_v,   Q = sum e_v d_v,
// the row's results are
//     S      = R + e_a
//     log p_a = -ln(1 + R / e_a)                  (no cancellation near p_a = 1)
//     H      = ln S - ln 2 (Q + e_a d_a) / S
//     1 - p_a = R / S
// and the gradient of g log p_a + h H for the logits is
//     dz_v = (1/T) [ g (1[v = a] - p_v) - h p_v (ln p_v + H) ],
//     p_v  = 2^(d_v - log2 S),
// the token's own element taken from 1 - p_a = R / S.  Leaving the token out
// of the sums keeps the log-probability and gradient of a confident row
// (p_a within 2^-24 of 1), where S itself would round them away.
// Everything between the loads and the stores is fp32, the losses' sums over
// rows and sequences are fp64; a gradient is rounded once, to the logits'
// type.
#pragma once

#include <float.h>

#include "eb_device.cuh"

namespace ebk {

enum { kScoreF32 = 0, kScoreBF16 = 1 };
enum { kModeScore = 0, kModeGrad = 1, kModePolicy = 2 };

constexpr int kPolicyTerms = 5;
constexpr uint32_t kScoreBadToken = 1u, kScoreNonFinite = 2u, kScoreTimeout = 4u,
                   kScoreBadOffsets = 8u;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
// Terms below 2^-kDeep of the maximum are zero in fp32 with flush to zero;
// holding their exponent there keeps e d = 0 where d would be -inf (a logit of
// -inf, or one whose distance to the maximum overflows).
constexpr float kDeep = 200.0f;
// NaN stays NaN.
__device__ __forceinline__ float hold_deep(float d) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(d), "f"(-kDeep));
  return r;
}
// Below fp32's smallest normal number 1/T and log2(e)/T are past its largest.
__device__ __forceinline__ bool row_temp_ok(float T) { return T >= FLT_MIN && T < INFINITY; }
// log2(e) / T, rounded once or nearly so, and what that left.
struct Scale {
  float c2, low, T;
};
__device__ __forceinline__ Scale row_scale(float T) {
  const float r = __frcp_rn(T), q = kLog2e * r;
  // log2(e) is kLog2e in fp32 plus 1.92596e-8
  constexpr float kLog2eLow = 1.925963033500e-8f;
  const float c2 = fmaf(fmaf(-q, T, kLog2e) + kLog2eLow, r, q);
  return Scale{c2, (fmaf(-c2, T, kLog2e) + kLog2eLow) * r, T};
}
__device__ __forceinline__ float log2e_over(float T) { return row_scale(T).c2; }

struct ScoreArgs {
  const void* logits;  // [rows][ld]
  void* d_logits;      // [rows][ldd], the logits' type
  int64_t ld, ldd;
  int rows, V;
  const int32_t* tokens;
  const float* temps;  // per row, or null: temp for all
  float temp;
  const int32_t* offsets;  // only rows in [offsets[0], offsets[n_off]) count, or null
  int n_off;
  float* logprobs;         // [rows] or null
  float* entropies;        // [rows] or null
  float4* stats;           // [rows] or null: M, log2 S and its low part, 1 - p_a
  const float* g_lp;       // kModeGrad: upstream gradients
  const float* g_h;        // kModeGrad: or null
  const float* old_lp;     // kModePolicy
  const float* ref_lp;     // or null
  const float* adv;
  const float* weights;    // or null
  float clip_lo, clip_hi;  // 1 - clip_low, 1 + clip_high
  float kl_coef, ent_coef;
  double scale;
  double* part;            // kModePolicy: [grid][kPolicyTerms]
  float* terms;            // kModePolicy: [kPolicyTerms]
  uint32_t* counter;       // arrivals of the grid, zero between launches
  uint32_t* status;
  uint64_t wait_ns;
};

template <int DT>
struct ScoreType;
template <>
struct ScoreType<kScoreF32> {
  static constexpr int kBytes = 4, kPer16 = 4;
};
template <>
struct ScoreType<kScoreBF16> {
  static constexpr int kBytes = 2, kPer16 = 8;
};

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if (DT == kScoreF32) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// Round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int DT>
__device__ __forceinline__ void store_grad(void* p, int64_t i, float v) {
  if (DT == kScoreF32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16(v, 0.f);
}

// ---------------------------------------------------------------------------
// A row's running sums, and what follows from them
// ---------------------------------------------------------------------------
struct RowSums {
  float m, R, Q;  // reference maximum; sums of e and e d relative to it
};

__device__ __forceinline__ RowSums row_sums_empty() { return RowSums{-FLT_MAX, 0.f, 0.f}; }

// The sums of two disjoint parts of a row against the larger maximum.
__device__ __forceinline__ RowSums row_sums_join(RowSums a, RowSums b, float c2) {
  const float m = fmaxf(a.m, b.m);
  const float da = fmaxf((a.m - m) * c2, -kDeep), db = fmaxf((b.m - m) * c2, -kDeep);
  const float fa = ex2(da), fb = ex2(db);
  // sum e d of a part, moved to the new maximum: f (Q + d R)
  return RowSums{m, fmaf(a.R, fa, b.R * fb),
                 fmaf(fa, fmaf(da, a.R, a.Q), fb * fmaf(db, b.R, b.Q))};
}

struct RowResult {
  float M;             // maximum over every logit (or near it, see kMuch)
  float l2S, l2S_low;  // log2 S, and what its rounding left
  float lp, lp_low;    // log p_a (nats), and what its rounding left
  float H;             // entropy (nats)
  float rest;          // 1 - p_a
  float pa;            // p_a
  bool finite;
};

// Beyond 2^24 nats the part of log p_a below fp32 is more than its roundings
// leave of it, so it is dropped.
constexpr float kNoLow = 16777216.f;

// s: the sums without the token; za: the token's logit (NaN: a bad token).
// log2 S is kept as a + b, a an integer or d_a and b small, so that the
// differences log p_a and H round only their own size.  ENT: Q is there; it
// also takes out the rounding of c2, by d log2 S / d c2 = (Q + e_a d_a) / (S c2).
template <bool ENT>
__device__ __forceinline__ RowResult row_result(RowSums s, float za, Scale sc) {
  const float c2 = sc.c2;
  RowResult r;
  const float M = fmaxf(s.m, za);
  const float ds = fmaxf((s.m - M) * c2, -kDeep);
  const float fs = ex2(ds);
  const float R = s.R * fs;
  const float Q = fs * fmaf(ds, s.R, s.Q);
  const float gap = za - M, da = gap * c2, da_low = fmaf(gap, c2, -da);
  const float ea = ex2(da);
  const float S = R + ea;
  r.finite = S > 0.f && S < INFINITY;
  // e_a = 0: no entropy term, whatever d_a
  const float W = ea == 0.f ? Q : fmaf(ea, da, Q);
  const float iS = __frcp_rn(S);
  const float w = W * iS;
  float a, b;
  if (ea >= R) {
    const float t = log1pf(__fdividef(R, ea));
    a = da;
    b = t * kLog2e;
    r.lp = -t;
    r.lp_low = 0.f;
  } else {
    // S = 2^k f, f in [1/sqrt 2, sqrt 2)
    const int k = (int)((__float_as_uint(S) + 0x004afb0du) >> 23) - 127;
    a = (float)k;
    b = log2f(S * __uint_as_float((uint32_t)(127 - k) << 23));
    // ln 2 (d_a - a - b), the low parts kept (two-sums and a two-product)
    const float s1 = da - a, u = s1 - da, e1 = (da - (s1 - u)) - (a + u);
    const float s2 = s1 - b, v = s2 - s1, e2 = (s1 - (s2 - v)) - (b + v);
    float low = e1 + e2 + da_low;
    if (ENT) low += sc.low * (gap - w / c2);
    constexpr float kLn2Low = -1.904654323148236e-9f;  // ln 2 - kLn2
    r.lp = kLn2 * s2;
    r.lp_low = fmaf(kLn2, s2, -r.lp) + fmaf(kLn2, low, kLn2Low * s2);
    const float sum = r.lp + r.lp_low;
    r.lp_low = r.lp_low - (sum - r.lp);
    r.lp = sum;
    if (!(da > -INFINITY) || !(r.lp > -kNoLow)) {
      r.lp_low = 0.f;
      // d_a may be past fp32 where log p_a is not, and so may M - z_a
      if (!(da > -INFINITY))
        r.lp = !(za > -INFINITY) ? za : gap > -INFINITY ? gap / sc.T : za / sc.T - M / sc.T;
    }
  }
  r.M = M;
  r.l2S = a + b;
  r.l2S_low = (a - r.l2S) + b;
  const float w_low = fmaf(-w, S, W) * iS;
  r.H = kLn2 * (((a - w) - w_low) + b);
  r.rest = R / S;
  r.pa = ea * iS;
  if (!r.finite) r.lp = r.lp_low = r.H = r.l2S = r.rest = r.pa = __int_as_float(0x7fc00000);
  return r;
}

struct RowCoef {
  float g, h;  // upstream gradients of log p_a and H
};

// What a row's gradient is made from.
struct RowGrad {
  float M, l2S;  // p = 2^((z - M) c2 - l2S)
  float a0, a1;  // gradient p (a0 + a1 log2 p)
  float own;     // the token's element
};

template <bool ENT>
__device__ __forceinline__ RowGrad row_grad(const RowResult& r, RowCoef c, float T) {
  const float iT = 1.f / T;
  // p = 2^(d - l2S) 2^-l2S_low: the second factor goes into the coefficients
  const float f = fmaf(-kLn2, r.l2S_low, 1.f) * -iT;
  RowGrad o;
  o.M = r.M;
  o.l2S = r.l2S;
  o.a0 = f * (ENT ? fmaf(c.h, r.H, c.g) : c.g);
  o.a1 = f * c.h * kLn2;
  // p_a = 0: log p_a may be -inf, its entropy term is 0
  const float ha = !ENT ? 0.f : r.pa > 0.f ? c.h * r.pa * (r.lp + r.H) : r.pa;
  o.own = iT * (c.g * r.rest - ha);
  return o;
}

// The rows that count: those of the sequences, where there are any.
struct RowRange {
  int lo, hi;
  __device__ __forceinline__ bool live(int row, int token, float weight) const {
    return token >= 0 && weight != 0.f && row >= lo && row < hi;
  }
};
__device__ __forceinline__ RowRange row_range(const ScoreArgs& p) {
  RowRange r{0, p.rows};
  if (p.offsets) r = RowRange{p.offsets[0], p.offsets[p.n_off]};
  return r;
}

// The policy loss of a row.
//   L = w [ max(-A r, -A clip(r)) + k KL - c H ],  r = exp(log p_a - old),
//   KL = exp(ref - log p_a) - 1 - (ref - log p_a)
// Formed in fp32 near the policy that drew the token.  Where the exponents or
// their products leave fp32's range (kFarExp, kFarSize), the row is `far`, and
// policy_far forms it in 64 bits: w may bring an A r past fp32 back into it.
// A factor of 0 takes its term out, whatever the term: an advantage of 0 beside
// an infinite ratio, a k of 0 beside an infinite KL.
constexpr float kFarExp = 80.0f, kFarSize = 1e30f;

struct PolicyRow {
  float pg;
  float gap, back;  // ref - log p_a, e^gap - 1
  bool cut;  // the clipped side is the larger: no gradient through the ratio
  bool far;  // fp32 does not hold it: policy_far does
};
struct PolicyFar {
  double pg, kl, dkl;
  bool cut;
};

__device__ __forceinline__ PolicyRow policy_row(const ScoreArgs& p, const RowResult& r,
                                                float old_lp, float adv, float ref_lp,
                                                float weight) {
  const float x = (r.lp - old_lp) + r.lp_low;
  const float ratio = expf(x);
  const float free = -adv * ratio;
  const float held = -adv * fminf(fmaxf(ratio, p.clip_lo), p.clip_hi);
  PolicyRow o;
  o.cut = held > free;
  o.pg = o.cut ? held : free;
  o.gap = o.back = 0.f;
  float reach = fabsf(x);
  if (p.ref_lp) {
    o.gap = (ref_lp - r.lp) - r.lp_low;
    o.back = expm1f(o.gap);
    reach += fabsf(o.gap);
  }
  // NaN is far, and so is a w that scale or weight brings past fp32's middle
  const float w = fabsf(weight * (float)p.scale);
  const bool near = reach < kFarExp && fabsf(o.pg) < kFarSize &&
                    w < kFarSize && w > 1.f / kFarSize;
  o.far = !near;
  return o;
}

// e^x - 1 - x, given e^x - 1.  The difference's relative error grows as
// 2^-23 / |x| near 0, so there the series x^2 (1/2! + x/3! + ... + x^7/9!): what
// it leaves out is below 2^-28 of the sum at |x| = 1/2, where the difference
// loses two bits.
__device__ __forceinline__ float exp_excess(float x, float back) {
  if (!(fabsf(x) < 0.5f)) return back - x;
  float s = 1.f / 362880.f;
  s = fmaf(s, x, 1.f / 40320.f);
  s = fmaf(s, x, 1.f / 5040.f);
  s = fmaf(s, x, 1.f / 720.f);
  s = fmaf(s, x, 1.f / 120.f);
  s = fmaf(s, x, 1.f / 24.f);
  s = fmaf(s, x, 1.f / 6.f);
  s = fmaf(s, x, 0.5f);
  return x * x * s;
}

static __device__ __noinline__ PolicyFar policy_far(float lp, float lp_low, float old_lp,
                                                    float adv, float ref_lp, bool has_ref,
                                                    float clip_lo, float clip_hi) {
  PolicyFar o;
  const double x = ((double)lp - (double)old_lp) + (double)lp_low;
  const double ratio = exp(x), A = (double)adv;
  // the comparisons keep a NaN ratio NaN
  const double held_ratio =
      ratio < (double)clip_lo ? (double)clip_lo : ratio > (double)clip_hi ? (double)clip_hi : ratio;
  double free = -A * ratio, held = -A * held_ratio;
  if (A == 0.0 && x == x) free = held = 0.0;
  o.cut = held > free;
  o.pg = o.cut ? held : free;
  o.kl = o.dkl = 0.0;
  if (has_ref) {
    const double gap = ((double)ref_lp - (double)lp) - (double)lp_low;
    const double back = expm1(gap);
    o.kl = back < (double)INFINITY ? back - gap : back;
    o.dkl = -back;
  }
  return o;
}

// The factors of log p_a and H in the gradient.
__device__ __forceinline__ RowCoef policy_coef(const ScoreArgs& p, const RowResult& r,
                                               const PolicyRow& o, float old_lp, float adv,
                                               float ref_lp, float weight) {
  RowCoef c;
  if (!o.far) {
    const float w = weight * (float)p.scale;
    c.g = w * fmaf(p.kl_coef, -o.back, o.cut ? 0.f : o.pg);
    c.h = -w * p.ent_coef;
  } else {
    const PolicyFar f = policy_far(r.lp, r.lp_low, old_lp, adv, ref_lp, p.ref_lp != nullptr,
                                   p.clip_lo, p.clip_hi);
    const double w = (double)weight * p.scale;
    double g = f.cut ? 0.0 : f.pg;
    if (p.kl_coef != 0.f) g += (double)p.kl_coef * f.dkl;
    c.g = (float)(w * g);
    c.h = (float)(-w * (double)p.ent_coef);
  }
  return c;
}

__device__ __forceinline__ void policy_add(const ScoreArgs& p, const RowResult& r,
                                           const PolicyRow& o, float old_lp, float adv,
                                           float ref_lp, float weight,
                                           double (&t)[kPolicyTerms]) {
  const double w = (double)weight * p.scale;
  double pg = o.pg, kl = exp_excess(o.gap, o.back);
  bool cut = o.cut;
  if (o.far) {
    const PolicyFar f = policy_far(r.lp, r.lp_low, old_lp, adv, ref_lp, p.ref_lp != nullptr,
                                   p.clip_lo, p.clip_hi);
    pg = f.pg;
    kl = f.kl;
    cut = f.cut;
  }
  const double k = p.kl_coef == 0.f ? 0.0 : (double)p.kl_coef * kl;
  t[0] += w * (pg + k - (double)p.ent_coef * r.H);
  t[1] += w * pg;
  t[2] += w * kl;
  t[3] += w * r.H;
  t[4] += cut ? w : 0.0;
}

// The loss's terms.  A CTA's part is the sum of its leaders' t (one thread
// each, numbered from 0); the last of n CTAs to arrive sums the parts, in an
// order of its own that does not depend on who arrived when: the same bits at
// every launch of one grid.  Called by whole blocks, this one being `index`.
template <int THREADS, int LEADERS>
__device__ __forceinline__ void policy_total(const ScoreArgs& p, int leader,
                                             const double (&t)[kPolicyTerms], int index, int n) {
  constexpr int kWarps = THREADS / 32;
  __shared__ double sums[kWarps][kPolicyTerms];
  __shared__ int last;
  if (leader >= 0)
    for (int k = 0; k < kPolicyTerms; ++k) sums[leader][k] = t[k];
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 0; k < kPolicyTerms; ++k) {
      double v = 0.0;
      for (int w = 0; w < LEADERS; ++w) v += sums[w][k];
      if (n > 1)
        p.part[(size_t)index * kPolicyTerms + k] = v;
      else
        p.terms[k] = (float)v;
    }
    last = 0;
    if (n > 1) {
      last = atom_add_acq_rel_gpu(reinterpret_cast<int*>(p.counter), 1) == n - 1;
      if (last) *p.counter = 0u;
    }
  }
  __syncthreads();
  if (!last) return;
  double s[kPolicyTerms] = {};
  for (int i = threadIdx.x; i < n; i += THREADS)
#pragma unroll
    for (int k = 0; k < kPolicyTerms; ++k) s[k] += __ldcg(p.part + (size_t)i * kPolicyTerms + k);
#pragma unroll
  for (int k = 0; k < kPolicyTerms; ++k)
    for (int m = 16; m > 0; m >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], m);
  if ((threadIdx.x & 31) == 0)
    for (int k = 0; k < kPolicyTerms; ++k) sums[threadIdx.x >> 5][k] = s[k];
  __syncthreads();
  if (threadIdx.x < kPolicyTerms) {
    double v = 0.0;
    for (int w = 0; w < kWarps; ++w) v += sums[w][threadIdx.x];
    p.terms[threadIdx.x] = (float)v;
  }
}

// ---------------------------------------------------------------------------
// Rows on thread-block clusters
//
// A cluster of C CTAs takes one row at a time; CTA c holds the c-th share of
// it.  Three roles:
//   producer   (a warp) copies the share into a ring of stages (bulk copies);
//   consumers  (NW warps) fold each stage into a running (reference, sum e,
//              sum e d); at the row's end every warp sends its sums into the
//              finishing CTAs' shared memory (st.async, counted by an
//              mbarrier);
//   finisher   (a warp) joins the C NW sums, in an order of its own, and
//              computes the row's results and its gradient's factors.
// Without a gradient only the first CTA finishes, and the consumers go on to
// the next row at once.  With one every CTA does (the same arithmetic, the
// same bits), and the consumers turn what the ring holds into the gradient:
//   ahead      where two shares fit the ring, they fold the next row first, so
//              that the exchange and the finisher's work run under that;
//   otherwise  they go through the share a second time in the opposite order.
//              Its last stages are still in the ring; the others are copied
//              again, the most recent first, so that most come from L2 (the
//              first copy asks L2 to keep them).
//
// Cluster c takes rows c, c + n, c + 2 n, ..., or (listed) the live rows number
// c, c + n, ... and as even a part of the ignored ones, whose gradient is only
// zeros to write: then every CTA counts the rows' liveness once, at the start.
//
// Rows start at any element.  A share is a range of 16-byte granules of the
// row's 16-byte-aligned image; the granules that the row fills only partly
// (at its two ends) are gathered element by element, with -inf in the places
// that are not the row's, and stored element by element.
//
// What bounds it: HBM, and close behind it the exponentials and the issue
// slots.  2048 rows of 262144 bf16: 178 us without a gradient (6.0 TB/s, 0.92
// of the measured copy rate; the exponential unit 60 % and the issue slots
// 57 % busy), 412 us with the policy loss's (5.2 TB/s counting one read and
// one write, 0.79; an earlier form's copies and stores alone took 359).  Kept
// up for seconds, the chip's power limit holds the SM clock at 1.76 GHz: 203
// and 445 us.
// One canvas of 256 rows, 31 and 66 us, has two waves of clusters of which
// the second is three quarters full, and the pipeline to fill and drain.
// Measured against: 8 KB and 32 KB stages, 6, 10 or 12 consumer warps, three
// CTAs per SM, clusters started in turn (all slower or the same); part of the
// exponentials as polynomials on the FMA pipe (slower: issue slots).
// ---------------------------------------------------------------------------
constexpr int kRingWarps = 8;  // consumers
constexpr int kRingThreads = (kRingWarps + 2) * 32;
constexpr int kRingCtas = 2;   // per SM
constexpr int kStageIter = 4;  // granules of a stage per consumer thread
constexpr int kStageGran = kRingWarps * 32 * kStageIter;
constexpr int kStageBytes = kStageGran * 16;
constexpr int kRingStages = 6;  // two CTAs of 96 KB rings share an SM
constexpr int kMaxCluster = 16;
constexpr int kListRows = 1024;  // of a cluster

// A thread's reference is the maximum of what it folds first.  It moves only
// when a fold's sum relative to it exceeds kMuch (or is not finite), so that
// the common fold looks for no maximum.  The sums are as exact relative to a
// nearby value; a logit that dominates its row is over kMuch times any other's
// term, so it becomes the reference, and its own term is exactly 1.
constexpr float kMuch = 64.0f;

struct RingArgs {
  int mode;
  int log2C;     // CTAs per cluster: a power of two
  int ahead;     // two shares fit: the next row is folded before this one's gradient
  int listed;    // the rows are shared out by lists, see below
};

// The ring's slots in their order of use, the same for the producer and the
// consumers, each slot with the parity of its next wait.
struct RingWalk {
  int slot, dir;
  uint32_t parity;  // by slot
  __device__ __forceinline__ uint32_t phase() const { return parity >> slot & 1u; }
  __device__ __forceinline__ void used() { parity ^= 1u << slot; }
  __device__ __forceinline__ void step(int n = 1) {
    slot += dir * n;
    if (slot >= kRingStages) slot -= kRingStages;
    if (slot < 0) slot += kRingStages;
  }
  // The next slot is the one used last.
  __device__ __forceinline__ void turn() {
    dir = -dir;
    step();
  }
};
constexpr int kSlots = 4;  // rows between a slot's uses, see the kernel

struct RingLayout {
  uint32_t part, grad, bars, flag, count, sent, list, total;
};
__host__ __device__ constexpr RingLayout ring_layout() {
  RingLayout y{};
  y.part = (uint32_t)(kRingStages * kStageBytes);
  y.grad = y.part + (uint32_t)(kSlots * kMaxCluster * kRingWarps * 16);
  y.bars = y.grad + kSlots * 32u;
  y.flag = y.bars + (2u * (uint32_t)kRingStages + 2u * kSlots) * 8u;
  y.count = y.flag + 16u;
  y.sent = y.count + 16u * 4u;
  y.list = y.sent + 16u * 4u;
  y.total = y.list + (uint32_t)kListRows * 4u;
  return y;
}

// -- packed fp32 pairs --------------------------------------------------------
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t bf2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// -- clusters -------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t smem_addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_async4(uint32_t addr, float a, float b, float c, float d,
                                          uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(addr),
      "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)),
      "r"(__float_as_uint(d)), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
// Words of another CTA of the cluster; the cluster's barriers order them.
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.relaxed.cluster.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Written once, not read again here: first to leave L2.
__device__ __forceinline__ void store_stream(uint4* p, const uint4& v) {
  __stcs(p, v);
}

// The two bf16 of a word minus m, in fp32.
__device__ __forceinline__ uint64_t bf_minus(uint32_t w, float m) {
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tsub.f32.bf16 %0, l, %3;\n\t"
      "sub.f32.bf16 %1, h, %3;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(w), "f"(m));
  return pack2(lo, hi);
}

// One granule of 16 bytes, minus m, as packed fp32 pairs.
template <int DT>
struct Granule {
  static constexpr int kPairs = ScoreType<DT>::kPer16 / 2;
  uint64_t v[kPairs];
};
template <int DT>
__device__ __forceinline__ Granule<DT> granule_minus(const uint4& w, float m) {
  Granule<DT> g;
  if constexpr (DT == kScoreF32) {
    const uint64_t nm = pack2(-m, -m);
    g.v[0] = add2(pack2(__uint_as_float(w.x), __uint_as_float(w.y)), nm);
    g.v[1] = add2(pack2(__uint_as_float(w.z), __uint_as_float(w.w)), nm);
  } else {
    g.v[0] = bf_minus(w.x, m);
    g.v[1] = bf_minus(w.y, m);
    g.v[2] = bf_minus(w.z, m);
    g.v[3] = bf_minus(w.w, m);
  }
  return g;
}

// A granule of -inf: no part of any sum.
template <int DT>
__device__ __forceinline__ uint4 nothing() {
  const uint32_t x = DT == kScoreF32 ? 0xff800000u : 0xff80ff80u;
  return make_uint4(x, x, x, x);
}

// Largest element of N granules (NaN is passed over: it shows in the sums).
template <int DT, int N>
__device__ __forceinline__ float granule_max(const uint4 (&w)[N]) {
  if constexpr (DT == kScoreF32) {
    float a[N];
#pragma unroll
    for (int n = 0; n < N; ++n)
      a[n] = fmaxf(fmaxf(__uint_as_float(w[n].x), __uint_as_float(w[n].y)),
                   fmaxf(__uint_as_float(w[n].z), __uint_as_float(w[n].w)));
#pragma unroll
    for (int n = 1; n < N; ++n) a[0] = fmaxf(a[0], a[n]);
    return a[0];
  } else {
    uint32_t a[N];
#pragma unroll
    for (int n = 0; n < N; ++n) a[n] = bf2_max(bf2_max(w[n].x, w[n].y), bf2_max(w[n].z, w[n].w));
#pragma unroll
    for (int n = 1; n < N; ++n) a[0] = bf2_max(a[0], a[n]);
    return fmaxf(bf_lo(a[0]), bf_hi(a[0]));
  }
}

// Element `at` of N granules, replaced by -inf.
template <int DT, int N>
__device__ __forceinline__ float granule_drop(uint4 (&w)[N], int at) {
  constexpr int kPer = ScoreType<DT>::kPer16, kWord = kPer / 4;  // elements per 32-bit word
  float z = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    uint32_t x[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (n * 4 + k != at / kWord) continue;
      if (DT == kScoreF32) {
        z = __uint_as_float(x[k]);
        x[k] = 0xff800000u;
      } else if (at & 1) {
        z = bf_hi(x[k]);
        x[k] = (x[k] & 0xffffu) | 0xff800000u;
      } else {
        z = bf_lo(x[k]);
        x[k] = (x[k] & 0xffff0000u) | 0xff80u;
      }
    }
    w[n] = make_uint4(x[0], x[1], x[2], x[3]);
  }
  return z;
}

// A thread's running sums: pairs, two chains each.
struct ThreadSums {
  float m;
  uint64_t R[2], Q[2];
};

__device__ __forceinline__ float pair_sum(const uint64_t (&v)[2]) {
  float a, b;
  unpack2(add2(v[0], v[1]), a, b);
  return a + b;
}

// Sums of N granules against the reference m.
template <int DT, bool ENT, int N>
__device__ __forceinline__ void granule_sums(const uint4 (&w)[N], float m, float c2,
                                             uint64_t (&R)[2], uint64_t (&Q)[2]) {
  const uint64_t cc = pack2(c2, c2);
  R[0] = R[1] = Q[0] = Q[1] = 0ull;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const Granule<DT> v = granule_minus<DT>(w[n], m);
#pragma unroll
    for (int k = 0; k < Granule<DT>::kPairs; ++k) {
      uint64_t d = mul2(v.v[k], cc);
      float d0, d1;
      unpack2(d, d0, d1);
      if (ENT) {
        d0 = hold_deep(d0);
        d1 = hold_deep(d1);
        d = pack2(d0, d1);
      }
      const uint64_t e = pack2(ex2(d0), ex2(d1));
      R[k & 1] = add2(R[k & 1], e);
      if (ENT) Q[k & 1] = fma2(e, d, Q[k & 1]);
    }
  }
}

// The thread's sums moved to the reference of N granules' maximum, where that
// is above theirs.
template <int DT, bool ENT, int N>
__device__ __forceinline__ void raise(ThreadSums& s, const uint4 (&w)[N], float c2) {
  const float hi = granule_max<DT, N>(w);
  if (!(hi > s.m)) return;  // the empty reference is -FLT_MAX
  const float d = fmaxf((s.m - hi) * c2, -kDeep), f = ex2(d);
  const uint64_t f2 = pack2(f, f), d2 = pack2(d, d);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (ENT) s.Q[k] = mul2(f2, fma2(d2, s.R[k], s.Q[k]));
    s.R[k] = mul2(f2, s.R[k]);
  }
  s.m = hi;
}

// Folds N granules into a thread's sums.  `fresh`: the row's first.  `drop`: the
// element that is left out (counted through the N granules), or -1; its value
// goes to `za`.
template <int DT, bool ENT, int N>
__device__ __forceinline__ void fold(ThreadSums& s, uint4 (&w)[N], bool fresh, int drop, float c2,
                                     float& za) {
  if (drop >= 0) za = granule_drop<DT, N>(w, drop);
  if (fresh) raise<DT, ENT, N>(s, w, c2);
  uint64_t R[2], Q[2];
  granule_sums<DT, ENT, N>(w, s.m, c2, R, Q);
  if (!(pair_sum(R) <= kMuch)) {
    raise<DT, ENT, N>(s, w, c2);
    granule_sums<DT, ENT, N>(w, s.m, c2, R, Q);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    s.R[k] = add2(s.R[k], R[k]);
    if (ENT) s.Q[k] = add2(s.Q[k], Q[k]);
  }
}

// The gradient p (a0 + a1 log2 p), p = 2^((z - M) c2 - l2S), of a granule.
template <int DT, bool ENT>
__device__ __forceinline__ void granule_grad(const uint4& w, float M, uint64_t c2, uint64_t nl,
                                             uint64_t A0, uint64_t A1,
                                             float (&o)[ScoreType<DT>::kPer16]) {
  const Granule<DT> z = granule_minus<DT>(w, M);
#pragma unroll
  for (int k = 0; k < Granule<DT>::kPairs; ++k) {
    uint64_t x = fma2(z.v[k], c2, nl);
    float xa, xb;
    unpack2(x, xa, xb);
    if (ENT) {
      xa = hold_deep(xa);
      xb = hold_deep(xb);
      x = pack2(xa, xb);
    }
    const uint64_t e = pack2(ex2(xa), ex2(xb));
    unpack2(mul2(e, ENT ? fma2(A1, x, A0) : A0), o[2 * k], o[2 * k + 1]);
  }
}

template <int DT>
__device__ __forceinline__ uint4 granule_pack(const float (&o)[ScoreType<DT>::kPer16]) {
  if constexpr (DT == kScoreF32)
    return make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                      __float_as_uint(o[3]));
  else
    return make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                      pack_bf16(o[6], o[7]));
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// The warp's parts joined in every lane.
__device__ __forceinline__ RowSums warp_join(RowSums s, float c2) {
  const float m = warp_max(s.m);
  const float d = fmaxf((s.m - m) * c2, -kDeep), f = ex2(d);
  float Q = f * fmaf(d, s.R, s.Q), R = s.R * f;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) {
    R += __shfl_xor_sync(0xffffffffu, R, k);
    Q += __shfl_xor_sync(0xffffffffu, Q, k);
  }
  return RowSums{m, R, Q};
}

// A CTA's share of a row.
struct RowShare {
  int64_t base;  // byte offset of the row's aligned image from the buffer's start (may be < 0)
  int shift;     // elements of the image before the row
  int g0, n;     // first granule, granules
  int whole0, whole1;  // granules of the image that lie inside the row: [whole0, whole1)
};

template <int DT>
__device__ __forceinline__ RowShare row_share(const void* buf, int64_t ld, int row, int V,
                                              int log2C, int rank) {
  constexpr int kB = ScoreType<DT>::kBytes, kPer = ScoreType<DT>::kPer16;
  RowShare s;
  const int64_t off = (int64_t)row * ld * kB;
  const int mis = (int)(((uintptr_t)buf + (uintptr_t)off) & 15u);
  s.base = off - mis;
  s.shift = mis / kB;
  const int end = s.shift + V;
  const int G = (end + kPer - 1) / kPer;
  const int per = (((G + (1 << log2C) - 1) >> log2C) + 7) & ~7;
  s.g0 = min(G, rank * per);
  s.n = min(G - s.g0, per);
  s.whole0 = s.shift ? 1 : 0;
  s.whole1 = end / kPer;
  return s;
}

// The rows of cluster `cid`, where they are listed: its live ones, then its
// ignored ones.  Returns how many, once every thread of the block has passed a
// barrier; the list is complete after the next.
__device__ __forceinline__ int list_rows(const ScoreArgs& p, const RingArgs& q,
                                         const RowRange& range, int cid, int ncl, int* count,
                                         int* list) {
  if (!q.listed) return 0;
  constexpr int kWarps = kRingThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.rows + kWarps * 32 - 1) / (kWarps * 32) * 32;
  const int r0 = min(p.rows, warp * per), r1 = min(p.rows, r0 + per);
  auto lives = [&](int r) {
    return __ballot_sync(0xffffffffu,
                         r < r1 && range.live(r, p.tokens[r], p.weights ? p.weights[r] : 1.f));
  };
  int n = 0;
#pragma unroll 8
  for (int r = r0; r < r1; r += 32) n += __popc(lives(r + lane));
  if (lane == 0) count[warp] = n;
  __syncthreads();
  int live = 0, before = 0;  // in all, and in the warps before this one
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = live;
    live += count[w];
  }
  // the clusters with a live row fewer are the first to take an ignored one
  const int back = ncl - 1 - cid;
  const int mine = (live - cid + ncl - 1) / ncl;  // live rows
#pragma unroll 4
  for (int r = r0; r < r1; r += 32) {
    const unsigned m = lives(r + lane);
    const bool on = m >> lane & 1u;
    const int ahead = before + __popc(m & ((1u << lane) - 1u));  // live rows before this one
    const int rank = on ? ahead : r + lane - ahead, k = rank / ncl;
    if (r + lane < r1 && rank - k * ncl == (on ? cid : back)) list[on ? k : mine + k] = r + lane;
    before += __popc(m);
  }
  return mine + (p.rows - live - back + ncl - 1) / ncl;
}

// A finisher's warp waits for every sum still on its way into this CTA, when
// nobody sends any more.  sent: rows sent by each of this CTA's consumers, rows
// finished (the next one's sums are awaited), whether the finisher gave up.  A
// row is sent only after the one kSlots before it was finished everywhere, so at
// most kSlots rows are in question; of a row of which some sums come, or which
// is awaited, the warp sends itself those that will not.
static __device__ __noinline__ void drain_sums(float4* part, uint64_t* sums_in, uint32_t* sent,
                                               int C) {
  constexpr int NW = kRingWarps;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), done = sent[NW];
  for (uint32_t k = done; k < done + kSlots; ++k) {
    const uint32_t par = k % kSlots;
    unsigned come = 0u;
    for (int j = 0; j < kMaxCluster * NW / 32; ++j) {
      const int e = lane + 32 * j;
      if (e < C * NW && ld_cluster(map_rank(smem_u32(sent + e % NW), e / NW)) > k) come |= 1u << j;
    }
    if (k > done && !__any_sync(0xffffffffu, come != 0u)) break;
    if (k > done && lane == 0) mbar_arrive_expect_tx(&sums_in[par], (uint32_t)(C * NW * 16));
    __syncwarp();
    for (int j = 0; j < kMaxCluster * NW / 32; ++j) {
      const int e = lane + 32 * j;
      if (e < C * NW && !(come >> j & 1u))
        st_async4(map_rank(smem_u32(part + par * kMaxCluster * NW + e), rank), 0.f, 0.f, 0.f, 0.f,
                  map_rank(smem_u32(&sums_in[par]), rank));
    }
    mbar_wait(&sums_in[par], (k / kSlots) & 1u, kDrainLimitNs);
    __syncwarp();
  }
}

template <int DT, bool ENT, bool GRAD>
__global__ void __launch_bounds__(kRingThreads, kRingCtas)
    score_ring_kernel(const ScoreArgs p, const RingArgs q) {
  constexpr int NW = kRingWarps;
  constexpr int kB = ScoreType<DT>::kBytes, kPer = ScoreType<DT>::kPer16;
  constexpr int kT = NW * 32;
  constexpr int kIter = kStageIter;
  extern __shared__ __align__(128) unsigned char ring[];
  constexpr RingLayout lay = ring_layout();
  float4* part = reinterpret_cast<float4*>(ring + lay.part);  // [kSlots][C NW]
  RowGrad* grad = reinterpret_cast<RowGrad*>(ring + lay.grad);  // [kSlots], 32 bytes apart
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + lay.bars);
  uint64_t* empty = full + kRingStages;
  uint64_t* sums_in = empty + kRingStages;  // [kSlots] a row's sums have arrived
  uint64_t* result = sums_in + kSlots;   // [kSlots] its factors are there (no gradient: its sums are read)
  int* abort_flag = reinterpret_cast<int*>(ring + lay.flag);
  int* list = reinterpret_cast<int*>(ring + lay.list);
  uint32_t* sent = reinterpret_cast<uint32_t*>(ring + lay.sent);  // see drain_sums

  uint64_t begun = p.wait_ns < kSuspendHintNs ? global_ns() : 0;  // see wait_limited
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool is_policy = ENT && q.mode == kModePolicy;  // always with entropies
  const int C = 1 << q.log2C;
  const int rank = (int)cluster_rank();
  const int cid = blockIdx.x >> q.log2C, ncl = gridDim.x >> q.log2C;
  if (tid == 0) {
    for (int s = 0; s < kRingStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], NW);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sums_in[s], 1);
      mbar_init(&result[s], 1);
    }
    *abort_flag = 0;
    sent[NW + 1] = 0u;
    fence_mbar_init();
  }
  const RowRange range = row_range(p);
  const int n_rows = list_rows(p, q, range, cid, ncl, reinterpret_cast<int*>(ring + lay.count), list);
  __syncthreads();
  cluster_sync_all();
  // this cluster's k-th row, or the number of rows
  auto row_at = [&](int k) {
    return !q.listed ? min(p.rows, cid + k * ncl) : k < n_rows ? list[k] : p.rows;
  };

  // A wait that gave up cuts the cluster short.
  auto fail = [&]() {
    atomicOr(p.status, kScoreTimeout);
#pragma unroll 1
    for (int c = 0; c < C; ++c) st_cluster(map_rank(smem_u32(abort_flag), c), 1u);
  };
  // A barrier's phase has completed: one test and a vote, the bounded wait
  // only where that fails.  The outcome is the whole warp's.  The test may
  // suspend the thread until the phase completes, whatever the limit.
  auto wait = [&](uint64_t* bar, uint32_t ph) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, ph))) return true;
    return (bool)__all_sync(0xffffffffu, mbar_wait_timed(bar, ph, p.wait_ns, abort_flag));
  };
  // The same, but a limit shorter than that is kept: the finisher's wait for a
  // row's sums, counted from the last one's end (the first one's from the
  // kernel's start, so that sums which are there before the finisher is have
  // taken their time too): a short limit runs out in every call.  In every wait
  // the look at the limit costs up to 3 % (2048 rows of 262144 bf16, scores:
  // 194.6 us against 188.4), in this one nothing (188.4).
  auto wait_limited = [&](uint64_t* bar, uint32_t ph) {
    if (p.wait_ns >= kSuspendHintNs) return wait(bar, ph);
    const bool came = mbar_wait_timed(bar, ph, p.wait_ns, abort_flag) &&
                      global_ns() - begun <= p.wait_ns;
    begun = global_ns();
    return (bool)__all_sync(0xffffffffu, came);
  };
  bool ok = true;
  const float nan = __int_as_float(0x7fc00000);
  double t[kPolicyTerms] = {};  // the finisher's

  if (warp == NW) {
    // ------------------------------------------------------------ producer
    const uint64_t once = evict_first_policy(), again = evict_last_policy();
    RingWalk walk{0, 1, 0xffffffffu};  // an empty stage's first wait passes at once
    uint32_t fills = 0u;  // parity of each slot's copies
    // One stage of a share, granules g .. end - 1, into the walk's slot.
    auto copy_stage = [&](const RowShare& s, const char* img, int g, int end, uint64_t policy) {
      if (!wait(&empty[walk.slot], walk.phase())) {
        ok = false;
        return;
      }
      unsigned char* dst = ring + (size_t)walk.slot * kStageBytes;
      const int b0 = max(g, s.whole0), b1 = max(b0, min(end, s.whole1));
      if (b0 != g || b1 != end) {
        // granules the row fills in part: at most the first and the last
        for (int e = lane; e < 2 * kPer; e += 32) {
          const int gr = e < kPer ? 0 : s.whole1;
          const bool mine = gr >= g && gr < end && (gr < b0 || gr >= b1) &&
                            (e < kPer || s.whole1 != 0 || s.whole0 == 0);
          const int at = gr * kPer + (e & (kPer - 1));  // element of the image
          if (mine) {
            const int v = at - s.shift;
            const bool in = v >= 0 && v < p.V;
            unsigned char* to = dst + (size_t)(gr - g) * 16 + (e & (kPer - 1)) * kB;
            if (kB == 4)
              *reinterpret_cast<uint32_t*>(to) =
                  in ? reinterpret_cast<const uint32_t*>(img)[at] : 0xff800000u;
            else
              *reinterpret_cast<uint16_t*>(to) =
                  in ? reinterpret_cast<const uint16_t*>(img)[at] : (uint16_t)0xff80u;
          }
        }
        __syncwarp();
      }
      if (lane == 0) {
        const uint32_t bytes = (uint32_t)(b1 - b0) * 16u;
        mbar_arrive_expect_tx(&full[walk.slot], bytes);
        if (bytes)
          bulk_load(dst + (size_t)(b0 - g) * 16, img + (size_t)b0 * 16, bytes, &full[walk.slot],
                    policy);
      }
      __syncwarp();
      fills ^= 1u << walk.slot;
      walk.used();
      walk.step();
    };
    int next = row_at(0);
    int token = -1;
    float weight = 1.f;
    if (next < p.rows) {
      token = p.tokens[next];
      if (p.weights) weight = p.weights[next];
    }
    for (int i = 1; next < p.rows && ok; ++i) {
      const int row = next;
      const bool on = range.live(row, token, weight);
      next = row_at(i);
      if (next < p.rows) {
        token = p.tokens[next];
        if (p.weights) weight = p.weights[next];
      }
      if (!on) continue;
      const RowShare s = row_share<DT>(p.logits, p.ld, row, p.V, q.log2C, rank);
      const char* img = static_cast<const char*>(p.logits) + s.base;
      const int n_st = (s.n + kStageGran - 1) / kStageGran;
      const bool back = GRAD && !q.ahead;
      const int kept = min(n_st, kRingStages);
      for (int k = 0; k < n_st && ok; ++k)
        copy_stage(s, img, s.g0 + k * kStageGran, s.g0 + min(s.n, (k + 1) * kStageGran),
                   (back && k < n_st - kept) || p.stats ? again : once);
      if (back) {
        walk.turn();
        walk.step(kept);
        for (int k = n_st - kept - 1; k >= 0 && ok; --k)
          copy_stage(s, img, s.g0 + k * kStageGran, s.g0 + (k + 1) * kStageGran, once);
      }
    }
    if (!ok && lane == 0) fail();
    // every copy issued has landed before the CTA may leave
    if (lane == 0)
      for (int k = 0; k < kRingStages; ++k)
        mbar_wait(&full[k], (fills >> k & 1u) ^ 1u, kDrainLimitNs);
    __syncwarp();
  } else if (warp == NW + 1) {
    // ------------------------------------------------------------ finisher
    uint32_t count = 0;  // rows finished
    const bool first = rank == 0;
    if (GRAD || first) {
      // a row's inputs, fetched one row ahead
      int token = -1;
      float weight = 1.f, T = p.temp, x0 = 0.f, x1 = 0.f, x2 = 0.f;
      auto fetch = [&](int row) {
        token = p.tokens[row];
        if (p.weights) weight = p.weights[row];
        if (p.temps) T = p.temps[row];
        if (is_policy) {
          x0 = p.old_lp[row];
          x1 = p.adv[row];
          if (p.ref_lp) x2 = p.ref_lp[row];
        } else if (q.mode == kModeGrad) {
          x0 = p.g_lp[row];
          if (p.g_h) x1 = p.g_h[row];
        }
      };
      int next = row_at(0), i = 1;
      if (next < p.rows) fetch(next);
      for (; next < p.rows && ok; ++i) {
        const int row = next;
        const int a = token;
        const float wt = weight, y0 = x0, y1 = x1, y2 = x2;
        const float Trow = row_temp_ok(T) ? T : nan;
        next = row_at(i);
        if (next < p.rows) fetch(next);
        if (!range.live(row, a, wt)) {
          if (first && lane == 0) {
            if (p.logprobs) p.logprobs[row] = 0.f;
            if (p.entropies) p.entropies[row] = 0.f;
          }
          continue;
        }
        const uint32_t par = count % kSlots, ph = (count / kSlots) & 1u;
        const Scale sc = row_scale(Trow);
        const float c2 = sc.c2;
        if (lane == 0) mbar_arrive_expect_tx(&sums_in[par], (uint32_t)(C * NW * 16));
        __syncwarp();
        if (!wait_limited(&sums_in[par], ph)) {
          ok = false;
          break;
        }
        // the warps' sums against their largest reference; the token's logit
        // comes from the warp that holds it, the others send 0
        float4 v[kMaxCluster * NW / 32];
        float m = -FLT_MAX;
#pragma unroll
        for (int k = 0; k < kMaxCluster * NW / 32; ++k) {
          const int e = lane + 32 * k;
          v[k] = e < C * NW ? part[par * kMaxCluster * NW + e]
                            : make_float4(-FLT_MAX, 0.f, 0.f, 0.f);
          m = fmaxf(m, v[k].x);
        }
        m = warp_max(m);
        RowSums all{m, 0.f, 0.f};
        float za = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxCluster * NW / 32; ++k) {
          const float d = fmaxf((v[k].x - m) * c2, -kDeep), f = ex2(d);
          all.R = fmaf(f, v[k].y, all.R);
          all.Q = fmaf(f, fmaf(d, v[k].y, v[k].z), all.Q);
          za += v[k].w;
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) {
          all.R += __shfl_xor_sync(0xffffffffu, all.R, k);
          all.Q += __shfl_xor_sync(0xffffffffu, all.Q, k);
          za += __shfl_xor_sync(0xffffffffu, za, k);
        }
        if (!GRAD) {  // the slots are free again
          __syncwarp();
          if (lane < C) arrive_remote(map_rank(smem_u32(&result[par]), lane));
        }
        const bool bad = a >= p.V;
        const RowResult r = row_result<ENT>(all, bad ? nan : za, sc);
        RowCoef c{y0, y1};
        PolicyRow o{};
        if (is_policy) {
          o = policy_row(p, r, y0, y1, y2, wt);
          c = policy_coef(p, r, o, y0, y1, y2, wt);
        }
        if (GRAD) {
          if (lane == 0) {
            const RowGrad f = row_grad<ENT>(r, c, Trow);
            *reinterpret_cast<RowGrad*>(reinterpret_cast<char*>(grad) + par * 32) = f;
            mbar_arrive(&result[par]);
          }
          __syncwarp();
        }
        if (first && lane == 0) {
          if (p.logprobs) p.logprobs[row] = r.lp;
          if (ENT && p.entropies) p.entropies[row] = r.H;
          if (p.stats) p.stats[row] = make_float4(r.M, r.l2S, r.l2S_low, r.rest);
          const uint32_t bits = (bad ? kScoreBadToken : 0u) | (r.finite ? 0u : kScoreNonFinite);
          if (bits) atomicOr(p.status, bits);
          if (is_policy) policy_add(p, r, o, y0, y1, y2, wt, t);
        }
        ++count;
      }
      if (!ok) {
        // the rows left, this one first: NaN, not what was there before
        if (lane == 0) {
          sent[NW] = count;
          sent[NW + 1] = 1u;
          fail();
        }
        for (int k = i - 1 + lane; first && row_at(k) < p.rows; k += 32) {
          const int row = row_at(k);
          if (p.logprobs) p.logprobs[row] = nan;
          if (p.entropies) p.entropies[row] = nan;
          if (p.stats) p.stats[row] = make_float4(nan, nan, nan, nan);
        }
      }
    }
  } else {
    // ----------------------------------------------------------- consumers
    RingWalk walk{0, 1, 0u};
    int held = 0;        // ahead: the first slot still held
    uint32_t count = 0;  // rows folded
    if (lane == 0) sent[warp] = 0u;
    // A folded row whose gradient is still to be written.
    struct Pending {
      int row, token;
      float c2;
      int k;  // its number among this cluster's rows
    } last{-1, 0, 0.f, 0};

    // The token's place in this CTA's share: this thread's granule (counted
    // along its own granules, -1: another thread's) and element.
    auto place = [&](const RowShare& sh, int token, int& el) {
      const int at = min(token, p.V) + sh.shift, ag = at / kPer - sh.g0;
      el = at & (kPer - 1);
      return token < p.V && ag >= 0 && ag < sh.n && (ag & (kT - 1)) == tid ? ag / kT : -1;
    };
    auto grad_image = [&](int row, const RowShare& sh) {
      return static_cast<char*>(p.d_logits) + (int64_t)row * p.ldd * kB - sh.shift * kB;
    };

    // Pass 2: a folded row's gradient, number `k` of the rows folded.
    auto write_grad = [&](const Pending& w, uint32_t k) {
      if (!wait(&result[k % kSlots], (k / kSlots) & 1u)) {
        ok = false;
        return;
      }
      const RowGrad r =
          *reinterpret_cast<const RowGrad*>(reinterpret_cast<char*>(grad) + (k % kSlots) * 32);
      const RowShare sh = row_share<DT>(p.logits, p.ld, w.row, p.V, q.log2C, rank);
      char* dz = grad_image(w.row, sh);
      // aligned as the logits, or written element by element
      const bool dz_vec = ((uintptr_t)dz & 15u) == 0;
      int el;
      const int mine = place(sh, w.token, el);
      const float c2 = w.c2;
      const uint64_t cc = pack2(c2, c2), nl = pack2(-r.l2S, -r.l2S), A0 = pack2(r.a0, r.a0), A1 = pack2(r.a1, r.a1);
      const int n_st = (sh.n + kStageGran - 1) / kStageGran;
      if (!q.ahead) walk.turn();
      for (int i = 0; i < n_st; ++i) {
        const int st_no = q.ahead ? i : n_st - 1 - i;  // the stage of the share
        if (!q.ahead && i >= kRingStages) {
          if (!wait(&full[walk.slot], walk.phase())) {
            ok = false;
            return;
          }
          walk.used();
        }
        const int at = q.ahead ? held : walk.slot;
        const uint4* st = reinterpret_cast<const uint4*>(ring + (size_t)at * kStageBytes) + tid;
        const int n = sh.n - st_no * kStageGran, first = st_no * kIter;
        const int g = sh.g0 + st_no * kStageGran + tid;
        // this thread's granules of the stage: whole ones without the token?
        const int many = min(kIter, (n - tid + kT - 1) / kT);
        const bool plain = dz_vec && (unsigned)(mine - first) >= (unsigned)kIter &&
                           g >= sh.whole0 && g + (many - 1) * kT < sh.whole1;
        uint4* out = reinterpret_cast<uint4*>(dz) + g;
        if (plain && many == kIter) {
#pragma unroll
          for (int j = 0; j < kIter; ++j) {
            float o[kPer];
            granule_grad<DT, ENT>(st[j * kT], r.M, cc, nl, A0, A1, o);
            store_stream(out + j * kT, granule_pack<DT>(o));
          }
        } else if (plain) {
#pragma unroll 1
          for (int j = 0; j < many; ++j) {
            float o[kPer];
            granule_grad<DT, ENT>(st[j * kT], r.M, cc, nl, A0, A1, o);
            store_stream(out + j * kT, granule_pack<DT>(o));
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < many; ++j) {
            const int gj = g + j * kT;
            float o[kPer];
            granule_grad<DT, ENT>(st[j * kT], r.M, cc, nl, A0, A1, o);
            if (first + j == mine) {
#pragma unroll
              for (int k = 0; k < kPer; ++k)
                if (k == el) o[k] = r.own;
            }
            if (dz_vec && gj >= sh.whole0 && gj < sh.whole1) {
              store_stream(reinterpret_cast<uint4*>(dz) + gj, granule_pack<DT>(o));
            } else {
#pragma unroll
              for (int k = 0; k < kPer; ++k) {
                const int v = gj * kPer + k - sh.shift;
                if (v >= 0 && v < p.V) store_grad<DT>(dz, (int64_t)gj * kPer + k, o[k]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[at]);
        if (q.ahead)
          held = held + 1 == kRingStages ? 0 : held + 1;
        else
          walk.step();
      }
    };

    int next = row_at(0), i = 1;
    int token = -1;
    float weight = 1.f, T = p.temp;
    if (next < p.rows) {
      token = p.tokens[next];
      if (p.weights) weight = p.weights[next];
      if (p.temps) T = p.temps[next];
    }
    for (; next < p.rows && ok; ++i) {
      const int row = next;
      const int a = token;
      const float wt = weight;
      const float c2 = log2e_over(row_temp_ok(T) ? T : nan);
      next = row_at(i);
      if (next < p.rows) {
        token = p.tokens[next];
        if (p.weights) weight = p.weights[next];
        if (p.temps) T = p.temps[next];
      }
      const RowShare sh = row_share<DT>(p.logits, p.ld, row, p.V, q.log2C, rank);
      if (!range.live(row, a, wt)) {
        if (GRAD) {
          char* dz = grad_image(row, sh);
          const bool dz_vec = ((uintptr_t)dz & 15u) == 0;
          for (int g = sh.g0 + tid; g < sh.g0 + sh.n; g += kT) {
            if (dz_vec && g >= sh.whole0 && g < sh.whole1) {
              *reinterpret_cast<uint4*>(dz + (int64_t)g * 16) = make_uint4(0, 0, 0, 0);
            } else {
#pragma unroll 1
              for (int k = 0; k < kPer; ++k) {
                const int v = g * kPer + k - sh.shift;
                if (v >= 0 && v < p.V) store_grad<DT>(dz, (int64_t)g * kPer + k, 0.f);
              }
            }
          }
        }
        continue;
      }
      int el;
      const int mine = place(sh, a, el);

      // pass 1: the sums
      ThreadSums s;
      s.m = -FLT_MAX;
      s.R[0] = s.R[1] = s.Q[0] = s.Q[1] = 0ull;
      float za = 0.f;
      const int n_st = (sh.n + kStageGran - 1) / kStageGran;
      // stages that stay for the gradient: all (ahead), or the last ones
      const int stay = !GRAD ? 0 : q.ahead ? n_st : min(n_st, kRingStages);
      for (int k = 0; k < n_st; ++k) {
        if (!wait(&full[walk.slot], walk.phase())) {
          ok = false;
          break;
        }
        walk.used();
        const uint4* st =
            reinterpret_cast<const uint4*>(ring + (size_t)walk.slot * kStageBytes) + tid;
        const int n = sh.n - k * kStageGran, first = k * kIter;
        const int drop =
            (unsigned)(mine - first) < (unsigned)kIter ? (mine - first) * kPer + el : -1;
        if ((kIter - 1) * kT + tid < n) {
          uint4 w[kIter];
#pragma unroll
          for (int j = 0; j < kIter; ++j) w[j] = st[j * kT];
          fold<DT, ENT, kIter>(s, w, k == 0, drop, c2, za);
        } else if (tid < n) {  // nothing past the share's end
          uint4 w[kIter];
#pragma unroll
          for (int j = 0; j < kIter; ++j) w[j] = j * kT + tid < n ? st[j * kT] : nothing<DT>();
          fold<DT, ENT, kIter>(s, w, k == 0, drop, c2, za);
        }
        if (k < n_st - stay) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[walk.slot]);
        }
        walk.step();
      }
      if (!ok) break;
      // this warp's sums to the finishing CTAs, with the token's logit where
      // this warp holds it
      const uint32_t par = count % kSlots;
      const RowSums rs = warp_join(RowSums{s.m, pair_sum(s.R), ENT ? pair_sum(s.Q) : 0.f}, c2);
      const unsigned holder = __ballot_sync(0xffffffffu, mine >= 0);
      za = holder ? __shfl_sync(0xffffffffu, za, __ffs(holder) - 1) : 0.f;
      // A slot's last sums have been read.  Without a gradient the first CTA's
      // finisher says so.  With one it follows: a CTA sends row k + kSlots
      // after its result of row k + 2, which needed this CTA's sums of row
      // k + 2, sent after this CTA's result of row k.
      if (!GRAD && count >= kSlots && !wait(&result[par], (count / kSlots - 1u) & 1u)) {
        ok = false;
        break;
      }
      if (lane < (GRAD ? C : 1)) {
        const uint32_t to = smem_u32(&part[par * kMaxCluster * NW + rank * NW + warp]);
        st_async4(map_rank(to, lane), rs.m, rs.R, rs.Q, za,
                  map_rank(smem_u32(&sums_in[par]), lane));
      }
      if (lane == 0) sent[warp] = count + 1u;
      if (GRAD) {
        const Pending now{row, a, c2, i - 1};
        if (!q.ahead)
          write_grad(now, count);
        else if (last.row >= 0)
          write_grad(last, count - 1u);
        if (!ok) break;
        last = now;
      }
      ++count;
    }
    if (GRAD && ok && q.ahead && last.row >= 0) write_grad(last, count - 1u);
    if (!ok) {
      if (lane == 0) fail();
      // this warp's first granule of each row whose gradient it has not finished: NaN
      for (int k = q.ahead && last.row >= 0 ? last.k : i - 1;
           GRAD && lane == 0 && row_at(k) < p.rows; ++k) {
        const RowShare sh = row_share<DT>(p.logits, p.ld, row_at(k), p.V, q.log2C, rank);
        for (int e = 0; tid < sh.n && e < kPer; ++e) {
          const int v = (sh.g0 + tid) * kPer + e - sh.shift;
          if (v >= 0 && v < p.V)
            store_grad<DT>(grad_image(row_at(k), sh), (int64_t)(sh.g0 + tid) * kPer + e, nan);
        }
      }
      __syncwarp();
    }
  }
  __syncthreads();
  cluster_sync_all();
  // after a pass cut short sums may still be on their way
  if (*(volatile int*)abort_flag) {
    if (warp == NW + 1 && sent[NW + 1]) drain_sums(part, sums_in, sent, C);
    __syncthreads();
    cluster_sync_all();
  }
  if (is_policy && rank == 0) {
    // a cut-short pass gives NaN, not a part of the sums
    if (*(volatile int*)abort_flag)
      for (int k = 0; k < kPolicyTerms; ++k) t[k] = (double)nan;
    policy_total<kRingThreads, 1>(p, tid == (NW + 1) * 32 ? 0 : -1, t, cid, ncl);
  }
}

// ---------------------------------------------------------------------------
// Short rows: held in registers
//
// W warps take a row, each lane up to 8 of its granules, and keep it from the
// one read to the gradient's write.  A short row's cost is its latency (load,
// sums, logarithms, store), so what counts is how many are in flight: W = 1
// up to 4 KB, W = 4 up to 16 KB, four warps to a block, six to eight blocks to
// an SM.  A policy step: 16 rows of 1024 fp32 5.0 us (one row's latency), 16384
// rows of 4096 bf16 107 us (2.5 TB/s; the issue slots, 62 % busy, go half to
// the row's logarithms and loss terms, which each of its warps computes so
// that no second barrier waits for them).
// ---------------------------------------------------------------------------
constexpr int kShortThreads = 128;
constexpr int kShortGran = 8;  // granules per lane
constexpr int kShortChunk = 2;
constexpr __host__ __device__ int short_bytes(int W) { return W * 32 * kShortGran * 16; }

template <int DT, bool ENT, bool GRAD, int W>
__global__ void __launch_bounds__(kShortThreads, GRAD ? 6 : 8)
    score_short_kernel(const ScoreArgs p, const int mode) {
  constexpr int kB = ScoreType<DT>::kBytes, kPer = ScoreType<DT>::kPer16;
  constexpr int kRows = kShortThreads / 32 / W;  // per block
  constexpr int kT = W * 32;
  __shared__ float4 warp_part[2][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tid = threadIdx.x % kT;  // in the row
  const RowRange range = row_range(p);
  const float nan = __int_as_float(0x7fc00000);
  const bool is_policy = ENT && mode == kModePolicy;  // always with entropies
  double t[kPolicyTerms] = {};
  int flip = 0;
  // W = 4: the block's warps share a row and meet at barriers
  for (int i = blockIdx.x * kRows + warp / W; i < p.rows; i += gridDim.x * kRows) {
    const int row = i;
    const int token = p.tokens[row];
    const float weight = p.weights ? p.weights[row] : 1.f;
    const RowShare sh = row_share<DT>(p.logits, p.ld, row, p.V, 0, 0);
    char* dz = nullptr;
    bool dz_vec = false;
    if (GRAD) {
      dz = static_cast<char*>(p.d_logits) + (int64_t)row * p.ldd * kB - sh.shift * kB;
      dz_vec = ((uintptr_t)dz & 15u) == 0;
    }
    // one granule of the gradient
    auto put = [&](int g, const float (&o)[kPer]) {
      if (dz_vec && g >= sh.whole0 && g < sh.whole1) {
        store_stream(reinterpret_cast<uint4*>(dz) + g, granule_pack<DT>(o));
      } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int v = g * kPer + k - sh.shift;
          if (v >= 0 && v < p.V) store_grad<DT>(dz, (int64_t)g * kPer + k, o[k]);
        }
      }
    };
    if (!range.live(row, token, weight)) {
      if (tid == 0) {
        if (p.logprobs) p.logprobs[row] = 0.f;
        if (p.entropies) p.entropies[row] = 0.f;
      }
      if (GRAD) {
        const float zero[kPer] = {};
        for (int g = tid; g < sh.n; g += kT) put(g, zero);
      }
      continue;
    }
    // the row, in registers
    const char* img = static_cast<const char*>(p.logits) + sh.base;
    uint4 w[kShortGran / kShortChunk][kShortChunk];
#pragma unroll
    for (int c = 0; c < kShortGran; ++c) {
      const int g = c * kT + tid;
      uint4 x = nothing<DT>();
      if (g < sh.n) {
        if (g >= sh.whole0 && g < sh.whole1) {
          x = reinterpret_cast<const uint4*>(img)[g];
        } else {
          uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int v = g * kPer + k - sh.shift;
            if (v < 0 || v >= p.V) continue;
            if (kB == 4)
              e[k & 3] = reinterpret_cast<const uint32_t*>(img)[g * 4 + (k & 3)];
            else {
              const uint32_t h = reinterpret_cast<const uint16_t*>(img)[g * 8 + k];
              e[(k >> 1) & 3] = (k & 1) ? (e[(k >> 1) & 3] & 0xffffu) | h << 16
                                        : (e[(k >> 1) & 3] & 0xffff0000u) | h;
            }
          }
          x = make_uint4(e[0], e[1], e[2], e[3]);
        }
      }
      w[c / kShortChunk][c % kShortChunk] = x;
    }
    float T = p.temps ? p.temps[row] : p.temp;
    if (!row_temp_ok(T)) T = nan;
    float x0 = 0.f, x1 = 0.f, x2 = 0.f;
    if (is_policy) {
      x0 = p.old_lp[row];
      x1 = p.adv[row];
      if (p.ref_lp) x2 = p.ref_lp[row];
    } else if (mode == kModeGrad) {
      x0 = p.g_lp[row];
      if (p.g_h) x1 = p.g_h[row];
    }
    const Scale sc = row_scale(T);
    const float c2 = sc.c2;
    const bool bad = token >= p.V;
    const int at = min(token, p.V) + sh.shift, ag = at / kPer, el = at & (kPer - 1);
    const int mine = !bad && ag % kT == tid ? ag / kT : -1;
    ThreadSums s;
    s.m = -FLT_MAX;
    s.R[0] = s.R[1] = s.Q[0] = s.Q[1] = 0ull;
    float za = 0.f;
#pragma unroll
    for (int c = 0; c < kShortGran / kShortChunk; ++c) {
      if (c * kShortChunk * kT >= sh.n) break;  // the same in every lane
      uint4 v[kShortChunk];
#pragma unroll
      for (int k = 0; k < kShortChunk; ++k) v[k] = w[c][k];
      const int j = mine - c * kShortChunk;
      fold<DT, ENT, kShortChunk>(s, v, c == 0, j >= 0 && j < kShortChunk ? j * kPer + el : -1, c2,
                                 za);
    }
    RowSums all = warp_join(RowSums{s.m, pair_sum(s.R), ENT ? pair_sum(s.Q) : 0.f}, c2);
    const unsigned holder = __ballot_sync(0xffffffffu, mine >= 0);
    za = holder ? __shfl_sync(0xffffffffu, za, __ffs(holder) - 1) : 0.f;
    if (W > 1) {
      if (lane == 0) warp_part[flip][warp] = make_float4(all.m, all.R, all.Q, za);
      __syncthreads();
      all = row_sums_empty();
      za = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const float4 v = warp_part[flip][k];
        all = row_sums_join(all, RowSums{v.x, v.y, v.z}, c2);
        za += v.w;
      }
      flip ^= 1;  // the next row's sums do not meet a slow reader of these
    }
    const RowResult r = row_result<ENT>(all, bad ? nan : za, sc);
    RowCoef c{x0, x1};
    if (is_policy) {
      const PolicyRow o = policy_row(p, r, x0, x1, x2, weight);
      c = policy_coef(p, r, o, x0, x1, x2, weight);
      if (tid == 0) policy_add(p, r, o, x0, x1, x2, weight, t);
    }
    if (tid == 0) {
      if (p.logprobs) p.logprobs[row] = r.lp;
      if (ENT && p.entropies) p.entropies[row] = r.H;
      if (p.stats) p.stats[row] = make_float4(r.M, r.l2S, r.l2S_low, r.rest);
      const uint32_t bits = (bad ? kScoreBadToken : 0u) | (r.finite ? 0u : kScoreNonFinite);
      if (bits) atomicOr(p.status, bits);
    }
    if (GRAD) {
      const RowGrad f = row_grad<ENT>(r, c, T);
      const uint64_t cc = pack2(c2, c2), nl = pack2(-f.l2S, -f.l2S), A0 = pack2(f.a0, f.a0), A1 = pack2(f.a1, f.a1);
#pragma unroll
      for (int c1 = 0; c1 < kShortGran; ++c1) {
        const int g = c1 * kT + tid;
        if (g >= sh.n) break;
        float o[kPer];
        granule_grad<DT, ENT>(w[c1 / kShortChunk][c1 % kShortChunk], f.M, cc, nl, A0, A1, o);
        if (c1 == mine) {
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            if (k == el) o[k] = f.own;
        }
        put(g, o);
      }
    }
  }
  if (is_policy)
    policy_total<kShortThreads, kRows>(p, tid == 0 ? warp / W : -1, t, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------------------
// The gradient of g log p_a from the rows' statistics
//
// One read and one write: for a loss whose factor g needs every row's sums
// first (the preference loss).  A block takes 32 KB of a row.  The rows go in
// the opposite order of the pass that made the statistics, so that what that
// pass read last is still in L2.  A copy in its cost: 1024 rows of 262144 bf16
// take 169 us, 6.35 TB/s (0.97 of the measured copy rate).  The rows' own pass
// before it (94 us) cannot be saved above L2's size: a pair's factor needs both
// of its sequences first.
// ---------------------------------------------------------------------------
constexpr int kApplyThreads = 256, kApplyGran = 8;  // granules per thread

template <int DT>
__global__ void __launch_bounds__(kApplyThreads)
    score_apply_kernel(const ScoreArgs p, const int tiles) {  // per row
  constexpr int kB = ScoreType<DT>::kBytes, kPer = ScoreType<DT>::kPer16;
  const int row = p.rows - 1 - (int)(blockIdx.x / (unsigned)tiles);
  const int tile = tiles - 1 - (int)(blockIdx.x % (unsigned)tiles);
  const RowShare sh = row_share<DT>(p.logits, p.ld, row, p.V, 0, 0);
  const int g0 = tile * (kApplyThreads * kApplyGran) + (int)threadIdx.x;
  const char* img = static_cast<const char*>(p.logits) + sh.base;
  char* dz = static_cast<char*>(p.d_logits) + (int64_t)row * p.ldd * kB - sh.shift * kB;
  const bool vec = ((uintptr_t)dz & 15u) == 0;
  const int token = p.tokens[row];
  float T = p.temps ? p.temps[row] : p.temp;
  if (!row_temp_ok(T)) T = __int_as_float(0x7fc00000);
  const Scale sc = row_scale(T);
  const float iT = 1.f / T;
  const RowRange range = row_range(p);
  griddep_wait();  // the statistics and factors
  const bool on = range.live(row, token, 1.f);
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
  float g = 0.f;
  if (on) {
    st = __ldcg(p.stats + row);
    g = __ldcg(p.g_lp + row);
  }
  // p = 2^(d - l2S) 2^-l2S_low: the second factor goes into the coefficient
  const float a0 = fmaf(-kLn2, st.z, 1.f) * (-iT * g), own = iT * g * st.w;
  const uint64_t cc = pack2(sc.c2, sc.c2), nl = pack2(-st.y, -st.y), A0 = pack2(a0, a0);
  const int at = min(token, p.V) + sh.shift, ag = at / kPer, el = at & (kPer - 1);
  uint4 w[kApplyGran];
#pragma unroll
  for (int j = 0; j < kApplyGran; ++j) {
    const int gj = g0 + j * kApplyThreads;
    if (on && gj >= sh.whole0 && gj < sh.whole1)
      w[j] = __ldcs(reinterpret_cast<const uint4*>(img) + gj);
  }
#pragma unroll
  for (int j = 0; j < kApplyGran; ++j) {
    const int gj = g0 + j * kApplyThreads;
    if (gj >= sh.n) break;
    const bool whole = gj >= sh.whole0 && gj < sh.whole1;
    float o[kPer];
    if (!on) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) o[k] = 0.f;
    } else if (whole) {
      granule_grad<DT, false>(w[j], st.x, cc, nl, A0, A0, o);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int v = gj * kPer + k - sh.shift;
        o[k] = 0.f;
        if (v >= 0 && v < p.V)
          o[k] = a0 * ex2(fmaf(load_logit<DT>(img, (int64_t)gj * kPer + k) - st.x, sc.c2, -st.y));
      }
    }
    if (on && gj == ag) {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (k == el) o[k] = own;
    }
    if (vec && whole) {
      store_stream(reinterpret_cast<uint4*>(dz) + gj, granule_pack<DT>(o));
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int v = gj * kPer + k - sh.shift;
        if (v >= 0 && v < p.V) store_grad<DT>(dz, (int64_t)gj * kPer + k, o[k]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The preference loss of the pairs, from the rows' log-probabilities: a block
// per pair, sums in 64 bits.  Latency only: four pairs of 128 rows each side 9 us
// alone and with cold caches.
// ---------------------------------------------------------------------------
struct PrefArgs {
  const float* lp;         // [rows]
  const int32_t* tokens;   // [rows]
  const int32_t* offsets;  // [2 pairs + 1]
  const float* ref;        // [2 pairs] or null
  int rows, pairs, average;
  double beta, smooth, margin, scale;
  float* loss;      // [1]
  float* losses;    // [pairs]
  float* seq;       // [2 pairs]
  float* g_lp;      // [rows] or null
  uint32_t* counter;
  uint32_t* status;
};

constexpr int kPrefThreads = 256;

__device__ __forceinline__ double block_sum(double v, double* buf) {
  for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kPrefThreads / 32; ++w) s += buf[w];
  return s;
}

// Block k: pair k.  m = beta ((S_c - R_c) - (S_r - R_r)) - margin,
// L = -(1 - eps) ln sigmoid(m) - eps ln sigmoid(-m), S a sequence's sum (or
// mean) of log-probabilities; every row of the pair gets dL / d log p.  The
// last block sums the losses in pair order.
__global__ void __launch_bounds__(kPrefThreads) preference_kernel(const PrefArgs p) {
  __shared__ double buf[kPrefThreads / 32];
  __shared__ int last;
  const int k = blockIdx.x, tid = threadIdx.x;
  double S[2], share[2];
  int lo[2], hi[2];
  bool bad = false;
  griddep_wait();  // the rows' log-probabilities
  for (int q = 0; q < 2; ++q) {
    const int s = k + q * p.pairs;
    const int a = p.offsets[s], b = p.offsets[s + 1];
    bad = bad || a < 0 || b < a || b > p.rows;
    lo[q] = max(0, min(a, p.rows));
    hi[q] = max(lo[q], min(b, p.rows));
    double v = 0.0, n = 0.0;
    for (int i = lo[q] + tid; i < hi[q]; i += kPrefThreads)
      if (p.tokens[i] >= 0) {
        v += (double)__ldcg(p.lp + i);
        n += 1.0;
      }
    v = block_sum(v, buf);
    n = block_sum(n, buf);
    share[q] = p.average ? 1.0 / fmax(n, 1.0) : 1.0;
    S[q] = v * share[q];
    if (tid == 0) p.seq[s] = (float)S[q];
  }
  double gap = S[0] - S[1];
  if (p.ref) gap -= (double)p.ref[k] - (double)p.ref[k + p.pairs];
  double m = p.beta * gap - p.margin;
  if (bad) m = (double)__int_as_float(0x7fc00000);
  const double soft = log1p(exp(-fabs(m)));
  // -ln sigmoid(m) = soft + max(-m, 0), kept NaN for a NaN margin
  double loss = (1.0 - p.smooth) * (soft + (m > 0.0 ? 0.0 : -m));
  if (p.smooth > 0.0) loss += p.smooth * (soft + (m < 0.0 ? 0.0 : m));
  const double dm = p.smooth / (1.0 + exp(-m)) - (1.0 - p.smooth) / (1.0 + exp(m));
  if (p.g_lp)
    for (int q = 0; q < 2; ++q) {
      const float g = (float)((q ? -dm : dm) * p.scale * p.beta * share[q]);
      for (int i = lo[q] + tid; i < hi[q]; i += kPrefThreads) p.g_lp[i] = g;
    }
  if (tid == 0) {
    p.losses[k] = (float)loss;
    if (bad) atomicOr(p.status, kScoreBadOffsets);
    const int old = atom_add_acq_rel_gpu(reinterpret_cast<int*>(p.counter), 1);
    last = old == p.pairs - 1;
    if (last) *p.counter = 0u;
  }
  __syncthreads();
  if (!last) return;
  double v = 0.0;
  for (int i = tid; i < p.pairs; i += kPrefThreads) v += (double)__ldcg(p.losses + i);
  v = block_sum(v, buf);
  if (tid == 0) *p.loss = (float)(v * p.scale);
}

}  // namespace ebk
