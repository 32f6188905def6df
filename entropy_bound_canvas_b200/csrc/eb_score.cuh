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
// clamping their exponent keeps e d = 0 where d would be -inf (a logit of
// -inf, or one whose distance to the maximum overflows).
constexpr float kDeep = 200.0f;

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

__device__ __forceinline__ RowSums row_sums_shuffle(RowSums s, int mask, float c2) {
  RowSums o;
  o.m = __shfl_xor_sync(0xffffffffu, s.m, mask);
  o.R = __shfl_xor_sync(0xffffffffu, s.R, mask);
  o.Q = __shfl_xor_sync(0xffffffffu, s.Q, mask);
  return row_sums_join(s, o, c2);
}

struct RowResult {
  float M;     // maximum over every logit
  float l2S;   // log2 S
  float lp;    // log p_a (nats)
  float H;     // entropy (nats)
  float rest;  // 1 - p_a
  float pa;    // p_a
  bool finite;
};

// s: the sums without the token; za: the token's logit (NaN: a bad token).
__device__ __forceinline__ RowResult row_result(RowSums s, float za, float c2) {
  RowResult r;
  const float M = fmaxf(s.m, za);
  const float ds = fmaxf((s.m - M) * c2, -kDeep);
  const float fs = ex2(ds);
  const float R = s.R * fs;
  const float Q = fs * fmaf(ds, s.R, s.Q);
  const float da = (za - M) * c2;
  const float ea = ex2(da);
  const float S = R + ea;
  float lnS;
  if (ea >= R) {
    const float t = log1pf(R / ea);
    lnS = fmaf(da, kLn2, t);
    r.lp = -t;
  } else {
    lnS = logf(S);
    r.lp = fmaf(da, kLn2, -lnS);
  }
  r.M = M;
  r.l2S = lnS * kLog2e;
  // e_a = 0: no entropy term, whatever d_a
  const float W = ea == 0.f ? Q : fmaf(ea, da, Q);
  r.H = fmaf(-kLn2, W / S, lnS);
  r.rest = R / S;
  r.pa = ea / S;
  r.finite = S > 0.f && S < INFINITY;
  if (!r.finite) r.lp = r.H = r.l2S = r.rest = r.pa = __int_as_float(0x7fc00000);
  return r;
}

// Per-row inputs, read once per row.
struct RowIn {
  int token;
  bool live;  // counts: token >= 0, weight not 0, inside the sequences
  bool bad;   // token >= V
  float T, c2, iT, weight;
};

__device__ __forceinline__ bool row_temp_ok(float T) { return T > 0.f && T < INFINITY; }

__device__ __forceinline__ RowIn row_in(const ScoreArgs& p, int row) {
  RowIn r;
  r.token = p.tokens[row];
  r.weight = p.weights ? p.weights[row] : 1.f;
  r.live = r.token >= 0 && r.weight != 0.f;
  if (p.offsets) r.live = r.live && row >= p.offsets[0] && row < p.offsets[p.n_off];
  r.bad = r.token >= p.V;
  r.T = p.temps ? p.temps[row] : p.temp;
  // a temperature that is not finite and positive gives a row of NaN
  if (!row_temp_ok(r.T)) r.T = __int_as_float(0x7fc00000);
  r.c2 = kLog2e / r.T;
  r.iT = 1.f / r.T;
  return r;
}

struct RowCoef {
  float g, h;  // upstream gradients of log p_a and H
};

// The policy loss of a row: its gradients, and its terms added to t.
//   L = w [ max(-A r, -A clip(r)) + k KL - c H ],  r = exp(log p_a - old),
//   KL = exp(ref - log p_a) - 1 - (ref - log p_a)
__device__ __forceinline__ RowCoef policy_row(const ScoreArgs& p, int row, const RowResult& r,
                                              float weight, double (&t)[kPolicyTerms]) {
  const double w = (double)weight * p.scale;
  const float A = p.adv[row];
  const float ratio = expf(r.lp - p.old_lp[row]);
  const float free = -A * ratio;
  // the comparisons keep a NaN ratio NaN
  const float held_ratio = ratio < p.clip_lo ? p.clip_lo : ratio > p.clip_hi ? p.clip_hi : ratio;
  const float held = -A * held_ratio;
  const bool cut = held > free;
  float kl = 0.f, dkl = 0.f;
  if (p.ref_lp) {
    const float gap = p.ref_lp[row] - r.lp;
    const float back = expm1f(gap);
    kl = back - gap;
    dkl = -back;
  }
  const float pg = cut ? held : free;
  const float H = r.H;
  t[0] += w * ((double)pg + (double)p.kl_coef * kl - (double)p.ent_coef * H);
  t[1] += w * pg;
  t[2] += w * kl;
  t[3] += w * H;
  t[4] += cut ? w : 0.0;
  RowCoef c;
  c.g = (float)(w * ((cut ? 0.0 : (double)free) + (double)p.kl_coef * dkl));
  c.h = (float)(-w * (double)p.ent_coef);
  return c;
}

// The last CTA of the grid sums the CTAs' terms in CTA order (the same order
// at every launch of one grid).  Called by one whole block, after its own
// thread 0 wrote part[blockIdx.x].
__device__ __forceinline__ void policy_total(const ScoreArgs& p, int n) {
  __shared__ int last;
  if (threadIdx.x == 0) {
    const int old = atom_add_acq_rel_gpu(reinterpret_cast<int*>(p.counter), 1);
    last = old == n - 1;
    if (last) *p.counter = 0u;
  }
  __syncthreads();
  if (!last) return;
  if (threadIdx.x < kPolicyTerms) {
    double s = 0.0;
    for (int i = 0; i < n; ++i) s += __ldcg(p.part + (size_t)i * kPolicyTerms + threadIdx.x);
    p.terms[threadIdx.x] = (float)s;
  }
}

// ---------------------------------------------------------------------------
// One block per row
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 512;

template <int DT>
__global__ void __launch_bounds__(kRowThreads)
    score_rows_kernel(const ScoreArgs p, const int mode, const bool reverse) {
  constexpr int kB = ScoreType<DT>::kBytes;
  __shared__ RowSums warp_sums[kRowThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  double t[kPolicyTerms] = {};
  for (int i = blockIdx.x; i < p.rows; i += gridDim.x) {
    const int row = reverse ? p.rows - 1 - i : i;
    const RowIn in = row_in(p, row);
    const char* z = static_cast<const char*>(p.logits) + (size_t)row * (size_t)p.ld * kB;
    char* dz = p.d_logits ? static_cast<char*>(p.d_logits) + (size_t)row * (size_t)p.ldd * kB
                          : nullptr;
    if (!in.live) {
      if (tid == 0) {
        if (p.logprobs) p.logprobs[row] = 0.f;
        if (p.entropies) p.entropies[row] = 0.f;
      }
      if (dz)
        for (int v = tid; v < p.V; v += kRowThreads) store_grad<DT>(dz, v, 0.f);
      continue;
    }
    const float za = in.bad ? __int_as_float(0x7fc00000) : load_logit<DT>(z, in.token);
    RowSums s = row_sums_empty();
    for (int v = tid; v < p.V; v += kRowThreads) {
      if (v == in.token) continue;
      const float x = load_logit<DT>(z, v);
      if (x > s.m) s = row_sums_join(s, RowSums{x, 0.f, 0.f}, in.c2);
      // a NaN logit stays NaN through the clamp's comparison
      float d = (x - s.m) * in.c2;
      d = d < -kDeep ? -kDeep : d;
      const float e = ex2(d);
      s.R += e;
      s.Q = fmaf(e, d, s.Q);
    }
    for (int k = 16; k > 0; k >>= 1) s = row_sums_shuffle(s, k, in.c2);
    __syncthreads();
    if (lane == 0) warp_sums[warp] = s;
    __syncthreads();
    s = warp_sums[lane % (kRowThreads / 32)];
    for (int k = 8; k > 0; k >>= 1) s = row_sums_shuffle(s, k, in.c2);
    const RowResult r = row_result(s, za, in.c2);
    RowCoef c{0.f, 0.f};
    if (mode == kModePolicy) {
      c = policy_row(p, row, r, in.weight, t);
    } else if (mode == kModeGrad) {
      c.g = p.g_lp[row];
      c.h = p.g_h ? p.g_h[row] : 0.f;
    }
    if (tid == 0) {
      if (p.logprobs) p.logprobs[row] = r.lp;
      if (p.entropies) p.entropies[row] = r.H;
      const uint32_t bits = (in.bad ? kScoreBadToken : 0u) | (r.finite ? 0u : kScoreNonFinite);
      if (bits) atomicOr(p.status, bits);
    }
    if (dz) {
      const float a0 = -in.iT * fmaf(c.h, r.H, c.g), a1 = -in.iT * c.h * kLn2;
      // p_a = 0: log p_a may be -inf, its entropy term is 0
      const float ha = r.pa > 0.f ? c.h * r.pa * (r.lp + r.H) : r.pa;
      const float at = in.iT * (c.g * r.rest - ha);
      const bool ent = c.h != 0.f;
      for (int v = tid; v < p.V; v += kRowThreads) {
        float d = (load_logit<DT>(z, v) - r.M) * in.c2;
        d = d < -kDeep ? -kDeep : d;
        const float x = d - r.l2S;
        const float pv = ex2(x);
        float dv = pv * (ent ? fmaf(a1, x, a0) : a0);
        if (v == in.token) dv = at;
        store_grad<DT>(dz, v, dv);
      }
    }
  }
  if (mode == kModePolicy) {
    if (tid == 0)
      for (int k = 0; k < kPolicyTerms; ++k)
        p.part[(size_t)blockIdx.x * kPolicyTerms + k] = t[k];
    policy_total(p, gridDim.x);
  }
}

// ---------------------------------------------------------------------------
// The preference loss of the pairs, from the rows' log-probabilities
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
