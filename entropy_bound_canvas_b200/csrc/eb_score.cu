// eb_score.cu -- host side of the scorer (eb_scorer_*, eb_token_logprobs*,
// eb_policy_loss, eb_preference_loss, eb_lmhead_logprobs of
// include/eb_sampler.h): validation, workspace, launches.
#include "eb_sampler.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <functional>
#include <mutex>
#include <new>

#include "eb_host.cuh"
#include "eb_lmscore.cuh"
#include "eb_score.cuh"

using ebk::DeviceGuard;
using ebk::ScoreArgs;
using ebk::align256;

namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxGrid = 8192;  // partial sums of a policy launch

// The row kernels' variants: [bf16][entropy][gradient].
constexpr int kVariants = 8;
template <int DT, bool ENT, bool GRAD>
const void* ring_fn() {
  return reinterpret_cast<const void*>(&ebk::score_ring_kernel<DT, ENT, GRAD>);
}
const void* const kRing[kVariants] = {
    ring_fn<ebk::kScoreF32, false, false>(),  ring_fn<ebk::kScoreF32, false, true>(),
    ring_fn<ebk::kScoreF32, true, false>(),   ring_fn<ebk::kScoreF32, true, true>(),
    ring_fn<ebk::kScoreBF16, false, false>(), ring_fn<ebk::kScoreBF16, false, true>(),
    ring_fn<ebk::kScoreBF16, true, false>(),  ring_fn<ebk::kScoreBF16, true, true>()};
template <int DT, bool ENT, bool GRAD, int W>
const void* short_fn() {
  return reinterpret_cast<const void*>(&ebk::score_short_kernel<DT, ENT, GRAD, W>);
}
const void* const kShort[2][kVariants] = {
    {short_fn<ebk::kScoreF32, false, false, 1>(), short_fn<ebk::kScoreF32, false, true, 1>(),
     short_fn<ebk::kScoreF32, true, false, 1>(), short_fn<ebk::kScoreF32, true, true, 1>(),
     short_fn<ebk::kScoreBF16, false, false, 1>(), short_fn<ebk::kScoreBF16, false, true, 1>(),
     short_fn<ebk::kScoreBF16, true, false, 1>(), short_fn<ebk::kScoreBF16, true, true, 1>()},
    {short_fn<ebk::kScoreF32, false, false, 4>(), short_fn<ebk::kScoreF32, false, true, 4>(),
     short_fn<ebk::kScoreF32, true, false, 4>(), short_fn<ebk::kScoreF32, true, true, 4>(),
     short_fn<ebk::kScoreBF16, false, false, 4>(), short_fn<ebk::kScoreBF16, false, true, 4>(),
     short_fn<ebk::kScoreBF16, true, false, 4>(), short_fn<ebk::kScoreBF16, true, true, 4>()}};

using ebk::kListRows;
using ebk::kRingStages;
constexpr double kListUs = 100.0;
constexpr int kMaxLog2C = 4;

struct DeviceInfo {
  std::once_flag once;
  int rc = EB_ERR_CUDA;
  int sms = 0;
  int clusters[kVariants][kMaxLog2C + 1];  // ring clusters of 2^c CTAs that fit at once
};
DeviceInfo g_info[kMaxDevices];

void ring_config(cudaLaunchConfig_t& lc, cudaLaunchAttribute& attr, int clusters, int log2C,
                 cudaStream_t st) {
  std::memset(&lc, 0, sizeof(lc));
  lc.gridDim = dim3((unsigned)clusters << log2C);
  lc.blockDim = dim3(ebk::kRingThreads);
  lc.dynamicSmemBytes = ebk::ring_layout().total;
  lc.stream = st;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 1u << log2C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  lc.attrs = &attr;
  lc.numAttrs = 1;
}

void info_setup(DeviceInfo& d, int device) {
  int sms = 0, optin = 0, major = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
      cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device) !=
          cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess) {
    cudaGetLastError();
    d.rc = EB_ERR_CUDA;
    return;
  }
  if (major != 10) {
    d.rc = EB_ERR_UNSUPPORTED;
    return;
  }
  const int lm_smem[4] = {(int)ebk::LsShape<true>::kSmem, (int)ebk::LsShape<false>::kSmem,
                          (int)ebk::FewShape<1>::kSmem, (int)ebk::FewShape<2>::kSmem};
  const void* lm_fn[4] = {reinterpret_cast<const void*>(&ebk::lmscore_kernel<true>),
                          reinterpret_cast<const void*>(&ebk::lmscore_kernel<false>),
                          reinterpret_cast<const void*>(&ebk::lmfew_kernel<1>),
                          reinterpret_cast<const void*>(&ebk::lmfew_kernel<2>)};
  for (int k = 0; k < 4; ++k) {
    if (lm_smem[k] > optin) {
      d.rc = EB_ERR_UNSUPPORTED;
      return;
    }
    if (cudaFuncSetAttribute(lm_fn[k], cudaFuncAttributeMaxDynamicSharedMemorySize, lm_smem[k]) !=
        cudaSuccess) {
      cudaGetLastError();
      d.rc = EB_ERR_CUDA;
      return;
    }
  }
  const uint32_t ring_smem = ebk::ring_layout().total;
  if (ring_smem > (uint32_t)optin) {
    d.rc = EB_ERR_UNSUPPORTED;
    return;
  }
  for (int v = 0; v < kVariants; ++v)
    if (cudaFuncSetAttribute(kRing[v], cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)ring_smem) != cudaSuccess ||
        cudaFuncSetAttribute(kRing[v], cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess) {
      cudaGetLastError();
      d.rc = EB_ERR_CUDA;
      return;
    }
  for (int v = 0; v < kVariants; ++v)
    for (int c = 0; c <= kMaxLog2C; ++c) {
      cudaLaunchConfig_t lc;
      cudaLaunchAttribute attr;
      ring_config(lc, attr, 1, c, nullptr);
      int most = 0;
      if (cudaOccupancyMaxActiveClusters(&most, kRing[v], &lc) != cudaSuccess) {
        cudaGetLastError();
        most = 0;  // this size is not used
      }
      d.clusters[v][c] = std::max(0, std::min(most, kMaxGrid));
    }
  if (d.clusters[0][0] < 1) {
    d.rc = EB_ERR_CUDA;
    return;
  }
  d.sms = sms;
  d.rc = EB_OK;
}

}  // namespace

struct eb_scorer {
  int device = 0;
  int max_rows = 0;
  int sms = 0;
  uint64_t wait_ns = ebk::kWaitLimitNs;
  void* ws = nullptr;
  size_t ws_bytes = 0;
  uint32_t* status = nullptr;
  uint32_t* counter = nullptr;
  double* part = nullptr;           // [kMaxGrid][terms]
  float* lp = nullptr;              // [max_rows] log-probabilities (preference)
  float* g = nullptr;               // [max_rows] their gradients (preference)
  float4* stats = nullptr;          // [max_rows] the rows' statistics (preference)
  ebk::LmSums* lm = nullptr;        // [lm_slots] the LM-head pass's partial sums
  float* lm_za = nullptr;           // [max_rows] the tokens' logits
  size_t lm_slots = 0;
};

namespace {

size_t elt_bytes(int dtype) { return dtype == EB_F32 ? 4 : 2; }

// Positive, normal and finite, as the fp32 that the kernels use.
bool temperature_ok(double t) { return (float)t >= FLT_MIN && std::isfinite((float)t); }

// Sizes, types and pointers every call over logits shares.
int check_input(const eb_scorer* h, const eb_score_input_t* in) {
  if (!h || !in) return EB_ERR_INVALID_ARG;
  if (in->dtype != EB_F32 && in->dtype != EB_BF16) return EB_ERR_UNSUPPORTED;
  if (in->rows < 0 || in->V < 1 || in->ld < in->V) return EB_ERR_INVALID_ARG;
  if (in->rows > h->max_rows || in->V > (1 << 30) || in->ld > (1ll << 40)) return EB_ERR_OVERFLOW;
  if (in->rows > 0 && (!in->logits || !in->tokens)) return EB_ERR_INVALID_ARG;
  if ((uintptr_t)in->logits % elt_bytes(in->dtype) != 0) return EB_ERR_INVALID_ARG;
  if (!in->temperatures && !temperature_ok(in->temperature)) return EB_ERR_INVALID_ARG;
  return EB_OK;
}

// A gradient may be written over its own logits (same address and stride).
int check_grad(const eb_score_input_t* in, const void* d_logits, int64_t ldd) {
  if (ldd < in->V) return EB_ERR_INVALID_ARG;
  if (ldd > (1ll << 40)) return EB_ERR_OVERFLOW;
  if ((uintptr_t)d_logits % elt_bytes(in->dtype) != 0) return EB_ERR_INVALID_ARG;
  if (in->rows > 1 && d_logits == in->logits && ldd != in->ld) return EB_ERR_INVALID_ARG;
  return EB_OK;
}

void fill_args(const eb_scorer* h, const eb_score_input_t* in, ScoreArgs& a) {
  std::memset(&a, 0, sizeof(a));
  a.logits = in->logits;
  a.ld = in->ld;
  a.rows = in->rows;
  a.V = in->V;
  a.tokens = in->tokens;
  a.temps = in->temperatures;
  a.temp = (float)in->temperature;
  a.part = h->part;
  a.counter = h->counter;
  a.status = h->status;
  a.wait_ns = h->wait_ns;
}

int share_stages(int64_t row_bytes, int log2C) {
  // the aligned image of a row spans up to one granule more than its bytes
  const int64_t G = (row_bytes + 15) / 16 + 1;
  const int64_t per = (((G + (1ll << log2C) - 1) >> log2C) + 7) / 8 * 8;
  return (int)std::min<int64_t>((per + ebk::kStageGran - 1) / ebk::kStageGran, 1 << 20);
}

// The cluster size of a ring launch.  A row on 2^c CTAs costs a CTA its share
// of the row at the CTA's rate, and one to two microseconds for the exchange;
// rows go in waves of the clusters that fit.  More CTAs per row shorten the
// last, partly filled wave and (with a gradient, whose second look at a row
// should find it in L2) keep fewer rows in flight; fewer pay the exchange less
// often.  The rates are what one CTA was measured to take, in KB/us: alone on
// its SM, and with every SM holding two; the other constants were fitted to
// 22 shapes of 100 to 2048 rows on one to eight CTAs each, where the size
// taken is within 2 % of the best on average and 8 % at most.  262144 bf16:
// one row, forward, 22.6 us on one CTA and 5.5 on 16; a policy step of 2048 rows
// 489 us on one CTA each, 411 on two, 438 on four, 534 on eight; of 2048 rows of
// 16000, 52 on one, 61 on two, 80 on four.
int ring_log2C(const eb_scorer* h, int variant, bool f32, bool grad, int64_t rows,
               int64_t row_bytes, double& best_t) {
  const double alone = (grad ? 12.0 : 26.0) * (f32 ? 1.4 : 1.0);
  const double full = (grad ? 9.3 : 18.0) * (f32 ? 1.25 : 1.0);
  const double kb = (double)row_bytes / 1024.0;
  int best = 0;
  best_t = 0.0;
  for (int c = 0; c <= kMaxLog2C; ++c) {
    const int n = g_info[h->device].clusters[variant][c];
    if (n < 1) break;
    const double share = kb / (1 << c), fixed = grad ? 1.2 + 0.3 * c : 1.1 + 0.1 * c;
    // the part of a share that the ring does not keep is copied again, from
    // L2, or from HBM where the rows in flight ask for more than L2 keeps
    double again = 1.0;
    const int stages = share_stages(row_bytes, c);
    if (grad && stages > kRingStages) {
      const double part = 1.0 - (double)kRingStages / stages;
      const double asked = (double)std::min<int64_t>(n, rows) * kb / 1024.0 * part;
      const double over = std::min(1.0, std::max(0.0, (asked - 40.0) / 60.0));
      again = 1.0 + part * (0.1 + 0.5 * over);
    }
    const int64_t waves = rows / n, left = rows - waves * n;
    double t = (double)waves * (fixed + share / full * again);
    if (left > 0) {
      const double ctas = (double)(left << c);
      const double crowd = std::min(1.0, std::max(0.0, (ctas - h->sms) / (double)h->sms));
      t += fixed + share / (alone + (full - alone) * crowd) * again;
    }
    if (c == 0 || t < best_t) {
      best = c;
      best_t = t;
    }
  }
  return best;
}

int launch_rows(const eb_scorer* h, const ScoreArgs& a, int dtype, int mode, bool ent, bool grad,
                cudaStream_t st) {
  const int v = (dtype == EB_BF16 ? 4 : 0) + (ent ? 2 : 0) + (grad ? 1 : 0);
  const int64_t row_bytes = (int64_t)a.V * (int64_t)elt_bytes(dtype);
  // the aligned image of a row holds a granule more where rows start off 16 bytes
  const bool even = (uintptr_t)a.logits % 16 == 0 && (a.ld * (int64_t)elt_bytes(dtype)) % 16 == 0;
  const int64_t image = (row_bytes + 15) / 16 * 16 + (even ? 0 : 16);
  if (image <= ebk::short_bytes(4)) {
    // four warps to a row also where one would do but every row has its SM's
    // attention anyway (16 rows of 1024 fp32: 2.1 us against 2.8; 2000: 6.8
    // against 4.6)
    const int wide = image > ebk::short_bytes(1) || (image > 1024 && a.rows <= 4 * h->sms);
    const int per_block = wide ? 1 : 4;
    const int blocks = (int)std::min<int64_t>(((int64_t)a.rows + per_block - 1) / per_block,
                                              (int64_t)h->sms * (grad ? 6 : 8));
    int m = mode;
    void* args[] = {const_cast<ScoreArgs*>(&a), &m};
    return cudaLaunchKernel(kShort[wide][v], dim3(std::max(1, blocks)), dim3(ebk::kShortThreads),
                            args, 0, st) == cudaSuccess
               ? EB_OK
               : EB_ERR_CUDA;
  }
  double us;
  const int c = ring_log2C(h, v, dtype == EB_F32, grad, a.rows, row_bytes, us);
  const int most = g_info[h->device].clusters[v][c];
  if (most < 1) return EB_ERR_CUDA;
  ebk::RingArgs q;
  q.mode = mode;
  q.log2C = c;
  q.ahead = 2 * share_stages(row_bytes, c) <= kRingStages;
  // Rows shared out by lists: where a cluster takes more than two, and the launch
  // is long enough for the counting (a policy step of 2048 rows of 262144 bf16:
  // none ignored 413 us against 408, 128 scattered ones 393 against 402, 512
  // 351 against 396; 1000 rows, scores, none ignored: 104 against 101).
  const int clusters = std::max(1, std::min(a.rows, most));
  q.listed = a.rows > 2 * clusters && us > kListUs && a.rows <= (kListRows - 2) * clusters;
  cudaLaunchConfig_t lc;
  cudaLaunchAttribute attr;
  ring_config(lc, attr, clusters, c, st);
  void* args[] = {const_cast<ScoreArgs*>(&a), &q};
  return cudaLaunchKernelExC(&lc, kRing[v], args) == cudaSuccess ? EB_OK : EB_ERR_CUDA;
}

}  // namespace

extern "C" {

int eb_scorer_init(eb_scorer_t** out, int32_t max_rows, int device) {
  if (!out) return EB_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_rows < 1) return EB_ERR_INVALID_ARG;
  if (max_rows > EB_MAX_SCORE_ROWS) return EB_ERR_OVERFLOW;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess) return EB_ERR_CUDA;
  if (device < 0 || device >= ndev) return EB_ERR_INVALID_ARG;
  if (device >= kMaxDevices) return EB_ERR_UNSUPPORTED;
  DeviceGuard guard(device);
  if (!guard.ok) return EB_ERR_CUDA;
  DeviceInfo& d = g_info[device];
  std::call_once(d.once, info_setup, std::ref(d), device);
  if (d.rc != EB_OK) return d.rc;

  eb_scorer* h = new (std::nothrow) eb_scorer();
  if (!h) return EB_ERR_OUT_OF_MEMORY;
  h->device = device;
  h->max_rows = max_rows;
  h->sms = d.sms;
  h->lm_slots = ebk::lm_score_slots(d.sms, max_rows);
  size_t off = 0;
  const size_t o_status = off;
  off = align256(off + 2 * sizeof(uint32_t));
  const size_t o_part = off;
  off = align256(off + sizeof(double) * kMaxGrid * ebk::kPolicyTerms);
  const size_t o_lp = off;
  off = align256(off + sizeof(float) * (size_t)max_rows);
  const size_t o_g = off;
  off = align256(off + sizeof(float) * (size_t)max_rows);
  const size_t o_stats = off;
  off = align256(off + sizeof(float4) * (size_t)max_rows);
  const size_t o_lm = off;
  off = align256(off + sizeof(ebk::LmSums) * h->lm_slots);
  const size_t o_za = off;
  off = align256(off + sizeof(float) * (size_t)max_rows);
  h->ws_bytes = off;
  if (cudaMalloc(&h->ws, h->ws_bytes) != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return EB_ERR_OUT_OF_MEMORY;
  }
  if (!ebk::clear_now(h->ws, h->ws_bytes)) {
    cudaFree(h->ws);
    delete h;
    return EB_ERR_CUDA;
  }
  char* base = static_cast<char*>(h->ws);
  h->status = reinterpret_cast<uint32_t*>(base + o_status);
  h->counter = h->status + 1;
  h->part = reinterpret_cast<double*>(base + o_part);
  h->lp = reinterpret_cast<float*>(base + o_lp);
  h->g = reinterpret_cast<float*>(base + o_g);
  h->stats = reinterpret_cast<float4*>(base + o_stats);
  h->lm = reinterpret_cast<ebk::LmSums*>(base + o_lm);
  h->lm_za = reinterpret_cast<float*>(base + o_za);
  *out = h;
  return EB_OK;
}

int eb_token_logprobs(eb_scorer_t* h, const eb_score_input_t* in, float* logprobs,
                      float* entropies, void* stream) {
  int rc = check_input(h, in);
  if (rc != EB_OK) return rc;
  if (in->rows == 0) return EB_OK;
  if (!logprobs) return EB_ERR_INVALID_ARG;
  DeviceGuard guard(h->device);
  if (!guard.ok) return EB_ERR_CUDA;
  ScoreArgs a;
  fill_args(h, in, a);
  a.logprobs = logprobs;
  a.entropies = entropies;
  return launch_rows(h, a, in->dtype, ebk::kModeScore, entropies != nullptr, false,
                     (cudaStream_t)stream);
}

int eb_token_logprobs_backward(eb_scorer_t* h, const eb_score_input_t* in,
                               const float* d_logprobs, const float* d_entropies, void* d_logits,
                               int64_t ldd, void* stream) {
  int rc = check_input(h, in);
  if (rc != EB_OK) return rc;
  if ((rc = check_grad(in, d_logits, ldd)) != EB_OK) return rc;
  if (in->rows == 0) return EB_OK;
  if (!d_logprobs || !d_logits) return EB_ERR_INVALID_ARG;
  DeviceGuard guard(h->device);
  if (!guard.ok) return EB_ERR_CUDA;
  ScoreArgs a;
  fill_args(h, in, a);
  a.d_logits = d_logits;
  a.ldd = ldd;
  a.g_lp = d_logprobs;
  a.g_h = d_entropies;
  return launch_rows(h, a, in->dtype, ebk::kModeGrad, d_entropies != nullptr, true,
                     (cudaStream_t)stream);
}

int eb_policy_loss(eb_scorer_t* h, const eb_score_input_t* in, const eb_policy_t* p, float* terms,
                   float* logprobs, float* entropies, void* d_logits, int64_t ldd, void* stream) {
  int rc = check_input(h, in);
  if (rc != EB_OK) return rc;
  if (!p || !terms) return EB_ERR_INVALID_ARG;
  if (!(p->clip_low >= 0.0 && p->clip_low <= 1.0) || !(p->clip_high >= 0.0) ||
      !std::isfinite((float)p->clip_high) || !std::isfinite((float)p->kl_coef) ||
      !std::isfinite((float)p->entropy_coef) || !std::isfinite(p->scale))
    return EB_ERR_INVALID_ARG;
  if (p->kl_coef != 0.0 && !p->ref_logprobs && in->rows > 0) return EB_ERR_INVALID_ARG;
  if (in->rows > 0 && (!p->old_logprobs || !p->advantages)) return EB_ERR_INVALID_ARG;
  if (d_logits && (rc = check_grad(in, d_logits, ldd)) != EB_OK) return rc;
  DeviceGuard guard(h->device);
  if (!guard.ok) return EB_ERR_CUDA;
  ScoreArgs a;
  fill_args(h, in, a);
  a.logprobs = logprobs;
  a.entropies = entropies;
  a.d_logits = d_logits;
  a.ldd = ldd;
  a.old_lp = p->old_logprobs;
  a.ref_lp = p->ref_logprobs;
  a.adv = p->advantages;
  a.weights = p->weights;
  a.clip_lo = (float)(1.0 - p->clip_low);
  a.clip_hi = (float)(1.0 + p->clip_high);
  a.kl_coef = (float)p->kl_coef;
  a.ent_coef = (float)p->entropy_coef;
  a.scale = p->scale;
  a.terms = terms;
  return launch_rows(h, a, in->dtype, ebk::kModePolicy, true, d_logits != nullptr,
                     (cudaStream_t)stream);
}

int eb_preference_loss(eb_scorer_t* h, const eb_score_input_t* in, const eb_preference_t* p,
                       float* loss, float* losses, float* sequence_logprobs, float* logprobs,
                       void* d_logits, int64_t ldd, void* stream) {
  int rc = check_input(h, in);
  if (rc != EB_OK) return rc;
  if (!p || !loss || p->pairs < 0) return EB_ERR_INVALID_ARG;
  if (p->pairs > EB_MAX_SCORE_ROWS) return EB_ERR_OVERFLOW;
  if (!(p->beta >= 0.0) || !std::isfinite(p->beta) ||
      !(p->label_smoothing >= 0.0 && p->label_smoothing < 1.0) || !std::isfinite(p->margin) ||
      !std::isfinite(p->scale) || (p->average != 0 && p->average != 1))
    return EB_ERR_INVALID_ARG;
  if (!p->offsets || (p->pairs > 0 && (!losses || !sequence_logprobs))) return EB_ERR_INVALID_ARG;
  if (d_logits && (rc = check_grad(in, d_logits, ldd)) != EB_OK) return rc;
  DeviceGuard guard(h->device);
  if (!guard.ok) return EB_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  ScoreArgs a;
  fill_args(h, in, a);
  a.offsets = p->offsets;
  a.n_off = 2 * p->pairs;
  a.logprobs = logprobs ? logprobs : h->lp;
  // the gradient's blocks, 32 KB of a row's aligned image each
  constexpr int kBlock = ebk::kApplyThreads * ebk::kApplyGran * 16;
  const int64_t image = (int64_t)in->V * (int64_t)elt_bytes(in->dtype) + 16;
  int tiles = (int)((image + kBlock - 1) / kBlock);
  if (d_logits && (int64_t)in->rows * tiles > 0x7fffffffll) return EB_ERR_OVERFLOW;
  a.stats = d_logits ? h->stats : nullptr;
  if (in->rows > 0 &&
      (rc = launch_rows(h, a, in->dtype, ebk::kModeScore, false, false, st)) != EB_OK)
    return rc;
  if (p->pairs == 0) {
    if (cudaMemsetAsync(loss, 0, sizeof(float), st) != cudaSuccess) return EB_ERR_CUDA;
  } else {
    ebk::PrefArgs q;
    q.lp = a.logprobs;
    q.tokens = in->tokens;
    q.offsets = p->offsets;
    q.ref = p->ref_logprobs;
    q.rows = in->rows;
    q.pairs = p->pairs;
    q.average = p->average;
    q.beta = p->beta;
    q.smooth = p->label_smoothing;
    q.margin = p->margin;
    q.scale = p->scale;
    q.loss = loss;
    q.losses = losses;
    q.seq = sequence_logprobs;
    q.g_lp = d_logits ? h->g : nullptr;
    q.counter = h->counter;
    q.status = h->status;
    void* args[] = {&q};
    if (!ebk::launch_dependent(reinterpret_cast<const void*>(&ebk::preference_kernel),
                               dim3(p->pairs), dim3(ebk::kPrefThreads), 0, args, st))
      return EB_ERR_CUDA;
  }
  if (!d_logits || in->rows == 0) return EB_OK;
  a.logprobs = nullptr;
  a.d_logits = d_logits;
  a.ldd = ldd;
  a.g_lp = h->g;
  void* args[] = {&a, &tiles};
  const void* fn = in->dtype == EB_F32
                       ? reinterpret_cast<const void*>(&ebk::score_apply_kernel<ebk::kScoreF32>)
                       : reinterpret_cast<const void*>(&ebk::score_apply_kernel<ebk::kScoreBF16>);
  return ebk::launch_dependent(fn, dim3((unsigned)in->rows * (unsigned)tiles),
                               dim3(ebk::kApplyThreads), 0, args, st)
             ? EB_OK
             : EB_ERR_CUDA;
}

int eb_lmhead_logprobs(eb_scorer_t* h, const void* hidden, const void* weight, int32_t rows,
                       int32_t V, int32_t d, const int32_t* tokens, const float* temperatures,
                       double temperature, float* logprobs, float* entropies, void* stream) {
  if (!h || rows < 0 || V < 1 || d < 1) return EB_ERR_INVALID_ARG;
  if (d % 8 != 0) return EB_ERR_UNSUPPORTED;
  if (rows > h->max_rows || V > (1 << 30) || d > (1 << 20)) return EB_ERR_OVERFLOW;
  if (!temperatures && !temperature_ok(temperature)) return EB_ERR_INVALID_ARG;
  if (rows == 0) return EB_OK;
  if (!hidden || !weight || !tokens || !logprobs) return EB_ERR_INVALID_ARG;
  if ((uintptr_t)hidden % 16 != 0 || (uintptr_t)weight % 16 != 0) return EB_ERR_INVALID_ARG;
  DeviceGuard guard(h->device);
  if (!guard.ok) return EB_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  ebk::LmScoreArgs p;
  std::memset(&p, 0, sizeof(p));
  p.tokens = tokens;
  p.temps = temperatures;
  p.temp = (float)temperature;
  p.sums = h->lm;
  p.za = h->lm_za;
  p.rows = rows;
  p.V = V;
  p.d = d;
  p.wait_ns = h->wait_ns;
  p.status = h->status;
  p.logprobs = logprobs;
  p.entropies = entropies;
  // An odd number of 128-row tiles leaves half of the last pair's work padding;
  // single CTAs take longer for the same tiles, so they win up to 9 tiles.  Single
  // CTAs against pairs, us:
  //   ids, d           100 rows  300        600        1100         1400
  //   32003, 256       17 / 18   21 / 23    26 / 29    34 / 37      39 / 41
  //   32003, 2560      39 / 48   70 / 76    101 / 107  163 / 167    204 / 199
  //   131072, 1024     60 / 69   105 / 115  152 / 162  275 / 281    344 / 324
  //   262144, 2560     220 / 264 484 / 568  808 / 825  1358 / 1330  1678 / 1575
  // (2000 ids, where one launch's latency is most of it: within 2 us.)
  const int tiles = (rows + ebk::kLsRows - 1) / ebk::kLsRows;
  const bool few = rows <= ebk::kLfRows, pair = tiles % 2 == 0 || tiles > 9;
  if (few) {
    p.n_split = std::min(h->sms, (V + 127) / 128);
    p.n_rec = p.n_split;
  } else {
    p.n_split = pair ? ebk::lm_score_split<true>(h->sms, rows, V)
                     : ebk::lm_score_split<false>(h->sms, rows, V);
    p.n_rec = 2 * p.n_split;
  }
  if ((size_t)p.n_rec * (size_t)rows > h->lm_slots) return EB_ERR_OVERFLOW;
  const bool wide = rows > 32;  // of the few: 64 columns
  CUtensorMap th, tw;
  if (!ebk::make_tmap(&th, hidden, (uint64_t)d, (uint64_t)rows, ebk::kLsBK,
                      !few ? ebk::kLsRows : wide ? 64 : 32) ||
      !ebk::make_tmap(&tw, weight, (uint64_t)d, (uint64_t)V, ebk::kLsBK, 128))
    return EB_ERR_CUDA;
  if (!few && pair) {
    ebk::lmscore_kernel<true><<<(tiles + 1) / 2 * 2 * p.n_split, ebk::kLsThreads,
                                ebk::LsShape<true>::kSmem, st>>>(th, tw, p);
  } else if (!few) {
    ebk::lmscore_kernel<false><<<tiles * p.n_split, ebk::kLsThreads, ebk::LsShape<false>::kSmem,
                                 st>>>(th, tw, p);
  } else if (wide) {
    ebk::lmfew_kernel<2><<<p.n_split, ebk::FewShape<2>::kThreads, ebk::FewShape<2>::kSmem, st>>>(
        th, tw, p);
  } else {
    ebk::lmfew_kernel<1><<<p.n_split, ebk::FewShape<1>::kThreads, ebk::FewShape<1>::kSmem, st>>>(
        th, tw, p);
  }
  if (cudaGetLastError() != cudaSuccess) return EB_ERR_CUDA;
  void* args[] = {&p};
  return ebk::launch_dependent(reinterpret_cast<const void*>(&ebk::lmscore_finish_kernel),
                               dim3((rows + 3) / 4), dim3(128), 0, args, st)
             ? EB_OK
             : EB_ERR_CUDA;
}

int eb_scorer_status(eb_scorer_t* h, uint32_t* status, int clear, void* stream) {
  if (!h || !status) return EB_ERR_INVALID_ARG;
  DeviceGuard guard(h->device);
  if (!guard.ok) return EB_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  if (cudaMemcpyAsync(status, h->status, sizeof(uint32_t), cudaMemcpyDeviceToHost, st) !=
      cudaSuccess)
    return EB_ERR_CUDA;
  if (clear && cudaMemsetAsync(h->status, 0, sizeof(uint32_t), st) != cudaSuccess)
    return EB_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return EB_ERR_CUDA;
  return EB_OK;
}

int eb_scorer_set_wait_limit(eb_scorer_t* h, uint64_t limit_ns) {
  if (!h) return EB_ERR_INVALID_ARG;
  h->wait_ns = limit_ns == 0 ? ebk::kWaitLimitNs : limit_ns;
  return EB_OK;
}

size_t eb_scorer_workspace_bytes(const eb_scorer_t* h) { return h ? h->ws_bytes : 0; }

void eb_scorer_destroy(eb_scorer_t* h) {
  if (!h) return;
  {
    DeviceGuard guard(h->device);
    if (h->ws) cudaFree(h->ws);
  }
  delete h;
}

}  // extern "C"
