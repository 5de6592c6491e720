// MI355X (gfx950) training on drafted blocks: the log-probabilities of a
// block's tokens under the corrected logits, the clipped policy loss with a KL
// term, and the gradients of the base logits, w1 and w2.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "markov.h"
#include "numbers.h"

namespace {

constexpr float LOG2E = 1.44269504088896341f;
constexpr float LN2 = 0.69314718055994531f;

// What the scoring kernels take. Row-step m = r * k + s.
struct ScoreArgs {
  const uint16_t* base;       // [M][V]
  const uint16_t* w1;         // [V][R]
  const uint16_t* w2;         // [V][R]
  const int64_t* prev;        // [rows]
  const int64_t* tokens;      // [M]
  const int32_t* lengths;     // [rows] or null
  const float* temperature;   // [rows] or null
  float* logprobs;            // [M]
  float* lse;                 // [M]
  const float* grad;          // [M]
  uint16_t* grad_base;        // [M][V]
  uint16_t* grad_w1;          // [V][R]
  uint16_t* grad_w2;          // [V][R]
  float* grad_emb;            // [M][R]
  int M, k, V, R;
  float mult, cap, inv_cap;
};

__device__ __forceinline__ bool scored(const int64_t* tokens, const int32_t* lengths, int m, int k,
                                       int V) {
  const int r = m / k, s = m - r * k;
  const int64_t t = tokens[m];
  return (!lengths || s < lengths[r]) && t >= 0 && t < V;
}

// The w1 row that feeds row-step m: the loop's clamp, as unsigned.
__device__ __forceinline__ int fed_row(const ScoreArgs& a, int m) {
  const int r = m / a.k;
  const uint64_t t = (uint64_t)(m == r * a.k ? a.prev[r] : a.tokens[m - 1]);
  return (int)(t < (uint64_t)a.V ? t : (uint64_t)(a.V - 1));
}

__device__ __forceinline__ float inverse_temperature(const ScoreArgs& a, int m) {
  const float T = a.temperature ? a.temperature[m / a.k] : 1.0f;
  return T == 0.0f ? 1.0f : 1.0f / T;
}

// z of x, and dz/dx. With e = exp(-2|y|): tanh = (1 - e)/(1 + e) and its
// slope 4e/(1 + e)^2, neither of which cancels.
__device__ __forceinline__ float transform(float x, float mult, float cap, float inv_cap, float* slope) {
  if (!(cap > 0.0f)) {
    *slope = mult;
    return mult * x;
  }
  const float y = mult * x * inv_cap;
  const float e = __builtin_amdgcn_exp2f(-2.0f * LOG2E * fabsf(y));
  const float q = 1.0f / (1.0f + e);
  *slope = mult * 4.0f * e * q * q;
  return cap * __builtin_copysignf((1.0f - e) * q, y);
}

__device__ __forceinline__ float logit(const ScoreArgs& a, int m, int v, const uint16_t* emb, float* slope) {
  float dot = 0.0f;
  for (int j = 0; j < a.R; ++j) dot += bf_one(emb[j]) * bf_one(a.w2[(size_t)v * a.R + j]);
  return transform(bf_one(a.base[(size_t)m * a.V + v]) + dot, a.mult, a.cap, a.inv_cap, slope);
}

// (m, s) += (m2, s2) of a running log2-domain maximum and sum.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float at = top == -INFINITY ? 0.0f : top;
  s = s * __builtin_amdgcn_exp2f(m - at) + s2 * __builtin_amdgcn_exp2f(m2 - at);
  m = top;
}

// One workgroup per row-step.
__global__ __launch_bounds__(256) void score_kernel(ScoreArgs a) {
  const int m = blockIdx.x, tid = threadIdx.x;
  __shared__ float sm[256], ss[256];
  __shared__ float su;
  if (!scored(a.tokens, a.lengths, m, a.k, a.V)) {
    if (tid == 0) a.logprobs[m] = a.lse[m] = 0.0f;
    return;
  }
  const uint16_t* emb = a.w1 + (size_t)fed_row(a, m) * a.R;
  const float c = inverse_temperature(a, m) * LOG2E;
  const int t = (int)a.tokens[m];
  float mx = -INFINITY, sum = 0.0f;
  for (int v = tid; v < a.V; v += 256) {
    float slope;
    const float u = logit(a, m, v, emb, &slope) * c;
    if (v == t) su = u;
    join(mx, sum, u, u == -INFINITY ? 0.0f : 1.0f);
  }
  sm[tid] = mx;
  ss[tid] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < 256; ++i) join(mx, sum, sm[i], ss[i]);
    const float l2 = mx + __log2f(sum);
    a.lse[m] = l2 * LN2;
    a.logprobs[m] = su == -INFINITY ? -INFINITY : (su - l2) * LN2;
  }
}

// ---------------------------------------------------------------- the loss

// One workgroup: N first, then the terms; sums in binary64 in a fixed order.
constexpr int LT = 1024;

__device__ double block_sum(double v, double* red) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int sh = 32; sh >= 1; sh >>= 1) v += __shfl_xor(v, sh);
  __syncthreads();
  if (lane == 0) red[wave] = v;
  __syncthreads();
  double t = 0.0;
  for (int w = 0; w < LT / 64; ++w) t += red[w];
  return t;
}

__global__ __launch_bounds__(LT) void policy_loss_kernel(
    const float* logprobs, const float* old, const float* ref, const float* advantages,
    const int64_t* tokens, const int32_t* lengths, int M, int k, int V, float clip_low,
    float clip_high, float beta, float* stats, float* grad) {
  __shared__ double red[LT / 64];
  const int tid = threadIdx.x;
  int mine = 0;
  for (int m = tid; m < M; m += LT) mine += scored(tokens, lengths, m, k, V);
  const double n = block_sum((double)mine, red);
  const double inv = n > 0.0 ? 1.0 / n : 0.0;
  const double low = 1.0 - (double)clip_low, high = 1.0 + (double)clip_high, b = (double)beta;
  double s0 = 0.0, s1 = 0.0;
  int held_n = 0;
  for (int m = tid; m < M; m += LT) {
    if (!scored(tokens, lengths, m, k, V)) {
      grad[m] = 0.0f;
      continue;
    }
    const double lp = (double)logprobs[m], adv = (double)advantages[m];
    // (an advantage of 0 takes ratio 0: an infinite one would make NaN of it)
    const double ratio = adv == 0.0 ? 0.0 : exp(lp - (double)old[m]);
    const double held = (ratio < low ? low : ratio > high ? high : ratio) * adv;   // 0 where adv is
    const double open = ratio * adv;
    const bool clipped = held < open;
    double g = clipped ? 0.0 : -open;
    s0 += clipped ? held : open;
    held_n += clipped;
    if (b != 0.0 || ref) {
      const double gap = (double)ref[m] - lp, e = expm1(gap);
      s1 += e - gap;
      if (b != 0.0) g -= b * e;
    }
    grad[m] = (float)(g * inv);
  }
  const double surrogate = block_sum(s0, red) * inv;
  const double kl = block_sum(s1, red) * inv;
  const double share = block_sum((double)held_n, red) * inv;
  if (tid == 0) {
    stats[0] = (float)((b != 0.0 ? b * kl : 0.0) - surrogate);
    stats[1] = (float)surrogate;
    stats[2] = (float)kl;
    stats[3] = (float)share;
  }
}

// ---------------------------------------------------------------- the gradients

// grid (ceil(V/256), M): d of one element per thread.
__global__ __launch_bounds__(256) void grad_base_kernel(ScoreArgs a) {
  const int m = blockIdx.y, v = blockIdx.x * 256 + threadIdx.x;
  if (v >= a.V) return;
  float d = 0.0f;
  const float g = a.grad[m];
  if (scored(a.tokens, a.lengths, m, a.k, a.V) && g != 0.0f) {
    const float it = inverse_temperature(a, m);
    float slope;
    const float z = logit(a, m, v, a.w1 + (size_t)fed_row(a, m) * a.R, &slope);
    const float u = z * it * LOG2E;
    const float p = __builtin_amdgcn_exp2f(u - a.lse[m] * LOG2E);
    d = u == -INFINITY ? 0.0f : g * ((v == (int)a.tokens[m] ? 1.0f : 0.0f) - p) * it * slope;
  }
  a.grad_base[(size_t)m * a.V + v] = (uint16_t)pack_bf16(d, 0.0f);
}

// grid V, R threads: grad_w2[v].
__global__ void grad_w2_kernel(ScoreArgs a) {
  const int v = blockIdx.x, j = threadIdx.x;
  float sum = 0.0f;
  for (int m = 0; m < a.M; ++m)
    sum += bf_one(a.grad_base[(size_t)m * a.V + v]) * bf_one(a.w1[(size_t)fed_row(a, m) * a.R + j]);
  a.grad_w2[(size_t)v * a.R + j] = (uint16_t)pack_bf16(sum, 0.0f);
  a.grad_w1[(size_t)v * a.R + j] = 0;
}

// grid M, R threads: the gradient of row-step m's embedding.
__global__ void grad_emb_kernel(ScoreArgs a) {
  const int m = blockIdx.x, j = threadIdx.x;
  float sum = 0.0f;
  for (int v = 0; v < a.V; ++v)
    sum += bf_one(a.grad_base[(size_t)m * a.V + v]) * bf_one(a.w2[(size_t)v * a.R + j]);
  a.grad_emb[(size_t)m * a.R + j] = sum;
}

// grid M, R threads: the first row-step of those fed by one token adds them
// up, in rising row-step.
__global__ void grad_w1_kernel(ScoreArgs a) {
  const int m = blockIdx.x, j = threadIdx.x;
  const int row = fed_row(a, m);
  float sum = 0.0f;
  for (int i = 0; i < a.M; ++i) {
    if (fed_row(a, i) != row) continue;
    if (i < m) return;
    sum += a.grad_emb[(size_t)i * a.R + j];
  }
  a.grad_w1[(size_t)row * a.R + j] = (uint16_t)pack_bf16(sum, 0.0f);
}

// ---------------------------------------------------------------- host side

int check(const markov_shape_t* sh, int32_t k) {
  if (!sh) return MARKOV_ERR_NULL;
  if (sh->vocab > MARKOV_MAX_VOCAB) return MARKOV_ERR_VOCAB;
  if (sh->rows < 1 || k < 1 || sh->vocab < 8 || (sh->vocab & 7)) return MARKOV_ERR_SHAPE;
  if (sh->rank < 16 || sh->rank > 512 || (sh->rank & (sh->rank - 1))) return MARKOV_ERR_RANK;
  if ((int64_t)sh->rows * k > MARKOV_MAX_TOKENS) return MARKOV_ERR_ROWS;
  return MARKOV_OK;
}

ScoreArgs arguments(const void* base, const void* w1, const void* w2, const int64_t* prev,
                    const int64_t* tokens, const int32_t* lengths, int32_t k,
                    const float* temperature, const markov_shape_t* sh) {
  ScoreArgs a = {};
  a.base = (const uint16_t*)base;
  a.w1 = (const uint16_t*)w1;
  a.w2 = (const uint16_t*)w2;
  a.prev = prev;
  a.tokens = tokens;
  a.lengths = lengths;
  a.temperature = temperature;
  a.M = sh->rows * k;
  a.k = k;
  a.V = sh->vocab;
  a.R = sh->rank;
  a.mult = sh->mult;
  a.cap = sh->softcap > 0.0f ? sh->softcap : 0.0f;
  a.inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f;
  return a;
}

}  // namespace

extern "C" {

size_t markov_score_workspace_bytes(const markov_shape_t* shape, int32_t k) {
  if (check(shape, k)) return 0;
  return (size_t)shape->rows * k * shape->rank * 4;
}

int markov_score_sequential(const void* base_logits, const void* w1, const void* w2,
                            const int64_t* prev, const int64_t* tokens, const int32_t* lengths,
                            int32_t k, const float* temperature, float* logprobs, float* lse,
                            markov_stream_t stream, const markov_shape_t* shape, void* workspace,
                            size_t workspace_bytes) {
  const int rc = check(shape, k);
  if (rc) return rc;
  if (!base_logits || !w1 || !w2 || !prev || !tokens || !logprobs || !lse || !workspace)
    return MARKOV_ERR_NULL;
  if (!aligned_to(base_logits, 16) || !aligned_to(w1, 16) || !aligned_to(w2, 16) ||
      !aligned_to(workspace, 16))
    return MARKOV_ERR_ALIGN;
  if (workspace_bytes < markov_score_workspace_bytes(shape, k)) return MARKOV_ERR_WORKSPACE;
  ScoreArgs a = arguments(base_logits, w1, w2, prev, tokens, lengths, k, temperature, shape);
  a.logprobs = logprobs;
  a.lse = lse;
  score_kernel<<<dim3((unsigned)a.M), 256, 0, (hipStream_t)stream>>>(a);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

int markov_policy_loss(const float* logprobs, const float* old_logprobs, const float* ref_logprobs,
                       const float* advantages, const int64_t* tokens, const int32_t* lengths,
                       int32_t k, float clip_low, float clip_high, float beta, float* stats,
                       float* grad_logprobs, markov_stream_t stream, const markov_shape_t* shape) {
  const int rc = check(shape, k);
  if (rc) return rc;
  if (!logprobs || !old_logprobs || !advantages || !tokens || !stats || !grad_logprobs ||
      (!ref_logprobs && beta != 0.0f))
    return MARKOV_ERR_NULL;
  if (!(clip_low >= 0.0f) || !(clip_high >= 0.0f) || !isfinite(beta)) return MARKOV_ERR_VALUE;
  policy_loss_kernel<<<1, LT, 0, (hipStream_t)stream>>>(
      logprobs, old_logprobs, ref_logprobs, advantages, tokens, lengths, shape->rows * k, k,
      shape->vocab, clip_low, clip_high, beta, stats, grad_logprobs);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

int markov_score_backward(const void* base_logits, const void* w1, const void* w2,
                          const int64_t* prev, const int64_t* tokens, const int32_t* lengths,
                          int32_t k, const float* temperature, const float* lse,
                          const float* grad_logprobs, void* grad_base, void* grad_w1,
                          void* grad_w2, markov_stream_t stream, const markov_shape_t* shape,
                          void* workspace, size_t workspace_bytes) {
  const int rc = check(shape, k);
  if (rc) return rc;
  if (!base_logits || !w1 || !w2 || !prev || !tokens || !lse || !grad_logprobs || !grad_base ||
      !grad_w1 || !grad_w2 || !workspace)
    return MARKOV_ERR_NULL;
  if (!aligned_to(base_logits, 16) || !aligned_to(w1, 16) || !aligned_to(w2, 16) ||
      !aligned_to(grad_base, 16) || !aligned_to(grad_w1, 16) || !aligned_to(grad_w2, 16) ||
      !aligned_to(workspace, 16))
    return MARKOV_ERR_ALIGN;
  if (workspace_bytes < markov_score_workspace_bytes(shape, k)) return MARKOV_ERR_WORKSPACE;
  ScoreArgs a = arguments(base_logits, w1, w2, prev, tokens, lengths, k, temperature, shape);
  a.lse = (float*)lse;
  a.grad = grad_logprobs;
  a.grad_base = (uint16_t*)grad_base;
  a.grad_w1 = (uint16_t*)grad_w1;
  a.grad_w2 = (uint16_t*)grad_w2;
  a.grad_emb = (float*)workspace;
  const hipStream_t st = (hipStream_t)stream;
  grad_base_kernel<<<dim3((unsigned)((a.V + 255) / 256), (unsigned)a.M), 256, 0, st>>>(a);
  if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
  grad_w2_kernel<<<dim3((unsigned)a.V), a.R, 0, st>>>(a);
  if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
  grad_emb_kernel<<<dim3((unsigned)a.M), a.R, 0, st>>>(a);
  if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
  grad_w1_kernel<<<dim3((unsigned)a.M), a.R, 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

}  // extern "C"
