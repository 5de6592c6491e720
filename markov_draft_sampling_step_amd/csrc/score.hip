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
  // the workspace: per row-step, written by rows_kernel
  int32_t* fed;               // [M] the w1 row
  int32_t* own;               // [M] the token, -1 if the row-step takes no part
  float* heat;                // [M] log2(e) / T
  float* scale;               // [M] grad / T
  float* lse2;                // [M] lse log2(e)
  float* own_u;               // [M] the token's tempered logit, in powers of 2
  f32x2_t* parts;             // [slabs][M] maximum and sum over a slab's vocabulary
  float* grad_emb;            // [splits][M][R]
  int M, k, V, R;
  int slabs, chunks_per, shares;   // scoring: slabs, 64-token chunks per workgroup, workgroups per slab
  int splits, tiles_per;           // gradients: vocabulary splits, 64-entry tiles of each
  float mult, cap, inv_cap;
};

__device__ __forceinline__ bool scored(const int64_t* tokens, const int32_t* lengths, int m, int k,
                                       int V) {
  const int r = m / k, s = m - r * k;
  const int64_t t = tokens[m];
  return (!lengths || s < lengths[r]) && t >= 0 && t < V;
}

// Everything the kernels need of a row-step, once per call.
template <bool BACKWARD>
__global__ __launch_bounds__(256) void rows_kernel(ScoreArgs a) {
  const int m = blockIdx.x * 256 + threadIdx.x;
  if (m >= a.M) return;
  const int r = m / a.k;
  // the w1 row that feeds it: the loop's clamp, as unsigned
  const uint64_t f = (uint64_t)(m == r * a.k ? a.prev[r] : a.tokens[m - 1]);
  a.fed[m] = (int)(f < (uint64_t)a.V ? f : (uint64_t)(a.V - 1));
  const float T = a.temperature ? a.temperature[r] : 1.0f, it = T == 0.0f ? 1.0f : 1.0f / T;
  a.heat[m] = it * LOG2E;
  bool part = scored(a.tokens, a.lengths, m, a.k, a.V);
  if (BACKWARD) {
    const float g = a.grad[m];
    part = part && g != 0.0f;
    a.scale[m] = part ? g * it : 0.0f;
    a.lse2[m] = part ? a.lse[m] * LOG2E : 0.0f;
  }
  a.own[m] = part ? (int)a.tokens[m] : -1;
}

// The output transform of one logit. With e = exp(-2|y|), y = mult x / cap:
// tanh = (1 - e)/(1 + e) and its slope 4e/(1 + e)^2, neither of which cancels
// (a relative error of a small tanh is a small error of the logit).
struct Transform {
  float mult, cap, bend;      // bend = -2 log2(e) mult / cap
  __device__ __forceinline__ explicit Transform(const ScoreArgs& a)
      : mult(a.mult), cap(a.cap), bend(2.0f * LOG2E * a.mult * a.inv_cap) {}
  template <bool CAP>
  __device__ __forceinline__ float logit(float x) const {
    if (!CAP) return mult * x;
    const float y = bend * x, e = __builtin_amdgcn_exp2f(-fabsf(y));
    return cap * __builtin_copysignf((1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e), y);
  }
  template <bool CAP>
  __device__ __forceinline__ float logit(float x, float* slope) const {
    if (!CAP) {
      *slope = mult;
      return mult * x;
    }
    const float y = bend * x, e = __builtin_amdgcn_exp2f(-fabsf(y)), q = __builtin_amdgcn_rcpf(1.0f + e);
    *slope = 4.0f * mult * e * q * q;
    return cap * __builtin_copysignf((1.0f - e) * q, y);
  }
};

// (m, s) += (m2, s2) of a running maximum and sum of powers of 2.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float at = top == -INFINITY ? 0.0f : top;
  s = s * __builtin_amdgcn_exp2f(m - at) + s2 * __builtin_amdgcn_exp2f(m2 - at);
  m = top;
}

__device__ __forceinline__ void load_lds(const void* src, void* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

__device__ __forceinline__ void landed() {
  __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): this wave's asynchronous loads
  __syncthreads();
}

// ---------------------------------------------------------------- scoring
//
// A workgroup of 4 waves takes a slab of the vocabulary and some of the 64-token
// chunks of the block. A wave holds its w2 rows as matrix operands for the
// whole call (16 NT rows x R, 128 registers at R = 256), so the table is read
// once per workgroup; the chunk's embeddings come through LDS, two buffers,
// and the base logits straight from memory, 16 tokens ahead. Per 16 tokens:
// the product in fp32, the base logit, the transform, and the running maximum
// and sum of the softmax over the lane's 4 NT neighbouring entries. Nothing
// of the size of the logits is written.
//
// A operand: w2 rows, B operand: tokens; row i of tile n is entry
// (i / 4) 4 NT + 4 n + i % 4 of the wave's, so that a lane's entries are
// neighbours. LDS: 16-byte group c of token t is at place c ^ (t & KEY).

template <int R>
struct Rank {
  static constexpr int G = R / 8;                        // 16-byte groups of a row
  static constexpr int KEY = G < 8 ? G - 1 : 7;
  static constexpr int KS = R < 32 ? 1 : R / 32;         // matrix steps over the rank
};

template <int R, bool CAP>
__global__ __launch_bounds__(256, R <= 256 ? 2 : 1) void score_kernel(ScoreArgs a) {
  typedef Rank<R> Q;
  constexpr int NT = R <= 256 ? 4 : 2, NE = 4 * NT;      // entries of a lane
  __shared__ __attribute__((aligned(16))) uint8_t one[64 * R * 2], two[64 * R * 2];
  __shared__ f32x2_t stat[64][17];
  const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // a slab's workgroups follow each other on one XCD and share its w2 rows
  const int local = blockIdx.x >> 3, slab = (local / a.shares) * 8 + (blockIdx.x & 7);
  if (slab >= a.slabs) return;
  const int chunks = (a.M + 63) / 64;
  const int c0 = (local % a.shares) * a.chunks_per, c1 = min(chunks, c0 + a.chunks_per);
  if (c0 >= c1) return;

  auto request = [&](int c, uint8_t* __restrict__ to) {
#pragma unroll
    for (int i = 0; i < (Q::G + 3) / 4; ++i) {
      const int n = wave + 4 * i;
      if (Q::G % 4 != 0 && n >= Q::G) break;
      const int at = n * 64 + lane, t = at / Q::G, place = at % Q::G;
      load_lds(a.w1 + (size_t)a.fed[min(c * 64 + t, a.M - 1)] * R + (place ^ (t & Q::KEY)) * 8, to + n * 1024);
    }
  };
  request(c0, one);

  const int vw = slab * 64 * NT + wave * 16 * NT;        // the wave's first entry, then the lane's
  const int vl = vw + lg * NE;
  bf16x8_t A[NT][Q::KS];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int v = min(vw + (li >> 2) * NE + 4 * n + (li & 3), a.V - 1);
    const uint16_t* row = a.w2 + (size_t)v * R + lg * 8;
#pragma unroll
    for (int s = 0; s < Q::KS; ++s)
      A[n][s] = R >= 32 || lg < 2 ? *(const bf16x8_t*)(row + s * 32) : (bf16x8_t){};
  }
  const Transform f(a);

  // a group of 16 tokens: this lane's base logits, token and temperature
  struct Ahead {
    u32x4_t base[NT / 2];
    int own;
    float heat;
  };
  const int m1 = min(a.M, c1 * 64);
  auto ahead = [&](int c, int g) {
    Ahead h;
    const int m = c * 64 + g * 16 + li;
    h.own = -1;
    h.heat = 0.0f;
    if (m < m1) {
      h.own = a.own[m];
      h.heat = a.heat[m];
    }
#pragma unroll
    for (int i = 0; i < NT / 2; ++i)
      h.base[i] = m < m1 && vl + 8 * i < a.V ? *(const u32x4_t*)(a.base + (size_t)m * a.V + vl + 8 * i)
                                             : (u32x4_t){0u, 0u, 0u, 0u};
    return h;
  };

  auto group = [&](int c, int g, const Ahead& h, const uint8_t* __restrict__ from) {
    f32x4_t z[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) z[n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    const int t = g * 16 + li;
#pragma unroll
    for (int s = 0; s < Q::KS; ++s) {
      const int place = (R >= 32 ? s * 4 + lg : lg & 1) ^ (t & Q::KEY);
      bf16x8_t B = *(const bf16x8_t*)(from + t * R * 2 + place * 16);
      if (R < 32 && lg >= 2) B = (bf16x8_t){};
#pragma unroll
      for (int n = 0; n < NT; ++n) z[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[n][s], B, z[n], 0, 0, 0);
    }
    float u[NE], top = -INFINITY;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const uint32_t w = h.base[e >> 3][(e >> 1) & 3];
      u[e] = f.logit<CAP>(((e & 1) ? bf_hi(w) : bf_lo(w)) + z[e >> 2][e & 3]) * h.heat;
      if (vl + (e & ~7) >= a.V || h.own < 0) u[e] = -INFINITY;
      top = fmaxf(top, u[e]);
    }
    const float at = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < NE; ++e) sum += __builtin_amdgcn_exp2f(u[e] - at);
    stat[t][wave * 4 + lg] = (f32x2_t){top, sum};
    const unsigned d = (unsigned)(h.own - vl);
    if (d < (unsigned)NE) {
      float mine = u[0];
#pragma unroll
      for (int e = 1; e < NE; ++e) mine = d == (unsigned)e ? u[e] : mine;
      a.own_u[c * 64 + t] = mine;
    }
  };

  Ahead now = ahead(c0, 0);
  auto chunk = [&](int c, const uint8_t* __restrict__ from, uint8_t* __restrict__ to) {
    landed();
    if (c + 1 < c1) request(c + 1, to);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (c * 64 + g * 16 >= a.M) break;
      const Ahead next = ahead(g < 3 ? c : c + 1, (g + 1) & 3);
      group(c, g, now, from);
      now = next;
    }
    __syncthreads();
    // the workgroup's maximum and sum of each token, 4 threads a token
    const int t = tid >> 2, m = c * 64 + t;
    if (m < a.M) {
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2_t q = stat[t][(tid & 3) * 4 + i];
        join(top, sum, q[0], q[1]);
      }
#pragma unroll
      for (int sh = 1; sh <= 2; sh <<= 1) {
        const float m2 = __shfl_xor(top, sh), s2 = __shfl_xor(sum, sh);
        join(top, sum, m2, s2);
      }
      if ((tid & 3) == 0) a.parts[(size_t)slab * a.M + m] = (f32x2_t){top, sum};
    }
  };
  int c = c0;
  for (; c + 1 < c1; c += 2) {
    chunk(c, one, two);
    chunk(c + 1, two, one);
  }
  if (c < c1) chunk(c, one, two);
}

// 8 row-steps per workgroup, 32 threads each over the slabs.
__global__ __launch_bounds__(256) void score_finish_kernel(ScoreArgs a) {
  const int tid = threadIdx.x, m = blockIdx.x * 8 + (tid & 7), j = tid >> 3;
  float top = -INFINITY, sum = 0.0f;
  if (m < a.M)
    for (int s = j; s < a.slabs; s += 32) {
      const f32x2_t p = a.parts[(size_t)s * a.M + m];
      join(top, sum, p[0], p[1]);
    }
  __shared__ f32x2_t part[32][8];
  part[j][tid & 7] = (f32x2_t){top, sum};
  __syncthreads();
  if (j > 0 || m >= a.M) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) join(top, sum, part[i][tid][0], part[i][tid][1]);
  if (a.own[m] < 0) {
    a.logprobs[m] = a.lse[m] = 0.0f;
    return;
  }
  const float l2 = top + __log2f(sum), u = a.own_u[m];
  a.lse[m] = l2 * LN2;
  a.logprobs[m] = u == -INFINITY ? -INFINITY : (u - l2) * LN2;
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
template <bool CAP>
__global__ __launch_bounds__(256) void grad_base_kernel(ScoreArgs a) {
  const int m = blockIdx.y, v = blockIdx.x * 256 + threadIdx.x;
  if (v >= a.V) return;
  float d = 0.0f;
  if (a.own[m] >= 0) {
    float dot = 0.0f, slope;
    const uint16_t* emb = a.w1 + (size_t)a.fed[m] * a.R;
    for (int j = 0; j < a.R; ++j) dot += bf_one(emb[j]) * bf_one(a.w2[(size_t)v * a.R + j]);
    const float z = Transform(a).logit<CAP>(bf_one(a.base[(size_t)m * a.V + v]) + dot, &slope), u = z * a.heat[m];
    const float p = __builtin_amdgcn_exp2f(u - a.lse2[m]);
    d = u == -INFINITY ? 0.0f : a.scale[m] * ((v == a.own[m] ? 1.0f : 0.0f) - p) * slope;
  }
  a.grad_base[(size_t)m * a.V + v] = (uint16_t)pack_bf16(d, 0.0f);
}

// grid V, R threads: grad_w2[v].
__global__ void grad_w2_kernel(ScoreArgs a) {
  const int v = blockIdx.x, j = threadIdx.x;
  float sum = 0.0f;
  for (int m = 0; m < a.M; ++m)
    sum += bf_one(a.grad_base[(size_t)m * a.V + v]) * bf_one(a.w1[(size_t)a.fed[m] * a.R + j]);
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
  const int row = a.fed[m];
  float sum = 0.0f;
  for (int i = 0; i < a.M; ++i) {
    if (a.fed[i] != row) continue;
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

size_t aligned(size_t n) { return (n + 255) & ~(size_t)255; }

// How a call is split, and the workspace that this takes: a function of the
// shape alone.
struct Plan {
  int slabs, shares, chunks_per, splits, tiles_per;
  size_t rows_bytes, bytes;
};

constexpr int ROW_ARRAYS = 6;   // of 4 bytes per row-step

Plan plan_of(const markov_shape_t* sh, int32_t k) {
  Plan p;
  const int M = sh->rows * k, slab = sh->rank <= 256 ? 256 : 128;
  p.slabs = (int)(((int64_t)sh->vocab + slab - 1) / slab);
  // about 2500 workgroups: two fit a CU at the largest rank, and a few rounds
  // of them even out the end
  const int chunks = (M + 63) / 64, want = (2560 + p.slabs - 1) / p.slabs;
  p.shares = want < chunks ? want : chunks;
  p.chunks_per = (chunks + p.shares - 1) / p.shares;
  p.shares = (chunks + p.chunks_per - 1) / p.chunks_per;
  p.splits = 1;
  p.tiles_per = (int)(((int64_t)sh->vocab + 63) / 64);
  p.rows_bytes = aligned((size_t)M * 4);
  const size_t score = (size_t)p.slabs * M * 8, grad = (size_t)p.splits * M * sh->rank * 4;
  p.bytes = ROW_ARRAYS * p.rows_bytes + aligned(score > grad ? score : grad);
  return p;
}

ScoreArgs arguments(const void* base, const void* w1, const void* w2, const int64_t* prev,
                    const int64_t* tokens, const int32_t* lengths, int32_t k,
                    const float* temperature, const markov_shape_t* sh, const Plan& p, void* workspace) {
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
  a.slabs = p.slabs;
  a.shares = p.shares;
  a.chunks_per = p.chunks_per;
  a.splits = p.splits;
  a.tiles_per = p.tiles_per;
  uint8_t* at = (uint8_t*)workspace;
  void** rows[ROW_ARRAYS] = {(void**)&a.fed, (void**)&a.own, (void**)&a.heat,
                             (void**)&a.scale, (void**)&a.lse2, (void**)&a.own_u};
  for (void** r : rows) {
    *r = at;
    at += p.rows_bytes;
  }
  a.parts = (f32x2_t*)at;
  a.grad_emb = (float*)at;
  return a;
}

template <typename K>
int launch(K kernel, int64_t grid, int threads, hipStream_t stream, const ScoreArgs& a) {
  if (grid > 0xffffffffll / threads) return MARKOV_ERR_SHAPE;
  kernel<<<dim3((unsigned)grid), threads, 0, stream>>>(a);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

typedef void (*ScoreKernel)(ScoreArgs);

template <bool CAP>
ScoreKernel score_kernel_of(int rank) {
  switch (rank) {
    case 16: return score_kernel<16, CAP>;
    case 32: return score_kernel<32, CAP>;
    case 64: return score_kernel<64, CAP>;
    case 128: return score_kernel<128, CAP>;
    case 256: return score_kernel<256, CAP>;
    default: return score_kernel<512, CAP>;
  }
}

}  // namespace

extern "C" {

size_t markov_score_workspace_bytes(const markov_shape_t* shape, int32_t k) {
  if (check(shape, k)) return 0;
  return plan_of(shape, k).bytes;
}

int markov_score_sequential(const void* base_logits, const void* w1, const void* w2,
                            const int64_t* prev, const int64_t* tokens, const int32_t* lengths,
                            int32_t k, const float* temperature, float* logprobs, float* lse,
                            markov_stream_t stream, const markov_shape_t* shape, void* workspace,
                            size_t workspace_bytes) {
  int rc = check(shape, k);
  if (rc) return rc;
  if (!base_logits || !w1 || !w2 || !prev || !tokens || !logprobs || !lse || !workspace)
    return MARKOV_ERR_NULL;
  if (!aligned_to(base_logits, 16) || !aligned_to(w1, 16) || !aligned_to(w2, 16) ||
      !aligned_to(workspace, 16))
    return MARKOV_ERR_ALIGN;
  const Plan p = plan_of(shape, k);
  if (workspace_bytes < p.bytes) return MARKOV_ERR_WORKSPACE;
  ScoreArgs a = arguments(base_logits, w1, w2, prev, tokens, lengths, k, temperature, shape, p, workspace);
  a.logprobs = logprobs;
  a.lse = lse;
  const hipStream_t st = (hipStream_t)stream;
  if ((rc = launch(rows_kernel<false>, (a.M + 255) / 256, 256, st, a))) return rc;
  const ScoreKernel kernel = a.cap > 0.0f ? score_kernel_of<true>(a.R) : score_kernel_of<false>(a.R);
  if ((rc = launch(kernel, (int64_t)((a.slabs + 7) / 8) * 8 * a.shares, 256, st, a))) return rc;
  return launch(score_finish_kernel, (a.M + 7) / 8, 256, st, a);
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
  int rc = check(shape, k);
  if (rc) return rc;
  if (!base_logits || !w1 || !w2 || !prev || !tokens || !lse || !grad_logprobs || !grad_base ||
      !grad_w1 || !grad_w2 || !workspace)
    return MARKOV_ERR_NULL;
  if (!aligned_to(base_logits, 16) || !aligned_to(w1, 16) || !aligned_to(w2, 16) ||
      !aligned_to(grad_base, 16) || !aligned_to(grad_w1, 16) || !aligned_to(grad_w2, 16) ||
      !aligned_to(workspace, 16))
    return MARKOV_ERR_ALIGN;
  const Plan p = plan_of(shape, k);
  if (workspace_bytes < p.bytes) return MARKOV_ERR_WORKSPACE;
  ScoreArgs a = arguments(base_logits, w1, w2, prev, tokens, lengths, k, temperature, shape, p, workspace);
  a.lse = (float*)lse;
  a.grad = grad_logprobs;
  a.grad_base = (uint16_t*)grad_base;
  a.grad_w1 = (uint16_t*)grad_w1;
  a.grad_w2 = (uint16_t*)grad_w2;
  const hipStream_t st = (hipStream_t)stream;
  if ((rc = launch(rows_kernel<true>, (a.M + 255) / 256, 256, st, a))) return rc;
  (a.cap > 0.0f ? grad_base_kernel<true> : grad_base_kernel<false>)<<<dim3((unsigned)((a.V + 255) / 256), (unsigned)a.M), 256, 0, st>>>(a);
  if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
  if ((rc = launch(grad_w2_kernel, a.V, a.R, st, a))) return rc;
  if ((rc = launch(grad_emb_kernel, a.M, a.R, st, a))) return rc;
  return launch(grad_w1_kernel, a.M, a.R, st, a);
}

}  // extern "C"
