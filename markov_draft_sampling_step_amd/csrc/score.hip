// MI355X (gfx950) training on drafted blocks: the log-probabilities of a
// block's tokens under the corrected logits, the clipped policy loss with a KL
// term, and the gradients of the base logits, w1 and w2.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "markov.h"
#include "numbers.h"

namespace {

constexpr float LOG2E = 1.44269504088896341f, LN2 = 0.693147180559945309f;

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
  // the workspace: per row-step, written by rows_kernel or grad_base_kernel
  uint16_t* emb;              // [M rounded up to 64][R] its w1 row, 0 if it takes no part
  int32_t* fed;               // [M] the w1 row's number
  int32_t* own;               // [M] the token, -1 if the row-step takes no part
  float* heat;                // [M] what takes a logit to a power of 2: log2(e) / T, times mult without a cap
  float* rest;                // [M] what rounding d of the token itself to bf16 left off
  f32x2_t* parts;             // [slabs][M] maximum and sum over a slab's vocabulary
  float* grad_emb;            // [splits][M][R]
  int M, k, V, R;
  int slabs, shares;               // scoring: slabs of the vocabulary, workgroups
  int splits, tiles_per;           // gradients: vocabulary splits, tiles of each
  float mult, cap, inv_cap;
};

__device__ __forceinline__ bool scored(const int64_t* tokens, const int32_t* lengths, int m, int k,
                                       int V) {
  const int r = m / k, s = m - r * k;
  const int64_t t = tokens[m];
  return (!lengths || s < lengths[r]) && t >= 0 && t < V;
}

// The largest factor of a logit: a distance of 0 times it is 0, times infinity NaN.
constexpr float MOST = 0x1p126f;
__device__ __forceinline__ float bounded(float f) { return fabsf(f) > MOST ? __builtin_copysignf(MOST, f) : f; }

// 1 / T of a row, as the formulas have it (1 for a T of 0).
__device__ __forceinline__ float inverse_temperature(const ScoreArgs& a, int r) {
  const float T = a.temperature ? a.temperature[r] : 1.0f;
  return T == 0.0f ? 1.0f : bounded(1.0f / T);
}

// What the kernels need of a row-step: the w1 row that feeds it (the loop's clamp,
// as unsigned), its token if it takes part, else -1, and its factors.
struct RowStep {
  int fed, own;
  float inverse, heat, scale, lse;   // 1 / T, log2(e) / T, grad / T, the lse
};

template <bool BACKWARD>
__device__ __forceinline__ RowStep row_step(const ScoreArgs& a, int m) {
  const int r = m / a.k;
  const uint64_t f = (uint64_t)(m == r * a.k ? a.prev[r] : a.tokens[m - 1]);
  const float it = inverse_temperature(a, r);
  bool part = scored(a.tokens, a.lengths, m, a.k, a.V);
  float g = 0.0f, lse = 0.0f;
  if (BACKWARD) {
    g = a.grad[m];
    lse = a.lse[m];
    // (nothing to follow from a gradient of 0, nor where all is masked: by -inf, or
    // by finite logits beside which binary32 does not hold the logarithm of a sum;
    // nor at a temperature that takes the logits to the end of binary32)
    part = part && g != 0.0f && !(lse < -0x1p24f * fabsf(it)) && !(fabsf(lse) > MOST);
  }
  RowStep s;
  s.fed = (int)(f < (uint64_t)a.V ? f : (uint64_t)(a.V - 1));
  s.own = part ? (int)a.tokens[m] : -1;
  s.inverse = it;
  s.heat = it * LOG2E;
  s.scale = part ? g * it : 0.0f;
  s.lse = part ? lse : 0.0f;
  return s;
}

// The factor that takes a logit to a power of 2. An infinite temperature and a
// multiplier of 0 flatten every logit but a mask's: with the smallest number for 0
// the largest logits still differ by 2^-20 at most, and -inf times it is -inf.
__device__ __forceinline__ float factor(float f) { return f == 0.0f ? __builtin_copysignf(0x1p-149f, f) : bounded(f); }

// A 16-byte group x of row m of the gathered embeddings, which are padded to 64
// rows; zeros past the last row-step and where one does not take part.
template <bool BACKWARD>
__device__ __forceinline__ RowStep gather_embedding(const ScoreArgs& a, int m, int x) {
  RowStep s = {0, -1, 0.0f, 0.0f, 0.0f, 0.0f};
  if (m < a.M) s = row_step<BACKWARD>(a, m);
  ((u32x4_t*)(a.emb + (size_t)m * a.R))[x] =
      s.own >= 0 ? ((const u32x4_t*)(a.w1 + (size_t)s.fed * a.R))[x] : (u32x4_t){0u, 0u, 0u, 0u};
  return s;
}

// Once before the scoring: R / 8 threads a row-step.
__global__ __launch_bounds__(256) void rows_kernel(ScoreArgs a) {
  const int across = a.R / 8;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int m = (int)(at / across), x = (int)(at - (int64_t)m * across);
  if (m >= ((a.M + 63) & ~63)) return;
  const RowStep s = gather_embedding<false>(a, m, x);
  if (x > 0 || m >= a.M) return;
  a.heat[m] = factor(s.heat * (a.cap > 0.0f ? 1.0f : a.mult));
  a.own[m] = s.own;
}

// The output transform of one logit, y = mult x / cap. For the scores tanh = 1 -
// 2 / (1 + exp(2y)), a few steps of 1 off, so the logit a few of the cap; infinities
// and NaN come out right (the cap as 1 - e over 1 + e, which is what the slope has
// anyway, took 77 us instead of 73 for 320 x 163840 x 256). For the gradients, with
// e = exp(-2|y|), tanh = (1 - e)/(1 + e), likewise a few steps of 1 off, and its
// slope 4e/(1 + e)^2, which neither cancels nor overflows; it is without the factor
// mult. A cap past WIDE, whose steps would show in logits that it hardly bends, takes
// tanh to a few steps of itself in both: its series below 1/8 (2048 x 163840 x 256
// scored in 375 us for 299, its gradients in 827 for 760).
struct Transform {
  static constexpr float WIDE = 64.0f;   // (a few steps of 64 are 2^-16)
  float mult, cap, bend;      // bend = 2 log2(e) mult / cap
  float rate;                 // mult / cap
  bool wide;
  __device__ __forceinline__ explicit Transform(const ScoreArgs& a)
      : mult(a.mult), cap(a.cap), bend(2.0f * LOG2E * a.mult * a.inv_cap), rate(a.mult * a.inv_cap), wide(a.cap > WIDE) {}
  // For any cap, and for one up to WIDE.
  __device__ __forceinline__ float exact(float x) const {
    const float y = rate * x, s = y * y, e = __builtin_amdgcn_exp2f(-fabsf(bend * x));
    const float t = __builtin_fmaf(y * s, s * (s * (-17.0f / 315.0f) + 2.0f / 15.0f) - 1.0f / 3.0f, y);
    const float far = __builtin_copysignf((1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e), y);
    return cap * (fabsf(y) < 0.125f ? t : far);
  }
  __device__ __forceinline__ float near(float x) const {
    return __builtin_fmaf(-2.0f * cap, __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(bend * x)), cap);
  }
  __device__ __forceinline__ float capped(float x) const { return wide ? exact(x) : near(x); }
  // One up to WIDE, with the slope.
  __device__ __forceinline__ float near(float x, float* slope) const {
    const float y = bend * x, e = __builtin_amdgcn_exp2f(-fabsf(y)), q = __builtin_amdgcn_rcpf(1.0f + e);
    *slope = 4.0f * e * q * q;
    return cap * __builtin_copysignf((1.0f - e) * q, y);
  }
};

// (m, s) += (m2, s2): a running maximum of logits and sum of 2^(h (logit - m)), h >
// 0. The maximum is kept as a logit, so that one of any size loses nothing.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2, float h) {
  const float top = fmaxf(m, m2);
  const float at = top == -INFINITY ? 0.0f : top;
  s = s * __builtin_amdgcn_exp2f((m - at) * h) + s2 * __builtin_amdgcn_exp2f((m2 - at) * h);
  m = top;
}

// Beyond this a logit's power of 2 is taken from its distance to the largest: the
// product with h is rounded by up to 2^-14 and more there, and from 2^31 by more than
// binary32 has exponents. Both passes then also round z / T and lse alike, so that
// the only token that a small temperature leaves has probability 1 exactly. (Rows
// past it, at T = 0.01, beside rows at 1: 2048 x 163840 x 256 scored in 274 us for
// 252 and its gradients in 770 for 721, 320 with the soft cap 80 for 75 and 219 for
// 167. The largest logit and lse up to it lose 2^-14 of a probability at most.)
constexpr float FAR = 1024.0f;

// (ONCE: what nothing reads again, kept out of the caches as far as they allow)
template <bool ONCE = false>
__device__ __forceinline__ void load_lds(const void* src, void* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, ONCE ? 2 : 0);
}

// From a scalar base and a lane's 32-bit offset (both opaque, so that the
// address is not made a 64-bit value per lane and held).
template <bool ONCE = false>
__device__ __forceinline__ void load_lds(const void* base, uint32_t off, void* dst) {
  asm volatile("" : "+s"(base), "+v"(off));
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)((const __attribute__((address_space(1))) uint8_t*)base + off),
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, ONCE ? 2 : 0);
}

// ---------------------------------------------------------------- scoring
//
// The work is a list of units, a slab of the vocabulary and a chunk of 32 tokens
// each, slab by slab, cut into equal shares for as many workgroups of 4 waves as
// fit. A wave holds its slab's w2 rows as matrix operands (16 NT rows x R, 128
// registers at R = 256) until the slab changes, so the table is read about once;
// a chunk's embeddings and base logits come through LDS by asynchronous loads, a
// unit ahead (base logits straight to registers, 16 tokens ahead, were too few
// bytes under way: 64 x 5 x 163840 x 256 took 72 us). Per 16 tokens: the product
// in fp32, the base logit, the transform, and the maximum and sum of the softmax
// over the lane's 4 NT neighbouring entries. Nothing of the size of the logits is
// written.
//
// Measured (the kernel, V = 163840, no cap but where it is named): 320 tokens at rank
// 256 52-56 us, 3.5 TB/s of the logits and the table, with the soft cap 61-70; 2048
// tokens 230-252 us (the product 710 TF, the matrix units 34 % busy, vector
// instructions about as much), at rank 64 145-159 us, 4.5 TB/s. The matrix units
// and the memory both wait, for the turns that products, exponentials and loads
// take, and for each slab's table, which is asked for when the slab begins.
//
// A operand: w2 rows, B operand: tokens; row i of tile n is entry
// (i / 4) 4 NT + 4 n + i % 4 of the wave's, so that a lane's entries are
// neighbours. LDS: 16-byte group c of token t's embedding is at place
// c ^ (t & KEY), of its base logits at c ^ (t & 15). (A read of 16 bytes a lane
// takes 16 lanes at a time over 256 bytes of banks: with rows of 256 bytes or more
// a key of 3 bits puts them on half of the banks and takes 1.65 times as long.)

template <int R>
struct Rank {
  static constexpr int G = R / 8;                        // 16-byte groups of a row
  static constexpr int KEY = G < 16 ? G - 1 : 15;
  static constexpr int KS = R < 32 ? 1 : R / 32;         // matrix steps over the rank
};

template <int R, bool CAP>
struct Score {
  typedef Rank<R> Q;
  static constexpr int NT = R <= 256 ? 4 : 2, NE = 4 * NT;   // entries of a lane
  static constexpr int SLAB = 64 * NT, GB = SLAB / 8;        // entries of a slab, 16-byte groups of a token's base
  static constexpr int E = 32 * R * 2, B = 32 * SLAB * 2;    // bytes of a chunk
  static constexpr int NLE = E / 1024, NLB = B / 1024;       // loads of 64 lanes
  static constexpr int LE = (NLE + 3) / 4, LB = NLB / 4;     // of a wave
  const ScoreArgs& a;
  const Transform f;
  int tid, lane, li, lg, wave, chunks;
  static constexpr int EV = R >= 512 ? 4 : 2;                // permutations of a wave's embedding loads
  uint32_t e_off[EV], b_off;
  bf16x8_t A[NT][Q::KS];
  float heat[2];         // of this lane's two tokens of the chunk

  __device__ __forceinline__ void place() {
#pragma unroll
    for (int i = 0; i < EV; ++i) {
      // (a wave's loads are 4 apart; 16 tokens on the permutation is the same)
      const int at = (wave + 4 * i) * 64 + lane;
      e_off[i] = (uint32_t)(lane / Q::G) * R * 2 + ((at % Q::G) ^ ((at / Q::G) & Q::KEY)) * 16;
    }
    // (a load holds 64 / GB tokens, and a wave's loads are 4 loads apart)
    b_off = (uint32_t)(lane / GB) * (uint32_t)a.V * 2;
  }

  __device__ __forceinline__ void request(int slab, int c, uint8_t* __restrict__ e, uint8_t* __restrict__ b) const {
#pragma unroll
    for (int i = 0; i < LE; ++i) {
      const int n = wave + 4 * i;
      if (NLE % 4 != 0 && n >= NLE) break;
      load_lds(a.emb + (size_t)c * 32 * R + n * 512, e_off[i & (EV - 1)], e + n * 1024);
    }
    if (c * 32 + 32 <= a.M && (slab + 1) * SLAB <= a.V) {
#pragma unroll
      for (int i = 0; i < LB; ++i) {
        const int n = wave + 4 * i, t0 = n * (64 / GB);        // the load's first token
        load_lds(a.base + (size_t)(c * 32 + t0) * a.V + slab * SLAB, b_off + ((lane % GB) ^ ((t0 + lane / GB) & 15)) * 16,
                 b + n * 1024);
      }
      return;
    }
    // rows past the last row-step repeat it, columns past the last entry are
    // any (the lane is opaque, so that none of this is computed ahead and held)
    int l = lane;
    asm volatile("" : "+v"(l));
#pragma unroll 1
    for (int n = wave; n < NLB; n += 4) {
      const int t = n * (64 / GB) + l / GB, v = slab * SLAB + ((l % GB) ^ (t & 15)) * 8;
      load_lds(a.base + (size_t)min(c * 32 + t, a.M - 1) * a.V + (v < a.V ? v : 0), b + n * 1024);
    }
  }

  // The slab's w2 rows; those past the last entry repeat it.
  __device__ __forceinline__ void table(int slab) {
    const int vw = slab * SLAB + wave * 16 * NT;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int v = min(vw + (li >> 2) * NE + 4 * n + (li & 3), a.V - 1);
      const uint16_t* row = a.w2 + (size_t)v * R + lg * 8;
#pragma unroll
      for (int s = 0; s < Q::KS; ++s)
        A[n][s] = R >= 32 || lg < 2 ? *(const bf16x8_t*)(row + s * 32) : (bf16x8_t){};
    }
  }

  __device__ __forceinline__ void tokens(int c) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      heat[g] = a.heat[min(c * 32 + g * 16 + li, a.M - 1)];   // (a row-step past the last: what it does is not kept)
    }
  }

  // The logits of 16 tokens. The base logits are added last, in one rounding: as
  // the product's accumulator they took one for each 32 of the rank, at their own size,
  // and lse and log-probabilities were 1.4 times as far off (2048 x 163840 x 256 262
  // us for 269, now 253).
  // PRODUCT: their products alone, REST: what follows them.
  template <bool PRODUCT, bool REST>
  __device__ __forceinline__ void logits(int slab, int g, float h, const uint8_t* __restrict__ e,
                                         const uint8_t* __restrict__ b, f32x4_t (&z)[NT]) const {
    const int t = g * 16 + li, vl = slab * SLAB + wave * 16 * NT + lg * NE;
#pragma unroll
    for (int n = 0; PRODUCT && n < NT; ++n) z[n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; PRODUCT && s < Q::KS; ++s) {
      const int place = (R >= 32 ? s * 4 + lg : lg & 1) ^ (t & Q::KEY);
      bf16x8_t B = *(const bf16x8_t*)(e + t * R * 2 + place * 16);
      if (R < 32 && lg >= 2) B = (bf16x8_t){};
#pragma unroll
      for (int n = 0; n < NT; ++n) z[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[n][s], B, z[n], 0, 0, 0);
    }
    if (!REST) return;
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) {
      const u32x4_t x = *(const u32x4_t*)(b + t * SLAB * 2 + ((wave * 2 * NT + lg * (NT / 2) + i) ^ (t & 15)) * 16);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        z[2 * i + h] += (f32x4_t){bf_lo(x[2 * h]), bf_hi(x[2 * h]), bf_lo(x[2 * h + 1]), bf_hi(x[2 * h + 1])};
    }
    if (CAP && !f.wide) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[n][k] = f.near(z[n][k]);
    } else if (CAP) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[n][k] = f.exact(z[n][k]);
          __builtin_amdgcn_sched_barrier(0);   // (one at a time: there are no registers for more)
        }
    }
    if ((slab + 1) * SLAB > a.V) {   // uniform: past the last entry there is no mass
      const float none = h < 0.0f ? INFINITY : -INFINITY;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (vl + (n & ~1) * 4 >= a.V) z[n] = (f32x4_t){none, none, none, none};
    }
  }

  // Their maximum and sum over the lane's entries; h takes a logit to a power of
  // 2 (without a cap it holds the factor mult as well). With a negative h (a
  // negative temperature or multiplier) the maximum is that of -z.
  __device__ __forceinline__ f32x2_t soften(const f32x4_t (&z)[NT], float h) const {
    float top = z[0][0];
#pragma unroll
    for (int k = 1; k < NE; ++k) top = fmaxf(top, z[k >> 2][k & 3]);
    float most = top, from = top == -INFINITY ? 0.0f : top, sum = 0.0f;
    const float at = from * h;
    float off = __builtin_fmaf(from, h, -at);   // what at was rounded by, at most 2^-15
    const bool apart = h < 0.0f || fabsf(at) > FAR;
    if (__builtin_expect(__ballot(apart) == 0, 1)) {
#pragma unroll
      for (int k = 0; k < NE; ++k) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(z[k >> 2][k & 3], h, -at));
    } else {
      float low = z[0][0];
#pragma unroll
      for (int k = 1; k < NE; ++k) low = fminf(low, z[k >> 2][k & 3]);
      if (h < 0.0f) {
        most = -low;
        from = most == -INFINITY ? 0.0f : low;
      }
#pragma unroll
      for (int k = 0; k < NE; ++k) {
        const float x = z[k >> 2][k & 3];
        sum += __builtin_amdgcn_exp2f(apart ? (x - from) * h : __builtin_fmaf(x, h, -at));
      }
      off = apart ? 0.0f : off;
    }
    sum = __builtin_fmaf(sum, -LN2 * off, sum);   // (2^-off is 1 - off ln 2)
    return (f32x2_t){most, sum};
  }

  __device__ __forceinline__ void unit(int slab, int c, const uint8_t* __restrict__ e, const uint8_t* __restrict__ b,
                                       f32x2_t (&stat)[32][17], const float (&heat)[2]) const {
    f32x4_t z0[NT], z1[NT];
    // (the second product hides the first one's end; with the cap, and with twice the
    // rank, there are no registers for it: 2048 x 163840 x 256 252 us for 255, with
    // the cap 301 and 296, 160 x 131072 x 512 77 and 72)
    constexpr bool AHEAD = !CAP && R <= 256;
    if (AHEAD) {
      logits<true, false>(slab, 0, heat[0], e, b, z0);
      logits<true, false>(slab, 1, heat[1], e, b, z1);
    }
    logits<!AHEAD, true>(slab, 0, heat[0], e, b, z0);
    logits<!AHEAD, true>(slab, 1, heat[1], e, b, z1);
    stat[li][wave * 4 + lg] = soften(z0, heat[0]);
    stat[16 + li][wave * 4 + lg] = soften(z1, heat[1]);
    if (tid < 16) {   // (for the join)
      stat[li][16][0] = fabsf(heat[0]);
      stat[16 + li][16][0] = fabsf(heat[1]);
    }
  }

  // The workgroup's maximum and sum of each of a unit's tokens, 8 threads a token.
  __device__ __forceinline__ void join_unit(int slab, int c, const f32x2_t (&stat)[32][17]) const {
    const int t = tid >> 3, m = c * 32 + t;
    const f32x2_t p = stat[t][(tid & 7) * 2], q = stat[t][(tid & 7) * 2 + 1];
    const float h = stat[t][16][0];
    float top = p[0], sum = p[1];
    join(top, sum, q[0], q[1], h);
#pragma unroll
    for (int sh = 1; sh <= 4; sh <<= 1) {
      const float m2 = __shfl_xor(top, sh), s2 = __shfl_xor(sum, sh);
      join(top, sum, m2, s2, h);
    }
    if ((tid & 7) == 0 && m < a.M) a.parts[(size_t)slab * a.M + m] = (f32x2_t){top, sum};
  }

  // A unit, whose loads have landed, and the joins of the one before.
  int slab, c, slab_before, c_before;
  bool fresh, joined;     // the unit's w2 rows are to be read; there is no unit before
  __device__ __forceinline__ void step(bool more, const uint8_t* __restrict__ e, const uint8_t* __restrict__ b,
                                       uint8_t* __restrict__ e_next, uint8_t* __restrict__ b_next,
                                       f32x2_t (&stat)[32][17], const f32x2_t (&stat_before)[32][17]) {
    const float heat_now[2] = {heat[0], heat[1]};
    barrier_but<0>();
    const bool last = c + 1 == chunks;
    const int slab_next = last ? slab + 1 : slab, c_next = last ? 0 : c + 1;
    if (fresh) {
      table(slab);
      // (waited for here: at its use the wait would be for the next unit's
      // loads as well, in every step)
      __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
    }
    if (more) {
      tokens(c_next);
      request(slab_next, c_next, e_next, b_next);
    }
    if (!joined) join_unit(slab_before, c_before, stat_before);
    unit(slab, c, e, b, stat, heat_now);
    slab_before = slab;
    c_before = c;
    slab = slab_next;
    c = c_next;
    fresh = last;
    joined = false;
  }
};

template <int R, bool CAP>
__global__ __launch_bounds__(256, R <= 256 ? 2 : 1) void score_kernel(ScoreArgs a) {
  typedef Score<R, CAP> T;
  __shared__ __attribute__((aligned(16))) uint8_t e0[T::E], e1[T::E], b0[T::B], b1[T::B];
  __shared__ f32x2_t s0[32][17], s1[32][17];
  T g{a, Transform(a)};
  g.tid = threadIdx.x;
  g.lane = g.tid & 63;
  g.li = g.lane & 15;
  g.lg = g.lane >> 4;
  g.wave = __builtin_amdgcn_readfirstlane(g.tid >> 6);
  g.chunks = (a.M + 31) / 32;
  // neighbouring shares on one XCD (workgroups go round the 8 of them)
  const int share = a.shares % 8 == 0 ? (blockIdx.x & 7) * (a.shares / 8) + (blockIdx.x >> 3) : blockIdx.x;
  const int64_t units = (int64_t)a.slabs * g.chunks;
  const int begin = (int)(units * share / a.shares), end = (int)(units * (share + 1) / a.shares);
  g.place();
  g.slab = begin / g.chunks;
  g.c = begin - g.slab * g.chunks;
  g.fresh = false;
  g.joined = true;
  g.request(g.slab, g.c, e0, b0);
  g.tokens(g.c);
  g.table(g.slab);
  int u = begin;
  for (; u + 1 < end; u += 2) {
    g.step(true, e0, b0, e1, b1, s0, s1);
    g.step(u + 2 < end, e1, b1, e0, b0, s1, s0);
  }
  if (u < end) {
    g.step(false, e0, b0, e1, b1, s0, s1);
    __syncthreads();
    g.join_unit(g.slab_before, g.c_before, s0);
  } else {
    __syncthreads();
    g.join_unit(g.slab_before, g.c_before, s1);
  }
}

// 4 row-steps per workgroup, 64 threads each: the join over the slabs in binary32,
// and the token's own logit once more, its product and all that follows in
// binary64. (The binary32 logits of the pass are half a step off, which the sum over
// the vocabulary evens out but a single token's would not.)
template <bool CAP>
__global__ __launch_bounds__(256) void score_finish_kernel(ScoreArgs a) {
  const int tid = threadIdx.x, m = blockIdx.x * 4 + (tid & 3), mm = min(m, a.M - 1), j = tid >> 2;
  const int own = a.own[mm];
  const float heat = a.heat[mm], h = fabsf(heat);
  const float base = bf_one(a.base[(size_t)mm * a.V + max(own, 0)]);
  const uint16_t *emb = a.emb + (size_t)mm * a.R, *row = a.w2 + (size_t)max(own, 0) * a.R;
  double dot = 0.0;
  for (int i = j; i < a.R; i += 64) dot += (double)bf_one(emb[i]) * (double)bf_one(row[i]);
  float top = -INFINITY, sum = 0.0f;
  for (int s0 = j; s0 < a.slabs; s0 += 8 * 64) {
    f32x2_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      p[i] = s0 + 64 * i < a.slabs ? a.parts[(size_t)(s0 + 64 * i) * a.M + mm] : (f32x2_t){-INFINITY, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) join(top, sum, p[i][0], p[i][1], h);
  }
#pragma unroll
  for (int sh = 4; sh <= 32; sh <<= 1) {
    const float m2 = __shfl_xor(top, sh), s2 = __shfl_xor(sum, sh);
    join(top, sum, m2, s2, h);
    dot += __shfl_xor(dot, sh);
  }
  __shared__ f32x2_t part[4][4];
  __shared__ double dots[4][4];
  if ((tid & 63) < 4) {
    part[tid >> 6][tid & 3] = (f32x2_t){top, sum};
    dots[tid >> 6][tid & 3] = dot;
  }
  __syncthreads();
  if (tid >= 64) return;   // (16 lanes of the first wave do the same for each row-step)
  top = part[0][tid & 3][0];
  sum = part[0][tid & 3][1];
  dot = dots[0][tid & 3];
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    join(top, sum, part[i][tid & 3][0], part[i][tid & 3][1], h);
    dot += dots[i][tid & 3];
  }
  // mult / T in full: the pass's factor is a binary32 number, which only the sum's
  // distances to the largest logit feel
  const float T = a.temperature ? a.temperature[mm / a.k] : 1.0f;
  const double full = (T == 0.0f ? 1.0 : 1.0 / (double)T) * (CAP ? 1.0 : (double)a.mult);
  const double by = h == MOST || h == 0x1p-149f ? (double)h * 0.693147180559945309 : fabs(full);
  const double x = (double)base + dot;
  const double z = (CAP ? (double)a.cap * tanh((double)a.mult * x * (double)a.inv_cap) : x) * (heat < 0.0f ? -1.0 : 1.0);
  const double rest = log((double)sum);
  double lse = (double)top * by + rest, d = (z - (double)top) * by - rest;
  const bool far = own >= 0 && fabs(lse) > (double)FAR - 24.0;   // (at least what the gradients take for far)
  if (__ballot(far) != 0) {
    // the token's logit as the pass had it, to which its distance is exact: the
    // same products in the same order, in rows and columns i of row-step i % 4
    const Transform f(a);
    const int li = tid & 15, lg = tid >> 4;
    f32x4_t p = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < a.R; i += 32) {
      bf16x8_t A = {}, B = {};
      if (i + lg * 8 < a.R) {
        A = *(const bf16x8_t*)(row + i + lg * 8);
        B = *(const bf16x8_t*)(emb + i + lg * 8);
      }
      p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B, p, 0, 0, 0);
    }
    float now = li & 2 ? (li & 1 ? p[3] : p[2]) : (li & 1 ? p[1] : p[0]);
    now += base;
    if (CAP) now = f.capped(now);
    if (heat < 0.0f) now = -now;
    if (far) {
      // (rounded as the gradients round it, which a factor of both does)
      lse = (double)(top * fabsf(factor(inverse_temperature(a, mm / a.k) * (CAP ? 1.0f : a.mult)))) + rest;
      d = ((double)now - (double)top) * by - rest;
    }
  }
  if (tid >= 4 || m >= a.M) return;
  if (own < 0) {
    a.logprobs[m] = a.lse[m] = 0.0f;
    return;
  }
  a.lse[m] = (float)lse;
  // (a masked token, unless the row-step is NaN; a row-step of nothing but masks is not)
  a.logprobs[m] = z == -INFINITY && lse == lse ? -INFINITY : d > 0.0 ? 0.0f : (float)d;
}

// ---------------------------------------------------------------- the loss

// One workgroup: N first, then the terms; sums in binary64 in a fixed order. Bound
// by the latency of its loads and steps: a thread's first row-step is loaded while
// N is counted, and the three sums are joined at once.
constexpr int LT = 1024;

template <int N>
__device__ __forceinline__ void block_sums(double (&v)[N], double (&red)[LT / 64][N]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int sh = 32; sh >= 1; sh >>= 1) v[i] += __shfl_xor(v[i], sh);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[wave][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0;
#pragma unroll
  for (int w = 0; w < LT / 64; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += red[w][i];
}

__global__ __launch_bounds__(LT) void policy_loss_kernel(
    const float* logprobs, const float* old, const float* ref, const float* advantages,
    const int64_t* tokens, const int32_t* lengths, int M, int k, int V, float clip_low,
    float clip_high, float beta, float* stats, float* grad) {
  __shared__ double count[LT / 64][1], red[LT / 64][3];
  const int tid = threadIdx.x, first = min(tid, M - 1);
  const float lp0 = logprobs[first], old0 = old[first], adv0 = advantages[first], ref0 = ref ? ref[first] : 0.0f;
  int mine = 0;
  for (int m = tid; m < M; m += LT) mine += scored(tokens, lengths, m, k, V);
  double n[1] = {(double)mine};
  block_sums(n, count);
  const double inv = n[0] > 0.0 ? 1.0 / n[0] : 0.0;
  const double low = 1.0 - (double)clip_low, high = 1.0 + (double)clip_high, b = (double)beta;
  double s0 = 0.0, s1 = 0.0;
  int held_n = 0;
  for (int m = tid; m < M; m += LT) {
    if (!scored(tokens, lengths, m, k, V)) {
      grad[m] = 0.0f;
      continue;
    }
    const bool loaded = m == first;
    const double lp = (double)(loaded ? lp0 : logprobs[m]), adv = (double)(loaded ? adv0 : advantages[m]);
    const double before = (double)(loaded ? old0 : old[m]);
    // (equal log-probabilities are 0 apart, two of a masked token also)
    const double gone = before == lp ? 0.0 : lp - before;
    // (an advantage of 0 takes ratio 0: an infinite one would make NaN of it)
    const double ratio = adv == 0.0 ? 0.0 : exp(gone);
    const double held = (ratio < low ? low : ratio > high ? high : ratio) * adv;   // 0 where adv is
    const double open = ratio * adv;
    const bool clipped = held < open;
    double g = clipped ? 0.0 : -open;
    s0 += clipped ? held : open;
    held_n += clipped;
    if (b != 0.0 || ref) {
      const double at = (double)(loaded ? ref0 : ref[m]);
      const double gap = at == lp ? 0.0 : at - lp, e = expm1(gap);
      s1 += gap == INFINITY ? gap : e - gap;
      if (b != 0.0) g -= b * e;
    }
    grad[m] = (float)(g * inv);
  }
  double sums[3] = {s0, s1, (double)held_n};
  block_sums(sums, red);
  const double surrogate = sums[0] * inv, kl = sums[1] * inv, share = sums[2] * inv;
  if (tid == 0) {
    stats[0] = (float)((b != 0.0 ? b * kl : 0.0) - surrogate);
    stats[1] = (float)surrogate;
    stats[2] = (float)kl;
    stats[3] = (float)share;
  }
}

// ---------------------------------------------------------------- the gradients
//
// Two launches, each a pass over the vocabulary.
//
// grad_base_kernel: a workgroup takes TB tokens and a split of the vocabulary,
// a tile at a time: the logits again (w2 rows from LDS, the tokens'
// embeddings in registers), d in place of the base logits in LDS, d out to
// grad_base, and d times w2 into the tokens' embedding gradients, which stay
// in registers over the whole split. The second product needs w2 with the
// vocabulary along the lane, and reads it from the same LDS tile with the
// transposing read. It leaves the gathered embeddings, and grad_w1 zeroed.
//
// grad_tables_kernel: for grad_w2 a workgroup takes a tile of the vocabulary
// and runs over all tokens, d read back from grad_base and the gathered
// embeddings, both through LDS with transposing reads; for grad_w1 one adds up
// the splits of every row-step fed by one token.
//
// Measured (V = 163840, rank 256, no cap but where it is named): 320 tokens,
// grad_base_kernel 94-106 us (2.9 TB/s of the logits, d and the tables), with the soft
// cap 111-131, and grad_tables_kernel 44-52 (3.7 TB/s); 2048 tokens 462-484 us (3.0
// TB/s, 730 TF) and 235-242 (3.2 TB/s, 720 TF); at rank 64 263-281 and 148-158 us
// (5.0 TB/s both). At rank 256 and 2048 tokens the first took 407 us without its
// arithmetic and 270 without its stores as well: it waits for loads and stores in
// turn (with three buffers each barrier waits for the stores of d too), with the
// matrix units 34 % and the LDS 29 % busy.
//
// Row-steps fed by one token are added up one after another by one workgroup
// (sum_w1), as the own d of one token's row-steps are (rests): backward of 320 x
// 163840 x 256 takes 166 us where few share a token, 283 with one prev for all rows,
// 769 with one token throughout; of 2048 745, 950 and 3660; 745 with a prev for 8 rows.
//
// The base logits and d are each read once, and past the caches: so d stays in
// the 256 MB cache between the launches where it fits (320 x 163840 x 256 with
// the soft cap 176 -> 162 us of backward, 2048 tokens at rank 64 464 -> 422; d
// stored past them as well: 16 x 5 x 129280 x 256 68 -> 76).
//
// Writing d between the two products costs a bf16 rounding, which the matrix
// units' operands need anyway, and no traffic of its own: it is grad_base. The
// token's own d, which is larger than all the others of its row-step together,
// enters both products whole: what its rounding left off is added as two rows
// scaled in fp32 (without, the gradients of a short block were twice as far off).

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

// Four rows x 16 columns of 16-bit values per 16 lanes, transposed: lane i
// gives the address of row i / 4, columns 4 (i % 4).. and receives column i.
__device__ __forceinline__ s16x4_t read_transposed(const uint8_t* at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)at);
}

__device__ __forceinline__ bf16x8_t both(s16x4_t lo, s16x4_t hi) {
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// A workgroup of 8 waves and NB LDS buffers, each a tile of VT w2 rows and of the
// tokens' base logits, one barrier a tile: after it a wave stores d of tile i - 1,
// asks for tile i + NB - 2, gathers tile i - 1 and differentiates tile i. (The two
// waves of a SIMD doing the last two in opposite order, so that one's exponentials
// run beside the other's products, measured no faster; two barriers a tile and so
// one more tile on its way 9 % slower.)
//
// Differentiating, WV waves side by side over the tile's vocabulary and the rest
// over the tokens: a wave's w2 rows come from LDS, its tokens' embeddings lie in
// registers, so that four over the vocabulary halve the LDS reads where there are
// registers for it (64 tokens; two measured 172 us for 169 at 320 x 163840 x 256).
// Gathering, NRW waves over the rank (RT tiles of 16) and the rest over the tokens
// (T2 tiles).
template <int R, int TB, bool CAP>
struct Gradient {
  typedef Rank<R> Q;
  static constexpr int VT = R <= 256 ? 64 : 32;
  static constexpr int WV = VT == 64 && TB == 64 ? 4 : 2, NV = VT / 16 / WV, T1 = TB / 16 / (8 / WV);
  static constexpr int RT = R >= 64 ? 4 : R / 16, NRW = R / 16 / RT;
  static constexpr int T2 = TB / 16 / (8 / NRW) > 0 ? TB / 16 / (8 / NRW) : 1;
  static constexpr int GD = VT / 8;                              // 16-byte groups of a token's d
  static constexpr int W = VT * R * 2, D = TB * VT * 2;          // bytes of the two tiles
  static constexpr int NLW = W / 1024, NLD = D / 1024;           // loads of 64 lanes
  static constexpr int LW = (NLW + 7) / 8, LD = (NLD + 7) / 8;   // of a wave, at most
  static constexpr int LEAST = NLW / 8 + NLD / 8;                // and at least
  static constexpr int NB = 4 * (W + D) <= 163840 ? 4 : 3;
  const ScoreArgs& a;
  const Transform f;
  int tid, lane, li, lg, wave, m0;
  // this lane's places in LDS and byte offsets of its loads
  int at_row, at_d, at_b, at_t;
  uint32_t w_off[2], d_off[LD];
  // this lane's tokens, one of each 16
  bf16x8_t emb[T1][Q::KS];
  int own[T1];
  float heat[T1], scale[T1], lse2[T1];   // (scale holds the factor mult, without a cap heat also)
  bool odd;                              // (of the wave) some token's scale is INFINITE, or its lse far

  // A token whose lse is past FAR: heat holds 1 / T and lse2 twice the lse, which is
  // how it is known (lse log2(e) of another is below).
  static __device__ __forceinline__ bool far(float lse2) { return fabsf(lse2) > 1.5f * FAR; }

  // An infinite gradient's scale. It is finite so that what has no mass or no slope
  // gets 0 of it, and not NaN; all else gets infinity.
  static constexpr float INFINITE = 0x1.fffffep127f;
  static __device__ __forceinline__ float finite(float scale) {
    if (__builtin_isinf(scale)) return __builtin_copysignf(INFINITE, scale);
    return fabsf(scale) == INFINITE ? __builtin_copysignf(0x1.fffffcp127f, scale) : scale;
  }

  // 16-byte group c of w2 row v is at place c ^ key(v): 16 rows side by side
  // spread over all banks (a transposing read has no preference). Group c of
  // token t's d is at place c ^ key_d(t): 16 tokens side by side likewise.
  static __device__ __forceinline__ int key(int v) { return v & Q::KEY; }
  static __device__ __forceinline__ int key_d(int t) { return VT == 64 ? t & 7 : (t >> 1) & 3; }

  __device__ __forceinline__ void place() {
    const int wv = wave % WV, wt = wave / WV, row = wv * NV * 16 + li;
    at_row = row * R * 2 + (((R >= 32 ? lg : lg & 1) ^ key(row)) * 16);
    at_d = (wt * T1 * 16 + li) * VT * 2 + ((wv * NV * 2 + (lg >> 1)) ^ key_d(li)) * 16 + (lg & 1) * 8;
    const int wr = wave % NRW, w2 = wave / NRW;
    at_b = (w2 * T2 * 16 + li) * VT * 2 + (lg ^ key_d(li)) * 16;
    const int v = lg * 8 + (li >> 2);
    at_t = v * R * 2 + ((wr * RT * 2 + ((li >> 1) & 1)) ^ key(v)) * 16 + (li & 1) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // (a wave's loads are 8 apart: at R = 512 every other has another permutation)
      const int at = (wave + 8 * i) * 64 + lane;
      w_off[i] = (uint32_t)(lane / Q::G) * R * 2 + ((at % Q::G) ^ key(at / Q::G)) * 16;
    }
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int at = i * 512 + tid, t = at / GD;
      d_off[i] = (uint32_t)min(t, a.M - 1 - m0) * (uint32_t)a.V * 2 + ((at % GD) ^ key_d(t)) * 16;
    }
  }

  __device__ __forceinline__ void request(int tile, uint8_t* __restrict__ w, uint8_t* __restrict__ d) const {
    if (tile * VT + VT <= a.V) {
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int n = wave + 8 * i;
        if (NLD % 8 != 0 && n >= NLD) break;
        load_lds<true>(a.base + (size_t)m0 * a.V + tile * VT, d_off[i], d + n * 1024);
      }
#pragma unroll
      for (int i = 0; i < LW; ++i) {
        const int n = wave + 8 * i;
        if (NLW % 8 != 0 && n >= NLW) break;
        load_lds((const uint8_t*)(a.w2 + (size_t)tile * VT * R) + n * 1024, w_off[i & 1], w + n * 1024);
      }
      return;
    }
    // the last tile, if it is a smaller one: rows past the last entry repeat
    // it, columns past it are any (the lane is opaque, so that none of this is
    // computed ahead and held)
    int l = lane;
    asm volatile("" : "+v"(l));
#pragma unroll 1
    for (int n = wave; n < NLD; n += 8) {
      const int at = n * 64 + l, t = at / GD, v = tile * VT + ((at % GD) ^ key_d(t)) * 8;
      load_lds(a.base + (size_t)min(m0 + t, a.M - 1) * a.V + (v < a.V ? v : 0), d + n * 1024);
    }
#pragma unroll 1
    for (int n = wave; n < NLW; n += 8) {
      const int at = n * 64 + l, r = at / Q::G;
      load_lds(a.w2 + (size_t)min(tile * VT + r, a.V - 1) * R + ((at % Q::G) ^ key(r)) * 8, w + n * 1024);
    }
  }

  // d of the tile in place of its base logits.
  __device__ __forceinline__ void differentiate(int tile, const uint8_t* __restrict__ w, uint8_t* __restrict__ d) const {
#pragma unroll
    for (int n = 0; n < NV; ++n) differentiate(tile, n, w, d);
  }

  __device__ __forceinline__ void differentiate(int tile, int n, const uint8_t* __restrict__ w,
                                                uint8_t* __restrict__ d) const {
    f32x4_t z[T1];
#pragma unroll
    for (int i = 0; i < T1; ++i) z[i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    // (operands are read one step ahead, and the barriers keep the scheduler
    // from reading more of them ahead than there are registers)
    auto row = [&](int s) {
      const bf16x8_t A = *(const bf16x8_t*)(w + (at_row ^ ((s & 3) * 64)) + (s >> 2) * 256 + n * 16 * R * 2);
      return R >= 32 || lg < 2 ? A : (bf16x8_t){};
    };
    bf16x8_t A = row(0);
#pragma unroll
    for (int s = 0; s < Q::KS; ++s) {
      const bf16x8_t next = row(s + 1 < Q::KS ? s + 1 : s);
#pragma unroll
      for (int i = 0; i < T1; ++i) z[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, emb[i][s], z[i], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      A = next;
    }
    const int v = tile * VT + (wave % WV) * NV * 16 + n * 16 + lg * 4;   // this lane's four entries
#pragma unroll
    for (int i = 0; i < T1; ++i) {
      u32x2_t* at = (u32x2_t*)(d + (at_d ^ (n * 32)) + i * 16 * VT * 2);
      const u32x2_t x = *at;
      z[i] += (f32x4_t){bf_lo(x[0]), bf_hi(x[0]), bf_lo(x[1]), bf_hi(x[1])};   // (as in the scoring pass: the logits come out equal)
      float g[4], u[4], slope[4];   // u: the power of 2 that the probability is
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        slope[e] = 1.0f;
        u[e] = CAP ? f.near(z[i][e], &slope[e]) * heat[i] - lse2[i] : __builtin_fmaf(z[i][e], heat[i], -lse2[i]);
      }
      if (CAP && __builtin_expect(f.wide, 0)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = f.exact(z[i][e]) * heat[i] - lse2[i];
      }
      if (__builtin_expect(odd, 0)) {
        const bool apart = far(lse2[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (z / T is rounded as in the lse, the doubling is exact)
          const float x = (CAP ? f.capped(z[i][e]) : z[i][e]) * heat[i], t = __builtin_fmaf(x, 2.0f, -lse2[i]) * (0.5f * LOG2E);
          u[e] = apart ? (t > 0.0f ? 0.0f : t) : u[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = CAP ? scale[i] * slope[e] * __builtin_amdgcn_exp2f(u[e]) : scale[i] * __builtin_amdgcn_exp2f(u[e]);
      const unsigned hit = (unsigned)(own[i] - v);
      if (__builtin_expect(__ballot(hit < 4u) != 0, 0)) {
        // the token's own entry (unless its logit is masked): scale holds -g / T
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (hit == (unsigned)e) {
            if ((CAP ? z[i][e] : z[i][e] * heat[i]) != -INFINITY) g[e] -= scale[i] * slope[e];
            const float stored = bf_lo(pack_bf16(g[e], 0.0f));
            a.rest[m0 + ((wave / WV) * T1 + i) * 16 + li] =
                __builtin_isinf(stored) || fabsf(scale[i]) == INFINITE ? 0.0f : g[e] - stored;
          }
        }
      }
      if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (fabsf(scale[i]) == INFINITE && g[e] != 0.0f) g[e] *= INFINITY;
      }
      const bool out = own[i] < 0 || v >= a.V;
      *at = (u32x2_t){out ? 0u : pack_bf16(g[0], g[1]), out ? 0u : pack_bf16(g[2], g[3])};
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // d out to grad_base.
  __device__ __forceinline__ void store(int tile, const uint8_t* __restrict__ d) const {
    uint16_t* out = a.grad_base + (size_t)m0 * a.V + tile * VT;
    asm volatile("" : "+s"(out));
    const int left = a.V - tile * VT;   // the tile's entries
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      uint32_t off = d_off[i];
      asm volatile("" : "+v"(off));
      const int at = i * 512 + tid, t = at / GD;
      if ((NLD % 8 == 0 || at * 16 < D) && t < a.M - m0 && (left >= VT || ((at % GD) ^ key_d(t)) * 8 < left))
        *(__attribute__((address_space(1))) u32x4_t*)((__attribute__((address_space(1))) uint8_t*)out + off) =
            *(const u32x4_t*)(d + at * 16);
    }
  }

  // d times w2 into the embeddings' gradients.
  __device__ __forceinline__ void gather(const uint8_t* __restrict__ w, const uint8_t* __restrict__ d,
                                         f32x4_t (&acc)[RT][T2]) const {
    if ((wave / NRW) * T2 * 16 >= TB) return;
    int from = at_t;   // (opaque: its variants are made where they are used, not held)
    asm volatile("" : "+v"(from));
    auto column = [&](int n) {
      // (a wave's first group is a multiple of 8 where it has four tiles)
      const int at = (from ^ (n % RT * 32)) + n / RT * 32 * R * 2;
      return both(read_transposed(w + at), read_transposed(w + ((at ^ ((4 & Q::KEY) * 16)) + 4 * R * 2)));
    };
    bf16x8_t A = column(0);
#pragma unroll
    for (int s = 0; s < VT / 32; ++s) {
      bf16x8_t B[T2];
#pragma unroll
      for (int i = 0; i < T2; ++i) B[i] = *(const bf16x8_t*)(d + (at_b ^ (s * 64)) + i * 16 * VT * 2);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int n = s * RT + j;
        const bf16x8_t next = column(n + 1 < VT / 32 * RT ? n + 1 : n);
#pragma unroll
        for (int i = 0; i < T2; ++i) acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B[i], acc[j][i], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        A = next;
      }
    }
  }

  // Waits for tile i. With four buffers a wave has, since its loads, stored tile
  // i - 2 (if there is one, and every token of the block is one: else perhaps
  // not) and asked for tile i + 1.
  __device__ __forceinline__ void wait(int i, int begin, int end) const {
    if (NB > 3 && i + 1 < end) {
      if (i - 2 >= begin && m0 + TB <= a.M && NLD % 8 == 0) barrier_but<LEAST + LD>();
      else barrier_but<LEAST>();
    } else {
      barrier_but<0>();
    }
  }

  // Tile i, whose loads are under way, and tile i - 1, whose d is written.
  __device__ __forceinline__ void step(int i, int begin, int end, const uint8_t* __restrict__ w_before,
                                       const uint8_t* __restrict__ d_before, const uint8_t* __restrict__ w,
                                       uint8_t* __restrict__ d, uint8_t* __restrict__ w_next,
                                       uint8_t* __restrict__ d_next, f32x4_t (&acc)[RT][T2]) const {
    wait(i, begin, end);
    store(i - 1, d_before);
    __builtin_amdgcn_sched_barrier(0);   // (the order that the waits count on)
    if (i + NB - 2 < end) request(i + NB - 2, w_next, d_next);
    gather(w_before, d_before, acc);
    differentiate(i, w, d);
  }

  __device__ __forceinline__ void finish(int i, const uint8_t* __restrict__ w, const uint8_t* __restrict__ d,
                                         f32x4_t (&acc)[RT][T2]) const {
    barrier_but<0>();
    store(i, d);
    gather(w, d, acc);
  }
};

template <int R, int TB, bool CAP>
__global__ __launch_bounds__(512, 2) void grad_base_kernel(ScoreArgs a) {
  typedef Gradient<R, TB, CAP> T;
  typedef Rank<R> Q;
  __shared__ __attribute__((aligned(16))) uint8_t w0[T::W], w1[T::W], w2[T::W], w3[T::NB > 3 ? T::W : 16],
      d0[T::D], d1[T::D], d2[T::D], d3[T::NB > 3 ? T::D : 16];
  const int blocks = (a.M + TB - 1) / TB;
  int split, block;
  if (a.splits % 8 == 0) {   // a split's workgroups on one XCD share its w2 rows
    const int local = blockIdx.x >> 3;
    split = (local / blocks) * 8 + (blockIdx.x & 7);
    block = local % blocks;
  } else {
    split = blockIdx.x % a.splits;
    block = blockIdx.x / a.splits;
  }
  T g{a, Transform(a)};
  g.tid = threadIdx.x;
  g.lane = g.tid & 63;
  g.li = g.lane & 15;
  g.lg = g.lane >> 4;
  g.wave = __builtin_amdgcn_readfirstlane(g.tid >> 6);
  g.m0 = block * TB;
  g.place();
  const int begin = split * a.tiles_per;
  const int end = min(begin + a.tiles_per, (a.V + T::VT - 1) / T::VT);
#pragma unroll
  for (int i = 0; i < T::T1; ++i) {
    const int m = g.m0 + ((g.wave / T::WV) * T::T1 + i) * 16 + g.li, mm = min(m, a.M - 1);
    const RowStep s = row_step<true>(a, mm);
    g.own[i] = m < a.M ? s.own : -1;
    const bool far = fabsf(s.lse) > FAR;
    g.heat[i] = factor((far ? s.inverse : s.heat) * (CAP ? 1.0f : a.mult));
    g.scale[i] = T::finite(-s.scale * a.mult);
    g.lse2[i] = s.lse * (far ? 2.0f : LOG2E);
    const uint16_t* row = a.w1 + (size_t)s.fed * R + g.lg * 8;   // (d is 0 where it does not take part)
#pragma unroll
    for (int s = 0; s < Q::KS; ++s)
      g.emb[i][s] = R >= 32 || g.lg < 2 ? *(const bf16x8_t*)(row + s * 32) : (bf16x8_t){};
  }
  bool odd = false;
#pragma unroll
  for (int i = 0; i < T::T1; ++i) odd = odd || fabsf(g.scale[i]) == T::INFINITE || T::far(g.lse2[i]);
  g.odd = __ballot(odd) != 0;
  f32x4_t acc[T::RT][T::T2];
#pragma unroll
  for (int j = 0; j < T::RT; ++j)
#pragma unroll
    for (int i = 0; i < T::T2; ++i) acc[j][i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  g.request(begin, w0, d0);
  __builtin_amdgcn_sched_barrier(0);
  if (T::NB > 3 && begin + 1 < end) g.request(begin + 1, w1, d1);
  g.wait(begin, begin, end);
  int i = begin + 1;
  if constexpr (T::NB > 3) {
    if (begin + 2 < end) g.request(begin + 2, w2, d2);
    g.differentiate(begin, w0, d0);
    for (; i + 3 < end; i += 4) {
      g.step(i, begin, end, w0, d0, w1, d1, w3, d3, acc);
      g.step(i + 1, begin, end, w1, d1, w2, d2, w0, d0, acc);
      g.step(i + 2, begin, end, w2, d2, w3, d3, w1, d1, acc);
      g.step(i + 3, begin, end, w3, d3, w0, d0, w2, d2, acc);
    }
    if (i == end) {
      g.finish(end - 1, w0, d0, acc);
    } else {
      g.step(i, begin, end, w0, d0, w1, d1, w3, d3, acc);
      if (i + 1 == end) {
        g.finish(end - 1, w1, d1, acc);
      } else {
        g.step(i + 1, begin, end, w1, d1, w2, d2, w0, d0, acc);
        if (i + 2 == end) {
          g.finish(end - 1, w2, d2, acc);
        } else {
          g.step(i + 2, begin, end, w2, d2, w3, d3, w1, d1, acc);
          g.finish(end - 1, w3, d3, acc);
        }
      }
    }
  } else {
    if (begin + 1 < end) g.request(begin + 1, w1, d1);
    g.differentiate(begin, w0, d0);
    for (; i + 2 < end; i += 3) {
      g.step(i, begin, end, w0, d0, w1, d1, w2, d2, acc);
      g.step(i + 1, begin, end, w1, d1, w2, d2, w0, d0, acc);
      g.step(i + 2, begin, end, w2, d2, w0, d0, w1, d1, acc);
    }
    if (i == end) {
      g.finish(end - 1, w0, d0, acc);
    } else {
      g.step(i, begin, end, w0, d0, w1, d1, w2, d2, acc);
      if (i + 1 == end) {
        g.finish(end - 1, w1, d1, acc);
      } else {
        g.step(i + 1, begin, end, w1, d1, w2, d2, w0, d0, acc);
        g.finish(end - 1, w2, d2, acc);
      }
    }
  }
  if ((g.wave / T::NRW) * T::T2 * 16 < TB) {
#pragma unroll
    for (int j = 0; j < T::RT; ++j)
#pragma unroll
      for (int i = 0; i < T::T2; ++i) {
        const int m = g.m0 + ((g.wave / T::NRW) * T::T2 + i) * 16 + g.li;
        if (m < a.M)
          *(f32x4_t*)(a.grad_emb + ((size_t)split * a.M + m) * R + ((g.wave % T::NRW) * T::RT + j) * 16 + g.lg * 4) = acc[j][i];
      }
  }
  // for the next launch: the block's embeddings, a part in each split, what it
  // needs of its row-steps, and a part of grad_w1's zeros
  for (int i = split * 512 + g.tid; i < TB * Q::G; i += a.splits * 512) {
    const int m = g.m0 + i / Q::G;
    if (m < ((a.M + 63) & ~63)) gather_embedding<true>(a, m, i % Q::G);
  }
  if (split == 0 && g.tid < TB && g.m0 + g.tid < a.M) {
    const RowStep s = row_step<true>(a, g.m0 + g.tid);
    a.own[g.m0 + g.tid] = s.own;
    a.fed[g.m0 + g.tid] = s.fed;
  }
  for (size_t i = (size_t)blockIdx.x * 512 + g.tid; i < (size_t)a.V * Q::G; i += (size_t)gridDim.x * 512)
    __builtin_nontemporal_store((u32x4_t){0u, 0u, 0u, 0u}, (u32x4_t*)a.grad_w1 + i);
}

// grad_w2 = d^T emb over all tokens, 32 at a time. A wave has RW of the rank x
// VW of the vocabulary; A operand: the rank, so that a lane holds neighbouring
// rank entries of one vocabulary row: rows i of the tile pair (2p, 2p + 1)
// are rank entries 32 p + 8 (i / 4) + 4 ((n + i / 4) % 2) + i % 4, which
// also lets a transposing read use all banks.
template <int R>
struct Outer {
  typedef Rank<R> Q;
  static constexpr int WR = R >= 512 ? 4 : R >= 128 ? 2 : 1;   // waves over the rank
  static constexpr int RW = R / WR, NR = RW / 16;
  static constexpr int VB = R >= 512 ? 64 : 128;               // vocabulary of a workgroup
  static constexpr int VW = VB / (4 / WR), NV = VW / 16;
  static constexpr int GV = VB / 8;
  static constexpr int LE = (Q::G / 2 + 3) / 4, LD = GV / 8;    // loads of a wave per 32 tokens
  const ScoreArgs& a;
  int tid, lane, li, lg, wave, v0;
  uint32_t e_off[2], d_off;

  static __device__ __forceinline__ int key(int t) { return ((t & 3) << 1) | ((t >> 3) & 1); }

  __device__ __forceinline__ void place() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // (token rows of one load, and those of the loads 4 or, at R = 512, 8
      // further on, whose permutation is another)
      const int at = (wave + (R >= 512 ? 8 : 4) * i) * 64 + lane, t = at / Q::G;
      e_off[i] = (uint32_t)(lane / Q::G) * R * 2 + ((at % Q::G) ^ (key(t) & Q::KEY)) * 16;
    }
    const int t = wave * (64 / GV) + lane / GV, c = (lane % GV) ^ key(t);
    // (columns past the last entry repeat the first ones)
    d_off = (uint32_t)t * (uint32_t)a.V * 2 + (v0 + c * 8 < a.V ? c * 16 : 0);
  }

  __device__ __forceinline__ void request(int c, uint8_t* __restrict__ e, uint8_t* __restrict__ d) const {
#pragma unroll
    for (int i = 0; i < LE; ++i) {
      const int n = wave + 4 * i;
      if (Q::G / 2 % 4 != 0 && n >= Q::G / 2) break;
      load_lds(a.emb + (size_t)c * 32 * R + n * 512, e_off[R >= 512 ? (i >> 1) & 1 : i & 1], e + n * 1024);
    }
    if (c * 32 + 32 <= a.M) {
#pragma unroll
      for (int i = 0; i < LD; ++i)
        load_lds<true>(a.grad_base + ((size_t)c * 32 + i * (256 / GV)) * a.V + v0, d_off, d + (wave + 4 * i) * 1024);
      return;
    }
    // past the last row-step zeros, which its embedding's padding is (products of 0
    // with another row's d would be NaN where that is infinite)
    int l = lane;
    asm volatile("" : "+v"(l));
#pragma unroll 1
    for (int n = wave; n < GV / 2; n += 4) {
      const int at = n * 64 + l, t = at / GV, v = v0 + ((at % GV) ^ key(t)) * 8;
      load_lds(c * 32 + t < a.M ? a.grad_base + (size_t)(c * 32 + t) * a.V + (v < a.V ? v : 0) : a.emb + (size_t)a.M * R,
               d + n * 1024);
    }
  }

  // What the roundings of the tokens' own d left off, for those of this wave's
  // entries: looked for in rising row-step, while the first loads are under way.
  __device__ __forceinline__ void rests(f32x4_t (&acc)[NR][NV]) const {
    const int r0 = (wave % WR) * RW, vv = v0 + (wave / WR) * VW;
#pragma unroll 1
    for (int i0 = 0; i0 < a.M; i0 += 512) {
      unsigned at[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) at[k] = (unsigned)(a.own[min(i0 + k * 64 + lane, a.M - 1)] - vv);
      uint64_t left[8], any = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) any |= left[k] = __ballot(at[k] < (unsigned)VW && i0 + k * 64 + lane < a.M);
      if (any == 0) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll 1
        for (; left[k]; left[k] &= left[k] - 1) {
          const int l = __builtin_ctzll(left[k]);
          add_rest(i0 + k * 64 + l, __builtin_amdgcn_readlane((int)at[k], l), r0, acc);
        }
    }
  }

  // (the other tiles of the wave take 0 of it, which is cheaper than a choice)
  __device__ __forceinline__ void add_rest(int m, int v, int r0, f32x4_t (&acc)[NR][NV]) const {
    const float rest = (v & 15) == li ? a.rest[m] : 0.0f;
    const uint16_t* row = a.emb + (size_t)m * R + r0;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const u32x2_t x = *(const u32x2_t*)(row + (NR == 1 ? lg * 4 : 32 * (n >> 1) + 8 * lg + 4 * ((n + lg) & 1)));
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const float f = k == v >> 4 ? rest : 0.0f;
        acc[n][k] += (f32x4_t){f * bf_lo(x[0]), f * bf_hi(x[0]), f * bf_lo(x[1]), f * bf_hi(x[1])};
      }
    }
  }

  __device__ __forceinline__ void step(int c, int chunks, const uint8_t* __restrict__ e, const uint8_t* __restrict__ d,
                                       uint8_t* __restrict__ e_next, uint8_t* __restrict__ d_next,
                                       f32x4_t (&acc)[NR][NV]) const {
    barrier_but<0>();
    if (c + 1 < chunks) request(c + 1, e_next, d_next);
    const int r0 = (wave % WR) * RW, vv = (wave / WR) * VW;
    bf16x8_t B[NV];
    const int t = lg * 8 + (li >> 2), q = li & 3;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int g = (vv + n * 16) / 8 + (q >> 1);
      const s16x4_t lo = read_transposed(d + t * VB * 2 + (g ^ key(t)) * 16 + (q & 1) * 8);
      const s16x4_t hi = read_transposed(d + (t + 4) * VB * 2 + (g ^ key(t + 4)) * 16 + (q & 1) * 8);
      B[n] = both(lo, hi);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int r = r0 + (NR == 1 ? q * 4 : 32 * (n >> 1) + 8 * q + 4 * ((n + q) & 1));
      const int g = r >> 3, h = (r >> 2) & 1;
      const s16x4_t lo = read_transposed(e + t * R * 2 + (g ^ (key(t) & Q::KEY)) * 16 + h * 8);
      const s16x4_t hi = read_transposed(e + (t + 4) * R * 2 + (g ^ (key(t + 4) & Q::KEY)) * 16 + h * 8);
      const bf16x8_t A = both(lo, hi);
#pragma unroll
      for (int v = 0; v < NV; ++v) acc[n][v] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B[v], acc[n][v], 0, 0, 0);
    }
  }
};

// One workgroup per row-step; that of the first row-step that takes part and is
// fed by its token adds up all of them, in rising row-step: R / 4 threads across
// and the rest over the splits. The row-step's own sums are on their way while
// the others' tokens are compared (that no other is fed by its token is the
// common case).
template <int R>
__device__ __forceinline__ void sum_w1(const ScoreArgs& a, int m, uint64_t* hits, f32x4_t* part) {
  const int tid = threadIdx.x;
  constexpr int across = R / 4, deep = 256 / across;
  const int x = tid % across, y = tid / across;
  const size_t stride = (size_t)a.M * across;
  auto splits_of = [&](int i) {
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    const f32x4_t* at = (const f32x4_t*)(a.grad_emb + (size_t)i * R) + x;
#pragma unroll 8
    for (int s = y; s < a.splits; s += deep) sum += at[s * stride];
    if (y == 0 && a.own[i] >= 0) {
      const u32x2_t row = ((const u32x2_t*)(a.w2 + (size_t)a.own[i] * R))[x];
      const float rest = a.rest[i];
      sum += (f32x4_t){rest * bf_lo(row[0]), rest * bf_hi(row[0]), rest * bf_lo(row[1]), rest * bf_hi(row[1])};
    }
    return sum;
  };
  f32x4_t sum = splits_of(m);
  if (a.own[m] < 0) return;
  const int row = a.fed[m];
  bool before = false, after = false;
  for (int i0 = 0; i0 < a.M; i0 += 256) {
    const int i = i0 + tid;
    const bool hit = i < a.M && i != m && a.fed[i] == row && a.own[i] >= 0;
    before = before || (hit && i < m);
    after = after || (hit && i > m);
    const uint64_t h = __ballot(hit);
    if ((tid & 63) == 0) hits[i >> 6] = h;
  }
  if (__syncthreads_or(before)) return;
  if (__syncthreads_or(after))
    for (int w = m >> 6; w < (a.M + 63) / 64; ++w)
      for (uint64_t left = hits[w]; left; left &= left - 1) sum += splits_of(w * 64 + __builtin_ctzll(left));
  part[tid] = sum;
  __syncthreads();
  if (y > 0) return;
  for (int j = 1; j < deep; ++j) sum += part[j * across + x];
  *(u32x2_t*)(a.grad_w1 + (size_t)row * R + x * 4) = (u32x2_t){pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
}

// The first M workgroups are grad_w1's (short, and waiting for memory most of the
// time: in a launch of their own they took 8 us after 320 tokens, 18 after 2048),
// the others a vocabulary tile each.
template <int R>
__global__ __launch_bounds__(256, 2) void grad_tables_kernel(ScoreArgs a) {
  typedef Outer<R> T;
  __shared__ __attribute__((aligned(16))) uint8_t e_one[32 * R * 2], e_two[32 * R * 2], d_one[32 * T::VB * 2],
      d_two[32 * T::VB * 2];
  if (blockIdx.x < (unsigned)a.M) {
    uint8_t *hits = R >= 512 ? e_one : d_one, *part = R >= 512 ? e_two : d_two;
    static_assert((R >= 512 ? sizeof(e_one) : sizeof(d_one)) >= MARKOV_MAX_TOKENS / 8, "");
    static_assert((R >= 512 ? sizeof(e_two) : sizeof(d_two)) >= 256 * sizeof(f32x4_t), "");
    sum_w1<R>(a, blockIdx.x, (uint64_t*)hits, (f32x4_t*)part);
    return;
  }
  T g{a};
  g.tid = threadIdx.x;
  g.lane = g.tid & 63;
  g.li = g.lane & 15;
  g.lg = g.lane >> 4;
  g.wave = __builtin_amdgcn_readfirstlane(g.tid >> 6);
  g.v0 = (blockIdx.x - a.M) * T::VB;
  g.place();
  g.request(0, e_one, d_one);
  f32x4_t acc[T::NR][T::NV];
#pragma unroll
  for (int n = 0; n < T::NR; ++n)
#pragma unroll
    for (int v = 0; v < T::NV; ++v) acc[n][v] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  g.rests(acc);
  const int chunks = (a.M + 31) / 32;
  int c = 0;
  for (; c + 1 < chunks; c += 2) {
    g.step(c, chunks, e_one, d_one, e_two, d_two, acc);
    g.step(c + 1, chunks, e_two, d_two, e_one, d_one, acc);
  }
  if (c < chunks) g.step(c, chunks, e_one, d_one, e_two, d_two, acc);
  const int r0 = (g.wave % T::WR) * T::RW, vv = g.v0 + (g.wave / T::WR) * T::VW;
#pragma unroll
  for (int v = 0; v < T::NV; ++v) {
    const int row = vv + v * 16 + g.li;
    if (row >= a.V) continue;
    uint16_t* out = a.grad_w2 + (size_t)row * R + r0;
    if constexpr (T::NR == 1) {
      *(u32x2_t*)(out + g.lg * 4) = (u32x2_t){pack_bf16(acc[0][v][0], acc[0][v][1]), pack_bf16(acc[0][v][2], acc[0][v][3])};
    } else {
#pragma unroll
      for (int n = 0; n < T::NR; n += 2) {
        const f32x4_t lo = g.lg & 1 ? acc[n + 1][v] : acc[n][v], hi = g.lg & 1 ? acc[n][v] : acc[n + 1][v];
        *(u32x4_t*)(out + 16 * n + g.lg * 8) =
            (u32x4_t){pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3]), pack_bf16(hi[0], hi[1]), pack_bf16(hi[2], hi[3])};
      }
    }
  }
}

// ---------------------------------------------------------------- host side

int check(const markov_shape_t* sh, int32_t k) {
  if (!sh) return MARKOV_ERR_NULL;
  if (sh->vocab > MARKOV_MAX_SCORED_VOCAB) return MARKOV_ERR_VOCAB;
  if (sh->rows < 1 || k < 1 || sh->vocab < 8 || (sh->vocab & 7)) return MARKOV_ERR_SHAPE;
  if (sh->rank < 16 || sh->rank > 512 || (sh->rank & (sh->rank - 1))) return MARKOV_ERR_RANK;
  if ((int64_t)sh->rows * k > MARKOV_MAX_TOKENS) return MARKOV_ERR_ROWS;
  return MARKOV_OK;
}

size_t aligned(size_t n) { return (n + 255) & ~(size_t)255; }

// How a call is split, and the workspace that this takes: a function of the
// shape alone.
struct Plan {
  int slabs, shares, block, splits, tiles_per;
  size_t rows_bytes, emb_bytes, bytes;
};

// Tokens of a workgroup of grad_base_kernel: their embeddings and gradients are
// held in registers. More share a w2 tile, fewer leave registers and LDS for more
// loads under way (backward of 320 x 163840 x 256 170 us with 64 and 196 with 128,
// of 512 230 and 229, of 768 366 and 321, of 2048 785 and 744).
int grad_tokens(int M, int rank) { return rank > 256 || M <= 512 ? 64 : 128; }

constexpr int ROW_ARRAYS = 4;   // of 4 bytes per row-step

Plan plan_of(const markov_shape_t* sh, int32_t k) {
  Plan p;
  const int M = sh->rows * k, slab = sh->rank <= 256 ? 256 : 128;
  p.slabs = (int)(((int64_t)sh->vocab + slab - 1) / slab);
  // as many workgroups as 256 CUs hold at once, two each (three up to rank 64,
  // one at rank 512): 2048 x 163840 x 256 252 us with two, 333 with one, 272 with
  // three; rank 64 159 with three, 169 with two, 177 with four; 1024 at rank 512
  // 346 with one, 351 with two
  const int64_t units = (int64_t)p.slabs * ((M + 31) / 32);
  p.shares = sh->rank <= 64 ? 768 : sh->rank <= 256 ? 512 : 256;
  if (units < p.shares) p.shares = (int)units;
  p.block = grad_tokens(M, sh->rank);
  const int tile = sh->rank <= 256 ? 64 : 32, tiles = (sh->vocab + tile - 1) / tile, blocks = (M + p.block - 1) / p.block;
  // a workgroup a CU, or two up to rank 32 (two also fit up to rank 128, with twice
  // as many partial sums: 320 x 163840 x 64 73 us with one, 82 with two, 2048 at
  // rank 32 423 and 407); the splits in eights to go round the XCDs
  const int most = (sh->rank <= 32 ? 512 : 256) / blocks;
  p.splits = most >= 8 ? most / 8 * 8 : most > 1 ? most : 1;
  if (p.splits > tiles) p.splits = tiles;
  p.tiles_per = (tiles + p.splits - 1) / p.splits;
  p.splits = (tiles + p.tiles_per - 1) / p.tiles_per;
  p.rows_bytes = aligned((size_t)M * 4);
  const size_t score = (size_t)p.slabs * M * 8, grad = (size_t)p.splits * M * sh->rank * 4;
  p.emb_bytes = aligned((size_t)((M + 63) & ~63) * sh->rank * 2);
  p.bytes = ROW_ARRAYS * p.rows_bytes + p.emb_bytes + aligned(score > grad ? score : grad);
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
  a.splits = p.splits;
  a.tiles_per = p.tiles_per;
  uint8_t* at = (uint8_t*)workspace;
  void** rows[ROW_ARRAYS] = {(void**)&a.fed, (void**)&a.own, (void**)&a.heat, (void**)&a.rest};
  for (void** r : rows) {
    *r = at;
    at += p.rows_bytes;
  }
  a.emb = (uint16_t*)at;
  at += p.emb_bytes;
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

int64_t rows_grid(const ScoreArgs& a) { return ((int64_t)((a.M + 63) & ~63) * (a.R / 8) + 255) / 256; }

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

template <int R, bool CAP>
ScoreKernel grad_base_kernel_of(int block) {
  if constexpr (R <= 256)
    if (block == 128) return grad_base_kernel<R, 128, CAP>;
  return grad_base_kernel<R, 64, CAP>;
}

template <bool CAP>
ScoreKernel grad_base_kernel_of(int rank, int block) {
  switch (rank) {
    case 16: return grad_base_kernel_of<16, CAP>(block);
    case 32: return grad_base_kernel_of<32, CAP>(block);
    case 64: return grad_base_kernel_of<64, CAP>(block);
    case 128: return grad_base_kernel_of<128, CAP>(block);
    case 256: return grad_base_kernel_of<256, CAP>(block);
    default: return grad_base_kernel_of<512, CAP>(block);
  }
}

ScoreKernel grad_tables_kernel_of(int rank, int* tile) {
  *tile = rank >= 512 ? Outer<512>::VB : Outer<256>::VB;
  switch (rank) {
    case 16: return grad_tables_kernel<16>;
    case 32: return grad_tables_kernel<32>;
    case 64: return grad_tables_kernel<64>;
    case 128: return grad_tables_kernel<128>;
    case 256: return grad_tables_kernel<256>;
    default: return grad_tables_kernel<512>;
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
  if ((rc = launch(rows_kernel, rows_grid(a), 256, st, a))) return rc;
  const ScoreKernel kernel = a.cap > 0.0f ? score_kernel_of<true>(a.R) : score_kernel_of<false>(a.R);
  if ((rc = launch(kernel, a.shares, 256, st, a))) return rc;
  return launch(a.cap > 0.0f ? score_finish_kernel<true> : score_finish_kernel<false>, (a.M + 3) / 4, 256, st, a);
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
  const int64_t blocks = (a.M + p.block - 1) / p.block;
  if ((rc = launch(a.cap > 0.0f ? grad_base_kernel_of<true>(a.R, p.block) : grad_base_kernel_of<false>(a.R, p.block),
                   blocks * a.splits, 512, st, a)))
    return rc;
  int tile;
  const ScoreKernel tables = grad_tables_kernel_of(a.R, &tile);
  return launch(tables, a.M + ((int64_t)a.V + tile - 1) / tile, 256, st, a);
}

}  // extern "C"
