// MI355X (gfx950) base logits: hidden states times an E4M3 head with one
// scale per block of 128 x 128, and the two quantizers.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "markov.h"
#include "numbers.h"

namespace {

// E4M3 code of x: nearest, ties to even, saturating at +-448, NaN to the NaN
// code of its sign. Integer rounding on x's bits: at or above 2^-6 the top 3
// fraction bits are kept (a carry moves into the exponent), the exponent
// rebiased from 127 to 7; below, the subnormal m 2^-9 with m = RN(|x| 2^9).
__device__ __forceinline__ uint32_t e4m3_encode(float x) {
  const uint32_t u = __float_as_uint(x), sgn = (u >> 24) & 0x80u, a = u & 0x7fffffffu;
  if (a > 0x7f800000u) return sgn | 0x7fu;
  if (a >= 0x43e00000u) return sgn | 0x7eu;
  if (a < 0x3c800000u) return sgn | (uint32_t)rintf(__uint_as_float(a) * 512.0f);
  return sgn | (((a + 0x7ffffu + ((a >> 20) & 1u)) >> 20) - (120u << 3));
}

// RN32(top / 448) of a block whose largest magnitude has the bits `top` (as
// integers they order like the magnitudes, with infinity and then NaN last).
__device__ __forceinline__ float block_scale(uint32_t top) { return __uint_as_float(top) / 448.0f; }

// The larger of two words' four magnitudes' bits so far and `top`.
__device__ __forceinline__ uint32_t top_of(uint32_t top, u32x4_t w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top = max(top, (w[i] << 16) & 0x7fffffffu);
    top = max(top, w[i] & 0x7fff0000u);
  }
  return top;
}

// The codes of 8 values. A finite scale takes the hardware conversion (nearest,
// ties to even; the clamp is the saturation, which only a subnormal scale can
// reach); any other scale the general one, for its NaN codes.
__device__ __forceinline__ u32x2_t codes_of(u32x4_t w, float scale) {
  u32x2_t out = {0u, 0u};
  if (scale == 0.0f) return out;
  const bool finite = __builtin_isfinite(scale);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = bf_lo(w[i]) / scale, b = bf_hi(w[i]) / scale;
    if (finite) {
      a = __builtin_amdgcn_fmed3f(a, -448.0f, 448.0f);
      b = __builtin_amdgcn_fmed3f(b, -448.0f, 448.0f);
      if (i & 1) out[i >> 1] = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, out[i >> 1], true);
      else out[i >> 1] = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, out[i >> 1], false);
    } else {
      out[i >> 1] |= (e4m3_encode(a) | (e4m3_encode(b) << 8)) << (16 * (i & 1));
    }
  }
  return out;
}

// The head: one workgroup per block of 128 x 128, held in registers between
// the maximum and the codes, so the weights are read once. Thread i takes
// 16-byte groups i % 16 of rows i / 16 + 16 s. Bound by memory, and streamed past
// the caches both ways: 163840 x 4096 372 -> 343 us (5.9 TB/s), 8192 x 2048 14.6
// -> 12.0, 4096 x 2048 8.7 -> 8.8.
__global__ __launch_bounds__(256) void quantize_head_kernel(const uint16_t* w, uint8_t* q, float* scales,
                                                            int V, int H, int wide) {
  const int bi = blockIdx.x / wide, bj = blockIdx.x - bi * wide, tid = threadIdx.x;
  const int j = bj * 128 + (tid & 15) * 8, r0 = bi * 128 + (tid >> 4);
  u32x4_t x[8];
  uint32_t top = 0;
#pragma unroll
  for (int s = 0; s < 8; ++s)
    x[s] = j < H && r0 + 16 * s < V ? __builtin_nontemporal_load((const u32x4_t*)(w + (size_t)(r0 + 16 * s) * H + j)) : (u32x4_t){0u, 0u, 0u, 0u};
#pragma unroll
  for (int s = 0; s < 8; ++s) top = top_of(top, x[s]);
#pragma unroll
  for (int sh = 32; sh >= 1; sh >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, sh));
  __shared__ uint32_t tops[4];
  if ((tid & 63) == 0) tops[tid >> 6] = top;
  __syncthreads();
  const float scale = block_scale(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
#pragma unroll
  for (int s = 0; s < 8; ++s)
    if (j < H && r0 + 16 * s < V) __builtin_nontemporal_store(codes_of(x[s], scale), (u32x2_t*)(q + (size_t)(r0 + 16 * s) * H + j));
  if (tid == 0) scales[blockIdx.x] = scale;
}

// Tokens per row of the states' scales: whole 1 KiB loads of 256.
__host__ __device__ constexpr int scale_stride(int tokens) { return (tokens + 255) & ~255; }

// The hidden states: 16 threads per 128 values of a row. Codes go to rows of
// `wide` * 128 bytes (zeros past H), scales to [wide][scale_stride(tokens)], the
// order the product reads them in.
__global__ __launch_bounds__(256) void quantize_states_kernel(const uint16_t* x, uint8_t* q, float* scales,
                                                              int tokens, int H, int wide) {
  const int64_t block = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (block >= (int64_t)tokens * wide) return;   // (whole groups of 16 lanes)
  const int t = (int)(block / wide), b = (int)(block - (int64_t)t * wide), j = b * 128 + (threadIdx.x & 15) * 8;
  const u32x4_t v = j < H ? *(const u32x4_t*)(x + (size_t)t * H + j) : (u32x4_t){0u, 0u, 0u, 0u};
  uint32_t top = top_of(0u, v);
#pragma unroll
  for (int sh = 8; sh >= 1; sh >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, sh));
  const float scale = block_scale(top);
  // (the padding's codes are 0 whatever the scale)
  *(u32x2_t*)(q + (size_t)t * wide * 128 + j) = j < H ? codes_of(v, scale) : (u32x2_t){0u, 0u};
  if ((threadIdx.x & 15) == 0) scales[(size_t)b * scale_stride(tokens) + t] = scale;
}

// ---------------------------------------------------------------- the product
//
// A workgroup of WM x WN waves takes a tile of WM TT 16 tokens x WN NV 16
// vocabulary rows, a wave TT x NV tiles of 16 x 16. One K step is one block of
// 128 hidden values: a single v_mfma_f32_16x16x128_f8f6f4 per 16 x 16 tile
// from a zero accumulator, whose fp32 result is added to the running sum with
// the product of its two scales (one FMA per element). The tile shapes do these
// in the same order, but for the step that calls of few tokens begin with.
//
// A operand: head rows, B operand: tokens, so that a lane holds one token (its
// lane % 16) and 4 vocabulary entries per tile. Row i of a wave's tile vt is
// vocabulary entry (i / 4) 4 NV + 4 vt + i % 4 of the wave's 16 NV, so that a
// lane's entries over its NV tiles are neighbours, stored 16 bytes at a time.
//
// Both operands and the tokens' scales come through LDS by asynchronous
// 16-byte loads. With two buffers a step waits for its own, asks for the next
// step's, and reads and multiplies while that load is in flight; with three
// (tiles of up to 32 tokens, which wait for memory most: 5 x 129280 x 7168 170
// -> 154 us; 320 tokens 262 -> 269) it asks for the one after. (Each
// step's buffers are restrict arguments of an inlined function: the compiler
// would otherwise hold every LDS read until the loads before it had landed.)
//
// LDS: rows of 128 bytes; 16-byte group c of row r is at place c ^ key(r), so
// that 8 neighbouring lanes of a read touch all 32 banks. Loads put 64
// consecutive places per instruction, so the permutation is in their source
// addresses.
//
// Measured (the kernel): 5 x 129280 x 7168 132 us, 7.0 TB/s of codes (bound by
// memory); 320 x 163840 x 4096 249 us, 1720 TF, 3.1 TB/s (the two floors are equal
// here, 150 us each, and LDS reads and the sums' vector instructions take turns with
// them); 2048 tokens 1270-1285 us, 2150 TF, the matrix units 54 % busy (the rest is
// the fp32 sum with two scales of every 128 values, a vector instruction per
// element, and LDS reads).

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// (ONCE: what is not read again, past the caches)
template <bool ONCE = false>
__device__ __forceinline__ void load_lds(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, ONCE ? 2 : 0);
}

constexpr int FEW = 64;   // tokens that one tile of a memory-bound call takes

template <int WM, int WN, int TT, int NV, bool ONCE>
struct Tile {
  static constexpr int NW = WM * WN, BM = WM * TT * 16, BN = WN * NV * 16;
  static constexpr int GX = BM / 8, GW = BN / 8;     // load instructions per step
  static constexpr int LX = (GX + NW - 1) / NW, LW = GW / NW;
  static constexpr int LEAST = GX / NW + LW;         // loads of a wave per step, at least
  static constexpr int BYTES = (BM + BN) * 128 + 1024;
  static_assert(GW % NW == 0 && BM <= 256, "");

  const uint8_t *xq, *wq, *xs, *zeros;   // at the tile's first row and token
  const __attribute__((address_space(4))) float* ws;   // (scalar loads: a vector load would wait for the requests)
  float weight;                          // the next block's head scale
  uint32_t offx[LX], offw[LW];           // of this lane's group in the first block
  int first, c, H, wide, stride_s, wave, wm, wn, li, lg;
  int atx, atw, ats;                     // this lane's operands and scale in a buffer

  // head row r's place permutation: the 8 rows that 8 neighbouring lanes read
  // (i % 4, then i / 4 in steps of 4 NV rows) have 8 different keys
  static __device__ __forceinline__ int key(int r) {
    return NV == 1 ? r & 7 : (r & 3) | ((r / (4 * NV)) & 1) << 2;
  }

  // The block of step i.
  __device__ __forceinline__ int block(int i) const { return i + first < wide ? i + first : i + first - wide; }

  // FULL: the block of step i is known to be a whole one.
  template <bool FULL>
  __device__ __forceinline__ void request(int i0, uint8_t* __restrict__ to) const {
    const int b = block(i0);
    if (wave == NW - 1) load_lds(xs + (size_t)b * stride_s * 4 + (threadIdx.x & 63) * 16, to + (BM + BN) * 128);
    // (opaque, so that they stay scalars beside the lanes' 32-bit offsets)
    const uint8_t *x = xq + (size_t)b * 128, *w = wq + (size_t)b * 128;
    asm("" : "+s"(x));
    asm("" : "+s"(w));
#pragma unroll
    for (int i = 0; i < LX; ++i)
      if (GX % NW == 0 || wave + i * NW < GX) load_lds(x + offx[i], to + (wave + i * NW) * 1024);
    uint8_t* tw = to + BM * 128;
    if (FULL || b * 128 + 128 <= H) {
#pragma unroll
      for (int i = 0; i < LW; ++i) load_lds<ONCE>(w + offw[i], tw + (wave + i * NW) * 1024);
    } else {
      // past the head's last column, the zeros that pad the states' rows
      // (there are some exactly if there is such a column)
#pragma unroll
      for (int i = 0; i < LW; ++i)
        load_lds<ONCE>(b * 128 + c * 16 < H ? w + offw[i] : zeros, tw + (wave + i * NW) * 1024);
    }
  }

  template <bool FULL>
  __device__ __forceinline__ void step(int b, int ahead, bool more, const uint8_t* __restrict__ from, uint8_t* __restrict__ to,
                                       f32x4_t (&acc)[TT][NV]) {
    if (more) request<FULL>(ahead, to);
    const float by = weight;             // asked for in the step before
    weight = ws[block(b + 1 < wide ? b + 1 : b)];
    i32x8_t A[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) A[v] = operand(from, atw + v * 512);
    // one token tile's products are issued, then the tile before's are scaled
    // and added while they run, with the next tile's operand on its way; the
    // barriers keep the scheduler from holding more tiles in registers
    i32x8_t B = operand(from, atx);
    float s = *(const float*)(from + ats) * by, s_before = 0.0f;
    f32x4_t p[NV], before[NV];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      i32x8_t B_next = B;
      float s_next = 0.0f;
      if (t + 1 < TT) {
        B_next = operand(from, atx + (t + 1) * 2048);
        s_next = *(const float*)(from + ats + (t + 1) * 64);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v)   // (scale operands of 0: the instruction without block scales)
        p[v] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A[v], B, (f32x4_t){0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
      if (t > 0) {
        add(acc[t - 1], before, s_before);
        __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);   // the operand's reads,
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0); // then a product
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0); // and four sums in turn
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int v = 0; v < NV; ++v) before[v] = p[v];
      s_before = s;
      s = s_next * by;
      B = B_next;
    }
    add(acc[TT - 1], before, s_before);
  }

  // A lane's 32 of a row's 128 values: groups lane / 16 and lane / 16 + 4.
  __device__ __forceinline__ static i32x8_t operand(const uint8_t* from, int at) {
    const i32x4_t lo = *(const i32x4_t*)(from + at);
    const i32x4_t hi = *(const i32x4_t*)(from + (at ^ 64));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }

  __device__ __forceinline__ static void add(f32x4_t (&acc)[NV], const f32x4_t (&p)[NV], float s) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[v][e] = __builtin_fmaf(p[v][e], s, acc[v][e]);
    // (the sums are wanted here: left alone the compiler puts them off to the
    // end of the step, with every product held in registers)
#pragma unroll
    for (int v = 0; v < NV; ++v) asm volatile("" : "+v"(acc[v]));
  }
};

template <int WM, int WN, int TT, int NV, int NB, bool ONCE>
__global__ __launch_bounds__(WM * WN * 64) void product_kernel(
    const uint8_t* __restrict__ xq, const float* __restrict__ xs, const uint8_t* __restrict__ wq,
    const float* __restrict__ ws, uint16_t* __restrict__ out, int tokens, int V, int H, int token_tiles,
    int tiles) {
  typedef Tile<WM, WN, TT, NV, ONCE> T;
  __shared__ __attribute__((aligned(16))) uint8_t one[T::BYTES], two[T::BYTES], three[NB == 3 ? T::BYTES : 16];
  // a vocabulary tile's token tiles follow each other on one XCD (workgroups
  // go round the 8 XCDs), so they share its rows in that XCD's L2
  const int local = blockIdx.x >> 3, tile = (local / token_tiles) * 8 + (blockIdx.x & 7);
  const int t0 = (local % token_tiles) * T::BM, v0 = tile * T::BN;
  if (tile >= tiles) return;
  const int wide = (H + 127) / 128, lane = threadIdx.x & 63;
  const uint32_t stride = (uint32_t)wide * 128;
  T a;
  a.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  a.wm = a.wave / WN;
  a.wn = a.wave % WN;
  a.li = lane & 15;
  a.lg = lane >> 4;
  a.H = H;
  a.wide = wide;
  // Where the head's rows bound the call, each 256 vocabulary entries start
  // with another block, so that the workgroups at work read other columns:
  // rows a power of two apart put one column on few memory channels (32 tokens
  // x 163840 x 4096: 165 -> 129 us; 24 x 129280 x 7168: 161 -> 162). With more
  // tokens, tiles of one column share its states in L2 instead (2048 tokens:
  // 1293 us, and 1373 with such starts). Smaller last blocks come last.
  a.first = H % 128 || tokens > FEW ? 0 : (v0 / 256) % wide;
  a.stride_s = scale_stride(tokens);
  a.xq = xq + (size_t)t0 * stride;
  a.wq = wq + (size_t)v0 * H;
  a.xs = (const uint8_t*)(xs + t0);
  a.zeros = xq + stride - 16;
  const int wave_v = v0 + a.wn * NV * 16;
  a.ws = (const __attribute__((address_space(4))) float*)(ws + (size_t)(min(wave_v, V - 1) / 128) * wide);
  // (every row that a lane reads has the key lane % 8)
  const int place = (a.lg ^ (lane & 7)) * 16;
  a.atx = (a.wm * TT * 16 + a.li) * 128 + place;
  a.atw = (T::BM + a.wn * NV * 16 + (a.li >> 2) * 4 * NV + (a.li & 3)) * 128 + place;
  a.ats = (T::BM + T::BN) * 128 + (a.wm * TT * 16 + a.li) * 4;
  // lane l of a load is at row l / 8 of its 8, place l % 8; the loads of a
  // wave are 8 NW rows apart, which have the same key. Rows past the last
  // token or vocabulary entry read the last one's.
  const int r0 = a.wave * 8 + (lane >> 3);
  a.c = (lane & 7) ^ T::key(r0);
#pragma unroll
  for (int i = 0; i < T::LX; ++i)
    a.offx[i] = (uint32_t)min(r0 + i * T::NW * 8, tokens - 1 - t0) * stride + ((lane & 7) ^ (r0 & 7)) * 16;
#pragma unroll
  for (int i = 0; i < T::LW; ++i) a.offw[i] = (uint32_t)min(r0 + i * T::NW * 8, V - 1 - v0) * (uint32_t)H + a.c * 16;

  f32x4_t acc[TT][NV];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int v = 0; v < NV; ++v) acc[t][v] = (f32x4_t){0.f, 0.f, 0.f, 0.f};

  // a step's own buffer has landed: with three buffers the next step's may
  // still be on its way
  auto landed = [] { barrier_but<NB == 3 ? T::LEAST : 0>(); };
  a.weight = a.ws[a.first];
  int b = 0;
  if constexpr (NB == 2) {
    a.template request<false>(0, one);
    for (; b + 3 < wide; b += 2) {   // only the last block may be a smaller one
      landed();
      a.template step<true>(b, b + 1, true, one, two, acc);
      landed();
      a.template step<true>(b + 1, b + 2, true, two, one, acc);
    }
    landed();
    a.template step<false>(b, b + 1, b + 1 < wide, one, two, acc);
    if (b + 1 < wide) {
      landed();
      a.template step<false>(b + 1, b + 2, b + 2 < wide, two, one, acc);
    }
    if (b + 2 < wide) {
      landed();
      a.template step<false>(b + 2, 0, false, one, two, acc);
    }
  } else {
    a.template request<false>(0, one);
    __builtin_amdgcn_sched_barrier(0);   // (the first block's loads first: the first wait counts on it)
    if (wide > 1) a.template request<false>(1, two);
    for (; b + 5 < wide; b += 3) {
      landed();
      a.template step<true>(b, b + 2, true, one, three, acc);
      landed();
      a.template step<true>(b + 1, b + 3, true, two, one, acc);
      landed();
      a.template step<true>(b + 2, b + 4, true, three, two, acc);
    }
    auto rest = [&](int b, const uint8_t* from, uint8_t* to) {
      if (b >= wide) return;
      if (b + 1 < wide) landed();
      else barrier_but<0>();
      a.template step<false>(b, b + 2, b + 2 < wide, from, to, acc);
    };
    rest(b, one, three);
    rest(b + 1, two, one);
    rest(b + 2, three, two);
    rest(b + 3, one, three);
    rest(b + 4, two, one);
  }

  const int v = wave_v + a.lg * 4 * NV;
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int token = t0 + (a.wm * TT + t) * 16 + a.li;
    if (token >= tokens) continue;
    uint16_t* row = out + (size_t)token * V + v;
    if constexpr (NV == 1) {
      if (v < V) *(u32x2_t*)row = (u32x2_t){pack_bf16(acc[t][0][0], acc[t][0][1]), pack_bf16(acc[t][0][2], acc[t][0][3])};
    } else {
#pragma unroll
      for (int n = 0; n < NV; n += 2)
        if (v + 4 * n < V)
          *(u32x4_t*)(row + 4 * n) =
              (u32x4_t){pack_bf16(acc[t][n][0], acc[t][n][1]), pack_bf16(acc[t][n][2], acc[t][n][3]),
                        pack_bf16(acc[t][n + 1][0], acc[t][n + 1][1]), pack_bf16(acc[t][n + 1][2], acc[t][n + 1][3])};
    }
  }
}

constexpr int64_t MOST_THREADS = 0xffffffffll;   // of one launch

struct Product {
  const uint8_t* xq;
  const float* xs;
  const uint8_t* wq;
  const float* ws;
  uint16_t* out;
  int tokens, V, H;
};

// A head that the 256 MB cache behind the L2 holds stays there for the next call;
// a larger one is streamed past it (5 tokens x 129280 x 7168: 157 -> 137 us; 320 x
// 98304 x 4096: 162 -> 158; but 5 x 32768 x 4096 23 -> 26, 320 tokens 52 -> 58).
constexpr int64_t CACHE = 256 << 20;

template <int WM, int WN, int TT, int NV, int NB>
int launch_product(const Product& p, hipStream_t stream) {
  constexpr int BM = WM * TT * 16, BN = WN * NV * 16;
  const int token_tiles = (p.tokens + BM - 1) / BM, tiles = (p.V + BN - 1) / BN;
  const int64_t grid = (int64_t)((tiles + 7) / 8) * 8 * token_tiles;
  if (grid > MOST_THREADS / (WM * WN * 64)) return MARKOV_ERR_SHAPE;
  const auto kernel = (int64_t)p.V * p.H > CACHE ? product_kernel<WM, WN, TT, NV, NB, true> : product_kernel<WM, WN, TT, NV, NB, false>;
  kernel<<<dim3((unsigned)grid), WM * WN * 64, 0, stream>>>(p.xq, p.xs, p.wq, p.ws, p.out, p.tokens, p.V, p.H, token_tiles, tiles);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

int blocks(int32_t n) { return (n + 127) / 128; }

int check_head(int32_t vocab, int32_t hidden) {
  if (vocab > MARKOV_MAX_VOCAB) return MARKOV_ERR_VOCAB;
  if (vocab < 1 || hidden < 16 || (hidden & 15) || hidden > 1048576) return MARKOV_ERR_SHAPE;
  return MARKOV_OK;
}

// Workgroups of the states' quantizer, 0 if they are more than a launch takes.
int64_t states_grid(int32_t tokens, int32_t hidden) {
  const int64_t grid = ((int64_t)tokens * blocks(hidden) + 15) / 16;
  return grid > MOST_THREADS / 256 ? 0 : grid;
}

size_t codes_bytes(int32_t tokens, int32_t hidden) { return (size_t)tokens * blocks(hidden) * 128; }

}  // namespace

extern "C" {

int markov_quantize_head_fp8(const void* w, uint8_t* wq, float* scales, int32_t vocab,
                             int32_t hidden, markov_stream_t stream) {
  const int rc = check_head(vocab, hidden);
  if (rc) return rc;
  if (!w || !wq || !scales) return MARKOV_ERR_NULL;
  if (!aligned_to(w, 16) || !aligned_to(wq, 16) || !aligned_to(scales, 4)) return MARKOV_ERR_ALIGN;
  const int wide = blocks(hidden);
  const int64_t grid = (int64_t)wide * blocks(vocab);
  if (grid > MOST_THREADS / 256) return MARKOV_ERR_SHAPE;
  quantize_head_kernel<<<dim3((unsigned)grid), 256, 0, (hipStream_t)stream>>>((const uint16_t*)w, wq, scales, vocab,
                                                                             hidden, wide);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

size_t markov_head_workspace_bytes(int32_t tokens, int32_t hidden) {
  if (tokens < 1 || tokens > MARKOV_MAX_TOKENS || check_head(8, hidden) || !states_grid(tokens, hidden)) return 0;
  return codes_bytes(tokens, hidden) + (size_t)scale_stride(tokens) * blocks(hidden) * 4;
}

int markov_head_logits_fp8(const void* x, const uint8_t* wq, const float* scales, void* logits,
                           int32_t tokens, int32_t vocab, int32_t hidden, void* workspace,
                           size_t workspace_bytes, markov_stream_t stream) {
  const int rc = check_head(vocab, hidden);
  if (rc) return rc;
  if (tokens < 1 || (vocab & 7)) return MARKOV_ERR_SHAPE;
  if (tokens > MARKOV_MAX_TOKENS) return MARKOV_ERR_ROWS;
  const int64_t grid = states_grid(tokens, hidden);
  if (!grid) return MARKOV_ERR_SHAPE;
  if (!x || !wq || !scales || !logits || !workspace) return MARKOV_ERR_NULL;
  if (!aligned_to(x, 16) || !aligned_to(wq, 16) || !aligned_to(scales, 4) || !aligned_to(logits, 16) ||
      !aligned_to(workspace, 16))
    return MARKOV_ERR_ALIGN;
  if (workspace_bytes < markov_head_workspace_bytes(tokens, hidden)) return MARKOV_ERR_WORKSPACE;
  uint8_t* xq = (uint8_t*)workspace;
  float* xs = (float*)(xq + codes_bytes(tokens, hidden));
  const int wide = blocks(hidden);
  const hipStream_t st = (hipStream_t)stream;
  quantize_states_kernel<<<dim3((unsigned)grid), 256, 0, st>>>(
      (const uint16_t*)x, xq, xs, tokens, hidden, wide);
  if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
  const Product p = {xq, xs, wq, scales, (uint16_t*)logits, tokens, vocab, hidden};
  // Few tokens: the smallest tile that takes them all (x 129280 x 7168: 16 tokens
  // 142 us in a tile of 16 or 32, 156 in one of 64, 229 in one of 96; 32 tokens
  // 157, 163, 236; 64 tokens 180 and 235; 16 x 32768 x 4096 23.3, 23.7, 25.3, 53).
  // More: tiles of up to 256, of the height that pads the tokens least (320: two
  // of 160).
  if (tokens <= 16) return launch_product<1, 4, 1, 1, 3>(p, st);
  if (tokens <= 32) return launch_product<1, 4, 2, 1, 3>(p, st);
  if (tokens <= FEW) return launch_product<1, 4, 4, 2, 2>(p, st);
  const int tiles = (tokens + 255) / 256;
  switch ((tokens + 32 * tiles - 1) / (32 * tiles)) {
    case 3: return launch_product<2, 4, 3, 4, 2>(p, st);
    case 4: return launch_product<2, 4, 4, 4, 2>(p, st);
    case 5: return launch_product<2, 4, 5, 4, 2>(p, st);
    case 6: return launch_product<2, 4, 6, 4, 2>(p, st);
    case 7: return launch_product<2, 4, 7, 4, 2>(p, st);
    default: return launch_product<2, 4, 8, 4, 2>(p, st);
  }
}

}  // extern "C"
