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

__device__ __forceinline__ float e4m3_decode(uint32_t code) {
  const uint32_t e = (code >> 3) & 15u, f = code & 7u;
  float x = e ? __uint_as_float(((e + 120u) << 23) | (f << 20)) : (float)f * 0x1p-9f;
  if ((code & 0x7fu) == 0x7fu) x = __uint_as_float(0x7fc00000u);
  return code & 0x80u ? -x : x;
}

// The scale of a block whose largest magnitude has the bits `top` (as
// integers they order like the magnitudes, with infinity and then NaN last).
__device__ __forceinline__ float block_scale(uint32_t top) { return __uint_as_float(top) / 448.0f; }

__device__ __forceinline__ uint32_t code_of(float v, float scale) {
  return scale == 0.0f ? 0u : e4m3_encode(v / scale);
}

// One workgroup per block of `height` rows x 128 columns of x [n][h]; codes
// with a row stride of `stride` (columns past h up to the stride get 0).
__global__ __launch_bounds__(256) void quantize_kernel(const uint16_t* x, uint8_t* q, float* scales,
                                                       int n, int h, int stride, int height) {
  const int b = blockIdx.x, r0 = blockIdx.y * height, tid = threadIdx.x;
  const int rows = min(height, n - r0), j0 = b * 128;
  __shared__ uint32_t top;
  if (tid == 0) top = 0;
  __syncthreads();
  uint32_t mine = 0;
  for (int i = tid; i < rows * 128; i += 256) {
    const int r = r0 + i / 128, j = j0 + i % 128;
    if (j < h) mine = max(mine, ((uint32_t)x[(size_t)r * h + j] << 16) & 0x7fffffffu);
  }
  atomicMax(&top, mine);
  __syncthreads();
  const float scale = block_scale(top);
  for (int i = tid; i < rows * 128; i += 256) {
    const int r = r0 + i / 128, j = j0 + i % 128;
    if (j < stride) q[(size_t)r * stride + j] = j < h ? (uint8_t)code_of(bf_one(x[(size_t)r * h + j]), scale) : 0;
  }
  if (tid == 0) scales[(size_t)blockIdx.y * gridDim.x + b] = scale;
}

// One thread per logit.
__global__ __launch_bounds__(256) void product_kernel(const uint8_t* xq, const float* xs, const uint8_t* wq,
                                                      const float* ws, uint16_t* out, int tokens, int V,
                                                      int H, int stride) {
  const int v = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (v >= V) return;
  const int nb = (H + 127) / 128;
  float sum = 0.0f;
  for (int b = 0; b < nb; ++b) {
    float part = 0.0f;
    for (int j = b * 128; j < min(H, b * 128 + 128); ++j)
      part += e4m3_decode(xq[(size_t)t * stride + j]) * e4m3_decode(wq[(size_t)v * H + j]);
    sum += xs[(size_t)t * nb + b] * ws[(size_t)(v / 128) * nb + b] * part;
  }
  out[(size_t)t * V + v] = (uint16_t)pack_bf16(sum, 0.0f);
}

int blocks(int32_t n) { return (n + 127) / 128; }

int check_head(int32_t vocab, int32_t hidden) {
  if (vocab > MARKOV_MAX_VOCAB) return MARKOV_ERR_VOCAB;
  if (vocab < 1 || hidden < 16 || (hidden & 15) || hidden > 1048576) return MARKOV_ERR_SHAPE;
  return MARKOV_OK;
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
  quantize_kernel<<<dim3((unsigned)blocks(hidden), (unsigned)blocks(vocab)), 256, 0, (hipStream_t)stream>>>(
      (const uint16_t*)w, wq, scales, vocab, hidden, hidden, 128);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

size_t markov_head_workspace_bytes(int32_t tokens, int32_t hidden) {
  if (tokens < 1 || tokens > MARKOV_MAX_TOKENS || check_head(8, hidden)) return 0;
  return codes_bytes(tokens, hidden) + (((size_t)tokens * blocks(hidden) * 4 + 15) & ~(size_t)15);
}

int markov_head_logits_fp8(const void* x, const uint8_t* wq, const float* scales, void* logits,
                           int32_t tokens, int32_t vocab, int32_t hidden, void* workspace,
                           size_t workspace_bytes, markov_stream_t stream) {
  const int rc = check_head(vocab, hidden);
  if (rc) return rc;
  if (tokens < 1 || (vocab & 7)) return MARKOV_ERR_SHAPE;
  if (tokens > MARKOV_MAX_TOKENS) return MARKOV_ERR_ROWS;
  if (!x || !wq || !scales || !logits || !workspace) return MARKOV_ERR_NULL;
  if (!aligned_to(x, 16) || !aligned_to(wq, 16) || !aligned_to(scales, 4) || !aligned_to(logits, 16) ||
      !aligned_to(workspace, 16))
    return MARKOV_ERR_ALIGN;
  if (workspace_bytes < markov_head_workspace_bytes(tokens, hidden)) return MARKOV_ERR_WORKSPACE;
  uint8_t* xq = (uint8_t*)workspace;
  float* xs = (float*)(xq + codes_bytes(tokens, hidden));
  const int stride = blocks(hidden) * 128;
  quantize_kernel<<<dim3((unsigned)blocks(hidden), (unsigned)tokens), 256, 0, (hipStream_t)stream>>>(
      (const uint16_t*)x, xq, xs, tokens, hidden, stride, 1);
  if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
  product_kernel<<<dim3((unsigned)((vocab + 255) / 256), (unsigned)tokens), 256, 0, (hipStream_t)stream>>>(
      xq, xs, wq, scales, (uint16_t*)logits, tokens, vocab, hidden, stride);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

}  // extern "C"
