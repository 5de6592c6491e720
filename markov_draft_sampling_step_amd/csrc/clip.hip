// MI355X (gfx950) gradient clipping: the norm over many tensors, and the
// tensors scaled to it.
//
// Two passes with the kernel boundary between them. The first reads every
// element once and leaves a binary64 sum of squares per workgroup (binary64:
// a square of a large fp32 gradient is past the largest fp32); the second adds
// those sums up in a fixed order in every workgroup -- they are few, and a
// launch of its own would cost more -- and scales. Both are bound by memory:
// the second goes through the chunks backwards, so that it begins with what the
// first left in the 256 MB cache, and its stores stream past it (40 tensors of 321
// MB together: 55 us, 5.8 TB/s, and 103 us, 6.2 TB/s; loads that stream as well
// 131 us for 125 on a smaller set). Tensors come as a table in the kernel's
// arguments, so a captured graph holds its own copy.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "markov.h"
#include "numbers.h"

namespace {

constexpr int CT = 256;           // threads
constexpr int GROUP = 64;         // tensors per launch
constexpr int64_t CHUNK = 8192;   // elements a workgroup takes at a time
constexpr int BLOCKS = 2048;      // the most workgroups over all groups' first pass, about

struct Tensors {
  const void* src[GROUP];
  void* dst[GROUP];
  int64_t count[GROUP];
  int64_t chunk0[GROUP + 1];      // the first chunk of each tensor
  uint64_t fp32;                  // bit i: tensor i is fp32, else bf16
  int n;
};

// The tensor that chunk c belongs to: the last with chunk0 <= c.
__device__ __forceinline__ int tensor_of(const Tensors& t, int64_t c) {
  int i = 0;
#pragma unroll
  for (int step = GROUP / 2; step > 0; step >>= 1)
    if (i + step < t.n && t.chunk0[i + step] <= c) i += step;
  return i;
}

__device__ __forceinline__ double block_total(double v, double* red) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int sh = 32; sh >= 1; sh >>= 1) v += __shfl_xor(v, sh);
  __syncthreads();
  if (lane == 0) red[wave] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < CT / 64; ++w) s += red[w];
  return s;
}

// The squares of a word's two bf16 values, or of a binary32 value, exact.
__device__ __forceinline__ double square(float g) { return (double)g * (double)g; }

__global__ __launch_bounds__(CT) void square_kernel(Tensors t, double* partial) {
  __shared__ double red[CT / 64];
  double s0 = 0.0, s1 = 0.0;
  for (int64_t c = blockIdx.x; c < t.chunk0[t.n]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t e0 = (c - t.chunk0[i]) * CHUNK;
    const int left = (int)(t.count[i] - e0 < CHUNK ? t.count[i] - e0 : CHUNK);
    const bool f32 = (t.fp32 >> i) & 1;
    const int per = f32 ? 4 : 8;                     // elements in 16 bytes
    const uint8_t* src = (const uint8_t*)t.src[i] + e0 * (f32 ? 4 : 2);
    int done = 0;
    if (aligned_to(src, 16)) {
      const u32x4_t* at = (const u32x4_t*)src;
      const int groups = left / per;
      done = groups * per;
      for (int g0 = threadIdx.x; g0 < groups; g0 += 4 * CT) {
        u32x4_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = g0 + u * CT < groups ? at[g0 + u * CT] : (u32x4_t){0u, 0u, 0u, 0u};
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (f32) {
              s0 += square(__uint_as_float(w[u][k]));
            } else {
              s0 += square(bf_lo(w[u][k]));
              s1 += square(bf_hi(w[u][k]));
            }
          }
      }
    }
#pragma unroll 4
    for (int e = done + threadIdx.x; e < left; e += CT)
      s0 += square(f32 ? ((const float*)src)[e] : bf_one(((const uint16_t*)src)[e]));
  }
  const double s = block_total(s0 + s1, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(CT) void scale_kernel(Tensors t, const double* partial, int partials,
                                                   float max_norm, float* norm) {
  __shared__ double red[CT / 64];
  double s = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < partials; i += CT) s += partial[i];
  const double total = sqrt(block_total(s, red));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
  const double want = (double)max_norm / (total + 1e-6);
  // (finite as the caller sees it: a root past binary32 is reported as infinite)
  const bool clips = isfinite((float)total) && want < 1.0;
  // a factor below the smallest normal number would have few bits: 2^120 of it go
  // into another, which takes a gradient whose product is not 0 as it is
  const bool small = clips && want < 0x1p-126;
  const float by = !clips ? 1.0f : (float)(small ? want * 0x1p120 : want), first = small ? 0x1p-120f : 1.0f;
  for (int64_t c = t.chunk0[t.n] - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int i = tensor_of(t, c);
    if (!clips && t.src[i] == t.dst[i]) continue;
    const int64_t e0 = (c - t.chunk0[i]) * CHUNK;
    const int left = (int)(t.count[i] - e0 < CHUNK ? t.count[i] - e0 : CHUNK);
    const bool f32 = (t.fp32 >> i) & 1;
    const int per = f32 ? 4 : 8;
    const uint8_t* src = (const uint8_t*)t.src[i] + e0 * (f32 ? 4 : 2);
    uint8_t* dst = (uint8_t*)t.dst[i] + e0 * (f32 ? 4 : 2);
    int done = 0;
    if (aligned_to(src, 16) && aligned_to(dst, 16)) {
      const u32x4_t* at = (const u32x4_t*)src;
      u32x4_t* to = (u32x4_t*)dst;
      const int groups = left / per;
      done = groups * per;
      for (int g0 = threadIdx.x; g0 < groups; g0 += 4 * CT) {
        u32x4_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = g0 + u * CT < groups ? at[g0 + u * CT] : (u32x4_t){0u, 0u, 0u, 0u};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[u][k] = f32 ? __float_as_uint(__uint_as_float(w[u][k]) * first * by)
                          : pack_bf16(bf_lo(w[u][k]) * first * by, bf_hi(w[u][k]) * first * by);
          if (g0 + u * CT < groups) __builtin_nontemporal_store(w[u], to + g0 + u * CT);
        }
      }
    }
#pragma unroll 4
    for (int e = done + threadIdx.x; e < left; e += CT) {
      if (f32) ((float*)dst)[e] = ((const float*)src)[e] * first * by;
      else ((uint16_t*)dst)[e] = (uint16_t)pack_bf16(bf_one(((const uint16_t*)src)[e]) * first * by, 0.0f);
    }
  }
}

int groups_of(int32_t n) { return n < 1 ? 1 : (n + GROUP - 1) / GROUP; }

// The most workgroups of one group's first pass.
int blocks_of(int groups) { return BLOCKS / groups < 32 ? 32 : BLOCKS / groups; }

}  // namespace

extern "C" {

size_t markov_clip_workspace_bytes(int32_t n) {
  if (n < 0) return 0;
  const int g = groups_of(n);
  return (size_t)g * blocks_of(g) * sizeof(double);
}

int markov_clip_gradients(const void* const* grads, void* const* out, const int64_t* counts,
                          const int32_t* types, int32_t n, float max_norm, float* norm,
                          void* workspace, size_t workspace_bytes, markov_stream_t stream) {
  if (n < 0) return MARKOV_ERR_SHAPE;
  if (!norm || !workspace || (n > 0 && (!grads || !out || !counts || !types))) return MARKOV_ERR_NULL;
  if (!(max_norm >= 0.0f)) return MARKOV_ERR_VALUE;
  for (int32_t i = 0; i < n; ++i) {
    if (counts[i] < 0 || (types[i] != MARKOV_BF16 && types[i] != MARKOV_FP32)) return MARKOV_ERR_SHAPE;
    if (counts[i] > 0 && (!grads[i] || !out[i])) return MARKOV_ERR_NULL;
    const uintptr_t size = types[i] == MARKOV_FP32 ? 4 : 2;
    if (counts[i] > 0 && (!aligned_to(grads[i], size) || !aligned_to(out[i], size))) return MARKOV_ERR_ALIGN;
  }
  if (!aligned_to(workspace, 16) || !aligned_to(norm, 4)) return MARKOV_ERR_ALIGN;
  if (workspace_bytes < markov_clip_workspace_bytes(n)) return MARKOV_ERR_WORKSPACE;
  const int groups = groups_of(n), most = blocks_of(groups);
  double* partial = (double*)workspace;
  int partials = 0;
  for (int pass = 0; pass < 2; ++pass) {
    for (int g = 0; g < groups; ++g) {
      Tensors t = {};
      // (tensors by their place in the list: an empty one leaves its place unused)
      const int32_t first = g * GROUP, last = n - first < GROUP ? n : first + GROUP;
      for (int32_t i = first; i < last; ++i) {
        if (counts[i] == 0) continue;
        t.src[t.n] = grads[i];
        t.dst[t.n] = out[i];
        t.count[t.n] = counts[i];
        t.chunk0[t.n + 1] = t.chunk0[t.n] + (counts[i] + CHUNK - 1) / CHUNK;
        if (types[i] == MARKOV_FP32) t.fp32 |= 1ull << t.n;
        ++t.n;
      }
      const int64_t chunks = t.chunk0[t.n];
      // an empty group still writes its (zero) sum, and the last pass the norm
      if (pass == 0) {
        const int grid = (int)(chunks < 1 ? 1 : chunks < most ? chunks : most);
        square_kernel<<<dim3((unsigned)grid), CT, 0, (hipStream_t)stream>>>(t, partial + partials);
        partials += grid;
      } else {
        const int grid = (int)(chunks < 1 ? 1 : chunks < BLOCKS ? chunks : BLOCKS);
        scale_kernel<<<dim3((unsigned)grid), CT, 0, (hipStream_t)stream>>>(t, partial, partials, max_norm,
                                                                           g == 0 ? norm : nullptr);
      }
      if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
    }
  }
  return MARKOV_OK;
}

}  // extern "C"
