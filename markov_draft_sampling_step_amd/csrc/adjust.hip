// MI355X (gfx950) penalties for seen tokens, biases and grammar masks on logits,
// and the state of the tokens that a request has seen.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "markov.h"
#include "numbers.h"

namespace {

constexpr int64_t MOST_THREADS = 0xffffffffll;   // of one launch

// ---------------------------------------------------------------- the state

struct Count {
  uint32_t *prompt, *output;
  int32_t* counts;
  const int64_t* tokens;
  const int32_t *lengths, *prompt_lengths, *slots;
  int rows, length, slots_count, V, words;
};

// The slot of a row, or -1.
__device__ __forceinline__ int slot_of(const int32_t* slots, int row, int slots_count) {
  const int slot = slots ? slots[row] : row;
  return slot >= 0 && slot < slots_count ? slot : -1;
}

constexpr int RESET = 4096;   // counts that a workgroup empties

__global__ __launch_bounds__(256) void reset_kernel(Count a, int parts) {
  const int row = blockIdx.x / parts, v0 = (int)(blockIdx.x - (unsigned)row * parts) * RESET;
  const int slot = slot_of(a.slots, row, a.slots_count);
  if (slot < 0) return;
  int32_t* counts = a.counts + (size_t)slot * a.V;
  for (int v = v0 + threadIdx.x; v < min(v0 + RESET, a.V); v += 256) counts[v] = 0;
  const int w = v0 / 32 + threadIdx.x;
  if (threadIdx.x < RESET / 32 && w < a.words) {
    a.prompt[(size_t)slot * a.words + w] = 0;
    a.output[(size_t)slot * a.words + w] = 0;
  }
}

// A thread per token. Whole numbers: the order of the additions changes nothing.
__global__ __launch_bounds__(256) void count_kernel(Count a) {
  const int i = blockIdx.x * 256 + (int)threadIdx.x;
  if (i >= a.rows * a.length) return;
  const int row = i / a.length, j = i - row * a.length;
  if (a.lengths && j >= a.lengths[row]) return;
  const int slot = slot_of(a.slots, row, a.slots_count);
  const int64_t t = a.tokens[i];
  if (slot < 0 || t < 0 || t >= a.V) return;
  const size_t word = (size_t)slot * a.words + ((uint32_t)t >> 5);
  const uint32_t bit = 1u << ((uint32_t)t & 31);
  if (a.prompt_lengths && j < a.prompt_lengths[row]) {
    atomicOr(a.prompt + word, bit);
  } else {
    atomicOr(a.output + word, bit);
    atomicAdd(a.counts + (size_t)slot * a.V + t, 1);
  }
}

// ---------------------------------------------------------------- the logits

constexpr int SLAB = 4096, CHUNKS = SLAB / (256 * 8);   // tokens of a workgroup, groups of 8 of a thread

// A workgroup per row-step and slab. What a group of 8 tokens needs is decided by
// its bits: most of them have none set and are copied, or not touched in place.
// The row's biases, and which of the slab's tokens were drafted, are put
// into LDS first.
template <bool F32, bool IN_PLACE>
__global__ __launch_bounds__(256) void adjust_kernel(markov_adjust_t a, int slabs) {
  __shared__ int bias_at[SLAB];              // a token's entry + 1, 0 where it has none
  __shared__ uint32_t marked[SLAB / 32];     // tokens with a bias, or drafted before this step
  const int at = blockIdx.x / slabs, slab = blockIdx.x - (unsigned)at * slabs, tid = threadIdx.x;
  const int row = at / a.k, step = at - row * a.k, v0 = slab * SLAB, V = a.vocab, words = (V + 31) >> 5;
  const size_t here = (size_t)at * (V >> 3) + (v0 >> 3);   // in groups of 8
  Eight<F32> x[CHUNKS];
  if constexpr (!IN_PLACE) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      x[i] = {};
      if (v0 + (tid + i * 256) * 8 < V) x[i] = load8<F32>(a.logits, here + tid + i * 256);
    }
  }
  const int slot = a.counts ? slot_of(a.slots, row, a.slots_count) : -1;
  const int drafted = a.drafted ? step : 0;
  int b0 = 0, b1 = 0;
  if (a.bias_starts) {   // (kept within the entries, whatever the starts are)
    b0 = max(0, min(a.bias_starts[row], a.biases));
    b1 = max(b0, min(a.bias_starts[row + 1], a.biases));
  }
  const bool marks = drafted > 0 || b1 > b0;
  if (marks) {
    for (int i = tid; i < SLAB; i += 256) bias_at[i] = 0;
    for (int i = tid; i < SLAB / 32; i += 256) marked[i] = 0;
    __syncthreads();
    for (int b = b0 + tid; b < b1; b += 256) {
      const int64_t t = a.bias_tokens[b];
      if (t >= v0 && t < min(v0 + SLAB, V)) {
        atomicMax(&bias_at[t - v0], b + 1);
        atomicOr(&marked[(t - v0) >> 5], 1u << ((t - v0) & 31));
      }
    }
    for (int j = tid; j < drafted; j += 256) {
      const int64_t t = a.drafted[(size_t)row * a.drafted_stride + j];
      if (t >= v0 && t < min(v0 + SLAB, V)) atomicOr(&marked[(t - v0) >> 5], 1u << ((t - v0) & 31));
    }
    __syncthreads();
  }
  const float rep = a.repetition ? a.repetition[row] : 1.0f, freq = a.frequency ? a.frequency[row] : 0.0f;
  const float pres = a.presence ? a.presence[row] : 0.0f;
  // (byte g of a row's words: its tokens 8 g to 8 g + 7)
  const uint8_t* allow = a.allowed ? (const uint8_t*)(a.allowed + (size_t)at * words) : nullptr;
  const uint8_t* prompt = slot >= 0 ? (const uint8_t*)(a.prompt + (size_t)slot * words) : nullptr;
  const uint8_t* output = slot >= 0 ? (const uint8_t*)(a.output + (size_t)slot * words) : nullptr;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int g = tid + i * 256, v = v0 + g * 8;
    if (v >= V) continue;
    const uint32_t open = allow ? allow[v >> 3] : 255u;
    const uint32_t in_prompt = prompt ? prompt[v >> 3] : 0u, in_output = output ? output[v >> 3] : 0u;
    const uint32_t mark = marks ? (marked[g >> 2] >> ((g & 3) * 8)) & 255 : 0u;
    const uint32_t touched = (in_prompt | in_output | mark) & open;
    if constexpr (IN_PLACE) {
      if (open == 255 && !touched) continue;
      x[i] = {};
      if (open) x[i] = load8<F32>(a.logits, here + g);
    }
    if (open != 255 || touched) {
      float f[8];
      values8(x[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t bit = 1u << e;
        if (touched & bit) {
          int count = in_output & bit ? a.counts[(size_t)slot * V + v + e] : 0, bias = 0;
          if (mark & bit) {
            for (int j = 0; j < drafted; ++j) count += a.drafted[(size_t)row * a.drafted_stride + j] == v + e;
            bias = bias_at[g * 8 + e];
          }
          if ((in_prompt & bit) || count > 0) f[e] = f[e] > 0.0f ? f[e] / rep : f[e] * rep;
          if (count > 0) f[e] = f[e] - freq * (float)count - pres;
          if (bias) f[e] += a.bias_values[bias - 1];
        }
      }
      // (a logit that nothing names keeps its bits)
      Eight<F32> y = round8<F32>(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool keeps = !((touched >> e) & 1), shut = !((open >> e) & 1);
        if constexpr (F32) {
          if (shut) x[i].w[e >> 2][e & 3] = 0xff800000u;
          else if (!keeps) x[i].w[e >> 2][e & 3] = y.w[e >> 2][e & 3];
        } else {
          const uint32_t part = e & 1 ? 0xffff0000u : 0xffffu, from = shut ? 0xff80ff80u : y.w[0][e >> 1];
          if (shut || !keeps) x[i].w[0][e >> 1] = (x[i].w[0][e >> 1] & ~part) | (from & part);
        }
      }
    }
    store8<F32>(a.out, here + g, x[i]);
  }
}

int check_vocab(int32_t vocab) {
  if (vocab > MARKOV_MAX_VOCAB) return MARKOV_ERR_VOCAB;
  return vocab < 8 || (vocab & 7) ? MARKOV_ERR_SHAPE : MARKOV_OK;
}

int64_t slabs_of(int32_t vocab) { return ((int64_t)vocab + SLAB - 1) / SLAB; }

template <bool F32>
int adjust(const markov_adjust_t& a, hipStream_t st) {
  const int64_t slabs = slabs_of(a.vocab), grid = slabs * a.rows * a.k;
  if (a.out == a.logits) adjust_kernel<F32, true><<<dim3((unsigned)grid), 256, 0, st>>>(a, (int)slabs);
  else adjust_kernel<F32, false><<<dim3((unsigned)grid), 256, 0, st>>>(a, (int)slabs);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

}  // namespace

extern "C" {

int markov_count_tokens(uint32_t* prompt, uint32_t* output, int32_t* counts, const int64_t* tokens,
                        const int32_t* lengths, const int32_t* prompt_lengths,
                        const int32_t* slots, int32_t rows, int32_t length, int32_t slots_count,
                        int32_t vocab, int32_t reset, markov_stream_t stream) {
  const int rc = check_vocab(vocab);
  if (rc) return rc;
  if (rows < 1 || length < 0 || slots_count < 1 || (int64_t)rows * length > 0x7fffffff) return MARKOV_ERR_SHAPE;
  const int64_t parts = ((int64_t)vocab + RESET - 1) / RESET;
  if (reset && parts * rows > MOST_THREADS / 256) return MARKOV_ERR_SHAPE;
  if (!prompt || !output || !counts || (length > 0 && !tokens)) return MARKOV_ERR_NULL;
  for (const void* p : {(const void*)prompt, (const void*)output, (const void*)counts, (const void*)lengths,
                        (const void*)prompt_lengths, (const void*)slots})
    if (!aligned_to(p, 4)) return MARKOV_ERR_ALIGN;
  if (!aligned_to(tokens, 8)) return MARKOV_ERR_ALIGN;
  const Count a = {prompt, output, counts, tokens, lengths, prompt_lengths, slots, rows, length, slots_count, vocab, (vocab + 31) / 32};
  const hipStream_t st = (hipStream_t)stream;
  if (reset) {
    reset_kernel<<<dim3((unsigned)(parts * rows)), 256, 0, st>>>(a, (int)parts);
    if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
  }
  if (length > 0) {
    count_kernel<<<dim3((unsigned)(((int64_t)rows * length + 255) / 256)), 256, 0, st>>>(a);
    if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
  }
  return MARKOV_OK;
}

int markov_adjust_logits(const markov_adjust_t* args, markov_stream_t stream) {
  if (!args) return MARKOV_ERR_NULL;
  const markov_adjust_t& a = *args;
  const int rc = check_vocab(a.vocab);
  if (rc) return rc;
  const bool state = a.prompt || a.output || a.counts, bias = a.bias_tokens || a.bias_values || a.bias_starts;
  if (a.rows < 1 || a.k < 1 || unknown_type(a.type) || (state && a.slots_count < 1) ||
      (a.drafted && a.drafted_stride < a.k - 1) || a.biases < 0)
    return MARKOV_ERR_SHAPE;
  if ((int64_t)a.rows * a.k > MARKOV_MAX_TOKENS) return MARKOV_ERR_ROWS;
  if (slabs_of(a.vocab) * a.rows * a.k > MOST_THREADS / 256) return MARKOV_ERR_SHAPE;
  if (!a.logits || !a.out || (state && (!a.prompt || !a.output || !a.counts)) ||
      (bias && (!a.bias_starts || (a.biases > 0 && (!a.bias_tokens || !a.bias_values)))))
    return MARKOV_ERR_NULL;
  if (!aligned_to(a.logits, 16) || !aligned_to(a.out, 16) || !aligned_to(a.drafted, 8) || !aligned_to(a.bias_tokens, 8))
    return MARKOV_ERR_ALIGN;
  for (const void* p : {(const void*)a.prompt, (const void*)a.output, (const void*)a.counts, (const void*)a.slots,
                        (const void*)a.repetition, (const void*)a.frequency, (const void*)a.presence,
                        (const void*)a.bias_values, (const void*)a.bias_starts, (const void*)a.allowed})
    if (!aligned_to(p, 4)) return MARKOV_ERR_ALIGN;
  const size_t size = (size_t)a.rows * a.k * a.vocab * size_of_type(a.type);
  if (a.out != a.logits && overlap(a.out, size, a.logits, size)) return MARKOV_ERR_VALUE;
  return a.type == MARKOV_FP32 ? adjust<true>(a, (hipStream_t)stream) : adjust<false>(a, (hipStream_t)stream);
}

}  // extern "C"
