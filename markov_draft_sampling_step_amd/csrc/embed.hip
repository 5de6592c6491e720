// MI355X (gfx950) embeddings of tokens, scaled, and the gradient of their table
// by sorted tokens.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "markov.h"
#include "numbers.h"

namespace {

// L lanes take a row, 256 / L rows a workgroup.
template <bool F32, int L>
__global__ __launch_bounds__(256) void embed_kernel(const void* table, const int64_t* tokens, void* out, int n, int V,
                                                    int groups, float scale) {
  const int lane = threadIdx.x % L, row = blockIdx.x * (256 / L) + (int)threadIdx.x / L;
  if (row >= n) return;
  const int64_t t = tokens[row];
  const bool live = t >= 0 && t < V;
  const size_t from = (size_t)(live ? t : 0) * groups, to = (size_t)row * groups;
#pragma unroll 4
  for (int c = lane; c < groups; c += L) {
    Eight<F32> e = {};
    if (live) {
      float v[8];
      values8(load8<F32>(table, from + c), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= scale;
      e = round8<F32>(v);
    }
    store8<F32>(out, to + c, e);
  }
}

// ---------------------------------------------------------------- the gradient

constexpr int ST = 1024, SW = ST / 64;   // threads and waves of the sort

struct Sort {
  const int64_t* tokens;
  uint32_t* key[2];    // a token, or V where it is none; the sorted ones end up in key[0], index[0]
  uint32_t* index[2];
  int n, V, passes;
};

// A stable sort by 8 bits at a time, the lowest first, by one workgroup: each wave
// counts the digits of its stretch of entries, the counts are added up over
// digits and waves, then each wave puts its entries where they belong, 64 at a time.
__device__ void sort_tokens(const Sort& s, uint32_t (&count)[SW][256], uint32_t (&sums)[4]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int each = ((s.n + SW - 1) / SW + 63) & ~63, first = min(wave * each, s.n), last = min(first + each, s.n);
  for (int pass = 0; pass < s.passes; ++pass) {
    // (the last pass writes to buffer 0)
    const int to = (s.passes - 1 - pass) & 1, from = to ^ 1, shift = pass * 8;
    auto key_of = [&](int i) -> uint32_t {
      if (pass) return s.key[from][i];
      const int64_t t = s.tokens[i];
      return t >= 0 && t < s.V ? (uint32_t)t : (uint32_t)s.V;
    };
    for (int i = tid; i < SW * 256; i += ST) count[i >> 8][i & 255] = 0;
    __syncthreads();
    for (int i = first + lane; i < last; i += 64) atomicAdd(&count[wave][(key_of(i) >> shift) & 255], 1u);
    __syncthreads();
    // where each wave's entries of each digit begin
    uint32_t total = 0, before = 0;
    if (tid < 256) {
      for (int w = 0; w < SW; ++w) {
        const uint32_t c = count[w][tid];
        count[w][tid] = total;
        total += c;
      }
      before = total;
#pragma unroll
      for (int sh = 1; sh < 64; sh <<= 1) {
        const uint32_t other = (uint32_t)__shfl_up((int)before, sh);
        if (lane >= sh) before += other;
      }
      if (lane == 63) sums[wave] = before;
    }
    __syncthreads();
    if (tid < 256) {
      before -= total;
      for (int w = 0; w < wave; ++w) before += sums[w];
      for (int w = 0; w < SW; ++w) count[w][tid] += before;
    }
    __syncthreads();
    for (int i0 = first; i0 < last; i0 += 64) {
      const int i = i0 + lane;
      const bool in = i < last;
      const uint32_t key = in ? key_of(i) : 0u, index = in ? pass ? s.index[from][i] : (uint32_t)i : 0u;
      const uint32_t digit = (key >> shift) & 255;
      uint64_t same = __ballot(in);   // the lanes with this lane's digit
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const uint64_t set = __ballot((digit >> b) & 1);
        same &= (digit >> b) & 1 ? set : ~set;
      }
      const int leader = in ? __ffsll((unsigned long long)same) - 1 : lane;
      uint32_t at = 0;
      if (in && lane == leader) at = atomicAdd(&count[wave][digit], (uint32_t)__popcll(same));
      at = (uint32_t)__shfl((int)at, leader) + (uint32_t)__popcll(same & ((1ull << lane) - 1));
      if (in) {
        s.key[to][at] = key;
        s.index[to][at] = index;
      }
    }
    __syncthreads();
  }
}

// The first workgroup sorts, the others fill the table with zeros meanwhile.
__global__ __launch_bounds__(ST) void sort_kernel(Sort s, u32x4_t* table, int64_t vectors) {
  __shared__ uint32_t count[SW][256], sums[4];
  if (blockIdx.x == 0) {
    sort_tokens(s, count, sums);
    return;
  }
  const int64_t step = (int64_t)(gridDim.x - 1) * ST;
  for (int64_t i = (int64_t)(blockIdx.x - 1) * ST + threadIdx.x; i < vectors; i += step)
    __builtin_nontemporal_store((u32x4_t){0u, 0u, 0u, 0u}, table + i);
}

// Entries of the sorted list that one row of lanes adds up: enough such segments
// for the chip, and few partial sums.
int segment_of(int n) {
  const int s = (n / 256) & ~7;
  return s < 8 ? 8 : s > 64 ? 64 : s;
}

struct Sums {
  const void* grad;
  const uint32_t *key, *index;
  void* table;
  float* partial;   // [segments][2][hidden]: of a token that began before the segment, of one that goes on after it
  int n, V, groups, segment, segments, chunks;
  float scale;
};

template <bool T32>
__device__ __forceinline__ void store_row(const Sums& a, uint32_t key, int c, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= a.scale;
  store8<T32>(a.table, (size_t)key * a.groups + c, round8<T32>(v));
}

// L lanes add up the rows of one segment's entries, 8 columns each: a token that
// lies within it goes to the table, others leave a partial sum.
template <bool F32, bool T32, int L>
__global__ __launch_bounds__(256) void sums_kernel(Sums a) {
  constexpr int U = 8;
  const int seg = blockIdx.x / a.chunks * (256 / L) + (int)threadIdx.x / L;
  const int c = (int)(blockIdx.x % a.chunks) * L + (int)threadIdx.x % L;
  if (seg >= a.segments || c >= a.groups) return;
  const int s0 = seg * a.segment, s1 = min(s0 + a.segment, a.n);
  float sum[8] = {};
  uint32_t now = a.key[s0];
  bool before = s0 > 0 && a.key[s0 - 1] == now;
  auto close = [&](bool after) {
    if (now < (uint32_t)a.V) {
      if (before || after)
        store8<true>(a.partial, ((size_t)seg * 2 + (before ? 0 : 1)) * a.groups + c, round8<true>(sum));
      else
        store_row<T32>(a, now, c, sum);
    }
  };
  for (int i0 = s0; i0 < s1; i0 += U) {
    uint32_t key[U];
    Eight<F32> row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u, s1 - 1);
      key[u] = a.key[i];
      row[u] = {};
      if (key[u] < (uint32_t)a.V) row[u] = load8<F32>(a.grad, (size_t)a.index[i] * a.groups + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= s1) continue;
      if (key[u] != now) {
        close(false);
        now = key[u];
        before = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
      }
      float v[8];
      values8(row[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += v[e];
    }
  }
  close(s1 < a.n && a.key[s1] == now);
}

// The tokens that go over a segment's end: the segment where one begins adds up
// its partial sums, 64 columns a workgroup, each wave a share of them.
template <bool T32>
__global__ __launch_bounds__(512) void join_kernel(Sums a) {
  const int seg = blockIdx.x / a.chunks, hidden = a.groups * 8;
  const int s0 = seg * a.segment, s1 = s0 + a.segment;
  if (s1 >= a.n) return;
  const uint32_t key = a.key[s1];
  if (key >= (uint32_t)a.V || a.key[s1 - 1] != key || (s0 > 0 && a.key[s0 - 1] == key)) return;
  int end = s1 + 1, past = a.n;   // the first entry after this token's
  while (end < past) {
    const int mid = (end + past) / 2;
    if (a.key[mid] == key) end = mid + 1;
    else past = mid;
  }
  const int last = (end - 1) / a.segment, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = (int)(blockIdx.x % a.chunks) * 64 + lane;
  float s = 0.0f;
  if (j < hidden) {
#pragma unroll 8
    for (int q = seg + wave; q <= last; q += 8) s += a.partial[((size_t)q * 2 + (q == seg ? 1 : 0)) * hidden + j];
  }
  __shared__ float part[8][64];
  part[wave][lane] = s;
  __syncthreads();
  if (wave || j >= hidden) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += part[w][lane];
  s *= a.scale;
  if constexpr (T32) ((float*)a.table)[(size_t)key * hidden + j] = s;
  else ((uint16_t*)a.table)[(size_t)key * hidden + j] = (uint16_t)pack_bf16(s, 0.0f);
}

int check_embed(int32_t n, int32_t vocab, int32_t hidden) {
  if (vocab > MARKOV_MAX_VOCAB) return MARKOV_ERR_VOCAB;
  if (n < 1 || vocab < 1 || hidden < 16 || (hidden & 15) || hidden > MARKOV_MAX_NORM_HIDDEN) return MARKOV_ERR_SHAPE;
  return n > MARKOV_MAX_TOKENS ? MARKOV_ERR_ROWS : MARKOV_OK;
}

size_t list_bytes(int32_t n) { return ((size_t)n * 4 + 255) & ~(size_t)255; }

int segments_of(int32_t n) { return (n + segment_of(n) - 1) / segment_of(n); }

template <bool F32, int L>
void launch_embed(const void* table, const int64_t* tokens, void* out, int n, int V, int groups, float scale,
                  hipStream_t st) {
  constexpr int ROWS = 256 / L;
  embed_kernel<F32, L><<<dim3((unsigned)((n + ROWS - 1) / ROWS)), 256, 0, st>>>(table, tokens, out, n, V, groups, scale);
}

template <bool F32>
void embed_by_hidden(const void* table, const int64_t* tokens, void* out, int n, int V, int groups, float scale,
                     hipStream_t st) {
  if (groups <= 16) launch_embed<F32, 16>(table, tokens, out, n, V, groups, scale, st);
  else if (groups <= 64) launch_embed<F32, 64>(table, tokens, out, n, V, groups, scale, st);
  else launch_embed<F32, 256>(table, tokens, out, n, V, groups, scale, st);
}

template <bool F32, bool T32, int L>
void launch_sums(Sums a, hipStream_t st) {
  a.chunks = (a.groups + L - 1) / L;
  const unsigned grid = (unsigned)((a.segments + 256 / L - 1) / (256 / L)) * a.chunks;
  sums_kernel<F32, T32, L><<<dim3(grid), 256, 0, st>>>(a);
}

template <bool F32, bool T32>
int sums(Sums a, hipStream_t st) {
  if (a.groups <= 16) launch_sums<F32, T32, 16>(a, st);
  else if (a.groups <= 64) launch_sums<F32, T32, 64>(a, st);
  else launch_sums<F32, T32, 256>(a, st);
  if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
  a.chunks = (a.groups + 7) / 8;
  join_kernel<T32><<<dim3((unsigned)a.segments * a.chunks), 512, 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

}  // namespace

extern "C" {

int markov_embed(const void* table, const int64_t* tokens, void* out, int32_t tokens_count,
                 int32_t vocab, int32_t hidden, int32_t type, float scale, markov_stream_t stream) {
  const int rc = check_embed(tokens_count, vocab, hidden);
  if (rc) return rc;
  if (unknown_type(type)) return MARKOV_ERR_SHAPE;
  if (!table || !tokens || !out) return MARKOV_ERR_NULL;
  if (!isfinite(scale)) return MARKOV_ERR_VALUE;
  if (!aligned_to(table, 16) || !aligned_to(out, 16) || !aligned_to(tokens, 8)) return MARKOV_ERR_ALIGN;
  const size_t row = (size_t)hidden * size_of_type(type);
  if (overlap(out, row * tokens_count, table, row * vocab) ||
      overlap(out, row * tokens_count, tokens, (size_t)tokens_count * 8))
    return MARKOV_ERR_VALUE;
  if (type == MARKOV_FP32)
    embed_by_hidden<true>(table, tokens, out, tokens_count, vocab, hidden / 8, scale, (hipStream_t)stream);
  else
    embed_by_hidden<false>(table, tokens, out, tokens_count, vocab, hidden / 8, scale, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MARKOV_OK : MARKOV_ERR_HIP;
}

size_t markov_embed_workspace_bytes(int32_t tokens_count, int32_t hidden) {
  if (check_embed(tokens_count, 1, hidden)) return 0;
  return 4 * list_bytes(tokens_count) + (size_t)segments_of(tokens_count) * 2 * hidden * 4;
}

int markov_embed_backward(const void* grad_out, const int64_t* tokens, void* grad_table,
                          int32_t tokens_count, int32_t vocab, int32_t hidden, int32_t type,
                          int32_t table_type, float scale, void* workspace,
                          size_t workspace_bytes, markov_stream_t stream) {
  const int rc = check_embed(tokens_count, vocab, hidden);
  if (rc) return rc;
  if (unknown_type(type) || unknown_type(table_type)) return MARKOV_ERR_SHAPE;
  if (!grad_out || !tokens || !grad_table || !workspace) return MARKOV_ERR_NULL;
  if (!isfinite(scale)) return MARKOV_ERR_VALUE;
  if (!aligned_to(grad_out, 16) || !aligned_to(grad_table, 16) || !aligned_to(workspace, 16) || !aligned_to(tokens, 8))
    return MARKOV_ERR_ALIGN;
  const size_t need = markov_embed_workspace_bytes(tokens_count, hidden);
  if (workspace_bytes < need) return MARKOV_ERR_WORKSPACE;
  const size_t size = (size_t)vocab * hidden * size_of_type(table_type);
  const size_t rows = (size_t)tokens_count * hidden * size_of_type(type), list = (size_t)tokens_count * 8;
  if (overlap(grad_table, size, grad_out, rows) || overlap(grad_table, size, tokens, list) ||
      overlap(grad_table, size, workspace, need) || overlap(workspace, need, grad_out, rows) ||
      overlap(workspace, need, tokens, list))
    return MARKOV_ERR_VALUE;
  uint8_t* w = (uint8_t*)workspace;
  const size_t l = list_bytes(tokens_count);
  Sort s = {tokens, {(uint32_t*)w, (uint32_t*)(w + l)}, {(uint32_t*)(w + 2 * l), (uint32_t*)(w + 3 * l)}, tokens_count, vocab, 1};
  while (s.passes < 4 && (vocab >> (8 * s.passes)) > 0) ++s.passes;
  const hipStream_t st = (hipStream_t)stream;
  const int64_t vectors = (int64_t)(size / 16);
  const int64_t fill = (vectors + 4 * ST - 1) / (4 * ST);
  sort_kernel<<<dim3((unsigned)(1 + (fill < 1024 ? fill : 1024))), ST, 0, st>>>(s, (u32x4_t*)grad_table, vectors);
  if (hipGetLastError() != hipSuccess) return MARKOV_ERR_HIP;
  const Sums a = {grad_out, s.key[0], s.index[0], grad_table, (float*)(w + 4 * l), tokens_count, vocab, hidden / 8,
                  segment_of(tokens_count), segments_of(tokens_count), 0, scale};
  if (type == MARKOV_FP32) return table_type == MARKOV_FP32 ? sums<true, true>(a, st) : sums<true, false>(a, st);
  return table_type == MARKOV_FP32 ? sums<false, true>(a, st) : sums<false, false>(a, st);
}

}  // extern "C"
