// Embedding lookup with scaling and an addend, and its gradient by sorted tokens
// (fsdp_embedding, fsdp_embedding_backward).
//
//   out_r = scale table[token_r] + addend_r
//   dtable_v (+)= scale sum over the rows r with token_r = v of dout_r
//
// Gradient. The rows are put in the order of their tokens (a stable radix sort of row
// indexes by token, so equal tokens keep the rows' order), and the sorted list is cut into chunks of
// kChunk rows. A block adds the rows of a chunk, run by run of equal tokens, for
// its columns: a run that lies in the chunk goes to the table at once, the parts of
// one that crosses chunks go to the workspace in fp32 and are added in order by a second
// kernel. Every sum is fp32 in an order fixed by the tokens alone.
#include "host_internal.h"
#include "launch.h"
#include "strided.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace fsdp {
namespace {

__device__ __forceinline__ void begin_after_previous() {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ int64_t index_at(const void* p, int bits, int64_t i) {
  return bits == 64 ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

__device__ __forceinline__ void unpack_bf16(uint32_t two, float* v) {
  v[0] = __uint_as_float(two << 16);
  v[1] = __uint_as_float(two & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&two);
}

// kVec consecutive elements (kVec > 1: at a 16-byte boundary).
template <int kVec>
__device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[kVec]) {
  if constexpr (kVec == 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    unpack_bf16(a.x, v), unpack_bf16(a.y, v + 2), unpack_bf16(a.z, v + 4), unpack_bf16(a.w, v + 6);
  } else {
    v[0] = __bfloat162float(*p);
  }
}
template <int kVec>
__device__ __forceinline__ void load(const float* p, float (&v)[kVec]) {
  if constexpr (kVec == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = *p;
  }
}
template <int kVec>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[kVec]) {
  if constexpr (kVec == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else
    *p = __float2bfloat16_rn(v[0]);
}
template <int kVec>
__device__ __forceinline__ void store(float* p, const float (&v)[kVec]) {
  if constexpr (kVec == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}

// -------------------------------------------------------------------- lookup

struct LookupParams {
  const void* tokens;
  const void* table;
  const void* addend;
  void* out;
  int64_t rows, cols, vocab, table_stride, addend_stride, out_stride;
  int32_t index_bits;
  float scale;
};

constexpr int kLookupThreads = 128;

template <typename T, int kVec>
__global__ void __launch_bounds__(kLookupThreads) embed_rows(const __grid_constant__ LookupParams p) {
  begin_after_previous();
  const int64_t groups = (p.cols + kVec - 1) / kVec, per_row = (groups + kLookupThreads - 1) / kLookupThreads;
  const int64_t blocks = p.rows * per_row;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t row = b / per_row, col = ((b - row * per_row) * kLookupThreads + threadIdx.x) * kVec;
    if (col >= p.cols) continue;
    const int64_t token = index_at(p.tokens, p.index_bits, row);
    float v[kVec];
    if (token >= 0 && token < p.vocab) {
      load<kVec>(static_cast<const T*>(p.table) + token * p.table_stride + col, v);
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[e] *= p.scale;
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[e] = token < 0 ? 0.0f : NAN;
    }
    if (p.addend) {
      float a[kVec];
      load<kVec>(static_cast<const T*>(p.addend) + row * p.addend_stride + col, a);
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[e] += a[e];
    }
    store<kVec>(static_cast<T*>(p.out) + row * p.out_stride + col, v);
  }
}

// ---------------------------------------------------------------------- sort

constexpr int kSortThreads = 256, kSortItems = 8, kSortBlock = kSortThreads * kSortItems;
constexpr int kMaxBins = 512;

struct SortParams {
  const void* tokens;      // first pass: the caller's, else null
  int32_t index_bits;
  int64_t vocab;
  const uint32_t *keys_in, *rows_in;
  uint32_t *keys_out, *rows_out;
  uint32_t* counts;        // [bin][block], then their running sums
  int32_t n, blocks, shift, bins;
};

// Tokens that are no row of the table are sorted behind the others.
__device__ __forceinline__ uint32_t sort_key(const SortParams& p, int i) {
  if (!p.tokens) return p.keys_in[i];
  const int64_t t = index_at(p.tokens, p.index_bits, i);
  return static_cast<uint32_t>(t >= 0 && t < p.vocab ? t : p.vocab);
}

__global__ void __launch_bounds__(kSortThreads) sort_count(const __grid_constant__ SortParams p) {
  begin_after_previous();
  __shared__ uint32_t bins[kMaxBins];
  for (int b = threadIdx.x; b < p.bins; b += kSortThreads) bins[b] = 0;
  __syncthreads();
  for (int k = 0; k < kSortItems; ++k) {
    const int i = blockIdx.x * kSortBlock + k * kSortThreads + threadIdx.x;
    if (i < p.n) atomicAdd(&bins[(sort_key(p, i) >> p.shift) & (p.bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < p.bins; b += kSortThreads) p.counts[b * p.blocks + blockIdx.x] = bins[b];
}

// Exclusive running sums of counts, in place, by one block.
__global__ void __launch_bounds__(1024) sort_offsets(const __grid_constant__ SortParams p) {
  begin_after_previous();
  __shared__ uint32_t warps[32];
  __shared__ uint32_t carry;
  const int n = p.bins * p.blocks, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (threadIdx.x == 0) carry = 0;
  for (int i0 = 0; i0 < n; i0 += 4096) {
    uint32_t v[4], sum = 0;
    const int at = i0 + threadIdx.x * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = at + e < n ? p.counts[at + e] : 0;
      sum += v[e];
    }
    uint32_t run = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += u;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = run;
    __syncthreads();
    uint32_t before = carry;
    for (int w = 0; w < warp; ++w) before += warps[w];
    uint32_t next = before + run - sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (at + e < n) p.counts[at + e] = next;
      next += v[e];
    }
    __syncthreads();
    if (threadIdx.x == 1023) carry = next;
    __syncthreads();
  }
}

// Moves the block's items to their places: 32 at a time for each warp, in the order of the input.
__global__ void __launch_bounds__(kSortThreads) sort_move(const __grid_constant__ SortParams p) {
  begin_after_previous();
  constexpr int kWarps = kSortThreads / 32;
  __shared__ uint32_t next[kWarps][kMaxBins];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int b = threadIdx.x; b < kWarps * kMaxBins; b += kSortThreads) next[b / kMaxBins][b % kMaxBins] = 0;
  __syncthreads();
  const int first = blockIdx.x * kSortBlock + warp * (kSortItems * 32) + lane;
  uint32_t key[kSortItems], rank[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = first + k * 32;
    key[k] = i < p.n ? sort_key(p, i) : 0;
    const uint32_t bin = i < p.n ? (key[k] >> p.shift) & (p.bins - 1) : 0xffffffffu;
    const uint32_t same = __match_any_sync(0xffffffffu, bin);
    const uint32_t below = same & ((1u << lane) - 1);
    uint32_t old = 0;
    if (i < p.n) old = next[warp][bin];
    __syncwarp();
    if (i < p.n && below == 0) next[warp][bin] = old + __popc(same);
    __syncwarp();
    rank[k] = old + __popc(below);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < p.bins; b += kSortThreads) {
    uint32_t at = p.counts[b * p.blocks + blockIdx.x];
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t count = next[w][b];
      next[w][b] = at;
      at += count;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = first + k * 32;
    if (i >= p.n) continue;
    const uint32_t to = next[warp][(key[k] >> p.shift) & (p.bins - 1)] + rank[k];
    p.keys_out[to] = key[k];
    p.rows_out[to] = p.tokens ? static_cast<uint32_t>(i) : p.rows_in[i];
  }
}

// ------------------------------------------------------------------ gradient

constexpr int kChunk = 32;
constexpr int kSumThreads = 128;

struct SumParams {
  const uint32_t *keys, *rows;  // sorted
  int32_t n, chunks;
  int32_t tiles, join_tiles;    // blocks of columns of a chunk, in the two kernels
  int64_t vocab, cols;
  const void* dout;
  int64_t dout_stride;
  void* dtable;
  int64_t dtable_stride;
  float* parts;                 // [2 chunk + (0: the run that came in, 1: the run that goes on)][part_stride]
  int64_t part_stride;
  float scale;
  bool accumulate;
};

template <typename TTable, int kVec>
__device__ __forceinline__ void finish_row(const SumParams& p, uint32_t token, int64_t col, float (&sum)[kVec]) {
  TTable* to = static_cast<TTable*>(p.dtable) + token * p.dtable_stride + col;
  float old[kVec] = {};
  if (p.accumulate) load<kVec>(to, old);
#pragma unroll
  for (int e = 0; e < kVec; ++e) sum[e] = old[e] + sum[e] * p.scale;
  store<kVec>(to, sum);
}

template <typename T, typename TTable, int kVec>
__global__ void __launch_bounds__(kSumThreads) embed_sum(const __grid_constant__ SumParams p) {
  begin_after_previous();
  __shared__ uint32_t keys[kChunk + 2], rows[kChunk];  // keys[0]: of the row before the chunk; the last: behind it
  const int chunk = blockIdx.x / p.tiles, tile = blockIdx.x - chunk * p.tiles;
  const int first = chunk * kChunk, count = min(kChunk, p.n - first);
  const uint32_t none = static_cast<uint32_t>(p.vocab);
  for (int i = threadIdx.x; i < kChunk + 2; i += kSumThreads) {
    const int at = first + i - 1;
    keys[i] = at >= 0 && at < p.n ? p.keys[at] : none;
    if (i >= 1 && i <= count) rows[i - 1] = p.rows[at];
  }
  __syncthreads();
  const int64_t col = (static_cast<int64_t>(tile) * kSumThreads + threadIdx.x) * kVec;
  if (col >= p.cols) return;
  const T* dout = static_cast<const T*>(p.dout) + col;
  float sum[kVec] = {};
  int begin = 0;
  for (int i = 0; i < count && keys[i + 1] != none; ++i) {
    float v[kVec];
    load<kVec>(dout + rows[i] * p.dout_stride, v);
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum[e] += v[e];
    const bool last = i + 1 == count;
    if (!last && keys[i + 2] == keys[i + 1]) continue;
    const bool came = begin == 0 && first > 0 && keys[0] == keys[1];
    const bool goes = last && keys[count + 1] == keys[count];
    if (came || goes) {
      store<kVec>(p.parts + (2 * static_cast<int64_t>(chunk) + (came ? 0 : 1)) * p.part_stride + col, sum);
    } else {
      finish_row<TTable, kVec>(p, keys[i + 1], col, sum);
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum[e] = 0.0f;
    begin = i + 1;
  }
}

// Adds up a run that begins in this block's chunk and goes on behind it: eight
// groups of threads each a share of the chunks, then the groups in order.
constexpr int kJoinGroups = 8;

template <typename TTable, int kVec>
__global__ void __launch_bounds__(32 * kJoinGroups) embed_join(const __grid_constant__ SumParams p) {
  begin_after_previous();
  const int chunk = blockIdx.x / p.join_tiles, end = min(p.n, (chunk + 1) * kChunk);
  const uint32_t none = static_cast<uint32_t>(p.vocab);
  if (end >= p.n) return;
  const uint32_t token = p.keys[end - 1];
  if (token == none || p.keys[end] != token) return;
  if (chunk > 0 && p.keys[chunk * kChunk] == token && p.keys[chunk * kChunk - 1] == token) return;  // began before
  int lo = end, hi = p.n;  // the run's end: the first key beyond `token`
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (p.keys[mid] == token) lo = mid + 1;
    else hi = mid;
  }
  const int last = (lo - 1) / kChunk, parts = last - chunk;  // after the first one
  const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
  const int each = (parts + kJoinGroups - 1) / kJoinGroups;
  const int from = chunk + 1 + min(parts, group * each), to = chunk + 1 + min(parts, (group + 1) * each);
  const int64_t col = (static_cast<int64_t>(blockIdx.x - chunk * p.join_tiles) * 32 + lane) * kVec;
  __shared__ float sums[kJoinGroups][kVec][32];
  float sum[kVec] = {};
  if (col < p.cols) {
    if (group == 0) load<kVec>(p.parts + (2 * static_cast<int64_t>(chunk) + 1) * p.part_stride + col, sum);
    for (int c = from; c < to; ++c) {
      float v[kVec];
      load<kVec>(p.parts + 2 * static_cast<int64_t>(c) * p.part_stride + col, v);
#pragma unroll
      for (int e = 0; e < kVec; ++e) sum[e] += v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < kVec; ++e) sums[group][e][lane] = sum[e];
  __syncthreads();
  if (group != 0 || col >= p.cols) return;
#pragma unroll
  for (int g = 1; g < kJoinGroups; ++g)
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum[e] += sums[g][e][lane];
  finish_row<TTable, kVec>(p, token, col, sum);
}

// ---------------------------------------------------------------------- host

constexpr int64_t kMaxCols = int64_t(1) << 30, kMaxVocab = int64_t(1) << 30, kMaxRows = int64_t(1) << 30;

int64_t round_to(int64_t n, int64_t k) { return (n + k - 1) / k * k; }

bool vector_rows(const void* p, int64_t rows, int64_t stride, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows < 2 || stride * size % 16 == 0);
}

struct Workspace {
  int64_t keys[2], rows[2], counts, parts, bytes;
  int64_t part_stride;
  int32_t chunks, blocks;
};

Workspace carve(int64_t rows, int64_t cols) {
  Workspace w{};
  int64_t at = 256;  // the caller's pointer may have any alignment
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_to(bytes, 256);
    return here;
  };
  w.chunks = static_cast<int32_t>((rows + kChunk - 1) / kChunk);
  w.blocks = static_cast<int32_t>((rows + kSortBlock - 1) / kSortBlock);
  w.part_stride = round_to(cols, 8);
  for (int k = 0; k < 2; ++k) {
    w.keys[k] = take(rows * 4);
    w.rows[k] = take(rows * 4);
  }
  w.counts = take(static_cast<int64_t>(w.blocks) * kMaxBins * 4);
  w.parts = take(2 * static_cast<int64_t>(w.chunks) * w.part_stride * 4);
  w.bytes = at;
  return w;
}

template <typename T, typename TTable, int kVec>
int run_sum(SumParams p, cudaStream_t st) {
  const int64_t groups = (p.cols + kVec - 1) / kVec;
  const int64_t tiles = (groups + kSumThreads - 1) / kSumThreads, join_tiles = (groups + 31) / 32;
  if (join_tiles * p.chunks > INT32_MAX) return FSDP_EINVAL;  // more than any memory holds
  p.tiles = static_cast<int32_t>(tiles);
  p.join_tiles = static_cast<int32_t>(join_tiles);
  if (int rc = launch_after(embed_sum<T, TTable, kVec>, p.chunks * p.tiles, 1, kSumThreads, 0, st, p)) return rc;
  return launch_after(embed_join<TTable, kVec>, p.chunks * p.join_tiles, 1, 32 * kJoinGroups, 0, st, p);
}

template <typename T, typename TTable>
int run_sum_as(const SumParams& p, bool vectors, cudaStream_t st) {
  return vectors ? run_sum<T, TTable, 8>(p, st) : run_sum<T, TTable, 1>(p, st);
}

bool is_index(int32_t dtype) { return dtype == FSDP_DTYPE_I32 || dtype == FSDP_DTYPE_I64; }
bool is_float(int32_t dtype) { return dtype == FSDP_DTYPE_F32 || dtype == FSDP_DTYPE_BF16; }

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" int fsdp_embedding(const fsdp_embedding_t* a, const void* tokens, const void* table, const void* addend,
                              void* out, fsdp_stream_t stream) {
  if (!a || a->rows < 0 || a->rows > kMaxRows || a->cols < 1 || a->cols > kMaxCols || a->vocab < 1 || a->vocab > kMaxVocab)
    return FSDP_EINVAL;
  if (!is_float(a->dtype) || !is_index(a->token_dtype) || !std::isfinite(static_cast<float>(a->scale))) return FSDP_EINVAL;
  if (a->rows == 0) return FSDP_OK;
  const int es = size_of_dtype(a->dtype), is = size_of_dtype(a->token_dtype);
  const Strided st{tokens, 1, a->rows, a->rows, is}, sw{table, a->vocab, a->cols, a->table_stride, es},
      sa{addend, a->rows, a->cols, a->addend_stride, es}, so{out, a->rows, a->cols, a->out_stride, es};
  if (!st.ok() || !sw.ok() || !so.ok() || (addend && !sa.ok())) return FSDP_EINVAL;
  if (so.overlaps(st) || so.overlaps(sw) || (addend && so.overlaps(sa) && !so.same_place(sa))) return FSDP_EALIAS;
  const LookupParams p{tokens, table, addend, out, a->rows, a->cols, a->vocab, a->table_stride, a->addend_stride,
                       a->out_stride, 8 * is, static_cast<float>(a->scale)};
  const bool vectors = a->cols % 8 == 0 && vector_rows(table, a->vocab, a->table_stride, es) &&
                       vector_rows(out, a->rows, a->out_stride, es) &&
                       (!addend || vector_rows(addend, a->rows, a->addend_stride, es));
  const int64_t groups = vectors ? a->cols / 8 : a->cols;
  const int grid = static_cast<int>(std::min<int64_t>(a->rows * ((groups + kLookupThreads - 1) / kLookupThreads), 1 << 20));
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (a->dtype == FSDP_DTYPE_F32)
    return launch_after(vectors ? embed_rows<float, 8> : embed_rows<float, 1>, grid, 1, kLookupThreads, 0, cs, p);
  return launch_after(vectors ? embed_rows<__nv_bfloat16, 8> : embed_rows<__nv_bfloat16, 1>, grid, 1, kLookupThreads, 0, cs, p);
}

extern "C" int fsdp_embedding_backward_workspace(int64_t rows, int64_t cols, int64_t vocab, int64_t* bytes_out) {
  if (!bytes_out || rows < 0 || rows > kMaxRows || cols < 1 || cols > kMaxCols || vocab < 1 || vocab > kMaxVocab)
    return FSDP_EINVAL;
  *bytes_out = carve(rows, cols).bytes;
  return FSDP_OK;
}

extern "C" int fsdp_embedding_backward(const fsdp_embedding_backward_t* a, const void* tokens, const void* dout,
                                       void* dtable, void* workspace, int64_t workspace_bytes, fsdp_stream_t stream) {
  if (!a || !is_float(a->dtype) || !is_float(a->table_dtype) || !is_index(a->token_dtype) ||
      !std::isfinite(static_cast<float>(a->scale)))
    return FSDP_EINVAL;
  int64_t need = 0;
  if (int rc = fsdp_embedding_backward_workspace(a->rows, a->cols, a->vocab, &need)) return rc;
  const int es = size_of_dtype(a->dtype), ts = size_of_dtype(a->table_dtype), is = size_of_dtype(a->token_dtype);
  const Strided st{tokens, 1, a->rows, a->rows, is}, sd{dout, a->rows, a->cols, a->dout_stride, es},
      sw{dtable, a->vocab, a->cols, a->dtable_stride, ts}, ws{workspace, 1, need, need, 1};
  if (!sw.ok()) return FSDP_EINVAL;
  if (a->rows > 0) {
    if (!st.ok() || !sd.ok() || !ws.ok()) return FSDP_EINVAL;
    if (workspace_bytes < need) return FSDP_EWORKSPACE;
    if (sw.overlaps(st) || sw.overlaps(sd) || sw.overlaps(ws) || ws.overlaps(st) || ws.overlaps(sd)) return FSDP_EALIAS;
  }
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (!a->accumulate &&
      cudaMemset2DAsync(dtable, static_cast<size_t>(sw.pitch() ? sw.pitch() : a->cols * ts), 0,
                        static_cast<size_t>(a->cols) * ts, static_cast<size_t>(a->vocab), cs) != cudaSuccess)
    return FSDP_ECUDA;
  if (a->rows == 0) return FSDP_OK;

  const Workspace w = carve(a->rows, a->cols);
  auto* base = reinterpret_cast<unsigned char*>(round_to(reinterpret_cast<intptr_t>(workspace), 256) - 256);
  uint32_t *keys[2], *rows[2];
  for (int k = 0; k < 2; ++k) {
    keys[k] = reinterpret_cast<uint32_t*>(base + w.keys[k]);
    rows[k] = reinterpret_cast<uint32_t*>(base + w.rows[k]);
  }
  int bits = 1;
  while (a->vocab >> bits) ++bits;  // of the keys 0 .. vocab
  const int passes = (bits + 8) / 9, digit = (bits + passes - 1) / passes;
  int now = 0;
  for (int k = 0; k < passes; ++k, now ^= 1) {
    const SortParams p{k == 0 ? tokens : nullptr, 8 * is, a->vocab, keys[now], rows[now], keys[now ^ 1], rows[now ^ 1],
                       reinterpret_cast<uint32_t*>(base + w.counts), static_cast<int32_t>(a->rows), w.blocks, k * digit, 1 << digit};
    if (int rc = launch_after(sort_count, w.blocks, 1, kSortThreads, 0, cs, p)) return rc;
    if (int rc = launch_after(sort_offsets, 1, 1, 1024, 0, cs, p)) return rc;
    if (int rc = launch_after(sort_move, w.blocks, 1, kSortThreads, 0, cs, p)) return rc;
  }
  const SumParams p{keys[now], rows[now], static_cast<int32_t>(a->rows), w.chunks, 0, 0, a->vocab, a->cols, dout, a->dout_stride,
                    dtable, a->dtable_stride, reinterpret_cast<float*>(base + w.parts), w.part_stride,
                    static_cast<float>(a->scale), a->accumulate != 0};
  const bool vectors = a->cols % 8 == 0 && vector_rows(dout, a->rows, a->dout_stride, es) &&
                       vector_rows(dtable, a->vocab, a->dtable_stride, ts);
  const bool in32 = a->dtype == FSDP_DTYPE_F32, table32 = a->table_dtype == FSDP_DTYPE_F32;
  return in32 ? table32 ? run_sum_as<float, float>(p, vectors, cs) : run_sum_as<float, __nv_bfloat16>(p, vectors, cs)
         : table32 ? run_sum_as<__nv_bfloat16, float>(p, vectors, cs) : run_sum_as<__nv_bfloat16, __nv_bfloat16>(p, vectors, cs);
}
