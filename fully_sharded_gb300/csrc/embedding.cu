// Embedding lookup with scaling and an addend, and its gradient by sorted tokens
// (fsdp_embedding, fsdp_embedding_backward).
//
//   out_r = scale table[token_r] + addend_r
//   dtable_v (+)= scale sum over the rows r with token_r = v of dout_r
//
// Gradient. The rows are put in the order of their tokens (places counted, or a stable radix sort of row
// indexes by token: equal tokens keep the rows' order), and the sorted list is cut into chunks of
// 16 rows. A block adds the rows of a chunk, run by run of equal tokens, for
// its columns: a run that lies in the chunk goes to the table at once, the parts of
// one that crosses chunks go to the workspace in fp32 and are added in order by a
// last kernel. Every sum is fp32 in an order fixed by the tokens alone.
// Where the table is not added to, zeros go to its other rows: to all of a small table during the sort,
// by the SMs that have no part in it; to the rows that no token names of a large table, by blocks between
// those that add.
#include "host_internal.h"
#include "launch.h"
#include "strided.h"
#include "tensor_core.cuh"

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

// kVec consecutive elements (kVec > 1: at a boundary of their size, 16 bytes at most).
template <int kVec>
__device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[kVec]) {
  if constexpr (kVec == 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    unpack_bf16(a.x, v), unpack_bf16(a.y, v + 2), unpack_bf16(a.z, v + 4), unpack_bf16(a.w, v + 6);
  } else if constexpr (kVec == 4) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    unpack_bf16(a.x, v), unpack_bf16(a.y, v + 2);
  } else {
    v[0] = __bfloat162float(*p);
  }
}
template <int kVec>
__device__ __forceinline__ void load(const float* p, float (&v)[kVec]) {
  if constexpr (kVec >= 4) {
#pragma unroll
    for (int e = 0; e < kVec; e += 4) {
      const float4 a = *reinterpret_cast<const float4*>(p + e);
      v[e] = a.x, v[e + 1] = a.y, v[e + 2] = a.z, v[e + 3] = a.w;
    }
  } else {
    v[0] = *p;
  }
}
template <int kVec>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[kVec]) {
  if constexpr (kVec == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else if constexpr (kVec == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  else
    *p = __float2bfloat16_rn(v[0]);
}
template <int kVec>
__device__ __forceinline__ void store(float* p, const float (&v)[kVec]) {
  if constexpr (kVec >= 4) {
#pragma unroll
    for (int e = 0; e < kVec; e += 4) *reinterpret_cast<float4*>(p + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  } else {
    *p = v[0];
  }
}

// kVec elements as they lie in memory.
template <typename T, int kVec>
struct alignas(sizeof(T) * kVec < 16 ? sizeof(T) * kVec : 16) Piece {
  T v[kVec];
  __device__ __forceinline__ void to(float (&x)[kVec]) const { load<kVec>(v, x); }
};

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

constexpr int kLookupWarps = 8;

// How many groups of kVec elements a lane has in flight.
template <int kVec>
constexpr int kGroups = kVec > 1 ? 4 : 8;

// A warp takes 32 kGroups kVec consecutive elements of a row (a unit) at a time; the next token is on its way meanwhile,
// with kAhead the next unit too. Bound by HBM; the rows stay packed until they are used, so that many warps fit.
// kAhead takes the registers of two units, which pays where nearly all lanes have their part (bf16, units of 1024:
// 16384 x 4096 31.3 us against 34.9, but 60000 x 1032 37.7 against 32.2; fp32, units of 512: 30000 x 1000 27.1 against 31.0).
// Off 16-byte boundaries an element a lane, kVec 1 (16384 x 4096 of evenly drawn tokens 61 us, 43 by vectors).
template <typename T, int kVec, bool kAdd, bool kAhead>
__global__ void __launch_bounds__(32 * kLookupWarps) embed_rows(const __grid_constant__ LookupParams p) {
  begin_after_previous();
  constexpr int kQ = kGroups<kVec>, kUnit = 32 * kQ * kVec;
  const uint32_t per_row = static_cast<uint32_t>((p.cols + kUnit - 1) / kUnit);
  const int64_t units = p.rows * per_row, step = static_cast<int64_t>(gridDim.x) * kLookupWarps;
  const int lane = threadIdx.x % 32;
  const auto row_of = [&](int64_t u) { return units >> 31 ? u / per_row : static_cast<uint32_t>(u) / per_row; };
  struct Unit {  // a unit on its way
    int64_t row, col;
    bool there;
    float none;
    Piece<T, kVec> v[kQ], a[kAdd ? kQ : 1];
  };
  const auto fetch = [&](Unit& w, int64_t u, int64_t token) {
    w.row = row_of(u);
    w.col = (u - w.row * per_row) * kUnit + lane * kVec;
    w.there = token >= 0 && token < p.vocab;
    w.none = token < 0 ? 0.0f : NAN;
    const T* from = static_cast<const T*>(p.table) + (w.there ? token : 0) * p.table_stride + w.col;
    const T* addend = static_cast<const T*>(p.addend) + w.row * p.addend_stride + w.col;
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      if (w.col + q * 32 * kVec < p.cols) {
        w.v[q] = *reinterpret_cast<const Piece<T, kVec>*>(from + q * 32 * kVec);
        if constexpr (kAdd) w.a[q] = *reinterpret_cast<const Piece<T, kVec>*>(addend + q * 32 * kVec);
      }
  };
  const auto finish = [&](const Unit& w) {
    T* out = static_cast<T*>(p.out) + w.row * p.out_stride + w.col;
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      if (w.col + q * 32 * kVec < p.cols) {
        float x[kVec], y[kVec] = {};
        w.v[q].to(x);
        if constexpr (kAdd) w.a[q].to(y);
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] = (w.there ? x[e] * p.scale : w.none) + (kAdd ? y[e] : 0.0f);
        store<kVec>(out + q * 32 * kVec, x);
      }
  };
  const auto token_of = [&](int64_t u) { return u < units ? index_at(p.tokens, p.index_bits, row_of(u)) : 0; };
  int64_t u = static_cast<int64_t>(blockIdx.x) * kLookupWarps + threadIdx.x / 32;
  if (u >= units) return;
  Unit one;
  if constexpr (!kAhead) {
    for (int64_t token = token_of(u); u < units; u += step) {
      fetch(one, u, token);
      token = token_of(u + step);
      finish(one);
    }
    return;
  }
  Unit two;
  int64_t token = token_of(u + step);
  fetch(one, u, token_of(u));
  for (;;) {
    u += step;
    if (u >= units) break;
    int64_t next = token_of(u + step);
    fetch(two, u, token);
    finish(one);
    u += step;
    if (u >= units) {
      finish(two);
      return;
    }
    token = token_of(u + step);
    fetch(one, u, next);
    finish(two);
  }
  finish(one);
}

// ---------------------------------------------------------------------- sort

// Zeros: rows of `row_bytes` bytes, `pitch` apart, by `parts` blocks of which this is number `part`.
struct FillParams {
  unsigned char* to;
  int64_t rows, row_bytes, pitch;  // row_bytes 0: nothing
};

// A row's bytes (an even number from an even address): vectors inside, 2 bytes at a time at the ends.
__device__ __forceinline__ void fill_row(unsigned char* row, int64_t bytes, int64_t first, int64_t step) {
  const int64_t head = min(bytes, static_cast<int64_t>(-reinterpret_cast<uintptr_t>(row) & 15u));
  const int64_t vectors = (bytes - head) / 16, tail = head + vectors * 16;
  for (int64_t i = first; i < vectors; i += step) reinterpret_cast<uint4*>(row + head)[i] = make_uint4(0, 0, 0, 0);
  for (int64_t i = first; i < head / 2; i += step) reinterpret_cast<uint16_t*>(row)[i] = 0;
  for (int64_t i = first; i < (bytes - tail) / 2; i += step) reinterpret_cast<uint16_t*>(row + tail)[i] = 0;
}

__device__ __forceinline__ void fill_zeros(const FillParams& f, int part, int parts) {
  if (f.row_bytes == 0) return;
  if (f.rows == 1) {
    fill_row(f.to, f.row_bytes, static_cast<int64_t>(part) * blockDim.x + threadIdx.x, static_cast<int64_t>(parts) * blockDim.x);
    return;
  }
  const int warps = blockDim.x / 32;
  for (int64_t r = static_cast<int64_t>(part) * warps + threadIdx.x / 32; r < f.rows; r += static_cast<int64_t>(parts) * warps)
    fill_row(f.to + r * f.pitch, f.row_bytes, threadIdx.x % 32, 32);
}

// Up to 8192 rows: every row's place is counted, as the number of rows with a smaller token, or the same token before
// it. A block finds the places of 64 rows, 8 by each warp, whose lanes share out the comparisons with all rows.
// Bound by those, 2 instructions each; in fp32 (tokens below 2^24 are exact), because integer additions and all
// comparisons run at half its rate (8192 rows 13 us by integers).
constexpr int kRankRows = 8192, kRankTile = 64, kRankEach = 8, kRankThreads = 1024, kRankWarps = kRankThreads / 32;
constexpr int64_t kRankVocab = (1 << 24) - 2;

struct RankParams {
  const void* tokens;
  uint32_t *keys, *rows;
  uint32_t* active;        // lists that embed_sum makes: their counts
  int64_t vocab;
  int32_t index_bits, n, tiles;
  FillParams fill;
};

__device__ __forceinline__ uint32_t key_of(int64_t token, int64_t vocab) {
  // tokens that are no row of the table are sorted behind the others
  return static_cast<uint32_t>(token >= 0 && token < vocab ? token : vocab);
}

__global__ void __launch_bounds__(kRankThreads) embed_rank(const __grid_constant__ RankParams p) {
  begin_after_previous();
  if (static_cast<int>(blockIdx.x) >= p.tiles) {
    fill_zeros(p.fill, blockIdx.x - p.tiles, gridDim.x - p.tiles);
    return;
  }
  extern __shared__ float4 rank_shared[];  // the rows' keys, four to a vector
  constexpr int kShares = kRankWarps * kRankEach / kRankTile;  // warps that share 8 rows
  __shared__ float counts[kShares][kRankTile];
  float* keys = reinterpret_cast<float*>(rank_shared);
  if (blockIdx.x == 0 && threadIdx.x < 2) p.active[threadIdx.x] = 0;
  const int vectors = (p.n + 3) / 4;
#pragma unroll 4
  for (int i = threadIdx.x; i < 4 * vectors; i += kRankThreads)  // behind the last row: smaller than none
    keys[i] = i < p.n ? static_cast<float>(key_of(index_at(p.tokens, p.index_bits, i), p.vocab)) : 3e38f;
  __syncthreads();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, first = blockIdx.x * kRankTile;
  const int group = warp / kShares * kRankEach, share = warp % kShares * 32 + lane;
  float own[kRankEach], count[kRankEach] = {};
#pragma unroll
  for (int k = 0; k < kRankEach; ++k) own[k] = first + group + k < p.n ? keys[first + group + k] : 0.0f;
  const auto compare = [&](int from, int to, float or_same) {
#pragma unroll 2
    for (int v = from + share; v < to; v += 32 * kShares) {
      const float4 other = rank_shared[v];
#pragma unroll
      for (int k = 0; k < kRankEach; ++k) {  // bound - other, cut to [0, 1], is 1 where other is smaller and 0 elsewhere
        const float bound = own[k] + or_same;
        count[k] += __saturatef(bound - other.x);
        count[k] += __saturatef(bound - other.y);
        count[k] += __saturatef(bound - other.z);
        count[k] += __saturatef(bound - other.w);
      }
    }
  };
  compare(0, first / 4, 1.0f);                                 // rows before the tile: the same token counts too
  compare((first + kRankTile) / 4, vectors, 0.0f);             // rows behind it
  for (int j = first + share; j < min(first + kRankTile, p.n); j += 32 * kShares) {
    const float other = keys[j];
#pragma unroll
    for (int k = 0; k < kRankEach; ++k) count[k] += other < own[k] || (other == own[k] && j < first + group + k) ? 1.0f : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < kRankEach; ++k) {
    const uint32_t sum = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(count[k]));
    if (lane == 0) counts[warp % kShares][group + k] = static_cast<float>(sum);
  }
  __syncthreads();
  const int row = first + static_cast<int>(threadIdx.x);
  if (threadIdx.x >= kRankTile || row >= p.n) return;
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kShares; ++w) sum += counts[w][threadIdx.x];
  const int place = static_cast<int>(sum);
  p.keys[place] = static_cast<uint32_t>(keys[row]);
  p.rows[place] = row;
}

// Up to 8 x 8192 rows are sorted by one cluster of up to eight blocks, which holds them in
// registers and moves them through (distributed) shared memory. In a pass each warp ranks its rows by digit, 32 at a
// time; the places follow from the counts of all digits, blocks and warps. Bound by its own latencies (cycles of a
// pass of 16384 rows on eight blocks: ranking 3000, running sums 1300, exchange of the blocks' totals 2000, their sums
// 500, moving 2000 and waiting for it 2100).
constexpr int kMaxBins = 512;
constexpr int kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32, kMaxRounds = 8, kMaxCluster = 8;
constexpr int kClusterRows = kMaxCluster * kMaxRounds * kClusterThreads;

struct ClusterSortParams {
  const void* tokens;
  uint32_t *keys, *rows;
  uint32_t* active;        // as above
  int64_t vocab;
  int32_t index_bits, n, cluster, rounds, passes, digit;
  FillParams fill;
};

__device__ __forceinline__ void remote_store(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ uint32_t remote_load(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The lanes whose `bin` (of `bits`, at most nine) is this lane's, by a ballot for each bit: a match of 32 lanes takes
// several times as long.
__device__ __forceinline__ uint32_t same_bin(uint32_t bin, int bits, bool there) {
  uint32_t same = __ballot_sync(0xffffffffu, there);
#pragma unroll
  for (int b = 0; b < 9; ++b) {
    if (b > 4 && b >= bits) break;
    const bool set = bin >> b & 1;
    const uint32_t others = __ballot_sync(0xffffffffu, set);
    same &= set ? others : ~others;
  }
  return same;
}

// A row's place among those of its warp with the same digit (lanes in order, earlier steps first), counted in `count`.
__device__ __forceinline__ uint32_t rank_in_warp(uint32_t* count, uint32_t bin, uint32_t same, bool there, int lane) {
  const uint32_t below = same & ((1u << lane) - 1);
  uint32_t old = 0;
  if (there) old = count[bin];
  __syncwarp();
  if (there && below == 0) count[bin] = old + __popc(same);
  __syncwarp();
  return old + __popc(below);
}

__global__ void __launch_bounds__(kClusterThreads, 1) embed_sort(const __grid_constant__ ClusterSortParams p) {
  begin_after_previous();
  if (static_cast<int>(blockIdx.x) >= p.cluster) {
    fill_zeros(p.fill, blockIdx.x - p.cluster, gridDim.x - p.cluster);
    return;
  }
  extern __shared__ uint32_t sort_shared[];
  const int each = p.rounds * kClusterThreads, bins = 1 << p.digit;
  uint2* items = reinterpret_cast<uint2*>(sort_shared);  // key, row
  uint32_t* counts = sort_shared + 2 * each;             // [warp][bin]
  uint32_t *totals = counts + kClusterWarps * bins, *base = totals + bins;
  __shared__ uint32_t warp_sums[kClusterWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, rank = static_cast<int>(blockIdx.x);
  const int digit_of = threadIdx.x;
  const bool has_digit = digit_of < bins;
  if (rank == 0 && threadIdx.x < 2) p.active[threadIdx.x] = 0;
  const int mine = warp * 32 * p.rounds + lane;  // of the block's rows: mine, mine + 32, ...
  const int left = p.n - rank * each;
  uint32_t key[kMaxRounds], row[kMaxRounds];
#pragma unroll
  for (int k = 0; k < kMaxRounds; ++k) {
    if (k >= p.rounds) break;
    const int i = mine + 32 * k;
    row[k] = rank * each + i;
    key[k] = i < left ? key_of(index_at(p.tokens, p.index_bits, row[k]), p.vocab) : 0;
  }
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.digit;
    for (int b = threadIdx.x; b < kClusterWarps * bins / 4; b += kClusterThreads)
      reinterpret_cast<uint4*>(counts)[b] = make_uint4(0, 0, 0, 0);
    uint32_t at[kMaxRounds];  // first the lanes of the same digit, then the row's place among its warp's
#pragma unroll
    for (int k = 0; k < kMaxRounds; ++k) {
      if (k >= p.rounds) break;
      at[k] = same_bin(key[k] >> shift & (bins - 1), p.digit, mine + 32 * k < left);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMaxRounds; ++k) {
      if (k >= p.rounds) break;
      at[k] = rank_in_warp(counts + warp * bins, key[k] >> shift & (bins - 1), at[k], mine + 32 * k < left, lane);
    }
    __syncthreads();
    // thread b: digit b. Running sums over the warps; its count in all blocks, and in those before this one.
    uint32_t all = 0, before = 0;
    if (has_digit) {
#pragma unroll 8
      for (int w = 0; w < kClusterWarps; ++w) {
        const uint32_t c = counts[w * bins + digit_of];
        counts[w * bins + digit_of] = all;
        all += c;
      }
      totals[digit_of] = all;
    }
    if (p.cluster > 1) {
      tc::cluster_sync();
      if (has_digit) {
        uint32_t of[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          of[r] = r < p.cluster ? remote_load(tc::in_block(tc::smem_addr(&totals[digit_of]), r)) : 0;
        all = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          before += r < rank ? of[r] : 0;
          all += of[r];
        }
      }
    }
    uint32_t run = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += u;
    }
    if (lane == 31) warp_sums[warp] = run;
    __syncthreads();
    // by whole warps: there may be fewer digits than lanes
    const uint32_t lower = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0);
    if (has_digit) base[digit_of] = before + run - all + lower;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMaxRounds; ++k) {
      if (k >= p.rounds) break;
      if (mine + 32 * k >= left) continue;
      const uint32_t bin = key[k] >> shift & (bins - 1);
      const uint32_t to = base[bin] + counts[warp * bins + bin] + at[k];
      if (p.cluster > 1) {
        const uint32_t block = to / each, slot = to - block * each;
        remote_store(tc::in_block(tc::smem_addr(&items[slot]), block), key[k], row[k]);
      } else {
        items[to] = make_uint2(key[k], row[k]);
      }
    }
    if (p.cluster > 1)
      tc::cluster_sync();
    else
      __syncthreads();
#pragma unroll
    for (int k = 0; k < kMaxRounds; ++k) {
      if (k >= p.rounds) break;
      key[k] = items[mine + 32 * k].x;
      row[k] = items[mine + 32 * k].y;
    }
  }
#pragma unroll
  for (int k = 0; k < kMaxRounds; ++k) {
    if (k >= p.rounds) break;
    const int i = mine + 32 * k;
    if (i >= left) continue;
    p.keys[rank * each + i] = key[k];
    p.rows[rank * each + i] = row[k];
  }
}

__global__ void __launch_bounds__(kClusterThreads) embed_fill(const __grid_constant__ FillParams p) {
  begin_after_previous();
  fill_zeros(p, blockIdx.x, gridDim.x);
}

// More rows: three launches a pass, counts of the blocks' digits in memory (the whole gradient with 64 columns, in
// this form and on a cluster: 36000 rows 44 and 37 us, 65536 53 and 53, 131072 75 and 92). Bound by the launches' chain
// and the one block that adds up the counts: 131072 rows have 3.6 us of bytes.
constexpr int kSortThreads = 256, kSortItems = 8, kSortBlock = kSortThreads * kSortItems;

struct SortParams {
  const void* tokens;      // first pass: the caller's, else null
  int32_t index_bits;
  int64_t vocab;
  const uint32_t *keys_in, *rows_in;
  uint32_t *keys_out, *rows_out;
  uint32_t* counts;        // [bin][block], then their running sums
  uint32_t* active;        // as above
  int32_t n, blocks, shift, bins;
};

__device__ __forceinline__ uint32_t sort_key(const SortParams& p, int i) {
  if (!p.tokens) return p.keys_in[i];
  return key_of(index_at(p.tokens, p.index_bits, i), p.vocab);
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
  if (threadIdx.x < 2) p.active[threadIdx.x] = 0;
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
    const uint32_t bin = key[k] >> p.shift & (p.bins - 1);
    rank[k] = rank_in_warp(next[warp], bin, same_bin(bin, 31 - __clz(p.bins), i < p.n), i < p.n, lane);
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

// Rows of a chunk: few follow one another, and few runs cross chunks (with 32: 8192 x 768 22.6 us against 19.1, 333 x
// 769 15.2 against 11.6, 4000 x 4096 22.8 against 24.7, 16384 x 4096 83.3 against 82.6).
constexpr int kChunk = 16;
constexpr int kSumThreads = 128;
constexpr int kSumBatch = 8;  // rows of a thread in flight

struct SumParams {
  const uint32_t *keys, *rows;  // sorted
  int32_t n, chunks;
  int32_t tiles, join_tiles;    // parts of the columns, in the two kernels
  int32_t join_lanes;           // threads that the columns of a part take (a power of two, 32 at most)
  int64_t vocab, cols;
  const void* dout;
  int64_t dout_stride;
  void* dtable;
  int64_t dtable_stride;
  float* parts;                 // [2 chunk + (0: the run that came in, 1: the run that goes on)][part_stride]
  int64_t part_stride;
  // Runs that go on behind their first chunk, as (chunk, token): counts of the short and the long ones, then the
  // short ones from the front, the long ones (more than kShortRun chunks behind the first) from the end.
  uint32_t* active;
  int64_t zero_row_bytes;       // of the table's rows; 0: the table needs no more zeros
  int32_t zero_blocks, sum_blocks;
  float scale;
  bool accumulate;
};

template <typename TTable, int kVec>
__device__ __forceinline__ TTable* table_at(const SumParams& p, uint32_t token, int64_t col) {
  return static_cast<TTable*>(p.dtable) + token * p.dtable_stride + col;
}

constexpr int kShortRun = 16;
constexpr int kZeroRows = 8;  // rows of the table for each block that writes zeros

// Zeros to the rows of its part that no token names, a warp for each row: whether the row is among the sorted
// keys is found in steps of 32 lanes (16384 keys: 3).
__device__ __forceinline__ void zero_unnamed(const SumParams& p, uint32_t part) {
  const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
  const int64_t end = min(static_cast<int64_t>(part + 1) * kZeroRows, p.vocab);
  for (int64_t v = static_cast<int64_t>(part) * kZeroRows + threadIdx.x / 32; v < end; v += warps) {
    int lo = 0, left = p.n;  // the first key that is not below v lies in [lo, lo + left]
    while (left > 0) {
      const int step = (left + 31) / 32;
      const bool below = lane * step < left && p.keys[lo + lane * step] < v;
      const int count = __popc(__ballot_sync(0xffffffffu, below));
      if (count == 0) break;
      left = min(count * step, left) - (count - 1) * step - 1;
      lo += (count - 1) * step + 1;
    }
    if (lo < p.n && p.keys[lo] == v) continue;
    fill_row(static_cast<unsigned char*>(p.dtable) + v * p.dtable_stride * (p.zero_row_bytes / p.cols), p.zero_row_bytes, lane, 32);
  }
}

// kQ pieces of kVec columns for each thread. Bound by reading dout (HBM); kSumBatch rows, and the table's rows
// that are added to, are on their way together. kVec 1 where dout or dtable lies off 16 bytes (16384 x 4096, 32000 rows, the
// whole gradient of evenly drawn tokens: written 114 us, 80 by vectors; added 159 us, 74 by vectors; 8192 x 768, 50257
// added 34 us, 18 by vectors).
template <typename T, typename TTable, int kVec, int kQ, bool kAccumulate>
__global__ void __launch_bounds__(kSumThreads) embed_sum(const __grid_constant__ SumParams p) {
  begin_after_previous();
  __shared__ uint32_t keys[kChunk + 2], rows[kChunk];  // keys[0]: of the row before the chunk; the last: behind it
  int block = blockIdx.x;
  if (!kAccumulate && p.zero_blocks) {  // blocks that write zeros, spread evenly between the others
    const uint32_t all = p.zero_blocks + p.sum_blocks;
    const uint32_t zeros = static_cast<uint32_t>(static_cast<uint64_t>(block) * p.zero_blocks / all);
    const uint32_t next = static_cast<uint32_t>(static_cast<uint64_t>(block + 1) * p.zero_blocks / all);
    if (next != zeros) {
      zero_unnamed(p, zeros);
      return;
    }
    block -= zeros;
  }
  const int chunk = block / p.tiles, tile = block - chunk * p.tiles;
  const int first = chunk * kChunk;
  const uint32_t none = static_cast<uint32_t>(p.vocab);
  bool token = false;
  const int i = threadIdx.x;
  if (i < kChunk + 2) {
    const int at = first + i - 1;
    const bool there = at >= 0 && at < p.n, inside = i >= 1 && i <= kChunk;
    const uint32_t key = there ? p.keys[at] : none, row = there && inside ? p.rows[at] : 0;
    keys[i] = key;
    token = inside && key != none;
    if (inside) rows[i - 1] = row;
  }
  const int count = __syncthreads_count(token);  // rows with a token come first
  if (count == 0) return;
  const bool came = first > 0 && keys[0] == keys[1];                              // the first run began before
  const bool goes = count == kChunk && keys[kChunk + 1] == keys[kChunk];       // the last one goes on
  if (tile == 0 && i == 0 && goes && !(came && keys[1] == keys[kChunk])) {
    const int64_t far = first + static_cast<int64_t>(kShortRun + 1) * kChunk;
    const bool is_long = far < p.n && p.keys[far] == keys[kChunk];
    const uint32_t index = atomicAdd(&p.active[is_long], 1u);
    uint32_t* to = p.active + 2 + 2 * static_cast<int64_t>(is_long ? p.chunks - 1 - index : index);
    to[0] = chunk;
    to[1] = keys[kChunk];
  }
  const int64_t col0 = (static_cast<int64_t>(tile) * kQ * blockDim.x + i) * kVec, step = blockDim.x * kVec;
  const T* dout = static_cast<const T*>(p.dout) + col0;
  float sum[kQ][kVec] = {};
  bool begun = came;  // whether the present run has rows before the chunk
  for (int i0 = 0; i0 < count; i0 += kSumBatch) {
    Piece<T, kVec> v[kSumBatch][kQ];
    Piece<TTable, kVec> old[kAccumulate ? kSumBatch : 1][kQ];
#pragma unroll
    for (int k = 0; k < kSumBatch; ++k) {
      if (i0 + k >= count) break;
      const T* from = dout + rows[i0 + k] * p.dout_stride;
#pragma unroll
      for (int q = 0; q < kQ; ++q)
        if (col0 + q * step < p.cols) v[k][q] = *reinterpret_cast<const Piece<T, kVec>*>(from + q * step);
      if constexpr (kAccumulate) {
        const uint32_t key = keys[i0 + k + 1];
        if (key == keys[i0 + k + 2]) continue;  // the run's last row brings the table's
#pragma unroll
        for (int q = 0; q < kQ; ++q)
          if (col0 + q * step < p.cols)
            old[k][q] = *reinterpret_cast<const Piece<TTable, kVec>*>(table_at<TTable, kVec>(p, key, col0 + q * step));
      }
    }
#pragma unroll
    for (int k = 0; k < kSumBatch; ++k) {
      const int r = i0 + k;
      if (r >= count) break;
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        float x[kVec];
        v[k][q].to(x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum[q][e] += x[e];
      }
      const bool last = r + 1 == count, on = last && goes;
      if (!last && keys[r + 2] == keys[r + 1]) continue;
      const bool part = begun || on;
      float* to = p.parts + (2 * static_cast<int64_t>(chunk) + (begun ? 0 : 1)) * p.part_stride;
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const int64_t col = col0 + q * step;
        if (col < p.cols) {
          if (part) {
            store<kVec>(to + col, sum[q]);
          } else {
            float x[kVec] = {};
            if constexpr (kAccumulate) old[k][q].to(x);
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] += sum[q][e] * p.scale;
            store<kVec>(table_at<TTable, kVec>(p, keys[r + 1], col), x);
          }
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum[q][e] = 0.0f;
      }
      begun = false;
    }
  }
}

// Adds up the runs that cross chunks. Short ones by a warp for each 32 kVec columns, chunk after chunk; long ones
// by a block: groups of as many threads as the columns take, up to 32, each a share of the chunks, then the groups
// pair by pair.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

template <typename TTable, int kVec>
__device__ __forceinline__ void add_to_table(const SumParams& p, uint32_t token, int64_t col, const float (&sum)[kVec]) {
  TTable* to = table_at<TTable, kVec>(p, token, col);
  float x[kVec] = {};
  if (p.accumulate) load<kVec>(to, x);
#pragma unroll
  for (int e = 0; e < kVec; ++e) x[e] += sum[e] * p.scale;
  store<kVec>(to, x);
}

// Adds the parts that chunks [from, to) hold of the run that came in.
template <int kVec>
__device__ __forceinline__ void add_parts(const SumParams& p, int from, int to, int64_t col, float (&sum)[kVec]) {
#pragma unroll 4
  for (int c = from; c < to; ++c) {
    float v[kVec];
    load<kVec>(p.parts + 2 * static_cast<int64_t>(c) * p.part_stride + col, v);
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum[e] += v[e];
  }
}

template <typename TTable, int kVec>
__global__ void __launch_bounds__(kJoinThreads) embed_join(const __grid_constant__ SumParams p) {
  begin_after_previous();
  const int64_t shorts = static_cast<int64_t>(p.active[0]) * p.join_tiles, longs = static_cast<int64_t>(p.active[1]) * p.join_tiles;
  const int lane = threadIdx.x % 32;
  __shared__ float sums[kVec][kJoinThreads];
  int64_t turn = blockIdx.x;  // the long items, then eight short ones at a time
  const int lanes = p.join_lanes, groups = kJoinThreads / lanes, in_group = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes;
  for (; turn < longs; turn += gridDim.x) {
    const int64_t item = turn, index = item / p.join_tiles;
    const uint32_t* run = p.active + 2 + 2 * (p.chunks - 1 - index);
    const int chunk = static_cast<int>(run[0]);
    const uint32_t token = run[1];
    int parts = 0;  // chunks behind the first that begin with the run
    for (int c0 = chunk + 1;; c0 += kJoinThreads) {
      const int64_t at = (c0 + static_cast<int64_t>(threadIdx.x)) * kChunk;
      const int more = __syncthreads_count(at < p.n && p.keys[at] == token);
      parts += more;
      if (more < kJoinThreads) break;
    }
    const int each = (parts + groups - 1) / groups;
    const int64_t col = ((item - index * p.join_tiles) * 32 + in_group) * kVec;
    float sum[kVec] = {};
    if (col < p.cols) {
      if (group == 0) load<kVec>(p.parts + (2 * static_cast<int64_t>(chunk) + 1) * p.part_stride + col, sum);
      const int64_t from = min(static_cast<int64_t>(parts), static_cast<int64_t>(group) * each);
      const int64_t to = min(static_cast<int64_t>(parts), from + each);
      add_parts<kVec>(p, chunk + 1 + static_cast<int>(from), chunk + 1 + static_cast<int>(to), col, sum);
    }
    for (int half = groups / 2; half > 0; half /= 2) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) sums[e][threadIdx.x] = sum[e];
      __syncthreads();
      if (group < half)
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum[e] += sums[e][threadIdx.x + half * lanes];
      __syncthreads();
    }
    if (group == 0 && col < p.cols) add_to_table<TTable, kVec>(p, token, col, sum);
  }
  for (;; turn += gridDim.x) {
    const int64_t item = (turn - longs) * kJoinWarps + threadIdx.x / 32;
    if (item >= shorts) return;
    const int64_t index = item / p.join_tiles;
    const uint32_t* run = p.active + 2 + 2 * index;
    const int chunk = static_cast<int>(run[0]);
    const uint32_t token = run[1];
    const int64_t at = (chunk + 1 + static_cast<int64_t>(lane)) * kChunk;
    const int64_t col = ((item - index * p.join_tiles) * 32 + lane) * kVec;
    // on their way together: the keys that tell how far the run goes, its first two parts and the table's row
    const bool more = lane < kShortRun && at < p.n && p.keys[at] == token;
    float sum[kVec] = {}, next[kVec] = {}, old[kVec] = {};
    if (col < p.cols) {
      const float* from = p.parts + (2 * static_cast<int64_t>(chunk) + 1) * p.part_stride + col;
      load<kVec>(from, sum);
      load<kVec>(from + p.part_stride, next);
      if (p.accumulate) load<kVec>(table_at<TTable, kVec>(p, token, col), old);
    }
    const int parts = __popc(__ballot_sync(0xffffffffu, more));  // at least one
    if (col >= p.cols) continue;
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum[e] += next[e];
    add_parts<kVec>(p, chunk + 2, chunk + 1 + parts, col, sum);
#pragma unroll
    for (int e = 0; e < kVec; ++e) old[e] += sum[e] * p.scale;
    store<kVec>(table_at<TTable, kVec>(p, token, col), old);
  }
}

// ---------------------------------------------------------------------- host

constexpr int64_t kMaxCols = int64_t(1) << 30, kMaxVocab = int64_t(1) << 30, kMaxRows = int64_t(1) << 30;

int64_t round_to(int64_t n, int64_t k) { return (n + k - 1) / k * k; }

bool vector_rows(const void* p, int64_t rows, int64_t stride, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows < 2 || stride * size % 16 == 0);
}

struct Workspace {
  int64_t keys[2], rows[2], counts, active, parts, bytes;
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
  const bool many = rows > kClusterRows;
  for (int k = 0; k < (many ? 2 : 1); ++k) {
    w.keys[k] = take(rows * 4);
    w.rows[k] = take(rows * 4);
  }
  if (many) w.counts = take(static_cast<int64_t>(w.blocks) * kMaxBins * 4);
  w.active = take((static_cast<int64_t>(w.chunks) + 1) * 8);
  w.parts = take(2 * static_cast<int64_t>(w.chunks) * w.part_stride * 4);
  w.bytes = at;
  return w;
}

template <typename T, typename TTable, int kVec>
int run_sum(SumParams p, int sms, cudaStream_t st) {
  constexpr int kQ = kVec == 8 ? 1 : kVec == 4 ? 2 : 4;
  const int64_t groups = (p.cols + kVec - 1) / kVec;
  const int threads = static_cast<int>(std::max<int64_t>(64, std::min<int64_t>(kSumThreads, round_to((groups + kQ - 1) / kQ, 32))));
  const int64_t tiles = (groups + threads * kQ - 1) / (threads * kQ), join_tiles = (groups + 31) / 32;
  if (tiles * p.chunks > INT32_MAX || join_tiles > INT32_MAX) return FSDP_EINVAL;  // more than any memory holds
  p.tiles = static_cast<int32_t>(tiles);
  p.join_tiles = static_cast<int32_t>(join_tiles);
  p.join_lanes = 1;
  while (p.join_lanes < 32 && p.join_lanes < groups) p.join_lanes *= 2;
  p.sum_blocks = p.chunks * p.tiles;
  p.zero_blocks = p.zero_row_bytes ? static_cast<int32_t>((p.vocab + kZeroRows - 1) / kZeroRows) : 0;
  if (static_cast<int64_t>(p.sum_blocks) + p.zero_blocks > INT32_MAX) return FSDP_EINVAL;
  const auto kernel = p.accumulate ? embed_sum<T, TTable, kVec, kQ, true> : embed_sum<T, TTable, kVec, kQ, false>;
  if (int rc = launch_after(kernel, p.sum_blocks + p.zero_blocks, 1, threads, 0, st, p)) return rc;
  if (p.chunks == 1) return FSDP_OK;  // no run crosses chunks
  const int64_t items = p.chunks * join_tiles;  // at most
  return launch_after(embed_join<TTable, kVec>, static_cast<int>(std::min<int64_t>(items, 6 * sms)), 1, kJoinThreads, 0, st, p);
}

template <typename T, typename TTable>
int run_sum_as(const SumParams& p, bool vectors, int sms, cudaStream_t st) {
  // vectors of 16 bytes of the wider type
  constexpr int kVec = sizeof(T) == 2 && sizeof(TTable) == 2 ? 8 : 4;
  return vectors ? run_sum<T, TTable, kVec>(p, sms, st) : run_sum<T, TTable, 1>(p, sms, st);
}

// Blocks that fill beside a sort: a vector for each thread, at most `most`.
int fill_blocks(const FillParams& f, int most) {
  return static_cast<int>(std::min<int64_t>((f.rows * f.row_bytes + 16383) / 16384, most));
}

int run_rank(RankParams p, int sms, cudaStream_t st) {
  p.tiles = (p.n + kRankTile - 1) / kRankTile;
  return launch_after(embed_rank, p.tiles + fill_blocks(p.fill, sms), 1, kRankThreads, (p.n + 3) / 4 * 16, st, p);
}

// The sort of up to kClusterRows rows; the other blocks fill. Two steps of 32 rows for each warp, then more blocks,
// then more steps.
int run_cluster_sort(ClusterSortParams p, int sms, cudaStream_t st) {
  p.cluster = 1;
  while (p.cluster < kMaxCluster && p.n > p.cluster * 2 * kClusterThreads) p.cluster *= 2;
  p.rounds = (p.n + p.cluster * kClusterThreads - 1) / (p.cluster * kClusterThreads);
  const int bins = 1 << p.digit;
  const int smem = (2 * p.rounds * kClusterThreads + (kClusterWarps + 2) * bins) * 4;
  constexpr int kMost = (2 * kMaxRounds * kClusterThreads + (kClusterWarps + 2) * kMaxBins) * 4;
  if (cudaFuncSetAttribute(embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess) return FSDP_ECUDA;
  const int grid = p.cluster + static_cast<int>(round_to(fill_blocks(p.fill, (sms / p.cluster - 1) * p.cluster), p.cluster));
  return launch_after(embed_sort, grid, p.cluster, kClusterThreads, smem, st, p);
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
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const auto go = [&](auto kernel, int vec, int groups, int per_sm) {  // per_sm: blocks that run at once
    const int64_t unit = 32 * groups * vec, units = a->rows * ((a->cols + unit - 1) / unit);
    const int grid = static_cast<int>(std::min<int64_t>((units + kLookupWarps - 1) / kLookupWarps, 152 * per_sm));
    return launch_after(kernel, grid, 1, 32 * kLookupWarps, 0, cs, p);
  };
  const auto filled = [&](int64_t unit) {  // whether nine tenths of the units' elements are in the rows
    return vectors && 10 * a->cols >= 9 * ((a->cols + unit - 1) / unit * unit);
  };
  if (a->dtype == FSDP_DTYPE_F32) {
    if (addend) return vectors ? go(embed_rows<float, 4, true, false>, 4, 4, 4) : go(embed_rows<float, 1, true, false>, 1, 8, 4);
    if (filled(512)) return go(embed_rows<float, 4, false, true>, 4, 4, 3);
    return vectors ? go(embed_rows<float, 4, false, false>, 4, 4, 5) : go(embed_rows<float, 1, false, false>, 1, 8, 5);
  }
  if (addend)
    return vectors ? go(embed_rows<__nv_bfloat16, 8, true, false>, 8, 4, 3) : go(embed_rows<__nv_bfloat16, 1, true, false>, 1, 8, 4);
  if (filled(1024)) return go(embed_rows<__nv_bfloat16, 8, false, true>, 8, 4, 3);
  return vectors ? go(embed_rows<__nv_bfloat16, 8, false, false>, 8, 4, 5) : go(embed_rows<__nv_bfloat16, 1, false, false>, 1, 8, 5);
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
  FillParams fill{static_cast<unsigned char*>(dtable), a->vocab, a->accumulate ? 0 : a->cols * ts, sw.pitch()};
  if (fill.rows > 1 && fill.pitch == fill.row_bytes) fill.row_bytes *= fill.rows, fill.rows = 1;  // one long row
  Device dev;
  if (int rc = device_facts(&dev)) return rc;
  // A table beyond what is filled during a sort (about 8 us) leaves its zeros to the blocks between the sums' (see
  // the top): 16384 x 4096, 32000 rows 104 -> 84 us. Not narrow rows, which take a warp each there.
  const bool sorted_at_once = a->rows <= kClusterRows;
  const bool later = fill.row_bytes && a->rows > 0 && a->cols * ts >= 256 &&
                     (!sorted_at_once || a->vocab * a->cols * ts > (int64_t(32) << 20));
  if (later) fill.row_bytes = 0;
  if (fill.row_bytes && (a->rows == 0 || !sorted_at_once)) {
    if (int rc = launch_after(embed_fill, 2 * dev.sms, 1, kClusterThreads, 0, cs, fill)) return rc;
  }
  if (a->rows == 0) return FSDP_OK;

  const Workspace w = carve(a->rows, a->cols);
  auto* base = reinterpret_cast<unsigned char*>(round_to(reinterpret_cast<intptr_t>(workspace), 256) - 256);
  uint32_t *keys[2], *rows[2], *active = reinterpret_cast<uint32_t*>(base + w.active);
  for (int k = 0; k < 2; ++k) {
    keys[k] = reinterpret_cast<uint32_t*>(base + w.keys[k]);
    rows[k] = reinterpret_cast<uint32_t*>(base + w.rows[k]);
  }
  int bits = 1;
  while (a->vocab >> bits) ++bits;  // of the keys 0 .. vocab
  const int passes = (bits + 8) / 9, digit = (bits + passes - 1) / passes;
  const int32_t n = static_cast<int32_t>(a->rows);
  int now = 0;
  if (a->rows <= kRankRows && a->vocab <= kRankVocab) {
    if (int rc = run_rank(RankParams{tokens, keys[0], rows[0], active, a->vocab, 8 * is, n, 0, fill}, dev.sms, cs)) return rc;
  } else if (sorted_at_once) {
    const ClusterSortParams p{tokens, keys[0], rows[0], active, a->vocab, 8 * is, n, 0, 0, passes, digit, fill};
    if (int rc = run_cluster_sort(p, dev.sms, cs)) return rc;
  } else {
    for (int k = 0; k < passes; ++k, now ^= 1) {
      const SortParams p{k == 0 ? tokens : nullptr, 8 * is, a->vocab, keys[now], rows[now], keys[now ^ 1], rows[now ^ 1],
                         reinterpret_cast<uint32_t*>(base + w.counts), active, n, w.blocks, k * digit, 1 << digit};
      if (int rc = launch_after(sort_count, w.blocks, 1, kSortThreads, 0, cs, p)) return rc;
      if (int rc = launch_after(sort_offsets, 1, 1, 1024, 0, cs, p)) return rc;
      if (int rc = launch_after(sort_move, w.blocks, 1, kSortThreads, 0, cs, p)) return rc;
    }
  }
  const SumParams p{keys[now], rows[now], n, w.chunks, 0, 0, 0, a->vocab, a->cols, dout, a->dout_stride, dtable,
                    a->dtable_stride, reinterpret_cast<float*>(base + w.parts), w.part_stride, active,
                    later ? a->cols * ts : 0, 0, 0, static_cast<float>(a->scale), a->accumulate != 0};
  const bool vectors = a->cols % 8 == 0 && vector_rows(dout, a->rows, a->dout_stride, es) &&
                       vector_rows(dtable, a->vocab, a->dtable_stride, ts);
  const bool in32 = a->dtype == FSDP_DTYPE_F32, table32 = a->table_dtype == FSDP_DTYPE_F32;
  const int sms = dev.sms;
  return in32 ? table32 ? run_sum_as<float, float>(p, vectors, sms, cs) : run_sum_as<float, __nv_bfloat16>(p, vectors, sms, cs)
         : table32 ? run_sum_as<__nv_bfloat16, float>(p, vectors, sms, cs)
                   : run_sum_as<__nv_bfloat16, __nv_bfloat16>(p, vectors, sms, cs);
}
