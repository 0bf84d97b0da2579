// Newton-Schulz orthogonalisation (fsdp_newton_schulz; also the update of
// fsdp_muon_step).
//
// X_0 = G / (|G|_F + eps); per step, with the Gram matrix on the short side,
//   A = X X^T,  P = b A + c A^2,  X <- a X + P X
// (X^T X and X P for a matrix with more rows than columns: no transposes, the
// tensor cores take operands whose long index is the contiguous one).
//
// Representation. The products run on fp16 operands with fp32 accumulation, at
// the rate of bf16 and with 11 instead of 8 bits; powers of two keep the values in
// fp16's range: X is held times 2^12, A and P times 2^10 (X's singular values
// stay below 7 and P's below 30, which ns_plan() checks). X itself is held as two
// fp16 parts, hi + lo, 22 bits: only the products see it rounded. A rounding of X
// would put noise into the directions that X lacks, and each step multiplies
// those by a = 3.4 (measured on matrices of low rank: 3 % of the result's
// norm, 0.06 % with the two parts); the operands' rounding stays inside X's row or
// column space. With terms = 3 every operand has both parts: hi hi + lo hi + hi lo.
//
// Late steps round less still. Once the mean squared singular value m = |X|^2 / side
// is large (1/4 or more: most of the space is filled, nothing is left to keep clean)
// A is close to m I, and what is rounded is only the rest, A' = A - m I:
//   b A + c A^2 = d I + P',  d = b m + c m^2,  P' = (b + 2 c m) A' + c A'^2,
//   X <- (a + d) X + P' X.
// P' is several times smaller than P, and so is the part of X' that comes from rounded
// operands (error of a 768 x 2304 matrix 1.5e-3 -> 0.5e-3 of its norm).
//
// Long Gram products are cut into segments. The tensor cores' sums are cut off, not
// rounded, at each addition, so a sum's error grows with the number of steps (measured:
// 7e-9 of the result per element of the long side; 12 % at 16.8 M). Where a
// product has more than 256 steps of 64, or few tiles and many steps, blocks take segments of
// it, and a pass adds the segments' fp32 results in order (1 x 16.8 M: 6e-5, and 757 -> 26 ms;
// 300 x 262144: 6e-5, 5.7 -> 1.6 ms; 50257 x 768 0.8 ms).
//
// Each of the three products is one launch over all matrices of the call: a
// persistent grid of tiles; in each block a producer lane (TMA), a product lane
// (tcgen05, two accumulators in tensor memory), a lane that fetches what the result
// is added to, and eight epilogue warps. Results leave through shared memory, 64
// columns at a time, as tiled stores. A and P are symmetric: tiles above the
// diagonal are not computed, and the others are written to both places.
#include "host_internal.h"
#include "newton_schulz.h"
#include "strided.h"
#include "tensor_core.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <type_traits>
#include <vector>

namespace fsdp {
namespace {

using namespace tc;

constexpr float kScaleX = 4096.0f, kScaleA = 1024.0f;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr int kMaxMats = 32;                      // matrices of one launch (24 KB of parameters)

// ------------------------------------------------- norm and first operands

// Warps take units of up to 1024 consecutive elements (of a row), each lane four
// times 8 elements: 128 bytes of fp32 in flight per lane.
constexpr int kUnit = 1024;
constexpr int kPassWarps = 8;
constexpr int kMaxParts = 608;

struct PassMat {
  const void* source;
  int64_t stride, rows, cols;
  __half *hi, *lo;
  int64_t ld;
  float* partial;
  int64_t flat;       // the first element's place in the unit (momentum)
  int32_t dtype;
  int32_t parts;      // blocks (and partial sums) of this matrix
  int32_t block_end;  // running total of parts
};

struct PassParams {
  PassMat mat[kMaxMats];
  int32_t count;
  float eps;
};

struct MomentumParams {
  PassParams pass;
  NsMomentum m;
};

__device__ __forceinline__ const PassMat& pass_mat(const PassParams& p, int* part) {
  int i = 0, first = 0;
  while (static_cast<int>(blockIdx.x) >= p.mat[i].block_end) first = p.mat[i++].block_end;
  *part = blockIdx.x - first;
  return p.mat[i];
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The block's sum, at `out` after the caller's next barrier.
__device__ __forceinline__ void block_sum_to(float sum, float* out) {
  __shared__ float shared[kPassWarps];
  sum = warp_sum(sum);
  if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < kPassWarps; ++i) sum += shared[i];
  *out = sum;
}

__device__ __forceinline__ void unpack_bf16(uint32_t two, float* v) {
  v[0] = __uint_as_float(two << 16);
  v[1] = __uint_as_float(two & 0xffff0000u);
}

// 8 elements from element i of the source, zeros from `count` on.
__device__ __forceinline__ void load8(const PassMat& j, int64_t i, int count, float (&v)[8]) {
  if (j.dtype == FSDP_DTYPE_F32) {
    const float* q = static_cast<const float*>(j.source) + i;
    if (count >= 8 && (reinterpret_cast<uintptr_t>(q) & 15u) == 0) {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(q)), b = __ldcs(reinterpret_cast<const float4*>(q) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < count ? q[e] : 0.0f;
    return;
  }
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(j.source) + i;
  if (count >= 8 && (reinterpret_cast<uintptr_t>(q) & 15u) == 0) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(q));
    unpack_bf16(a.x, v), unpack_bf16(a.y, v + 2), unpack_bf16(a.z, v + 4), unpack_bf16(a.w, v + 6);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < count ? __bfloat162float(q[e]) : 0.0f;
}

// Calls f(row, column, values) for this lane's groups of 8 elements of its block's
// units (column beyond the row's end: not called; values beyond it: zero).
template <typename F>
__device__ __forceinline__ void each_group(const PassMat& j, int part, F f) {
  const int64_t segs = (j.cols + kUnit - 1) / kUnit, units = j.rows * segs;
  const int lane = threadIdx.x % 32;
  for (int64_t u = static_cast<int64_t>(part) * kPassWarps + threadIdx.x / 32; u < units;
       u += static_cast<int64_t>(j.parts) * kPassWarps) {
    const int64_t r = units >> 31 ? u / segs : static_cast<uint32_t>(u) / static_cast<uint32_t>(segs);
    const int64_t c0 = (u - r * segs) * kUnit + lane * 8;
    float v[4][8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t c = c0 + q * 256;
      if (c < j.cols) load8(j, r * j.stride + c, static_cast<int>(min(j.cols - c, int64_t(8))), v[q]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c0 + q * 256 < j.cols) f(r, c0 + q * 256, v[q]);
  }
}

// Sums of squares, one per block (4096 x 11008 fp32: 30 us, 6.0 TB/s): a lane adds its groups of 8, then trees. fp32
// throughout (fp64 runs at 1/64 of the rate): a lane has up to four groups of each unit of its warp, one after another,
// rows x ceil(cols / 1024) units over 608 x 8 warps. That is 40 terms in sequence for 4096 x 11008, 860 for
// 32768 x 32768 (|G|^2 off by 5e-5 of itself at most), 3400 for a column of 2^24.
__global__ void __launch_bounds__(32 * kPassWarps) ns_squares(const __grid_constant__ PassParams p) {
  int part;
  const PassMat j = pass_mat(p, &part);  // read ahead of the wait, as in ns_product
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float sum = 0.0f;
  each_group(j, part, [&](int64_t, int64_t, const float (&v)[8]) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += v[e] * v[e];
    sum += s;
  });
  block_sum_to(sum, &j.partial[part]);
}

__device__ __forceinline__ float mean_of(float sum, const NsMomentum& m) {
  return m.inv_w != 0.0f ? sum * m.inv_w : sum / static_cast<float>(m.w);
}

// The momentum update of a unit's matrices (W = kWorld ranks; 0: any), and the sums
// of squares of u. Bound by HBM: 2 W + 12 bytes an element (a Llama block's seven matrices,
// W = 8, 202 M elements: 0.82 ms, 6.9 TB/s).
template <int kWorld>
__global__ void __launch_bounds__(32 * kPassWarps) ns_momentum(const __grid_constant__ MomentumParams p) {
  int part;
  const PassMat j = pass_mat(p.pass, &part);
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const NsMomentum& m = p.m;
  const int world = kWorld ? kWorld : m.w;
  float* out = static_cast<float*>(const_cast<void*>(j.source));
  const int64_t begin = j.flat, end = j.flat + j.rows * j.cols;
  const int64_t units = (end - (begin & ~int64_t(7)) + 255) / 256;  // of 256 elements: 8 per lane
  uintptr_t bits = 0;
  for (int k = 0; k < world; ++k) bits |= reinterpret_cast<uintptr_t>(m.grads[k]);
  float sum = 0.0f;
  for (int64_t u = static_cast<int64_t>(part) * kPassWarps + threadIdx.x / 32; u < units;
       u += static_cast<int64_t>(j.parts) * kPassWarps) {
    const int64_t f = (begin & ~int64_t(7)) + u * 256 + threadIdx.x % 32 * 8;
    if (f >= end) continue;
    const int64_t rank = f / m.shard, at = f - rank * m.shard;
    float* mom = m.momentum[rank] + at;
    float* to = out + (f - begin);
    float s = 0.0f;
    if (f >= begin && f + 8 <= end && at + 8 <= m.shard &&
        ((bits | reinterpret_cast<uintptr_t>(mom) | reinterpret_cast<uintptr_t>(to)) & 15u) == 0) {
      float4 a = __ldcs(reinterpret_cast<const float4*>(mom)), b = __ldcs(reinterpret_cast<const float4*>(mom) + 1);
      float g[8] = {};
      constexpr int kBatch = kWorld ? (kWorld < 8 ? kWorld : 8) : 4;
      for (int k0 = 0; k0 < world; k0 += kBatch) {
        uint4 r[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (kWorld || k0 + k < world) r[k] = __ldcs(reinterpret_cast<const uint4*>(m.grads[k0 + k] + f));
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (!kWorld && k0 + k >= world) break;
          float w[8];
          unpack_bf16(r[k].x, w), unpack_bf16(r[k].y, w + 2), unpack_bf16(r[k].z, w + 4), unpack_bf16(r[k].w, w + 6);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] += w[e];
        }
      }
      float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float mean = mean_of(g[e], m);
        v[e] = m.mu * v[e] + mean;
        w[e] = m.nesterov ? mean + m.mu * v[e] : v[e];
        s += w[e] * w[e];
      }
      __stcs(reinterpret_cast<float4*>(mom), make_float4(v[0], v[1], v[2], v[3]));
      __stcs(reinterpret_cast<float4*>(mom) + 1, make_float4(v[4], v[5], v[6], v[7]));
      reinterpret_cast<float4*>(to)[0] = make_float4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<float4*>(to)[1] = make_float4(w[4], w[5], w[6], w[7]);
    } else {
      for (int64_t q = max(f, begin); q < min(f + 8, end); ++q) {
        float g = 0.0f;
        for (int k = 0; k < world; ++k) g += __bfloat162float(__ushort_as_bfloat16(m.grads[k][q]));
        g = mean_of(g, m);
        float* mq = m.momentum[q / m.shard] + q % m.shard;
        const float v = m.mu * *mq + g;
        *mq = v;
        const float w = m.nesterov ? g + m.mu * v : v;
        out[q - begin] = w;
        s += w * w;
      }
    }
    sum += s;
  }
  block_sum_to(sum, &j.partial[part]);
}

// X_0 as two parts. Bound by HBM: 8 bytes an element (4096 x 11008 fp32: 55 us, 6.5 TB/s).
__global__ void __launch_bounds__(32 * kPassWarps) ns_normalise(const __grid_constant__ PassParams p) {
  int part;
  const PassMat j = pass_mat(p, &part);  // read ahead of the wait, as in ns_product
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float sum = 0.0f;
  for (int i = threadIdx.x % 32; i < j.parts; i += 32) sum += j.partial[i];
  const float inv = 1.0f / (sqrtf(warp_sum(sum)) + p.eps);
  each_group(j, part, [&](int64_t r, int64_t c, const float (&v)[8]) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // inv first: a tiny norm's reciprocal times 2^12 may not fit
      const float a = v[2 * e] * inv * kScaleX, b = v[2 * e + 1] * inv * kScaleX;
      const __half2 h = __floats2half2_rn(a, b);
      const float2 f = __half22float2(h);
      const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
      hi[e] = *reinterpret_cast<const uint32_t*>(&h);
      lo[e] = *reinterpret_cast<const uint32_t*>(&l);
    }
    *reinterpret_cast<uint4*>(j.hi + r * j.ld + c) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(j.lo + r * j.ld + c) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  });
}

// ----------------------------------------------------------------- products

enum Kind : int32_t { kGram, kPoly, kUpdate };             // A = X X^T; P = b A + c A A; X <- a X + P X
enum Result : int32_t { kParts, kOut, kApply };            // hi/lo parts; bf16 out; the master's update

// C[m, n] = alpha sum_k p[i, k] q[j, k] + beta in[i, j].
struct GemmMat {
  CUtensorMap p[2], q[2], result[2];  // boxes of 64 x 64 elements of the hi and lo parts
  int32_t m, n, k;
  int32_t col_tiles, tiles;
  uint8_t p_mn, q_mn;      // the operand's row index (of C's rows, columns) is the contiguous one
  uint8_t symmetric;
  uint8_t in_q;            // `in` is q (else p)
  const float* squares;    // sums of squares of X over 32 x 32 blocks (null: X_0, no shift)
  float* new_squares;      // those of the next X
  int32_t squares_count;
  int32_t splits, seg_blocks;  // a long Gram product's segments (0: it is whole) and their length in steps of 64
  float* partial;              // their results, each a square of `square_of(n)` rows
  __half* joined[2];           // where their sum goes: hi, lo (null: not kept)
  int64_t joined_ld;
  uint16_t* out;
  int64_t out_stride;
  int64_t flat;
  float step;
};

template <int kMats>
struct GemmParams {
  GemmMat mat[kMats];
  NsApply apply;
  int32_t count, tiles, terms;
  int32_t kind, result;
  float a, b, c;           // the step's coefficients
  unsigned int* status;
};
static_assert(sizeof(GemmParams<kMaxMats>) <= 32764, "kernel parameter block too large");

constexpr float kShiftFrom = 0.25f;  // mean squared singular value from which A is shifted

constexpr int kTileK = 64;
constexpr int kChunk = 64;          // columns of a tile that leave together
constexpr int kEpilogueWarps = 8;
constexpr int kGemmThreads = 128 + 32 * kEpilogueWarps;  // producer, products, fetch of `in`, an idle warp, epilogue
constexpr int kSlotBytes = 128 * kChunk * 2;              // one part of a chunk
constexpr int kSlots = 4;

// A tile: 128 rows per block of the pair (or single block) and kN columns.
template <int kN, int kPair>
struct Tile {
  static constexpr int kM = 128 * kPair;
  static constexpr int kBRows = kN / kPair;  // a block's half of the second operand
  static constexpr int kABytes = 128 * kTileK * 2, kBBytes = kBRows * kTileK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = (230400 - 1024 - kSlots * kSlotBytes) / kStageBytes;
  static constexpr int kSmemBytes = kStages * kStageBytes + kSlots * kSlotBytes + 1024;
  static constexpr int kTmemCols = 2 * kN;

  // symmetric results: tiles of tile row i with an element on or below the diagonal
  __host__ __device__ static int below(int i, int col_tiles) {
    const int c = ((i + 1) * kM + kN - 1) / kN;
    return c < col_tiles ? c : col_tiles;
  }
};

__host__ __device__ constexpr int square_of(int side) { return (side + 31) / 32 * 32; }

// Tile t of a launch: its matrix and place. Calls come with growing t.
template <typename T, typename P, bool kLong = false>
struct Tiles {
  const P& p;
  int mat = 0, first = 0, split = 0;
  int row = 0, base = 0;  // symmetric: the current row of tiles and its first tile

  __device__ __forceinline__ const GemmMat& at(int t, int* i, int* j) {
    while (t - first >= p.mat[mat].tiles) {
      first += p.mat[mat++].tiles;
      row = base = split = 0;
    }
    const GemmMat& g = p.mat[mat];
    int l = t - first;
    if constexpr (kLong) {  // one segment's tiles after another's
      const int each = g.tiles / g.splits, s = l / each;
      if (s != split) split = s, row = base = 0;
      l -= s * each;
    }
    if (!g.symmetric) {
      // along the short side first: the tiles at work share the long operand's rows or
      // columns and the whole of the short one, which stays in L2
      const int short_tiles = g.in_q ? g.tiles / g.col_tiles : g.col_tiles;
      const int a = l / short_tiles, b = l - a * short_tiles;
      *i = g.in_q ? b : a;
      *j = g.in_q ? a : b;
      return g;
    }
    while (l - base >= T::below(row, g.col_tiles)) base += T::below(row++, g.col_tiles);
    *i = row;
    *j = l - base;
    return g;
  }
};

// Byte of the 16-byte piece `piece` of row `row` in a slot (rows of 128 bytes, swizzled as TMA does).
__device__ __forceinline__ uint32_t slot_at(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }

__device__ __forceinline__ uint4 shared_load(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void shared_store(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Writes the thread's 32 fp16 values (columns 32 half .. of row `row`) into a slot.
__device__ __forceinline__ void put_part(uint32_t slot, int row, int half, const uint32_t (&r)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    shared_store(slot + slot_at(row, half * 4 + q), r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
}

// The same values as columns of the transposed chunk: two boxes of 64 x 64, box b
// with rows 64 b .. of the tile as its columns. Pairs of lanes exchange two columns at a
// time, so that a store holds two rows of one column; the even lanes' columns and
// the odd lanes' are 4 apart, which puts them in different banks.
__device__ __forceinline__ void put_mirror(uint32_t slot, int row, int half, const uint32_t (&r)[16]) {
  const bool odd = row & 1;
  const int pair = row & 63 & ~1;
  const uint32_t base = slot + (row >> 6) * 8192 + (pair & 7) * 2;
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // columns 2 (c + k), + 1 of the even lane; 4 more of the odd lane
      const uint32_t mine = odd ? r[c + 2 + k] : r[c + k];
      const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? r[c + k] : r[c + 2 + k], 1);
      const uint32_t first = odd ? __byte_perm(other, mine, 0x5410) : __byte_perm(mine, other, 0x5410);
      const uint32_t second = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x7632);
      const int col = half * 32 + 2 * (c + k) + (odd ? 4 : 0);
      const uint32_t a = base + col * 128 + (((pair >> 3) ^ (col & 7)) << 4);
      const uint32_t b = base + (col + 1) * 128 + (((pair >> 3) ^ ((col + 1) & 7)) << 4);
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(first) : "memory");
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(b), "r"(second) : "memory");
    }
  }
}

__device__ __forceinline__ float shared_load1(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// The last step's chunk, fp32 in the slots (the caller's barrier ordered the writes):
// written as bf16, or applied to the master, a row by a warp at a time (any
// alignment, whole lines per access), eight rows in flight.
__device__ __forceinline__ void finish_rows(const GemmMat& g, const NsApply& ap, int32_t result, uint32_t slots, int row0,
                                            int col0, int warp, int lane) {
  constexpr int kRows = 128 / kEpilogueWarps, kBatch = 8;
  const int first = row0 + warp * kRows, rows = min(kRows, g.m - first);
  const int n = g.n;
  const bool there[2] = {col0 + lane < n, col0 + 32 + lane < n};
  uint32_t from[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) from[h] = slots + (lane >> 4) * kSlotBytes + (lane & 3) * 4;
  if (result == kOut) {
    uint16_t* out = g.out + first * g.out_stride + col0 + lane;
    const int64_t stride = g.out_stride;
#pragma unroll
    for (int r0 = 0; r0 < kRows; r0 += kBatch) {
      float v[kBatch][2];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[b][h] = shared_load1(from[h] + slot_at(warp * kRows + r0 + b, h * 4 + ((lane & 15) >> 2)));
#pragma unroll
      for (int b = 0; b < kBatch; ++b, out += stride)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (r0 + b < rows && there[h]) out[32 * h] = __bfloat16_as_ushort(__float2bfloat16_rn(v[b][h]));
    }
    return;
  }
  const int64_t shard = ap.shard;
  const float keep = ap.keep, step = g.step;
  int64_t f = g.flat + static_cast<int64_t>(first) * n + col0 + lane;
  int64_t rank = f / shard, at = f - rank * shard;  // of element (row, col0 + lane)
  uint16_t* full = ap.full + f;
#pragma unroll
  for (int r0 = 0; r0 < kRows; r0 += kBatch) {
    float v[kBatch][2], old[kBatch][2];
    float* where[kBatch][2];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v[b][h] = shared_load1(from[h] + slot_at(warp * kRows + r0 + b, h * 4 + ((lane & 15) >> 2)));
        const bool use = r0 + b < rows && there[h];
        int64_t a = at + 32 * h, r = rank;
        if (use)
          while (a >= shard) a -= shard, ++r;
        where[b][h] = use ? ap.master[r] + a : nullptr;
        old[b][h] = use ? *where[b][h] : 0.0f;
      }
      at += n;
      if (r0 + b + 1 < rows)
        while (at >= shard) at -= shard, ++rank;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b, full += n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!where[b][h]) continue;
        const float w = old[b][h] * keep - step * v[b][h];
        *where[b][h] = w;
        full[32 * h] = __bfloat16_as_ushort(__float2bfloat16_rn(w));
      }
  }
}

// One of the three products over all matrices of a launch (kLong: segments of the long Gram
// products, left as fp32 for ns_join); which tile by pair_time() and
// block_time() below. What bounds it, by size (measured on GB300):
//   - long sides from 2048 on: the tensor cores under the power cap. A step of 64 of a 256 x
//     256 tile takes 0.33 us at first, 2.0 PFLOP/s over 76 pairs; a long run of such launches
//     settles at 1.5 to 1.6 PFLOP/s, as cuBLAS does on fp16 operands (1.55 to 1.60; 1.69 on
//     bf16: more mantissa bits switch). Rounds that are not full cost the rest: 136 tiles of
//     a 4096-wide symmetric product are 1.8 rounds of 76.
//   - around 1000: shared memory. A step of a 128 x 128 tile writes 32 KB of operands and
//     the products read them once: 512 cycles at 128 bytes each, 0.27 us of the
//     measured 0.28, where the products themselves take half of that. And about 4 us of
//     each launch are its start and end (1 us from the previous kernel's end to the
//     wait's return, 0.8 to the first stage, 0.9 for a chunk to leave, 0.5 to the exit).
// (The whole of 5 steps: 4096 x 11008 2.3 ms, 1.35 PFLOP/s of the work that symmetry leaves;
// 768 x 2304, 768 x 768, 768 x 3072 and 3072 x 768 together 0.22 ms; 512 x 512 0.10 ms.)
// Halving the inner dimension between two blocks of a cluster where tiles are few was
// slower below 768 x 3072 (512 x 512 110 us) and 2 to 6 % faster above: not kept.
template <int kN, int kPair, int kMats, bool kLong>
__global__ void __launch_bounds__(kGemmThreads, 1) ns_product(const __grid_constant__ GemmParams<kMats> p) {
  using T = Tile<kN, kPair>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full_bar[T::kStages], empty_bar[T::kStages], done_bar[2], free_bar[2];
  __shared__ __align__(8) uint64_t in_bar[2], out_bar[2];     // a set of slots: `in` has come; the result has left
  __shared__ uint32_t tmem_slot;
  __shared__ int stop;
  __shared__ float squares[2][kEpilogueWarps];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t slots = smem + T::kStages * T::kStageBytes;
  const int rank = kPair == 2 ? static_cast<int>(block_rank()) : 0;
  // Tiles go round the clusters forwards, then backwards, and so on: they are sorted by
  // length, so who had a long one in one round gets a short one in the next.
  const int cluster = blockIdx.x / kPair, clusters = gridDim.x / kPair;
  const auto tile_of = [=](int turn) { return turn * clusters + (turn & 1 ? clusters - 1 - cluster : cluster); };
  const Guard guard{&stop, p.status, kWaitLimitNs};
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      bar_init(smem_addr(&full_bar[s]), 1);
      bar_init(smem_addr(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(smem_addr(&done_bar[b]), 1);
      bar_init(smem_addr(&free_bar[b]), kEpilogueWarps * kPair);
      bar_init(smem_addr(&in_bar[b]), 1);
      bar_init(smem_addr(&out_bar[b]), kEpilogueWarps);
    }
    stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Held while this grid waits for the previous one, which is safe: with its 225 KB a block shares its SM
  // with no other block that has tensor memory, and the next launch starts after this barrier.
  if (warp == 1) tmem_alloc<kPair>(smem_addr(&tmem_slot), T::kTmemCols);
  if (warp == 2 && lane < 3) {  // the first matrix's maps
    const GemmMat& g = p.mat[0];
    prefetch_map(lane == 0 ? g.p : lane == 1 ? g.q : g.result);
  }
  fence_before();
  __syncthreads();
  if constexpr (kPair == 2) cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_slot;
  // The previous kernel's results: each role waits for them right before its first
  // access, after it has read its part of the parameters (their first reads miss the
  // constant cache, about 1 us in all).
  asm volatile("griddepcontrol.launch_dependents;");
  const auto await_inputs = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };

  // sets of slots: a chunk needs hi and lo, or a part and its mirror image, or all four
  const int sets = p.terms == 3 && p.kind != kUpdate ? 1 : 2;
  const uint32_t set_bytes = sets == 1 ? kSlots * kSlotBytes : 2 * kSlotBytes;
  // steps of a tile's inner dimension from step `from` on
  const auto inner = [&](const GemmMat& g, int split, int* from) {
    const int blocks = (g.k + kTileK - 1) / kTileK;
    *from = kLong ? split * g.seg_blocks : 0;
    return kLong ? min(g.seg_blocks, blocks - *from) : blocks;
  };
  // whether this block finishes the chunk of a tile
  const auto has_chunk = [&](const GemmMat& g, int block, int col0) {
    return !(col0 >= g.n || block * 128 >= g.m || (g.symmetric && col0 / 128 > block));
  };

  if (warp == 0) {  // producer: this block's rows of both operands
    Tiles<T, GemmParams<kMats>, kLong> tiles{p};
    uint32_t it = 0;
    bool ok = true;
    for (int turn = 0, t = tile_of(0); ok && t < p.tiles; t = tile_of(++turn)) {
      int i, j;
      const GemmMat& g = tiles.at(t, &i, &j);
      int from;
      const int blocks = inner(g, tiles.split, &from);
      const int row0 = i * T::kM + rank * 128, col0 = j * kN + rank * T::kBRows;
      int term = 0, kb = 0;
      const bool p_mn = g.p_mn, q_mn = g.q_mn;
      for (int step = 0; step < blocks * p.terms; ++step, ++it) {
        const CUtensorMap* mp = &g.p[term == 1 ? 1 : 0];
        const CUtensorMap* mq = &g.q[term == 2 ? 1 : 0];
        const int s = it % T::kStages;
        ok = bar_wait_warp(smem_addr(&empty_bar[s]), ((it / T::kStages) & 1u) ^ 1u, guard);
        if (!ok) break;
        // the first block's barrier counts the bytes of both
        const uint32_t own = smem_addr(&full_bar[s]), bar = kPair == 2 ? in_block(own, 0) : own;
        const uint32_t a = smem + s * T::kStageBytes, b = a + T::kABytes;
        if (it == 0) await_inputs();
        if (elect_one()) {
          if (rank == 0) bar_expect(own, T::kStageBytes * kPair);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int r = row0 + 64 * q;
            tma_box<kPair>(a + q * 8192, mp, p_mn ? r : (from + kb) * kTileK, p_mn ? (from + kb) * kTileK : r, bar);
          }
#pragma unroll
          for (int q = 0; q < T::kBRows / 64; ++q) {
            const int c = col0 + 64 * q;
            tma_box<kPair>(b + q * 8192, mq, q_mn ? c : (from + kb) * kTileK, q_mn ? (from + kb) * kTileK : c, bar);
          }
        }
        __syncwarp();
        if (++kb == blocks) kb = 0, ++term;
      }
    }
    // every copy lands (its stage is used and released) before the block ends
    for (uint32_t back = 1; back <= T::kStages && back <= it; ++back) {
      const uint32_t last = it - back;
      const uint64_t* bar = rank == 0 ? full_bar : empty_bar;
      bar_drain(smem_addr(&bar[last % T::kStages]), (last / T::kStages) & 1u, kWaitLimitNs);
    }
  } else if (warp == 1 && rank == 0) {  // products, for both blocks of a pair
    Tiles<T, GemmParams<kMats>, kLong> tiles{p};
    uint32_t it = 0, n = 0;
    bool ok = true;
    for (int t = tile_of(0); ok && t < p.tiles; t = tile_of(++n)) {
      int i, j;
      const GemmMat& g = tiles.at(t, &i, &j);
      int from;
      const int steps = inner(g, tiles.split, &from) * p.terms;
      if (n == 0) await_inputs();  // the limit of the waits below does not run while earlier kernels do
      const uint32_t buf = n & 1u, d = tmem + buf * kN;
      ok = bar_wait_warp(smem_addr(&free_bar[buf]), ((n >> 1) & 1u) ^ 1u, guard);
      if (!ok) break;
      fence_after();
      const uint32_t kind = product_kind(T::kM, kN, g.p_mn, g.q_mn);
      // bytes from one 16-deep product's operand to the next, and between blocks of 64 rows
      const uint32_t a_step = g.p_mn ? 2048 : 32, b_step = g.q_mn ? 2048 : 32;
      const uint32_t a_block = g.p_mn ? 8192 : 0, b_block = g.q_mn ? 8192 : 0;
      for (int step = 0; step < steps; ++step, ++it) {
        const int s = it % T::kStages;
        ok = bar_wait_warp(smem_addr(&full_bar[s]), (it / T::kStages) & 1u, guard);
        if (!ok) break;
        fence_after();
        const uint32_t a = smem + s * T::kStageBytes, b = a + T::kABytes;
        const uint64_t da = operand(a, a_block, 1024), db = operand(b, b_block, 1024);
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < kTileK / 16; ++q)
            mma<kPair>(d, da + (q * a_step >> 4), db + (q * b_step >> 4), kind, step > 0 || q > 0);
          mma_commit<kPair>(smem_addr(&empty_bar[s]));
        }
        __syncwarp();
      }
      if (ok && elect_one()) mma_commit<kPair>(smem_addr(&done_bar[buf]));
      __syncwarp();
    }
    if (!ok && it > 0)  // products in flight end before the accumulators are freed
      bar_drain(smem_addr(&empty_bar[(it - 1) % T::kStages]), ((it - 1) / T::kStages) & 1u, kWaitLimitNs);
  } else if (warp == 2 && p.kind != kGram) {  // fetch of `in`, ahead of the epilogue
    Tiles<T, GemmParams<kMats>, kLong> tiles{p};
    const int parts = p.kind == kUpdate || p.terms == 3 ? 2 : 1;
    uint32_t e = 0;
    bool ok = true;
    for (int turn = 0, t = tile_of(0); ok && t < p.tiles; t = tile_of(++turn)) {
      int i, j;
      const GemmMat& g = tiles.at(t, &i, &j);
      const int block = i * kPair + rank;
      const CUtensorMap* in = g.in_q ? g.q : g.p;
      for (int c = 0; c < kN / kChunk; ++c) {
        const int col0 = j * kN + c * kChunk;
        if (!has_chunk(g, block, col0)) continue;
        const uint32_t set = e % sets, bar = smem_addr(&in_bar[set]), to = slots + set * set_bytes;
        ok = bar_wait_warp(smem_addr(&out_bar[set]), ((e / sets) & 1u) ^ 1u, guard);
        if (!ok) break;
        if (e == 0) await_inputs();
        if (elect_one()) {
          bar_expect(bar, parts * kSlotBytes);
          for (int part = 0; part < parts; ++part)
            for (int b = 0; b < 2; ++b)
              tma_box<1>(to + part * kSlotBytes + b * 8192, &in[part], col0, block * 128 + 64 * b, bar);
        }
        __syncwarp();
        ++e;
      }
    }
    for (uint32_t back = 1; back <= static_cast<uint32_t>(sets) && back <= e; ++back)
      bar_drain(smem_addr(&in_bar[(e - back) % sets]), ((e - back) / sets) & 1u, kWaitLimitNs);
  } else if (warp >= 4) {  // epilogue: this block's 128 rows
    Tiles<T, GemmParams<kMats>, kLong> tiles{p};
    const int own = warp - 4, quarter = own & 3, half = own >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    await_inputs();
    uint32_t n = 0, e = 0, left = 0;            // tiles, chunks, chunks whose slots this warp has released
    // a wait of this thread ran out; some thread's did (the same for all, known at the next barrier)
    bool lost = false, failed = false;
    int known = -1, side = 0;                   // the matrix whose m is `shift`; the set of sums in use
    float shift = 0.0f;
    for (int t = tile_of(0); !failed && t < p.tiles; t = tile_of(++n)) {
      int i, j;
      const GemmMat& g = tiles.at(t, &i, &j);
      if (!kLong && known != tiles.mat) {  // its m, from all blocks' sums in a fixed order
        known = tiles.mat;
        shift = 0.0f;
        if (g.squares) {
          float sum = 0.0f;
          const int count = g.squares_count;
#pragma unroll 8
          for (int k = threadIdx.x - 128; k < count; k += 32 * kEpilogueWarps) sum += g.squares[k];
          sum = warp_sum(sum);
          if (lane == 0) squares[side][own] = sum;
          failed = named_or(1, 32 * kEpilogueWarps, lost);
          if (failed) break;
          sum = 0.0f;
#pragma unroll
          for (int k = 0; k < kEpilogueWarps; ++k) sum += squares[side][k];
          side ^= 1;  // the next matrix's barrier comes before this set is written again
          shift = sum / (kScaleX * kScaleX) / static_cast<float>(min(g.m, min(g.n, g.k)));
          if (shift < kShiftFrom) shift = 0.0f;
        }
      }
      const float alpha = p.kind == kGram ? kScaleA / (kScaleX * kScaleX) : p.kind == kPoly ? p.c / kScaleA : 1.0f / kScaleA;
      const float beta = p.kind == kPoly ? p.b + 2.0f * p.c * shift : p.a + p.b * shift + p.c * shift * shift;
      const int block = i * kPair + rank;  // in rows of 128, as col0 / 128 in columns
      const uint32_t buf = n & 1u;
      lost |= !bar_wait(smem_addr(&done_bar[buf]), (n >> 1) & 1u, guard);
      fence_after();
      if constexpr (kLong) {
        failed = named_or(1, 32 * kEpilogueWarps, lost);
        const int64_t ld = square_of(g.n);
        for (int c = 0; c < kN / kChunk && !failed; ++c) {
          const int col0 = j * kN + c * kChunk + half * 32, row0 = block * 128 + quarter * 32;
          if (col0 >= ld || row0 >= ld) continue;  // the same for the warp
          float v[32];
          __syncwarp();
          tmem_load32(lanes + buf * kN + c * kChunk + half * 32, v);
          float4* to = reinterpret_cast<float4*>(g.partial + (tiles.split * ld + row0 + lane) * ld + col0);
#pragma unroll
          for (int q = 0; q < 8; ++q) to[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
      }
      for (int c = 0; !kLong && c < kN / kChunk; ++c) {
        const int col0 = j * kN + c * kChunk;
        if (!has_chunk(g, block, col0)) continue;
        const uint32_t set = e % sets, base = slots + set * set_bytes;
        float v[32];
        __syncwarp();
        tmem_load32(lanes + buf * kN + c * kChunk + half * 32, v);
#pragma unroll
        for (int q = 0; q < 32; ++q) v[q] *= alpha;
        if (p.kind == kGram) {
          lost |= !bar_wait(smem_addr(&out_bar[set]), ((e / sets) & 1u) ^ 1u, guard);
          const int diagonal = block * 128 + row - (col0 + half * 32);
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] -= q == diagonal ? shift * kScaleA : 0.0f;
        } else {
          lost |= !bar_wait(smem_addr(&in_bar[set]), (e / sets) & 1u, guard);
          for (int part = 0; part < (p.kind == kUpdate || p.terms == 3 ? 2 : 1); ++part) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint4 w = shared_load(base + part * kSlotBytes + slot_at(row, half * 4 + q));
              const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[k]));
                v[8 * q + 2 * k] += beta * f.x;
                v[8 * q + 2 * k + 1] += beta * f.y;
              }
            }
          }
        }
        const bool mirror = g.symmetric && col0 / 128 < block;
        if (p.result != kParts) {  // fp32 where the thread's own hi and lo were
#pragma unroll
          for (int q = 0; q < 8; ++q)
            shared_store(base + (q >> 2) * kSlotBytes + slot_at(row, half * 4 + (q & 3)),
                         __float_as_uint(v[4 * q] * (1.0f / kScaleX)), __float_as_uint(v[4 * q + 1] * (1.0f / kScaleX)),
                         __float_as_uint(v[4 * q + 2] * (1.0f / kScaleX)), __float_as_uint(v[4 * q + 3] * (1.0f / kScaleX)));
        } else {
          if (p.kind == kUpdate) {
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < 32; ++q) sum += v[q] * v[q];
            sum = warp_sum(sum);
            if (lane == 0) g.new_squares[(block * 4 + quarter) * ((g.n + 63) / 64 * 2) + col0 / 32 + half] = sum;
          }
          uint32_t r[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const __half2 h = __floats2half2_rn(v[2 * q], v[2 * q + 1]);
            const float2 f = __half22float2(h);
            v[2 * q] -= f.x, v[2 * q + 1] -= f.y;
            r[q] = *reinterpret_cast<const uint32_t*>(&h);
          }
          const bool lo_too = p.kind == kUpdate || p.terms == 3;
          put_part(base, row, half, r);
          if (mirror) put_mirror(base + (lo_too ? 2 : 1) * kSlotBytes, row, half, r);
          if (lo_too) {
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const __half2 l = __floats2half2_rn(v[2 * q], v[2 * q + 1]);
              r[q] = *reinterpret_cast<const uint32_t*>(&l);
            }
            put_part(base + kSlotBytes, row, half, r);
            if (mirror) put_mirror(base + 3 * kSlotBytes, row, half, r);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        failed = named_or(1, 32 * kEpilogueWarps, lost);
        if (failed) break;
        if (p.result != kParts) {
          finish_rows(g, p.apply, p.result, base, block * 128, col0, own, lane);
          // the slots were read by every warp, and may be written by the next fetch
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          named_or(1, 32 * kEpilogueWarps, false);
          if (lane == 0) bar_arrive(smem_addr(&out_bar[set]));
        } else if (lane == 0) {
          // up to eight boxes, one for each warp to send: part, half of the rows, direct or mirrored
          const int parts = p.kind == kUpdate || p.terms == 3 ? 2 : 1;
          const int b = own & 1, part = own >> 1 & 1, at = block * 128 + 64 * b;
          if (part < parts && at < g.m) {
            if (own < 4)
              tma_store(&g.result[part], col0, at, base + part * kSlotBytes + b * 8192);
            else if (mirror)
              tma_store(&g.result[part], at, col0, base + (parts + part) * kSlotBytes + b * 8192);
          }
          bulk_commit();
          // this warp's box of the chunk before this one (of this one, with a single set) has left its slot
          if (sets == 2)
            bulk_wait_read<1>();
          else
            bulk_wait_read<0>();
          for (const uint32_t gone = sets == 2 ? e : e + 1; left < gone; ++left) bar_arrive(smem_addr(&out_bar[left % sets]));
        }
        ++e;
      }
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair == 2)
          bar_arrive_cluster(in_block(smem_addr(&free_bar[buf]), 0));
        else
          bar_arrive(smem_addr(&free_bar[buf]));
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (kPair == 2) cluster_sync();  // neither block leaves while the other may signal it
  fence_after();
  if (warp == 1) tmem_free<kPair>(tmem, T::kTmemCols);
}

// The sum of the segments of the long Gram products: A (shifted, as two parts) from the fp32
// results, a block of 32 x 32 on or below the diagonal and its mirror image per block of
// threads. Bound by reading 4 bytes per element and segment.
template <int kMats>
__global__ void __launch_bounds__(32 * kEpilogueWarps) ns_join(const __grid_constant__ GemmParams<kMats> p) {
  __shared__ uint32_t mirror[32][33];
  __shared__ float squares[kEpilogueWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int i = 0, b = blockIdx.x;
  for (;; ++i) {
    const int wide = square_of(p.mat[i].n) / 32, blocks = p.mat[i].splits ? wide * (wide + 1) / 2 : 0;
    if (b < blocks) break;
    b -= blocks;
  }
  const GemmMat& g = p.mat[i];
  int bi = static_cast<int>((sqrtf(8.0f * b + 1.0f) - 1.0f) * 0.5f);
  while (bi * (bi + 1) / 2 > b) --bi;
  while ((bi + 1) * (bi + 2) / 2 <= b) ++bi;
  const int bj = b - bi * (bi + 1) / 2, splits = g.splits, n = g.n;
  const int64_t ld = square_of(n), next = ld * ld;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float shift = 0.0f;
  if (g.squares) {  // m, in the order of ns_product
    float sum = 0.0f;
    const int count = g.squares_count;
#pragma unroll 8
    for (int k = threadIdx.x; k < count; k += 32 * kEpilogueWarps) sum += g.squares[k];
    sum = warp_sum(sum);
    if (lane == 0) squares[warp] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kEpilogueWarps; ++k) sum += squares[k];
    shift = sum / (kScaleX * kScaleX) / static_cast<float>(n);
    if (shift < kShiftFrom) shift = 0.0f;
  }
  constexpr int kRows = 32 / kEpilogueWarps;
  const float* from = g.partial + (bi * 32 + warp) * ld + bj * 32 + lane;
  float v[kRows] = {};
#pragma unroll 4
  for (int s = 0; s < splits; ++s, from += next)
#pragma unroll
    for (int k = 0; k < kRows; ++k) v[k] += from[k * kEpilogueWarps * ld];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = bi * 32 + warp + k * kEpilogueWarps, c = bj * 32 + lane;
    v[k] = v[k] * (kScaleA / (kScaleX * kScaleX)) - (r == c ? shift * kScaleA : 0.0f);
    const __half hi = __float2half_rn(v[k]), lo = __float2half_rn(v[k] - __half2float(hi));
    mirror[warp + k * kEpilogueWarps][lane] = __half_as_ushort(hi) | static_cast<uint32_t>(__half_as_ushort(lo)) << 16;
    if (r >= n || c >= n) continue;
    g.joined[0][r * g.joined_ld + c] = hi;
    if (g.joined[1]) g.joined[1][r * g.joined_ld + c] = lo;
  }
  if (bi == bj) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = bj * 32 + warp + k * kEpilogueWarps, c = bi * 32 + lane;
    if (r >= n || c >= n) continue;
    const uint32_t two = mirror[lane][warp + k * kEpilogueWarps];
    g.joined[0][r * g.joined_ld + c] = __ushort_as_half(static_cast<unsigned short>(two));
    if (g.joined[1]) g.joined[1][r * g.joined_ld + c] = __ushort_as_half(static_cast<unsigned short>(two >> 16));
  }
}

// ----------------------------------------------------------- small matrices

// A matrix with a short side of at most 128 that fits the shared memory of one
// block goes through all its steps there, in one launch: X's two parts and those
// of A (then of P, in the same place) as 128-byte-swizzled operand tiles, the
// products in tensor memory, the short side's rows on its lanes. The three products
// of a step follow one another, so it is bound by their latency, about 1 us each
// with the passes between them (16 x 16: 15 us for 5 steps, 64 x 32 18, 128 x 128 42,
// 100 x 300 69 us, whatever the number of matrices up to one for each SM). Tall
// matrices are transposed as they are read.
constexpr int kSmallSide = 128;
constexpr int kSmallThreads = 256;
constexpr int kSmallBytes = 220 * 1024;
constexpr int kSmallSlack = 128 * 128;  // a product reads 128 rows whatever the short side
constexpr int kSmallMats = 48;
constexpr int kSmallCols = 256;         // of X per product

struct SmallMat {
  const void* source;
  int64_t source_stride;
  uint16_t* out;
  int64_t out_stride;
  int64_t flat;
  int32_t rows, cols;
  int32_t dtype;
  float step;
};

struct SmallParams {
  SmallMat mat[kSmallMats];
  NsApply apply;
  NsMomentum momentum;  // applies: the step's first part, done here too
  float coef[3 * 32];
  int32_t steps, terms;
  float eps;
  bool applies;
  unsigned int* status;
};
static_assert(sizeof(SmallParams) <= 32764, "kernel parameter block too large");

struct SmallShape {
  int side, length;      // of the wide orientation
  int side16, blocks;    // padded short side; 64-column blocks of X
  int part_x, part_a;    // bytes of one part
  __host__ __device__ SmallShape(int rows, int cols) {
    side = rows < cols ? rows : cols;
    length = rows < cols ? cols : rows;
    side16 = (side + 15) / 16 * 16;
    blocks = (length + 63) / 64;
    part_x = side16 * blocks * 128;
    part_a = side16 * ((side16 + 63) / 64) * 128;
  }
  __host__ __device__ int bytes() const { return 2 * part_x + 2 * part_a + kSmallSlack + 1024; }
};

// Byte of element (row, col) in a part: 64-column blocks of rows of 128 bytes, whose
// 16-byte pieces are exchanged by the row's place in its group of 8.
__device__ __forceinline__ int small_at(int rows, int row, int col) {
  return (col >> 6) * rows * 128 + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2;
}

__global__ void __launch_bounds__(kSmallThreads) ns_small(const __grid_constant__ SmallParams p) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t done_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int stop;
  __shared__ float norm;
  const SmallMat g = p.mat[blockIdx.x];
  const SmallShape s(g.rows, g.cols);
  const bool wide = g.rows <= g.cols;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  unsigned char* x = raw + (base - smem_addr(raw));
  unsigned char* a = x + 2 * s.part_x;
  const uint32_t x_addr = base, a_addr = base + 2 * s.part_x;
  const Guard guard{&stop, p.status, kWaitLimitNs};
  if (threadIdx.x == 0) {
    bar_init(smem_addr(&done_bar), 1);
    stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = threadIdx.x * 16; i < 2 * s.part_x; i += kSmallThreads * 16)
    *reinterpret_cast<uint4*>(x + i) = make_uint4(0, 0, 0, 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Tensor memory is held by no block that still waits for another grid (several of these blocks
  // share an SM), and the next launch starts when every block here has its columns: who queues
  // for columns queues behind blocks that run to their end.
  if (warp == 0) tmem_alloc<1>(smem_addr(&tmem_slot), kSmallCols);
  const int count = g.rows * g.cols;
  float squares = 0.0f;
  if (p.applies) {  // u, written to where this block reads it again after the barrier below
    const NsMomentum& m = p.momentum;
    float* u = static_cast<float*>(const_cast<void*>(g.source));
    int64_t at = g.flat + threadIdx.x, rank = at / m.shard;
    at -= rank * m.shard;
    constexpr int kBatch = 4;  // elements of a thread whose loads are in flight together
    for (int i0 = threadIdx.x; i0 < count; i0 += kBatch * kSmallThreads) {
      float* mom[kBatch];
      float old[kBatch], sum[kBatch] = {};
#pragma unroll
      for (int b = 0; b < kBatch; ++b, at += kSmallThreads) {
        const bool there = i0 + b * kSmallThreads < count;
        if (there)
          while (at >= m.shard) at -= m.shard, ++rank;
        mom[b] = there ? m.momentum[rank] + at : nullptr;
        old[b] = there ? *mom[b] : 0.0f;
      }
#pragma unroll 4
      for (int k = 0; k < m.w; ++k) {
        const uint16_t* row = m.grads[k] + g.flat + i0;
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          sum[b] += __bfloat162float(__ushort_as_bfloat16(mom[b] ? row[b * kSmallThreads] : uint16_t(0)));
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (!mom[b]) continue;
        const float mean = mean_of(sum[b], m);
        const float v = m.mu * old[b] + mean;
        *mom[b] = v;
        u[i0 + b * kSmallThreads] = m.nesterov ? mean + m.mu * v : v;
      }
    }
  }
  // Everything outside the products goes by pieces of 8 columns of X: piece t lies in row
  // `row` from column `col` on, `n` of its elements are inside, element e is at (r, c) of the
  // matrix. Neighbouring threads have neighbouring elements of the matrix.
  struct Piece {
    int row, col, n, at;
  };
  const int per_row = (s.length + 7) / 8, all = s.side * per_row;
  const auto piece = [&](int t) {
    const int q = wide ? t / per_row : t / s.side;
    const int row = wide ? q : t - q * s.side, col = 8 * (wide ? t - q * per_row : q);
    return Piece{row, col, min(8, s.length - col), small_at(s.side16, row, col)};
  };
  const int64_t along = wide ? 1 : g.source_stride, across = wide ? g.source_stride : 1;
  __syncthreads();  // the zeros, and u, are written, and the columns are held
  asm volatile("griddepcontrol.launch_dependents;");
  // The source is read once: its fp32 bits wait where the element's two parts will be,
  // until the norm is known.
  for (int t = threadIdx.x; t < all; t += kSmallThreads) {
    const Piece q = piece(t);
    const int64_t from = q.row * across + q.col * along;
    float v[8];
    if (g.dtype == FSDP_DTYPE_F32) {
      const float* src = static_cast<const float*>(g.source) + from;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = src[(e < q.n ? e : 0) * along];
    } else {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(g.source) + from;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __bfloat162float(src[(e < q.n ? e : 0) * along]);
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = e < q.n ? v[e] : 0.0f;
      squares += v[e] * v[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t a0 = __float_as_uint(v[2 * e]), a1 = __float_as_uint(v[2 * e + 1]);
      hi[e] = __byte_perm(a0, a1, 0x7632);
      lo[e] = __byte_perm(a0, a1, 0x5410);
    }
    *reinterpret_cast<uint4*>(x + q.at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(x + s.part_x + q.at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  block_sum_to(squares, &norm);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  const float inv = 1.0f / (sqrtf(norm) + p.eps);
  for (int t = threadIdx.x; t < all; t += kSmallThreads) {
    const Piece q = piece(t);
    const uint4 h = *reinterpret_cast<const uint4*>(x + q.at), l = *reinterpret_cast<const uint4*>(x + s.part_x + q.at);
    const uint32_t hi[4] = {h.x, h.y, h.z, h.w}, lo[4] = {l.x, l.y, l.z, l.w};
    uint32_t first[4], second[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a0 = __uint_as_float(__byte_perm(lo[e], hi[e], 0x5410)) * inv * kScaleX;
      const float a1 = __uint_as_float(__byte_perm(lo[e], hi[e], 0x7632)) * inv * kScaleX;
      const __half2 t0 = __floats2half2_rn(a0, a1);
      const float2 f = __half22float2(t0);
      const __half2 t1 = __floats2half2_rn(a0 - f.x, a1 - f.y);
      first[e] = *reinterpret_cast<const uint32_t*>(&t0);
      second[e] = *reinterpret_cast<const uint32_t*>(&t1);
    }
    *reinterpret_cast<uint4*>(x + q.at) = make_uint4(first[0], first[1], first[2], first[3]);
    *reinterpret_cast<uint4*>(x + s.part_x + q.at) = make_uint4(second[0], second[1], second[2], second[3]);
  }
  uint32_t phase = 0;
  // a wait of this thread ran out; some thread's did (the same for all, known at the next barrier)
  bool lost = false, failed = false;
  // Makes what the threads wrote visible to the products, lets warp 0 issue them, and waits for them.
  const auto run = [&](auto issue) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    fence_before();
    failed = __syncthreads_or(lost);
    if (failed) return;
    if (warp == 0) {
      fence_after();
      issue();
      if (elect_one()) mma_commit<1>(smem_addr(&done_bar));
      __syncwarp();
    }
    lost = !bar_wait(smem_addr(&done_bar), phase & 1u, guard);
    ++phase;
    fence_after();
  };
  const int row = (warp & 3) * 32 + lane;
  const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const bool busy = (warp & 3) * 32 < s.side16;  // some lane of the warp has a row
  // old = hi + lo of a piece; stores `v` as two parts
  const auto sum_of = [](const uint4& hi, const uint4& lo, float* out) {
    const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&l[e]));
      out[2 * e] = f.x + t.x;
      out[2 * e + 1] = f.y + t.y;
    }
  };
  const auto put = [](const float* v, uint4* hi, uint4* lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 t = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
      const float2 f = __half22float2(t);
      const __half2 u = __floats2half2_rn(v[2 * e] - f.x, v[2 * e + 1] - f.y);
      h[e] = *reinterpret_cast<const uint32_t*>(&t);
      l[e] = *reinterpret_cast<const uint32_t*>(&u);
    }
    *hi = make_uint4(h[0], h[1], h[2], h[3]);
    *lo = make_uint4(l[0], l[1], l[2], l[3]);
  };
  // Columns [col0, col0 + cols) of this thread's row of a region at `to` become alpha times
  // the products' plus beta times (kOld) what is there; the two warps of a lane
  // quarter take 32 columns by turns. All reads come before the first write.
  const auto update = [&](auto with_old, unsigned char* to, int part, int col0, int cols, float alpha, float beta) {
    constexpr bool kOld = decltype(with_old)::value;
    if (!busy) return;
    for (int c = (warp >> 2) * 32; c < cols; c += 64) {
      const int n = row < s.side16 ? min(4, (cols - c) / 8) : 0;
      unsigned char* at[4];
      uint4 hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        at[q] = to + small_at(s.side16, row, col0 + c + 8 * q);
        if (kOld && q < n) {
          hi[q] = *reinterpret_cast<const uint4*>(at[q]);
          lo[q] = *reinterpret_cast<const uint4*>(at[q] + part);
        }
      }
      float v[32];
      __syncwarp();
      tmem_load32(lanes + c, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q >= n) continue;
        float old[8];
        if (kOld) sum_of(hi[q], lo[q], old);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * q + e] = kOld ? beta * old[e] + alpha * v[8 * q + e] : alpha * v[8 * q + e];
        put(&v[8 * q], reinterpret_cast<uint4*>(at[q]), reinterpret_cast<uint4*>(at[q] + part));
      }
    }
  };
  const std::integral_constant<bool, true> added;
  const std::integral_constant<bool, false> fresh;
  const uint32_t block = static_cast<uint32_t>(s.side16) * 128;
  // One product over `deep` steps of 16 of the inner dimension, all terms: l and r are the hi
  // parts' descriptors, l_lo and r_lo their lo parts' distances, `mn`: r's steps are
  // 16 rows, else both operands' are 32 bytes within blocks of 64 columns.
  const auto product = [&](uint64_t l, int l_lo, uint64_t r, int r_lo, int deep, uint32_t kind, bool mn) {
    if (!elect_one()) return;
    for (int t = 0; t < p.terms; ++t) {
      const uint64_t lt = l + (t == 1 ? l_lo >> 4 : 0), rt = r + (t == 2 ? r_lo >> 4 : 0);
#pragma unroll 4
      for (int k = 0; k < deep; ++k) {
        const uint32_t at = ((k >> 2) * block + (k & 3) * 32) >> 4;
        mma<1>(tmem, lt + at, rt + (mn ? k * (2048 >> 4) : at), kind, t > 0 || k > 0);
      }
    }
  };
  const uint32_t square = product_kind(128, s.side16, false, false);
  const uint64_t x_rows = operand(x_addr, 0, 1024), a_rows = operand(a_addr, 0, 1024);
  for (int step = 0; step < p.steps && !failed; ++step) {
    const float ca = p.coef[3 * step], cb = p.coef[3 * step + 1], cc = p.coef[3 * step + 2];
    run([&] { product(x_rows, s.part_x, x_rows, s.part_x, (s.length + 15) / 16, square, false); });  // A = X X^T
    if (failed) break;
    update(fresh, a, s.part_a, 0, s.side16, kScaleA / (kScaleX * kScaleX), 0.0f);
    run([&] { product(a_rows, s.part_a, a_rows, s.part_a, s.side16 / 16, square, false); });  // A A
    if (failed) break;
    update(added, a, s.part_a, 0, s.side16, cc / kScaleA, cb);
    for (int col0 = 0; col0 < s.length && !failed; col0 += kSmallCols) {  // P X, columns from col0 on
      const int cols = min(kSmallCols, (s.length - col0 + 15) / 16 * 16);
      run([&] {
        product(a_rows, s.part_a, operand(x_addr + (col0 >> 6) * block, block, 1024), s.part_x, s.side16 / 16,
                product_kind(128, cols, false, true), true);
      });
      if (failed) break;
      update(added, x, s.part_x, col0, cols, 1.0f / kScaleA, ca);
    }
  }
  fence_before();
  failed = __syncthreads_or(lost);
  if (!failed) {
    for (int t = threadIdx.x; t < all; t += kSmallThreads) {
      const Piece q = piece(t);
      float v[8];
      sum_of(*reinterpret_cast<const uint4*>(x + q.at), *reinterpret_cast<const uint4*>(x + s.part_x + q.at), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= 1.0f / kScaleX;
      if (!p.applies) {
        const int64_t step = wide ? 1 : g.out_stride;
        uint16_t* out = g.out + (wide ? q.row * g.out_stride + q.col : q.col * g.out_stride + q.row);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < q.n) out[e * step] = __bfloat16_as_ushort(__float2bfloat16_rn(v[e]));
        continue;
      }
      const int64_t shard = p.apply.shard, step = wide ? 1 : g.cols;
      const int64_t f = g.flat + (wide ? static_cast<int64_t>(q.row) * g.cols + q.col : static_cast<int64_t>(q.col) * g.cols + q.row);
      int64_t rank = f / shard, at = f - rank * shard;
      float* master[8];
      float old[8];
#pragma unroll
      for (int e = 0; e < 8; ++e, at += step) {
        master[e] = nullptr;
        if (e < q.n) {
          while (at >= shard) at -= shard, ++rank;
          master[e] = p.apply.master[rank] + at;
        }
        old[e] = master[e] ? *master[e] : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!master[e]) continue;
        const float w = old[e] * p.apply.keep - g.step * v[e];
        *master[e] = w;
        p.apply.full[f + e * step] = __bfloat16_as_ushort(__float2bfloat16_rn(w));
      }
    }
  }
  if (warp == 0) {
    fence_after();
    tmem_free<1>(tmem, kSmallCols);
  }
}

// ------------------------------------------------------------- host side

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

int terms_of(const NsJob& j, const NsPlan& plan) {
  return plan.terms ? plan.terms : std::min(j.rows, j.cols) < 256 ? 3 : 1;
}

bool is_small(const NsJob& j) {
  if (std::min(j.rows, j.cols) > kSmallSide || std::max(j.rows, j.cols) > kSmallBytes) return false;
  return SmallShape(static_cast<int>(j.rows), static_cast<int>(j.cols)).bytes() <= kSmallBytes;
}

int parts_of(const NsJob& j) {
  const int64_t units = j.rows * ((j.cols + kUnit - 1) / kUnit);
  // two units a warp: the blocks of a GPT-2 block's matrices (528) then run at once
  return static_cast<int>(std::min<int64_t>(kMaxParts, (units + 2 * kPassWarps - 1) / (2 * kPassWarps)));
}

// The segments of a matrix's Gram product. Products of more than 256 steps are cut for their
// sums' sake. Others are cut where that saves one block a long wait: into segments of 24 steps or
// more, as many as give each of 152 SMs a tile, if at least 12 us of steps go (the second launch costs
// half of that; 31 x 5000 289 -> 112 us, 300 x 5000 169 -> 157, 1024 x 8192 328 -> 279; but twelve of
// 300 x 5000 471 -> 496; with
// 9 us 768 x 4096 would be cut, 192 -> 195 us alone and 575 -> 697 for eight of them). By the
// matrix alone, so that it gives the same bits in any company.
struct Segments {
  int splits = 0, blocks = 0;
};
Segments segments_of(const NsJob& j, int terms) {
  constexpr int kMostSteps = 256, kLeastSteps = 24, kSms = 152;
  const int64_t blocks = (std::max(j.rows, j.cols) + kTileK - 1) / kTileK, steps = blocks * terms;
  const int64_t rows = (std::min(j.rows, j.cols) + 127) / 128, tiles = rows * (rows + 1) / 2;
  const int64_t splits = std::max<int64_t>({(steps + kMostSteps - 1) / kMostSteps, std::min(kSms / tiles, steps / kLeastSteps), 1});
  const int64_t each = (blocks + splits - 1) / splits;
  if (steps <= kMostSteps && 0.28 * static_cast<double>(steps - each * terms) < 12.0) return {};
  return {static_cast<int>((blocks + each - 1) / each), static_cast<int>(each)};
}

// A matrix's share of the workspace: X twice (read and written by turns) and A, P,
// each as hi and, where it is used, lo part, rows a multiple of 128 bytes apart.
struct Buffers {
  __half *x[2][2], *a[2], *poly[2];
  float *partial, *squares[2], *segments;
  int64_t ld_x, ld_a;
  int64_t squares_count;
};

int64_t carve(const NsJob& j, const NsPlan& plan, unsigned char* base, Buffers* out) {
  const int terms = terms_of(j, plan);
  const int64_t side = std::min(j.rows, j.cols);
  Buffers b{};
  b.ld_x = round_up(j.cols, 64);
  b.ld_a = round_up(side, 64);
  if (is_small(j)) return 0;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    unsigned char* q = base ? base + at : nullptr;
    at += round_up(bytes, 256);
    return q;
  };
  for (int k = 0; k < 2; ++k)
    for (int part = 0; part < 2; ++part)
      b.x[k][part] = reinterpret_cast<__half*>(take(j.rows * b.ld_x * 2));
  for (int part = 0; part < (terms == 3 ? 2 : 1); ++part) {
    b.a[part] = reinterpret_cast<__half*>(take(side * b.ld_a * 2));
    b.poly[part] = reinterpret_cast<__half*>(take(side * b.ld_a * 2));
  }
  b.partial = reinterpret_cast<float*>(take(kMaxParts * 4));
  b.squares_count = (j.rows + 127) / 128 * 4 * (b.ld_x / 32);
  for (int k = 0; k < 2; ++k) b.squares[k] = reinterpret_cast<float*>(take(b.squares_count * 4));
  const int64_t square = square_of(static_cast<int>(side));
  b.segments = reinterpret_cast<float*>(take(segments_of(j, terms).splits * square * square * 4));
  if (out) *out = b;
  return at;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// Boxes of 64 x 64 elements of a rows x cols fp16 matrix; outside it they read zeros.
bool make_map(CUtensorMap* map, const __half* base, int64_t rows, int64_t cols, int64_t ld) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, 64}, step[2] = {1, 1};
  return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half*>(base), dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Device {
  int id = 0, sms = 0;
  unsigned int* status = nullptr;
};

int device_facts(Device* d) {
  if (cudaGetDevice(&d->id) != cudaSuccess ||
      cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, d->id) != cudaSuccess)
    return FSDP_ECUDA;
  return device_status_word(&d->status);
}

// Launches a kernel so that its blocks may be placed while the previous kernel of
// the stream ends; the kernels wait for that one's results themselves.
template <typename K, typename P>
int launch_after(K kernel, int grid, int cluster, int threads, int smem, cudaStream_t stream, const P& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? FSDP_OK : FSDP_ECUDA;
}

// How many clusters of the kernel run at once (looked up once per device).
template <int kN, int kPair, int kMats, bool kLong>
int resident_clusters(const Device& dev) {
  using T = Tile<kN, kPair>;
  static std::atomic<int> cached[64];
  if (dev.id >= 64) return 0;
  int n = cached[dev.id].load(std::memory_order_acquire);
  if (n) return n;
  const auto kernel = ns_product<kN, kPair, kMats, kLong>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmemBytes) != cudaSuccess) return 0;
  if (kPair == 1) {
    n = dev.sms;
  } else {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(dev.sms / kPair * kPair);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = T::kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPair;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return 0;
  }
  cached[dev.id].store(n, std::memory_order_release);
  return n;
}

template <int kN, int kPair, bool kLong = false, int kMats>
int launch_product(GemmParams<kMats>& p, const Device& dev, cudaStream_t stream) {
  using T = Tile<kN, kPair>;
  p.tiles = 0;
  for (int i = 0; i < p.count; ++i) {
    GemmMat& g = p.mat[i];
    const int rows = (g.m + T::kM - 1) / T::kM;
    g.col_tiles = (g.n + kN - 1) / kN;
    g.tiles = rows * g.col_tiles;
    if (g.symmetric) {
      g.tiles = 0;
      for (int r = 0; r < rows; ++r) g.tiles += T::below(r, g.col_tiles);
    }
    if (kLong) g.tiles *= g.splits;
    if (!kLong && g.splits) g.tiles = 0;
    p.tiles += g.tiles;
  }
  if (p.tiles == 0) return FSDP_OK;
  const int room = resident_clusters<kN, kPair, kMats, kLong>(dev);
  if (room < 1) return FSDP_ECUDA;
  return launch_after(ns_product<kN, kPair, kMats, kLong>, std::min(p.tiles, room) * kPair, kPair, kGemmThreads, T::kSmemBytes,
                      stream, p);
}

int launch_momentum(const MomentumParams& p, int blocks, cudaStream_t stream) {
  const auto go = [&](auto kernel) { return launch_after(kernel, blocks, 1, 32 * kPassWarps, 0, stream, p); };
  switch (p.m.w) {
    case 1: return go(ns_momentum<1>);
    case 2: return go(ns_momentum<2>);
    case 4: return go(ns_momentum<4>);
    case 8: return go(ns_momentum<8>);
    case 16: return go(ns_momentum<16>);
    default: return go(ns_momentum<0>);
  }
}

// Small matrices: one block each, all steps in one launch.
int run_small(const NsJob* const* jobs, int count, const NsPlan& plan, const NsMomentum* momentum, const NsApply* apply,
              const Device& dev, cudaStream_t stream) {
  static thread_local SmallParams p;
  if (momentum) p.momentum = *momentum;
  int smem = 0;
  for (int i = 0; i < count; ++i) {
    const NsJob& j = *jobs[i];
    p.mat[i] = {j.source, j.source_stride, j.out, j.out_stride, j.flat, static_cast<int32_t>(j.rows),
                static_cast<int32_t>(j.cols), j.dtype, j.step};
    smem = std::max(smem, SmallShape(static_cast<int>(j.rows), static_cast<int>(j.cols)).bytes());
  }
  if (apply) p.apply = *apply;
  p.applies = apply != nullptr;
  std::copy(plan.coef.begin(), plan.coef.end(), p.coef);
  p.steps = plan.steps;
  p.terms = plan.terms ? plan.terms : 3;
  p.eps = plan.eps;
  p.status = dev.status;
  if (cudaFuncSetAttribute(ns_small, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallBytes) != cudaSuccess)
    return FSDP_ECUDA;
  return launch_after(ns_small, count, 1, kSmallThreads, smem, stream, p);
}

// Estimated times, in microseconds, of a launch of `tiles` tiles of `steps` steps of 64
// of the inner dimension. Measured on GB300: a step of a 256 x 256 tile takes a pair 0.33 to
// 0.36, one of a 128 x 128 tile takes a block 0.28; a tile's results leave in 9 and 2.5
// beside the next tile's products, and the last one's in 11 and 2.5 after them.
// All steps of a GPT-2 block's matrices with pairs for the updates (12 steps each) 253 us,
// with single blocks 217; of 4096 x 4096 (64 steps) 1008 with pairs, 1233 with single blocks for the
// updates.
double pair_time(int64_t tiles, int steps, int sms) {
  const double rounds = static_cast<double>((tiles + sms / 2 - 1) / (sms / 2));
  return rounds * std::max(0.34 * steps, 9.0) + 11.0;
}
double block_time(int64_t tiles, int steps, int sms) {
  const double rounds = static_cast<double>((tiles + sms - 1) / sms);
  return rounds * std::max(0.28 * steps, 2.5) + 2.5;
}

// One launch's matrices through all steps.
template <int kMats>
int run_group(const NsJob* const* jobs, int count, const NsPlan& plan, int terms, const NsMomentum* momentum,
              const NsApply* apply, unsigned char* workspace, const Device& dev, cudaStream_t stream) {
  static thread_local MomentumParams first;
  PassParams& pass = first.pass;
  static thread_local GemmParams<kMats> p;
  struct Maps {
    CUtensorMap x[2][2], a[2], poly[2];
  };
  std::vector<Buffers> buffers(count);
  std::vector<Maps> maps(count);
  int blocks = 0;
  for (int i = 0; i < count; ++i) {
    const NsJob& j = *jobs[i];
    Buffers& b = buffers[i];
    workspace += carve(j, plan, workspace, &b);
    const int64_t side = std::min(j.rows, j.cols);
    bool ok = true;
    for (int part = 0; part < 2; ++part) {
      for (int k = 0; k < 2; ++k) ok = ok && make_map(&maps[i].x[k][part], b.x[k][part], j.rows, j.cols, b.ld_x);
      if (part == 1 && terms == 1) continue;
      ok = ok && make_map(&maps[i].a[part], b.a[part], side, side, b.ld_a);
      ok = ok && make_map(&maps[i].poly[part], b.poly[part], side, side, b.ld_a);
    }
    if (!ok) return FSDP_ECUDA;
    blocks += parts_of(j);
    pass.mat[i] = {j.source, j.source_stride, j.rows, j.cols, b.x[0][0], b.x[0][1], b.ld_x, b.partial, j.flat,
                   j.dtype, parts_of(j), blocks};
  }
  pass.count = count;
  pass.eps = plan.eps;
  if (momentum) {
    first.m = *momentum;
    if (int rc = launch_momentum(first, blocks, stream)) return rc;
  } else {
    if (int rc = launch_after(ns_squares, blocks, 1, 32 * kPassWarps, 0, stream, pass)) return rc;
  }
  if (int rc = launch_after(ns_normalise, blocks, 1, 32 * kPassWarps, 0, stream, pass)) return rc;
  p.count = count;
  p.terms = terms;
  p.status = dev.status;
  if (apply) p.apply = *apply;
  for (int s = 0; s < plan.steps; ++s) {
    const bool last = s + 1 == plan.steps;
    const int now = s & 1, next = now ^ 1;
    for (int kind = kGram; kind <= kUpdate; ++kind) {
      int64_t large_tiles = 0, small_tiles = 0;
      int steps = 0, join_blocks = 0;
      for (int i = 0; i < count; ++i) {
        const NsJob& j = *jobs[i];
        const Buffers& b = buffers[i];
        const Maps& q = maps[i];
        GemmMat& g = p.mat[i];
        const bool wide = j.rows <= j.cols;
        const int32_t side = static_cast<int32_t>(std::min(j.rows, j.cols));
        auto use = [&](CUtensorMap* to, const CUtensorMap* from) { std::memcpy(to, from, 2 * sizeof(CUtensorMap)); };
        g.symmetric = kind != kUpdate;
        g.m = g.n = g.k = side;
        g.p_mn = g.q_mn = g.in_q = 0;
        g.squares = s > 0 ? b.squares[now] : nullptr;
        g.new_squares = b.squares[next];
        g.squares_count = static_cast<int32_t>(b.squares_count);
        g.splits = 0;
        if (kind == kGram) {
          use(g.p, q.x[now]);
          use(g.q, q.x[now]);
          use(g.result, q.a);
          g.k = static_cast<int32_t>(std::max(j.rows, j.cols));
          g.p_mn = g.q_mn = !wide;
          const Segments cut = segments_of(j, terms);
          g.splits = cut.splits;
          g.seg_blocks = cut.blocks;
          g.partial = b.segments;
          g.joined[0] = b.a[0];
          g.joined[1] = b.a[1];
          g.joined_ld = b.ld_a;
          if (g.splits) {
            const int square = square_of(side) / 32;
            join_blocks += square * (square + 1) / 2;
            continue;
          }
        } else if (kind == kPoly) {
          use(g.p, q.a);
          use(g.q, q.a);
          use(g.result, q.poly);
        } else {
          use(g.p, wide ? q.poly : q.x[now]);
          use(g.q, wide ? q.x[now] : q.poly);
          use(g.result, q.x[next]);
          g.q_mn = g.in_q = wide;
          g.m = static_cast<int32_t>(j.rows);
          g.n = static_cast<int32_t>(j.cols);
          g.out = j.out;
          g.out_stride = j.out_stride;
          g.flat = j.flat;
          g.step = j.step;
        }
        const int64_t rows = (g.m + 127) / 128, cols = (g.n + 255) / 256;
        large_tiles += g.symmetric ? cols * (cols + 1) / 2 : (rows + 1) / 2 * cols;
        small_tiles += g.symmetric ? rows * (rows + 1) / 2 : rows * ((g.n + 127) / 128);
        steps = std::max(steps, (g.k + kTileK - 1) / kTileK * terms);
      }
      p.kind = kind;
      p.result = kind != kUpdate || !last ? kParts : apply ? kApply : kOut;
      p.a = plan.coef[3 * s];
      p.b = plan.coef[3 * s + 1];
      p.c = plan.coef[3 * s + 2];
      if (join_blocks) {
        if (int rc = launch_product<128, 1, true>(p, dev, stream)) return rc;
        if (int rc = launch_after(ns_join<kMats>, join_blocks, 1, 32 * kEpilogueWarps, 0, stream, p)) return rc;
      }
      // pairs of blocks on 256 x 256 tiles, or single ones on 128 x 128, whichever is estimated
      // faster: the sums and their order are the same, so that a matrix gives the same bits in
      // any company
      const bool pairs = pair_time(large_tiles, steps, dev.sms) < block_time(small_tiles, steps, dev.sms);
      const int rc = pairs ? launch_product<256, 2>(p, dev, stream) : launch_product<128, 1>(p, dev, stream);
      if (rc != FSDP_OK) return rc;
    }
  }
  return FSDP_OK;
}

}  // namespace

int ns_plan(const fsdp_newton_schulz_t* h, NsPlan* plan) {
  if (h) {
    if (h->steps < 1 || h->steps > 32 || (h->terms != 0 && h->terms != 1 && h->terms != 3)) return FSDP_EINVAL;
    const float eps = static_cast<float>(h->eps);
    if (!(eps >= 0x1p-126f) || !std::isfinite(eps)) return FSDP_EINVAL;  // 1 / eps has to be finite
    plan->steps = h->steps;
    plan->terms = h->terms;
    plan->eps = static_cast<float>(h->eps);
  }
  static const double kQuintic[3] = {3.4445, -4.7750, 2.0315};
  double top = 1.0;  // the largest singular value that a step can meet
  for (int i = 0; i < plan->steps; ++i) {
    const double* q = h && h->coefficients ? h->coefficients + 3 * i : kQuintic;
    const double a = q[0], b = q[1], c = q[2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return FSDP_EINVAL;
    // extrema of x (a + b s + c s^2) and of b s + c s^2, s = x^2 in [0, top^2]
    double at[4] = {top * top, 0.0, 0.0, 0.0};
    const double disc = 9.0 * b * b - 20.0 * a * c;
    if (c != 0.0 && disc >= 0.0) {
      at[1] = (-3.0 * b + std::sqrt(disc)) / (10.0 * c);
      at[2] = (-3.0 * b - std::sqrt(disc)) / (10.0 * c);
    } else if (c == 0.0 && b != 0.0) {
      at[1] = -a / (3.0 * b);
    }
    if (c != 0.0) at[3] = -b / (2.0 * c);
    double next = 0.0;
    for (double s : at) {
      if (!(s >= 0.0 && s <= top * top)) continue;
      next = std::max(next, std::fabs(std::sqrt(s) * (a + b * s + c * s * s)));
      if (std::fabs(b * s + c * s * s) > 30.0) return FSDP_EINVAL;
    }
    if (!(next <= 7.0)) return FSDP_EINVAL;
    top = next;
    for (int k = 0; k < 3; ++k) plan->coef.push_back(static_cast<float>(q[k]));
  }
  return FSDP_OK;
}

int64_t ns_workspace_bytes(const std::vector<NsJob>& jobs, const NsPlan& plan) {
  int64_t bytes = 256;
  for (const NsJob& j : jobs) bytes += carve(j, plan, nullptr, nullptr);
  return bytes;
}

int ns_run(const std::vector<NsJob>& jobs, const NsPlan& plan, const NsMomentum* momentum, const NsApply* apply,
           void* workspace, cudaStream_t stream) {
  Device dev;
  if (int rc = device_facts(&dev)) return rc;
  if (!encoder()) return FSDP_ECUDA;
  auto* base = reinterpret_cast<unsigned char*>(round_up(reinterpret_cast<intptr_t>(workspace), 256));
  std::vector<const NsJob*> small;
  for (const NsJob& j : jobs)
    if (is_small(j)) small.push_back(&j);
  for (size_t at = 0; at < small.size(); at += kSmallMats) {
    const int count = static_cast<int>(std::min<size_t>(kSmallMats, small.size() - at));
    if (int rc = run_small(&small[at], count, plan, momentum, apply, dev, stream)) return rc;
  }
  for (int terms : {1, 3}) {
    std::vector<const NsJob*> group;
    for (const NsJob& j : jobs)
      if (!is_small(j) && terms_of(j, plan) == terms) group.push_back(&j);
    // the tiles that take longest first, so that the short ones fill up the end
    std::stable_sort(group.begin(), group.end(), [](const NsJob* a, const NsJob* b) {
      return std::max(a->rows, a->cols) > std::max(b->rows, b->cols);
    });
    for (size_t at = 0; at < group.size(); at += kMaxMats) {
      const int count = static_cast<int>(std::min<size_t>(kMaxMats, group.size() - at));
      const int rc = count <= 8
                         ? run_group<8>(&group[at], count, plan, terms, momentum, apply, base, dev, stream)
                         : run_group<kMaxMats>(&group[at], count, plan, terms, momentum, apply, base, dev, stream);
      if (rc != FSDP_OK) return rc;
      for (int i = 0; i < count; ++i) base += carve(*group[at + i], plan, nullptr, nullptr);
    }
  }
  return FSDP_OK;
}

namespace {

constexpr int64_t kMaxSide = int64_t(1) << 30;

// The jobs of a call (empty matrices left out) and the overlap checks.
int make_jobs(const fsdp_matrix_t* matrices, int32_t n, bool pointers, std::vector<NsJob>* jobs) {
  if (n < 0 || (n > 0 && !matrices)) return FSDP_EINVAL;
  std::vector<Strided> in, out;
  for (int32_t i = 0; i < n; ++i) {
    const fsdp_matrix_t& q = matrices[i];
    if (q.rows < 0 || q.cols < 0 || q.rows > kMaxSide || q.cols > kMaxSide) return FSDP_EINVAL;
    if (q.dtype != FSDP_DTYPE_F32 && q.dtype != FSDP_DTYPE_BF16) return FSDP_EINVAL;
    if (q.rows == 0 || q.cols == 0) continue;
    if (pointers) {
      in.push_back({q.source, q.rows, q.cols, q.source_stride, size_of_dtype(q.dtype)});
      out.push_back({q.out, q.rows, q.cols, q.out_stride, 2});
      if (!in.back().ok() || !out.back().ok()) return FSDP_EINVAL;
    }
    jobs->push_back({q.source, q.source_stride, q.rows, q.cols, q.out, q.out_stride, 0, 0.0f, q.dtype});
  }
  for (size_t i = 0; i < out.size(); ++i)
    for (size_t k = 0; k < in.size(); ++k) {
      if (i != k && out[i].overlaps(out[k])) return FSDP_EALIAS;
      if (out[i].overlaps(in[k]) && !(i == k && out[i].same_place(in[k]))) return FSDP_EALIAS;
    }
  return FSDP_OK;
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" int fsdp_newton_schulz_workspace(const fsdp_matrix_t* matrices, int32_t n, const fsdp_newton_schulz_t* h,
                                            int64_t* bytes_out) try {
  if (!bytes_out) return FSDP_EINVAL;
  NsPlan plan;
  if (int rc = ns_plan(h, &plan)) return rc;
  std::vector<NsJob> jobs;
  if (int rc = make_jobs(matrices, n, false, &jobs)) return rc;
  *bytes_out = ns_workspace_bytes(jobs, plan);
  return FSDP_OK;
} catch (...) {
  return FSDP_ECUDA;
}

extern "C" int fsdp_newton_schulz(const fsdp_matrix_t* matrices, int32_t n, const fsdp_newton_schulz_t* h,
                                  void* workspace, int64_t workspace_bytes, fsdp_stream_t stream) try {
  NsPlan plan;
  if (int rc = ns_plan(h, &plan)) return rc;
  std::vector<NsJob> jobs;
  if (int rc = make_jobs(matrices, n, true, &jobs)) return rc;
  if (jobs.empty()) return FSDP_OK;
  if (!workspace) return FSDP_EINVAL;
  const int64_t need = ns_workspace_bytes(jobs, plan);
  if (workspace_bytes < need) return FSDP_EWORKSPACE;
  const Strided ws{workspace, 1, need, need, 1};
  for (const NsJob& j : jobs)
    if (ws.overlaps({j.source, j.rows, j.cols, j.source_stride, size_of_dtype(j.dtype)}) ||
        ws.overlaps({j.out, j.rows, j.cols, j.out_stride, 2}))
      return FSDP_EALIAS;
  return ns_run(jobs, plan, nullptr, nullptr, workspace, reinterpret_cast<cudaStream_t>(stream));
} catch (...) {
  return FSDP_ECUDA;
}
