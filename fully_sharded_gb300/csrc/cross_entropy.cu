// Softmax cross entropy of a projection onto a vocabulary, with its gradients
// (fsdp_cross_entropy).
//
//   x = H W^T,  lse_r = log sum_v exp(x_rv),  loss_r = lse_r - x_rt
//   dH = G W,  dW = G^T H,  G_rv = g_r (exp(x_rv - lse_r) - [v = t_r])
//
// The logits x exist only as tiles in tensor memory and registers. What is kept of a
// piece of rows is E = exp(x) in bf16, which the gradients' products read as it
// is: with S_r = exp(lse_r) and s_r = g_r / S_r,
//   dH_r = s_r sum_v E_rv W_v,   dW_v = sum_r E_rv (s_r H_r),
// so that normalising takes a factor per row (in the epilogue of the first product, in a scaled
// copy of H for the second) and no pass over E, and the targets' -1 is one element of each
// row: E_rt = S_r expm1(x_rt - lse_r). bf16's exponents hold exp(x) for |x| up to 87; a row
// with |lse| or the largest logit of some 128 columns beyond 40 (or not finite; s_r H_r then keeps 20 decades
// above bf16's smallest values for g_r) goes by the general form instead: such a span's E is kept in units of a power of
// two near its largest, and brought to units of one near S_r once that is known, which rounds nothing again.
//
// Fewer bits than fp32, each for the tensor cores' sake: E and s_r H_r are rounded to bf16 (a product's operands have one
// type, and the other ones are bf16 parameters; wider operands halve the rate and double E's bytes); sums are cut off
// at each addition in tensor memory (hence the segments); exp(x) is one instruction on a rounded x log2(e). Together with the
// results' own rounding the gradients are within 1.9e-3 to 2.3e-3 of 64 bits (1.65e-3 is that rounding alone), losses and lse
// within 4e-7 to 7e-7.
//
// Launches for each piece: the scores (product and statistics), the rows (lse, loss,
// targets, scaled H), the gradients' two products together.
#include "host_internal.h"
#include "launch.h"
#include "strided.h"
#include "tensor_core.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

namespace fsdp {
namespace {

using namespace tc;

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr float kPlainRange = 40.0f;              // of the logits of a row whose E is exp(x) itself

constexpr int kTileK = 64;
constexpr int kN = 256;                           // columns of a tile
constexpr int kSpan = 128;                        // columns of a tile that one thread holds; of one statistic
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 128 + 32 * kEpilogueWarps;  // producer, products, two idle warps, epilogue
constexpr int kBoxBytes = 32 * 128;               // what a warp sends at once: 32 rows of 128 bytes
constexpr int kOutBytes = kEpilogueWarps * 2 * kBoxBytes;
// Registers after the start: 384 threads come with 168 each.
constexpr int kLeanRegisters = 56, kEpilogueRegisters = 224;
static_assert(128 * kLeanRegisters + 32 * kEpilogueWarps * kEpilogueRegisters <= kThreads * 168, "register split");

// A tile: 128 rows per block of the pair (or single block) and 256 columns.
template <int kPair>
struct Tile {
  static constexpr int kM = 128 * kPair;
  static constexpr int kBRows = kN / kPair;  // a block's part of the second operand
  static constexpr int kABytes = 128 * kTileK * 2, kBBytes = kBRows * kTileK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = (230400 - 1024 - kOutBytes) / kStageBytes;
  static constexpr int kSmemBytes = kStages * kStageBytes + kOutBytes + 1024;
  static constexpr int kTmemCols = 2 * kN;
};

enum Result : int32_t {
  kScores,   // E and the statistics of a piece's logits
  kRows,     // bf16 rows, times a factor per row
  kPartial,  // fp32, a part of the inner dimension: joined later
  kSum,      // fp32, the first piece's; kAdd: a later piece's, added to it in memory
  kAdd,
};

// C[m, n] = sum_k A[m, k] B[n, k].
struct Product {
  CUtensorMap a, b, out;   // boxes of 64 x 64 of the operands; of the result 32 rows of 128 bytes (bf16 or fp32)
  int32_t m, n, k;
  int32_t row_tiles, col_tiles, tiles;
  int32_t splits, split_steps;  // parts of the inner dimension, and their length in steps of 64
  int32_t split_rows;      // kPartial: from one part's rows to the next's
  uint8_t a_mn, b_mn;      // the operand's row index (of C's rows, columns) is the contiguous one
  uint8_t rows_first;      // order of the tiles
  int32_t result;
  uint16_t* rows;          // kRows: where the rows go if `out` cannot describe them, else null
  int64_t rows_stride;
  const float* factor;     // kRows: of each row (null: 1)
};

struct Params {
  Product product[2];
  int32_t count, tiles;
  int32_t extra, fewer;    // see tile_of
  int32_t segment;         // steps of 64 that are summed in tensor memory
  int32_t index_bits;      // of the targets: 32 or 64
  bool keep;               // E is kept
  const void* targets;
  float2* stats;           // [row][span]: largest logit, sum of exp(x) in its unit
  int64_t spans;
  float* target_score;
  unsigned int* status;
};

__device__ __forceinline__ int64_t index_at(const void* p, int bits, int64_t i) {
  return bits == 64 ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// The unit of a span's exponentials, as a power of two: 1 where exp(x) itself can be kept.
__device__ __forceinline__ float unit_of(float most) {
  return !(fabsf(most) > kPlainRange) || most == -INFINITY ? 0.0f : rintf(most * kLog2e);
}

// 2^x to 2^-22 of itself; results below 2^-126 are zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two values at once: half the instructions.
struct Two {
  uint64_t bits;
  __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(bits) : "f"(a), "f"(b)); }
  __device__ __forceinline__ void to(float* a, float* b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(bits)); }
};
__device__ __forceinline__ Two fma_two(const Two& a, const Two& b, const Two& c) {
  Two d = a;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.bits) : "l"(a.bits), "l"(b.bits), "l"(c.bits));
  return d;
}
__device__ __forceinline__ Two add_two(const Two& a, const Two& b) {
  Two d = a;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.bits) : "l"(a.bits), "l"(b.bits));
  return d;
}
// The largest of three (a NaN among them counts for nothing).
__device__ __forceinline__ float max_of(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void shared_store(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint16_t shared_load_half(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t shared_load_word(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// bf16, bf16 -> fp32.
__device__ __forceinline__ uint32_t bf16_kind(int m, int n, bool a_mn, bool b_mn) {
  return product_kind(m, n, a_mn, b_mn) | (1u << 7) | (1u << 10);
}

// The cluster's tile number `turn`, or p.tiles behind its last. The first product's tiles, which take
// longest, go round the clusters; the `fewer` clusters that get one less than the others take `extra` rounds of
// the second product's, then those go round all clusters too.
__device__ __forceinline__ int tile_of(const Params& p, int cluster, int clusters, int turn) {
  const int first = p.product[0].tiles, more = clusters - p.fewer, own = first / clusters + (p.fewer < clusters && cluster < more && first % clusters ? 1 : 0);
  if (turn < own) return turn * clusters + cluster;
  turn -= own;
  int t;
  if (cluster >= more && turn < p.extra) {
    t = first + turn * p.fewer + cluster - more;
  } else {
    if (cluster >= more) turn -= p.extra;
    t = first + p.extra * p.fewer + turn * clusters + cluster;
  }
  return min(t, p.tiles);
}

struct Place {
  int product, split, i, j;
};

__device__ __forceinline__ Place place_of(const Params& p, int t) {
  Place q{0, 0, 0, 0};
  if (p.count > 1 && t >= p.product[0].tiles) {
    q.product = 1;
    t -= p.product[0].tiles;
  }
  const Product& g = p.product[q.product];
  const int each = g.row_tiles * g.col_tiles;
  q.split = t / each;
  t -= q.split * each;
  if (g.rows_first) {
    q.j = t / g.row_tiles;
    q.i = t - q.j * g.row_tiles;
  } else {
    q.i = t / g.col_tiles;
    q.j = t - q.i * g.col_tiles;
  }
  return q;
}

// Sends the warp's 32 rows of 128 columns (a lane's own row in value(c), as bf16), from (row0, col0) on: two boxes
// with one fence between the writes and the copies.
template <typename F>
__device__ __forceinline__ void send_rows(const Product& g, uint32_t boxes, int row0, int col0, int lane, F value) {
  if (lane == 0) bulk_wait_read<0>();  // the last boxes have left their places
  __syncwarp();
#pragma unroll
  for (int q = 0; q < kSpan / 8; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 two = __floats2bfloat162_rn(value(8 * q + 2 * k), value(8 * q + 2 * k + 1));
      w[k] = *reinterpret_cast<const uint32_t*>(&two);
    }
    shared_store(boxes + (q >> 3) * kBoxBytes + lane * 128 + (((q & 7) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
  }
  if (!g.rows) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      tma_store(&g.out, col0, row0, boxes);
      if (col0 + 64 < g.n) tma_store(&g.out, col0 + 64, row0, boxes + kBoxBytes);
      bulk_commit();
    }
    return;
  }
  // rows off 16-byte alignment: by pairs of elements at 4-byte boundaries, and single ones at the ends
  __syncwarp();
  const int rows = min(32, g.m - row0), cols = min(kSpan, g.n - col0);
  const int64_t stride = g.rows_stride;
  uint16_t* to = g.rows + row0 * stride + col0;
  constexpr int kAtOnce = 4;  // rows whose loads are in flight
  for (int r0 = 0; r0 < rows; r0 += kAtOnce) {
    uint32_t two[kAtOnce][2];
    bool odd[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int r = r0 + k;
      odd[k] = (reinterpret_cast<uintptr_t>(to + k * stride) >> 1 & 1) != 0;
      const auto at = [=](int c) {
        return boxes + (c >> 6) * kBoxBytes + r * 128 + (((c >> 3 & 7) ^ (r & 7)) << 4) + (c & 7) * 2;
      };
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // columns 64 h + 2 lane + odd, and the next one (the last lane's wraps to column 0)
        const int c = 64 * h + 2 * lane;
        two[k][h] = odd[k] ? shared_load_half(at(c + 1)) | static_cast<uint32_t>(shared_load_half(at((c + 2) % kSpan))) << 16
                           : shared_load_word(at(c));
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k, to += stride) {
      if (r0 + k >= rows) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 64 * h + 2 * lane + odd[k];
        if (c + 1 < cols)
          *reinterpret_cast<uint32_t*>(to + c) = two[k][h];
        else if (c < cols)
          to[c] = static_cast<uint16_t>(two[k][h]);
      }
      if (odd[k] && lane == 31) to[0] = static_cast<uint16_t>(two[k][1] >> 16);
    }
  }
  __syncwarp();
}

// The same in fp32, 64 columns at a time: stored, or added to what is there (each element by one block in a
// launch, and launches follow one another: the order of the additions is fixed).
__device__ __forceinline__ void send_wide(const Product& g, uint32_t boxes, int row0, int col0, int lane, const float (&x)[kSpan]) {
  const bool add = g.result == kAdd;
#pragma unroll
  for (int h = 0; h < kSpan; h += 64) {
    if (col0 + h >= g.n) break;
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 16; ++q)
      shared_store(boxes + (q >> 3) * kBoxBytes + lane * 128 + (((q & 7) ^ (lane & 7)) << 4), __float_as_uint(x[h + 4 * q]),
                   __float_as_uint(x[h + 4 * q + 1]), __float_as_uint(x[h + 4 * q + 2]), __float_as_uint(x[h + 4 * q + 3]));
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int col = col0 + h + 32 * b;
        if (col >= g.n) break;
        if (add)
          tma_add(&g.out, col, row0, boxes + b * kBoxBytes);
        else
          tma_store(&g.out, col, row0, boxes + b * kBoxBytes);
      }
      bulk_commit();
    }
  }
}

template <int kPair, bool kIsScores>
__global__ void __launch_bounds__(kThreads, 1) ce_product(const __grid_constant__ Params p) {
  using T = Tile<kPair>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full_bar[T::kStages], empty_bar[T::kStages], done_bar[2], free_bar[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int stop;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t boxes = smem + T::kStages * T::kStageBytes;
  const int rank = kPair == 2 ? static_cast<int>(block_rank()) : 0;
  const int cluster = blockIdx.x / kPair, clusters = gridDim.x / kPair;
  const Guard guard{&stop, p.status, kWaitLimitNs};
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      bar_init(smem_addr(&full_bar[s]), 1);
      bar_init(smem_addr(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(smem_addr(&done_bar[b]), 1);
      bar_init(smem_addr(&free_bar[b]), kEpilogueWarps * kPair);
    }
    stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Held while this grid waits for the previous one, which is safe: that grid's blocks have their own columns
  // before they let this one start (and so does this one, below), so none of them waits for these; with 209 KB of
  // shared memory or more no second block of such products is on the SM.
  if (warp == 1) tmem_alloc<kPair>(smem_addr(&tmem_slot), T::kTmemCols);
  fence_before();
  __syncthreads();
  if constexpr (kPair == 2) cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;");
  const auto await_inputs = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
  // steps of a tile's inner dimension, from step `from` on
  const auto inner = [](const Product& g, int split, int* from) {
    *from = split * g.split_steps;
    return min(g.split_steps, (g.k + kTileK - 1) / kTileK - *from);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLeanRegisters));
    if (warp == 0) {  // producer: this block's rows of both operands
      uint32_t it = 0;
      bool ok = true;
      for (int turn = 0, t = tile_of(p, cluster, clusters, 0); ok && t < p.tiles; t = tile_of(p, cluster, clusters, ++turn)) {
        const Place at = place_of(p, t);
        const Product& g = p.product[at.product];
        int from;
        const int steps = inner(g, at.split, &from);
        const int row0 = at.i * T::kM + rank * 128, col0 = at.j * kN + rank * T::kBRows;
        const bool a_mn = g.a_mn, b_mn = g.b_mn;
        for (int step = 0; step < steps; ++step, ++it) {
          const int s = it % T::kStages;
          ok = bar_wait_warp(smem_addr(&empty_bar[s]), ((it / T::kStages) & 1u) ^ 1u, guard);
          if (!ok) break;
          // the first block's barrier counts the bytes of both
          const uint32_t own = smem_addr(&full_bar[s]), bar = kPair == 2 ? in_block(own, 0) : own;
          const uint32_t a = smem + s * T::kStageBytes, b = a + T::kABytes;
          const int k0 = (from + step) * kTileK;
          if (it == 0) await_inputs();
          if (elect_one()) {
            if (rank == 0) bar_expect(own, T::kStageBytes * kPair);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int r = row0 + 64 * q;
              tma_box<kPair>(a + q * 8192, &g.a, a_mn ? r : k0, a_mn ? k0 : r, bar);
            }
#pragma unroll
            for (int q = 0; q < T::kBRows / 64; ++q) {
              const int c = col0 + 64 * q;
              tma_box<kPair>(b + q * 8192, &g.b, b_mn ? c : k0, b_mn ? k0 : c, bar);
            }
          }
          __syncwarp();
        }
      }
      // every copy lands (its stage is used and released) before the block ends
      for (uint32_t back = 1; back <= T::kStages && back <= it; ++back) {
        const uint32_t last = it - back;
        const uint64_t* bar = rank == 0 ? full_bar : empty_bar;
        bar_drain(smem_addr(&bar[last % T::kStages]), (last / T::kStages) & 1u, kWaitLimitNs);
      }
    } else if (warp == 1 && rank == 0) {  // products, for both blocks of a pair
      uint32_t it = 0, n = 0;             // steps; segments
      bool ok = true;
      for (int turn = 0, t = tile_of(p, cluster, clusters, 0); ok && t < p.tiles; t = tile_of(p, cluster, clusters, ++turn)) {
        const Place at = place_of(p, t);
        const Product& g = p.product[at.product];
        int from;
        const int steps = inner(g, at.split, &from);
        if (it == 0) await_inputs();  // the limit of the waits below does not run while earlier kernels do
        const uint32_t kind = bf16_kind(T::kM, kN, g.a_mn, g.b_mn);
        // bytes from one 16-deep product's operand to the next, and between blocks of 64 rows
        const uint32_t a_step = g.a_mn ? 2048 : 32, b_step = g.b_mn ? 2048 : 32;
        const uint32_t a_block = g.a_mn ? 8192 : 0, b_block = g.b_mn ? 8192 : 0;
        for (int step0 = 0; ok && step0 < steps; step0 += p.segment, ++n) {
          const uint32_t buf = n & 1u, d = tmem + buf * kN;
          ok = bar_wait_warp(smem_addr(&free_bar[buf]), ((n >> 1) & 1u) ^ 1u, guard);
          if (!ok) break;
          fence_after();
          const int count = min(p.segment, steps - step0);
          for (int step = 0; step < count; ++step, ++it) {
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
      }
      if (!ok && it > 0)  // products in flight end before the accumulators are freed
        bar_drain(smem_addr(&empty_bar[(it - 1) % T::kStages]), ((it - 1) / T::kStages) & 1u, kWaitLimitNs);
    }
  } else {  // epilogue: this block's 128 rows, 128 columns of one row in each thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegisters));
    const int own = warp - 4, quarter = own & 3, half = own >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kSpan;
    const uint32_t box = boxes + own * 2 * kBoxBytes;
    uint32_t n = 0;
    bool ok = true;
    await_inputs();
    for (int turn = 0, t = tile_of(p, cluster, clusters, 0); ok && t < p.tiles; t = tile_of(p, cluster, clusters, ++turn)) {
      const Place at = place_of(p, t);
      const Product& g = p.product[at.product];
      int from;
      const int steps = inner(g, at.split, &from);
      const int row0 = (at.i * kPair + rank) * 128 + quarter * 32, row = row0 + lane;
      const int col0 = at.j * kN + half * kSpan;
      int64_t target = -1;    // of the row, on its way during the wait; likewise its factor
      float factor = 1.0f;
      if (row < g.m) {
        if constexpr (kIsScores)
          target = index_at(p.targets, p.index_bits, row) - col0;
        else if (g.factor)
          factor = g.factor[row];
      }
      float x[kSpan];
      for (int step0 = 0; ok && step0 < steps; step0 += p.segment, ++n) {
        const uint32_t buf = n & 1u;
        ok = bar_wait_warp(smem_addr(&done_bar[buf]), (n >> 1) & 1u, guard);
        if (!ok) break;
        fence_after();
        if (step0 == 0) {
          tmem_load128(lanes + buf * kN, x);
        } else {
#pragma unroll
          for (int c = 0; c < kSpan; c += 32) {
            float v[32];
            tmem_load32(lanes + buf * kN + c, v);
#pragma unroll
            for (int q = 0; q < 32; ++q) x[c + q] += v[q];
          }
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
      if (!ok) break;
      if (row0 >= g.m || col0 >= g.n) continue;  // the same for the warp
      if constexpr (kIsScores) {
        if (col0 + kSpan > g.n)
#pragma unroll
          for (int c = 0; c < kSpan; ++c)
            if (col0 + c >= g.n) x[c] = -INFINITY;
        if (target >= 0 && target < kSpan) {
          float score = 0.0f;
#pragma unroll
          for (int c = 0; c < kSpan; ++c)  // in this form the compiler does not index x, which would move it out of registers
            asm("{\n .reg .pred p;\n setp.eq.s32 p, %1, 0;\n @p mov.f32 %0, %2;\n}\n"
                : "+f"(score)
                : "r"(static_cast<int>(target) - c), "f"(x[c]));
          p.target_score[row] = score;
        }
        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < kSpan - 4; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) top[k] = max_of(top[k], x[c + 2 * k], x[c + 2 * k + 1]);
        const float most = max_of(max_of(top[0], top[1], top[2]), max_of(top[3], x[kSpan - 4], x[kSpan - 3]),
                                  fmaxf(x[kSpan - 2], x[kSpan - 1]));
        const float unit = unit_of(most);
        const Two slope(kLog2e, kLog2e), offset(-unit, -unit);
        Two sums[2] = {Two(0.0f, 0.0f), Two(0.0f, 0.0f)};
#pragma unroll
        for (int c = 0; c < kSpan; c += 2) {
          fma_two(Two(x[c], x[c + 1]), slope, offset).to(&x[c], &x[c + 1]);
          x[c] = exp2_fast(x[c]);
          x[c + 1] = exp2_fast(x[c + 1]);
          sums[c / 2 & 1] = add_two(sums[c / 2 & 1], Two(x[c], x[c + 1]));
        }
        float sum[2];
        add_two(sums[0], sums[1]).to(&sum[0], &sum[1]);
        if (row < g.m) p.stats[row * p.spans + col0 / kSpan] = make_float2(most, sum[0] + sum[1]);
        if (!p.keep) continue;
        send_rows(g, box, row0, col0, lane, [&](int c) { return x[c]; });
      } else {
        if (g.result != kRows) {
          send_wide(g, box, at.split * g.split_rows + row0, col0, lane, x);
          continue;
        }
        if (g.factor) {
#pragma unroll
          for (int c = 0; c < kSpan; ++c) x[c] = factor == 0.0f ? 0.0f : x[c] * factor;
        }
        send_rows(g, box, row0, col0, lane, [&](int c) { return x[c]; });
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

// ------------------------------------------------------------------ the rows

constexpr int kRowThreads = 128;  // of a block: for one row, or for four

struct RowParams {
  const float2* stats;
  int64_t spans;
  const float* target_score;
  const void* targets;
  int32_t index_bits, rows, cols, vocab;
  bool keep;
  float scale;
  const float* dloss;
  float *loss, *lse;
  float* factor;           // s_r
  uint16_t* e;
  int64_t e_stride;
  const uint16_t* hidden;  // rows at 16-byte boundaries, as the scores read them
  int64_t hidden_stride;
  uint16_t* scaled;        // s_r H_r
  int64_t scaled_stride;
};

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// From one power of two to another, as far as a float's exponents go (a NaN counts as very small).
__device__ __forceinline__ int between(float from, float to) {
  return static_cast<int>(fminf(fmaxf(from - to, -300.0f), 300.0f));
}

// Over the threads of a row (the block, or a warp of it), the same for all of them.
template <int kLanes, typename F>
__device__ __forceinline__ float row_reduce(float v, float* shared, F f) {
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (kLanes == 32) return v;
  __syncthreads();  // the last use of `shared`
  if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = v;
  __syncthreads();
  v = shared[0];
#pragma unroll
  for (int w = 1; w < kRowThreads / 32; ++w) v = f(v, shared[w]);
  return v;
}

// A row of the piece by kLanes threads: its lse and loss from the spans' statistics; for the
// gradients its factor, its target's element of E and its scaled row of H. Bound by HBM for many rows, a warp each
// (8192 x 768, vocabulary 50257: 11 us; by blocks 21), by its chain of loads for few, a block each (61 x 4096,
// 32000: 8 us; by warps 13).
template <int kLanes>
__global__ void __launch_bounds__(kRowThreads) ce_rows(const __grid_constant__ RowParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float shared[kRowThreads / 32];
  const int tid = threadIdx.x % kLanes;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRowThreads / kLanes) + threadIdx.x / kLanes;
  if (row >= p.rows) return;  // a whole warp, or a whole block
  const auto add = [](float a, float b) { return a + b; };
  const auto larger = [](float a, float b) { return fmaxf(a, b); };
  const float2* stats = p.stats + row * p.spans;
  const int64_t target = index_at(p.targets, p.index_bits, row);
  const bool there = target >= 0, has = there && target < p.vocab;
  const float score = has ? p.target_score[row] : NAN;
  const float g = there ? (has ? p.scale * (p.dloss ? p.dloss[row] : 1.0f) : NAN) : 0.0f;
  float most = -INFINITY, far = 0.0f, sum = 0.0f;
  for (int64_t i = tid; i < p.spans; i += kLanes) {
    const float2 s = stats[i];
    most = fmaxf(most, s.x);
    far = fmaxf(far, fabsf(s.x));
    sum += s.y;
  }
  far = row_reduce<kLanes>(far, shared, larger);
  float unit = 0.0f;  // of the sum
  if (!(far > kPlainRange)) {
    sum = row_reduce<kLanes>(sum, shared, add);
  } else {
    unit = unit_of(row_reduce<kLanes>(most, shared, larger));
    sum = 0.0f;
    for (int64_t i = tid; i < p.spans; i += kLanes) {
      const float2 s = stats[i];
      sum += ldexpf(s.y, between(unit_of(s.x), unit));
    }
    sum = row_reduce<kLanes>(sum, shared, add);
  }
  const float log_sum = logf(sum), lse = fmaf(unit, kLn2, log_sum);
  // x_t - lse, in the sum's unit if it has one. A confident row's lse may round to less than its target's logit: its
  // loss is then 0, and p - 1 not above 0.
  float behind = (unit == 0.0f ? score : fmaf(score, kLog2e, -unit) * kLn2) - log_sum;
  if (behind > 0.0f) behind = 0.0f;
  if (tid == 0) {
    p.loss[row] = there ? 0.0f - behind : 0.0f;
    if (p.lse) p.lse[row] = lse;
  }
  if (!p.keep) return;
  uint16_t* e = p.e + row * p.e_stride;
  const bool plain = !(far > kPlainRange) && fabsf(lse) <= kPlainRange;
  if (!plain && sum > 0.0f && sum < INFINITY) {  // E in a unit near the sum
    const int more = ilogbf(sum);
    unit += static_cast<float>(more);
    sum = ldexpf(sum, -more);
  }
  // The target's element is the largest of the row's: its rounding to bf16 goes into the row's factor
  // (relative to which the others, rounded too, are then off by one more rounding).
  const float exact = has ? sum * expm1f(behind) : 0.0f;
  const uint16_t rounded = bf16_bits(exact);
  float factor = g == 0.0f ? 0.0f : g / sum;
  if (bf16_value(rounded) != 0.0f) factor *= exact / bf16_value(rounded);
  if (plain) {
    if (tid == 0 && has) e[target] = rounded;
  } else {
    for (int64_t v = tid * 8; v < p.vocab; v += kLanes * 8) {  // whole vectors: E's rows are whole lines
      const int by = between(unit_of(stats[v / kSpan].x), unit);
      const bool own = has && target >= v && target < v + 8;
      if (there && by == 0 && !own) continue;
      uint4* at = reinterpret_cast<uint4*>(e + v);
      const uint4 kept = *at;
      const uint32_t in[4] = {kept.x, kept.y, kept.z, kept.w};
      uint32_t out[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t two[2] = {in[k] & 0xffffu, in[k] >> 16};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          two[h] = there ? bf16_bits(ldexpf(bf16_value(static_cast<uint16_t>(two[h])), by)) : 0u;
          if (own && target == v + 2 * k + h) two[h] = rounded;
        }
        out[k] = two[0] | two[1] << 16;
      }
      *at = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
  if (tid == 0) p.factor[row] = factor;
  const uint16_t* h = p.hidden + row * p.hidden_stride;
  uint16_t* scaled = p.scaled + row * p.scaled_stride;
  for (int c = tid * 8; c < p.cols; c += kLanes * 8) {  // what lies behind the row's end is not used
    const uint4 v = *reinterpret_cast<const uint4*>(h + c);
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 two = __floats2bfloat162_rn(__uint_as_float(in[k] << 16) * factor, __uint_as_float(in[k] & 0xffff0000u) * factor);
      out[k] = factor == 0.0f ? 0u : *reinterpret_cast<const uint32_t*>(&two);
    }
    *reinterpret_cast<uint4*>(scaled + c) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// ------------------------------------------------- copies and joined results

struct CopyParams {
  const uint16_t* from;
  int64_t from_stride;
  uint16_t* to;
  int64_t to_stride;
  int64_t rows, cols;
};

// Eight two-byte elements from byte `off` (even) of two vectors on.
__device__ __forceinline__ uint4 eight_from(const uint4& a, const uint4& b, uint32_t off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 8)
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  if (off & 4)
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  if (off & 2)
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows off 16-byte alignment into rows that tensor maps can describe, 8 elements a thread: the (one or two)
// aligned vectors that hold them, shifted. Bound by HBM (65536 x 1795: 70 us, 6.7 TB/s).
__global__ void __launch_bounds__(256) ce_copy(const __grid_constant__ CopyParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t per_row = static_cast<uint32_t>((p.cols + 7) / 8);
  const int64_t vectors = p.rows * per_row;
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; v < vectors; v += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = vectors >> 31 ? v / per_row : static_cast<uint32_t>(v) / per_row, c = (v - r * per_row) * 8;
    const uintptr_t row = reinterpret_cast<uintptr_t>(p.from + r * p.from_stride), from = row + 2 * c, end = row + 2 * p.cols;
    const uintptr_t base = from & ~uintptr_t(15);
    const uint32_t off = static_cast<uint32_t>(from & 15);
    const uint4 a = *reinterpret_cast<const uint4*>(base);
    uint4 b = make_uint4(0, 0, 0, 0);
    if (off && base + 16 < end) b = *reinterpret_cast<const uint4*>(base + 16);
    *reinterpret_cast<uint4*>(p.to + r * p.to_stride + c) = eight_from(a, b, off);
  }
}

// The other way: rows at 16-byte boundaries to where they belong, an aligned vector of the result a thread,
// single elements at the rows' ends.
__global__ void __launch_bounds__(256) ce_place(const __grid_constant__ CopyParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t per_row = static_cast<uint32_t>((p.cols + 14) / 8);
  const int64_t vectors = p.rows * per_row;
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; v < vectors; v += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = vectors >> 31 ? v / per_row : static_cast<uint32_t>(v) / per_row;
    uint16_t* to = p.to + r * p.to_stride;
    const int64_t c = (v - r * per_row) * 8 - static_cast<int64_t>(reinterpret_cast<uintptr_t>(to) >> 1 & 7);  // the vector's first column
    if (c >= p.cols) continue;
    const int64_t first = c >= 0 ? c / 8 : -1;  // the row's vector that holds it
    const uint32_t off = static_cast<uint32_t>(c - 8 * first) * 2;
    const uint4* from = reinterpret_cast<const uint4*>(p.from + r * p.from_stride);
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (first >= 0) a = from[first];
    if (off && 8 * (first + 1) < p.cols) b = from[first + 1];
    const uint4 w = eight_from(a, b, off);
    if (c >= 0 && c + 8 <= p.cols) {
      *reinterpret_cast<uint4*>(to + c) = w;
    } else {
      const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e >= 0 && c + e < p.cols) to[c + e] = static_cast<uint16_t>(words[e / 2] >> (e & 1) * 16);
    }
  }
}

struct JoinParams {
  const float* wide;
  int64_t wide_stride, split_rows;
  int32_t splits;
  int64_t rows, cols;
  const float* factor;
  uint16_t* out;
  int64_t out_stride;
};

// The sum of a product's parts, times the row's factor: eight groups of threads each a share of the
// parts, then the groups in order.
constexpr int kJoinGroups = 8;

__global__ void __launch_bounds__(32 * kJoinGroups) ce_join(const __grid_constant__ JoinParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float4 sums[kJoinGroups][32];
  const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
  const int64_t per_row = (p.cols + 127) / 128;
  const int64_t row = blockIdx.x / per_row, col = ((blockIdx.x - row * per_row) * 32 + lane) * 4;
  const int each = (p.splits + kJoinGroups - 1) / kJoinGroups;
  const int from = min(p.splits, group * each), to = min(p.splits, from + each);
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const auto add = [&](const float4& v) { sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w; };
  if (col < p.cols)  // the parts' rows are whole groups of 8
#pragma unroll 4
    for (int s = from; s < to; ++s) add(*reinterpret_cast<const float4*>(p.wide + (s * p.split_rows + row) * p.wide_stride + col));
  sums[group][lane] = sum;
  const float factor = p.factor[row];
  __syncthreads();
  if (group != 0 || col >= p.cols) return;
#pragma unroll
  for (int g = 1; g < kJoinGroups; ++g) add(sums[g][lane]);
  const float v[4] = {sum.x, sum.y, sum.z, sum.w};
  uint16_t* out = p.out + row * p.out_stride + col;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (col + e < p.cols) out[e] = bf16_bits(factor == 0.0f ? 0.0f : v[e] * factor);
}

struct RoundParams {
  const float* sum;
  int64_t sum_stride;
  uint16_t* out;
  int64_t out_stride;
  int64_t rows, cols;
};

// The sum over the pieces, rounded: 8 elements a thread at 16-byte boundaries, else one. Bound by HBM.
template <int kVec>
__global__ void __launch_bounds__(256) ce_round(const __grid_constant__ RoundParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t per_row = static_cast<uint32_t>((p.cols + kVec - 1) / kVec);
  const int64_t groups = p.rows * per_row;
#pragma unroll 2
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; v < groups; v += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = groups >> 31 ? v / per_row : static_cast<uint32_t>(v) / per_row, c = (v - r * per_row) * kVec;
    const float* from = p.sum + r * p.sum_stride + c;
    uint16_t* to = p.out + r * p.out_stride + c;
    if constexpr (kVec == 8) {
      const float4 a = *reinterpret_cast<const float4*>(from), b = *reinterpret_cast<const float4*>(from + 4);
      const __nv_bfloat162 two[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w), __floats2bfloat162_rn(b.x, b.y),
                                     __floats2bfloat162_rn(b.z, b.w)};
      *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(two);
    } else {
      *to = bf16_bits(*from);
    }
  }
}

// ---------------------------------------------------------------------- host

constexpr int64_t kMaxCols = int64_t(1) << 24, kMaxVocab = int64_t(1) << 30, kMaxRows = int64_t(1) << 40;
constexpr int64_t kPieceBytes = int64_t(1) << 30;  // of E
constexpr int64_t kMaxPiece = 1 << 20;

int64_t round_to(int64_t n, int64_t k) { return (n + k - 1) / k * k; }

// The sizes of a call and its workspace.
struct Plan {
  int64_t piece, pieces;   // rows of a piece
  int64_t spans, e_stride, h_stride;
  int pair, splits, split_steps;
  int64_t stats, target_score, factor, e, scaled, hidden, weight, sum, aside, partial, bytes;  // offsets (0: not there)
};

int make_plan(const fsdp_cross_entropy_t& a, bool gradients, Plan* out) {
  if (a.rows < 0 || a.rows > kMaxRows || a.cols < 1 || a.cols > kMaxCols || a.vocab < 1 || a.vocab > kMaxVocab ||
      a.piece < 0)
    return FSDP_EINVAL;
  Plan p{};
  p.spans = (a.vocab + kSpan - 1) / kSpan;
  p.e_stride = round_to(a.vocab, 64);
  p.h_stride = round_to(a.cols, 64);  // whole lines: a box's row of 128 bytes is then one
  int64_t piece = a.piece;
  if (!piece) piece = std::max<int64_t>(256, kPieceBytes / (p.e_stride * 2) / 256 * 256);
  p.piece = std::max<int64_t>(1, std::min({piece, a.rows, kMaxPiece}));
  p.pieces = (a.rows + p.piece - 1) / p.piece;
  p.pair = p.piece <= 128 ? 1 : 2;
  const int clusters = 152 / p.pair;
  const int64_t tiles = ((p.piece + 128 * p.pair - 1) / (128 * p.pair)) * ((a.cols + kN - 1) / kN);
  const int64_t steps = (a.vocab + kTileK - 1) / kTileK;
  // Few tiles are cut along the vocabulary where that saves more than the launch that joins them (3 us) costs:
  // a step takes about 0.3 us.
  p.splits = static_cast<int>(std::max<int64_t>(1, std::min(clusters / tiles, steps / 8)));
  if (steps < 24) p.splits = 1;
  p.split_steps = static_cast<int>((steps + p.splits - 1) / p.splits);
  p.splits = static_cast<int>((steps + p.split_steps - 1) / p.split_steps);
  int64_t at = 256;  // the caller's pointer may have any alignment
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_to(bytes, 256);
    return here;
  };
  p.stats = take(p.piece * p.spans * 8);
  p.target_score = take(p.piece * 4);
  p.hidden = take(p.piece * p.h_stride * 2);
  p.weight = take(a.vocab * p.h_stride * 2);
  if (gradients) {
    p.factor = take(p.piece * 4);
    p.e = take(p.piece * p.e_stride * 2);
    p.scaled = take(p.piece * p.h_stride * 2);
    if (p.pieces > 1)
      p.sum = take(a.vocab * p.h_stride * 4);
    else if (a.cols % 8 != 0 && a.rows <= 2048)  // see run()
      p.aside = take(a.vocab * p.h_stride * 2);
    if (p.splits > 1) p.partial = take(p.splits * round_to(p.piece, 256) * p.h_stride * 4);
  }
  p.bytes = at;
  *out = p;
  return FSDP_OK;
}

// Whether a tensor map can describe these bf16 rows (its strides are below 2^40 bytes).
bool mappable(const void* p, int64_t rows, int64_t stride) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows < 2 || (stride % 8 == 0 && stride < (int64_t(1) << 39)));
}

// Whether tiled stores can write them: whole vectors of 16 bytes, for a store fills a row's last one up.
bool storable(const void* p, int64_t rows, int64_t cols, int64_t stride) { return cols % 8 == 0 && mappable(p, rows, stride); }

bool f32_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t stride) {
  return make_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, rows, cols, stride, 32);
}

bool bf16_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t stride, int box_rows) {
  if (rows < 2) stride = round_to(cols, 8);  // not used
  return make_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, rows, cols, stride, box_rows);
}

// How many clusters of the kernel run at once (looked up once per device).
template <int kPair, bool kIsScores>
int resident_clusters(const Device& dev) {
  using T = Tile<kPair>;
  static std::atomic<int> cached[64];
  if (dev.id >= 64) return 0;
  int n = cached[dev.id].load(std::memory_order_acquire);
  if (n) return n;
  const auto kernel = ce_product<kPair, kIsScores>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmemBytes) != cudaSuccess) return 0;
  if (kPair == 1) {
    n = dev.sms;
  } else {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(dev.sms / kPair * kPair);
    cfg.blockDim = dim3(kThreads);
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

template <int kPair, bool kIsScores>
int launch_products(Params& p, const Device& dev, cudaStream_t stream) {
  using T = Tile<kPair>;
  p.tiles = 0;
  for (int i = 0; i < p.count; ++i) {
    Product& g = p.product[i];
    g.row_tiles = (g.m + T::kM - 1) / T::kM;
    g.col_tiles = (g.n + kN - 1) / kN;
    g.tiles = g.row_tiles * g.col_tiles * g.splits;
    p.tiles += g.tiles;
  }
  const int room = resident_clusters<kPair, kIsScores>(dev);
  if (room < 1) return FSDP_ECUDA;
  const int clusters = std::min(p.tiles, room);
  p.fewer = p.extra = 0;
  if (p.count == 2 && p.product[0].tiles % clusters) {
    p.fewer = clusters - p.product[0].tiles % clusters;
    // As many as take as long as one of the first product's: a tile takes its steps or, with few, its epilogue and
    // store, about as long as 6 steps (61 x 4096, vocabulary 32000: by the steps alone a few SMs had most of the
    // one-step tiles, the launch took 130 us, now 75).
    p.extra = (2 * p.product[0].split_steps / std::max(6, p.product[1].split_steps) + 1) / 2;
  }
  return launch_after(ce_product<kPair, kIsScores>, clusters * kPair, kPair, kThreads, T::kSmemBytes, stream, p);
}

int steps_of(int64_t k) { return static_cast<int>((k + kTileK - 1) / kTileK); }

int copy_rows(const uint16_t* from, int64_t from_stride, uint16_t* to, int64_t to_stride, int64_t rows, int64_t cols,
              cudaStream_t st) {
  const CopyParams p{from, from_stride, to, to_stride, rows, cols};
  return launch_after(ce_copy, static_cast<int>(std::min<int64_t>((rows * ((cols + 7) / 8) + 255) / 256, 152 * 8)), 1, 256, 0, st, p);
}

struct Call {
  const uint16_t *hidden, *weight;
  const void* targets;
  const float* dloss;
  float *loss, *lse;
  uint16_t *dhidden, *dweight;
};

int run(const fsdp_cross_entropy_t& a, const Plan& plan, const Call& c, void* workspace, cudaStream_t st) {
  Device dev;
  if (int rc = device_facts(&dev)) return rc;
  if (!encoder()) return FSDP_ECUDA;
  auto* base = reinterpret_cast<unsigned char*>(round_to(reinterpret_cast<intptr_t>(workspace), 256) - 256);
  const auto at = [&](int64_t offset) { return base + offset; };
  const bool gradients = c.dhidden != nullptr;
  const int index_bytes = a.target_dtype == FSDP_DTYPE_I64 ? 8 : 4;
  const uint16_t* weight = c.weight;
  int64_t weight_stride = a.weight_stride;
  if (!mappable(weight, a.vocab, weight_stride)) {
    auto* copy = reinterpret_cast<uint16_t*>(at(plan.weight));
    if (int rc = copy_rows(weight, weight_stride, copy, plan.h_stride, a.vocab, a.cols, st)) return rc;
    weight = copy;
    weight_stride = plan.h_stride;
  }
  Params scores{}, products{};
  RowParams rows{};
  scores.count = 1;
  // The logits' sums are cut off at each addition, so segments are added in registers: of 1024 columns, 256 for few
  // rows, whose losses are not averaged over many and which are bound by reading the weight. (The losses of 4096 rows are
  // within 7e-7 of 64 bits, of 4 within 3e-6 by segments of 1024 and 1e-6 of 256; with 256 the Llama head would take 1958 us
  // for 1871, GPT-2's 1256 for 1111.)
  scores.segment = plan.pair == 1 ? 4 : 16;
  products.segment = 64;
  scores.status = products.status = dev.status;
  scores.index_bits = rows.index_bits = 8 * index_bytes;
  scores.keep = rows.keep = gradients;
  scores.stats = reinterpret_cast<float2*>(at(plan.stats));
  rows.stats = scores.stats;
  scores.spans = rows.spans = plan.spans;
  scores.target_score = reinterpret_cast<float*>(at(plan.target_score));
  rows.target_score = scores.target_score;
  rows.cols = static_cast<int32_t>(a.cols);
  rows.vocab = static_cast<int32_t>(a.vocab);
  rows.scale = static_cast<float>(a.scale);
  auto* sum = reinterpret_cast<float*>(at(plan.sum));  // several pieces: dweight's
  // Few rows: dweight's rows off 16-byte boundaries go there by a pass of their own (73 x 1795, 65536 348 us; stored by
  // the products in words 403; 1123 x 741, 43094 237 and 243), where odd widths make that certain enough for the workspace
  // to have room. With many the products hide their stores (4000 x 769, 50257: 752 and 725).
  auto* aside = plan.aside ? reinterpret_cast<uint16_t*>(at(plan.aside)) : nullptr;
  bool put_aside = false;
  if (gradients) {
    rows.factor = reinterpret_cast<float*>(at(plan.factor));
    rows.e = reinterpret_cast<uint16_t*>(at(plan.e));
    rows.e_stride = plan.e_stride;
    rows.scaled = reinterpret_cast<uint16_t*>(at(plan.scaled));
    rows.scaled_stride = plan.h_stride;
  }

  for (int64_t r0 = 0; r0 < a.rows; r0 += plan.piece) {
    const int64_t n = std::min(plan.piece, a.rows - r0);
    const uint16_t* hidden = c.hidden + r0 * a.hidden_stride;
    int64_t hidden_stride = a.hidden_stride;
    if (!mappable(hidden, n, hidden_stride)) {
      auto* copy = reinterpret_cast<uint16_t*>(at(plan.hidden));
      if (int rc = copy_rows(hidden, hidden_stride, copy, plan.h_stride, n, a.cols, st)) return rc;
      hidden = copy;
      hidden_stride = plan.h_stride;
    }
    rows.hidden = hidden;
    rows.hidden_stride = hidden_stride;
    scores.targets = static_cast<const unsigned char*>(c.targets) + r0 * index_bytes;
    rows.targets = scores.targets;
    rows.rows = static_cast<int32_t>(n);
    rows.dloss = c.dloss ? c.dloss + r0 : nullptr;
    rows.loss = c.loss + r0;
    rows.lse = c.lse ? c.lse + r0 : nullptr;

    Product& s = scores.product[0];
    s = Product{};
    s.m = static_cast<int32_t>(n);
    s.n = static_cast<int32_t>(a.vocab);
    s.k = static_cast<int32_t>(a.cols);
    s.splits = 1;
    s.split_steps = steps_of(s.k);
    s.rows_first = 1;
    s.result = kScores;
    bool ok = bf16_map(&s.a, hidden, n, a.cols, hidden_stride, 64) && bf16_map(&s.b, weight, a.vocab, a.cols, weight_stride, 64);
    if (gradients) ok = ok && bf16_map(&s.out, rows.e, n, a.vocab, plan.e_stride, 32);
    if (!ok) return FSDP_ECUDA;
    if (int rc = plan.pair == 2 ? launch_products<2, true>(scores, dev, st) : launch_products<1, true>(scores, dev, st))
      return rc;
    const bool many = n >= 2048;
    const int row_blocks = static_cast<int>(many ? (n + kRowThreads / 32 - 1) / (kRowThreads / 32) : n);
    if (int rc = launch_after(many ? ce_rows<32> : ce_rows<kRowThreads>, row_blocks, 1, kRowThreads, 0, st, rows)) return rc;
    if (!gradients) continue;

    products.count = 2;
    uint16_t* dhidden = c.dhidden + r0 * a.dhidden_stride;
    Product& dh = products.product[0];
    dh = Product{};
    dh.m = s.m;
    dh.n = s.k;
    dh.k = s.n;
    dh.b_mn = 1;
    dh.splits = plan.splits;
    dh.split_steps = plan.split_steps;
    dh.factor = rows.factor;
    auto* partial = reinterpret_cast<float*>(at(plan.partial));
    ok = bf16_map(&dh.a, rows.e, n, a.vocab, plan.e_stride, 64);
    dh.b = s.b;
    if (plan.splits > 1) {
      dh.result = kPartial;
      dh.split_rows = static_cast<int32_t>(round_to(n, 256));
      ok = ok && f32_map(&dh.out, partial, plan.splits * static_cast<int64_t>(dh.split_rows), a.cols, plan.h_stride);
    } else {
      dh.result = kRows;
      if (storable(dhidden, n, a.cols, a.dhidden_stride)) {
        ok = ok && bf16_map(&dh.out, dhidden, n, a.cols, a.dhidden_stride, 32);
      } else {
        dh.rows = dhidden;
        dh.rows_stride = a.dhidden_stride;
      }
    }
    Product& dw = products.product[1];
    dw = Product{};
    dw.m = s.n;
    dw.n = s.k;
    dw.k = s.m;
    dw.a_mn = dw.b_mn = 1;
    dw.splits = 1;
    dw.split_steps = steps_of(n);
    dw.a = dh.a;
    ok = ok && bf16_map(&dw.b, rows.scaled, n, a.cols, plan.h_stride, 64);
    if (plan.pieces > 1) {
      dw.result = r0 == 0 ? kSum : kAdd;
      ok = ok && f32_map(&dw.out, sum, a.vocab, a.cols, plan.h_stride);
    } else {
      dw.result = kRows;
      if (storable(c.dweight, a.vocab, a.cols, a.dweight_stride)) {
        ok = ok && bf16_map(&dw.out, c.dweight, a.vocab, a.cols, a.dweight_stride, 32);
      } else if (aside) {
        ok = ok && bf16_map(&dw.out, aside, a.vocab, a.cols, plan.h_stride, 32);
        put_aside = true;
      } else {
        dw.rows = c.dweight;
        dw.rows_stride = a.dweight_stride;
      }
    }
    if (!ok) return FSDP_ECUDA;
    if (int rc = plan.pair == 2 ? launch_products<2, false>(products, dev, st) : launch_products<1, false>(products, dev, st))
      return rc;
    if (plan.splits > 1) {
      const JoinParams j{partial, plan.h_stride, dh.split_rows, dh.splits, n, a.cols, rows.factor, dhidden, a.dhidden_stride};
      const int64_t blocks = n * ((a.cols + 127) / 128);  // few: a product is cut only where its result has few tiles
      if (int rc = launch_after(ce_join, static_cast<int>(blocks), 1, 32 * kJoinGroups, 0, st, j)) return rc;
    }
  }
  if (put_aside) {
    const CopyParams p{aside, plan.h_stride, c.dweight, a.dweight_stride, a.vocab, a.cols};
    const int64_t blocks = (a.vocab * ((a.cols + 14) / 8) + 255) / 256;
    return launch_after(ce_place, static_cast<int>(std::min<int64_t>(blocks, 152 * 8)), 1, 256, 0, st, p);
  }
  if (gradients && plan.pieces > 1) {
    const RoundParams p{sum, plan.h_stride, c.dweight, a.dweight_stride, a.vocab, a.cols};
    const bool vectors = storable(c.dweight, a.vocab, a.cols, a.dweight_stride);
    const int64_t groups = a.vocab * (vectors ? a.cols / 8 : a.cols);
    const int grid = static_cast<int>(std::min<int64_t>((groups + 255) / 256, 152 * 8));
    return launch_after(vectors ? ce_round<8> : ce_round<1>, grid, 1, 256, 0, st, p);
  }
  return FSDP_OK;
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" int fsdp_cross_entropy_workspace(const fsdp_cross_entropy_t* a, int32_t gradients, int64_t* bytes_out) {
  if (!a || !bytes_out) return FSDP_EINVAL;
  Plan plan;
  if (int rc = make_plan(*a, gradients != 0, &plan)) return rc;
  *bytes_out = plan.bytes;
  return FSDP_OK;
}

extern "C" int fsdp_cross_entropy(const fsdp_cross_entropy_t* a, const uint16_t* hidden, const uint16_t* weight,
                                  const void* targets, const float* dloss, float* loss, float* lse, uint16_t* dhidden,
                                  uint16_t* dweight, void* workspace, int64_t workspace_bytes, fsdp_stream_t stream) {
  if (!a || (a->rows > 0 && !dhidden != !dweight)) return FSDP_EINVAL;
  if (a->target_dtype != FSDP_DTYPE_I32 && a->target_dtype != FSDP_DTYPE_I64) return FSDP_EINVAL;
  const bool gradients = dweight != nullptr;  // an empty dhidden may have no address
  if (gradients ? !std::isfinite(static_cast<float>(a->scale)) : dloss != nullptr) return FSDP_EINVAL;
  Plan plan;
  if (int rc = make_plan(*a, gradients, &plan)) return rc;
  const int is = a->target_dtype == FSDP_DTYPE_I64 ? 8 : 4;
  const Strided sh{hidden, a->rows, a->cols, a->hidden_stride, 2}, sw{weight, a->vocab, a->cols, a->weight_stride, 2},
      st{targets, 1, a->rows, a->rows, is}, sg{dloss, 1, a->rows, a->rows, 4}, sl{loss, 1, a->rows, a->rows, 4},
      se{lse, 1, a->rows, a->rows, 4}, sdh{dhidden, a->rows, a->cols, a->dhidden_stride, 2},
      sdw{dweight, a->vocab, a->cols, a->dweight_stride, 2}, ws{workspace, 1, plan.bytes, plan.bytes, 1};
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (gradients && !sdw.ok()) return FSDP_EINVAL;
  if (a->rows == 0) {  // no rows: only the weight's gradient, zero
    if (!gradients) return FSDP_OK;
    return cudaMemset2DAsync(dweight, static_cast<size_t>(sdw.pitch() ? sdw.pitch() : a->cols * 2), 0,
                             static_cast<size_t>(a->cols) * 2, static_cast<size_t>(a->vocab), cs) == cudaSuccess
               ? FSDP_OK
               : FSDP_ECUDA;
  }
  if (!sh.ok() || !sw.ok() || !st.ok() || !sl.ok() || !ws.ok() || (dloss && !sg.ok()) || (lse && !se.ok()) ||
      (gradients && !sdh.ok()))
    return FSDP_EINVAL;
  if (workspace_bytes < plan.bytes) return FSDP_EWORKSPACE;
  const Strided* in[] = {&sh, &sw, &st, dloss ? &sg : nullptr};
  const Strided* out[] = {&sl, lse ? &se : nullptr, gradients ? &sdh : nullptr, gradients ? &sdw : nullptr, &ws};
  for (const Strided* o : out) {
    if (!o) continue;
    for (const Strided* q : out)
      if (q && q != o && o->overlaps(*q)) return FSDP_EALIAS;
    for (const Strided* i : in)
      if (i && o->overlaps(*i) && !(o == &sdh && i == &sh && o->same_place(*i))) return FSDP_EALIAS;
  }
  return run(*a, plan, Call{hidden, weight, targets, dloss, loss, lse, dhidden, dweight}, workspace, cs);
}
