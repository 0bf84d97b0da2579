// Dropout from a counter-based generator, with the residual's addition
// (fsdp_dropout). Its gradient is the same call on the gradient, without a residual.
//
// Element i of the matrix (row cols + column, whatever the strides) has draw i mod 8 of
// counter i / 8: Philox4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011), key = seed, counter = (i / 8, offset), whose four words are
// eight draws of 16 bits, the low half first. It stays where its draw is at least
// threshold = round(65536 p), times 65536 / (65536 - threshold): no mask is stored,
// and the mean is kept exactly although p is rounded to 16 bits.
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

struct DropoutParams {
  const void* x;
  const void* residual;
  void* out;
  int64_t rows, cols, x_stride, residual_stride, out_stride;
  uint64_t seed, offset;
  const uint64_t* counter;  // device: added to the offset (null: 0)
  uint32_t threshold;
  float scale;
};

constexpr int kThreads = 256;

// Eight draws of 16 bits, packed by two.
__device__ __forceinline__ uint4 philox(uint64_t at, uint64_t offset, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(at), c1 = static_cast<uint32_t>(at >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0, p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(p1);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ void unpack_bf16(uint32_t two, float* v) {
  v[0] = __uint_as_float(two << 16);
  v[1] = __uint_as_float(two & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&two);
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  unpack_bf16(a.x, v), unpack_bf16(a.y, v + 2), unpack_bf16(a.z, v + 4), unpack_bf16(a.w, v + 6);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float value_of(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float value_of(float v) { return v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

__device__ __forceinline__ uint32_t draw_of(const uint4& w, int e) {
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  return e & 1 ? words[e / 2] >> 16 : words[e / 2] & 0xffffu;
}

// Group g (of 8 consecutive elements), one element after another.
template <typename T>
__device__ __forceinline__ void drop_singly(const DropoutParams& p, int64_t g, uint64_t offset) {
  const T* x = static_cast<const T*>(p.x);
  const T* residual = static_cast<const T*>(p.residual);
  T* out = static_cast<T*>(p.out);
  const int64_t n = p.rows * p.cols;
  const uint4 w = philox(static_cast<uint64_t>(g), offset, p.seed);
  int64_t row = p.rows > 1 ? g * 8 / p.cols : 0, col = g * 8 - row * p.cols;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (g * 8 + e >= n) break;
    float v = draw_of(w, e) >= p.threshold ? value_of(x[row * p.x_stride + col]) * p.scale : 0.0f;
    if (residual) v += value_of(residual[row * p.residual_stride + col]);
    put(out + row * p.out_stride + col, v);
    if (++col == p.cols) col = 0, ++row;
  }
}

// kVector: every group of 8 elements lies in one row, at 16-byte boundaries (the last one of one long row may be
// short). Bound by HBM there: 16384 x 4096 bf16 with the residual 60 us, 6.7 TB/s (without it 54 us; rows 4104
// apart 61); ten rounds for 8 elements are a third of the instructions that the memory leaves room for. Else
// one element after another, bound by their loads and stores: the same matrix 2 bytes off a boundary 168 us.
template <typename T, bool kVector>
__global__ void __launch_bounds__(kThreads) dropout_rows(const __grid_constant__ DropoutParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint64_t offset = p.offset + (p.counter ? *p.counter : 0);
  const int64_t n = p.rows * p.cols, groups = kVector ? n / 8 : (n + 7) / 8;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, step = static_cast<int64_t>(gridDim.x) * kThreads;
  if (kVector && first == 0 && n % 8) drop_singly<T>(p, groups, offset);
  const T* x = static_cast<const T*>(p.x);
  const T* residual = static_cast<const T*>(p.residual);
  T* out = static_cast<T*>(p.out);
  for (int64_t g = first; g < groups; g += step) {
    if constexpr (kVector) {
      const uint4 w = philox(static_cast<uint64_t>(g), offset, p.seed);
      const int64_t row = p.rows > 1 ? g * 8 / p.cols : 0, col = g * 8 - row * p.cols;
      float v[8], r[8] = {};
      load8(x + row * p.x_stride + col, v);
      if (residual) load8(residual + row * p.residual_stride + col, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (draw_of(w, e) >= p.threshold ? v[e] * p.scale : 0.0f) + r[e];
      store8(out + row * p.out_stride + col, v);
    } else {
      drop_singly<T>(p, g, offset);
    }
  }
}

constexpr int64_t kMaxSide = int64_t(1) << 40;

template <typename T>
int run(const DropoutParams& p, bool vectors, cudaStream_t st) {
  const int64_t blocks = ((p.rows * p.cols + 7) / 8 + kThreads - 1) / kThreads;
  return launch_after(vectors ? dropout_rows<T, true> : dropout_rows<T, false>,
                      static_cast<int>(std::min<int64_t>(blocks, 152 * 8 * 4)), 1, kThreads, 0, st, p);
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" int fsdp_dropout(const fsdp_dropout_t* a, const void* x, const void* residual, const uint64_t* counter,
                            void* out, fsdp_stream_t stream) {
  if (!a || a->rows < 0 || a->cols < 1 || a->rows > kMaxSide || a->cols > kMaxSide) return FSDP_EINVAL;
  if (a->rows > 0 && a->cols > (int64_t(1) << 60) / a->rows) return FSDP_EINVAL;
  if (a->dtype != FSDP_DTYPE_F32 && a->dtype != FSDP_DTYPE_BF16) return FSDP_EINVAL;
  if (!(a->p >= 0.0 && a->p < 1.0)) return FSDP_EINVAL;
  const auto threshold = static_cast<uint32_t>(std::floor(a->p * 65536.0 + 0.5));
  if (threshold > 65535) return FSDP_EINVAL;
  if (a->rows == 0) return FSDP_OK;
  const int es = size_of_dtype(a->dtype);
  const Strided sx{x, a->rows, a->cols, a->x_stride, es}, sr{residual, a->rows, a->cols, a->residual_stride, es},
      so{out, a->rows, a->cols, a->out_stride, es}, sc{counter, 1, 1, 1, 8};
  if (!sx.ok() || !so.ok() || (residual && !sr.ok()) || (counter && !sc.ok())) return FSDP_EINVAL;
  if ((so.overlaps(sx) && !so.same_place(sx)) || (residual && so.overlaps(sr) && !so.same_place(sr)) ||
      (counter && so.overlaps(sc)))
    return FSDP_EALIAS;
  DropoutParams p{x, residual, out, a->rows, a->cols, a->x_stride, a->residual_stride, a->out_stride, a->seed, a->offset,
                  counter, threshold, 65536.0f / static_cast<float>(65536 - threshold)};
  const auto contiguous = [&](int64_t stride) { return a->rows < 2 || stride == a->cols; };
  if (contiguous(a->x_stride) && contiguous(a->out_stride) && (!residual || contiguous(a->residual_stride)))
    p.cols *= p.rows, p.rows = 1;  // one long row: the same elements
  const auto aligned = [&](const void* q, int64_t stride) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && (p.rows < 2 || stride * es % 16 == 0);
  };
  const bool vectors = (p.rows == 1 || p.cols % 8 == 0) && aligned(x, a->x_stride) && aligned(out, a->out_stride) &&
                       (!residual || aligned(residual, a->residual_stride));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return a->dtype == FSDP_DTYPE_F32 ? run<float>(p, vectors, st) : run<__nv_bfloat16>(p, vectors, st);
}
