// RMS norm with the residual's addition, and its gradients (fsdp_rmsnorm,
// fsdp_rmsnorm_backward).
//
// With h = x + residual, r = (mean h^2 + eps)^(-1/2), n = h r: y = n gain, and
// for u = dy gain, from dr/dh_j = -r^3 h_j / cols,
//   dx_j = r (u_j - n_j mean_i(u_i n_i)) + dh_j,   dgain_j = sum_rows dy_j n_j.
//
// Both are bound by HBM (5 to 10 operations for 4 to 8 bytes moved per element at
// bf16), so a row is read once: it stays in its threads' registers between the
// sum over the row and the writes. A row belongs to a part of a warp, to one warp (short
// rows, several to a block) or to one block; each thread holds up to kV groups of
// 8 elements. Rows longer than that are read twice (norm_long_rows and its like).
//
// Measured on GB300 (fraction of the copy bandwidth of 6.79 TB/s): 16384 x 4096 bf16 with
// the residual 82.9 us (95 %), backward with the residual's gradient 93.5 us (85 %);
// 4097 x 11008 bf16 to 8 bits in groups of 128 45 us (45 %, bound by instructions: about
// 25 an element, a conversion, two maxima and four products among them); one row of
// 4096 8.5 us, of which the launch from Python is all but 3.
#include "host_internal.h"
#include "row_map.h"
#include "strided.h"
#include "tensor_core.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

namespace fsdp {
namespace {

constexpr int64_t kMaxCols = int64_t(1) << 30;
constexpr int kMaxV = 4;              // groups of 8 elements per thread
constexpr int kMaxThreads = 512;      // of a row held in registers
constexpr int kLongThreads = 256;     // rows beyond the registers

template <RowMap kMap>
constexpr bool kByVectors = kMap == kVector || kMap == kShifted;

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ void store1(uint8_t* p, float v) { *p = to_e4m3(v); }

// 8 elements as loaded, and as floats.
template <typename T>
struct Raw8;
__device__ __forceinline__ void unpack(uint32_t two, float* v) {
  v[0] = __uint_as_float(two << 16);
  v[1] = __uint_as_float(two & 0xffff0000u);
}
template <>
struct Raw8<float> {
  float4 a, b;
  // first, second: whether the 4 elements of each half are wanted
  __device__ __forceinline__ void load(const float* p, bool first, bool second) {
    a = first ? __ldcs(reinterpret_cast<const float4*>(p)) : make_float4(0, 0, 0, 0);
    b = second ? __ldcs(reinterpret_cast<const float4*>(p) + 1) : make_float4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void take(const float* p, bool there) {
    a = there ? *reinterpret_cast<const float4*>(p) : make_float4(0, 0, 0, 0);
    b = there ? *(reinterpret_cast<const float4*>(p) + 1) : make_float4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void to(float* v) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool first, bool second) {
    a = first || second ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void take(const __nv_bfloat16* p, bool there) {
    a = there ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void to(float* v) const {
    unpack(a.x, v), unpack(a.y, v + 2), unpack(a.z, v + 4), unpack(a.w, v + 6);
  }
};
__device__ __forceinline__ void store_vec(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&two);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]));
}
__device__ __forceinline__ void store_vec(uint8_t* p, const float* v) {
  uint32_t two[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    two[e] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * e], v[2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
  *reinterpret_cast<uint2*>(p) = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
}

// The same to a place of any alignment: the aligned 4 bytes among them as one store, the rest around it.
__device__ __forceinline__ void store8_anywhere(uint8_t* p, const float* v) {
  uint32_t two[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    two[e] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * e], v[2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t lo = two[0] | two[1] << 16, hi = two[2] | two[3] << 16;
  const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3u);
  if (s == 0) {
    reinterpret_cast<uint32_t*>(p)[0] = lo;
    reinterpret_cast<uint32_t*>(p)[1] = hi;
  } else if (s == 2) {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(lo);
    *reinterpret_cast<uint32_t*>(p + 2) = __funnelshift_r(lo, hi, 16);
    *reinterpret_cast<uint16_t*>(p + 6) = static_cast<uint16_t>(hi >> 16);
  } else if (s == 1) {
    p[0] = static_cast<uint8_t>(lo);
    *reinterpret_cast<uint16_t*>(p + 1) = static_cast<uint16_t>(lo >> 8);
    *reinterpret_cast<uint32_t*>(p + 3) = __funnelshift_r(lo, hi, 24);
    p[7] = static_cast<uint8_t>(hi >> 24);
  } else {
    p[0] = static_cast<uint8_t>(lo);
    *reinterpret_cast<uint32_t*>(p + 1) = __funnelshift_r(lo, hi, 8);
    *reinterpret_cast<uint16_t*>(p + 5) = static_cast<uint16_t>(hi >> 8);
    p[7] = static_cast<uint8_t>(hi >> 24);
  }
}

__device__ __forceinline__ void store8_anywhere(__nv_bfloat16* p, const float* v) {
  const uint32_t w[4] = {pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7])};
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  if ((at & 15u) == 0) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if ((at & 3u) == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) reinterpret_cast<uint32_t*>(p)[e] = w[e];
  } else {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
#pragma unroll
    for (int e = 0; e < 3; ++e) reinterpret_cast<uint32_t*>(p + 1)[e] = __funnelshift_r(w[e], w[e + 1], 16);
    *reinterpret_cast<uint16_t*>(p + 7) = static_cast<uint16_t>(w[3] >> 16);
  }
}
__device__ __forceinline__ void store8_anywhere(float* p, const float* v) {
  if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    store_vec(p, v);
  } else if ((reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) *reinterpret_cast<float2*>(p + e) = make_float2(v[e], v[e + 1]);
  } else {
    p[0] = v[0];
#pragma unroll
    for (int e = 1; e < 7; e += 2) *reinterpret_cast<float2*>(p + e) = make_float2(v[e], v[e + 1]);
    p[7] = v[7];
  }
}

__device__ __forceinline__ float load_gain(const void* gain, int32_t dtype, int64_t j) {
  return dtype == FSDP_DTYPE_F32 ? load1(static_cast<const float*>(gain) + j)
                                 : load1(static_cast<const __nv_bfloat16*>(gain) + j);
}
// kWords 4-byte words from any 2-byte boundary, out of aligned vectors that each hold some of
// the first `bytes` bytes (what follows them is not defined).
template <int kWords>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&out)[kWords], int bytes = 4 * kWords) {
  constexpr int kVecs = kWords / 4 + 1;
  const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p) - s);
  uint32_t w[4 * kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const uint4 t = bytes > 0 && 16 * i < static_cast<int>(s) + bytes ? q[i] : make_uint4(0, 0, 0, 0);
    w[4 * i] = t.x, w[4 * i + 1] = t.y, w[4 * i + 2] = t.z, w[4 * i + 3] = t.w;
  }
#pragma unroll
  for (int i = 0; i + 2 < 4 * kVecs; ++i) w[i] = s & 8u ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i + 1 < 4 * kVecs; ++i) w[i] = s & 4u ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < kWords; ++i) out[i] = __funnelshift_r(w[i], w[i + 1], (s & 2u) * 8u);
}

// 8 consecutive elements from any place, by aligned vectors; zeros from `count` on.
template <typename T>
__device__ __forceinline__ void load8_anywhere(const T* p, int count, float (&v)[8]) {
  uint32_t w[2 * sizeof(T)];
  load_words(p, w, min(count, 8) * static_cast<int>(sizeof(T)));
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (sizeof(T) == 4)
      v[e] = __uint_as_float(w[e]);
    else
      v[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
  if (count < 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < count ? v[e] : 0.0f;
  }
}

// A thread's kV groups of a row, as loaded.
template <RowMap kMap, int kV, typename T>
struct RowLoad {
  Raw8<T> raw[kByVectors<kMap> ? kV : 1];
  float v[kByVectors<kMap> ? 1 : kV][8];
  __device__ __forceinline__ void load(const T* p, const RowThreads& r, int cols, bool there = true) {
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const int j = place<kMap>(r, k, 0);
      if constexpr (kByVectors<kMap>) {
        const bool first = there && holds_some<kMap>(j, 4, cols);
        raw[k].load(p + j, first, kMap == kVector ? first : there && holds_some<kMap>(j + 4, 4, cols));
      } else if constexpr (kMap == kGroups) {
        load8_anywhere(p + j, there ? cols - j : 0, v[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = place<kMap>(r, k, e);
          v[k][e] = there && i < cols ? load1(p + i) : 0.0f;
        }
      }
    }
  }
  __device__ __forceinline__ void take(const T* p, const RowThreads& r, int cols, bool there = true) {  // shared memory
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const int j = place<kMap>(r, k, 0);
      raw[k].take(p + j, there && j < cols);
    }
  }
  // Group k as floats, zeros outside the row.
  __device__ __forceinline__ void to(int k, const RowThreads& r, int cols, float* out) const {
    if constexpr (kByVectors<kMap>) {
      raw[k].to(out);
      const int j = place<kMap>(r, k, 0);
      if (kMap == kShifted && (j < 0 || j + 8 > cols)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = j + e >= 0 && j + e < cols ? out[e] : 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = v[k][e];
    }
  }
};

template <RowMap kMap, typename T>
__device__ __forceinline__ void store_group(T* p, const RowThreads& r, int v, int cols, const float* in) {
  const int j = place<kMap>(r, v, 0);
  if constexpr (kMap == kVector) {
    if (j < cols) store_vec(p + j, in);
  } else if (kMap == kShifted && j >= 0 && j + 8 <= cols) {
    store_vec(p + j, in);
  } else if (kMap == kGroups && j + 8 <= cols) {
    store8_anywhere(p + j, in);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = place<kMap>(r, v, e);
      if (i >= 0 && i < cols) store1(p + i, in[e]);
    }
  }
}

// The same one by one, to a place of any alignment.
template <RowMap kMap>
__device__ __forceinline__ void store_each(float* p, const RowThreads& r, int v, int cols, const float* in) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = place<kMap>(r, v, e);
    if (i >= 0 && i < cols) p[i] = in[e];
  }
}

// The gains of group v (zeros past the end); `vectors`: the gain starts on a
// 16-byte boundary.
template <RowMap kMap>
__device__ __forceinline__ void gain_group(const void* gain, int32_t dtype, bool vectors, const RowThreads& r, int v,
                                           int cols, float* out) {
  const int j = place<kMap>(r, v, 0);
  if ((kMap == kVector || (kMap == kGroups && j + 8 <= cols)) && vectors) {
    if (dtype == FSDP_DTYPE_F32) {
      Raw8<float> raw;
      raw.a = raw.b = make_float4(0, 0, 0, 0);
      if (j < cols) {
        raw.a = *reinterpret_cast<const float4*>(static_cast<const float*>(gain) + j);
        raw.b = *reinterpret_cast<const float4*>(static_cast<const float*>(gain) + j + 4);
      }
      raw.to(out);
    } else {
      Raw8<__nv_bfloat16> raw;
      raw.a = make_uint4(0, 0, 0, 0);
      if (j < cols) raw.a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(gain) + j);
      raw.to(out);
    }
    return;
  }
  if constexpr (kMap == kGroups) {
    float g[8];
    if (dtype == FSDP_DTYPE_F32)
      load8_anywhere(static_cast<const float*>(gain) + j, cols - j, g);
    else
      load8_anywhere(static_cast<const __nv_bfloat16*>(gain) + j, cols - j, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = g[e];
    return;
  }
  if (kMap == kShifted && j >= 0 && j + 8 <= cols) {
    if (dtype == FSDP_DTYPE_F32) {
      uint32_t w[8];
      load_words(static_cast<const float*>(gain) + j, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = __uint_as_float(w[e]);
    } else {
      uint32_t w[4];
      load_words(static_cast<const __nv_bfloat16*>(gain) + j, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) unpack(w[e], out + 2 * e);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = place<kMap>(r, v, e);
    out[e] = i >= 0 && i < cols ? load_gain(gain, dtype, i) : 0.0f;
  }
}

// The larger one, or a NaN if either is one: the maximum of a group with a NaN is a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

template <bool kMax>
__device__ __forceinline__ float warp_reduce(float v, int lanes = 32) {
  for (int o = lanes / 2; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? max_nan(v, w) : v + w;
  }
  return v;
}

// Over aligned groups of 4, 8, 16 or 32 lanes.
__device__ __forceinline__ float group_max(float v, int lanes) {
  v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 1));
  v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 2));
  if (lanes > 4) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 4));
  if (lanes > 8) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 8));
  if (lanes > 16) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 16));
  return v;
}

// Over the row's threads; every one gets the result. `shared`: 32 floats, free to
// be written (the caller's previous reduction used another one).
template <bool kMax>
__device__ __forceinline__ float row_reduce(float v, const RowThreads& r, float* shared) {
  v = warp_reduce<kMax>(v, min(r.n, 32));
  if (r.n <= 32) return v;
  if (r.t % 32 == 0) shared[r.t / 32] = v;
  __syncthreads();
  const int warps = r.n / 32;
  return warp_reduce<kMax>(r.t % 32 < warps ? shared[r.t % 32] : 0.0f);  // zero is neutral: maxima are of |y|
}

struct NormParams {
  fsdp_rmsnorm_t a;
  const void *x, *residual, *gain;
  void *h, *y;
  float *scales, *rstd;
  int32_t threads;  // of a row
  int32_t group_bits;  // log2 of the group
  // that share a group's maximum: no more than the row's (of 8 or 16 lanes), the next ones are another row's
  int32_t group_lanes;
  bool gain_vectors;
};

// The scale of a group whose largest |y| is `top`.
__device__ __forceinline__ float scale_of(float top) { return max_nan(top * (1.0f / 448.0f), 0x1p-126f); }

// Threads of a row at most, and blocks of them that an SM's registers are to hold:
// more rows in flight while others wait at their reductions. kWide: rows that need
// more threads at kMaxV groups each.
constexpr int forward_threads(int v, bool wide) { return v < 3 || wide ? 512 : 384; }
constexpr int forward_blocks(bool wide) { return wide ? 1 : 2; }
constexpr int backward_threads(bool wide) { return wide ? 512 : 256; }
constexpr int backward_blocks(int v, bool wide) { return wide ? 1 : v == 1 ? 4 : v == 2 ? 3 : 2; }

// kQuant 0: y of the inputs' type; 1: 8 bits, one scale per row; 2: 8 bits, scales per group.
template <typename T, bool kResidual, int kQuant, RowMap kMap, int kV, bool kWide = false>
__global__ void __launch_bounds__(forward_threads(kV, kWide), forward_blocks(kWide))
    norm_rows(const __grid_constant__ NormParams p) {
  __shared__ float shared[3][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int all = static_cast<int>(p.a.cols);
  RowThreads r{static_cast<int>(threadIdx.x) % p.threads, p.threads, 0};
  const int per_block = blockDim.x / p.threads;
  int turn = 0;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * per_block;
  // a warp of several short rows stays together while its first one is there
  const int lead = p.threads < 32 ? static_cast<int>(threadIdx.x) % 32 / p.threads : 0;
  int64_t row = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / p.threads;
  // kAhead: the next row is on its way while this one is worked on
  constexpr bool kAhead = !kResidual && kMap == kVector && kV > 1;
  RowLoad<kMap, kV, T> x, res;
  if constexpr (kAhead)
    x.load(static_cast<const T*>(p.x) + row * p.a.x_stride, r, all, row < p.a.rows);
  for (; row - lead < p.a.rows; row += row_step) {
    const int cols = row < p.a.rows ? all : 0;
    const T* x_row = static_cast<const T*>(p.x) + row * p.a.x_stride;
    if constexpr (kMap == kShifted) r.phase = static_cast<int>((reinterpret_cast<uintptr_t>(x_row) & 15u) / sizeof(T));
    if constexpr (!kAhead) x.load(x_row, r, cols);
    if constexpr (kResidual) res.load(static_cast<const T*>(p.residual) + row * p.a.residual_stride, r, cols);
    float v[kV][8], sum = 0.0f;
    T* h = static_cast<T*>(p.h) + row * p.a.h_stride;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      x.to(k, r, cols, v[k]);
      if constexpr (kResidual) {
        float w[8];
        res.to(k, r, cols, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] += w[e];
        store_group<kMap>(h, r, k, cols, v[k]);
      }
    }
    if constexpr (kAhead)
      x.load(static_cast<const T*>(p.x) + (row + row_step) * p.a.x_stride, r, all, row + row_step < p.a.rows);
#pragma unroll
    for (int k = 0; k < kV; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[k][e] * v[k][e];
    float g[kV][8];
    if constexpr (kV == 1) gain_group<kMap>(p.gain, p.a.gain_dtype, p.gain_vectors, r, 0, cols, g[0]);
    // a block alternates between two sets of partial sums: the barrier inside one
    // reduction ends every read of the one before the last
    float* room = shared[turn];
    turn ^= 1;
    const float rstd = rsqrtf(row_reduce<false>(sum, r, room) / static_cast<float>(all) + static_cast<float>(p.a.eps));
    if (p.rstd && r.t == 0 && cols > 0) p.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      if constexpr (kV > 1)
        gain_group<kMap>(p.gain, p.a.gain_dtype, p.gain_vectors, r, k, cols, g[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] *= kQuant == 0 ? rstd * g[k][e] : g[k][e];  // 8 bits: rstd goes into the scale
    }
    if constexpr (kQuant == 0) {
      T* y = static_cast<T*>(p.y) + row * p.a.y_stride;
#pragma unroll
      for (int k = 0; k < kV; ++k) store_group<kMap>(y, r, k, cols, v[k]);
    } else {
      uint8_t* y = static_cast<uint8_t*>(p.y) + row * p.a.y_stride;
      float top[kV], most = 0.0f;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        top[k] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top[k] = max_nan(top[k], fabsf(v[k][e]));
        most = max_nan(most, top[k]);
      }
      if constexpr (kQuant == 1) {
        most = row_reduce<true>(most, r, shared[2]);
        // the next row's first reduction has a barrier before shared[2] is written again
      }
      const int groups = kQuant == 1 ? 1 : (all + p.a.group - 1) >> p.group_bits;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        if constexpr (kQuant == 2) most = group_max(top[k], p.group_lanes);
        const float scale = scale_of(most * rstd);
        const int j = place<kMap>(r, k, 0);
        if (kQuant == 1 ? (k == 0 && r.t == 0 && cols > 0) : (j < cols && (j & (p.a.group - 1)) == 0))
          p.scales[row * groups + (kQuant == 1 ? 0 : j >> p.group_bits)] = scale;
        // y / scale as h gain (rstd / scale): three roundings, as y (1 / scale) has, and a product an element less
        float inverse = __frcp_rn(scale), q[8];
        if (rstd * inverse <= 0x1p127f) {
          inverse *= rstd;
        } else {  // a group of zeros or next to them: the product of the two factors would overflow
#pragma unroll
          for (int e = 0; e < 8; ++e) v[k][e] *= rstd;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = v[k][e] * inverse;
        store_group<kMap>(y, r, k, cols, q);
      }
    }
  }
}

template <bool kMax>
__device__ __forceinline__ float long_reduce(float v, float* shared) {
  __syncthreads();
  return row_reduce<kMax>(v, RowThreads{static_cast<int>(threadIdx.x), kLongThreads, 0}, shared);
}

// A thread's sum over a long row: what each addition rounds off is kept beside it (Knuth's two-sum), so that the
// error does not grow with the row (2^24 equal values in fp32: a plain running sum is off by up to
// 6e-4 of itself, this one by 2e-8).
struct LongSum {
  float sum = 0.0f, rest = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float next = sum + v, added = next - sum;
    rest += (sum - (next - added)) + (v - added);
    sum = next;
  }
  // past an infinity or a NaN, `rest` is a NaN and says nothing
  __device__ __forceinline__ float value() const { return isfinite(rest) ? sum + rest : sum; }
};

// Calls f(j, count) for the thread's groups of 8 elements of a long row; all threads of the
// block make the same number of calls (count, up to 8, may be 0 or less).
template <typename F>
__device__ __forceinline__ void each_long_group(int64_t cols, F f) {
#pragma unroll 2
  for (int64_t j0 = 0; j0 < cols; j0 += kLongThreads * 8) {
    const int64_t j = j0 + threadIdx.x * 8;
    f(j, static_cast<int>(min(cols - j, int64_t(8))));
  }
}

template <typename T>
__device__ __forceinline__ void store8_upto(T* p, int count, const float* v) {
  if (count >= 8) {
    store8_anywhere(p, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < count) store1(p + e, v[e]);
}

__device__ __forceinline__ void load8_gain(const void* gain, int32_t dtype, int64_t j, int count, float (&g)[8]) {
  if (dtype == FSDP_DTYPE_F32)
    load8_anywhere(static_cast<const float*>(gain) + j, count, g);
  else
    load8_anywhere(static_cast<const __nv_bfloat16*>(gain) + j, count, g);
}

// Rows beyond the registers: one block per row, the row read twice (thrice with one 8-bit
// scale). 1677 x 20000 bf16 with the residual 82 us (49 % of the copy rate), backward with
// the residual's gradient 181 us (22 %: also 8 bytes an element for dgain's share); element by element 129
// and 353 us.
template <typename T, int kQuant>
__global__ void __launch_bounds__(kLongThreads) norm_long_rows(const __grid_constant__ NormParams p) {
  __shared__ float shared[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t cols = p.a.cols;
  for (int64_t row = blockIdx.x; row < p.a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.a.x_stride;
    const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.a.residual_stride : nullptr;
    T* h = p.h ? static_cast<T*>(p.h) + row * p.a.h_stride : nullptr;
    const auto values = [&](int64_t j, int count, float (&v)[8]) {
      load8_anywhere(x + j, count, v);
      if (!res) return;
      float w[8];
      load8_anywhere(res + j, count, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += w[e];
    };
    LongSum squares;
    each_long_group(cols, [&](int64_t j, int count) {
      float v[8], sum = 0.0f;
      values(j, count, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[e] * v[e];
      squares.add(sum);
    });
    const float rstd = rsqrtf(long_reduce<false>(squares.value(), shared) / static_cast<float>(cols) + static_cast<float>(p.a.eps));
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    // y before it is rounded, and h on its way
    const auto normed = [&](int64_t j, int count, bool last, float (&v)[8]) {
      float g[8];
      values(j, count, v);
      load8_gain(p.gain, p.a.gain_dtype, j, count, g);
      if (last && h) store8_upto(h + j, count, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= rstd * g[e];
    };
    if constexpr (kQuant == 0) {
      T* y = static_cast<T*>(p.y) + row * p.a.y_stride;
      each_long_group(cols, [&](int64_t j, int count) {
        float v[8];
        normed(j, count, true, v);
        store8_upto(y + j, count, v);
      });
    } else {
      uint8_t* y = static_cast<uint8_t*>(p.y) + row * p.a.y_stride;
      float all = 0.0f;
      if constexpr (kQuant == 1) {
        each_long_group(cols, [&](int64_t j, int count) {
          float v[8];
          normed(j, count, false, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) all = max_nan(all, fabsf(v[e]));
        });
        all = long_reduce<true>(all, shared);
        if (threadIdx.x == 0) p.scales[row] = scale_of(all);
      }
      const int64_t groups = kQuant == 1 ? 1 : (cols + p.a.group - 1) >> p.group_bits;
      // a lane holds 8 consecutive elements, a group 4 to 32 lanes of a warp
      each_long_group(cols, [&](int64_t j, int count) {
        float v[8], top = 0.0f;
        normed(j, count, true, v);
        if constexpr (kQuant == 2) {
#pragma unroll
          for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(v[e]));
          all = warp_reduce<true>(top, p.a.group / 8);
        }
        const float scale = scale_of(all), inverse = __frcp_rn(scale);
        if (kQuant == 2 && count > 0 && (j & (p.a.group - 1)) == 0) p.scales[row * groups + (j >> p.group_bits)] = scale;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= inverse;
        store8_upto(y + j, count, v);
      });
    }
  }
}

struct NormBwdParams {
  fsdp_rmsnorm_backward_t a;
  const void *dy, *h, *gain, *dh;
  const float* rstd;
  void *dx, *dgain;
  float* partial;   // [parts][cols]
  int32_t threads;  // of a row
  int32_t parts;
  int32_t stages;   // rows in shared memory (norm_staged_backward)
  bool gain_vectors;
  unsigned int* status;
};

constexpr int kMaxStages = 8;
constexpr int kStagedBytes = 216 * 1024;  // of an SM, for all its blocks
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

// A block takes every gridDim-th row (or, with a warp per row, set of rows); a
// thread keeps its columns' share of dgain in registers over all its rows. The
// warps' shares are added in order, then written as the block's row of `partial`.
template <typename T, RowMap kMap, int kV, bool kWide = false>
__global__ void __launch_bounds__(backward_threads(kWide), backward_blocks(kV, kWide))
    norm_rows_backward(const __grid_constant__ NormBwdParams p) {
  __shared__ float shared[2][32];
  extern __shared__ float total[];  // [cols], with a warp per row
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int all = static_cast<int>(p.a.cols);
  RowThreads r{static_cast<int>(threadIdx.x) % p.threads, p.threads, 0};
  const int per_block = blockDim.x / p.threads;
  float acc[kV][8] = {};
  int turn = 0;
  const int lead = p.threads < 32 ? static_cast<int>(threadIdx.x) % 32 / p.threads : 0;  // as in norm_rows
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / p.threads; row - lead < p.a.rows;
       row += static_cast<int64_t>(gridDim.x) * per_block) {
    const int cols = row < p.a.rows ? all : 0;
    const T* dy_row = static_cast<const T*>(p.dy) + row * p.a.dy_stride;
    // kShifted: the rows of a thread are a multiple of 8 apart and have one phase
    if constexpr (kMap == kShifted)
      if (cols > 0) r.phase = static_cast<int>((reinterpret_cast<uintptr_t>(dy_row) & 15u) / sizeof(T));
    RowLoad<kMap, kV, T> dy, h, dh;
    dy.load(dy_row, r, cols);
    h.load(static_cast<const T*>(p.h) + row * p.a.h_stride, r, cols);
    const T* dh_row = static_cast<const T*>(p.dh) + row * p.a.dh_stride;
    if constexpr (kByVectors<kMap>) dh.load(dh_row, r, cols, p.dh != nullptr);  // early: it costs 4 registers a group
    const float rstd = cols > 0 ? p.rstd[row] : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      float u[8], n[8], g[8];
      dy.to(k, r, cols, u);
      h.to(k, r, cols, n);
      gain_group<kMap>(p.gain, p.a.gain_dtype, p.gain_vectors, r, k, cols, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = u[e] * (n[e] * rstd);
        acc[k][e] += t;
        sum += t * g[e];
      }
    }
    const float mean = row_reduce<false>(sum, r, shared[turn]) / static_cast<float>(all);
    turn ^= 1;
    if constexpr (!kByVectors<kMap>) dh.load(dh_row, r, cols, p.dh != nullptr);
    T* dx = static_cast<T*>(p.dx) + row * p.a.dx_stride;
#pragma unroll
    for (int k = 0; k < kV; ++k) {  // formed again from the row as loaded: fewer registers over the reduction
      float u[8], n[8], g[8], d[8];
      dy.to(k, r, cols, u);
      h.to(k, r, cols, n);
      dh.to(k, r, cols, d);
      gain_group<kMap>(p.gain, p.a.gain_dtype, p.gain_vectors, r, k, cols, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] += rstd * (u[e] * g[e] - n[e] * rstd * mean);
      store_group<kMap>(dx, r, k, cols, d);
    }
  }
  float* mine = p.partial + static_cast<int64_t>(blockIdx.x) * all;
  if (per_block > 1) {
    const int slot = threadIdx.x / p.threads;
    for (int w = 0; w < per_block; ++w) {
      if (w == slot) {
#pragma unroll
        for (int k = 0; k < kV; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int j = place<kMap>(r, k, e);
            if (j < 0 || j >= all) continue;
            if (w + 1 < per_block)
              total[j] = (w > 0 ? total[j] : 0.0f) + acc[k][e];
            else
              mine[j] = total[j] + acc[k][e];
          }
      }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int k = 0; k < kV; ++k) store_each<kMap>(mine, r, k, all, acc[k]);
  }
}

// The same for many aligned rows of a block each, the rows staged in shared memory by
// bulk copies: `stages` rows ahead of the one at work. The row's values are read
// into registers, and after the barrier inside the sum over the row its stage is free
// for the next copy, so that the memory stays busy through the reductions.
// (16384 x 4096 bf16 with dh: 131 us without the stages.)
template <typename T, int kV, bool kWide>
__global__ void __launch_bounds__(backward_threads(kWide), backward_blocks(kV, kWide))
    norm_staged_backward(const __grid_constant__ NormBwdParams p) {
  __shared__ float shared[2][32];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ int stop;
  extern __shared__ __align__(128) unsigned char staged[];  // stages x {dy, h, dh} rows
  const int cols = static_cast<int>(p.a.cols);
  const RowThreads r{static_cast<int>(threadIdx.x), p.threads, 0};
  const uint32_t row_bytes = static_cast<uint32_t>(cols) * sizeof(T), arrays = p.dh ? 3 : 2;
  const tc::Guard guard{&stop, p.status, kWaitLimitNs};
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) tc::bar_init(tc::smem_addr(&full[s]), 1);
    stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const auto fetch = [&](int64_t row, int s) {
    const uint32_t bar = tc::smem_addr(&full[s]), to = tc::smem_addr(staged) + s * arrays * row_bytes;
    tc::bar_expect(bar, arrays * row_bytes);
    tc::bulk_load(to, static_cast<const T*>(p.dy) + row * p.a.dy_stride, row_bytes, bar);
    tc::bulk_load(to + row_bytes, static_cast<const T*>(p.h) + row * p.a.h_stride, row_bytes, bar);
    if (p.dh) tc::bulk_load(to + 2 * row_bytes, static_cast<const T*>(p.dh) + row * p.a.dh_stride, row_bytes, bar);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < p.stages; ++s) {
      const int64_t row = blockIdx.x + static_cast<int64_t>(s) * gridDim.x;
      if (row < p.a.rows) fetch(row, s);
    }
  float acc[kV][8] = {};
  int turn = 0, stage = 0;
  uint32_t parity = 0, turns = 0;
  bool failed = false;
  for (int64_t row = blockIdx.x; row < p.a.rows; row += gridDim.x) {
    const float rstd = p.rstd[row];
    failed = !tc::bar_wait(tc::smem_addr(&full[stage]), parity, guard);
    const unsigned char* at = staged + stage * arrays * row_bytes;
    RowLoad<kVector, kV, T> dy, h, dh;
    dy.take(reinterpret_cast<const T*>(at), r, cols);
    h.take(reinterpret_cast<const T*>(at + row_bytes), r, cols);
    dh.take(reinterpret_cast<const T*>(at + 2 * row_bytes), r, cols, p.dh != nullptr);
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      float u[8], n[8], g[8];
      dy.to(k, r, cols, u);
      h.to(k, r, cols, n);
      gain_group<kVector>(p.gain, p.a.gain_dtype, p.gain_vectors, r, k, cols, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = u[e] * (n[e] * rstd);
        acc[k][e] += t;
        sum += t * g[e];
      }
    }
    sum = warp_reduce<false>(sum);
    if (r.t % 32 == 0) shared[turn][r.t / 32] = sum;
    failed = __syncthreads_or(failed);
    if (failed) break;
    const int64_t next = row + static_cast<int64_t>(p.stages) * gridDim.x;
    if (threadIdx.x == 0 && next < p.a.rows) fetch(next, stage);
    const float mean =
        warp_reduce<false>(r.t % 32 < r.n / 32 ? shared[turn][r.t % 32] : 0.0f) / static_cast<float>(cols);
    turn ^= 1;
    T* dx = static_cast<T*>(p.dx) + row * p.a.dx_stride;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      float u[8], n[8], g[8], d[8];
      dy.to(k, r, cols, u);
      h.to(k, r, cols, n);
      dh.to(k, r, cols, d);
      gain_group<kVector>(p.gain, p.a.gain_dtype, p.gain_vectors, r, k, cols, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] += rstd * (u[e] * g[e] - n[e] * rstd * mean);
      store_group<kVector>(dx, r, k, cols, d);
    }
    if (++stage == p.stages) stage = 0, parity ^= 1u;
    ++turns;
  }
  if (failed && threadIdx.x == 0) {  // copies in flight land before the block ends
    for (int s = 0; s < p.stages; ++s) {
      if (blockIdx.x + static_cast<int64_t>(turns + s) * gridDim.x < p.a.rows)
        tc::bar_drain(tc::smem_addr(&full[stage]), parity, kWaitLimitNs);
      if (++stage == p.stages) stage = 0, parity ^= 1u;
    }
  }
  float* mine = p.partial + static_cast<int64_t>(blockIdx.x) * cols;
#pragma unroll
  for (int k = 0; k < kV; ++k) store_each<kVector>(mine, r, k, cols, acc[k]);
}

// Rows beyond the registers: the row read twice, dgain's share kept in `partial`.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_long_rows_backward(const __grid_constant__ NormBwdParams p) {
  __shared__ float shared[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t cols = p.a.cols;
  float* mine = p.partial + blockIdx.x * cols;
  bool first = true;
  for (int64_t row = blockIdx.x; row < p.a.rows; row += gridDim.x, first = false) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.a.dy_stride;
    const T* h = static_cast<const T*>(p.h) + row * p.a.h_stride;
    const T* dh = p.dh ? static_cast<const T*>(p.dh) + row * p.a.dh_stride : nullptr;
    T* dx = static_cast<T*>(p.dx) + row * p.a.dx_stride;
    const float r = p.rstd[row];
    LongSum products;
    each_long_group(cols, [&](int64_t j, int count) {
      float u[8], n[8], g[8], acc[8] = {}, sum = 0.0f;
      load8_anywhere(dy + j, count, u);
      load8_anywhere(h + j, count, n);
      load8_gain(p.gain, p.a.gain_dtype, j, count, g);
      if (!first) load8_anywhere(mine + j, count, acc);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = u[e] * (n[e] * r);
        sum += t * g[e];
        acc[e] += t;
      }
      products.add(sum);
      store8_upto(mine + j, count, acc);
    });
    const float mean = long_reduce<false>(products.value(), shared) / static_cast<float>(cols);
    each_long_group(cols, [&](int64_t j, int count) {
      float u[8], n[8], g[8], d[8] = {};
      load8_anywhere(dy + j, count, u);
      load8_anywhere(h + j, count, n);
      load8_gain(p.gain, p.a.gain_dtype, j, count, g);
      if (dh) load8_anywhere(dh + j, count, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] += r * (u[e] * g[e] - n[e] * r * mean);
      store8_upto(dx + j, count, d);
    });
  }
}

// dgain: 32 columns per block, its 32 warps share the rows of `partial`.
__global__ void __launch_bounds__(1024) sum_partials(const __grid_constant__ NormBwdParams p) {
  __shared__ float shared[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float sum = 0.0f;
  if (j < p.a.cols) {
    for (int i = warp; i < p.parts; i += 256) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = i + 32 * k < p.parts ? p.partial[(i + 32 * k) * p.a.cols + j] : 0.0f;
      sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  }
  shared[warp][lane] = sum;
  __syncthreads();
  // warp w adds up column w
  sum = warp_reduce<false>(shared[lane][warp]);
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane != 0 || c >= p.a.cols) return;
  if (p.a.gain_dtype == FSDP_DTYPE_F32)
    static_cast<float*>(p.dgain)[c] = sum;
  else
    store1(static_cast<__nv_bfloat16*>(p.dgain) + c, sum);
}

// ------------------------------------------------------------- host side

template <typename P>
int launch_rows(void (*kernel)(P), int grid, int threads, int smem, cudaStream_t stream, const P& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? FSDP_OK : FSDP_ECUDA;
}

// How a row is spread: kV groups of 8 elements for each of `threads` threads.
struct Spread {
  int v = 0, threads = 0, per_block = 1;  // v = 0: a long row
};

int warps_for(int64_t cols, int v) { return static_cast<int>((cols + 256 * v - 1) / (256 * v)); }

constexpr int kFewRows = 512;  // about as many rows as blocks run at once

// `cols`: of the row, with up to 7 more where its groups are shifted. Short rows share a
// warp: 8 or 16 lanes each, so that few lanes are idle.
int threads_for(int64_t rows, int64_t cols, int v) {
  if (rows >= kFewRows && v == 1 && cols <= 128) return cols <= 64 ? 8 : 16;
  return 32 * warps_for(cols, v);
}

Spread forward_spread(int64_t rows, int64_t cols) {
  Spread s;
  if (cols > kMaxThreads * 8 * kMaxV) return s;
  s.v = rows < kFewRows ? 1 : static_cast<int>(std::min<int64_t>(kMaxV, (cols + 1023) / 1024));
  if (rows >= kFewRows && cols <= 1024) s.v = warps_for(cols, 1);  // a warp per row
  while (s.v < kMaxV && 32 * warps_for(cols, s.v) > forward_threads(s.v, false)) ++s.v;
  s.threads = threads_for(rows, cols, s.v);
  if (s.threads <= 32) s.per_block = 128 / s.threads;
  return s;
}

// A warp per row up to 512 columns only: beyond that the staged rows are faster
// (43690 x 768 bf16: 63 us with a warp per row).
Spread backward_spread(int64_t rows, int64_t cols) {
  Spread s;
  if (cols > kMaxThreads * 8 * kMaxV) return s;
  s.v = rows < kFewRows ? 1 : static_cast<int>(std::min<int64_t>(kMaxV, (cols + 2047) / 2048));
  if (rows >= kFewRows && cols <= 512) s.v = warps_for(cols, 1);
  while (s.v < kMaxV && 32 * warps_for(cols, s.v) > backward_threads(false)) ++s.v;
  s.threads = threads_for(rows, cols, s.v);
  if (s.threads <= 32) s.per_block = 256 / s.threads;
  return s;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 152;
  return sms;
}

// Blocks of the backward pass (rows of `partial`): as many as run at once, a multiple of 8
// where a block has several rows.
int backward_parts(int64_t rows, const Spread& s) {
  int per_sm = 4;
  if (s.v > 0) {
    const int threads = s.threads * s.per_block;
    const bool wide = threads > backward_threads(false);
    per_sm = std::max(1, backward_blocks(s.v, wide) * backward_threads(wide) / threads);
  }
  const int64_t most = std::max<int64_t>(8, static_cast<int64_t>(per_sm) * sm_count() / 8 * 8);
  return static_cast<int>(std::min<int64_t>((std::max<int64_t>(rows, 1) + s.per_block - 1) / s.per_block, most));
}

// The columns that a row's groups have to cover.
int64_t covered(int64_t cols, RowMap map) { return map == kShifted ? cols + 7 : cols; }

template <typename T, bool kResidual, int kQuant, RowMap kMap>
int run_forward(const NormParams& p, const Spread& s, int grid, cudaStream_t st) {
  const int threads = s.threads * s.per_block;
  switch (s.v) {
    case 1: return launch_rows(norm_rows<T, kResidual, kQuant, kMap, 1>, grid, threads, 0, st, p);
    case 2: return launch_rows(norm_rows<T, kResidual, kQuant, kMap, 2>, grid, threads, 0, st, p);
    case 3: return launch_rows(norm_rows<T, kResidual, kQuant, kMap, 3>, grid, threads, 0, st, p);
    default:
      return launch_rows(threads > forward_threads(kMaxV, false) ? norm_rows<T, kResidual, kQuant, kMap, kMaxV, true>
                                                                 : norm_rows<T, kResidual, kQuant, kMap, kMaxV>,
                         grid, threads, 0, st, p);
  }
}

template <typename T, bool kResidual>
int run_forward_as(const NormParams& p, const Spread& s, RowMap map, int grid, cudaStream_t st) {
  const int quant = p.a.y_dtype != FSDP_DTYPE_E4M3 ? 0 : p.a.group == 0 ? 1 : 2;
  if (map == kVector)
    return quant == 0   ? run_forward<T, kResidual, 0, kVector>(p, s, grid, st)
           : quant == 1 ? run_forward<T, kResidual, 1, kVector>(p, s, grid, st)
                        : run_forward<T, kResidual, 2, kVector>(p, s, grid, st);
  if (map == kShifted) return run_forward<T, kResidual, 0, kShifted>(p, s, grid, st);
  if (map == kSingles)  // a group of 8 per lane
    return launch_rows(quant == 1 ? norm_rows<T, kResidual, 1, kSingles, 1> : norm_rows<T, kResidual, 2, kSingles, 1>, grid,
                       s.threads * s.per_block, 0, st, p);
  return quant == 0   ? run_forward<T, kResidual, 0, kStrided>(p, s, grid, st)
         : quant == 1 ? run_forward<T, kResidual, 1, kGroups>(p, s, grid, st)
                      : run_forward<T, kResidual, 2, kGroups>(p, s, grid, st);
}

template <typename T>
int forward(NormParams p, RowMap map, cudaStream_t st) {
  const bool quant = p.a.y_dtype == FSDP_DTYPE_E4M3;
  // 8 bits: y's rows have a distance of their own
  if (quant && map != kVector) map = p.a.cols <= 256 ? kSingles : kGroups;
  const Spread s = forward_spread(p.a.rows, covered(p.a.cols, map));
  p.threads = s.threads;
  p.group_lanes = std::min(p.a.group / 8, s.threads);
  // as many blocks as run at once where a block works ahead, else one for each row
  int64_t most = 1 << 20;
  if (s.v > 1 && map == kVector && !p.residual)
    most = static_cast<int64_t>(sm_count()) * std::max(1, 768 / (s.threads * s.per_block));
  const int grid = static_cast<int>(std::min<int64_t>((p.a.rows + s.per_block - 1) / s.per_block, most));
  if (s.v == 0)
    return launch_rows(!quant ? norm_long_rows<T, 0> : p.a.group == 0 ? norm_long_rows<T, 1> : norm_long_rows<T, 2>, grid,
                       kLongThreads, 0, st, p);
  return p.residual ? run_forward_as<T, true>(p, s, map, grid, st) : run_forward_as<T, false>(p, s, map, grid, st);
}

template <typename T, RowMap kMap>
int run_backward(const NormBwdParams& p, const Spread& s, cudaStream_t st) {
  const int threads = s.threads * s.per_block, smem = s.per_block > 1 ? static_cast<int>(p.a.cols * 4) : 0;
  switch (s.v) {
    case 1: return launch_rows(norm_rows_backward<T, kMap, 1>, p.parts, threads, smem, st, p);
    case 2: return launch_rows(norm_rows_backward<T, kMap, 2>, p.parts, threads, smem, st, p);
    case 3: return launch_rows(norm_rows_backward<T, kMap, 3>, p.parts, threads, smem, st, p);
    default:
      return launch_rows(threads > backward_threads(false) ? norm_rows_backward<T, kMap, kMaxV, true>
                                                           : norm_rows_backward<T, kMap, kMaxV>,
                         p.parts, threads, smem, st, p);
  }
}

template <typename T>
int run_staged(const NormBwdParams& p, const Spread& s, int smem, cudaStream_t st) {
  const auto go = [&](auto kernel) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStagedBytes) != cudaSuccess)
      return FSDP_ECUDA;
    return launch_rows(kernel, p.parts, s.threads, smem, st, p);
  };
  switch (s.v) {
    case 1: return go(norm_staged_backward<T, 1, false>);
    case 2: return go(norm_staged_backward<T, 2, false>);
    case 3: return go(norm_staged_backward<T, 3, false>);
    default:
      return s.threads > backward_threads(false) ? go(norm_staged_backward<T, kMaxV, true>)
                                                 : go(norm_staged_backward<T, kMaxV, false>);
  }
}

template <typename T>
int backward(NormBwdParams p, RowMap map, cudaStream_t st) {
  const Spread s = backward_spread(p.a.rows, covered(p.a.cols, map));
  p.threads = s.threads;
  p.parts = backward_parts(p.a.rows, s);
  // several rows per block: staged, if an SM's shared memory holds two for each of its blocks
  const int64_t row_bytes = p.a.cols * static_cast<int64_t>(sizeof(T)) * (p.dh ? 3 : 2);
  const int per_sm = (p.parts + sm_count() - 1) / sm_count();
  const int64_t stages = std::min<int64_t>(kMaxStages, (kStagedBytes / per_sm - 1024) / row_bytes);
  int rc;
  if (s.v == 0) {
    rc = launch_rows(norm_long_rows_backward<T>, p.parts, kLongThreads, 0, st, p);
  } else if (map == kVector && s.per_block == 1 && p.a.rows > p.parts && stages >= 2) {
    p.stages = static_cast<int32_t>(stages);
    rc = device_status_word(&p.status);
    if (rc == FSDP_OK) rc = run_staged<T>(p, s, static_cast<int>(stages * row_bytes), st);
  } else {
    rc = map == kVector    ? run_backward<T, kVector>(p, s, st)
         : map == kShifted ? run_backward<T, kShifted>(p, s, st)
                           : run_backward<T, kStrided>(p, s, st);
  }
  if (rc != FSDP_OK) return rc;
  return launch_rows(sum_partials, static_cast<int>((p.a.cols + 31) / 32), 1024, 0, st, p);
}

struct Rows {
  const void* p;  // null: no such array
  int64_t stride;
};

// How rows of `size`-byte elements in these arrays can be read and written.
RowMap map_of(std::initializer_list<Rows> arrays, int64_t rows, int64_t cols, int size) {
  const Rows* first = nullptr;
  bool aligned = cols % 8 == 0, together = true;
  for (const Rows& q : arrays) {
    if (!q.p) continue;
    if (!first) first = &q;
    const auto at = reinterpret_cast<uintptr_t>(q.p), at0 = reinterpret_cast<uintptr_t>(first->p);
    aligned = aligned && at % 16 == 0 && (rows < 2 || q.stride * size % 16 == 0);
    together = together && at % 16 == at0 % 16 && (rows < 2 || (q.stride - first->stride) * size % 16 == 0);
  }
  return aligned ? kVector : together ? kShifted : kStrided;
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" int fsdp_rmsnorm(const fsdp_rmsnorm_t* a, const void* x, const void* residual, const void* gain,
                            void* h_out, void* y, float* scales, float* rstd, fsdp_stream_t stream) {
  if (!a || a->rows < 0 || a->cols < 1 || a->cols > kMaxCols) return FSDP_EINVAL;
  if (a->dtype != FSDP_DTYPE_F32 && a->dtype != FSDP_DTYPE_BF16) return FSDP_EINVAL;
  if (a->gain_dtype != FSDP_DTYPE_F32 && a->gain_dtype != FSDP_DTYPE_BF16) return FSDP_EINVAL;
  const bool e4m3 = a->y_dtype == FSDP_DTYPE_E4M3;
  if (!e4m3 && (a->y_dtype != a->dtype || a->group != 0 || scales)) return FSDP_EINVAL;
  if (a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128 && a->group != 256) return FSDP_EINVAL;
  if (!(a->eps > 0.0) || !std::isfinite(a->eps) || !(static_cast<float>(a->eps) > 0.0f)) return FSDP_EINVAL;
  if (!residual != !h_out) return FSDP_EINVAL;
  if (a->rows == 0) return FSDP_OK;
  const int es = size_of_dtype(a->dtype), gs = size_of_dtype(a->gain_dtype);
  const int64_t groups = a->group ? (a->cols + a->group - 1) / a->group : 1;
  const Strided sx{x, a->rows, a->cols, a->x_stride, es}, sr{residual, a->rows, a->cols, a->residual_stride, es},
      sh{h_out, a->rows, a->cols, a->h_stride, es}, sy{y, a->rows, a->cols, a->y_stride, size_of_dtype(a->y_dtype)},
      sg{gain, 1, a->cols, a->cols, gs}, ss{scales, a->rows, groups, groups, 4}, sd{rstd, a->rows, 1, 1, 4};
  if (!sx.ok() || !sy.ok() || !sg.ok() || (e4m3 && !ss.ok()) || (residual && (!sr.ok() || !sh.ok())) ||
      (rstd && !sd.ok()))
    return FSDP_EINVAL;
  const Strided* in[] = {&sx, residual ? &sr : nullptr, &sg};
  const Strided* out[] = {h_out ? &sh : nullptr, &sy, e4m3 ? &ss : nullptr, rstd ? &sd : nullptr};
  for (const Strided* o : out) {
    if (!o) continue;
    for (const Strided* q : out)
      if (q && q != o && o->overlaps(*q)) return FSDP_EALIAS;
    for (const Strided* i : in) {
      if (!i || !o->overlaps(*i)) continue;
      const bool in_place = (o == &sh && i != &sg && o->same_place(*i)) || (o == &sy && i == &sx && o->same_place(*i));
      if (!in_place) return FSDP_EALIAS;
    }
  }
  int group_bits = 0;
  while (a->group >> (group_bits + 1)) ++group_bits;
  const NormParams p{*a, x, residual, gain, h_out, y, scales, rstd, 0, group_bits, 0,
                     reinterpret_cast<uintptr_t>(gain) % 16 == 0};
  RowMap map = map_of({{x, a->x_stride}, {residual, a->residual_stride}, {h_out, a->h_stride}, {e4m3 ? nullptr : y, a->y_stride}},
                   a->rows, a->cols, es);
  if (e4m3 && (reinterpret_cast<uintptr_t>(y) % 8 != 0 || (a->rows > 1 && a->y_stride % 8 != 0))) map = kStrided;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return a->dtype == FSDP_DTYPE_F32 ? forward<float>(p, map, st) : forward<__nv_bfloat16>(p, map, st);
}

extern "C" int fsdp_rmsnorm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes_out) {
  if (!bytes_out || rows < 0 || cols < 1 || cols > kMaxCols) return FSDP_EINVAL;
  // whatever the rows' alignment will be
  const int parts = std::max(backward_parts(rows, backward_spread(rows, cols)),
                             backward_parts(rows, backward_spread(rows, covered(cols, kShifted))));
  *bytes_out = parts * cols * 4 + 16;
  return FSDP_OK;
}

extern "C" int fsdp_rmsnorm_backward(const fsdp_rmsnorm_backward_t* a, const void* dy, const void* h, const void* gain,
                                     const float* rstd, const void* dh, void* dx, void* dgain, void* workspace,
                                     int64_t workspace_bytes, fsdp_stream_t stream) {
  if (!a || a->rows < 0 || a->cols < 1) return FSDP_EINVAL;
  if (a->dtype != FSDP_DTYPE_F32 && a->dtype != FSDP_DTYPE_BF16) return FSDP_EINVAL;
  if (a->gain_dtype != FSDP_DTYPE_F32 && a->gain_dtype != FSDP_DTYPE_BF16) return FSDP_EINVAL;
  int64_t need = 0;
  if (int rc = fsdp_rmsnorm_backward_workspace(a->rows, a->cols, &need)) return rc;
  const int es = size_of_dtype(a->dtype), gs = size_of_dtype(a->gain_dtype);
  const Strided sdy{dy, a->rows, a->cols, a->dy_stride, es}, sh{h, a->rows, a->cols, a->h_stride, es},
      sdh{dh, a->rows, a->cols, a->dh_stride, es}, sdx{dx, a->rows, a->cols, a->dx_stride, es},
      sg{gain, 1, a->cols, a->cols, gs}, sdg{dgain, 1, a->cols, a->cols, gs}, sr{rstd, a->rows, 1, 1, 4},
      sw{workspace, 1, need, need, 1};
  if (!sdg.ok()) return FSDP_EINVAL;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->rows == 0)
    return cudaMemsetAsync(dgain, 0, static_cast<size_t>(a->cols) * gs, st) == cudaSuccess ? FSDP_OK : FSDP_ECUDA;
  if (!sdy.ok() || !sh.ok() || !sg.ok() || !sr.ok() || !sdx.ok() || !sw.ok() || (dh && !sdh.ok())) return FSDP_EINVAL;
  if (workspace_bytes < need) return FSDP_EWORKSPACE;
  const Strided* in[] = {&sdy, &sh, &sg, &sr, dh ? &sdh : nullptr};
  const Strided* out[] = {&sdx, &sdg, &sw};
  for (const Strided* o : out) {
    for (const Strided* q : out)
      if (q != o && o->overlaps(*q)) return FSDP_EALIAS;
    for (const Strided* i : in)
      if (i && o->overlaps(*i) && !(o == &sdx && (i == &sdy || i == &sdh) && o->same_place(*i))) return FSDP_EALIAS;
  }
  float* partial = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + 15) & ~uintptr_t(15));
  const NormBwdParams p{*a, dy, h, gain, dh, rstd, dx, dgain, partial, 0, 0, 0,
                        reinterpret_cast<uintptr_t>(gain) % 16 == 0, nullptr};
  const RowMap map =
      map_of({{dy, a->dy_stride}, {h, a->h_stride}, {dh, a->dh_stride}, {dx, a->dx_stride}}, a->rows, a->cols, es);
  return a->dtype == FSDP_DTYPE_F32 ? backward<float>(p, map, st) : backward<__nv_bfloat16>(p, map, st);
}
