// RMS norm with the residual's addition, and its gradients (fsdp_rmsnorm,
// fsdp_rmsnorm_backward).
//
// With h = x + residual, r = (mean h^2 + eps)^(-1/2), n = h r: y = n gain, and
// for u = dy gain, from dr/dh_j = -r^3 h_j / cols,
//   dx_j = r (u_j - n_j mean_i(u_i n_i)) + dh_j,   dgain_j = sum_rows dy_j n_j.
#include "fsdp.h"
#include "strided.h"

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace fsdp {
namespace {

constexpr int kNormThreads = 256;
constexpr int64_t kMaxCols = int64_t(1) << 30;

template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float load_gain(const void* gain, int32_t dtype, int64_t j) {
  return dtype == FSDP_DTYPE_F32 ? load1(static_cast<const float*>(gain) + j)
                                 : load1(static_cast<const __nv_bfloat16*>(gain) + j);
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}

template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* shared) {
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, w) : v + w;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = v;
  __syncthreads();
  v = shared[0];
  for (int i = 1; i < kNormThreads / 32; ++i) v = kMax ? fmaxf(v, shared[i]) : v + shared[i];
  return v;
}

struct NormParams {
  fsdp_rmsnorm_t a;
  const void *x, *residual, *gain;
  void *h, *y;
  float *scales, *rstd;
};

// One block per row, the row read twice.
template <typename T, bool kE4m3>
__global__ void __launch_bounds__(kNormThreads) norm_rows(const NormParams p) {
  __shared__ float shared[kNormThreads / 32];
  const int64_t cols = p.a.cols;
  for (int64_t row = blockIdx.x; row < p.a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.a.x_stride;
    const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.a.residual_stride : nullptr;
    T* h = p.h ? static_cast<T*>(p.h) + row * p.a.h_stride : nullptr;
    float sum = 0.0f;
    for (int64_t j = threadIdx.x; j < cols; j += kNormThreads) {
      const float v = load1(x + j) + (res ? load1(res + j) : 0.0f);
      sum += v * v;
    }
    const float rstd = rsqrtf(block_reduce<false>(sum, shared) / static_cast<float>(cols) + static_cast<float>(p.a.eps));
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    if constexpr (kE4m3) {
      uint8_t* y = static_cast<uint8_t*>(p.y) + row * p.a.y_stride;
      const int64_t group = p.a.group ? p.a.group : cols;
      const int64_t groups = (cols + group - 1) / group;
      for (int64_t g = 0; g < groups; ++g) {
        const int64_t end = min(cols, (g + 1) * group);
        float top = 0.0f;
        for (int64_t j = g * group + threadIdx.x; j < end; j += kNormThreads)
          top = fmaxf(top, fabsf((load1(x + j) + (res ? load1(res + j) : 0.0f)) * rstd * load_gain(p.gain, p.a.gain_dtype, j)));
        const float scale = fmaxf(block_reduce<true>(top, shared) / 448.0f, 0x1p-126f);
        if (threadIdx.x == 0) p.scales[row * groups + g] = scale;
        for (int64_t j = g * group + threadIdx.x; j < end; j += kNormThreads) {
          const float v = load1(x + j) + (res ? load1(res + j) : 0.0f);
          y[j] = to_e4m3(v * rstd * load_gain(p.gain, p.a.gain_dtype, j) / scale);
          if (h) store1(h + j, v);
        }
      }
    } else {
      T* y = static_cast<T*>(p.y) + row * p.a.y_stride;
      for (int64_t j = threadIdx.x; j < cols; j += kNormThreads) {
        const float v = load1(x + j) + (res ? load1(res + j) : 0.0f);
        if (h) store1(h + j, v);
        store1(y + j, v * rstd * load_gain(p.gain, p.a.gain_dtype, j));
      }
    }
  }
}

struct NormBwdParams {
  fsdp_rmsnorm_backward_t a;
  const void *dy, *h, *gain, *dh;
  const float* rstd;
  void *dx, *dgain;
  float* partial;  // [gridDim.x][cols]
};

// One block per row in turn; its share of dgain in its own row of `partial`.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_rows_backward(const NormBwdParams p) {
  __shared__ float shared[kNormThreads / 32];
  const int64_t cols = p.a.cols;
  float* mine = p.partial + blockIdx.x * cols;
  for (int64_t j = threadIdx.x; j < cols; j += kNormThreads) mine[j] = 0.0f;
  for (int64_t row = blockIdx.x; row < p.a.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.a.dy_stride;
    const T* h = static_cast<const T*>(p.h) + row * p.a.h_stride;
    const T* dh = p.dh ? static_cast<const T*>(p.dh) + row * p.a.dh_stride : nullptr;
    T* dx = static_cast<T*>(p.dx) + row * p.a.dx_stride;
    const float r = p.rstd[row];
    float sum = 0.0f;
    for (int64_t j = threadIdx.x; j < cols; j += kNormThreads) {
      const float g = load1(dy + j), n = load1(h + j) * r;
      sum += g * load_gain(p.gain, p.a.gain_dtype, j) * n;
      mine[j] += g * n;
    }
    const float mean = block_reduce<false>(sum, shared) / static_cast<float>(cols);
    for (int64_t j = threadIdx.x; j < cols; j += kNormThreads) {
      const float n = load1(h + j) * r;
      float v = r * (load1(dy + j) * load_gain(p.gain, p.a.gain_dtype, j) - n * mean);
      if (dh) v += load1(dh + j);
      store1(dx + j, v);
    }
  }
}

__global__ void __launch_bounds__(kNormThreads) sum_partials(const NormBwdParams p, int parts) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
  if (j >= p.a.cols) return;
  float sum = 0.0f;
  for (int i = 0; i < parts; ++i) sum += p.partial[i * p.a.cols + j];
  if (p.a.gain_dtype == FSDP_DTYPE_F32)
    static_cast<float*>(p.dgain)[j] = sum;
  else
    store1(static_cast<__nv_bfloat16*>(p.dgain) + j, sum);
}

int backward_blocks(int64_t rows) { return static_cast<int>(std::min<int64_t>(std::max<int64_t>(rows, 1), 608)); }

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
  const NormParams p{*a, x, residual, gain, h_out, y, scales, rstd};
  const int grid = static_cast<int>(std::min<int64_t>(a->rows, 1 << 16));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->dtype == FSDP_DTYPE_F32)
    e4m3 ? norm_rows<float, true><<<grid, kNormThreads, 0, st>>>(p) : norm_rows<float, false><<<grid, kNormThreads, 0, st>>>(p);
  else
    e4m3 ? norm_rows<__nv_bfloat16, true><<<grid, kNormThreads, 0, st>>>(p)
         : norm_rows<__nv_bfloat16, false><<<grid, kNormThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? FSDP_OK : FSDP_ECUDA;
}

extern "C" int fsdp_rmsnorm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes_out) {
  if (!bytes_out || rows < 0 || cols < 1 || cols > kMaxCols) return FSDP_EINVAL;
  *bytes_out = backward_blocks(rows) * cols * 4 + 16;
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
  const NormBwdParams p{*a, dy, h, gain, dh, rstd, dx, dgain, partial};
  const int grid = backward_blocks(a->rows);
  if (a->dtype == FSDP_DTYPE_F32)
    norm_rows_backward<float><<<grid, kNormThreads, 0, st>>>(p);
  else
    norm_rows_backward<__nv_bfloat16><<<grid, kNormThreads, 0, st>>>(p);
  sum_partials<<<static_cast<int>((a->cols + kNormThreads - 1) / kNormThreads), kNormThreads, 0, st>>>(p, grid);
  return cudaGetLastError() == cudaSuccess ? FSDP_OK : FSDP_ECUDA;
}
