// Newton-Schulz orthogonalisation (fsdp_newton_schulz; also the update of
// fsdp_muon_step).
//
// X_0 = G / (|G|_F + eps); per step, with the Gram matrix on the short side,
//   A = X X^T,  X <- a X + (b A + c A^2) X.
#include "newton_schulz.h"
#include "strided.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

namespace fsdp {
namespace {

constexpr int kSumBlocks = 64;

__device__ __forceinline__ float load_source(const void* p, int32_t dtype, int64_t i) {
  return dtype == FSDP_DTYPE_F32 ? static_cast<const float*>(p)[i]
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Sum of squares of a matrix, one partial sum per block.
__global__ void __launch_bounds__(256) ns_squares(const NsJob j, float* partial) {
  __shared__ double shared[8];
  double sum = 0.0;
  for (int64_t r = blockIdx.x; r < j.rows; r += gridDim.x) {
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < j.cols; c += 256) {
      const float v = load_source(j.source, j.dtype, r * j.source_stride + c);
      s += v * v;
    }
    sum += s;
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) sum += shared[i];
    partial[blockIdx.x] = static_cast<float>(sum);
  }
}

__global__ void __launch_bounds__(256) ns_normalise(const NsJob j, const float* partial, float eps, float* x) {
  double sum = 0.0;
  for (int i = 0; i < kSumBlocks; ++i) sum += partial[i];
  const float inv = static_cast<float>(1.0 / (sqrt(sum) + eps));
  for (int64_t r = blockIdx.x; r < j.rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < j.cols; c += 256)
      x[r * j.cols + c] = load_source(j.source, j.dtype, r * j.source_stride + c) * inv;
}

// C = alpha A B + beta D with any strides; 64 x 64 tiles, 4 x 4 per thread.
struct Product {
  const float *a, *b, *d;
  float* c;
  int64_t m, n, k;
  int64_t a_row, a_k, b_k, b_col, c_row;  // element strides (C and D: row stride, unit column stride)
  float alpha, beta;
};

__global__ void __launch_bounds__(256) ns_product(const Product p) {
  __shared__ float sa[16][65], sb[16][65];
  const int64_t i0 = static_cast<int64_t>(blockIdx.y) * 64, j0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.k; k0 += 16) {
    for (int e = threadIdx.x; e < 64 * 16; e += 256) {
      const int kk = e % 16, ii = e / 16;
      const int64_t k = k0 + kk;
      sa[kk][ii] = (k < p.k && i0 + ii < p.m) ? p.a[(i0 + ii) * p.a_row + k * p.a_k] : 0.0f;
      sb[kk][ii] = (k < p.k && j0 + ii < p.n) ? p.b[k * p.b_k + (j0 + ii) * p.b_col] : 0.0f;
    }
    __syncthreads();
    for (int kk = 0; kk < 16; ++kk)
      for (int r = 0; r < 4; ++r)
        for (int c = 0; c < 4; ++c) acc[r][c] += sa[kk][ty * 4 + r] * sb[kk][tx * 4 + c];
    __syncthreads();
  }
  for (int r = 0; r < 4; ++r)
    for (int c = 0; c < 4; ++c) {
      const int64_t i = i0 + ty * 4 + r, j = j0 + tx * 4 + c;
      if (i >= p.m || j >= p.n) continue;
      float v = p.alpha * acc[r][c];
      if (p.d) v += p.beta * p.d[i * p.c_row + j];
      p.c[i * p.c_row + j] = v;
    }
}

int product(const Product& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.n + 63) / 64), static_cast<unsigned>((p.m + 63) / 64));
  ns_product<<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FSDP_OK : FSDP_ECUDA;
}

__global__ void __launch_bounds__(256) ns_output(const NsJob j, const float* x, const __grid_constant__ NsApply ap,
                                                 bool apply) {
  for (int64_t r = blockIdx.x; r < j.rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < j.cols; c += 256) {
      const float o = x[r * j.cols + c];
      if (!apply) {
        j.out[r * j.out_stride + c] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
        continue;
      }
      const int64_t f = j.flat + r * j.cols + c;
      float* master = ap.master[f / ap.shard] + f % ap.shard;
      const float v = *master * ap.keep - j.step * o;
      *master = v;
      ap.full[f] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

int64_t matrix_floats(const NsJob& j) {
  const int64_t k = std::min(j.rows, j.cols);
  return 2 * j.rows * j.cols + 2 * k * k + kSumBlocks;
}

}  // namespace

int ns_plan(const fsdp_newton_schulz_t* h, NsPlan* plan) {
  if (h) {
    if (h->steps < 1 || h->steps > 32 || (h->terms != 0 && h->terms != 1 && h->terms != 3)) return FSDP_EINVAL;
    if (!(h->eps > 0.0) || !std::isfinite(h->eps) || !(static_cast<float>(h->eps) > 0.0f) ||
        !std::isfinite(static_cast<float>(h->eps)))
      return FSDP_EINVAL;
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
      if (std::fabs(b * s + c * s * s) > 60.0) return FSDP_EINVAL;
    }
    if (!(next <= 7.0)) return FSDP_EINVAL;
    top = next;
    for (int k = 0; k < 3; ++k) plan->coef.push_back(static_cast<float>(q[k]));
  }
  return FSDP_OK;
}

int64_t ns_workspace_bytes(const std::vector<NsJob>& jobs, const NsPlan&) {
  int64_t floats = 0;
  for (const NsJob& j : jobs) floats += matrix_floats(j);
  return floats * 4 + 16;
}

int ns_run(const std::vector<NsJob>& jobs, const NsPlan& plan, const NsApply* apply, void* workspace,
           cudaStream_t stream) {
  float* at = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + 15) & ~uintptr_t(15));
  const NsApply none{};
  for (const NsJob& j : jobs) {
    const int64_t m = j.rows, n = j.cols, k = std::min(m, n);
    float *x = at, *y = x + m * n, *gram = y + m * n, *poly = gram + k * k, *partial = poly + k * k;
    at += matrix_floats(j);
    ns_squares<<<kSumBlocks, 256, 0, stream>>>(j, partial);
    const int grid = static_cast<int>(std::min<int64_t>(m, 4096));
    ns_normalise<<<grid, 256, 0, stream>>>(j, partial, plan.eps, x);
    for (int s = 0; s < plan.steps; ++s) {
      const float a = plan.coef[3 * s], b = plan.coef[3 * s + 1], c = plan.coef[3 * s + 2];
      if (m <= n) {
        if (int rc = product({x, x, nullptr, gram, k, k, n, n, 1, 1, n, k, 1.0f, 0.0f}, stream)) return rc;
        if (int rc = product({gram, gram, gram, poly, k, k, k, k, 1, k, 1, k, c, b}, stream)) return rc;
        if (int rc = product({poly, x, x, y, m, n, k, k, 1, n, 1, n, 1.0f, a}, stream)) return rc;
      } else {
        if (int rc = product({x, x, nullptr, gram, k, k, m, 1, n, n, 1, k, 1.0f, 0.0f}, stream)) return rc;
        if (int rc = product({gram, gram, gram, poly, k, k, k, k, 1, k, 1, k, c, b}, stream)) return rc;
        if (int rc = product({x, poly, x, y, m, n, k, n, 1, k, 1, n, 1.0f, a}, stream)) return rc;
      }
      std::swap(x, y);
    }
    ns_output<<<grid, 256, 0, stream>>>(j, x, apply ? *apply : none, apply != nullptr);
    if (cudaGetLastError() != cudaSuccess) return FSDP_ECUDA;
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
} catch (const std::bad_alloc&) {
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
  if (workspace_bytes < ns_workspace_bytes(jobs, plan)) return FSDP_EWORKSPACE;
  const Strided ws{workspace, 1, workspace_bytes, workspace_bytes, 1};
  for (const NsJob& j : jobs)
    if (ws.overlaps({j.source, j.rows, j.cols, j.source_stride, size_of_dtype(j.dtype)}) ||
        ws.overlaps({j.out, j.rows, j.cols, j.out_stride, 2}))
      return FSDP_EALIAS;
  return ns_run(jobs, plan, nullptr, workspace, reinterpret_cast<cudaStream_t>(stream));
} catch (const std::bad_alloc&) {
  return FSDP_ECUDA;
}
