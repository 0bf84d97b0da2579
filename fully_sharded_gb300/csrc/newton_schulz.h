// Newton-Schulz orthogonalisation of a list of matrices: the part shared by
// fsdp_newton_schulz and fsdp_muon_step (host interface). Not public.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <vector>

#include "fsdp.h"

namespace fsdp {

// One matrix: where it is read, and where its result goes. Plain
// orthogonalisation writes bf16 to `out`; with an NsApply the result updates the
// master elements [flat, flat + rows * cols) of a unit instead.
struct NsJob {
  const void* source;
  int64_t source_stride;
  int64_t rows, cols;
  uint16_t* out;
  int64_t out_stride;
  int64_t flat;
  float step;      // lr * scale
  int32_t dtype;
};

struct NsApply {
  float* master[FSDP_MAX_WORLD];
  uint16_t* full;
  int64_t shard;  // S: element f of the unit is master[f / S][f % S]
  float keep;     // 1 - lr * weight_decay
};

// The step's first part, where the matrices are a unit's momentum updates: the
// pass that sums squares also folds the gradients and updates the momentum, and
// writes each u to its job's (fp32, contiguous) source.
struct NsMomentum {
  const uint16_t* grads[FSDP_MAX_WORLD];
  float* momentum[FSDP_MAX_WORLD];
  int64_t shard;
  int32_t w;
  float mu;
  float inv_w;  // 1 / W where W is a power of two, else 0
  int32_t nesterov;
};

// The checked parameters of a call.
struct NsPlan {
  int steps = 5;
  int terms = 0;
  float eps = 1e-7f;
  std::vector<float> coef;  // a, b, c per step
};

int ns_plan(const fsdp_newton_schulz_t* h, NsPlan* plan);
int64_t ns_workspace_bytes(const std::vector<NsJob>& jobs, const NsPlan& plan);
int ns_run(const std::vector<NsJob>& jobs, const NsPlan& plan, const NsMomentum* momentum, const NsApply* apply,
           void* workspace, cudaStream_t stream);

}  // namespace fsdp
