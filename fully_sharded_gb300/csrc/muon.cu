// fsdp_muon_step: the step of one unit whose matrices are updated along their
// orthogonalised momentum, its other tensors by Adam.
//
// Matrices: g = fold of the W gradients / W (fp32, rank order), m = mu m + g,
// u = g + mu m (Nesterov) or m; then the Newton-Schulz products on u, whose
// last one updates the master shards and writes the gathered bf16 parameters.
// Other tensors and the padding: segments of the Adam step (segment_kernel.cuh).
#include "host_internal.h"
#include "newton_schulz.h"
#include "strided.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

namespace fsdp {
namespace {

struct Muon {
  std::vector<NsJob> jobs;
  SegmentList adam;
  NsPlan plan;
  NsApply apply{};
  Scalars scalars{};
  int64_t u_elems = 0;

  int64_t bytes() const { return jobs.empty() ? 0 : u_elems * 4 + 16 + ns_workspace_bytes(jobs, plan); }
};

// Checks the unit and the hyper-parameters and lists the work. `pointers`
// false: sizes only.
int make(const fsdp_muon_unit_t* unit, const fsdp_muon_t* h, bool pointers, Muon* out) {
  if (!unit || !h || !layout_ok(unit->layout) || !unit->tensors) return FSDP_EINVAL;
  const fsdp_layout_t& L = *unit->layout;
  if (L.shard_factor != L.world_size) return FSDP_EINVAL;
  const int W = L.world_size;
  const int64_t S = L.shard_numel, padded = L.padded_numel;
  if (!std::isfinite(h->lr) || !std::isfinite(h->weight_decay) || !(h->momentum >= 0.0 && h->momentum < 1.0))
    return FSDP_EINVAL;
  if (int rc = make_scalars(&h->adam, W, &out->scalars)) return rc;
  if (int rc = ns_plan(h->newton_schulz, &out->plan)) return rc;
  AliasCheck alias;
  if (pointers && padded > 0) {
    if (!unit->grads || !unit->master || !unit->exp_avg || !unit->exp_avg_sq || !unit->full_out) return FSDP_EINVAL;
    alias.output(unit->full_out, padded * 2);
    for (int k = 0; k < W; ++k) {
      float* state[] = {unit->master[k], unit->exp_avg[k], unit->exp_avg_sq[k]};
      if (!unit->grads[k] || reinterpret_cast<uintptr_t>(unit->grads[k]) % 2) return FSDP_EINVAL;
      alias.input(unit->grads[k], padded * 2);
      for (float* q : state) {
        if (!q || reinterpret_cast<uintptr_t>(q) % 4) return FSDP_EINVAL;
        alias.output(q, S * 4);
      }
      out->apply.master[k] = unit->master[k];
    }
    if (reinterpret_cast<uintptr_t>(unit->full_out) % 2) return FSDP_EINVAL;
    if (!alias.ok()) return FSDP_EALIAS;
  }
  out->apply.full = unit->full_out;
  out->apply.shard = S;
  out->apply.keep = static_cast<float>(1.0 - h->lr * h->weight_decay);
  // Adam segments: [begin, end) of the unit, cut at the shards' ends
  auto adam = [&](int64_t begin, int64_t end) {
    while (pointers && begin < end) {
      const int64_t r = begin / S, stop = std::min(end, (r + 1) * S), at = begin - r * S;
      std::vector<const void*> ptrs;
      for (int k = 0; k < W; ++k) ptrs.push_back(unit->grads[k] + begin);
      ptrs.insert(ptrs.end(), {unit->master[r] + at, unit->exp_avg[r] + at, unit->exp_avg_sq[r] + at,
                               unit->full_out + begin});
      out->adam.add_elementwise(kStep, stop - begin, 1, ptrs);
      begin = stop;
    }
  };
  int64_t flat = 0, pending = 0;  // [pending, flat): not yet listed Adam elements
  for (int32_t i = 0; i < L.n_tensors; ++i) {
    const fsdp_muon_tensor_t& t = unit->tensors[i];
    if (t.rows < 0 || t.cols < 0) return FSDP_EINVAL;
    const int64_t left = L.numel - flat;
    if (t.rows > (t.cols == 0 ? left : left / t.cols)) return FSDP_EINVAL;
    if (t.cols == 0) {
      flat += t.rows;
      continue;
    }
    if (t.rows > (int64_t(1) << 30) || t.cols > (int64_t(1) << 30) || !std::isfinite(t.scale)) return FSDP_EINVAL;
    if (t.rows > 0) {
      adam(pending, flat);
      out->jobs.push_back({nullptr, t.cols, t.rows, t.cols, nullptr, 0, flat, static_cast<float>(h->lr * t.scale),
                           FSDP_DTYPE_F32});
      // each u starts at its place in the unit modulo 8, so that groups of 8 elements
      // are aligned in both
      out->u_elems += (t.rows * t.cols + 7) / 8 * 8 + 8;
      flat += t.rows * t.cols;
      pending = flat;
    }
  }
  if (flat != L.numel) return FSDP_EINVAL;
  adam(pending, padded);
  return FSDP_OK;
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" int fsdp_muon_workspace(const fsdp_muon_unit_t* unit, const fsdp_muon_t* muon, int64_t* bytes_out) try {
  if (!bytes_out) return FSDP_EINVAL;
  Muon m;
  if (int rc = make(unit, muon, false, &m)) return rc;
  *bytes_out = m.bytes();
  return FSDP_OK;
} catch (...) {
  return FSDP_ECUDA;
}

extern "C" int fsdp_muon_step(const fsdp_muon_unit_t* unit, const fsdp_muon_t* h, void* workspace,
                              int64_t workspace_bytes, fsdp_stream_t stream) try {
  Muon m;
  if (int rc = make(unit, h, true, &m)) return rc;
  if (unit->layout->padded_numel == 0) return FSDP_OK;
  const int64_t need = m.bytes();
  if (need > 0 && !workspace) return FSDP_EINVAL;
  if (workspace_bytes < need) return FSDP_EWORKSPACE;
  const int W = unit->layout->world_size;
  const int64_t S = unit->layout->shard_numel, padded = unit->layout->padded_numel;
  if (need > 0) {
    const Strided ws{workspace, 1, need, need, 1};
    if (ws.overlaps({unit->full_out, 1, padded, padded, 2})) return FSDP_EALIAS;
    for (int k = 0; k < W; ++k)
      if (ws.overlaps({unit->grads[k], 1, padded, padded, 2}) || ws.overlaps({unit->master[k], 1, S, S, 4}) ||
          ws.overlaps({unit->exp_avg[k], 1, S, S, 4}) || ws.overlaps({unit->exp_avg_sq[k], 1, S, S, 4}))
        return FSDP_EALIAS;
  }
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (int rc = launch(m.adam, m.scalars, st)) return rc;
  if (m.jobs.empty()) return FSDP_OK;
  float* u = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + 15) & ~uintptr_t(15));
  void* rest = u + m.u_elems;
  for (NsJob& j : m.jobs) {
    j.source = u + j.flat % 8;
    u += (j.rows * j.cols + 7) / 8 * 8 + 8;
  }
  NsMomentum p{};
  for (int k = 0; k < W; ++k) {
    p.grads[k] = unit->grads[k];
    p.momentum[k] = unit->exp_avg[k];
  }
  p.shard = S;
  p.w = W;
  p.mu = static_cast<float>(h->momentum);
  p.inv_w = m.scalars.inv_w;
  p.nesterov = h->nesterov != 0;
  return ns_run(m.jobs, m.plan, &p, &m.apply, rest, st);
} catch (...) {
  return FSDP_ECUDA;
}
