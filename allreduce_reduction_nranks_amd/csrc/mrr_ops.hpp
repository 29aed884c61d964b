// mrr_ops.hpp -- argument blocks and launchers of the operators that follow
// the rank sum in a training step: layer norm and sharded cross entropy.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mrr.h"

namespace mrr {

// ---- layer norm of a rank sum -------------------------------------------------
struct NormFwdArgs {
  const void* in[MRR_MAX_RANKS];
  const void* residual;  // may be null
  const void* weight;    // may be null: 1
  const void* bias;      // may be null: 0
  void* sum;             // may be null
  void* out;
  float* mean;           // may be null
  float* rstd;           // may be null
  uint64_t rows, ld_in, ld_out;
  uint32_t cols;
  int nranks;
  float eps;
  int wf32;              // weight and bias are f32 (otherwise the data type)
};

struct NormBwdArgs {
  const void* dout;
  const void* sum;
  const void* weight;     // may be null: 1
  const float* mean;
  const float* rstd;
  const void* dresidual;  // may be null
  void* dsum;             // may be null
  void* dweight;          // may be null
  void* dbias;            // may be null
  float* partial;         // [groups][2][cols]: dweight and dbias of a group of rows
  uint64_t rows, ld_in, ld_out;
  uint32_t cols;
  uint32_t groups;
  int wf32;
};

// Groups of rows whose weight gradients are summed apart, for a call of this shape.
uint32_t norm_bwd_groups(uint64_t rows, uint32_t cols);
hipError_t launch_norm_fwd(const NormFwdArgs& a, int t, hipStream_t stream);
hipError_t launch_norm_bwd(NormBwdArgs a, int t, hipStream_t stream);

}  // namespace mrr
