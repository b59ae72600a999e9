// Launcher interface of the group norm with an activation (group_norm.hip).
// The arguments are validated by the C ABI before the launch.
#pragma once

#include "launch.h"

namespace ssm {

struct NormArgs {
  int64_t S, T, D, G;   // statistics over T tokens x D / G channels
  DType dt;
  const void *x;        // (S, T, D)
  const void *z;        // (S, T, D) or null: the gate
  const float *w, *b;   // (D) or null
  float eps;
  bool center;          // subtract the mean
  bool act;             // SiLU of the normalised value
  bool gate_first;      // x silu(z) is normalised; else the result is multiplied
  void *y;
  float *mean, *rstd;   // (S, G): written by the forward (may be null), read by
                        // the backward (mean null where not centred)
  // backward
  const void *dy;
  void *dx, *dz;        // dz null without z
  float *dw, *db;       // (D) or null
  float *ws;
};

// Floats of workspace: of this call (its type and alignment choose the path), and
// the most that a call of these sizes takes.
int64_t group_norm_fwd_ws_floats(const NormArgs &a);
int64_t group_norm_bwd_ws_floats(const NormArgs &a);
int64_t group_norm_fwd_ws_floats(int64_t S, int64_t T, int64_t D, int64_t G);
int64_t group_norm_bwd_ws_floats(int64_t S, int64_t T, int64_t D, int64_t G);
hipError_t launch_group_norm_fwd(const NormArgs &a, hipStream_t s);
hipError_t launch_group_norm_bwd(const NormArgs &a, hipStream_t s);

}  // namespace ssm
