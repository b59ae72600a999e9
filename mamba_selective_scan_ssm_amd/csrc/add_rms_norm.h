// Launcher interface of the root-mean-square norm with the residual's addition
// (add_rms_norm.hip).  The arguments are validated by the C ABI before the launch.
#pragma once

#include "launch.h"

namespace ssm {

constexpr int kAddNormLeastGroup = 8;  // channels of a scale
constexpr float kE4m3Max = 448.f, kInt8Max = 127.f;
constexpr float kLeastScale = 7.888609052210118e-31f;  // 2^-100

struct AddNormArgs {
  int64_t rows, D;
  DType dt, stream;       // of x, y, dy, dx; of residual, h, dh, dresidual
  const void *x, *residual;
  const float *w;         // (D) or null: ones
  float eps;
  int quant;              // 0: y in dt; 1: e4m3; 2: int8
  int64_t group;          // channels of a scale
  void *h, *y;
  float *scale;           // (rows, D / group)
  float *rstd;            // (rows) or null
  // backward
  const void *dy, *dh;    // dh may be null
  void *dx, *dresidual;   // either may be null
  float *dw;              // or null
  float *ws;
};

hipError_t launch_add_norm_fwd(const AddNormArgs &a, hipStream_t s);
int64_t add_norm_bwd_ws_floats(int64_t rows, int64_t D);
hipError_t launch_add_norm_bwd(const AddNormArgs &a, hipStream_t s);

}  // namespace ssm
