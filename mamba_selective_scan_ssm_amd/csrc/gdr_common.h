// Device helpers of the gated delta rule's token path: rows of the state spread
// over LPC adjacent lanes, NV groups of four consecutive states per lane.
#pragma once

#include "device_common.h"

namespace ssm {

// Sum over the LPC (1, 2, 4, 8 or 16) adjacent lanes of a row, every lane
// getting it: DPP quad permutations, then mirrors within half rows and rows.
template <int kCtrl>
__device__ __forceinline__ float dpp_get(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kCtrl, 0xF, 0xF, true));
}
template <int LPC>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (LPC >= 2) v += dpp_get<0xB1>(v);
  if constexpr (LPC >= 4) v += dpp_get<0x4E>(v);
  if constexpr (LPC >= 8) v += dpp_get<0x141>(v);
  if constexpr (LPC >= 16) v += dpp_get<0x140>(v);
  return v;
}

__device__ __forceinline__ void load4(const float *p, float *v) {
  const float4 f = *reinterpret_cast<const float4 *>(p);
  v[0] = f.x;
  v[1] = f.y;
  v[2] = f.z;
  v[3] = f.w;
}
__device__ __forceinline__ void load4(const bf16_t *p, float *v) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xffff0000u);
}

// A lane's part of a row of N values; states past N read as 0.  VEC: N is a
// multiple of 4 and the row is aligned to four elements.
template <bool VEC, int LPC, int NV, typename T>
__device__ __forceinline__ void load_row(const T *p, int lq, int64_t N, float *v) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int n = 4 * (lq + LPC * j);
    if constexpr (VEC) {
      if (n < N) load4(p + n, v + 4 * j);
      else v[4 * j] = v[4 * j + 1] = v[4 * j + 2] = v[4 * j + 3] = 0.f;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * j + e] = n + e < N ? to_f32(p[n + e]) : 0.f;
    }
  }
}
// The same in the tensor's own type.
template <bool VEC, int LPC, int NV, typename T>
__device__ __forceinline__ void load_raw(const T *p, int lq, int64_t N, T *v) {
  struct alignas(4 * sizeof(T)) Four {
    T v[4];
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int n = 4 * (lq + LPC * j);
    Four f = {};
    if constexpr (VEC) {
      if (n < N) f = *reinterpret_cast<const Four *>(p + n);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < N) f.v[e] = p[n + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * j + e] = f.v[e];
  }
}
template <bool VEC, int LPC, int NV>
__device__ __forceinline__ void store_row(float *p, int lq, int64_t N, const float *v) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int n = 4 * (lq + LPC * j);
    if constexpr (VEC) {
      if (n < N) *reinterpret_cast<float4 *>(p + n) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < N) p[n + e] = v[4 * j + e];
    }
  }
}
// The same part of a padded row in LDS.
template <int LPC, int NV>
__device__ __forceinline__ void lds_row(const float *p, int lq, float *v) {
#pragma unroll
  for (int j = 0; j < NV; ++j) load4(p + 4 * (lq + LPC * j), v + 4 * j);
}

template <int LPC, int NV>
__device__ __forceinline__ float row_dot(const float *x, const float *y) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int i = 0; i < 4 * NV; i += 2) {
    s0 = fmaf(x[i], y[i], s0);
    s1 = fmaf(x[i + 1], y[i + 1], s1);
  }
  return row_sum<LPC>(s0 + s1);
}

// One token of one row: S <- a S + (beta e rk) k with e = v - a rk (S . k);
// returns rq (S . q).
template <int LPC, int NV>
__device__ __forceinline__ float gdr_token(float *S, const float *k, const float *q, float v, float a, float beta,
                                           float rk, float rq) {
  const float e = fmaf(-(a * rk), row_dot<LPC, NV>(S, k), v);
  const float u = beta * e * rk;
#pragma unroll
  for (int i = 0; i < 4 * NV; ++i) S[i] = fmaf(a, S[i], u * k[i]);
  return rq * row_dot<LPC, NV>(S, q);
}

}  // namespace ssm
