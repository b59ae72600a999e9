// Device helpers of the gated delta rule's token path: rows of the state spread
// over LPC adjacent lanes, NV groups of four consecutive states per lane.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace ssm {

// Lanes' values from others by DPP, without the LDS: kCtrl 0xB1 and 0x4E permute
// quads, 0x141 and 0x140 mirror halves of rows and rows of 16, 0x120 + n rotates rows.
template <int kCtrl>
__device__ __forceinline__ float dpp_get(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kCtrl, 0xF, 0xF, true));
}
// x's sum over the lanes' two halves in the lower 32 lanes, y's in the upper
__device__ __forceinline__ float join_halves(float x, float y) {
  const auto u = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(u[0]) + __uint_as_float(u[1]);
}
// x's sums over pairs of rows of 16 lanes in the even rows, y's in the odd
__device__ __forceinline__ float join_rows(float x, float y) {
  const auto u = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(u[0]) + __uint_as_float(u[1]);
}
// Sum over the LPC (1, 2, 4, 8, 16, 32 or 64) adjacent lanes of a row, every lane
// getting it.
template <int LPC>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (LPC == 32) v = join_rows(v, v);
  if constexpr (LPC >= 2) v += dpp_get<0xB1>(v);
  if constexpr (LPC >= 4) v += dpp_get<0x4E>(v);
  if constexpr (LPC >= 8) v += dpp_get<0x141>(v);
  if constexpr (LPC >= 16) v += dpp_get<0x140>(v);
  if constexpr (LPC == 64) v = join_halves(join_rows(v, v), join_rows(v, v));
  return v;
}

// A buffer of that many bytes: loads behind them give 0, stores nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, uint32_t bytes) {
  // the same in all lanes, and said so: a descriptor in vector registers is
  // loaded from in a loop over its values
  bytes = __builtin_amdgcn_readfirstlane(bytes);
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at)));
  const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(hi << 32 | lo), 0, static_cast<int>(bytes),
                                           0x00020000);
}
constexpr uint32_t kNowhere = 0xfffffff0u;  // an offset outside every buffer
template <typename T>
__device__ __forceinline__ T load_one(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  if constexpr (sizeof(T) == 4)
    return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, static_cast<int>(at), 0, 0));
  else
    return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, static_cast<int>(at), 0, 0));
}
__device__ __forceinline__ void store_one(float v, __amdgpu_buffer_rsrc_t r, uint32_t at) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, static_cast<int>(at), 0, 0);
}
__device__ __forceinline__ void store_one(bf16_t v, __amdgpu_buffer_rsrc_t r, uint32_t at) {
  __builtin_amdgcn_raw_buffer_store_b16(v.bits, r, static_cast<int>(at), 0, 0);
}
// Four consecutive elements of a row at byte `at` of the buffer, as they are
// stored: VEC at once, else one by one, up to element n + e < N.
template <bool VEC, typename T>
struct alignas(4 * sizeof(T)) Four {
  T v[4];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at, int n, int64_t N) {
    if constexpr (VEC && sizeof(T) == 4) {
      *this = __builtin_bit_cast(Four, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(at), 0, 0));
    } else if constexpr (VEC) {
      *this = __builtin_bit_cast(Four, __builtin_amdgcn_raw_buffer_load_b64(r, static_cast<int>(at), 0, 0));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = load_one<T>(r, n + e < N ? at + e * static_cast<uint32_t>(sizeof(T)) : kNowhere);
    }
  }
};
// All waves of the workgroup: the LDS alone is waited for, not the loads on their way.
__device__ __forceinline__ void meet_in_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// f(0) .. f(n - 1), the numbers known to the compiler
template <int n, int i = 0, typename F>
__device__ __forceinline__ void each(F &&f) {
  if constexpr (i < n) {
    f(std::integral_constant<int, i>());
    each<n, i + 1>(f);
  }
}
// 1 / sqrt(x): the instruction's, with one step of Newton's
__device__ __forceinline__ float inverse_root(float x) {
  const float r = __builtin_amdgcn_rsqf(x);
  const float s = x * r;  // sqrt(x)
  const float out = fmaf(0.5f * r, fmaf(-s, r, 1.f), r);
  return x < __builtin_huge_valf() ? out : r;  // x = inf: 0, and NaN as it is
}
// A row's value in its lane j of 16, for all of them.
template <int j>
__device__ __forceinline__ float row_lane(float v) {
  return dpp_get<0x150 + j>(v);
}

__device__ __forceinline__ void load4(const float *p, float *v) {
  const float4 f = *reinterpret_cast<const float4 *>(p);
  v[0] = f.x;
  v[1] = f.y;
  v[2] = f.z;
  v[3] = f.w;
}

// A lane's part of a row of N values; states past N read as 0.  VEC: N is a
// multiple of 4 and the row is aligned to four elements.
template <bool VEC, int LPC, int NV>
__device__ __forceinline__ void load_row(const float *p, int lq, int64_t N, float *v) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int n = 4 * (lq + LPC * j);
    if constexpr (VEC) {
      if (n < N) load4(p + n, v + 4 * j);
      else v[4 * j] = v[4 * j + 1] = v[4 * j + 2] = v[4 * j + 3] = 0.f;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * j + e] = n + e < N ? p[n + e] : 0.f;
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

// The products of a row's states: of four at a time, fours 16 lanes apart added so
// that 16 and 32 lanes a row give the same sum to the last bit.
template <int LPC, int NV>
__device__ __forceinline__ float row_dot(const float *x, const float *y) {
  float s[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const float *u = x + 4 * j, *v = y + 4 * j;
    s[j] = fmaf(u[2], v[2], u[0] * v[0]) + fmaf(u[3], v[3], u[1] * v[1]);
  }
  if constexpr (NV == 4) return row_sum<LPC>((s[0] + s[2]) + (s[1] + s[3]));
  if constexpr (NV == 3) return row_sum<LPC>((s[0] + s[2]) + s[1]);
  if constexpr (NV == 2) return row_sum<LPC>(s[0] + s[1]);
  return row_sum<LPC>(s[0]);
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
