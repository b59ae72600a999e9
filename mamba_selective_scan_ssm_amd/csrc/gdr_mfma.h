// Matrix-core helpers of the gated delta rule's chunked kernels.
//
// v_mfma_f32_16x16x32_bf16 on lane l = 16 g + r: A holds A[r][k], B holds
// B[k][r] for the 8 values k of slot (g, 0..7), the result C[4 g + e][r].  The
// contraction may be taken in any order, so slot (g, 4 u + e) is made to stand
// for k = 16 u + 4 g + e: two result tiles, one above the other, then are a B
// operand lane by lane, and a chain of products keeps its 16 columns in the
// registers of one wave.  Operands in LDS are stored in that order (kpos), so
// that a slot's 8 values are 16 consecutive bytes.
#pragma once

#include "device_common.h"

namespace ssm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
// v_mfma_f32_16x16x4_f32: A[r][g], B[g][r]; with k = 4 g + s in step s a result
// tile is a B operand here too.
__device__ __forceinline__ f32x4 mma_f32(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
  for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
  return c;
}

// Position of contraction index k (a multiple of 4) in an LDS row.
__device__ __forceinline__ constexpr int kpos(int k) { return (k & ~31) + 8 * ((k >> 2) & 3) + 4 * ((k >> 4) & 1); }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {  // rounded to nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
// v less the low (or high) bf16 of a pair: v_dot2_f32_bf16 with -1 and 0, one
// instruction in place of an unpacking and a subtraction, and exact (checked
// over 2^20 values of all exponents).  The constants are kept from the
// compiler, which would write them as the inline constant -1.0, another value.
struct MinusOne {
  uint32_t low = 0x0000bf80u, high = 0xbf800000u;
  __device__ __forceinline__ MinusOne() { asm volatile("" : "+s"(low), "+s"(high)); }
};
__device__ __forceinline__ float less_half(float v, uint32_t pair, uint32_t minus) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, minus), v, false);
}
// fp32 as a sum of NP bf16 parts, each the rounded rest of those before it (the
// differences are exact): three hold all 24 bits; two leave out at most 2^-16
// of the value, and 3e-6 of it on the average.
template <int NP>
__device__ __forceinline__ void split4(f32x4 v, u32x2 *out, const MinusOne &m) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    out[p] = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    if (p + 1 < NP)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = less_half(v[e], out[p][e / 2], e & 1 ? m.high : m.low);
  }
}
// Two result tiles as a B operand of 32 contraction indices, in NP parts.
template <int NP>
__device__ __forceinline__ void split_operand(f32x4 top, f32x4 bottom, u32x4 *out, const MinusOne &m) {
  u32x2 a[NP], b[NP];
  split4<NP>(top, a, m);
  split4<NP>(bottom, b, m);
#pragma unroll
  for (int p = 0; p < NP; ++p) out[p] = u32x4{a[p][0], a[p][1], b[p][0], b[p][1]};
}

}  // namespace ssm
