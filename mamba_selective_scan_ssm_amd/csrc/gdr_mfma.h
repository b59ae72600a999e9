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

#include "gdr_common.h"

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
// differences are exact): three hold all 24 bits.
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


// ------------------------------------------------------------ chunks
constexpr int kC = 64;          // tokens per chunk
constexpr int kCols = 64;       // columns per workgroup

// X, [i][j] by kpos(j): rows 0..31 meet 32 tokens, rows 32..63 all 64;
// 16 bytes of padding put 16 rows on different banks.
constexpr int kTriSize = 32 * 40 + 32 * 72;
__device__ __forceinline__ constexpr int tri_at(int i) { return i < 32 ? i * 40 : 32 * 40 + (i - 32) * 72; }
// M the same without the padding, for which the LDS has no room: the 16-byte pieces
// `ch` (kpos / 8) of a row are exchanged by the row, so that one piece of eight rows
// lies on 32 banks.
constexpr int kMixSize = 32 * 32 + 32 * 64;
__device__ __forceinline__ constexpr int mix_at(int i, int ch) {
  return i < 32 ? i * 32 + 8 * (ch ^ (i / 2 % 4)) : 32 * 32 + (i - 32) * 64 + 8 * (ch ^ (i % 8));
}
// 16-byte piece `ch` (kpos / 8) of token `tok` in a K or Q tile.  Eight lanes
// of an operand read (eight rows, one piece) and sixteen of a transposing one
// (four rows by four pieces, half of each) share a cycle: the pieces of a row
// are exchanged by the row so that the former meet 32 banks and the latter as
// many as their halves allow.
template <int NT>
__device__ __forceinline__ int tile_at(int tok, int ch) {
  const int f = 4 * (tok % 2) + tok / 2 % 4 + (NT == 8 ? 8 * (tok / 8 % 2) : 0);
  return tok * 16 * NT + 8 * (ch ^ f);
}

// LDS by address.  A lane keeps the few addresses it reads around (`hold` hides
// how they were formed, or the compiler keeps one per read) and the rest is in
// the instructions' offsets, 16 bits each.
typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_char *)(p)));
}
__device__ __forceinline__ uint32_t hold(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}
template <typename T>
__device__ __forceinline__ T lds_get(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T *>(at);
}
template <typename T>
__device__ __forceinline__ void lds_put(uint32_t at, T v) {
  *reinterpret_cast<__attribute__((address_space(3))) T *>(at) = v;
}
// Four values of 4 rows by 16 columns, transposed on their way out of LDS: lane
// 16 g + i names the 8 bytes (row i / 4, columns 4 (i % 4) .. + 3) of its group
// and lane 16 g + r receives column r of the 4 rows.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 lds_transposed(uint32_t at) {
  return __builtin_bit_cast(
      u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<__attribute__((address_space(3))) s16x4 *>(at)));
}

// Rows t0 .. of a (.., rows, row elements) tensor of 16-bit values from one
// element on: reads behind the last row give 0 and writes there are dropped.
// `left` rows from t0 (0 and less: none), of which `tail` elements count in the
// last.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void *base, int left, uint32_t row, uint32_t tail) {
  return buffer_of(base, left > 0 ? 2 * (static_cast<uint32_t>(left - 1) * row + tail) : 0);
}
__device__ __forceinline__ u32x4 buffer_b128(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t more = 0) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(at), static_cast<int>(more), 0));
}

// exp2 of a difference of two cumulative decays
__device__ __forceinline__ float decay_of(double d) { return fast_exp2(static_cast<float>(d)); }

// Inclusive sum over the 64 lanes in 64 bits: shifts by 1, 2, 4, 8 within rows
// of 16 lanes (0 where there is no source), then the rows' ends.
template <int kCtrl>
__device__ __forceinline__ double dpp_shift(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<uint32_t>(u), kCtrl, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<uint32_t>(u >> 32), kCtrl, 0xf, 0xf, true);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(u), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(u >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// Inclusive sums within rows of 16 lanes, from the first lane on and from the
// last one back.
__device__ __forceinline__ double row_prefix(double v) {
  v += dpp_shift<0x111>(v);
  v += dpp_shift<0x112>(v);
  v += dpp_shift<0x114>(v);
  v += dpp_shift<0x118>(v);
  return v;
}
__device__ __forceinline__ double row_suffix(double v) {
  v += dpp_shift<0x101>(v);
  v += dpp_shift<0x102>(v);
  v += dpp_shift<0x104>(v);
  v += dpp_shift<0x108>(v);
  return v;
}
__device__ __forceinline__ double wave_scan(double v) {
  v = row_prefix(v);
  const double e0 = lane_value(v, 15), e1 = lane_value(v, 31), e2 = lane_value(v, 47);
  const int row = threadIdx.x % 64 / 16;
  if (row >= 1) v += row == 1 ? e0 : row == 2 ? e0 + e1 : e0 + e1 + e2;
  return v;
}
// Sums over the lanes before this one, and over this one and those behind it:
// sums alone, so that nothing is left where there is nothing to add.
__device__ __forceinline__ double wave_before(double v) {
  const double in = row_prefix(v), e0 = lane_value(in, 15), e1 = lane_value(in, 31), e2 = lane_value(in, 47);
  const int row = threadIdx.x % 64 / 16;
  return dpp_shift<0x111>(in) + (row == 0 ? 0.0 : row == 1 ? e0 : row == 2 ? e0 + e1 : e0 + e1 + e2);
}
__device__ __forceinline__ double wave_from(double v) {
  const double in = row_suffix(v), e1 = lane_value(in, 16), e2 = lane_value(in, 32), e3 = lane_value(in, 48);
  const int row = threadIdx.x % 64 / 16;
  return in + (row == 3 ? 0.0 : row == 2 ? e3 : row == 1 ? e2 + e3 : e1 + e2 + e3);
}

}  // namespace ssm
