// Root-mean-square norm with the residual's addition, an output in 8 bits, and
// the gradients.
//
// Per row of D channels:
//   h = round(x + residual) in the stream's type,  r = 1 / sqrt(mean(h^2) + eps)
//   y = h r w;  in 8 bits: scale = max |y| / most over a group, q = round(y / scale)
// and for dy and the stream's own gradient dh:
//   u = dy w,  dx = dresidual = r (u - h r^2 mean(u h)) + dh,  dw = sum over rows of dy h r
//
// THREADS threads hold a row in registers, NP pieces of eight consecutive channels
// each, so up to 16384 channels everything is read and written once: a wave where rows are
// many and at most 4096 wide (no barrier), 256 threads for few rows or up to 16384, else
// 1024.  NP is what the row has, not a power of two: 2560 channels are 5 pieces and not 8.
// Of 1024 threads each has 128 registers, which the row and the weights fill: wider rows
// pass through scratch memory too (208 to 645 registers a thread, by types and pass): 2048 x
// 32768 of bf16 222 us forward (2.4 TB/s), 339 in 8 bits, 1136 backward, where 4096 x 16384
// take 144, 128 and 253.
// Bound by bytes: 32768 x 2560 bf16, stream in bf16, 143 us (4.7 TB/s); 16384 x 5120 with
// the stream in fp32 and an output of e4m3 by 128 channels 182 us (5.1 TB/s, what a copy
// of 1 GiB by copy_ reaches); forward and backward of 8192 x 2560, stream in fp32, 123 us
// (kernels of 53, 64 and, for the sums of dw, 5; 4.8 TB/s).  256 rows in 8 bits take 5 us of
// kernel, one row 3, in calls of 9 to 12.  Rows that are no whole 16 bytes: 8000 x 2001 fp32 41 us (6.3 TB/s,
// partly from the cache), bf16 78 (1.7: two bytes a lane and load).
#include "add_rms_norm.h"
#include "device_common.h"
#include "gdr_common.h"

namespace ssm {
namespace {

constexpr int64_t kCus = 256;
constexpr int kLeastGroup = kAddNormLeastGroup;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Channel e of a thread's piece i: pieces are eight consecutive channels where rows are
// whole 16 bytes (VEC), else a channel of each thread after another's, so that a wave's
// single elements lie side by side all the same.
template <bool VEC, int THREADS>
__device__ __forceinline__ int channel_of(int tid, int i, int e) {
  return VEC ? 8 * (tid + THREADS * i) + e : tid + THREADS * (8 * i + e);
}
// A piece of a row; channels behind D are 0.
template <typename T, bool VEC, int THREADS>
__device__ __forceinline__ void load8(const T *row, int tid, int i, int D, float *v) {
  if constexpr (VEC) {  // D is a multiple of 8
    struct alignas(16) Raw {
      T v[16 / sizeof(T)];
    };
    constexpr int kEach = 16 / sizeof(T);
    const int n = channel_of<VEC, THREADS>(tid, i, 0);
    if (n < D) {
#pragma unroll
      for (int q = 0; q < 8 / kEach; ++q) {
        const Raw x = *reinterpret_cast<const Raw *>(row + n + q * kEach);
#pragma unroll
        for (int e = 0; e < kEach; ++e) v[q * kEach + e] = to_f32(x.v[e]);
      }
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = channel_of<VEC, THREADS>(tid, i, e);
      v[e] = n < D ? to_f32(row[n]) : 0.f;
    }
  }
}
template <typename T, bool VEC, int THREADS>
__device__ __forceinline__ void store8(T *row, int tid, int i, int D, const float *v) {
  if constexpr (VEC) {
    const int n = channel_of<VEC, THREADS>(tid, i, 0);
    if (n >= D) return;
    constexpr int kEach = 16 / sizeof(T);
    struct alignas(16) Raw {
      T v[kEach];
    };
#pragma unroll
    for (int q = 0; q < 8 / kEach; ++q) {
      Raw x;
#pragma unroll
      for (int e = 0; e < kEach; ++e) x.v[e] = from_f32<T>(v[q * kEach + e]);
      *reinterpret_cast<Raw *>(row + n + q * kEach) = x;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = channel_of<VEC, THREADS>(tid, i, e);
      if (n < D) row[n] = from_f32<T>(v[e]);
    }
  }
}

// Sum over the row's threads, all of them getting it; s: a float for each wave.
template <int THREADS>
__device__ __forceinline__ float threads_sum(float v, float *s) {
  v = row_sum<64>(v);
  if constexpr (THREADS > 64) {
    __syncthreads();
    if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) v += s[i];
  }
  return v;
}
// The largest over adjacent lanes of an 8-, 16-, 32- or 64-lane span (1, 2, 4 too).
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int span) {
  for (int d = 1; d < span; d *= 2) {
    const uint32_t o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}

// Four values to e4m3, to nearest even
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

// Eight values in 8 bits: to nearest even, NaN to NaN (e4m3) or 0 (int8).
template <bool VEC, int THREADS>
__device__ __forceinline__ void store8_quant(uint8_t *row, int tid, int piece, int D, const float *u, bool e4m3) {
  uint32_t q[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (e4m3) {
      q[i] = pack_e4m3(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
    } else {
      q[i] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // a NaN is neither below nor above: taken as 0
        const float a = u[4 * i + e], t = a > -128.f && a < 128.f ? a : 0.f;
        q[i] |= (static_cast<uint32_t>(static_cast<int>(__builtin_rintf(t))) & 0xffu) << (8 * e);
      }
    }
  }
  if constexpr (VEC) {
    const int n = channel_of<VEC, THREADS>(tid, piece, 0);
    if (n < D) *reinterpret_cast<u32x2_t *>(row + n) = u32x2_t{q[0], q[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = channel_of<VEC, THREADS>(tid, piece, e);
      if (n < D) row[n] = static_cast<uint8_t>(q[e / 4] >> (8 * (e % 4)));
    }
  }
}

// The scale of values whose largest has these bits.  NaN has bits above infinity's, and
// stays.
__device__ __forceinline__ float scale_of(uint32_t bits, float most) {
  const float s = __uint_as_float(bits) / most;
  return s < kLeastScale ? kLeastScale : s;
}

// Eight values divided by the scale of their group, each rounded once: times the rounded
// 1 / s, and what that lacks of the value (an fma has it exactly) times 1 / s once more,
// which rounds as the division does (Markstein's theorem).  Outside of these scales what is
// lacking can fall below the least number, or 1 / s is none.  16384 x 5120 by 128 channels
// 185 us, by divisions 188, times 1 / s alone (one e4m3 in 2^19 a step off) 184; 32768 x
// 2560 in bf16 by 64 channels 144, 150 and 142.
__device__ __forceinline__ void divide8(float *v, float s) {
  const float inverse = 1.f / s;
  if (s > 0x1p-90f && s < __builtin_huge_valf()) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q = v[e] * inverse;
      v[e] = fmaf(fmaf(-q, s, v[e]), inverse, q);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] /= s;
  }
}

// kRows rows a workgroup at a time, a wave each where THREADS is 64.  QUANT 0: none;
// 1: a scale for each token, or for groups that lie on a power of two of adjacent
// lanes; 2: any other groups, their largest kept in LDS.
template <typename X, typename H, bool VEC, int NP, int THREADS, int QUANT>
__global__ __launch_bounds__(THREADS == 64 ? 256 : THREADS) void add_norm_kernel(AddNormArgs a) {
  constexpr int kRows = THREADS == 64 ? 4 : 1, kWaves = THREADS / 64;
  __shared__ float s_sum[kWaves];
  __shared__ uint32_t s_top[kWaves];
  __shared__ uint32_t s_max[QUANT == 2 ? 8 * NP * THREADS / kLeastGroup : 1];
  const int D = static_cast<int>(a.D), tid = threadIdx.x % THREADS;
  const int sub = kRows == 1 ? 0 : threadIdx.x / THREADS;
  const X *x = static_cast<const X *>(a.x);
  const H *res = static_cast<const H *>(a.residual);
  const int groups = QUANT ? static_cast<int>(a.D / a.group) : 1, group = QUANT ? static_cast<int>(a.group) : D;
  const bool e4m3 = a.quant == 1;
  const float most = e4m3 ? kE4m3Max : kInt8Max;
  float w[NP][8];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (a.w != nullptr) {
      load8<float, VEC, THREADS>(a.w, tid, i, D, w[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = 1.f;
    }
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t at = row * D;
    float v[NP][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) load8<X, VEC, THREADS>(x + at, tid, i, D, v[i]);
    if (res != nullptr) {
      float o[NP][8];
#pragma unroll
      for (int i = 0; i < NP; ++i) load8<H, VEC, THREADS>(res + at, tid, i, D, o[i]);
      // h may be the residual itself: it is written where it has been read
#pragma unroll
      for (int i = 0; i < NP; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = to_f32(from_f32<H>(v[i][e] + o[i][e]));
        store8<H, VEC, THREADS>(static_cast<H *>(a.h) + at, tid, i, D, v[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    const float r = inverse_root(threads_sum<THREADS>(ss, s_sum) / static_cast<float>(D) + a.eps);
    if (a.rstd != nullptr && tid == 0) a.rstd[row] = r;
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * r * w[i][e];
    if constexpr (QUANT == 0) {
#pragma unroll
      for (int i = 0; i < NP; ++i) store8<X, VEC, THREADS>(static_cast<X *>(a.y) + at, tid, i, D, v[i]);
    } else {
      uint8_t *q = static_cast<uint8_t *>(a.y) + at;
      float *scale = a.scale + row * groups;
      uint32_t top[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        top[i] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t b = __float_as_uint(v[i][e]) & 0x7fffffffu;
          top[i] = b > top[i] ? b : top[i];
        }
      }
      if constexpr (QUANT == 2) {
        __syncthreads();  // the row before has been read
        for (int i = tid; i < groups; i += THREADS) s_max[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int n = channel_of<VEC, THREADS>(tid, i, e);
            if (n < D) atomicMax(&s_max[n / group], __float_as_uint(v[i][e]) & 0x7fffffffu);
          }
        __syncthreads();
        for (int i = tid; i < groups; i += THREADS) scale[i] = scale_of(s_max[i], most);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          float u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int n = channel_of<VEC, THREADS>(tid, i, e);
            u[e] = n < D ? v[i][e] / scale_of(s_max[n / group], most) : 0.f;
          }
          store8_quant<VEC, THREADS>(q, tid, i, D, u, e4m3);
        }
      } else if (groups == 1) {
        uint32_t all = top[0];
#pragma unroll
        for (int i = 1; i < NP; ++i) all = top[i] > all ? top[i] : all;
        all = lanes_max(all, 64);
        if constexpr (THREADS > 64) {
          // the sum's barriers have passed since these were read
          if (tid % 64 == 0) s_top[tid / 64] = all;
          __syncthreads();
#pragma unroll
          for (int i = 0; i < kWaves; ++i) all = s_top[i] > all ? s_top[i] : all;
        }
        const float sc = scale_of(all, most);
        if (tid == 0) scale[0] = sc;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          divide8(v[i], sc);
          store8_quant<VEC, THREADS>(q, tid, i, D, v[i], e4m3);
        }
      } else if constexpr (VEC) {
        const int span = group / 8;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int piece = tid + THREADS * i;
          const float sc = scale_of(lanes_max(top[i], span), most);
          if (piece % span == 0 && 8 * piece < D) scale[piece / span] = sc;
          divide8(v[i], sc);
          store8_quant<VEC, THREADS>(q, tid, i, D, v[i], e4m3);
        }
      }
    }
  }
}

template <typename X, typename H, bool VEC, int NP, int THREADS>
__global__ __launch_bounds__(THREADS == 64 ? 256 : THREADS) void add_norm_bwd_kernel(AddNormArgs a) {
  constexpr int kRows = THREADS == 64 ? 4 : 1;
  __shared__ float s_sum[THREADS / 64];
  const int D = static_cast<int>(a.D), tid = threadIdx.x % THREADS;
  const int64_t part = static_cast<int64_t>(blockIdx.x) * kRows + (kRows == 1 ? 0 : threadIdx.x / THREADS);
  const X *dy = static_cast<const X *>(a.dy);
  const H *h = static_cast<const H *>(a.h), *dh = static_cast<const H *>(a.dh);
  float w[NP][8], dw[NP][8];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (a.w != nullptr) {
      load8<float, VEC, THREADS>(a.w, tid, i, D, w[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = 1.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  }
  for (int64_t row = part; row < a.rows; row += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t at = row * D;
    const float r = a.rstd[row];
    float hv[NP][8], u[NP][8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      load8<H, VEC, THREADS>(h + at, tid, i, D, hv[i]);
      load8<X, VEC, THREADS>(dy + at, tid, i, D, u[i]);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hv[i][e] *= r;  // normalised
        dw[i][e] = fmaf(u[i][e], hv[i][e], dw[i][e]);
        u[i][e] *= w[i][e];
        s = fmaf(u[i][e], hv[i][e], s);
      }
    s = threads_sum<THREADS>(s, s_sum) / static_cast<float>(D);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float o[8];
      if (dh != nullptr) {
        load8<H, VEC, THREADS>(dh + at, tid, i, D, o);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) u[i][e] = fmaf(r, fmaf(-hv[i][e], s, u[i][e]), o[e]);
      if (a.dx != nullptr) store8<X, VEC, THREADS>(static_cast<X *>(a.dx) + at, tid, i, D, u[i]);
      if (a.dresidual != nullptr) store8<H, VEC, THREADS>(static_cast<H *>(a.dresidual) + at, tid, i, D, u[i]);
    }
  }
  if (a.dw == nullptr) return;
  if constexpr (kRows > 1) {  // the four waves' sums, one after the other
    __shared__ float s_dw[kRows > 1 ? 8 * 64 * NP : 1];
    for (int q = 0; q < kRows; ++q) {
      if (static_cast<int>(threadIdx.x) / THREADS == q)
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = tid + THREADS * (8 * i + e);  // a place of its own, not its channel's
            if (q > 0) dw[i][e] += s_dw[at];
            s_dw[at] = dw[i][e];
          }
      __syncthreads();
    }
    if (static_cast<int>(threadIdx.x) / THREADS != kRows - 1) return;
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) store8<float, VEC, THREADS>(a.ws + static_cast<int64_t>(blockIdx.x) * D, tid, i, D, dw[i]);
}

// dw: 64 channels a workgroup, 16 threads each over every 16th partial sum.
constexpr int kOver = 16;
__global__ __launch_bounds__(64 * kOver) void add_norm_dw_kernel(const float *part, int64_t parts, int64_t D, float *dw) {
  __shared__ float s[kOver][64];
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x % 64;
  const int o = threadIdx.x / 64;
  float sum = 0.f;
  if (n < D) {
#pragma unroll 4
    for (int64_t i = o; i < parts; i += kOver) sum += part[i * D + n];
  }
  s[o][threadIdx.x % 64] = sum;
  __syncthreads();
  if (o != 0 || n >= D) return;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < kOver; ++i) sum += s[i][threadIdx.x];
  dw[n] = sum;
}

__global__ void add_norm_zero_kernel(float *dw, int64_t D) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (n < D) dw[n] = 0.f;
}

// Threads and pieces of a row.
struct Shape {
  int threads, pieces;
};
Shape shape_of(int64_t rows, int64_t D, bool one_row) {
  const int64_t all = (D + 7) / 8;
  auto pieces = [&](int64_t threads) {
    const int64_t n = (all + threads - 1) / threads;
    return static_cast<int>(n <= 4 ? (n < 1 ? 1 : n) : n <= 6 ? 6 : 8);
  };
  if (!one_row && all <= 64 * 8 && rows >= 4 * kCus) return {64, static_cast<int>((all + 63) / 64)};
  if (all <= 256 * 8) return {256, pieces(256)};
  return {1024, 8};
}

bool aligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename F>
hipError_t by_shape(Shape z, F &&f) {
  using std::integral_constant;
#define SSM_AN(T, N) \
  if (z.threads == T && z.pieces == N) f(integral_constant<int, T>(), integral_constant<int, N>())
  SSM_AN(64, 1);
  SSM_AN(64, 2);
  SSM_AN(64, 3);
  SSM_AN(64, 4);
  SSM_AN(64, 5);
  SSM_AN(64, 6);
  SSM_AN(64, 7);
  SSM_AN(64, 8);
  SSM_AN(256, 1);
  SSM_AN(256, 2);
  SSM_AN(256, 3);
  SSM_AN(256, 4);
  SSM_AN(256, 6);
  SSM_AN(256, 8);
  SSM_AN(1024, 8);
#undef SSM_AN
  return hipGetLastError();
}

// Workgroups, of one row a thread group up to 2^14 of them (65536 rows by waves), where
// the weights they load are few beside the rows: 32768 rows of 2560 channels 181 us with
// 4 workgroups a CU, 154 with 8, 147 with 32 and more.
unsigned grid_of(int64_t rows, Shape z) {
  const int64_t blocks = z.threads == 64 ? (rows + 3) / 4 : rows;
  const int64_t most = kCus * (z.threads == 1024 ? 2 : z.threads == 64 ? 64 : 8);
  return static_cast<unsigned>(blocks < most ? blocks : most);
}
// The gradients': fewer, since each leaves a partial sum of dw: 8192 x 2560, forward and
// backward, 123 us with 2 a CU, 129 with 4, 136 with 6.
Shape bwd_shape(int64_t rows, int64_t D) { return shape_of(rows, D, false); }
unsigned bwd_grid(int64_t rows, Shape z) {
  const int64_t blocks = z.threads == 64 ? (rows + 3) / 4 : rows;
  const int64_t most = kCus * (z.threads == 1024 ? 1 : 2);
  return static_cast<unsigned>(blocks < most ? blocks : most);
}
int64_t bwd_parts(int64_t rows, Shape z) { return bwd_grid(rows, z); }

template <typename X, typename H>
hipError_t launch_fwd(const AddNormArgs &a, hipStream_t s) {
  const bool vec = a.D % 8 == 0 && aligned(a.x) && aligned(a.residual) && aligned(a.w) && aligned(a.h) && aligned(a.y);
  const int64_t span = a.quant ? a.group / 8 : 0;
  const bool lanes = a.quant == 0 || a.group == a.D || (vec && a.group % 8 == 0 && span <= 64 && (span & (span - 1)) == 0);
  const Shape z = shape_of(a.rows, a.D, !lanes);
  const unsigned grid = grid_of(a.rows, z);
  return by_shape(z, [&](auto threads, auto pieces) {
    constexpr int T = decltype(threads)::value, N = decltype(pieces)::value, kBlock = T == 64 ? 256 : T;
    auto go = [&](auto v) {
      constexpr bool V = decltype(v)::value;
      if (a.quant == 0) {
        add_norm_kernel<X, H, V, N, T, 0><<<grid, kBlock, 0, s>>>(a);
      } else if (lanes) {
        add_norm_kernel<X, H, V, N, T, 1><<<grid, kBlock, 0, s>>>(a);
      } else {
        if constexpr (T != 64) add_norm_kernel<X, H, V, N, T, 2><<<grid, kBlock, 0, s>>>(a);
      }
    };
    if (vec) go(std::true_type());
    else go(std::false_type());
  });
}
template <typename X, typename H>
hipError_t launch_bwd(const AddNormArgs &a, hipStream_t s) {
  if (a.rows == 0) {
    if (a.dw != nullptr) add_norm_zero_kernel<<<static_cast<unsigned>((a.D + 255) / 256), 256, 0, s>>>(a.dw, a.D);
    return hipGetLastError();
  }
  const bool vec = a.D % 8 == 0 && aligned(a.h) && aligned(a.w) && aligned(a.dy) && aligned(a.dh) && aligned(a.dx) &&
                   aligned(a.dresidual);
  const Shape z = bwd_shape(a.rows, a.D);
  const unsigned grid = bwd_grid(a.rows, z);
  const hipError_t e = by_shape(z, [&](auto threads, auto pieces) {
    constexpr int T = decltype(threads)::value, N = decltype(pieces)::value, kBlock = T == 64 ? 256 : T;
    if (vec) add_norm_bwd_kernel<X, H, true, N, T><<<grid, kBlock, 0, s>>>(a);
    else add_norm_bwd_kernel<X, H, false, N, T><<<grid, kBlock, 0, s>>>(a);
  });
  if (e != hipSuccess || a.dw == nullptr) return e;
  add_norm_dw_kernel<<<static_cast<unsigned>((a.D + 63) / 64), 64 * kOver, 0, s>>>(a.ws, bwd_parts(a.rows, z), a.D, a.dw);
  return hipGetLastError();
}

}  // namespace

int64_t add_norm_bwd_ws_floats(int64_t rows, int64_t D) {
  return rows == 0 ? 0 : bwd_parts(rows, bwd_shape(rows, D)) * D;
}

hipError_t launch_add_norm_fwd(const AddNormArgs &a, hipStream_t s) {
  if (a.dt == DType::F32) return launch_fwd<float, float>(a, s);
  return a.stream == DType::F32 ? launch_fwd<bf16_t, float>(a, s) : launch_fwd<bf16_t, bf16_t>(a, s);
}
hipError_t launch_add_norm_bwd(const AddNormArgs &a, hipStream_t s) {
  if (a.dt == DType::F32) return launch_bwd<float, float>(a, s);
  return a.stream == DType::F32 ? launch_bwd<bf16_t, float>(a, s) : launch_bwd<bf16_t, bf16_t>(a, s);
}

}  // namespace ssm
