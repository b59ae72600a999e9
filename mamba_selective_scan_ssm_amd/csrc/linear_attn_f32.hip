// Linear attention by chunks of C tokens on the fp32 matrix instructions: fp32 inputs
// of any size and alignment.
//
// Within a chunk of `left` tokens entered by the state S (n down, m across), with
// the powers a^d of the head's decay, f = 1 and (where the pass runs backwards) 0:
//   out_i = c_out (a^(i+f) S^T x_i + c_in sum_{j<=i} a^(i-j) (x_i . key_j) val_j)
//   S    <- a^left S + c_in sum_j a^(left-1-j+(1-f)) key_j val_j^T
// and the tangent T = dS / d log a, for the gradient of the decay (f = 1, c_in = 1):
//   out'_i = c_out (a^(i+1) ((i+1) S + T)^T x_i + sum_{j<=i} (i-j) a^(i-j) (x_i . key_j) val_j)
//   T     <- a^left (T + left S) + sum_j (left-1-j) a^(left-1-j) key_j val_j^T
// All powers are of distances >= 0: nothing is divided by a decay, whatever it is.
//
// A workgroup of four waves runs 64 columns m of one head's chain over a segment;
// 16 columns a wave, whose part of S stays in its registers.  A result tile of
// v_mfma_f32_16x16x4_f32 is the B operand of the next product as it is (mma_f32),
// so S goes into S^T x without leaving them.  The scores x . key are shared: each
// wave forms tiles of 16 x 16 and leaves them in LDS.
//
// Chunks of 32 tokens, single-buffered, the next one's rows on their way in registers: two
// workgroups a CU, one's loads and barriers under the other's products (232 registers a lane
// at K = 128, 176 at 64; the 47 KB of LDS would hold three).  64 tokens (102 KB, one workgroup): 2048 tokens, 64 heads of 128 x 128 323
// against 231 us; without the registers ahead 418 and 290.  Bound by the matrix products
// and the phases about them: the recurrence's 66 KFLOP a token and head and 12 of a chunk's
// scores, 10 GFLOP, in these 231 us are 44 TFLOP/s of the 131 of a large product in fp32.
// The inputs in bf16 parts instead were not tried.
//
// Values that are not finite stay behind their token: scores above the diagonal are
// selected away, and a value's column is left out of the products and set to NaN
// from its token on (0 times one of them would reach the tokens before it).
#include "device_common.h"
#include "linear_attn.h"
#include "linear_attn_common.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kColumns = 64;
constexpr int C = 32;  // tokens of a chunk

// Four consecutive elements of a row; elements from `left` on are 0
template <bool VEC>
__device__ __forceinline__ f32x4 load_four(const float *p, int left) {
  if constexpr (VEC)
    if (left >= 4) return *reinterpret_cast<const f32x4 *>(p);
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) v[e] = p[e];
  return v;
}

// KT: tiles of 16 that K is rounded up to.  Y: outputs (or the tangent's sum); else
// the segment's own addition to the state.
template <int KT, bool Y, bool TAN, bool VEC>
__global__ __launch_bounds__(kThreads) void la_f32_kernel(LaArgs a, LaPasses all, int64_t items, int64_t sub,
                                                          int64_t base) {
  constexpr int kPitch = 16 * KT + 4, kVal = kColumns + 4, kScore = C + 4;
  constexpr int CT = C / 16, kPairs = CT * (CT + 1) / 2;
  __shared__ __attribute__((aligned(16))) float s_x[Y ? C : 1][kPitch];
  __shared__ __attribute__((aligned(16))) float s_k[C][kPitch];
  __shared__ __attribute__((aligned(16))) float s_v[C][kVal];
  __shared__ __attribute__((aligned(16))) float s_a[Y ? C : 1][kScore];
  __shared__ float s_pw[C + 1];
  __shared__ double s_sum[kThreads / 64];

  const LaPass &p = all.p[blockIdx.y];
  const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, r = lane % 16, g = lane / 16;
  int64_t unit, in;
  la_place(blockIdx.x, sub, unit, in);
  const int64_t item = base + unit * sub + in;
  if (item >= items) return;
  const int64_t cols = (p.M + kColumns - 1) / kColumns;
  const int64_t h = item / cols % a.H, slot = item / (cols * a.H);
  const int m0 = static_cast<int>(item % cols) * kColumns, m = m0 + 16 * wave + r;
  const bool col = m < p.M;
  const LaSlot z = la_slot(a, slot, p.reverse);
  if constexpr (TAN && Y) {  // every partial sum is written
    if (z.len < 0 && tid == 0) p.dot_sum[item] = 0.0;
  }
  if (z.len < 0 || (!Y && z.last)) return;  // nothing follows the last segment
  const double log_a = a.log_decay[h];
  for (int d = tid; d <= C; d += kThreads) s_pw[d] = la_power(log_a, d);
  const int f = p.reverse ? 0 : 1;
  const float c_in = p.c_in, c_out = p.c_out;

  // ---- the state that enters the segment
  f32x4 S[KT], U[TAN ? KT : 1];
  const int64_t at = (z.seq * a.H + h) * a.state + static_cast<int64_t>(m) * p.sm;
#pragma unroll
  for (int j = 0; j < KT; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = 16 * j + 4 * g + e;
      S[j][e] = Y && p.s0 != nullptr && col && n < p.K ? p.s0[at + n * p.sn] : 0.f;
      if constexpr (TAN) U[j][e] = 0.f;
    }
  }
  const int64_t Kp = (p.K + 15) / 16 * 16;
  if constexpr (Y) {
    const LaWhole whole(log_a, a.seg_len);
    const float n_whole = static_cast<float>(a.seg_len);
    for (int64_t b = 0; b < z.before; ++b) {
      const int64_t from = (((z.slot0 + b) * a.H + h) * p.M + m) * Kp;
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        const bool there = col && 16 * j < Kp;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const f32x4 own = there ? *reinterpret_cast<const f32x4 *>(p.local + from + 16 * j + 4 * g) : zero;
        if constexpr (TAN) {
          const f32x4 tan = there ? *reinterpret_cast<const f32x4 *>(p.local_tan + from + 16 * j + 4 * g) : zero;
#pragma unroll
          for (int e = 0; e < 4; ++e) U[j][e] = whole(U[j][e]) + fmaf(n_whole, whole(S[j][e]), tan[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][e] = whole(S[j][e]) + own[e];
      }
    }
  }

  const float *x = static_cast<const float *>(p.x) + h / p.x_per * p.x_width;
  const float *key = static_cast<const float *>(p.key) + h / p.key_per * p.key_width;
  const float *val = static_cast<const float *>(p.val) + h / p.val_per * p.val_width;
  const float *dot = TAN ? static_cast<const float *>(p.dot) + h / p.val_per * p.val_width : nullptr;
  double sum = 0.0;

  // ---- x, keys and values of the next chunk, on their way in registers; zeros behind
  // the last token and width
  constexpr int kFours = C * 4 * KT / kThreads, kFoursV = C * kColumns / 4 / kThreads;
  f32x4 px[Y ? kFours : 1], pk[kFours], pv[kFoursV];
  auto row_of = [&](int t) { return z.first + static_cast<int64_t>(t) * z.step; };
  auto load = [&](int t0) {
    const int left = z.len - t0 < C ? z.len - t0 : C;
#pragma unroll
    for (int i = 0; i < kFours; ++i) {
      const int q = tid + kThreads * i, t = q / (4 * KT), n = q % (4 * KT) * 4;
      const int have = t < left ? p.K - n : 0;
      const int64_t row = have > 0 ? row_of(t0 + t) : 0;
      if constexpr (Y) px[i] = load_four<VEC>(x + row * p.x_row + n, have);
      pk[i] = load_four<VEC>(key + row * p.key_row + n, have);
    }
#pragma unroll
    for (int i = 0; i < kFoursV; ++i) {
      const int q = tid + kThreads * i, t = q / (kColumns / 4), n = q % (kColumns / 4) * 4;
      const int have = t < left ? p.M - m0 - n : 0;
      const int64_t row = have > 0 ? row_of(t0 + t) : 0;
      pv[i] = load_four<VEC>(val + row * p.val_row + m0 + n, have);
    }
  };
  if (z.len > 0) load(0);

  const LaCarry full(log_a, C);
  for (int t0 = 0; t0 < z.len; t0 += C) {
    const int left = z.len - t0 < C ? z.len - t0 : C;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFours; ++i) {
      const int q = tid + kThreads * i, t = q / (4 * KT), n = q % (4 * KT) * 4;
      if constexpr (Y) *reinterpret_cast<f32x4 *>(&s_x[t][n]) = px[i];
      *reinterpret_cast<f32x4 *>(&s_k[t][n]) = pk[i];
    }
#pragma unroll
    for (int i = 0; i < kFoursV; ++i) {
      const int q = tid + kThreads * i, t = q / (kColumns / 4), n = q % (kColumns / 4) * 4;
      *reinterpret_cast<f32x4 *>(&s_v[t][n]) = pv[i];
    }
    __syncthreads();
    if (t0 + C < z.len) load(t0 + C);

    // ---- scores, from the diagonal down, tile by tile
    if constexpr (Y) {
      for (int pair = wave; pair < kPairs; pair += kThreads / 64) {
        int bt = 0;
        while ((bt + 1) * (bt + 2) / 2 <= pair) ++bt;
        const int bs = pair - bt * (bt + 1) / 2;
        f32x4 w = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KT; ++j)
          w = mma_f32(*reinterpret_cast<const f32x4 *>(&s_k[16 * bs + r][16 * j + 4 * g]),
                      *reinterpret_cast<const f32x4 *>(&s_x[16 * bt + r][16 * j + 4 * g]), w);
        // token 16 bt + r, keys 16 bs + 4 g + e
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = 16 * (bt - bs) + r - 4 * g - e;
          const float pw = c_in * s_pw[d < 0 ? 0 : d];
          w[e] = d < 0 ? 0.f : w[e] * (TAN ? pw * static_cast<float>(d) : pw);
        }
        *reinterpret_cast<f32x4 *>(&s_a[16 * bt + r][16 * bs + 4 * g]) = w;
      }
    }
    // ---- this lane's values, tokens 16 j + 4 g + e
    f32x4 v[CT];
    int bad = C;
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = s_v[16 * j + 4 * g + e][16 * wave + r];
#pragma unroll
    for (int j = CT - 1; j >= 0; --j)
#pragma unroll
      for (int e = 3; e >= 0; --e)
        if (!(fabsf(v[j][e]) < __builtin_huge_valf())) {
          bad = 16 * j + 4 * g + e;
          v[j][e] = 0.f;
        }
    if (__ballot(bad < C) != 0) {
      bad = min(bad, __shfl_xor(bad, 16));
      bad = min(bad, __shfl_xor(bad, 32));
    }
    f32x4 y[CT];
    if constexpr (Y) {
      // ---- what the state answers
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        f32x4 w = {0.f, 0.f, 0.f, 0.f}, u = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KT; ++j) {
          const f32x4 q = *reinterpret_cast<const f32x4 *>(&s_x[16 * i + r][16 * j + 4 * g]);
          w = mma_f32(q, S[j], w);
          if constexpr (TAN) u = mma_f32(q, U[j], u);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 16 * i + 4 * g + e;
          if constexpr (TAN) w[e] = fmaf(static_cast<float>(t + 1), w[e], u[e]);
          w[e] *= s_pw[t + f];
        }
        y[i] = w;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j)
          y[i] = mma_f32(*reinterpret_cast<const f32x4 *>(&s_a[16 * i + r][16 * j + 4 * g]), v[j], y[i]);
      // ---- out
#pragma unroll
      for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 16 * i + 4 * g + e;
          const float out = t >= bad ? __builtin_nanf("") : c_out * y[i][e];
          if (t < left && col) {
            if constexpr (TAN) {
              sum += static_cast<double>(out) * dot[row_of(t0 + t) * p.val_row + m];
            } else {
              static_cast<float *>(p.out)[row_of(t0 + t) * p.out_row + h * p.out_width + m] = out;
            }
          }
        }
    }
    // ---- the state that leaves the chunk
    const LaCarry carry = left == C ? full : LaCarry(log_a, left);
    const float n_left = static_cast<float>(left) * s_pw[left];
    f32x4 u[TAN ? CT : 1];
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = left - 1 - (16 * j + 4 * g + e);
        const float w = d < 0 ? 0.f : v[j][e] * (c_in * s_pw[d + 1 - f]);
        if constexpr (TAN) u[j][e] = d < 0 ? 0.f : w * static_cast<float>(d);
        v[j][e] = w;
      }
    // What the chunk adds is summed from zero and joined with the state in one rounding: a
    // large state in the products would round each of their sums to its own steps.
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      f32x4 add = {0.f, 0.f, 0.f, 0.f}, add_u = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        f32x4 k;
#pragma unroll
        for (int e = 0; e < 4; ++e) k[e] = s_k[16 * j + 4 * g + e][16 * i + r];
        add = mma_f32(k, v[j], add);
        if constexpr (TAN) add_u = mma_f32(k, u[j], add_u);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (TAN) U[i][e] = fmaf(n_left, S[i][e], carry(U[i][e])) + add_u[e];
        S[i][e] = carry(S[i][e], add[e]);
      }
      if (bad < C) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          S[i][e] = __builtin_nanf("");
          if constexpr (TAN) U[i][e] = __builtin_nanf("");
        }
      }
    }
  }

  // ---- the state behind the segment
  if constexpr (!Y) {
    if (col) {
      const int64_t to = ((slot * a.H + h) * p.M + m) * Kp;
#pragma unroll
      for (int j = 0; j < KT; ++j)
        if (16 * j < Kp) {
          *reinterpret_cast<f32x4 *>(p.local + to + 16 * j + 4 * g) = S[j];
          if constexpr (TAN) *reinterpret_cast<f32x4 *>(p.local_tan + to + 16 * j + 4 * g) = U[j];
        }
    }
  } else {
    if (z.last && p.s_last != nullptr && col) {
#pragma unroll
      for (int j = 0; j < KT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = 16 * j + 4 * g + e;
          if (n < p.K) p.s_last[at + n * p.sn] = S[j][e];
        }
    }
    if constexpr (TAN) {
      if (z.last && p.s_dot != nullptr && col) {
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = 16 * j + 4 * g + e;
            if (n < p.K) sum += static_cast<double>(U[j][e]) * p.s_dot[at + n * p.sn];
          }
      }
#pragma unroll
      for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
      if (lane == 0) s_sum[wave] = sum;
      __syncthreads();
      if (tid == 0) p.dot_sum[item] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
    }
  }
}

template <int KT, bool TAN, bool VEC>
hipError_t launch_kt(const LaArgs &a, const LaPasses &all, int n, int64_t cols, int64_t sub, hipStream_t s) {
  for (int y = la_cut(a) ? 0 : 1; y < 2; ++y) {
    const hipError_t e = la_launches(a, cols, sub, n, [&](dim3 grid, int64_t items, int64_t base) {
      if (y) la_f32_kernel<KT, true, TAN, VEC><<<grid, kThreads, 0, s>>>(a, all, items, sub, base);
      else la_f32_kernel<KT, false, TAN, VEC><<<grid, kThreads, 0, s>>>(a, all, items, sub, base);
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

bool fours(const LaPass &p) {
  for (const void *q : {p.x, p.key, p.val})
    if (reinterpret_cast<uintptr_t>(q) % 16 != 0) return false;
  for (int64_t n : {p.x_row, p.key_row, p.val_row, p.x_width, p.key_width, p.val_width})
    if (n % 4 != 0) return false;
  return true;
}

template <bool TAN>
hipError_t launch_width(const LaArgs &a, const LaPass *p, int n, hipStream_t s) {
  LaPasses all{};
  bool vec = true;
  for (int i = 0; i < n; ++i) {
    all.p[i] = p[i];
    vec = vec && fours(p[i]);
  }
  const int64_t cols = la_columns(p[0].M);
  const int64_t sub = la_sub(a, p[0].x_per, cols);
#define SSM_LA_KT(KT)                                                    \
  return vec ? launch_kt<KT, TAN, true>(a, all, n, cols, sub, s)         \
             : launch_kt<KT, TAN, false>(a, all, n, cols, sub, s)
  if (p[0].K <= 64) SSM_LA_KT(4);
  if (p[0].K <= 128) SSM_LA_KT(8);
  SSM_LA_KT(16);
#undef SSM_LA_KT
}

}  // namespace

hipError_t launch_la_f32(const LaArgs &a, const LaPass *p, int n, hipStream_t s) {
  // dot may be empty
  return p[0].dot_sum != nullptr ? launch_width<true>(a, p, n, s) : launch_width<false>(a, p, n, s);
}

}  // namespace ssm
