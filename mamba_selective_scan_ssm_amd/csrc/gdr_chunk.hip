// The gated delta rule by chunks of C = 64 tokens on the gfx950 matrix cores
// (bf16 inputs, N <= 128).
//
// Within a chunk entered by the state S0 (N, P) -- n down, p across -- with the
// cumulative log decay c_i, k and q rows normalised by rk, rq (or 1):
//   A'[i][j] = rk_i rk_j beta_j exp(c_i - c_j) (k_i . k_j),  j < i
//   X = (I + A')^-1                              (unit lower triangular)
//   R_i = v_i - a_i (K S0)_i                     a_i = exp(c_i) rk_i
//   E = X R                                      the corrected values
//   y_i = b_i (Q S0)_i + sum_{j<=i} M_ij E_j     b_i = scale exp(c_i) rq_i
//     M_ij = scale rq_i rk_j beta_j exp(c_i - c_j) (q_i . k_j)
//   S1 = exp(c_C) S0 + K^T (w E)                 w_j = exp(c_C - c_j) rk_j beta_j
// which is the token-by-token recurrence regrouped: only S, E and y depend on
// the column p, so a column of the state is a chain of products of its own.
//
// One workgroup of 8 waves per (sequence, head, 64 columns).  Four waves, the
// chain, hold 16 columns each: the state stays in their registers over the
// whole sequence, and S0 -> R -> E -> S1 moves from product to product in
// registers (gdr_mfma.h).  The other four prepare the next chunk meanwhile: K
// and Q into LDS, K K^T and Q K^T, the decays (c in 64 bits: its differences
// count, not its size), X by substitution in 16 x 16 blocks (the chunk's keys
// may be all alike, where a series for the inverse loses everything) and block
// rows joined by fp32 MFMA.  Nothing but the inputs, y and the two states
// touches memory.  Four barriers per chunk pair the chain's products with the
// preparation's steps:
//   chain:   split S, K S0 | R, X R        | w E, K^T (w E) | Q S0, M E, y
//   prepare: X, M, K, Q in | K K^T, Q K^T  | block inverses | block rows, loads
//
// Precision: k, q and v are exact in bf16.  What is computed -- S, R, E, X --
// enters a product that makes S in three bf16 parts (all 24 bits; products of
// two such operands leave out what is below 2^-24), what only y depends on in
// two (at most 2^-16 of each term; y is rounded to bf16, by up to 2^-8).
// Accumulation is fp32.
#include "device_common.h"
#include "gdr.h"
#include "gdr_common.h"
#include "gdr_mfma.h"

namespace ssm {
namespace {

constexpr int kC = 64;          // tokens per chunk
constexpr int kCols = 64;       // columns per workgroup
constexpr int kThreads = 512;
constexpr int kTokPitch = 72;   // uint16 per row of 64 contraction tokens (144 bytes)
constexpr int kAtPitch = 68;    // floats
constexpr int kXtPitch = 20;    // floats

// The conflict-free place of tokens 8 ch .. + 7 in row n of K^T: rows 16 bytes
// apart modulo the banks for reads, chunks spread over the banks for the
// transposing writes.
__device__ __forceinline__ int kt_at(int n, int ch) { return n * kTokPitch + 8 * (ch ^ ((n >> 4) & 7)); }

template <int NT>
struct ChunkLds {
  static constexpr int kNPitch = 16 * NT + 8;  // uint16 per row of N
  __attribute__((aligned(16))) uint16_t k[2][kC * kNPitch];
  __attribute__((aligned(16))) uint16_t q[2][kC * kNPitch];
  __attribute__((aligned(16))) uint16_t kt[16 * NT * kTokPitch];
  __attribute__((aligned(16))) uint16_t x[3][kC * kTokPitch];
  __attribute__((aligned(16))) uint16_t m[2][kC * kTokPitch];
  __attribute__((aligned(16))) float at[kC * kAtPitch];         // A'[i][j] at [j][i]
  __attribute__((aligned(16))) float xt[4][16 * kXtPitch];      // diagonal blocks of X, transposed
  __attribute__((aligned(16))) float va[2][kC], vb[2][kC], vw[2][kC];
  __attribute__((aligned(16))) double c[kC];                    // in units of log 2
  __attribute__((aligned(16))) float rk[kC], rq[kC], beta[kC];
  float whole[2];
};

__device__ __forceinline__ u32x4 lds128(const uint16_t *p) { return *reinterpret_cast<const u32x4 *>(p); }
__device__ __forceinline__ f32x4 lds_f4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

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
__device__ __forceinline__ double wave_scan(double v) {
  v += dpp_shift<0x111>(v);
  v += dpp_shift<0x112>(v);
  v += dpp_shift<0x114>(v);
  v += dpp_shift<0x118>(v);
  const double e0 = lane_value(v, 15), e1 = lane_value(v, 31), e2 = lane_value(v, 47);
  const int row = threadIdx.x % 64 / 16;
  if (row >= 1) v += row == 1 ? e0 : row == 2 ? e0 + e1 : e0 + e1 + e2;
  return v;
}

// ---------------------------------------------------------------- the chain
template <int NT>
struct Chain {
  static constexpr int KB = NT / 2;   // blocks of 32 states
  static constexpr int kNP = ChunkLds<NT>::kNPitch;
  const GdrArgs &a;
  ChunkLds<NT> &s;
  const MinusOne minus;
  const int r, g;      // lane = 16 g + r
  const bool col;      // this lane's column is inside P
  const uint16_t *v;   // of this column, token 0
  bf16_t *y;
  int64_t row;         // elements from token to token
  f32x4 S[NT];
  u32x4 planes[KB][2];  // the two leading parts of S0, kept for y
  f32x4 R[4], E[4];
  uint16_t vr[16];
  int bad;             // first token whose value is not finite (kC: none)

  __device__ __forceinline__ void load_v(int64_t t0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {  // clamped: every load is in bounds, and none waits behind a branch
      const int64_t t = t0 + 16 * (i / 4) + 4 * g + i % 4;
      vr[i] = v[(t < a.L ? t : a.L - 1) * row];
    }
  }
  // K S0 into R, S0's leading parts kept
  __device__ __forceinline__ void ks(int buf) {
    const uint16_t *kp = &s.k[buf][r * kNP + 8 * g];
    u32x4 ka[2][4], sp[2][3];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      ka[0][rt] = lds128(kp + 16 * rt * kNP);
      R[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    split_operand<3>(S[0], S[1], sp[0], minus);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      planes[kb][0] = sp[kb % 2][0];
      planes[kb][1] = sp[kb % 2][1];
      if (kb + 1 < KB) {
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) ka[(kb + 1) % 2][rt] = lds128(kp + 16 * rt * kNP + 32 * (kb + 1));
        split_operand<3>(S[2 * kb + 2], S[2 * kb + 3], sp[(kb + 1) % 2], minus);
      }
#pragma unroll
      for (int pl = 2; pl >= 0; --pl)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) R[rt] = mma(ka[kb % 2][rt], sp[kb % 2][pl], R[rt]);
    }
  }
  // R = v - a (K S0); E = X R.  A row that is not finite is left out of the
  // products, where 0 times it would reach the tokens before it.
  __device__ __forceinline__ void xr(int buf) {
    u32x4 xa[4][2][3];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int kb = 0; kb <= rt / 2; ++kb)
#pragma unroll
        for (int pl = 0; pl < 3; ++pl)
          xa[rt][kb][pl] = lds128(&s.x[pl][(16 * rt + r) * kTokPitch + 32 * kb + 8 * g]);
    float test = 0.f;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const f32x4 av = lds_f4(&s.va[buf][16 * rt + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        R[rt][e] = fmaf(-av[e], R[rt][e], __uint_as_float(static_cast<uint32_t>(vr[4 * rt + e]) << 16));
        test = fmaf(R[rt][e], 0.f, test);
      }
    }
    bad = kC;
    if (__builtin_expect(__any(test != 0.f), 0)) {
#pragma unroll
      for (int i = 15; i >= 0; --i)
        if (!(fabsf(R[i / 4][i % 4]) < __builtin_inff())) {
          bad = 16 * (i / 4) + 4 * g + i % 4;
          R[i / 4][i % 4] = 0.f;
        }
      bad = min(bad, __shfl_xor(bad, 16));
      bad = min(bad, __shfl_xor(bad, 32));
    }
    u32x4 rp[2][3];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) split_operand<3>(R[2 * kb], R[2 * kb + 1], rp[kb], minus);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) E[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
    // small terms first; the four row tiles side by side
    constexpr int kX[6] = {2, 0, 1, 1, 0, 0}, kR[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int kb = 0; kb <= rt / 2; ++kb) E[rt] = mma(xa[rt][kb][kX[i]], rp[kb][kR[i]], E[rt]);
  }
  // S1 = whole S0 + K^T (w E)
  __device__ __forceinline__ void update(int buf) {
    u32x4 up[2][3];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
      split_operand<3>(E[2 * kb] * lds_f4(&s.vw[buf][32 * kb + 4 * g]),
                       E[2 * kb + 1] * lds_f4(&s.vw[buf][32 * kb + 16 + 4 * g]), up[kb], minus);
    const float whole = s.whole[buf];
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += 4) {
      u32x4 ka[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) ka[i][kb] = lds128(&s.kt[kt_at(16 * (n0 + i) + r, 4 * kb + g)]);
        S[n0 + i] = S[n0 + i] * whole;
      }
#pragma unroll
      for (int pl = 2; pl >= 0; --pl)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 4; ++i) S[n0 + i] = mma(ka[i][kb], up[kb][pl], S[n0 + i]);
    }
    if (__builtin_expect(__any(bad < kC), 0))
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (bad < kC) S[nt][e] = __builtin_nanf("");
  }
  __device__ __forceinline__ void output(int buf, int64_t t0) {
    const uint16_t *qp = &s.q[buf][r * kNP + 8 * g];
    u32x4 ep[2][2], qa[2][4];
    f32x4 acc[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      qa[0][rt] = lds128(qp + 16 * rt * kNP);
      acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if (kb + 1 < KB)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) qa[(kb + 1) % 2][rt] = lds128(qp + 16 * rt * kNP + 32 * (kb + 1));
#pragma unroll
      for (int pl = 1; pl >= 0; --pl)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) acc[rt] = mma(qa[kb % 2][rt], planes[kb][pl], acc[rt]);
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) split_operand<2>(E[2 * kb], E[2 * kb + 1], ep[kb], minus);
    u32x4 ma[4][2][2];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int kb = 0; kb <= rt / 2; ++kb)
#pragma unroll
        for (int pl = 0; pl < 2; ++pl)
          ma[rt][kb][pl] = lds128(&s.m[pl][(16 * rt + r) * kTokPitch + 32 * kb + 8 * g]);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) acc[rt] = acc[rt] * lds_f4(&s.vb[buf][16 * rt + 4 * g]);
    constexpr int kM[3] = {1, 0, 0}, kE[3] = {0, 1, 0};
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int kb = 0; kb <= rt / 2; ++kb) acc[rt] = mma(ma[rt][kb][kM[i]], ep[kb][kE[i]], acc[rt]);
    if (__builtin_expect(__any(bad < kC), 0))
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (16 * (i / 4) + 4 * g + i % 4 >= bad) acc[i / 4][i % 4] = __builtin_nanf("");
    if (!col) return;
    bf16_t *out = y + (t0 + 4 * g) * row;
    if (t0 + kC <= a.L) {
#pragma unroll
      for (int i = 0; i < 16; ++i) out[(16 * (i / 4) + i % 4) * row] = from_f32<bf16_t>(acc[i / 4][i % 4]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (t0 + 16 * (i / 4) + 4 * g + i % 4 < a.L)
          out[(16 * (i / 4) + i % 4) * row] = from_f32<bf16_t>(acc[i / 4][i % 4]);
    }
  }
};

// ------------------------------------------------------------ the preparation
// Threads 0..255 of four waves; thread (tq, m) holds tokens 4 tq .. + 3 and the
// 8 values n = 8 m .. + 7 of K and Q (m < 2 NT).
template <int NT>
struct Prepare {
  static constexpr int KB = NT / 2;
  static constexpr int kNP = ChunkLds<NT>::kNPitch;
  const GdrArgs &a;
  ChunkLds<NT> &s;
  const MinusOne minus;
  const int tid, lane, wave, r, g;
  const int64_t b, h, grp;
  const float A2, bias;
  static constexpr int kPieces = 2 * NT;                    // 16-byte pieces of a row
  static constexpr int kLoaders = kPieces * kC / 4;         // threads that hold a piece
  static_assert(kLoaders <= 256, "four tokens by one piece per thread");
  u32x4 kr[4], qr[4], kstaged[4];
  bf16_t dtr, ber;
  f32x4 X[4], M[4];

  __device__ __forceinline__ void load(int64_t t0) {
    const int m = tid % kPieces;
    // behind the last token the last one's address, and zeros in its place
    // when it is staged; no load waits behind a branch
    const int64_t n = 8 * m < a.N ? 8 * m : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + 4 * (tid / kPieces) + i;
      const int64_t at = ((b * a.L + (t < a.L ? t : a.L - 1)) * a.G + grp) * a.N + n;
      kr[i] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.k) + at);
      qr[i] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.q) + at);
    }
    const int64_t at = (b * a.L + (t0 + lane < a.L ? t0 + lane : a.L - 1)) * a.H + h;
    dtr = static_cast<const bf16_t *>(a.dt)[at];
    ber = static_cast<const bf16_t *>(a.beta)[at];
  }
  static __device__ __forceinline__ float sum_squares(u32x4 u) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = u[e];
      ss = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, w), ss, false);
    }
    return row_sum<(kPieces < 16 ? kPieces : 16)>(ss);
  }
  // K, Q, the norms, beta and the cumulative decay of the loaded chunk
  __device__ __forceinline__ void stage(int buf, int64_t t0) {
    const int m = tid % kPieces;
    if (tid < kLoaders) {
      float ss[4], qq[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 4 * (tid / kPieces) + i;
        const bool in = t0 + tok < a.L && 8 * m < a.N;
        kstaged[i] = in ? kr[i] : u32x4{0, 0, 0, 0};
        qr[i] = in ? qr[i] : u32x4{0, 0, 0, 0};
        const int at = tok * kNP + kpos(8 * m);
        *reinterpret_cast<u32x2 *>(&s.k[buf][at]) = u32x2{kstaged[i][0], kstaged[i][1]};
        *reinterpret_cast<u32x2 *>(&s.k[buf][at + 8]) = u32x2{kstaged[i][2], kstaged[i][3]};
        *reinterpret_cast<u32x2 *>(&s.q[buf][at]) = u32x2{qr[i][0], qr[i][1]};
        *reinterpret_cast<u32x2 *>(&s.q[buf][at + 8]) = u32x2{qr[i][2], qr[i][3]};
      }
      if (a.qk_norm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ss[i] = __builtin_amdgcn_rsqf(sum_squares(kstaged[i]) + kQkNormEps);
          qq[i] = a.scale * __builtin_amdgcn_rsqf(sum_squares(qr[i]) + kQkNormEps);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ss[i] = 1.f;
          qq[i] = a.scale;
        }
      }
      if (m == 0) {
        *reinterpret_cast<f32x4 *>(&s.rk[4 * (tid / kPieces)]) = f32x4{ss[0], ss[1], ss[2], ss[3]};
        *reinterpret_cast<f32x4 *>(&s.rq[4 * (tid / kPieces)]) = f32x4{qq[0], qq[1], qq[2], qq[3]};
      }
    }
    if (wave == 0) {
      const bool in = t0 + lane < a.L;  // behind the last token nothing decays and nothing is written
      s.beta[lane] = in ? to_f32(ber) : 0.f;
      // a step below -2000 leaves nothing of the state, however it is summed;
      // held there, the differences of later tokens keep their bits
      float lg = in ? step_size(to_f32(dtr), bias, a.dt_softplus) * A2 : 0.f;
      if (lg < -2000.f) lg = -2000.f;
      s.c[lane] = wave_scan(lg);
    }
  }
  __device__ __forceinline__ void transpose() {  // K^T of the staged chunk
    if (tid >= kLoaders) return;
    const int m = tid % kPieces, pos = kpos(4 * (tid / kPieces)), ch = pos >> 3, half = pos & 7;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
      *reinterpret_cast<u32x2 *>(&s.kt[kt_at(8 * m + e, ch) + half]) =
          u32x2{__builtin_amdgcn_perm(kstaged[1][e / 2], kstaged[0][e / 2], sel),
                __builtin_amdgcn_perm(kstaged[3][e / 2], kstaged[2][e / 2], sel)};
    }
  }
  // the chain's vectors
  __device__ __forceinline__ void vectors(int buf) {
    const double c = s.c[lane], end = s.c[kC - 1];
    const float into = decay_of(c), rk = s.rk[lane];
    s.va[buf][lane] = into * rk;
    s.vb[buf][lane] = into * s.rq[lane];
    s.vw[buf][lane] = decay_of(end - c) * rk * s.beta[lane];
    if (lane == kC - 1) s.whole[buf] = into;
  }
  // A' (transposed into LDS) for block row W, M^T for block row 3 - W (kept)
  template <int W>
  __device__ __forceinline__ void products(int buf) {
    constexpr int V = 3 - W;
    const uint16_t *kp = &s.k[buf][r * kNP + 8 * g], *qp = &s.q[buf][r * kNP + 8 * g];
    constexpr int kMost = (W > V ? W : V) + 1;  // block rows of K that either needs
    f32x4 ap[W + 1];
#pragma unroll
    for (int jt = 0; jt <= W; ++jt) ap[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int jt = 0; jt <= V; ++jt) M[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      u32x4 kf[kMost];
#pragma unroll
      for (int i = 0; i < kMost; ++i) kf[i] = lds128(kp + 16 * i * kNP + 32 * kb);
      const u32x4 qf = lds128(qp + 16 * V * kNP + 32 * kb);
#pragma unroll
      for (int jt = 0; jt <= W; ++jt) ap[jt] = mma(kf[W], kf[jt], ap[jt]);
#pragma unroll
      for (int jt = 0; jt <= V; ++jt) M[jt] = mma(kf[jt], qf, M[jt]);
    }
    double ci[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) ci[e] = s.c[16 * W + 4 * g + e];
    const f32x4 si = lds_f4(&s.rk[16 * W + 4 * g]);
#pragma unroll
    for (int jt = 0; jt <= W; ++jt) {
      const int j = 16 * jt + r;
      const double cj = s.c[j];
      const float sj = s.rk[j] * s.beta[j];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = ap[jt][e] * (si[e] * sj) * decay_of(ci[e] - cj);
        ap[jt][e] = jt < W || 4 * g + e > r ? f : 0.f;
      }
      *reinterpret_cast<f32x4 *>(&s.at[j * kAtPitch + 16 * W + 4 * g]) = ap[jt];
    }
    const double cv = s.c[16 * V + r];
    const float sv = s.rq[16 * V + r];
#pragma unroll
    for (int jt = 0; jt <= V; ++jt) {
      const f32x4 rkj = lds_f4(&s.rk[16 * jt + 4 * g]), bej = lds_f4(&s.beta[16 * jt + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = M[jt][e] * (sv * (rkj[e] * bej[e])) * decay_of(cv - s.c[16 * jt + 4 * g + e]);
        M[jt][e] = jt < V || 4 * g + e <= r ? f : 0.f;
      }
    }
  }
  // The inverses of the four diagonal blocks, by one wave: lane 16 blk + col
  // carries one column through the substitution, the next four rows of the
  // block on their way.
  __device__ __forceinline__ void diagonal() {
    const int blk = g, col = r;
    const float *at = &s.at[16 * blk * kAtPitch + 16 * blk];
    f32x4 l[2][4][4];
    auto fetch = [&](int k4) {  // A'[16 blk + i][16 blk + k], k = 4 k4 .. + 3, i >= 4 k4
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4)
          if (q4 >= k4) l[k4 % 2][kk][q4] = lds_f4(at + (4 * k4 + kk) * kAtPitch + 4 * q4);
    };
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.f : 0.f;
    fetch(0);
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4) {
      if (k4 < 3) fetch(k4 + 1);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int i = 4 * k4 + kk + 1; i < 16; ++i) x[i] = fmaf(-l[k4 % 2][kk][i / 4][i % 4], x[4 * k4 + kk], x[i]);
    }
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4)
      *reinterpret_cast<f32x4 *>(&s.xt[blk][col * kXtPitch + 4 * q4]) =
          f32x4{x[4 * q4], x[4 * q4 + 1], x[4 * q4 + 2], x[4 * q4 + 3]};
  }
  // Block row W of X, transposed tiles: X_Wj^T = -X_jj^T sum_{j<k<=W} A'_kj^T X_Wk^T
  template <int W>
  __device__ __forceinline__ void block_row() {
    f32x4 at[4][4], xj[4];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      xj[j] = lds_f4(&s.xt[j][r * kXtPitch + 4 * g]);
#pragma unroll
      for (int k = j + 1; k <= W; ++k) at[j][k] = lds_f4(&s.at[(16 * j + r) * kAtPitch + 16 * k + 4 * g]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) X[W][e] = s.xt[W][(4 * g + e) * kXtPitch + r];
#pragma unroll
    for (int j = W - 1; j >= 0; --j) {
      f32x4 t = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = W; k > j; --k) t = mma_f32(at[j][k], X[k], t);
      X[j] = -mma_f32(xj[j], t, f32x4{0.f, 0.f, 0.f, 0.f});
    }
  }
  // X and M of the prepared chunk where the chain reads them
  template <int W>
  __device__ __forceinline__ void publish() {
    constexpr int V = 3 - W;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
      u32x2 p[3];
      split4<3>(X[j], p, minus);
#pragma unroll
      for (int pl = 0; pl < 3; ++pl)
        *reinterpret_cast<u32x2 *>(&s.x[pl][(16 * W + r) * kTokPitch + kpos(16 * j) + 8 * g]) = p[pl];
    }
#pragma unroll
    for (int j = 0; j <= V; ++j) {
      u32x2 p[2];
      split4<2>(M[j], p, minus);
#pragma unroll
      for (int pl = 0; pl < 2; ++pl)
        *reinterpret_cast<u32x2 *>(&s.m[pl][(16 * V + r) * kTokPitch + kpos(16 * j) + 8 * g]) = p[pl];
    }
  }
  // Chunk c + 1 beside the chain's chunk c (chunk 0 has nobody to overlap with).
  template <int W>
  __device__ __forceinline__ void run(int64_t nc) {
    load(0);
    for (int64_t c = -1; c < nc; ++c) {
      const bool more = c + 1 < nc;
      const int buf = static_cast<int>((c + 1) & 1);
      if (c >= 0) publish<W>();
      if (more) {
        stage(buf, (c + 1) * kC);
        load((c + 2) * kC);
      }
      __syncthreads();
      if (more) products<W>(buf);
      __syncthreads();
      if (more) {
        if (W == 0) diagonal();
        if (W == 1) vectors(buf);
      }
      __syncthreads();
      if (more) {
        transpose();
        block_row<W>();
      }
      __syncthreads();
    }
  }
};

template <int NT>
__global__ __launch_bounds__(kThreads) void gdr_chunk_kernel(GdrArgs a, int64_t ptiles) {
  __shared__ ChunkLds<NT> s;
  const int64_t per = a.H / a.G * ptiles;  // workgroups of a (sequence, group), which share K and Q
  // workgroups of one (sequence, group) on one XCD (consecutive ids go to the
  // 8 XCDs in turn), so that its K and Q come from that L2
  const int64_t idx = blockIdx.x / 8, bg = blockIdx.x % 8 + 8 * (idx / per), mem = idx % per;
  if (bg >= a.B * a.G) return;
  const int64_t b = bg / a.G, grp = bg % a.G, h = grp * (a.H / a.G) + mem / ptiles, p0 = mem % ptiles * kCols;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int r = lane % 16, g = lane / 16;
  const int64_t nc = (a.L + kC - 1) / kC;

  // block pairs above the diagonal are read with their 32 tokens and stay 0
  for (int i = threadIdx.x; i < kC * kTokPitch / 2; i += kThreads) {
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) reinterpret_cast<uint32_t *>(s.x[pl])[i] = 0;
#pragma unroll
    for (int pl = 0; pl < 2; ++pl) reinterpret_cast<uint32_t *>(s.m[pl])[i] = 0;
  }
  __syncthreads();

  if (wave >= 4) {
    Prepare<NT> w{a, s, MinusOne(), static_cast<int>(threadIdx.x) - 256, lane, wave - 4, r, g, b, h, grp,
                  a.A[h] * kLog2e, a.dt_bias ? a.dt_bias[h] : 0.f, {}, {}, {}, {}, {}, {}, {}};
    if (wave == 4) w.template run<0>(nc);
    else if (wave == 5) w.template run<1>(nc);
    else if (wave == 6) w.template run<2>(nc);
    else w.template run<3>(nc);
    return;
  }

  const int64_t p = p0 + 16 * wave + r, row = a.H * a.P;
  const bool live = p0 + 16 * wave < a.P, col = p < a.P;  // some column, this lane's column
  const int64_t at0 = (b * a.L * a.H + h) * a.P + (col ? p : a.P - 1);
  Chain<NT> w{a, s, MinusOne(), r, g, col, static_cast<const uint16_t *>(a.v) + at0, static_cast<bf16_t *>(a.y) + at0,
              row, {}, {}, {}, {}, {}, kC};
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    w.S[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (a.h0 != nullptr && col && 16 * nt + 4 * g < a.N)
      w.S[nt] = *reinterpret_cast<const f32x4 *>(a.h0 + ((b * a.H + h) * a.P + p) * a.N + 16 * nt + 4 * g);
  }
  if (live) w.load_v(0);
#pragma unroll
  for (int i = 0; i < 4; ++i) __syncthreads();  // the preparation of chunk 0
  for (int64_t c = 0; c < nc; ++c) {
    const int buf = static_cast<int>(c & 1);
    if (live) w.ks(buf);
    __syncthreads();
    if (live) {
      w.xr(buf);
      w.load_v((c + 1) * kC);
    }
    __syncthreads();
    if (live) w.update(buf);
    __syncthreads();
    if (live) w.output(buf, c * kC);
    __syncthreads();
  }
  if (a.h_final != nullptr && col)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (16 * nt + 4 * g < a.N)
        *reinterpret_cast<f32x4 *>(a.h_final + ((b * a.H + h) * a.P + p) * a.N + 16 * nt + 4 * g) = w.S[nt];
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

bool gdr_chunk_applies(const GdrArgs &a) {
  return a.dt_type == DType::BF16 && a.N <= 128 && a.N % 8 == 0 && a.L >= kGdrChunkMinL && aligned16(a.q) &&
         aligned16(a.k) && aligned16(a.h0) && aligned16(a.h_final);
}

hipError_t launch_gdr_chunk(const GdrArgs &a, hipStream_t s) {
  const int64_t ptiles = (a.P + kCols - 1) / kCols, per = a.H / a.G * ptiles;
  const unsigned grid = static_cast<unsigned>((a.B * a.G + 7) / 8 * 8 * per);
  if (a.N <= 64) gdr_chunk_kernel<4><<<grid, kThreads, 0, s>>>(a, ptiles);
  else gdr_chunk_kernel<8><<<grid, kThreads, 0, s>>>(a, ptiles);
  return hipGetLastError();
}

}  // namespace ssm
