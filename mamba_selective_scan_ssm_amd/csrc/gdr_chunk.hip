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

// ---------------------------------------------------------------- the chain
template <int NT>
struct Chain {
  const GdrArgs &a;
  ChunkLds<NT> &s;
  const int r, g;      // lane = 16 g + r
  const int64_t b, h, p;
  const bool live;     // some column of this wave is inside P
  const bool col;      // this lane's column is
  f32x4 S[NT];
  u32x4 planes[NT / 2][2];  // the two leading parts of S0, kept for y
  f32x4 R[4];
  uint16_t v[16];

  __device__ __forceinline__ int64_t v_at(int64_t t) const { return ((b * a.L + t) * a.H + h) * a.P + p; }

  __device__ __forceinline__ void load_v(int64_t t0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t t = t0 + 16 * (i / 4) + 4 * g + i % 4;
      v[i] = col && t < a.L ? static_cast<const uint16_t *>(a.v)[v_at(t)] : 0;
    }
  }
  // K S0 into R (as products), S0's leading parts kept
  __device__ __forceinline__ void ks(int buf) {
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) R[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < NT / 2; ++kb) {
      u32x4 sp[3];
      split_operand<3>(S[2 * kb], S[2 * kb + 1], sp);
      planes[kb][0] = sp[0];
      planes[kb][1] = sp[1];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const u32x4 ka = lds128(&s.k[buf][(16 * rt + r) * ChunkLds<NT>::kNPitch + 32 * kb + 8 * g]);
#pragma unroll
        for (int pl = 2; pl >= 0; --pl) R[rt] = mma(ka, sp[pl], R[rt]);
      }
    }
  }
  // R = v - a (K S0); E = X R.  Returns the first token of the chunk at which
  // this lane's column is not finite (kC: none): such a row is left out of the
  // products, where 0 times it would reach the tokens before it.
  __device__ __forceinline__ int xr(int buf, f32x4 *E) {
    float test = 0.f;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const f32x4 av = lds_f4(&s.va[buf][16 * rt + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        R[rt][e] = fmaf(-av[e], R[rt][e], __uint_as_float(static_cast<uint32_t>(v[4 * rt + e]) << 16));
        test = fmaf(R[rt][e], 0.f, test);
      }
    }
    int bad = kC;
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
    for (int kb = 0; kb < 2; ++kb) split_operand<3>(R[2 * kb], R[2 * kb + 1], rp[kb]);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      E[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb <= rt / 2; ++kb) {
        u32x4 xa[3];
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) xa[pl] = lds128(&s.x[pl][(16 * rt + r) * kTokPitch + 32 * kb + 8 * g]);
        // small terms first
        E[rt] = mma(xa[2], rp[kb][0], E[rt]);
        E[rt] = mma(xa[0], rp[kb][2], E[rt]);
        E[rt] = mma(xa[1], rp[kb][1], E[rt]);
        E[rt] = mma(xa[1], rp[kb][0], E[rt]);
        E[rt] = mma(xa[0], rp[kb][1], E[rt]);
        E[rt] = mma(xa[0], rp[kb][0], E[rt]);
      }
    }
    return bad;
  }
  // S1 = whole S0 + K^T (w E)
  __device__ __forceinline__ void update(int buf, const f32x4 *E, int bad) {
    u32x4 up[2][3];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      f32x4 u[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) u[i] = E[2 * kb + i] * lds_f4(&s.vw[buf][16 * (2 * kb + i) + 4 * g]);
      split_operand<3>(u[0], u[1], up[kb]);
    }
    const float whole = s.whole[buf];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 acc = S[nt] * whole;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const u32x4 ka = lds128(&s.kt[kt_at(16 * nt + r, 4 * kb + g)]);
#pragma unroll
        for (int pl = 2; pl >= 0; --pl) acc = mma(ka, up[kb][pl], acc);
      }
      S[nt] = acc;
    }
    if (__builtin_expect(bad < kC, 0))
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[nt][e] = __builtin_nanf("");
  }
  __device__ __forceinline__ void output(int buf, int64_t t0, const f32x4 *E, int bad) {
    u32x4 ep[2][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) split_operand<2>(E[2 * kb], E[2 * kb + 1], ep[kb]);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < NT / 2; ++kb) {
        const u32x4 qa = lds128(&s.q[buf][(16 * rt + r) * ChunkLds<NT>::kNPitch + 32 * kb + 8 * g]);
        acc = mma(qa, planes[kb][1], acc);
        acc = mma(qa, planes[kb][0], acc);
      }
      acc = acc * lds_f4(&s.vb[buf][16 * rt + 4 * g]);
#pragma unroll
      for (int kb = 0; kb <= rt / 2; ++kb) {
        const u32x4 m0 = lds128(&s.m[0][(16 * rt + r) * kTokPitch + 32 * kb + 8 * g]);
        const u32x4 m1 = lds128(&s.m[1][(16 * rt + r) * kTokPitch + 32 * kb + 8 * g]);
        acc = mma(m1, ep[kb][0], acc);
        acc = mma(m0, ep[kb][1], acc);
        acc = mma(m0, ep[kb][0], acc);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * rt + 4 * g + e;
        if (col && t0 + i < a.L)
          static_cast<bf16_t *>(a.y)[v_at(t0 + i)] = from_f32<bf16_t>(i >= bad ? __builtin_nanf("") : acc[e]);
      }
    }
  }
};

// ------------------------------------------------------------ the preparation
// Threads 0..255 of four waves; thread (tq, m) holds tokens 4 tq .. + 3 and the
// 8 values n = 8 m .. + 7 of K and Q (m < 2 NT).
template <int NT>
struct Prepare {
  const GdrArgs &a;
  ChunkLds<NT> &s;
  const int tid, lane, wave, r, g;
  const int64_t b, h, grp;
  const float A2, bias;
  static constexpr int kPieces = 2 * NT;                    // 16-byte pieces of a row
  static constexpr int kLoaders = kPieces * kC / 4;         // threads that hold a piece
  static_assert(kLoaders <= 256, "four tokens by one piece per thread");
  u32x4 kr[4], qr[4];
  float dtv, bev;
  f32x4 X[4], M[4];

  __device__ __forceinline__ void load(int64_t t0) {
    const int m = tid % kPieces;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + 4 * (tid / kPieces) + i;
      kr[i] = qr[i] = u32x4{0, 0, 0, 0};
      if (tid < kLoaders && t < a.L && 8 * m < a.N) {
        const int64_t at = ((b * a.L + t) * a.G + grp) * a.N + 8 * m;
        kr[i] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.k) + at);
        qr[i] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.q) + at);
      }
    }
    dtv = bev = 0.f;
    if (wave == 0 && t0 + lane < a.L) {
      const int64_t at = (b * a.L + t0 + lane) * a.H + h;
      dtv = step_size(to_f32(static_cast<const bf16_t *>(a.dt)[at]), bias, a.dt_softplus);
      bev = to_f32(static_cast<const bf16_t *>(a.beta)[at]);
    }
  }
  static __device__ __forceinline__ float sum_squares(u32x4 u) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = __uint_as_float(u[e] << 16), hi = __uint_as_float(u[e] & 0xffff0000u);
      ss = fmaf(lo, lo, ss);
      ss = fmaf(hi, hi, ss);
    }
    return row_sum<(kPieces < 16 ? kPieces : 16)>(ss);
  }
  // K, Q, the norms, beta and the cumulative decay of the loaded chunk
  __device__ __forceinline__ void stage(int buf) {
    const int m = tid % kPieces;
    if (tid < kLoaders)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 4 * (tid / kPieces) + i;
        const int at = tok * ChunkLds<NT>::kNPitch + kpos(8 * m);
        *reinterpret_cast<u32x2 *>(&s.k[buf][at]) = u32x2{kr[i][0], kr[i][1]};
        *reinterpret_cast<u32x2 *>(&s.k[buf][at + 8]) = u32x2{kr[i][2], kr[i][3]};
        *reinterpret_cast<u32x2 *>(&s.q[buf][at]) = u32x2{qr[i][0], qr[i][1]};
        *reinterpret_cast<u32x2 *>(&s.q[buf][at + 8]) = u32x2{qr[i][2], qr[i][3]};
        float rk = 1.f, rq = 1.f;
        if (a.qk_norm) {
          rk = 1.f / sqrtf(sum_squares(kr[i]) + kQkNormEps);
          rq = 1.f / sqrtf(sum_squares(qr[i]) + kQkNormEps);
        }
        if (m == 0) {
          s.rk[tok] = rk;
          s.rq[tok] = a.scale * rq;
        }
      }
    if (wave == 0) {
      s.beta[lane] = bev;
      // a step below -2000 leaves nothing of the state, however it is summed;
      // held there, the differences of later tokens keep their bits
      float lg = dtv * A2;
      if (lg < -2000.f) lg = -2000.f;
      double c = lg;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(c, d);
        if (lane >= d) c += o;
      }
      s.c[lane] = c;
    }
  }
  __device__ __forceinline__ void transpose() {  // K^T of the staged chunk
    if (tid >= kLoaders) return;
    const int m = tid % kPieces, pos = kpos(4 * (tid / kPieces)), ch = pos >> 3, half = pos & 7;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
      *reinterpret_cast<u32x2 *>(&s.kt[kt_at(8 * m + e, ch) + half]) =
          u32x2{__builtin_amdgcn_perm(kr[1][e / 2], kr[0][e / 2], sel),
                __builtin_amdgcn_perm(kr[3][e / 2], kr[2][e / 2], sel)};
    }
  }
  // A' (transposed into LDS) for block row `wave`, M^T for block row 3 - wave
  // (kept), and the chain's vectors
  __device__ __forceinline__ void products(int buf) {
    const uint16_t *sk = s.k[buf], *sq = s.q[buf];
    constexpr int kNP = ChunkLds<NT>::kNPitch;
    if (wave == 0) {
      const double c = s.c[lane], end = s.c[kC - 1];
      const float into = decay_of(c), rk = s.rk[lane];
      s.va[buf][lane] = into * rk;
      s.vb[buf][lane] = into * s.rq[lane];
      s.vw[buf][lane] = decay_of(end - c) * rk * s.beta[lane];
      if (lane == kC - 1) s.whole[buf] = into;
    }
    {
      const int it = wave;
      u32x4 ki[NT / 2];
#pragma unroll
      for (int kb = 0; kb < NT / 2; ++kb) ki[kb] = lds128(&sk[(16 * it + r) * kNP + 32 * kb + 8 * g]);
      double ci[4];
      float si[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ci[e] = s.c[16 * it + 4 * g + e];
        si[e] = s.rk[16 * it + 4 * g + e];
      }
      for (int jt = 0; jt <= it; ++jt) {
        f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NT / 2; ++kb) acc = mma(ki[kb], lds128(&sk[(16 * jt + r) * kNP + 32 * kb + 8 * g]), acc);
        const int j = 16 * jt + r;
        const double cj = s.c[j];
        const float sj = s.rk[j] * s.beta[j];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[e] = 16 * it + 4 * g + e > j ? acc[e] * (si[e] * sj) * decay_of(ci[e] - cj) : 0.f;
        *reinterpret_cast<f32x4 *>(&s.at[j * kAtPitch + 16 * it + 4 * g]) = acc;
      }
    }
    {
      const int it = 3 - wave;
      u32x4 qi[NT / 2];
#pragma unroll
      for (int kb = 0; kb < NT / 2; ++kb) qi[kb] = lds128(&sq[(16 * it + r) * kNP + 32 * kb + 8 * g]);
      const int i = 16 * it + r;
      const double ci = s.c[i];
      const float si = s.rq[i];
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        if (jt > it) break;
        f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NT / 2; ++kb) acc = mma(lds128(&sk[(16 * jt + r) * kNP + 32 * kb + 8 * g]), qi[kb], acc);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * jt + 4 * g + e;
          acc[e] = j <= i ? acc[e] * (si * s.rk[j] * s.beta[j]) * decay_of(ci - s.c[j]) : 0.f;
        }
        M[jt] = acc;
      }
    }
  }
  // The inverses of the four diagonal blocks, by wave 0: lane 16 blk + col
  // carries one column through the substitution.
  __device__ __forceinline__ void diagonal() {
    if (wave != 0) return;
    const int blk = g, col = r;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.f : 0.f;
#pragma unroll
    for (int k = 0; k < 15; ++k) {
#pragma unroll
      for (int q4 = k / 4; q4 < 4; ++q4) {  // A'[16 blk + i][16 blk + k], 0 for i <= k
        const f32x4 l4 = lds_f4(&s.at[(16 * blk + k) * kAtPitch + 16 * blk + 4 * q4]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * q4 + e > k) x[4 * q4 + e] = fmaf(-l4[e], x[k], x[4 * q4 + e]);
      }
    }
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4)
      *reinterpret_cast<f32x4 *>(&s.xt[blk][col * kXtPitch + 4 * q4]) =
          f32x4{x[4 * q4], x[4 * q4 + 1], x[4 * q4 + 2], x[4 * q4 + 3]};
  }
  // Block row i = wave of X, transposed tiles: X_ij^T = -X_jj^T sum_{j<k<=i} A'_kj^T X_ik^T
  __device__ __forceinline__ void block_row() {
    const int i = wave;
#pragma unroll
    for (int j = 3; j >= 0; --j) {
      if (j > i) continue;
      if (j == i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) X[j][e] = s.xt[j][(4 * g + e) * kXtPitch + r];
        continue;
      }
      f32x4 t = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = j + 1; k < 4; ++k)
        if (k <= i) t = mma_f32(lds_f4(&s.at[(16 * j + r) * kAtPitch + 16 * k + 4 * g]), X[k], t);
      X[j] = -mma_f32(lds_f4(&s.xt[j][r * kXtPitch + 4 * g]), t, f32x4{0.f, 0.f, 0.f, 0.f});
    }
  }
  // X and M of the prepared chunk where the chain reads them
  __device__ __forceinline__ void publish() {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j <= wave) {
        u32x2 p[3];
        split4<3>(X[j], p);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl)
          *reinterpret_cast<u32x2 *>(&s.x[pl][(16 * wave + r) * kTokPitch + kpos(16 * j + 4 * g)]) = p[pl];
      }
      if (j <= 3 - wave) {
        u32x2 p[2];
        split4<2>(M[j], p);
#pragma unroll
        for (int pl = 0; pl < 2; ++pl)
          *reinterpret_cast<u32x2 *>(&s.m[pl][(16 * (3 - wave) + r) * kTokPitch + kpos(16 * j + 4 * g)]) = p[pl];
      }
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
    Prepare<NT> w{a, s, static_cast<int>(threadIdx.x) - 256, lane, wave - 4, r, g, b, h, grp, a.A[h] * kLog2e,
                  a.dt_bias ? a.dt_bias[h] : 0.f, {}, {}, 0.f, 0.f, {}, {}};
    // chunk 0 has nobody to overlap with; then chunk c + 1 beside the chain's c
    w.load(0);
    for (int64_t c = -1; c < nc; ++c) {
      const bool more = c + 1 < nc;
      const int buf = static_cast<int>((c + 1) & 1);
      if (c >= 0) w.publish();
      if (more) w.stage(buf);
      __syncthreads();
      if (more) w.products(buf);
      __syncthreads();
      if (more) w.diagonal();
      __syncthreads();
      if (more) {
        w.transpose();
        w.load((c + 2) * kC);
        w.block_row();
      }
      __syncthreads();
    }
    return;
  }

  const int64_t p = p0 + 16 * wave + r;
  Chain<NT> w{a, s, r, g, b, h, p, p0 + 16 * wave < a.P, p < a.P, {}, {}, {}, {}};
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    w.S[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (a.h0 != nullptr && w.col && 16 * nt + 4 * g < a.N)
      w.S[nt] = *reinterpret_cast<const f32x4 *>(a.h0 + ((b * a.H + h) * a.P + p) * a.N + 16 * nt + 4 * g);
  }
  if (w.live) w.load_v(0);
#pragma unroll
  for (int i = 0; i < 4; ++i) __syncthreads();  // the preparation of chunk 0
  for (int64_t c = 0; c < nc; ++c) {
    const int buf = static_cast<int>(c & 1);
    f32x4 E[4];
    int bad = kC;
    if (w.live) w.ks(buf);
    __syncthreads();
    if (w.live) bad = w.xr(buf, E);
    __syncthreads();
    if (w.live) {
      w.load_v((c + 1) * kC);
      w.update(buf, E, bad);
    }
    __syncthreads();
    if (w.live) w.output(buf, c * kC, E, bad);
    __syncthreads();
  }
  if (a.h_final != nullptr && w.col)
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
