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
// One workgroup of 8 waves per (sequence, head, 64 columns, or 32 or 16 where
// that leaves each a CU).  Four waves (two, one), the chain, hold 16 columns
// each: the state stays in their registers over the whole sequence, and S0 -> R
// -> E -> S1 moves from product to product in registers (gdr_mfma.h).  The last
// four prepare the next chunk meanwhile: K and Q into LDS, K K^T and Q K^T, the
// decays (c in 64 bits: its differences count, not its size), X by substitution
// in 16 x 16 blocks (the chunk's keys may be all alike, where a series for the
// inverse loses everything) and block rows joined by fp32 MFMA.  What they make
// is double-buffered, so one barrier a chunk joins the two; the preparing waves
// meet among themselves at a count in LDS.  Nothing but the inputs, y and the
// two states touches memory.
//
// Precision: k, q and v are exact in bf16.  What is computed -- S, R, E, X, M --
// enters a product in three bf16 parts (all 24 bits; products of two such operands
// leave out what is below 2^-24).  Accumulation is fp32.  Two parts of what only y
// depends on (S0, E and M there) took 0.56 instead of 0.60 ms at the first size
// below, and were off by up to 2^-16 of each term: y differed from the rounded exact
// value by 1.0e-4 of its norm, now by 1.4e-5, as by tokens.
//
// Values that are not finite stay behind their token: 0 times one of them, in the
// zeros above a diagonal, would reach the tokens before it.  Rows of A', R and E that
// are not finite are left out of the products, and y and the state set to NaN from
// their token on.
//
// Bound by the latency of both roles, not by a unit: 2 x 8192 tokens, 80 heads of
// 64 x 128 take 0.60 ms (107 TFLOP/s of the 64 GFLOP that the rule needs, 0.69 TB/s
// of its inputs and outputs), 11.3 thousand cycles a chunk, of which the preparation
// takes 8.3 and the chain 8.4 where the other is left out; the matrix cores are busy
// for 4.3 thousand a SIMD, the LDS for 5.1 (1.8 of them conflicts, of transposing
// reads and half-width writes).  160 workgroups on 256 CUs: a chunk's time is what
// counts.  4001 tokens, 32 heads of 128 x 128, 256 workgroups of 16 columns: 0.262
// ms.  A preparation of its own for all chunks would write and read 0.8 GB of tiles
// at the first of these sizes, a third of the time that it has now; at the second,
// where eight workgroups prepare the same chunk, 40 MB (not tried).
#include "device_common.h"
#include "gdr.h"
#include "gdr_common.h"
#include "gdr_mfma.h"

namespace ssm {
namespace {

constexpr int kThreads = 512;
constexpr int kAtPitch = 20;    // floats per row of a 16 x 16 block

// Block (j, k) of the transposed A', k >= j.
__device__ __forceinline__ constexpr int at_block(int j, int k) {
  return (j * 4 - j * (j - 1) / 2 + k - j) * 16 * kAtPitch;
}

template <int NT>
struct ChunkLds {
  __attribute__((aligned(16))) uint16_t k[2][kC * 16 * NT];
  __attribute__((aligned(16))) uint16_t q[2][kC * 16 * NT];
  __attribute__((aligned(16))) uint16_t x[2][3][kTriSize];
  __attribute__((aligned(128))) uint16_t m[2][3][kMixSize];  // a row's pieces by address bits
  // A'[i][j] at [j][i]; a diagonal block gives way to its inverse, transposed
  __attribute__((aligned(16))) float at[10 * 16 * kAtPitch];
  __attribute__((aligned(16))) float va[2][kC], vb[2][kC], vw[2][kC];
  __attribute__((aligned(16))) double c[2][kC];                 // in units of log 2
  __attribute__((aligned(16))) float beta[2][kC], rk[kC], rq[kC];
  float whole[2];
  int bad[2];  // the first token whose row of A' is not finite, kC where all are
  uint32_t met;
  // byte offsets between the parts
  static constexpr uint32_t kTile = 2 * kC * 16 * NT, kTri = 2 * kTriSize, kMix = 2 * kMixSize;
};

// ---------------------------------------------------------------- the chain
template <int NT, bool SAVE>
struct Chain {
  static constexpr int KB = NT / 2;   // blocks of 32 states
  const GdrArgs &a;
  const GdrSaved &keep;
  const int64_t item0, p;  // of this head and chunk 0; this lane's column
  const bool col;          // which is inside P
  ChunkLds<NT> &s;
  const MinusOne minus;
  const int r, g;        // lane = 16 g + r
  const uint16_t *v;     // of this head, token 0
  bf16_t *y;
  const uint32_t row;    // elements from token to token
  const uint32_t width;  // columns of a row from this head on that are its own
  const uint32_t rows16; // bytes of 16 rows
  uint32_t at[4];        // bytes to this lane's column in rows 4 g .. 4 g + 3
  // LDS addresses: rows r of K (Q behind it) by block of 32 states, the same
  // for the transposing reads, rows r of X and M (its last 32 by block of 32
  // tokens), element 4 g of the vectors
  uint32_t lk[KB], lt[KB], lx[2], lm[3], lv;
  f32x4 S[NT];
  uint16_t vr[16];  // v of the next chunk, on its way
  float vf[16];     // and of this one

  __device__ __forceinline__ void place() {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      lk[kb] = hold(lds_address(&s.k[0][tile_at<NT>(r, 4 * kb + g)]));
      lt[kb] = hold(lds_address(&s.k[0][tile_at<NT>(4 * g + r / 4, 4 * kb + r % 4)]));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)  // rows r and 32 + r
      lx[i] = hold(lds_address(&s.x[0][0][tri_at(32 * i + r) + 8 * g]));
#pragma unroll
    for (int i = 0; i < 3; ++i) lm[i] = hold(lds_address(&s.m[0][0][mix_at(i == 0 ? r : 32 + r, (i == 2 ? 4 : 0) + g)]));
    lv = hold(lds_address(&s.va[0][4 * g]));
  }
  // rows 16 rt + r, block kb of part `part` of X (M) in buffer buf
  template <int buf>
  __device__ __forceinline__ u32x4 row_x(int part, int rt, int kb) const {
    return lds_get<u32x4>(lx[rt / 2] + (3 * buf + part) * ChunkLds<NT>::kTri +
                          2 * (tri_at(16 * rt) - tri_at(32 * (rt / 2)) + 32 * kb));
  }
  template <int buf>
  __device__ __forceinline__ u32x4 row_m(int part, int rt, int kb) const {
    return lds_get<u32x4>(lm[rt < 2 ? 0 : 1 + kb] + (3 * buf + part) * ChunkLds<NT>::kMix +
                          2 * 16 * (rt % 2) * (rt < 2 ? 32 : 64));
  }
  // element 16 rt + 4 g .. + 3 of vector w (va, vb, vw) of the chunk
  template <int buf>
  __device__ __forceinline__ f32x4 vec(int w, int rt) const {
    return lds_get<f32x4>(lv + 4 * ((2 * w + buf) * kC + 16 * rt));
  }

  // v of the chunk of `left` tokens at t0
  __device__ __forceinline__ void load_v(int64_t t0, int left) {
    const __amdgpu_buffer_rsrc_t rv = rows_of(v + t0 * row, left, row, width);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      vr[i] = __builtin_amdgcn_raw_buffer_load_b16(rv, static_cast<int>(at[i % 4]), static_cast<int>(i / 4 * rows16), 0);
  }

  // Waits for the loads, before anything that is stored after them has to be
  // waited for too.
  __device__ __forceinline__ void take_v() {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      vf[i] = __uint_as_float(static_cast<uint32_t>(vr[i]) << 16);
      asm volatile("" : "+v"(vf[i]));
    }
  }

  // Zeros for what is not finite; its first token in this lane's column, or `bad`.
  __device__ __forceinline__ int leave_out(f32x4 *rows, int bad) {
#pragma unroll
    for (int i = 15; i >= 0; --i)
      if (!(fabsf(rows[i / 4][i % 4]) < __builtin_inff())) {
        bad = min(bad, 16 * (i / 4) + 4 * g + i % 4);
        rows[i / 4][i % 4] = 0.f;
      }
    bad = min(bad, __shfl_xor(bad, 16));
    return min(bad, __shfl_xor(bad, 32));
  }
  // A column whose token `bad` is not finite: its rows from there on, and the state.
  __device__ __forceinline__ void spoil(int bad, f32x4 *rows) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (16 * (i / 4) + 4 * g + i % 4 >= bad) rows[i / 4][i % 4] = __builtin_nanf("");
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (bad < kC) S[nt][e] = __builtin_nanf("");
  }

  // One chunk: y and the state behind it.
  template <int buf>
  __device__ __forceinline__ void step(int64_t t0) {
    const int more = static_cast<int>(a.L - t0 < 2 * kC ? a.L - t0 : 2 * kC), left = more < kC ? more : kC;
    const int64_t item = item0 + t0 / kC;
    if (SAVE && col)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (16 * nt + 4 * g < a.N)
          *reinterpret_cast<f32x4 *>(keep.S + (item * a.P + p) * a.N + 16 * nt + 4 * g) = S[nt];
    // K S0 and Q S0, the next block of the state split while one multiplies
    f32x4 R[4], Y[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) R[rt] = Y[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 sp[2][3];
    split_operand<3>(S[0], S[1], sp[0], minus);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      u32x4 ka[4], qa[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const uint32_t tile = buf * ChunkLds<NT>::kTile + 2 * 16 * rt * 16 * NT;
        ka[rt] = lds_get<u32x4>(lk[kb] + tile);
        if (!SAVE) qa[rt] = lds_get<u32x4>(lk[kb] + tile + 2 * ChunkLds<NT>::kTile);
      }
      if (kb + 1 < KB) split_operand<3>(S[2 * kb + 2], S[2 * kb + 3], sp[(kb + 1) % 2], minus);
#pragma unroll
      for (int pl = 2; pl >= 0; --pl)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) R[rt] = mma(ka[rt], sp[kb % 2][pl], R[rt]);
      if (!SAVE)
#pragma unroll
        for (int pl = 2; pl >= 0; --pl)
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) Y[rt] = mma(qa[rt], sp[kb % 2][pl], Y[rt]);
    }

    __builtin_amdgcn_sched_barrier(0);
    // R = v - a (K S0).  A row that is not finite is left out of the products,
    // where 0 times it would reach the tokens before it.
    float test = 0.f;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const f32x4 av = vec<buf>(0, rt);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        R[rt][e] = fmaf(-av[e], R[rt][e], vf[4 * rt + e]);
        test = fmaf(R[rt][e], 0.f, test);
      }
    }
    load_v(t0 + kC, more - kC);
    int bad = SAVE ? kC : s.bad[buf];  // the first such token of this lane's column
    bool any_bad = __any(test != 0.f) || bad < kC;
    if (__builtin_expect(any_bad, 0)) bad = leave_out(R, bad);

    __builtin_amdgcn_sched_barrier(0);
    // E = X R: small terms first, the four row tiles side by side
    f32x4 E[4];
    {
      u32x4 rp[2][3];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) split_operand<3>(R[2 * kb], R[2 * kb + 1], rp[kb], minus);
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) E[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int xp = 2; xp >= 0; --xp) {
        u32x4 xa[4][2];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
          for (int kb = 0; kb <= rt / 2; ++kb) xa[rt][kb] = row_x<buf>(xp, rt, kb);
#pragma unroll
        for (int pl = 2 - xp; pl >= 0; --pl)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int rt = 2 * kb; rt < 4; ++rt) E[rt] = mma(xa[rt][kb], rp[kb][pl], E[rt]);
      }
    }

    if (!SAVE) {  // sums that passed the largest number: left out of y's product likewise
      float over = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) over = fmaf(E[i / 4][i % 4], 0.f, over);
      if (__builtin_expect(__any(over != 0.f), 0)) {
        any_bad = true;
        bad = leave_out(E, bad);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // S1 = whole S0 + K^T (w E)
    {
      u32x4 up[2][3];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        split_operand<3>(E[2 * kb] * vec<buf>(2, 2 * kb), E[2 * kb + 1] * vec<buf>(2, 2 * kb + 1), up[kb], minus);
      const float whole = s.whole[buf];
      constexpr int kSide = 4;  // state tiles side by side
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += kSide) {
        u32x4 kt[kSide][2];
#pragma unroll
        for (int i = 0; i < kSide; ++i) {
          const int nt = n0 + i;
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) {
            u32x2 half[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
              half[u] = lds_transposed(lt[nt / 2] + buf * ChunkLds<NT>::kTile +
                                       2 * ((32 * kb + 16 * u) * 16 * NT + 4 * (nt % 2)));
            kt[i][kb] = u32x4{half[0][0], half[0][1], half[1][0], half[1][1]};
          }
          S[nt] = S[nt] * whole;
        }
#pragma unroll
        for (int pl = 2; pl >= 0; --pl)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < kSide; ++i) S[n0 + i] = mma(kt[i][kb], up[kb][pl], S[n0 + i]);
      }
    }

    __builtin_amdgcn_sched_barrier(0);
    if (SAVE) {
      if (__builtin_expect(any_bad, 0)) spoil(bad, E);
      take_v();
      __builtin_amdgcn_sched_barrier(0);
      if (col) {
        float *ep = keep.E + (item * kC + 4 * g) * a.P + p;
#pragma unroll
        for (int i = 0; i < 16; ++i) ep[(16 * (i / 4) + i % 4) * a.P] = E[i / 4][i % 4];
      }
      return;
    }
    // y = b (Q S0) + M E
    u32x4 ep[2][3];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) split_operand<3>(E[2 * kb], E[2 * kb + 1], ep[kb], minus);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) Y[rt] = Y[rt] * vec<buf>(1, rt);
#pragma unroll
    for (int mp = 2; mp >= 0; --mp) {
      u32x4 ma[4][2];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int kb = 0; kb <= rt / 2; ++kb) ma[rt][kb] = row_m<buf>(mp, rt, kb);
#pragma unroll
      for (int pl = 2 - mp; pl >= 0; --pl)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int rt = 2 * kb; rt < 4; ++rt) Y[rt] = mma(ma[rt][kb], ep[kb][pl], Y[rt]);
    }
    if (__builtin_expect(any_bad, 0)) spoil(bad, Y);
    take_v();
    __builtin_amdgcn_sched_barrier(0);
    const __amdgpu_buffer_rsrc_t ry = rows_of(y + t0 * row, left, row, width);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      __builtin_amdgcn_raw_buffer_store_b16(from_f32<bf16_t>(Y[i / 4][i % 4]).bits, ry, static_cast<int>(at[i % 4]),
                                            static_cast<int>(i / 4 * rows16), 0);
  }
};

// ------------------------------------------------------------ the preparation
// Threads 0..255 of four waves; thread (tq, m) holds tokens 4 tq .. + 3 and the
// 8 values n = 8 m .. + 7 of K and Q (m < 2 NT).
template <int NT, bool SAVE>
struct Prepare {
  static constexpr int KB = NT / 2;
  const GdrArgs &a;
  const GdrSaved &keep;
  const int64_t item0;   // of this head and chunk 0
  const bool first;      // the first columns of the head: they keep what all have in common
  ChunkLds<NT> &s;
  const MinusOne minus;
  const int tid, lane, r, g;
  const int64_t b, h, grp;
  const float A2, bias;
  static constexpr int kPieces = 2 * NT;                    // 16-byte pieces of a row
  static constexpr int kLoaders = kPieces * kC / 4;         // threads that hold a piece
  static_assert(kLoaders <= 256, "four tokens by one piece per thread");
  uint32_t meetings;
  // LDS addresses: this thread's pieces of K (two halves by four tokens), rows r
  // of K by block of 32 states, c and beta at r and at 4 g (rk and rq behind
  // beta), row r, element 4 g of the blocks of A'
  uint32_t lp[4][2], lk[KB], lc1, lc4, lf1, lf4, la;
  uint32_t piece;  // bytes to this thread's piece of K and Q, first token
  u32x4 kr[4], qr[4];
  bf16_t dtr, ber;
  f32x4 X[4], M[4];

  __device__ __forceinline__ void place() {
    const int pos = kpos(8 * (tid % kPieces)), tq = 4 * (tid / kPieces) % kC;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // the second four of a piece lie one piece further
#pragma unroll
      for (int u = 0; u < 2; ++u) lp[i][u] = hold(lds_address(&s.k[0][tile_at<NT>(tq + i, pos / 8 + u) + pos % 8]));
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) lk[kb] = hold(lds_address(&s.k[0][tile_at<NT>(r, 4 * kb + g)]));
    lc1 = hold(lds_address(&s.c[0][r]));
    lc4 = hold(lds_address(&s.c[0][4 * g]));
    lf1 = hold(lds_address(&s.beta[0][r]));
    lf4 = hold(lds_address(&s.beta[0][4 * g]));
    la = hold(lds_address(&s.at[r * kAtPitch + 4 * g]));
    const int m = tid % kPieces;
    piece = tid < kLoaders && 8 * m < a.N ? 2 * (tq * static_cast<uint32_t>(a.G * a.N) + 8 * m) : kNowhere;
  }
  __device__ __forceinline__ double c1(int t) const { return lds_get<double>(lc1 + 8 * t); }
  __device__ __forceinline__ double c4(int t) const { return lds_get<double>(lc4 + 8 * t); }
  enum { kBeta0, kBeta1, kRk, kRq };  // behind each other
  __device__ __forceinline__ float f1(int which, int t) const { return lds_get<float>(lf1 + 4 * (which * kC + t)); }
  __device__ __forceinline__ f32x4 f4(int which, int t) const { return lds_get<f32x4>(lf4 + 4 * (which * kC + t)); }
  static constexpr uint32_t block(int j, int k) { return 4 * at_block(j, k); }

  // The four preparing waves meet: all arrive without waiting for anybody else.
  __device__ __forceinline__ void meet() {
    meetings += 4;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    if (lane == 0) __hip_atomic_fetch_add(&s.met, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    while (__hip_atomic_load(&s.met, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) < meetings)
      __builtin_amdgcn_s_sleep(1);
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
  }

  __device__ __forceinline__ void load(int64_t t0) {
    const int left = static_cast<int>(a.L - t0 < kC ? a.L - t0 : kC);
    const uint32_t row = static_cast<uint32_t>(a.G * a.N);
    const int64_t base = ((b * a.L + t0) * a.G + grp) * a.N;
    const __amdgpu_buffer_rsrc_t rk = rows_of(static_cast<const uint16_t *>(a.k) + base, left, row, a.N);
    const __amdgpu_buffer_rsrc_t rq = rows_of(static_cast<const uint16_t *>(a.q) + base, left, row, a.N);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kr[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rk, static_cast<int>(piece),
                                                                              static_cast<int>(2 * i * row), 0));
      qr[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rq, static_cast<int>(piece),
                                                                              static_cast<int>(2 * i * row), 0));
    }
  }
  __device__ __forceinline__ void load_gates(int64_t t0) {
    const int left = static_cast<int>(a.L - t0 < kC ? a.L - t0 : kC);
    const uint32_t H = static_cast<uint32_t>(a.H);
    const int64_t gate = (b * a.L + t0) * a.H + h;
    dtr.bits = __builtin_amdgcn_raw_buffer_load_b16(rows_of(static_cast<const uint16_t *>(a.dt) + gate, left, H, 1),
                                                    static_cast<int>(2 * lane * H), 0, 0);
    ber.bits = __builtin_amdgcn_raw_buffer_load_b16(rows_of(static_cast<const uint16_t *>(a.beta) + gate, left, H, 1),
                                                    static_cast<int>(2 * lane * H), 0, 0);
  }
  // beta and the cumulative decay of the chunk at t0, by one wave; the next one's on their way
  __device__ __forceinline__ void gates(int buf, int64_t t0) {
    const bool in = t0 + lane < a.L;  // behind the last token nothing decays and nothing is written
    s.beta[buf][lane] = to_f32(ber);
    // a step below -2000 leaves nothing of the state, however it is summed; held
    // there, the differences of later tokens keep their bits
    float lg = in ? step_size(to_f32(dtr), bias, a.dt_softplus) * A2 : 0.f;
    if (lg < -2000.f) lg = -2000.f;
    s.c[buf][lane] = wave_scan(lg);
    load_gates(t0 + kC);
  }
  // 1 / norm of the rows of which u holds pieces, rows side by side
  static __device__ __forceinline__ void norms(const u32x4 (&u)[8], f32x4 *out) {
    float ss[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[i] = kQkNormEps / kPieces;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w = u[i][e];
        ss[i] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, w), ss[i], false);
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[i] += dpp_get<0xB1>(ss[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[i] += dpp_get<0x4E>(ss[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[i] += dpp_get<0x141>(ss[i]);
    if (kPieces > 8)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[i] += dpp_get<0x140>(ss[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i / 4][i % 4] = __builtin_amdgcn_rsqf(ss[i]);
  }
  // K, Q and their norms of the loaded chunk
  __device__ __forceinline__ void stage(int buf) {
    if (tid == 0) s.bad[buf] = kC;
    if (tid >= kLoaders) return;
    const int m = tid % kPieces, tq = 4 * (tid / kPieces);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t at = lp[i][u] + buf * ChunkLds<NT>::kTile;
        lds_put(at, u32x2{kr[i][2 * u], kr[i][2 * u + 1]});
        lds_put(at + 2 * ChunkLds<NT>::kTile, u32x2{qr[i][2 * u], qr[i][2 * u + 1]});
      }
    f32x4 n[2] = {f32x4{1.f, 1.f, 1.f, 1.f}, f32x4{1.f, 1.f, 1.f, 1.f}};
    if (a.qk_norm) {
      const u32x4 rows[8] = {kr[0], kr[1], kr[2], kr[3], qr[0], qr[1], qr[2], qr[3]};
      norms(rows, n);
    }
    if (m == 0) {
      *reinterpret_cast<f32x4 *>(&s.rk[tq]) = n[0];
      *reinterpret_cast<f32x4 *>(&s.rq[tq]) = n[1];
    }
  }
  // the chain's vectors
  __device__ __forceinline__ void vectors(int buf, int64_t c0) {
    const double c = s.c[buf][lane], end = s.c[buf][kC - 1];
    const float into = decay_of(c), rk = s.rk[lane];
    s.va[buf][lane] = into * rk;
    s.vb[buf][lane] = into * s.rq[lane] * a.scale;
    s.vw[buf][lane] = decay_of(end - c) * rk * s.beta[buf][lane];
    if (lane == kC - 1) s.whole[buf] = into;
    if (SAVE && first) {
      float *vp = keep.vec + (item0 + c0) * kGdrVec;
      vp[lane] = into * rk;
      vp[kC + lane] = into * s.rq[lane] * a.scale;
      vp[2 * kC + lane] = decay_of(end - c) * rk * s.beta[buf][lane];
      vp[3 * kC + lane] = rk;
      vp[4 * kC + lane] = s.rq[lane];
      reinterpret_cast<double *>(vp + 5 * kC)[lane] = c;
    }
  }
  // A' (transposed into LDS) for block row W, M^T for block row 3 - W (kept)
  template <int W>
  __device__ __forceinline__ void products(int buf) {
    constexpr int V = 3 - W;
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
      for (int i = 0; i < kMost; ++i)
        kf[i] = lds_get<u32x4>(lk[kb] + buf * ChunkLds<NT>::kTile + 2 * 16 * i * 16 * NT);
      const u32x4 qf = lds_get<u32x4>(lk[kb] + (2 + buf) * ChunkLds<NT>::kTile + 2 * 16 * V * 16 * NT);
#pragma unroll
      for (int jt = 0; jt <= W; ++jt) ap[jt] = mma(kf[W], kf[jt], ap[jt]);
#pragma unroll
      for (int jt = 0; jt <= V; ++jt) M[jt] = mma(kf[jt], qf, M[jt]);
    }
    double ci[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) ci[e] = c4(buf * kC + 16 * W + e);
    const f32x4 si = f4(kRk, 16 * W);
    float test = 0.f;
#pragma unroll
    for (int jt = 0; jt <= W; ++jt) {
      const double cj = c1(buf * kC + 16 * jt);
      const float sj = f1(kRk, 16 * jt) * f1(kBeta0 + buf, 16 * jt);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = ap[jt][e] * (si[e] * sj) * decay_of(ci[e] - cj);
        ap[jt][e] = jt < W || 4 * g + e > r ? f : 0.f;
        test = fmaf(ap[jt][e], 0.f, test);
      }
      lds_put(la + block(jt, W), ap[jt]);
    }
    // A row that is not finite would reach X's rows before it, 0 times it, where
    // blocks are joined.  It is left out, and the chain told from where on nothing
    // is finite.  (What is kept for the gradients stays as it is.)
    if (!SAVE && __builtin_expect(__any(test != 0.f), 0)) {
#pragma unroll
      for (int jt = 0; jt <= W; ++jt) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!(fabsf(ap[jt][e]) < __builtin_inff())) {
            atomicMin(&s.bad[buf], 16 * W + 4 * g + e);
            ap[jt][e] = 0.f;
          }
        lds_put(la + block(jt, W), ap[jt]);
      }
    }
    const double cv = c1(buf * kC + 16 * V);
    const float sv = f1(kRq, 16 * V) * a.scale;
#pragma unroll
    for (int jt = 0; jt <= V; ++jt) {
      const f32x4 sj = f4(kRk, 16 * jt) * f4(kBeta0 + buf, 16 * jt);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = M[jt][e] * (sv * sj[e]) * decay_of(cv - c4(buf * kC + 16 * jt + e));
        M[jt][e] = jt < V || 4 * g + e <= r ? f : 0.f;
      }
    }
  }
  // The inverses of the four diagonal blocks, by one wave: lane 16 blk + col
  // carries one column through the substitution, the next four rows of the
  // block on their way.
  __device__ __forceinline__ void diagonal() {
    const int blk = g, col = r;
    const uint32_t at = hold(lds_address(&s.at[(blk * 4 - blk * (blk - 1) / 2) * 16 * kAtPitch]));
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.f : 0.f;
#pragma unroll
    for (int k4 = 0; k4 < 16; k4 += 4) {
      f32x4 l[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k)  // A'[16 blk + i][16 blk + k4 + k], i >= k4
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4)
          if (q4 >= k4 / 4) l[k][q4] = lds_get<f32x4>(at + 4 * ((k4 + k) * kAtPitch + 4 * q4));
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i > k4 + k) x[i] = fmaf(-l[k][i / 4][i % 4], x[k4 + k], x[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4)
      lds_put(at + 4 * col * kAtPitch + 16 * q4, f32x4{x[4 * q4], x[4 * q4 + 1], x[4 * q4 + 2], x[4 * q4 + 3]});
  }
  // Block row W of X, transposed tiles: X_Wj^T = -X_jj^T sum_{j<k<=W} A'_kj^T X_Wk^T
  template <int W>
  __device__ __forceinline__ void block_row() {
    f32x4 at[4][4], xj[4];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      xj[j] = lds_get<f32x4>(la + block(j, j));
#pragma unroll
      for (int k = j + 1; k <= W; ++k) at[j][k] = lds_get<f32x4>(la + block(j, k));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) X[W][e] = s.at[at_block(W, W) + (4 * g + e) * kAtPitch + r];
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
  __device__ __forceinline__ void publish(int buf) {
    constexpr int V = 3 - W;
    const uint32_t xw = hold(lds_address(&s.x[buf][0][tri_at(16 * W + r) + 8 * g]));
    const uint32_t mv = hold(lds_address(&s.m[buf][0][mix_at(16 * V + r, g)]));
#pragma unroll
    for (int j = 0; j <= V; ++j) {
      u32x2 p[3];
      split4<3>(M[j], p, minus);
      // block 1 of 32 tokens lies four pieces on, or back
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) lds_put((j < 2 ? mv : mv ^ 64) + pl * ChunkLds<NT>::kMix + 8 * (j % 2), p[pl]);
    }
#pragma unroll
    for (int j = 0; j <= W; ++j) {
      u32x2 p[3];
      split4<3>(X[j], p, minus);
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) lds_put(xw + pl * ChunkLds<NT>::kTri + 2 * kpos(16 * j), p[pl]);
    }
  }
  // Chunk c + 1 beside the chain's chunk c (chunk 0 has nobody to overlap with).
  // One body for both buffers: the eight waves run five programs, and the
  // instruction cache holds 64 KB.
  template <int W>
  __device__ __forceinline__ void run(int64_t nc) {
    load(0);
    if (W == 0) {
      load_gates(0);
      gates(0, 0);
    }
    for (int64_t c = 0; c < nc; ++c) {
      const int buf = static_cast<int>(c & 1);
      stage(buf);
      meet();
      products<W>(buf);
      meet();
      if (W == 1) diagonal();
      if (W == 2) vectors(buf, c);
      if (W == 0) gates(buf ^ 1, (c + 1) * kC);
      if (W != 1) load((c + 1) * kC);
      meet();
      block_row<W>();
      publish<W>(buf);
      if (SAVE && first) {
        constexpr int V = 3 - W;
        float *xm = keep.XM + (item0 + c) * 20 * 256 + 4 * lane;
#pragma unroll
        for (int j = 0; j <= W; ++j) *reinterpret_cast<f32x4 *>(xm + (W * (W + 1) / 2 + j) * 256) = X[j];
#pragma unroll
        for (int j = 0; j <= V; ++j) *reinterpret_cast<f32x4 *>(xm + (10 + V * (V + 1) / 2 + j) * 256) = M[j];
      }
      if (W == 1) load((c + 1) * kC);
      __syncthreads();
    }
    __syncthreads();  // the chain's last chunk
  }
};

template <int NT, bool SAVE>
__global__ __launch_bounds__(kThreads) void gdr_chunk_kernel(GdrArgs a, GdrSaved keep, int64_t ptiles, int cols) {
  __shared__ ChunkLds<NT> s;
  const uint32_t heads = static_cast<uint32_t>(a.H / a.G);  // of a group
  const uint32_t per = heads * static_cast<uint32_t>(ptiles);  // workgroups of a (sequence, group), which share K and Q
  // workgroups of one (sequence, group) on one XCD (consecutive ids go to the
  // 8 XCDs in turn), so that its K and Q come from that L2
  const uint32_t idx = blockIdx.x / 8, bg = blockIdx.x % 8 + 8 * (idx / per), mem = idx % per;
  if (bg >= a.B * a.G) return;
  // the same for the workgroup, and said so: they address buffers
  auto same = [](uint32_t v) { return static_cast<int64_t>(__builtin_amdgcn_readfirstlane(v)); };
  const uint32_t G = static_cast<uint32_t>(a.G);
  const int64_t b = same(bg / G), grp = same(bg % G), h = same(bg % G * heads + mem / static_cast<uint32_t>(ptiles));
  const int64_t p0 = same(mem % static_cast<uint32_t>(ptiles) * cols);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int r = lane % 16, g = lane / 16;
  const int64_t nc = (a.L + kC - 1) / kC;

  // block pairs above the diagonal are read with their 32 tokens and stay 0
  for (int i = threadIdx.x; i < kTriSize / 2; i += kThreads)
#pragma unroll
    for (int bf = 0; bf < 2; ++bf)
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) {
        reinterpret_cast<uint32_t *>(s.x[bf][pl])[i] = 0;
        if (i < kMixSize / 2) reinterpret_cast<uint32_t *>(s.m[bf][pl])[i] = 0;
      }
  if (threadIdx.x == 0) s.met = 0;
  __syncthreads();

  if (wave >= 4) {
    __builtin_amdgcn_s_setprio(3);  // the chain waits for them rather than they for it

    Prepare<NT, SAVE> w{a, keep, (b * a.H + h) * nc, p0 == 0, s, MinusOne(), static_cast<int>(threadIdx.x) - 256, lane, r, g, b, h, grp,
                  a.A[h] * kLog2e, a.dt_bias ? a.dt_bias[h] : 0.f, 0u, {}, {}, 0, 0, 0, 0, 0, 0, {}, {}, {}, {}, {}, {}};
    w.place();
    if (wave == 4) w.template run<0>(nc);
    else if (wave == 5) w.template run<1>(nc);
    else if (wave == 6) w.template run<2>(nc);
    else w.template run<3>(nc);
    return;
  }

  const int64_t p = p0 + 16 * wave + r;
  const uint32_t row = static_cast<uint32_t>(a.H * a.P);
  const bool live = 16 * wave < cols && p0 + 16 * wave < a.P, col = live && p < a.P;  // some column, this lane's column
  const int64_t head = (b * a.L * a.H + h) * a.P;
  Chain<NT, SAVE> w{a, keep, (b * a.H + h) * nc, p, col, s, MinusOne(), r, g, static_cast<const uint16_t *>(a.v) + head, static_cast<bf16_t *>(a.y) + head,
              row, static_cast<uint32_t>(a.P), 32 * row, {}, {}, {}, {}, {}, 0, {}, {}, {}};
  w.place();
#pragma unroll
  for (int e = 0; e < 4; ++e) w.at[e] = col ? 2 * ((4 * g + e) * row + static_cast<uint32_t>(p)) : kNowhere;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    w.S[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (a.h0 != nullptr && col && 16 * nt + 4 * g < a.N)
      w.S[nt] = *reinterpret_cast<const f32x4 *>(a.h0 + ((b * a.H + h) * a.P + p) * a.N + 16 * nt + 4 * g);
  }
  if (live) {
    w.load_v(0, static_cast<int>(a.L < kC ? a.L : kC));
    w.take_v();
  }
  __syncthreads();  // the preparation of chunk 0
  for (int64_t c = 0; c < nc; c += 2) {
    if (live) w.template step<0>(c * kC);
    __syncthreads();
    if (c + 1 < nc) {
      if (live) w.template step<1>((c + 1) * kC);
      __syncthreads();
    }
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
         aligned16(a.k) && aligned16(a.h0) && aligned16(a.h_final) &&
         // the workgroups of the chains, eight groups side by side, in one dimension of
         // fewer than 2^32 threads
         (a.B * a.G + 7) / 8 * 8 * (a.H / a.G) * ((a.P + kCols - 1) / kCols) < (int64_t(1) << 32) / kThreads;
}

namespace {
template <bool SAVE>
hipError_t launch(const GdrArgs &a, const GdrSaved &keep, hipStream_t s) {
  const int cols = gdr_chain_columns(a.B, a.H, a.P);
  const int64_t ptiles = (a.P + cols - 1) / cols, per = a.H / a.G * ptiles;
  const unsigned grid = static_cast<unsigned>((a.B * a.G + 7) / 8 * 8 * per);
  if (a.N <= 64) gdr_chunk_kernel<4, SAVE><<<grid, kThreads, 0, s>>>(a, keep, ptiles, cols);
  else gdr_chunk_kernel<8, SAVE><<<grid, kThreads, 0, s>>>(a, keep, ptiles, cols);
  return hipGetLastError();
}
}  // namespace
hipError_t launch_gdr_chunk(const GdrArgs &a, hipStream_t s) { return launch<false>(a, GdrSaved{}, s); }
hipError_t launch_gdr_chunk_save(const GdrArgs &a, const GdrSaved &keep, hipStream_t s) {
  return launch<true>(a, keep, s);
}

}  // namespace ssm
