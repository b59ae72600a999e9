// Gradients of the gated delta rule by chunks of 64 tokens on the matrix cores
// (gdr_chunk.hip has the forward's formulas and names).
//
// 1. The forward's kernel again, keeping of each chunk the state S0 that enters
//    it, E, the tiles of X and M, and the tokens' vectors.
// 2. The chain backwards, a column of dS per lane as the forward's of S: with
//    dS1 the gradient of the state leaving the chunk,
//      gE = M^T dY + w (K dS1),  W = X^T gE,  dV = W
//      dS0 = exp(c_C) dS1 + Q^T (b dY) - K^T (a W)
//    keeping W and dS1.
// 3. Everything else, chunk by chunk and in parallel.  With the rows k^, q^ of
//    K and Q normalised, D_ij = exp(c_i - c_j), P_ij = dY_i . E_j, V_ij = W_i . E_j:
//      dq^_i = scale (exp(c_i) S0^T dY_i + sum_{j<=i} beta_j D_ij P_ij k^_j)
//      r_i   = -exp(c_i) S0^T W_i - sum_{j<i} beta_j D_ij V_ij k^_j       (k read)
//      T_j   = exp(c_C - c_j) dS1^T E_j + sum_{i>=j} scale D_ij P_ij q^_i
//              - sum_{i>j} D_ij V_ij k^_i                                 (k written)
//      dk^_j = r_j + beta_j T_j,  dbeta_j = k^_j . T_j
//    The gradient of the log decay of token t counts what passes it: reads of
//    S0 by tokens i >= t, writes to S1 by tokens j < t, pairs j < t <= i, and S0
//    as a whole,
//      dlog_t = exp(c_C) <S0, dS1> + sum_{i>=t} (q^_i . first term of dq^_i + k^_i . first of r_i)
//               + sum_{j<t} beta_j k^_j . first term of T_j + sum_{j<t<=i} z_ij,
//      z_ij = beta_j D_ij (scale P_ij q^_i . k^_j - V_ij k^_i . k^_j),
//    all of them sums of what does pass: a step that wipes the state leaves
//    zeros, however large its dt that dA multiplies them by.  (From the finished
//    dq, dk and dbeta the same follows by differences, in which their larger
//    part cancels, i = j above all.)
//
// Operands that are computed (or stored in fp32) are split into three bf16 parts
// throughout: dA and the bias' gradient are sums in fp32 of what goes through
// all of it.
//
// 2 x 4096 tokens, 80 heads of 64 x 128: 1.39 ms; 0.37 for part 1, 0.34 for part 2
// (both bound by the latency of a chunk, as the forward), 0.68 for part 3, which
// moves 2.0 GB (3 TB/s: two states of 32 KB, E and W a head and chunk, and spilled
// registers) and computes 290 products a wave and head (matrix cores busy 22%):
// one workgroup a CU, whose phases -- staging, products, scores -- follow each other.
#include "device_common.h"
#include "gdr.h"
#include "gdr_common.h"
#include "gdr_mfma.h"

namespace ssm {
namespace {

constexpr int kThreads = 512;

// X^T and M^T, [j][i] by kpos(i): rows 0..31 meet 64 tokens, rows 32..63 the
// last 32.
constexpr int kUpSize = 32 * 72 + 32 * 40;
__device__ __forceinline__ constexpr int up_at(int j) { return j < 32 ? j * 72 : 32 * 72 + (j - 32) * 40; }

template <int NT>
struct RevLds {
  __attribute__((aligned(16))) uint16_t k[2][kC * 16 * NT];
  __attribute__((aligned(16))) uint16_t q[2][kC * 16 * NT];
  __attribute__((aligned(16))) uint16_t x[2][3][kUpSize];
  __attribute__((aligned(16))) uint16_t m[2][3][kUpSize];
  __attribute__((aligned(16))) float va[2][kC], vb[2][kC], vw[2][kC];
  float whole[2];
  static constexpr uint32_t kTile = 2 * kC * 16 * NT, kTri = 2 * kUpSize;
};

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------- 2. the chain backwards
// The matrix cores' sums round downwards by a little, which shows in a gradient
// that sums over all tokens.  All here is linear in dY and dS1, so every other
// chunk (from the last, which is in buffer 0, backwards) is computed with both
// negated, and W and dS1 are kept so: what is rounded away changes its sign with
// the chunk.  Error of dA over 2 x 4096 tokens: 8.2e-7 -> 2.4e-7 (fp32 products
// with round to nearest: 2.5e-7), at no cost.
template <int NT>
struct RevChain {
  static constexpr int KB = NT / 2;
  const GdrBwdArgs &ba;
  const GdrSaved &keep;
  const int64_t item0, p;  // of this head and chunk 0; this lane's column
  const bool col;          // which is inside P
  RevLds<NT> &s;
  const MinusOne minus;
  const int r, g;          // lane = 16 g + r
  const uint16_t *dy;      // of this head, token 0
  uint16_t *dv;
  const uint32_t row, width, rows16;
  uint32_t at[4];
  uint32_t lk[KB], lt[KB], lx[2], lm[2], lv;
  f32x4 dS[NT];
  uint16_t dr[16];   // dY of the chunk to come, on its way
  u32x4 dO[2];       // and of this one, as an operand

  __device__ __forceinline__ void place() {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      lk[kb] = hold(lds_address(&s.k[0][tile_at<NT>(r, 4 * kb + g)]));
      lt[kb] = hold(lds_address(&s.k[0][tile_at<NT>(4 * g + r / 4, 4 * kb + r % 4)]));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // rows r and 32 + r
      lx[i] = hold(lds_address(&s.x[0][0][up_at(32 * i + r) + 8 * g]));
      lm[i] = hold(lds_address(&s.m[0][0][up_at(32 * i + r) + 8 * g]));
    }
    lv = hold(lds_address(&s.va[0][4 * g]));
  }
  // rows 16 jt + r of X^T or M^T, block kb (jt >= 2: block 1 alone)
  template <int buf>
  __device__ __forceinline__ u32x4 row_up(const uint32_t (&base)[2], int part, int jt, int kb) const {
    return lds_get<u32x4>(base[jt / 2] + (3 * buf + part) * RevLds<NT>::kTri +
                          2 * (up_at(16 * jt) - up_at(32 * (jt / 2)) + 32 * (kb - jt / 2)));
  }
  template <int buf>
  __device__ __forceinline__ f32x4 vec(int w, int rt) const {
    return lds_get<f32x4>(lv + 4 * ((2 * w + buf) * kC + 16 * rt));
  }
  __device__ __forceinline__ void load_dy(int64_t t0) {
    const int left = t0 < 0 ? 0 : static_cast<int>(ba.f.L - t0 < kC ? ba.f.L - t0 : kC);
    const __amdgpu_buffer_rsrc_t rd = rows_of(dy + (t0 < 0 ? 0 : t0) * row, left, row, width);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      dr[i] = __builtin_amdgcn_raw_buffer_load_b16(rd, static_cast<int>(at[i % 4]), static_cast<int>(i / 4 * rows16), 0);
  }
  template <int buf>  // with the sign of a chunk in that buffer
  __device__ __forceinline__ void take_dy() {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w = dr[8 * kb + 2 * e] | static_cast<uint32_t>(dr[8 * kb + 2 * e + 1]) << 16;
        asm volatile("" : "+v"(w));
        dO[kb][e] = buf == 0 ? w : w ^ 0x80008000u;
      }
  }
  // Zeros for dY's values that are not finite; the last such token of this lane's
  // column, -1 where there is none.
  __device__ __forceinline__ int leave_out() {
    int bad = -1;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t w = dO[i / 8][i % 8 / 2], half = i % 2 ? 0x7f800000u : 0x7f80u;
      if ((w & half) == half) {
        dO[i / 8][i % 8 / 2] = w & (i % 2 ? 0xffffu : 0xffff0000u);
        bad = 16 * (i / 4) + 4 * g + i % 4;
      }
    }
    bad = max(bad, __shfl_xor(bad, 16));
    return max(bad, __shfl_xor(bad, 32));
  }
  // dY of row tile rt in fp32
  __device__ __forceinline__ f32x4 dy_f32(int rt) const {
    const uint32_t lo = dO[rt / 2][rt % 2 * 2], hi = dO[rt / 2][rt % 2 * 2 + 1];
    return f32x4{__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u), __uint_as_float(hi << 16),
                 __uint_as_float(hi & 0xffff0000u)};
  }

  template <int buf>
  __device__ __forceinline__ void step(int64_t c) {
    const int64_t t0 = c * kC, item = item0 + c;
    const int left = static_cast<int>(ba.f.L - t0 < kC ? ba.f.L - t0 : kC);
    if (col)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (16 * nt + 4 * g < ba.f.N)
          *reinterpret_cast<f32x4 *>(keep.dS + (item * ba.f.P + p) * ba.f.N + 16 * nt + 4 * g) = dS[nt];
    // A dY that is not finite is left out of the products, where 0 times it would
    // reach the tokens behind it; what it enters is set below.
    u16x2 most = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, dO[i / 4][i % 4] & 0x7fff7fffu));
    const bool any_bad = __any(most[0] >= 0x7f80 || most[1] >= 0x7f80);
    int bad = -1;
    if (__builtin_expect(any_bad, 0)) bad = leave_out();
    // K dS1
    f32x4 G[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) G[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 sp[2][3];
    split_operand<3>(dS[0], dS[1], sp[0], minus);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      u32x4 ka[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) ka[rt] = lds_get<u32x4>(lk[kb] + buf * RevLds<NT>::kTile + 2 * 16 * rt * 16 * NT);
      if (kb + 1 < KB) split_operand<3>(dS[2 * kb + 2], dS[2 * kb + 3], sp[(kb + 1) % 2], minus);
#pragma unroll
      for (int pl = 2; pl >= 0; --pl)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) G[rt] = mma(ka[rt], sp[kb % 2][pl], G[rt]);
    }
    __builtin_amdgcn_sched_barrier(0);
    // gE = w (K dS1) + M^T dY
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) G[rt] = G[rt] * vec<buf>(2, rt);
#pragma unroll
    for (int mp = 2; mp >= 0; --mp) {
      u32x4 ma[4][2];
#pragma unroll
      for (int jt = 0; jt < 4; ++jt)
#pragma unroll
        for (int kb = jt / 2; kb < 2; ++kb) ma[jt][kb] = row_up<buf>(lm, mp, jt, kb);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int jt = 0; jt < 2 * kb + 2; ++jt) G[jt] = mma(ma[jt][kb], dO[kb], G[jt]);
    }
    __builtin_amdgcn_sched_barrier(0);
    // W = X^T gE
    f32x4 Wv[4];
    {
      u32x4 gp[2][3];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) split_operand<3>(G[2 * kb], G[2 * kb + 1], gp[kb], minus);
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) Wv[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int xp = 2; xp >= 0; --xp) {
        u32x4 xa[4][2];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
#pragma unroll
          for (int kb = jt / 2; kb < 2; ++kb) xa[jt][kb] = row_up<buf>(lx, xp, jt, kb);
#pragma unroll
        for (int pl = 2 - xp; pl >= 0; --pl)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int jt = 0; jt < 2 * kb + 2; ++jt) Wv[jt] = mma(xa[jt][kb], gp[kb][pl], Wv[jt]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // dS0 = whole dS1 + Q^T (b dY) - K^T (a W), its sign turned for the next chunk
    {
      u32x4 up[2][2][3];  // of K, of Q
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        split_operand<3>(Wv[2 * kb] * vec<buf>(0, 2 * kb), Wv[2 * kb + 1] * vec<buf>(0, 2 * kb + 1), up[0][kb], minus);
        split_operand<3>(-(dy_f32(2 * kb) * vec<buf>(1, 2 * kb)), -(dy_f32(2 * kb + 1) * vec<buf>(1, 2 * kb + 1)), up[1][kb], minus);
      }
      const float whole = -s.whole[buf];
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dS[n0 + i] = dS[n0 + i] * whole;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          u32x4 kt[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
              u32x2 half[2];
#pragma unroll
              for (int u = 0; u < 2; ++u)
                half[u] = lds_transposed(lt[(n0 + i) / 2] + (2 * o + buf) * RevLds<NT>::kTile +
                                         2 * ((32 * kb + 16 * u) * 16 * NT + 4 * ((n0 + i) % 2)));
              kt[i][kb] = u32x4{half[0][0], half[0][1], half[1][0], half[1][1]};
            }
#pragma unroll
          for (int pl = 2; pl >= 0; --pl)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
              for (int i = 0; i < 4; ++i) dS[n0 + i] = mma(kt[i][kb], up[o][kb][pl], dS[n0 + i]);
        }
      }
    }
    if (__builtin_expect(any_bad, 0)) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (16 * (i / 4) + 4 * g + i % 4 <= bad) Wv[i / 4][i % 4] = __builtin_nanf("");
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (bad >= 0) dS[nt][e] = __builtin_nanf("");
    }
    __builtin_amdgcn_sched_barrier(0);
    take_dy<1 - buf>();   // before anything stored after them has to be waited for
    load_dy(t0 - 2 * kC);
    __builtin_amdgcn_sched_barrier(0);
    const __amdgpu_buffer_rsrc_t rv = rows_of(dv + t0 * row, left, row, width);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      __builtin_amdgcn_raw_buffer_store_b16(from_f32<bf16_t>(buf == 0 ? Wv[i / 4][i % 4] : -Wv[i / 4][i % 4]).bits, rv, static_cast<int>(at[i % 4]),
                                            static_cast<int>(i / 4 * rows16), 0);
    if (col) {
      float *wp = keep.W + (item * kC + 4 * g) * ba.f.P + p;
#pragma unroll
      for (int i = 0; i < 16; ++i) wp[(16 * (i / 4) + i % 4) * ba.f.P] = Wv[i / 4][i % 4];
    }
  }
};

// The other four waves: K, Q, X^T, M^T and the vectors of the chunk before.
template <int NT>
struct RevPrepare {
  const GdrArgs &a;
  const GdrSaved &keep;
  const int64_t item0;
  RevLds<NT> &s;
  const MinusOne minus;
  const int tid, lane, wave, r, g;
  const int64_t b, h, grp;
  static constexpr int kPieces = 2 * NT, kLoaders = kPieces * kC / 4;
  uint32_t lp[4][2], piece, lx[2], lm[2];
  u32x4 kr[4], qr[4];
  f32x4 tile[5];
  float vec[3];
  double end;

  __device__ __forceinline__ void place() {
    const int m = tid % kPieces, pos = kpos(8 * m), tq = 4 * (tid / kPieces) % kC;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) lp[i][u] = hold(lds_address(&s.k[0][tile_at<NT>(tq + i, pos / 8 + u) + pos % 8]));
    piece = tid < kLoaders && 8 * m < a.N ? 2 * (tq * static_cast<uint32_t>(a.G * a.N) + 8 * m) : kNowhere;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lx[i] = hold(lds_address(&s.x[0][0][up_at(32 * i + r) + 8 * g]));
      lm[i] = hold(lds_address(&s.m[0][0][up_at(32 * i + r) + 8 * g]));
    }
  }
  // Tile n of a triangle: block row i and column j, row after row.
  static __device__ __forceinline__ constexpr int tile_i(int n) { return n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3; }
  static __device__ __forceinline__ constexpr int tile_j(int n) { return n - tile_i(n) * (tile_i(n) + 1) / 2; }
  template <int W>
  __device__ __forceinline__ void load(int64_t c) {
    const int64_t t0 = c * kC;
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
    // element (j' = r, i' = 4 g + e) of a tile whose lane 16 (j' / 4) + i' holds rows 4 (j' / 4) .. of column i'
    const float *xm = keep.XM + (item0 + c) * 20 * 256 + 64 * (r / 4) + 16 * g + r % 4;
#pragma unroll
    for (int i = 0; i < 5; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) tile[i][e] = xm[(4 * i + W) * 256 + 4 * e];
    if (W == 0) {
      const float *vp = keep.vec + (item0 + c) * kGdrVec;
#pragma unroll
      for (int i = 0; i < 3; ++i) vec[i] = vp[i * kC + lane];
      end = reinterpret_cast<const double *>(vp + 5 * kC)[kC - 1];
    }
  }
  template <int W>
  __device__ __forceinline__ void stage(int buf) {
    if (tid < kLoaders)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t at = lp[i][u] + buf * RevLds<NT>::kTile;
          lds_put(at, u32x2{kr[i][2 * u], kr[i][2 * u + 1]});
          lds_put(at + 2 * RevLds<NT>::kTile, u32x2{qr[i][2 * u], qr[i][2 * u + 1]});
        }
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      constexpr int kAll = 10;
      const int n = 4 * i + W, ti = tile_i(n % kAll), tj = tile_j(n % kAll);
      u32x2 p[3];
      split4<3>(tile[i], p, minus);
      const uint32_t at = (n < kAll ? lx : lm)[tj / 2] + 3 * buf * RevLds<NT>::kTri +
                          2 * (up_at(16 * tj) - up_at(32 * (tj / 2)) + kpos(16 * ti) - 32 * (tj / 2));
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) lds_put(at + pl * RevLds<NT>::kTri, p[pl]);
    }
    if (W == 0) {
      s.va[buf][lane] = vec[0];
      s.vb[buf][lane] = vec[1];
      s.vw[buf][lane] = vec[2];
      if (lane == 0) s.whole[buf] = decay_of(end);
    }
  }
  template <int W>
  __device__ __forceinline__ void run(int64_t nc) {
    load<W>(nc - 1);
    for (int64_t i = 0; i < nc; ++i) {
      stage<W>(static_cast<int>(i & 1));
      if (i + 1 < nc) load<W>(nc - 2 - i);
      __syncthreads();
    }
    __syncthreads();  // the chain's last chunk
  }
};

template <int NT>
__global__ __launch_bounds__(kThreads) void gdr_bwd_chain_kernel(GdrBwdArgs ba, GdrSaved keep, int64_t ptiles, int cols) {
  __shared__ RevLds<NT> s;
  const GdrArgs &a = ba.f;
  const uint32_t heads = static_cast<uint32_t>(a.H / a.G), per = heads * static_cast<uint32_t>(ptiles);
  const uint32_t idx = blockIdx.x / 8, bg = blockIdx.x % 8 + 8 * (idx / per), mem = idx % per;  // as the forward's
  if (bg >= a.B * a.G) return;
  auto same = [](uint32_t v) { return static_cast<int64_t>(__builtin_amdgcn_readfirstlane(v)); };
  const uint32_t G = static_cast<uint32_t>(a.G);
  const int64_t b = same(bg / G), grp = same(bg % G), h = same(bg % G * heads + mem / static_cast<uint32_t>(ptiles));
  const int64_t p0 = same(mem % static_cast<uint32_t>(ptiles) * cols);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int r = lane % 16, g = lane / 16;
  const int64_t nc = (a.L + kC - 1) / kC, item0 = (b * a.H + h) * nc;

  // blocks below the diagonal are read with their 32 tokens and stay 0
  for (int i = threadIdx.x; i < kUpSize / 2; i += kThreads)
#pragma unroll
    for (int bf = 0; bf < 2; ++bf)
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) {
        reinterpret_cast<uint32_t *>(s.x[bf][pl])[i] = 0;
        reinterpret_cast<uint32_t *>(s.m[bf][pl])[i] = 0;
      }
  __syncthreads();

  if (wave >= 4) {
    __builtin_amdgcn_s_setprio(3);
    RevPrepare<NT> w{a, keep, item0, s, MinusOne(), static_cast<int>(threadIdx.x) - 256, lane, wave - 4, r, g, b, h, grp,
                     {}, 0, {}, {}, {}, {}, {}, {}, 0.0};
    w.place();
    if (wave == 4) w.template run<0>(nc);
    else if (wave == 5) w.template run<1>(nc);
    else if (wave == 6) w.template run<2>(nc);
    else w.template run<3>(nc);
    return;
  }

  const int64_t p = p0 + 16 * wave + r;
  const uint32_t row = static_cast<uint32_t>(a.H * a.P);
  const bool live = 16 * wave < cols && p0 + 16 * wave < a.P, col = live && p < a.P;
  const int64_t head = (b * a.L * a.H + h) * a.P;
  RevChain<NT> w{ba, keep, item0, p, col, s, MinusOne(), r, g, static_cast<const uint16_t *>(ba.dy) + head,
                 static_cast<uint16_t *>(ba.dv) + head, row, static_cast<uint32_t>(a.P), 32 * row,
                 {}, {}, {}, {}, {}, 0, {}, {}, {}};
  w.place();
#pragma unroll
  for (int e = 0; e < 4; ++e) w.at[e] = col ? 2 * ((4 * g + e) * row + static_cast<uint32_t>(p)) : kNowhere;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    w.dS[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (ba.dh_final != nullptr && col && 16 * nt + 4 * g < a.N)
      w.dS[nt] = *reinterpret_cast<const f32x4 *>(ba.dh_final + ((b * a.H + h) * a.P + p) * a.N + 16 * nt + 4 * g);
  }
  if (live) {
    w.load_dy((nc - 1) * kC);
    w.template take_dy<0>();
    w.load_dy((nc - 2) * kC);
  }
  __syncthreads();  // the preparation of the last chunk
  for (int64_t i = 0; i < nc; i += 2) {
    if (live) w.template step<0>(nc - 1 - i);
    __syncthreads();
    if (i + 1 < nc) {
      if (live) w.template step<1>(nc - 2 - i);
      __syncthreads();
    }
  }
  if (ba.dh0 != nullptr && col)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (16 * nt + 4 * g < a.N)
        *reinterpret_cast<f32x4 *>(ba.dh0 + ((b * a.H + h) * a.P + p) * a.N + 16 * nt + 4 * g) = nc % 2 ? -w.dS[nt] : w.dS[nt];
}

// ------------------------------------------------------- 3. the other gradients
constexpr int kPitch = 72;  // uint16 per row of 64

template <int NT>
struct GradLds {
  // the small ones first, within the offsets that instructions hold
  __attribute__((aligned(16))) double c[kC];
  __attribute__((aligned(16))) float rk[kC], rq[kC], beta[kC], dt[kC];
  float head[4];  // A, bias
  float rows[2][3][kC];  // per half of N: the reads of S0, k^.T, k^.(first term of T)
  // z: sums of a column in a row tile below its own, of a row left of its
  // diagonal tile, and of the pairs of the diagonal tile that pass a token
  float cols[4][kC], zrow[kC], zdiag[kC];
  float dot[8];
  __attribute__((aligned(16))) uint16_t k[kC * 16 * NT], q[kC * 16 * NT];
  __attribute__((aligned(16))) uint16_t dy[kC * kPitch];         // [token][p by kpos]
  __attribute__((aligned(16))) uint16_t e[3][kC * kPitch];
  __attribute__((aligned(16))) uint16_t w[3][kC * kPitch];
  __attribute__((aligned(16))) uint16_t st[3][16 * NT * kPitch]; // [n][p by kpos], S0 then dS1
};

// One workgroup per (sequence, chunk, group): its heads one after the other, the
// sums over them in registers.  Wave 4 u + t: row tile t, half u of N.
// FOUR: P is a multiple of 4 (as a choice made here, at each load, it would make
// each wait for its value).
// SPLIT: the heads of a group are shared by `split` workgroups.
template <int NT, bool FOUR, bool SPLIT>
__global__ __launch_bounds__(kThreads) void gdr_bwd_grads_kernel(GdrBwdArgs ba, GdrSaved keep, int64_t split,
                                                                                        float *qk_part, float *red) {
  constexpr int NH = NT / 2;  // tiles of N per wave
  __shared__ GradLds<NT> s;
  const GdrArgs &a = ba.f;
  const int64_t nc = (a.L + kC - 1) / kC, heads = a.H / a.G;
  const int64_t part = SPLIT ? blockIdx.z % split : 0;
  const int64_t grp = blockIdx.y, b = SPLIT ? blockIdx.z / split : blockIdx.z, c = blockIdx.x;
  const int64_t before = SPLIT ? part * heads / split : 0;
  const int64_t first_head = grp * heads + before, count = SPLIT ? (part + 1) * heads / split - before : heads;
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int r = lane % 16, g = lane / 16, own = wave % 4, half = wave / 4;
  const MinusOne minus;
  const int64_t t0 = c * kC, P = a.P, N = a.N;
  const int left = static_cast<int>(a.L - t0 < kC ? a.L - t0 : kC);

  // K and Q
  constexpr int kPieces = 2 * NT;
  for (int i = tid; i < kC * kPieces; i += kThreads) {
    const int tok = i / kPieces, m = i % kPieces, pos = kpos(8 * m);
    u32x4 kr = {0, 0, 0, 0}, qr = {0, 0, 0, 0};
    if (tok < left && 8 * m < N) {
      const int64_t at = ((b * a.L + t0 + tok) * a.G + grp) * N + 8 * m;
      kr = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.k) + at);
      qr = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.q) + at);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = tile_at<NT>(tok, pos / 8 + u) + pos % 8;
      *reinterpret_cast<u32x2 *>(&s.k[at]) = u32x2{kr[2 * u], kr[2 * u + 1]};
      *reinterpret_cast<u32x2 *>(&s.q[at]) = u32x2{qr[2 * u], qr[2 * u + 1]};
    }
  }
  __syncthreads();
  // K (low) and Q (high) at the places of a result: rows 16 own + 4 g + e, columns n
  uint32_t kq[NH][4];
#pragma unroll
  for (int i = 0; i < NH; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int pos = kpos(16 * (NH * half + i) + r / 4 * 4) + r % 4;
      const int at = tile_at<NT>(16 * own + 4 * g + e, pos / 8) + pos % 8;
      kq[i][e] = s.k[at] | static_cast<uint32_t>(s.q[at]) << 16;
    }
  auto k_at = [&](int i, int e) { return __uint_as_float(kq[i][e] << 16); };
  auto q_at = [&](int i, int e) { return __uint_as_float(kq[i][e] & 0xffff0000u); };

  f32x4 GQ[NH], GK[NH];
#pragma unroll
  for (int i = 0; i < NH; ++i) GQ[i] = GK[i] = f32x4{0.f, 0.f, 0.f, 0.f};

  // columns 16 nt .. of K (o = 0) or Q (1) over 32 tokens, as an operand
  uint32_t lt[NH];
#pragma unroll
  for (int i = 0; i < NH; ++i)
    lt[i] = hold(lds_address(&s.k[tile_at<NT>(4 * g + r / 4, 4 * ((NH * half + i) / 2) + r % 4) + 4 * ((NH * half + i) % 2)]));
  auto columns = [&](int o, int i, int kb) {
    u32x2 u[2];
#pragma unroll
    for (int w = 0; w < 2; ++w)
      u[w] = lds_transposed(lt[i] + 2 * (o * kC * 16 * NT + (32 * kb + 16 * w) * 16 * NT));
    return u32x4{u[0][0], u[0][1], u[1][0], u[1][1]};
  };
  const uint32_t l_row = hold(2 * (r * kPitch + 8 * g));  // row r, slot g of a tile of rows
  const uint32_t l_dy = hold(lds_address(s.dy) + l_row), l_st = hold(lds_address(s.st[0]) + l_row);
  constexpr uint32_t kPart = 2 * kC * kPitch, kStPart = 2 * 16 * NT * kPitch, kTileRows = 2 * 16 * kPitch;

  const uint32_t l_rows = hold(lds_address(&s.dy[tid / 16 * kPitch + kpos(4 * (tid % 16))]));  // E and W behind dY
  const uint32_t l_k = hold(lds_address(&s.k[r * 16 * NT]));  // row r of a tile of K, its pieces exchanged
  const uint32_t swap = tile_at<NT>(r, 0) / 8 % (2 * NT);
  constexpr uint32_t kKTile = 2 * 16 * 16 * NT;
  const int ptiles = static_cast<int>((P + kCols - 1) / kCols);
  // What a thread loads of a head's columns p0 .. + 63: two times 4 columns of a
  // token of E, W and dY, and 4 p by 4 n of a state.  Always a step ahead of
  // where it is staged.
  f32x4 ev[2], wv[2], sv[4];
  u32x2 yv[2];
  auto load_rows = [&](int64_t h, int p0) {
    const int64_t item = (b * a.H + h) * nc + c;
    const uint32_t bytes = static_cast<uint32_t>(4 * kC * P);
    const __amdgpu_buffer_rsrc_t re = buffer_of(keep.E + item * kC * P, bytes), rw = buffer_of(keep.W + item * kC * P, bytes);
    const uint32_t row = static_cast<uint32_t>(a.H * P);
    const __amdgpu_buffer_rsrc_t ry =
        rows_of(static_cast<const uint16_t *>(ba.dy) + ((b * a.L + t0) * a.H + h) * P, left, row, static_cast<uint32_t>(P));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int me = hold(tid), tok = (me + i * kThreads) / 16, p = p0 + 4 * (me % 16);
      const uint32_t at = p < P ? 4 * (static_cast<uint32_t>(tok * P) + p) : kNowhere;
      ev[i] = __builtin_bit_cast(f32x4, buffer_b128(re, at));
      wv[i] = __builtin_bit_cast(f32x4, buffer_b128(rw, at));
      const uint32_t yat = p < P ? 2 * (tok * row + p) : kNowhere;
      if constexpr (FOUR) {
        yv[i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(ry, static_cast<int>(yat), 0, 0));
      } else {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[e] = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(
              ry, static_cast<int>(p + e < P ? yat + 2 * e : kNowhere), 0, 0));
        yv[i] = u32x2{y[0] | y[1] << 16, y[2] | y[3] << 16};
      }
    }
  };
  const float sign = (nc - 1 - c) % 2 ? -1.f : 1.f;  // as the chain's
  const uint32_t flip = (nc - 1 - c) % 2 ? 0x80008000u : 0u;
  auto stage_rows = [&](int p0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q4 = tid % 16;
      if constexpr (!FOUR)  // the columns behind P belong to the next row
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (p0 + 4 * q4 + e >= P) ev[i][e] = wv[i][e] = 0.f;
      u32x2 ep[3], wp[3];
      split4<3>(ev[i], ep, minus);
      split4<3>(wv[i], wp, minus);
      const uint32_t to = l_rows + i * 2 * kTileRows;  // 32 tokens on
      lds_put(to, u32x2{yv[i][0] ^ flip, yv[i][1] ^ flip});
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) {
        lds_put(to + (1 + pl) * kPart, ep[pl]);
        lds_put(to + (4 + pl) * kPart, wp[pl]);
      }
    }
  };
  const int st_p = 4 * (tid % 16), st_n = 4 * (tid / 16);
  const uint32_t l_stage = hold(lds_address(&s.st[0][(st_n < 16 * NT ? st_n : 0) * kPitch + kpos(st_p)]));
  auto load_state = [&](const float *from, int64_t h, int p0) {
    const int64_t item = (b * a.H + h) * nc + c;
    const __amdgpu_buffer_rsrc_t rs = buffer_of(from + item * P * N, static_cast<uint32_t>(4 * P * N));
    const int me = hold(tid), st_p = 4 * (me % 16), st_n = 4 * (me / 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = p0 + st_p + e;
      sv[e] = __builtin_bit_cast(
          f32x4, buffer_b128(rs, p < P && st_n < N ? 4 * (static_cast<uint32_t>(p * N) + st_n) : kNowhere));
    }
  };
  auto stage_state = [&]() {  // turned to rows of n
    if (st_n >= 16 * NT) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x2 sp[3];
      split4<3>(f32x4{sv[0][j], sv[1][j], sv[2][j], sv[3][j]}, sp, minus);
#pragma unroll
      for (int pl = 0; pl < 3; ++pl)
        lds_put(l_stage + pl * kStPart + j * 2 * kPitch, sp[pl]);
    }
  };
  // products of two three-part operands, small terms first
  constexpr int kA[6] = {2, 0, 1, 1, 0, 0}, kB[6] = {0, 2, 1, 0, 1, 0};

  // What is one number a token, a head ahead: an array (half of c) a wave, and A and
  // the bias, in one register.
  uint32_t gw = 0;
  auto load_gates = [&](int64_t h) {
    const uint32_t *vp = reinterpret_cast<const uint32_t *>(keep.vec + ((b * a.H + h) * nc + c) * kGdrVec);
    const __amdgpu_buffer_rsrc_t words = buffer_of(
        wave < 2 ? vp + 5 * kC + wave : wave < 4 ? vp + (1 + wave) * kC : wave == 6 ? reinterpret_cast<const uint32_t *>(a.A + h)
                                                                      : reinterpret_cast<const uint32_t *>(a.dt_bias + h),
        wave < 2 ? 8 * kC - 4 : wave < 4 ? 4 * kC : wave == 6 || a.dt_bias ? 4 : 0);
    const __amdgpu_buffer_rsrc_t halves =
        rows_of(static_cast<const uint16_t *>(wave == 4 ? a.beta : a.dt) + (b * a.L + t0) * a.H + h, left,
                static_cast<uint32_t>(a.H), 1);
    if (wave == 4 || wave == 5)
      gw = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(halves, 2 * lane * static_cast<int>(a.H), 0, 0));
    else
      gw = __builtin_amdgcn_raw_buffer_load_b32(words, (wave < 2 ? 8 : 4) * lane, 0, 0);
  };
  auto stage_gates = [&]() {
    if (wave < 2) reinterpret_cast<uint32_t *>(s.c)[2 * lane + wave] = gw;
    else if (wave == 2 || wave == 3) (wave == 2 ? s.rk : s.rq)[lane] = __uint_as_float(gw);
    else if (wave == 4 || wave == 5) (wave == 4 ? s.beta : s.dt)[lane] = __uint_as_float(gw << 16);
    else if (lane == 0) s.head[wave - 6] = __uint_as_float(gw);
  };

  load_gates(first_head);
  load_rows(first_head, 0);
  load_state(keep.S, first_head, 0);
  for (int64_t hh = 0; hh < count; ++hh) {
    const int64_t h = first_head + hh;
    // What comes from the lane is made anew for each head and part, not kept in registers.
    int r = hold(lane % 16), g = hold(lane / 16);
#pragma unroll
    for (int i = 0; i < NH; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) kq[i][e] = hold(kq[i][e]);
    __syncthreads();  // the head before
    stage_gates();
    // what goes through the states
    f32x4 DQ[NH], KR[NH], T[NH];
#pragma unroll
    for (int i = 0; i < NH; ++i) DQ[i] = KR[i] = T[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float dot = 0.f;
    for (int pt = 0; pt < ptiles; ++pt) {
      const int p0 = pt * kCols;
      if (pt > 0) {
        __syncthreads();
        load_rows(h, p0);
        load_state(keep.S, h, p0);
      }
      stage_rows(p0);
      stage_state();
      f32x4 before[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) before[e] = sv[e];
      load_state(keep.dS, h, p0);
      __syncthreads();
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const uint32_t mine = own * kTileRows + 64 * kb;
        const u32x4 dyo = lds_get<u32x4>(l_dy + mine);
        u32x4 wo[3];
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) wo[pl] = lds_get<u32x4>(l_dy + (4 + pl) * kPart + mine);
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          u32x4 sb[3];
#pragma unroll
          for (int pl = 0; pl < 3; ++pl)
            sb[pl] = lds_get<u32x4>(l_st + pl * kStPart + (NH * half + i) * kTileRows + 64 * kb);
#pragma unroll
          for (int k = 0; k < 6; ++k) {
            KR[i] = mma(wo[kA[k]], sb[kB[k]], KR[i]);
            if (k % 2 == 1) DQ[i] = mma(dyo, sb[2 - k / 2], DQ[i]);
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) dot = fmaf(sv[e][j], before[e][j], dot);
      stage_state();
      __syncthreads();
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        u32x4 eo[3];
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) eo[pl] = lds_get<u32x4>(l_dy + (1 + pl) * kPart + own * kTileRows + 64 * kb);
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          u32x4 sb[3];
#pragma unroll
          for (int pl = 0; pl < 3; ++pl)
            sb[pl] = lds_get<u32x4>(l_st + pl * kStPart + (NH * half + i) * kTileRows + 64 * kb);
#pragma unroll
          for (int k = 0; k < 6; ++k) T[i] = mma(eo[kA[k]], sb[kB[k]], T[i]);
        }
      }
    }
    f32x4 first = {0.f, 0.f, 0.f, 0.f}, read = first;  // k^ . (first term of T), and of S0's reads
    const f32x4 rko = *reinterpret_cast<const f32x4 *>(&s.rk[16 * own + 4 * g]);
    const f32x4 rqo = *reinterpret_cast<const f32x4 *>(&s.rq[16 * own + 4 * g]);
    {
      f32x4 into, out;
      const double end = s.c[kC - 1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const double ct = s.c[16 * own + 4 * g + e];
        into[e] = decay_of(ct);
        out[e] = decay_of(end - ct);
      }
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        DQ[i] = DQ[i] * (into * a.scale);
        KR[i] = -(KR[i] * into);
        T[i] = T[i] * out;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          first[e] = fmaf(k_at(i, e), T[i][e], first[e]);
          read[e] = fmaf(q_at(i, e) * rqo[e], DQ[i][e], fmaf(k_at(i, e) * rko[e], KR[i][e], read[e]));
        }
      }
    }
    r = hold(r), g = hold(g);
    // the scores.  Rows j and the own tile's i as columns: such a result is an
    // operand with the tokens i as rows.
    const double c_own = s.c[16 * own + r];
    {
      f32x4 PT[4], VT[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) PT[i] = VT[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int pt = 0; pt < ptiles; ++pt) {
        if (ptiles > 1) {
          __syncthreads();
          load_rows(h, pt * kCols);
          stage_rows(pt * kCols);
          __syncthreads();
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const uint32_t mine = own * kTileRows + 64 * kb;
          const u32x4 dyo = lds_get<u32x4>(l_dy + mine);
          u32x4 wo[3];
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) wo[pl] = lds_get<u32x4>(l_dy + (4 + pl) * kPart + mine);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j <= own) {
              u32x4 ej[3];
#pragma unroll
              for (int pl = 0; pl < 3; ++pl) ej[pl] = lds_get<u32x4>(l_dy + (1 + pl) * kPart + j * kTileRows + 64 * kb);
#pragma unroll
              for (int k = 0; k < 6; ++k) {
                VT[j] = mma(ej[kA[k]], wo[kB[k]], VT[j]);
                if (k % 2 == 1) PT[j] = mma(ej[2 - k / 2], dyo, PT[j]);
              }
            }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= own) {
          const f32x4 rkj = *reinterpret_cast<const f32x4 *>(&s.rk[16 * j + 4 * g]);
          const f32x4 bej = *reinterpret_cast<const f32x4 *>(&s.beta[16 * j + 4 * g]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = rkj[e] * bej[e] * decay_of(c_own - s.c[16 * j + 4 * g + e]);
            PT[j][e] = j < own || 4 * g + e <= r ? PT[j][e] * (f * a.scale) : 0.f;
            VT[j][e] = j < own || 4 * g + e < r ? -(VT[j][e] * f) : 0.f;
          }
        }
      if (half == 0) {  // z: the scores by q . k and k . k
        float zrow = 0.f;
        const float rq_own = s.rq[16 * own + r], rk_own = s.rk[16 * own + r];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 z = {0.f, 0.f, 0.f, 0.f};
          if (j <= own) {
            f32x4 gq = z, gk = z;
#pragma unroll
            for (int kb = 0; kb < NH; ++kb) {
              const uint32_t at = l_k + 2 * 8 * ((4 * kb + g) ^ swap);
              const u32x4 kj = lds_get<u32x4>(at + j * kKTile);
              gq = mma(kj, lds_get<u32x4>(at + own * kKTile + 2 * kC * 16 * NT), gq);
              gk = mma(kj, lds_get<u32x4>(at + own * kKTile), gk);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = fmaf(PT[j][e], gq[e] * rq_own, VT[j][e] * (gk[e] * rk_own));
          }
          if (j != own) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              zrow += z[e];
              z[e] = row_sum<16>(z[e]);
            }
            if (r == 0) *reinterpret_cast<f32x4 *>(&s.cols[own][16 * j + 4 * g]) = z;
          } else {
            // sum over j < t <= i, t = 4 g + e: down each column, then along the rows
            float sum[5];
            sum[0] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e + 1] = sum[e] + (4 * g + e < r ? z[e] : 0.f);
            float above = 0.f;
#pragma unroll
            for (int gg = 0; gg < 3; ++gg) {
              const float o = __shfl(sum[4], 16 * gg + r);
              if (gg < g) above += o;
            }
            f32x4 d;
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = row_sum<16>(4 * g + e <= r ? above + sum[e] : 0.f);
            if (r == 0) {
              *reinterpret_cast<f32x4 *>(&s.zdiag[16 * j + 4 * g]) = d;
              *reinterpret_cast<f32x4 *>(&s.cols[own][16 * j + 4 * g]) = f32x4{0.f, 0.f, 0.f, 0.f};
            }
          }
        }
        zrow += __shfl_xor(zrow, 16);
        zrow += __shfl_xor(zrow, 32);
        if (g == 0) s.zrow[16 * own + r] = zrow;
      }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        if (2 * kb <= own) {
          u32x4 pt[3], vt[3];
          split_operand<3>(PT[2 * kb], PT[2 * kb + 1], pt, minus);
          split_operand<3>(VT[2 * kb], VT[2 * kb + 1], vt, minus);
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            const u32x4 kt = columns(0, i, kb);
#pragma unroll
            for (int pl = 2; pl >= 0; --pl) {
              DQ[i] = mma(pt[pl], kt, DQ[i]);
              KR[i] = mma(vt[pl], kt, KR[i]);
            }
          }
        }
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      GQ[i] = GQ[i] + DQ[i] * sign;
      GK[i] = GK[i] + KR[i] * sign;
    }
    __builtin_amdgcn_sched_barrier(0);
    if (hh + 1 < count && ptiles == 1) load_rows(h + 1, 0);
    r = hold(r), g = hold(g);
    // Rows i and the own tile's j as columns.
    {
      f32x4 PN[4], VN[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) PN[i] = VN[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int pt = 0; pt < ptiles; ++pt) {
        if (ptiles > 1) {
          __syncthreads();
          load_rows(h, pt * kCols);
          stage_rows(pt * kCols);
          __syncthreads();
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          u32x4 eo[3];
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) eo[pl] = lds_get<u32x4>(l_dy + (1 + pl) * kPart + own * kTileRows + 64 * kb);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j >= own) {
              const u32x4 di = lds_get<u32x4>(l_dy + j * kTileRows + 64 * kb);
              u32x4 wi[3];
#pragma unroll
              for (int pl = 0; pl < 3; ++pl) wi[pl] = lds_get<u32x4>(l_dy + (4 + pl) * kPart + j * kTileRows + 64 * kb);
#pragma unroll
              for (int k = 0; k < 6; ++k) {
                VN[j] = mma(wi[kA[k]], eo[kB[k]], VN[j]);
                if (k % 2 == 1) PN[j] = mma(di, eo[2 - k / 2], PN[j]);
              }
            }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j >= own) {
          const f32x4 rqi = *reinterpret_cast<const f32x4 *>(&s.rq[16 * j + 4 * g]);
          const f32x4 rki = *reinterpret_cast<const f32x4 *>(&s.rk[16 * j + 4 * g]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = decay_of(s.c[16 * j + 4 * g + e] - c_own);
            PN[j][e] = j > own || 4 * g + e >= r ? PN[j][e] * (f * (a.scale * rqi[e])) : 0.f;
            VN[j][e] = j > own || 4 * g + e > r ? -(VN[j][e] * (f * rki[e])) : 0.f;
          }
        }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        if (2 * kb + 1 >= own) {
          u32x4 pn[3], vn[3];
          split_operand<3>(PN[2 * kb], PN[2 * kb + 1], pn, minus);
          split_operand<3>(VN[2 * kb], VN[2 * kb + 1], vn, minus);
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            const u32x4 kt = columns(0, i, kb), qt = columns(1, i, kb);
#pragma unroll
            for (int pl = 2; pl >= 0; --pl) {
              T[i] = mma(vn[pl], kt, T[i]);
              T[i] = mma(pn[pl], qt, T[i]);
            }
          }
        }
    }
    const f32x4 beo = *reinterpret_cast<const f32x4 *>(&s.beta[16 * own + 4 * g]) * sign;
    // sums over n of the own rows
    f32x4 kt_ = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NH; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) kt_[e] = fmaf(k_at(i, e), T[i][e], kt_[e]);
      GK[i] = GK[i] + T[i] * beo;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      read[e] = row_sum<16>(read[e]);
      kt_[e] = row_sum<16>(kt_[e]) * rko[e];
      first[e] = row_sum<16>(first[e]) * rko[e];
    }
    if (r == 0) {
      *reinterpret_cast<f32x4 *>(&s.rows[half][0][16 * own + 4 * g]) = read;
      *reinterpret_cast<f32x4 *>(&s.rows[half][1][16 * own + 4 * g]) = kt_;
      *reinterpret_cast<f32x4 *>(&s.rows[half][2][16 * own + 4 * g]) = first;
    }
    dot = row_sum<64>(dot);
    if (lane == 0) s.dot[wave] = dot;
    __builtin_amdgcn_sched_barrier(0);
    if (hh + 1 < count) {
      load_gates(h + 1);
      if (ptiles > 1) load_rows(h + 1, 0);
      load_state(keep.S, h + 1, 0);
    }
    __syncthreads();
    if (wave == 0) {
      const int t = lane;
      auto both = [&](int w) { return s.rows[0][w][t] + s.rows[1][w][t]; };
      const float dbeta = both(1) * sign;
      float d8 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) d8 += s.dot[i];
      double below = 0.0, tiles[4];  // column t in all tiles below its own; a tile's columns in tile w
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        below += s.cols[w][t];
        tiles[w] = row_prefix(s.cols[w][t]);
      }
      // tiles below t's and left of it (the lanes are read by all, outside the choice)
      const double c20 = lane_value(tiles[2], 15), c30 = lane_value(tiles[3], 15), c31 = lane_value(tiles[3], 31);
      const double corner = t / 16 == 1 ? c20 + c30 : t / 16 == 2 ? c30 + c31 : 0.0;
      const double pairs = corner + dpp_shift<0x111>(row_prefix(below)) + row_suffix(s.zrow[t]) + s.zdiag[t];
      const float dlog = static_cast<float>(sign * (static_cast<double>(decay_of(s.c[kC - 1])) * d8 + wave_from(both(0)) +
                                            wave_before(static_cast<double>(s.beta[t]) * both(2)) + pairs));
      const float A = s.head[0], bias = s.head[1];
      float sa = 0.f, sb = 0.f;
      if (t < left) {
        const int64_t at = (b * a.L + t0 + t) * a.H + h;
        const float raw = s.dt[t];
        const float d = step_size(raw, bias, a.dt_softplus);
        const float slope = a.dt_softplus ? 1.f / (1.f + fast_exp2(-(raw + bias) * kLog2e)) : 1.f;
        sa = dlog * d;
        sb = dlog * A * slope;
        static_cast<bf16_t *>(ba.dbeta)[at] = from_f32<bf16_t>(dbeta);
        static_cast<bf16_t *>(ba.ddt)[at] = from_f32<bf16_t>(sb);
      }
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        sa += __shfl_xor(sa, m);
        sb += __shfl_xor(sb, m);
      }
      if (lane == 0) {
        red[2 * (b * nc + c) * a.H + h] = sa;
        red[(2 * (b * nc + c) + 1) * a.H + h] = sb;
      }
    }
  }

  if constexpr (SPLIT) {  // the heads' parts are summed, and taken through the norms, behind this
    const int64_t all = a.B * a.L * a.G * N;
#pragma unroll
    for (int i = 0; i < NH; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = 16 * own + 4 * g + e, n = 16 * (NH * half + i) + r;
        if (tok < left && n < N) {
          float *to = qk_part + part * all + ((b * a.L + t0 + tok) * a.G + grp) * N + n;
          to[0] = GQ[i][e];
          to[split * all] = GK[i][e];
        }
      }
    return;
  }
  // through the norms: with u = r x, dx = r (g - u (g . u))
  const f32x4 rko = *reinterpret_cast<const f32x4 *>(&s.rk[16 * own + 4 * g]);
  const f32x4 rqo = *reinterpret_cast<const f32x4 *>(&s.rq[16 * own + 4 * g]);
  if (a.qk_norm) {
    f32x4 gq = {0.f, 0.f, 0.f, 0.f}, gk = gq;
#pragma unroll
    for (int i = 0; i < NH; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        gq[e] = fmaf(q_at(i, e), GQ[i][e], gq[e]);
        gk[e] = fmaf(k_at(i, e), GK[i][e], gk[e]);
      }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gq[e] = row_sum<16>(gq[e]) * rqo[e];
      gk[e] = row_sum<16>(gk[e]) * rko[e];
    }
    __syncthreads();  // wave 0 has read the rows
    if (r == 0) {
      *reinterpret_cast<f32x4 *>(&s.rows[half][0][16 * own + 4 * g]) = gq;
      *reinterpret_cast<f32x4 *>(&s.rows[half][1][16 * own + 4 * g]) = gk;
    }
    __syncthreads();
    gq = gq + *reinterpret_cast<const f32x4 *>(&s.rows[1 - half][0][16 * own + 4 * g]);
    gk = gk + *reinterpret_cast<const f32x4 *>(&s.rows[1 - half][1][16 * own + 4 * g]);
#pragma unroll
    for (int i = 0; i < NH; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        GQ[i][e] = rqo[e] * fmaf(-gq[e] * rqo[e], q_at(i, e), GQ[i][e]);
        GK[i][e] = rko[e] * fmaf(-gk[e] * rko[e], k_at(i, e), GK[i][e]);
      }
  }
#pragma unroll
  for (int i = 0; i < NH; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int tok = 16 * own + 4 * g + e, n = 16 * (NH * half + i) + r;
      if (tok < left && n < N) {
        const int64_t at = ((b * a.L + t0 + tok) * a.G + grp) * N + n;
        static_cast<bf16_t *>(ba.dq)[at] = from_f32<bf16_t>(GQ[i][e]);
        static_cast<bf16_t *>(ba.dk)[at] = from_f32<bf16_t>(GK[i][e]);
      }
    }
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
int64_t pad4(int64_t n) { return (n + 3) / 4 * 4; }

}  // namespace

bool gdr_bwd_chunk_applies(const GdrBwdArgs &a) {
  return gdr_chunk_applies(a.f) && aligned16(a.dy) && aligned16(a.dh_final) && aligned16(a.dh0) &&
         a.f.P <= (int64_t(1) << 20) &&  // what is kept of a chunk within 32-bit offsets
         (a.f.L + kC - 1) / kC < (int64_t(1) << 32) / kThreads;  // a workgroup a chunk, in one dimension
}

// Into how many workgroups the heads of a group are split: as many as make the
// turns of 256 CUs, times the heads of a turn, fewest.  2 sequences of 64 tokens,
// 80 heads of 64 x 128 in 8 groups: 170 us with a group's 10 heads one after the
// other, 69 split.
namespace {
int64_t head_split(int64_t B, int64_t nc, int64_t G, int64_t heads) {
  constexpr int64_t kCus = 256;
  int64_t best = 1, least = (B * nc * G + kCus - 1) / kCus * heads;
  for (int64_t split = 2; split <= heads && split <= 64 && B * split <= 65535; ++split) {
    const int64_t turns = (B * nc * G * split + kCus - 1) / kCus * ((heads + split - 1) / split);
    if (turns < least) {
      least = turns;
      best = split;
    }
  }
  return best;
}
int64_t split_floats(int64_t split, int64_t B, int64_t L, int64_t G, int64_t N) {
  return split > 1 ? pad4(2 * split * B * L * G * N) : 0;
}
}  // namespace

int64_t gdr_bwd_chunk_ws_floats(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N) {
  const int64_t nc = (L + kC - 1) / kC, items = B * H * nc;
  return items * (2 * pad4(P * N) + 2 * kC * P + 20 * 256 + kGdrVec) + pad4(2 * B * nc * H) +
         split_floats(head_split(B, nc, G, H / G), B, L, G, N);
}

hipError_t launch_gdr_bwd_chunk(const GdrBwdArgs &a, hipStream_t s) {
  const GdrArgs &f = a.f;
  const int64_t nc = (f.L + kC - 1) / kC, items = f.B * f.H * nc;
  GdrSaved k;
  k.S = a.ws;
  k.dS = k.S + items * pad4(f.P * f.N);
  k.E = k.dS + items * pad4(f.P * f.N);
  k.W = k.E + items * kC * f.P;
  k.XM = k.W + items * kC * f.P;
  k.vec = k.XM + items * 20 * 256;
  float *red = k.vec + items * kGdrVec;
  GdrArgs fw = f;
  fw.y = nullptr;
  fw.h_final = nullptr;
  hipError_t e = launch_gdr_chunk_save(fw, k, s);
  if (e != hipSuccess) return e;
  const int cols = gdr_chain_columns(f.B, f.H, f.P);
  const int64_t ptiles = (f.P + cols - 1) / cols, per = f.H / f.G * ptiles;
  const unsigned grid = static_cast<unsigned>((f.B * f.G + 7) / 8 * 8 * per);
  const int64_t split = head_split(f.B, nc, f.G, f.H / f.G);
  float *qk_part = red + pad4(2 * f.B * nc * f.H);
  const dim3 gg(static_cast<unsigned>(nc), static_cast<unsigned>(f.G), static_cast<unsigned>(f.B * split));
  if (f.N <= 64) gdr_bwd_chain_kernel<4><<<grid, kThreads, 0, s>>>(a, k, ptiles, cols);
  else gdr_bwd_chain_kernel<8><<<grid, kThreads, 0, s>>>(a, k, ptiles, cols);
  auto grads = [&](auto tiles, auto four) {
    constexpr int NT = decltype(tiles)::value;
    constexpr bool FOUR = decltype(four)::value;
    if (split > 1) gdr_bwd_grads_kernel<NT, FOUR, true><<<gg, kThreads, 0, s>>>(a, k, split, qk_part, red);
    else gdr_bwd_grads_kernel<NT, FOUR, false><<<gg, kThreads, 0, s>>>(a, k, split, qk_part, red);
  };
  auto of = [&](auto tiles) {
    if (f.P % 4 == 0) grads(tiles, std::true_type());
    else grads(tiles, std::false_type());
  };
  if (f.N <= 64) of(std::integral_constant<int, 4>());
  else of(std::integral_constant<int, 8>());
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (split > 1) {
    e = launch_gdr_reduce_qk(a, split, f.G, qk_part, qk_part + split * f.B * f.L * f.G * f.N, s);
    if (e != hipSuccess) return e;
  }
  return launch_gdr_reduce_params(a, f.B * nc, red, s);
}

}  // namespace ssm
