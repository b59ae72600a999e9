// Gradients of the gated delta rule, token by token on the vector ALU, and the
// sums that finish the gradients of both backward paths.
//
// With S the state before a token's decay, a its decay, B = a S, and q, k
// normalised where asked (e, u = beta e as in the forward):
//   after = B + u k^T            dq   = scale sum_p dy[p] after[p]
//   dS   += scale dy q^T         du   = dS k       dbeta = sum_p du e
//   de    = beta du = dv         dk   = sum_p u dS[p] - de B[p]
//   dS   -= de k^T               dlog = sum dS B   (d of the log decay)
//   dS    = a dS
// The states before the tokens are recomputed: the forward's token kernel
// saves the state entering every kGdrSeg tokens, and the reverse pass walks a
// segment forward from it, keeping the segment's states in registers.
//
// A workgroup holds 256 / LPC rows of one head (the forward's layout).  dq and
// dk sum over the head's rows: over the lanes of a wave by shuffles, over the
// waves in LDS, over the tiles of rows and the heads of a group by the sums
// below, always in the same order.
#include "device_common.h"
#include "gdr.h"
#include "gdr_common.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kSeg = kGdrSeg;

__host__ __device__ constexpr int lanes_per_row(int64_t N) { return N <= 16 ? 4 : N <= 32 ? 8 : 16; }
int64_t row_tiles(int64_t P, int64_t N) {
  const int64_t rows = kThreads / lanes_per_row(N);
  return (P + rows - 1) / rows;
}

template <typename T, int LPC, int NV, bool VEC>
__global__ __launch_bounds__(kThreads) void gdr_bwd_seq_kernel(GdrBwdArgs ba, const float *ckpt, float *dq_part,
                                                               float *dk_part, float *sc_part) {
  const GdrArgs &a = ba.f;
  constexpr int NP = 4 * LPC * NV;
  constexpr int kRows = kThreads / LPC;
  __shared__ __attribute__((aligned(16))) float s_k[kSeg][NP], s_q[kSeg][NP];
  __shared__ float s_r[kSeg][2];
  __shared__ float s_ab[kSeg][2];  // decay, beta
  __shared__ float s_dq[kWaves][kSeg][NP], s_dk[kWaves][kSeg][NP];
  __shared__ float s_sc[kWaves][kSeg][2];
  const int64_t L = a.L, H = a.H, P = a.P, G = a.G, N = a.N, B = a.B;
  const int tid = threadIdx.x, lq = tid % LPC, lr = tid / LPC, lane = tid % 64, wave = tid / 64;
  const int64_t tile = blockIdx.x, h = blockIdx.y, b = blockIdx.z, g = h / (H / G);
  const int64_t p_raw = tile * kRows + lr;
  const bool active = p_raw < P;
  const int64_t p = active ? p_raw : P - 1;
  const float A2 = a.A[h] * kLog2e, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  const int64_t nseg = (L + kSeg - 1) / kSeg;
  const T *kp = static_cast<const T *>(a.k), *qp = static_cast<const T *>(a.q);

  float dS[4 * NV];
  if (ba.dh_final != nullptr && active)
    load_row<VEC, LPC, NV>(ba.dh_final + ((b * H + h) * P + p) * N, lq, N, dS);
  else
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) dS[i] = 0.f;

  for (int64_t s = nseg - 1; s >= 0; --s) {
    const int64_t t0 = s * kSeg;
    const int nt = static_cast<int>(L - t0 < kSeg ? L - t0 : kSeg);
    for (int e = tid; e < kSeg * NP; e += kThreads) {
      const int j = e / NP, n = e % NP;
      const bool ok = j < nt && n < N;
      const int64_t at = ok ? ((b * L + t0 + j) * G + g) * N + n : 0;
      s_k[j][n] = ok ? to_f32(kp[at]) : 0.f;
      s_q[j][n] = ok ? to_f32(qp[at]) : 0.f;
    }
    if (tid < nt) {
      const int64_t at = (b * L + t0 + tid) * H + h;
      const float d = step_size(to_f32(static_cast<const T *>(a.dt)[at]), bias, a.dt_softplus);
      s_ab[tid][0] = fast_exp2(d * A2);
      s_ab[tid][1] = to_f32(static_cast<const T *>(a.beta)[at]);
    }
    __syncthreads();
    if (a.qk_norm) {  // 16 lanes per (token, q or k) row
      const int j = tid / 32, w = (tid / 16) % 2, i0 = tid % 16;
      static_assert(kSeg * 32 == kThreads, "32 lanes per token");
      float *x = w ? s_q[j] : s_k[j];
      float ss = 0.f;
      for (int n = i0; n < NP; n += 16) ss = fmaf(x[n], x[n], ss);
      ss = row_sum<16>(ss);
      if (i0 == 0) s_r[j][w] = 1.f / sqrtf(ss + kQkNormEps);
      __syncthreads();
      for (int e = tid; e < kSeg * NP; e += kThreads) {
        const int jj = e / NP, n = e % NP;
        s_k[jj][n] *= s_r[jj][0];
        s_q[jj][n] *= s_r[jj][1];
      }
      __syncthreads();
    }

    // forward through the segment: the state before each token, and e
    float Sv[kSeg][4 * NV], E[kSeg], v[kSeg], dy[kSeg];
#pragma unroll
    for (int j = 0; j < kSeg; ++j) {
      const int64_t t = t0 + (j < nt ? j : nt - 1);
      const int64_t at = ((b * L + t) * H + h) * P + p;
      v[j] = to_f32(static_cast<const T *>(a.v)[at]);
      dy[j] = active ? a.scale * to_f32(static_cast<const T *>(ba.dy)[at]) : 0.f;
    }
    load_row<VEC, LPC, NV>(ckpt + (((b * H + h) * nseg + s) * P + p) * N, lq, N, Sv[0]);
#pragma unroll
    for (int j = 0; j < kSeg; ++j) {
      E[j] = 0.f;
      if (j < nt) {
        float kv[4 * NV];
        lds_row<LPC, NV>(s_k[j], lq, kv);
        const float al = s_ab[j][0];
        E[j] = active ? fmaf(-al, row_dot<LPC, NV>(Sv[j], kv), v[j]) : 0.f;
        if (j + 1 < kSeg) {
          const float u = s_ab[j][1] * E[j];
#pragma unroll
          for (int i = 0; i < 4 * NV; ++i) Sv[j + 1][i] = fmaf(al, Sv[j][i], u * kv[i]);
        }
      }
    }
    // back through it
#pragma unroll
    for (int j = kSeg - 1; j >= 0; --j) {
      if (j < nt) {
        float kv[4 * NV], qv[4 * NV];
        lds_row<LPC, NV>(s_k[j], lq, kv);
        lds_row<LPC, NV>(s_q[j], lq, qv);
        const float al = s_ab[j][0], be = s_ab[j][1], u = be * E[j];
        float gq[4 * NV], gk[4 * NV];
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) {
          const float before = al * Sv[j][i];
          gq[i] = dy[j] * fmaf(u, kv[i], before);
          dS[i] = fmaf(dy[j], qv[i], dS[i]);
        }
        const float du = row_dot<LPC, NV>(dS, kv);
        const float de = be * du;
        float dl = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) {
          const float before = al * Sv[j][i];
          gk[i] = fmaf(dS[i], u, -(before * de));
          dS[i] = fmaf(-de, kv[i], dS[i]);
          dl = fmaf(dS[i], before, dl);
          dS[i] *= al;
        }
        if (active && lq == 0)
          static_cast<T *>(ba.dv)[((b * L + t0 + j) * H + h) * P + p] = from_f32<T>(de);
        // rows past P add nothing: their dy, e and dS are 0, but their saved
        // state is a copy of row P - 1
        float db = active && lq == 0 ? du * E[j] : 0.f;
        if (!active) dl = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) {
          if (!active) gq[i] = gk[i] = 0.f;
#pragma unroll
          for (int m = LPC; m < 64; m <<= 1) {
            gq[i] += __shfl_xor(gq[i], m);
            gk[i] += __shfl_xor(gk[i], m);
          }
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
          db += __shfl_xor(db, m);
          dl += __shfl_xor(dl, m);
        }
        if (lane < LPC) {
#pragma unroll
          for (int i = 0; i < 4 * NV; ++i) {
            const int n = 4 * (lq + LPC * (i / 4)) + i % 4;
            s_dq[wave][j][n] = gq[i];
            s_dk[wave][j][n] = gk[i];
          }
        }
        if (lane == 0) {
          s_sc[wave][j][0] = db;
          s_sc[wave][j][1] = dl;
        }
      }
    }
    __syncthreads();
    for (int e = tid; e < nt * NP; e += kThreads) {
      const int j = e / NP, n = e % NP;
      if (n < N) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          x += s_dq[w][j][n];
          y += s_dk[w][j][n];
        }
        const int64_t at = (((tile * B + b) * L + t0 + j) * H + h) * N + n;
        dq_part[at] = x;
        dk_part[at] = y;
      }
    }
    if (tid < 2 * nt) {
      const int j = tid / 2, w2 = tid % 2;
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) x += s_sc[w][j][w2];
      sc_part[(((w2 * static_cast<int64_t>(gridDim.x) + tile) * B + b) * L + t0 + j) * H + h] = x;
    }
    __syncthreads();  // the next segment stages into the same LDS
  }
  if (ba.dh0 != nullptr && active)
    store_row<VEC, LPC, NV>(ba.dh0 + ((b * H + h) * P + p) * N, lq, N, dS);
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T, int LPC, int NV>
hipError_t launch_shape(const GdrBwdArgs &a, const float *ckpt, float *dqp, float *dkp, float *scp, int64_t tiles,
                        hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.f.H), static_cast<unsigned>(a.f.B));
  if (a.f.N % 4 == 0 && aligned16(a.dh_final) && aligned16(a.dh0) && aligned16(ckpt))
    gdr_bwd_seq_kernel<T, LPC, NV, true><<<grid, kThreads, 0, s>>>(a, ckpt, dqp, dkp, scp);
  else
    gdr_bwd_seq_kernel<T, LPC, NV, false><<<grid, kThreads, 0, s>>>(a, ckpt, dqp, dkp, scp);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const GdrBwdArgs &a, const float *ckpt, float *dqp, float *dkp, float *scp, int64_t tiles,
                    hipStream_t s) {
  const int64_t N = a.f.N;
  if (N <= 16) return launch_shape<T, 4, 1>(a, ckpt, dqp, dkp, scp, tiles, s);
  if (N <= 32) return launch_shape<T, 8, 1>(a, ckpt, dqp, dkp, scp, tiles, s);
  if (N <= 64) return launch_shape<T, 16, 1>(a, ckpt, dqp, dkp, scp, tiles, s);
  if (N <= 128) return launch_shape<T, 16, 2>(a, ckpt, dqp, dkp, scp, tiles, s);
  if (N <= 192) return launch_shape<T, 16, 3>(a, ckpt, dqp, dkp, scp, tiles, s);
  return launch_shape<T, 16, 4>(a, ckpt, dqp, dkp, scp, tiles, s);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// dq (blockIdx.y 0) and dk (1): one wave per (token, group) sums the partial
// gradients of the group's heads and tiles, in order, and takes them through
// the norm: with u = r x, dx = r (g - u (g . u)).
template <typename T>
__global__ __launch_bounds__(kThreads) void gdr_reduce_qk_kernel(GdrBwdArgs ba, int64_t tiles, const float *dq_part,
                                                                 const float *dk_part) {
  const GdrArgs &a = ba.f;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  if (item >= a.B * a.L * a.G) return;
  const bool is_k = blockIdx.y != 0;
  const float *part = is_k ? dk_part : dq_part;
  const T *x = static_cast<const T *>(is_k ? a.k : a.q) + item * a.N;
  T *out = static_cast<T *>(is_k ? ba.dk : ba.dq) + item * a.N;
  const int64_t tok = item / a.G, g = item % a.G, per = a.H / a.G;
  constexpr int kPer = 4;  // N <= 256
  float sum[kPer], xv[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t n = lane + 64 * i;
    sum[i] = 0.f;
    xv[i] = n < a.N ? to_f32(x[n]) : 0.f;
    if (n < a.N)
      for (int64_t t = 0; t < tiles; ++t)
        for (int64_t hh = 0; hh < per; ++hh)
          sum[i] += part[((t * a.B * a.L + tok) * a.H + g * per + hh) * a.N + n];
  }
  if (a.qk_norm) {
    float ss = 0.f, gx = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      ss = fmaf(xv[i], xv[i], ss);
      gx = fmaf(sum[i], xv[i], gx);
    }
    const float r = 1.f / sqrtf(wave_sum(ss) + kQkNormEps);
    const float gu = wave_sum(gx) * r;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum[i] = r * fmaf(-gu * r, xv[i], sum[i]);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t n = lane + 64 * i;
    if (n < a.N) out[n] = from_f32<T>(sum[i]);
  }
}

// dbeta and ddt, one thread per (token, head), and the sums of a block of
// tokens for dA and the bias (64 heads by 4 tokens per round).
constexpr int kTokBlock = 128;
template <typename T>
__global__ __launch_bounds__(kThreads) void gdr_reduce_gates_kernel(GdrBwdArgs ba, int64_t tiles,
                                                                    const float *sc_part, float *red) {
  const GdrArgs &a = ba.f;
  __shared__ float s_a[kWaves][64], s_b[kWaves][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t h = static_cast<int64_t>(blockIdx.y) * 64 + lane, H = a.H, BL = a.B * a.L;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * kTokBlock;
  float sa = 0.f, sb = 0.f;
  if (h < H) {
    const float Ah = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    for (int64_t tok = tok0 + wave; tok < tok0 + kTokBlock && tok < BL; tok += kWaves) {
      float db = 0.f, dl = 0.f;
      for (int64_t t = 0; t < tiles; ++t) {
        db += sc_part[(t * BL + tok) * H + h];
        dl += sc_part[((tiles + t) * BL + tok) * H + h];
      }
      const float raw = to_f32(static_cast<const T *>(a.dt)[tok * H + h]);
      const float d = step_size(raw, bias, a.dt_softplus);
      const float slope = a.dt_softplus ? 1.f / (1.f + fast_exp2(-(raw + bias) * kLog2e)) : 1.f;
      const float dd = dl * Ah * slope;
      static_cast<T *>(ba.dbeta)[tok * H + h] = from_f32<T>(db);
      static_cast<T *>(ba.ddt)[tok * H + h] = from_f32<T>(dd);
      sa = fmaf(dl, d, sa);
      sb += dd;
    }
  }
  s_a[wave][lane] = sa;
  s_b[wave][lane] = sb;
  __syncthreads();
  if (wave == 0 && h < H) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      x += s_a[w][lane];
      y += s_b[w][lane];
    }
    red[(2 * static_cast<int64_t>(blockIdx.x)) * H + h] = x;
    red[(2 * static_cast<int64_t>(blockIdx.x) + 1) * H + h] = y;
  }
}
// one wave per head: the blocks' sums, in a fixed order
__global__ __launch_bounds__(64) void gdr_reduce_params_kernel(GdrBwdArgs ba, int64_t nblk, const float *red) {
  const int64_t h = blockIdx.x, H = ba.f.H;
  float x = 0.f, y = 0.f;
  for (int64_t i = threadIdx.x; i < nblk; i += 64) {
    x += red[2 * i * H + h];
    y += red[(2 * i + 1) * H + h];
  }
  x = wave_sum(x);
  y = wave_sum(y);
  if (threadIdx.x == 0) {
    ba.dA[h] = x;
    if (ba.dbias) ba.dbias[h] = y;
  }
}

int64_t pad4(int64_t n) { return (n + 3) / 4 * 4; }

}  // namespace

int64_t gdr_reduce_ws_floats(int64_t B, int64_t L, int64_t H) {
  return pad4((B * L + kTokBlock - 1) / kTokBlock * 2 * H);
}

hipError_t launch_gdr_reduce(const GdrBwdArgs &a, int64_t tiles, const float *dq_part, const float *dk_part,
                             const float *sc_part, float *red, hipStream_t s) {
  const GdrArgs &f = a.f;
  const int64_t BL = f.B * f.L;
  const int64_t nblk = (BL + kTokBlock - 1) / kTokBlock;
  const bool bf = f.dt_type == DType::BF16;
  if (BL > 0) {
    const dim3 gq(static_cast<unsigned>((BL * f.G + kWaves - 1) / kWaves), 2);
    const dim3 gg(static_cast<unsigned>(nblk), static_cast<unsigned>((f.H + 63) / 64));
    if (bf) {
      gdr_reduce_qk_kernel<bf16_t><<<gq, kThreads, 0, s>>>(a, tiles, dq_part, dk_part);
      gdr_reduce_gates_kernel<bf16_t><<<gg, kThreads, 0, s>>>(a, tiles, sc_part, red);
    } else {
      gdr_reduce_qk_kernel<float><<<gq, kThreads, 0, s>>>(a, tiles, dq_part, dk_part);
      gdr_reduce_gates_kernel<float><<<gg, kThreads, 0, s>>>(a, tiles, sc_part, red);
    }
  }
  return launch_gdr_reduce_params(a, nblk, red, s);
}
hipError_t launch_gdr_reduce_params(const GdrBwdArgs &a, int64_t nblk, const float *red, hipStream_t s) {
  gdr_reduce_params_kernel<<<static_cast<unsigned>(a.f.H), 64, 0, s>>>(a, nblk, red);
  return hipGetLastError();
}

int64_t gdr_bwd_seq_ws_floats(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N) {
  const int64_t nseg = (L + kSeg - 1) / kSeg, tiles = row_tiles(P, N);
  return pad4(B * H * nseg * P * N) + 2 * pad4(tiles * B * L * H * N) + pad4(2 * tiles * B * L * H) +
         gdr_reduce_ws_floats(B, L, H);
}

hipError_t launch_gdr_bwd_seq(const GdrBwdArgs &a, hipStream_t s) {
  const GdrArgs &f = a.f;
  const int64_t nseg = (f.L + kSeg - 1) / kSeg, tiles = row_tiles(f.P, f.N);
  float *ckpt = a.ws, *dqp = ckpt + pad4(f.B * f.H * nseg * f.P * f.N);
  float *dkp = dqp + pad4(tiles * f.B * f.L * f.H * f.N), *scp = dkp + pad4(tiles * f.B * f.L * f.H * f.N);
  float *red = scp + pad4(2 * tiles * f.B * f.L * f.H);
  GdrArgs fw = f;
  fw.y = nullptr;
  fw.h_final = nullptr;
  fw.h_ckpt = ckpt;
  hipError_t e = f.L > 0 ? launch_gdr_seq(fw, s) : hipSuccess;
  if (e != hipSuccess) return e;
  e = f.dt_type == DType::BF16 ? launch_t<bf16_t>(a, ckpt, dqp, dkp, scp, tiles, s)
                               : launch_t<float>(a, ckpt, dqp, dkp, scp, tiles, s);
  if (e != hipSuccess) return e;
  return launch_gdr_reduce(a, tiles, dqp, dkp, scp, red, s);
}

}  // namespace ssm
