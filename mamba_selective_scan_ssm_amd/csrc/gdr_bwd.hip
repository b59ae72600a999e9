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
// A workgroup holds 16 rows of one head, 16 lanes each.  dq and dk sum over the
// head's rows: over a wave's four by exchanges of lanes, two values at a time
// that end side by side (3 swaps for 4 values), over the waves in LDS, over the
// tiles of rows and the heads of a group by the sums below, always in the same
// order.
//
// Bound by the chain of a token, forwards and back (six sums between lanes): 2 x
// 515 tokens of fp32, 6 heads of 40 x 48: 0.216 ms, 0.42 us a token, with the next
// segment's loads under it; before it the states, 0.059 ms, behind it the sums,
// 0.017 ms.
#include "device_common.h"
#include "gdr.h"
#include "gdr_common.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kSeg = kGdrSeg;

constexpr int kLanes = 16, kRows = kThreads / kLanes;
int64_t row_tiles(int64_t P) { return (P + kRows - 1) / kRows; }

template <typename T, int NV, bool VEC>
__global__ __launch_bounds__(kThreads) void gdr_bwd_seq_kernel(GdrBwdArgs ba, const float *ckpt, float *dq_part,
                                                               float *dk_part, float *sc_part) {
  const GdrArgs &a = ba.f;
  constexpr int LPC = kLanes, NP = 4 * LPC * NV;
  constexpr uint32_t kSize = sizeof(T);
  static_assert(kSeg == 8 && kThreads == 16 * 2 * kSeg, "16 lanes for each of a segment's rows of k and q");
  __shared__ __attribute__((aligned(16))) float s_x[2][kSeg][NP];          // k, q, normalised
  __shared__ __attribute__((aligned(16))) float s_d[2][kWaves][kSeg][NP];  // dq, dk
  __shared__ float s_sc[kWaves][2 * kSeg];                                 // dbeta, then dlog
  const int64_t L = a.L, H = a.H, P = a.P, G = a.G, N = a.N, B = a.B;
  const int tid = threadIdx.x, lq = tid % LPC, mine = tid % 8, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int64_t tile = blockIdx.x, h = blockIdx.y, b = blockIdx.z, g = h / (H / G);
  const int64_t p_raw = tile * kRows + tid / LPC;
  const bool active = p_raw < P;
  const int64_t p = active ? p_raw : P - 1;
  const float A2 = a.A[h] * kLog2e, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  const int64_t nseg = (L + kSeg - 1) / kSeg;

  float dS[4 * NV];
  if (ba.dh_final != nullptr && active)
    load_row<VEC, LPC, NV>(ba.dh_final + ((b * H + h) * P + p) * N, lq, N, dS);
  else
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) dS[i] = 0.f;

  // a segment's rows of `width` elements, `pitch` apart
  auto rows = [&](const void *base, int64_t s, int64_t first, int64_t pitch, int64_t width) {
    const int64_t left = s < 0 ? 0 : L - s * kSeg < kSeg ? L - s * kSeg : kSeg;
    return buffer_of(static_cast<const T *>(base) + (s < 0 ? 0 : (b * L + s * kSeg) * pitch + first),
                     left > 0 ? static_cast<uint32_t>((left - 1) * pitch + width) * kSize : 0);
  };
  constexpr int kFours = NP / 64;
  const int tok = 4 * (wave % 2) + lane / 16;  // staged by this lane: of k by waves 0, 1, of q by 2, 3
  const uint32_t row_at = static_cast<uint32_t>(tok * G * N) * kSize;
  const uint32_t gate_at = static_cast<uint32_t>(mine * H) * kSize, v_at = static_cast<uint32_t>(mine * H * P + p) * kSize;
  Four<VEC, T> x[kFours];
  T dn, bn, vn, yn;
  float S0[4 * NV];
  auto load = [&](int64_t s) {
    const __amdgpu_buffer_rsrc_t r = rows(wave < 2 ? a.k : a.q, s, g * N, G * N, N);
#pragma unroll
    for (int j = 0; j < kFours; ++j) {
      const int n = 4 * (tid % 16 + 16 * j);
      x[j].load(r, n < N ? row_at + n * kSize : kNowhere, n, N);
    }
    dn = load_one<T>(rows(a.dt, s, h, H, 1), gate_at);
    bn = load_one<T>(rows(a.beta, s, h, H, 1), gate_at);
    vn = load_one<T>(rows(a.v, s, h * P, H * P, P), v_at);
    yn = load_one<T>(rows(ba.dy, s, h * P, H * P, P), v_at);
    load_row<VEC, LPC, NV>(ckpt + (((b * H + h) * nseg + (s < 0 ? 0 : s)) * P + p) * N, lq, N, S0);
  };
  auto stage = [&]() {
    float f[4 * kFours], ss = kQkNormEps / 16;
#pragma unroll
    for (int i = 0; i < 4 * kFours; ++i) {
      f[i] = to_f32(x[i / 4].v[i % 4]);
      ss = fmaf(f[i], f[i], ss);
    }
    if (a.qk_norm) {
      const float r = inverse_root(row_sum<16>(ss));
#pragma unroll
      for (int i = 0; i < 4 * kFours; ++i) f[i] *= r;
    }
#pragma unroll
    for (int j = 0; j < kFours; ++j)
      *reinterpret_cast<float4 *>(&s_x[wave / 2][tok][4 * (tid % 16 + 16 * j)]) =
          make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
  };

  if (nseg > 0) {
    load(nseg - 1);
    stage();
    meet_in_lds();
  }
  for (int64_t s = nseg - 1; s >= 0; --s) {
    const int64_t t0 = s * kSeg;
    const int nt = static_cast<int>(L - t0 < kSeg ? L - t0 : kSeg);
    // Tokens behind the last are read as zeros and leave all as it is; so do rows
    // behind P, whose dy and e are 0, but their saved state is a copy of row P - 1.
    const float decay = mine < nt ? fast_exp2(step_size(to_f32(dn), bias, a.dt_softplus) * A2) : 1.f;
    const float beta = to_f32(bn), v = to_f32(vn), dy = active ? a.scale * to_f32(yn) : 0.f;
    float Sv[kSeg][4 * NV], E[kSeg];
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) Sv[0][i] = S0[i];
    load(s - 1);
    // forward through the segment: the state before each token, and e
    each<kSeg>([&](auto number) {
      constexpr int j = decltype(number)::value;
      float kv[4 * NV];
      lds_row<LPC, NV>(s_x[0][j], lq, kv);
      const float al = row_lane<j>(decay);
      const float e = fmaf(-al, row_dot<LPC, NV>(Sv[j], kv), row_lane<j>(v));
      E[j] = active ? e : 0.f;
      if constexpr (j + 1 < kSeg) {
        const float u = row_lane<j>(beta) * E[j];
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) Sv[j + 1][i] = fmaf(al, Sv[j][i], u * kv[i]);
      }
    });
    // back through it
    float dv = 0.f, db[kSeg], dl[kSeg];
    each<kSeg>([&](auto number) {
      constexpr int j = kSeg - 1 - decltype(number)::value;
      float kv[4 * NV], qv[4 * NV], gq[4 * NV], gk[4 * NV];
      lds_row<LPC, NV>(s_x[0][j], lq, kv);
      lds_row<LPC, NV>(s_x[1][j], lq, qv);
      const float al = row_lane<j>(decay), be = row_lane<j>(beta), dyj = row_lane<j>(dy), u = be * E[j];
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) {
        Sv[j][i] *= al;
        gq[i] = dyj * fmaf(u, kv[i], Sv[j][i]);
        dS[i] = fmaf(dyj, qv[i], dS[i]);
      }
      const float du = row_dot<LPC, NV>(dS, kv);
      const float de = be * du;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) {
        gk[i] = fmaf(dS[i], u, -(Sv[j][i] * de));
        dS[i] = fmaf(-de, kv[i], dS[i]);
        sum = fmaf(dS[i], Sv[j][i], sum);
        dS[i] *= al;
      }
      if (mine == j) dv = de;
      db[j] = active && lq == 0 ? du * E[j] : 0.f;
      dl[j] = active ? sum : 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NV; i += 4) {
        float f[4];  // of q in the lower 32 lanes, of k in the upper
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = join_halves(active ? gq[i + e] : 0.f, active ? gk[i + e] : 0.f);
        // elements 0, 1 in the even rows of lanes, 2, 3 in the odd
        *reinterpret_cast<float2 *>(&s_d[lane / 32][wave][j][4 * (lq + LPC * (i / 4)) + lane / 16 % 2 * 2]) =
            make_float2(join_rows(f[0], f[2]), join_rows(f[1], f[3]));
      }
    });
    store_one(from_f32<T>(dv), rows(ba.dv, s, h * P, H * P, P), active && lq < 8 ? v_at : kNowhere);
    // dbeta of the segment's tokens in the lower lanes, dlog in the upper; tokens 0 .. 3
    // in the even rows, 4 .. 7 in the odd
#pragma unroll
    for (int j = 0; j < kSeg; ++j) db[j] = join_halves(db[j], dl[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x4 = row_sum<16>(join_rows(db[j], db[j + 4]));
      if (lq == 0) s_sc[wave][8 * (lane / 32) + 4 * (lane / 16 % 2) + j] = x4;
    }
    meet_in_lds();
    for (int e = tid; e < nt * NP; e += kThreads) {
      const int j = e / NP, n = e % NP;
      if (n < N) {
        float sq = 0.f, sk = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          sq += s_d[0][w][j][n];
          sk += s_d[1][w][j][n];
        }
        const int64_t at = (((tile * B + b) * L + t0 + j) * H + h) * N + n;
        dq_part[at] = sq;
        dk_part[at] = sk;
      }
    }
    if (tid < 2 * kSeg && tid % kSeg < nt) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) sum += s_sc[w][tid];
      sc_part[((tid / kSeg * static_cast<int64_t>(gridDim.x) + tile) * B + b) * L * H + (t0 + tid % kSeg) * H + h] = sum;
    }
    stage();
    meet_in_lds();  // the next segment's rows are there, and this one's sums taken
  }
  if (ba.dh0 != nullptr && active)
    store_row<VEC, LPC, NV>(ba.dh0 + ((b * H + h) * P + p) * N, lq, N, dS);
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T, int NV>
hipError_t launch_shape(const GdrBwdArgs &a, const float *ckpt, float *dqp, float *dkp, float *scp, int64_t tiles,
                        hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.f.H), static_cast<unsigned>(a.f.B));
  auto fours = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0; };
  if (a.f.N % 4 == 0 && aligned16(a.dh_final) && aligned16(a.dh0) && aligned16(ckpt) && fours(a.f.q) && fours(a.f.k))
    gdr_bwd_seq_kernel<T, NV, true><<<grid, kThreads, 0, s>>>(a, ckpt, dqp, dkp, scp);
  else
    gdr_bwd_seq_kernel<T, NV, false><<<grid, kThreads, 0, s>>>(a, ckpt, dqp, dkp, scp);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const GdrBwdArgs &a, const float *ckpt, float *dqp, float *dkp, float *scp, int64_t tiles,
                    hipStream_t s) {
  const int64_t N = a.f.N;
  if (N <= 64) return launch_shape<T, 1>(a, ckpt, dqp, dkp, scp, tiles, s);
  if (N <= 128) return launch_shape<T, 2>(a, ckpt, dqp, dkp, scp, tiles, s);
  if (N <= 192) return launch_shape<T, 3>(a, ckpt, dqp, dkp, scp, tiles, s);
  return launch_shape<T, 4>(a, ckpt, dqp, dkp, scp, tiles, s);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// dq (blockIdx.y 0) and dk (1): one wave per (token, group) sums the partial
// gradients (tiles, B, L, parts, N) of the group's share of the parts (its heads, or
// itself) and the tiles, in order, and takes them through the norm: with u = r x,
// dx = r (g - u (g . u)).  More items than a grid of kMostBlocks holds take turns.
constexpr int64_t kMostBlocks = int64_t(1) << 22;  // of 256 threads: a dimension holds fewer than 2^32
template <typename T>
__global__ __launch_bounds__(kThreads) void gdr_reduce_qk_kernel(GdrBwdArgs ba, int64_t tiles, int64_t parts,
                                                                 const float *dq_part, const float *dk_part) {
  const GdrArgs &a = ba.f;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const bool is_k = blockIdx.y != 0;
  const float *part = is_k ? dk_part : dq_part;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWaves + wave; item < a.B * a.L * a.G;
       item += static_cast<int64_t>(gridDim.x) * kWaves) {
    const T *x = static_cast<const T *>(is_k ? a.k : a.q) + item * a.N;
    T *out = static_cast<T *>(is_k ? ba.dk : ba.dq) + item * a.N;
    const int64_t tok = item / a.G, g = item % a.G, per = parts / a.G;
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
            sum[i] += part[((t * a.B * a.L + tok) * parts + g * per + hh) * a.N + n];
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
}

// dbeta and ddt, one thread per (token, head), and the sums of a block of
// tokens for dA and the bias (64 heads by 4 tokens per round).
constexpr int kTokBlock = 16;
template <typename T>
__global__ __launch_bounds__(kThreads) void gdr_reduce_gates_kernel(GdrBwdArgs ba, int64_t tiles,
                                                                    const float *sc_part, float *red) {
  const GdrArgs &a = ba.f;
  __shared__ float s_a[kWaves][64], s_b[kWaves][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t h = static_cast<int64_t>(blockIdx.y) * 64 + lane, H = a.H, BL = a.B * a.L;
  for (int64_t blk = blockIdx.x; blk * kTokBlock < BL; blk += gridDim.x) {
    const int64_t tok0 = blk * kTokBlock;
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
      red[2 * blk * H + h] = x;
      red[(2 * blk + 1) * H + h] = y;
    }
    __syncthreads();
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
    const dim3 gg(static_cast<unsigned>(nblk < kMostBlocks ? nblk : kMostBlocks), static_cast<unsigned>((f.H + 63) / 64));
    const hipError_t e = launch_gdr_reduce_qk(a, tiles, f.H, dq_part, dk_part, s);
    if (e != hipSuccess) return e;
    if (bf) {
      gdr_reduce_gates_kernel<bf16_t><<<gg, kThreads, 0, s>>>(a, tiles, sc_part, red);
    } else {
      gdr_reduce_gates_kernel<float><<<gg, kThreads, 0, s>>>(a, tiles, sc_part, red);
    }
  }
  return launch_gdr_reduce_params(a, nblk, red, s);
}
hipError_t launch_gdr_reduce_qk(const GdrBwdArgs &a, int64_t tiles, int64_t parts, const float *dq_part,
                                const float *dk_part, hipStream_t s) {
  const GdrArgs &f = a.f;
  const int64_t blocks = (f.B * f.L * f.G + kWaves - 1) / kWaves;
  const dim3 grid(static_cast<unsigned>(blocks < kMostBlocks ? blocks : kMostBlocks), 2);
  if (f.dt_type == DType::BF16) gdr_reduce_qk_kernel<bf16_t><<<grid, kThreads, 0, s>>>(a, tiles, parts, dq_part, dk_part);
  else gdr_reduce_qk_kernel<float><<<grid, kThreads, 0, s>>>(a, tiles, parts, dq_part, dk_part);
  return hipGetLastError();
}
hipError_t launch_gdr_reduce_params(const GdrBwdArgs &a, int64_t nblk, const float *red, hipStream_t s) {
  gdr_reduce_params_kernel<<<static_cast<unsigned>(a.f.H), 64, 0, s>>>(a, nblk, red);
  return hipGetLastError();
}

int64_t gdr_bwd_seq_ws_floats(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N) {
  const int64_t nseg = (L + kSeg - 1) / kSeg, tiles = row_tiles(P);
  return pad4(B * H * nseg * P * N) + 2 * pad4(tiles * B * L * H * N) + pad4(2 * tiles * B * L * H) +
         gdr_reduce_ws_floats(B, L, H);
}

hipError_t launch_gdr_bwd_seq(const GdrBwdArgs &a, hipStream_t s) {
  const GdrArgs &f = a.f;
  const int64_t nseg = (f.L + kSeg - 1) / kSeg, tiles = row_tiles(f.P);
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
