// The gated delta rule token by token on the vector ALU: prefill for the
// shapes and types the matrix-core kernels are not built for, the decode step
// over a pool of states, and the segment states of the token-path backward.
//
// What is computed, per sequence, head h and row p of the state S (P, N), with
// group g = h / (H / G), the decay a = exp(d A[h]) of the step size d, and q, k
// optionally divided by their 2-norms (rq, rk the factors, 1 otherwise):
//   e   = v[p] - a rk sum_n S[p,n] k[n]
//   S  <- a S + (beta e rk) k
//   y[p] = scale rq sum_n S[p,n] q[n]
// Rows of the state never meet: a row is a recurrence of its own, fed by the
// head's k, q, decay and beta.
//
// Work decomposition: LPC adjacent lanes hold one row, each NV groups of four
// consecutive states (lane i of the row: states 4 (i + LPC j) .. + 3), so the
// row moves in 16-byte pieces that are contiguous over the lanes, and both
// contractions end in log2(LPC) DPP steps.  All state is fp32 in registers from
// the first token to the last.  A workgroup holds 256 / LPC rows of one head.
#include "device_common.h"
#include "gdr.h"
#include "gdr_common.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kTB = 16;  // tokens staged per round
constexpr int64_t kCus = 256;

// State row of sequence b: false where its slot is outside the pool.
__device__ __forceinline__ bool state_row(const GdrArgs &a, int64_t b, int64_t &row) {
  row = b;
  if (a.slots == nullptr) return true;
  const int32_t sl = a.slots[b];
  if (sl < 0 || sl >= a.pool_rows) return false;
  row = sl;
  return true;
}

// Prefill: tokens move in blocks of kTB; all threads load the next block's k,
// q, v, dt and beta into registers while the current block computes from LDS.
template <typename T, int LPC, int NV, bool VEC>
__global__ __launch_bounds__(kThreads) void gdr_seq_kernel(GdrArgs a) {
  constexpr int NP = 4 * LPC * NV;               // states, padded to the lanes
  constexpr int kRows = kThreads / LPC;
  constexpr int kKR = kTB * NP / kThreads;       // (token, n) entries per thread
  constexpr int kVR = (kTB * kRows + kThreads - 1) / kThreads;
  static_assert(kTB * NP % kThreads == 0, "staging must tile");
  __shared__ __attribute__((aligned(16))) float s_k[kTB][NP], s_q[kTB][NP];
  __shared__ __attribute__((aligned(16))) float s_sc[kTB][4];  // a, beta, rk, scale rq
  __shared__ float s_v[kTB][kRows], s_y[kTB][kRows];
  const int64_t L = a.L, H = a.H, P = a.P, G = a.G, N = a.N;
  const int tid = threadIdx.x, lq = tid % LPC, lr = tid / LPC;
  const int64_t h = blockIdx.y, b = blockIdx.z, g = h / (H / G);
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kRows, p = p0 + lr;
  int64_t row;
  if (!state_row(a, b, row)) return;  // the same for the whole workgroup
  const bool active = p < P;
  const float A2 = a.A[h] * kLog2e, bias = a.dt_bias ? a.dt_bias[h] : 0.f;

  float S[4 * NV];
  if (a.h0 != nullptr && active)
    load_row<VEC, LPC, NV>(a.h0 + ((row * H + h) * P + p) * N, lq, N, S);
  else
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) S[i] = 0.f;

  const T *kp = static_cast<const T *>(a.k), *qp = static_cast<const T *>(a.q);
  const T *vp = static_cast<const T *>(a.v);
  T rk[kKR], rq[kKR], rv[kVR], rd{}, rb{};
  auto issue = [&](int64_t t0) {  // indices clamped to the last token, so every load is in bounds
#pragma unroll
    for (int i = 0; i < kKR; ++i) {
      const int e = tid + i * kThreads, j = e / NP, n = e % NP;
      const int64_t t = t0 + j < L ? t0 + j : L - 1;
      const int64_t at = ((b * L + t) * G + g) * N + (n < N ? n : N - 1);
      rk[i] = kp[at];
      rq[i] = qp[at];
    }
#pragma unroll
    for (int i = 0; i < kVR; ++i) {
      const int e = tid + i * kThreads, j = (e / kRows) % kTB;
      const int64_t pp = p0 + e % kRows;
      const int64_t t = t0 + j < L ? t0 + j : L - 1;
      rv[i] = vp[((b * L + t) * H + h) * P + (pp < P ? pp : P - 1)];
    }
    const int64_t t = t0 + tid % kTB < L ? t0 + tid % kTB : L - 1;
    rd = static_cast<const T *>(a.dt)[(b * L + t) * H + h];
    rb = static_cast<const T *>(a.beta)[(b * L + t) * H + h];
  };
  auto stage = [&]() {
#pragma unroll
    for (int i = 0; i < kKR; ++i) {
      const int e = tid + i * kThreads, j = e / NP, n = e % NP;
      s_k[j][n] = n < N ? to_f32(rk[i]) : 0.f;
      s_q[j][n] = n < N ? to_f32(rq[i]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kVR; ++i) {
      const int e = tid + i * kThreads;
      if (e < kTB * kRows) s_v[e / kRows][e % kRows] = to_f32(rv[i]);
    }
    if (tid < kTB) {
      s_sc[tid][0] = fast_exp2(step_size(to_f32(rd), bias, a.dt_softplus) * A2);
      s_sc[tid][1] = to_f32(rb);
      if (!a.qk_norm) {
        s_sc[tid][2] = 1.f;
        s_sc[tid][3] = a.scale;
      }
    }
    if (a.qk_norm) {  // 16 lanes per token: its sums of squares
      __syncthreads();
      const int j = tid / 16, i0 = tid % 16;
      float sk = 0.f, sq = 0.f;
      for (int n = i0; n < NP; n += 16) {
        sk = fmaf(s_k[j][n], s_k[j][n], sk);
        sq = fmaf(s_q[j][n], s_q[j][n], sq);
      }
      sk = row_sum<16>(sk);
      sq = row_sum<16>(sq);
      if (i0 == 0) {
        s_sc[j][2] = 1.f / sqrtf(sk + kQkNormEps);
        s_sc[j][3] = a.scale * (1.f / sqrtf(sq + kQkNormEps));
      }
    }
  };
  static_assert(kThreads == 16 * kTB, "16 lanes per staged token");

  if (L > 0) issue(0);
  for (int64_t t0 = 0; t0 < L; t0 += kTB) {
    stage();
    __syncthreads();
    if (t0 + kTB < L) issue(t0 + kTB);
    const int nt = static_cast<int>(L - t0 < kTB ? L - t0 : kTB);
    for (int j = 0; j < nt; ++j) {
      if (a.h_ckpt != nullptr && (t0 + j) % kGdrSeg == 0 && active) {
        const int64_t nseg = (L + kGdrSeg - 1) / kGdrSeg;
        store_row<VEC, LPC, NV>(a.h_ckpt + (((b * H + h) * nseg + (t0 + j) / kGdrSeg) * P + p) * N, lq, N, S);
      }
      const float4 sc = *reinterpret_cast<const float4 *>(s_sc[j]);
      float kv[4 * NV], qv[4 * NV];
      lds_row<LPC, NV>(s_k[j], lq, kv);
      lds_row<LPC, NV>(s_q[j], lq, qv);
      const float y = gdr_token<LPC, NV>(S, kv, qv, s_v[j][lr], sc.x, sc.y, sc.z, sc.w);
      if (lq == 0) s_y[j][lr] = y;
    }
    __syncthreads();
    if (a.y != nullptr)
#pragma unroll
      for (int i = 0; i < kVR; ++i) {
        const int e = tid + i * kThreads, j = e / kRows;
        const int64_t pp = p0 + e % kRows;
        if (j < nt && pp < P)
          static_cast<T *>(a.y)[((b * L + t0 + j) * H + h) * P + pp] = from_f32<T>(s_y[j][e % kRows]);
      }
  }
  if (a.h_final != nullptr && active)
    store_row<VEC, LPC, NV>(a.h_final + ((row * H + h) * P + p) * N, lq, N, S);
}

// Decode: T tokens (few) for each sequence, the state in place.  Every lane
// loads its own part of k and q, a token ahead; the norms are formed where they
// are used.  A lane group holds R rows, kThreads / LPC apart.
template <typename T, int LPC, int NV, int R, bool VEC>
__global__ __launch_bounds__(kThreads) void gdr_step_kernel(GdrArgs a) {
  constexpr int kRows = kThreads / LPC;
  const int64_t L = a.L, H = a.H, P = a.P, G = a.G, N = a.N;
  const int tid = threadIdx.x, lq = tid % LPC, lr = tid / LPC;
  const int64_t h = blockIdx.y, b = blockIdx.z, g = h / (H / G);
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * (kRows * R) + lr;
  int64_t row;
  if (!state_row(a, b, row)) return;
  float *st = a.h_final + (row * H + h) * P * N;
  float S[R][4 * NV];
#pragma unroll
  for (int i = 0; i < R; ++i) {  // rows behind P: the last one's, never stored
    const int64_t p = p0 + kRows * i < P ? p0 + kRows * i : P - 1;
    load_row<VEC, LPC, NV>(st + p * N, lq, N, S[i]);
  }
  const float A2 = a.A[h] * kLog2e, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  T kn[4 * NV], qn[4 * NV], vn[R], dn, bn;
  auto load = [&](int64_t t) {
    const int64_t tok = b * L + t;
    load_raw<VEC, LPC, NV>(static_cast<const T *>(a.k) + (tok * G + g) * N, lq, N, kn);
    load_raw<VEC, LPC, NV>(static_cast<const T *>(a.q) + (tok * G + g) * N, lq, N, qn);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t p = p0 + kRows * i < P ? p0 + kRows * i : P - 1;
      vn[i] = static_cast<const T *>(a.v)[(tok * H + h) * P + p];
    }
    dn = static_cast<const T *>(a.dt)[tok * H + h];
    bn = static_cast<const T *>(a.beta)[tok * H + h];
  };
  load(0);
  for (int64_t t = 0; t < L; ++t) {
    float kv[4 * NV], qv[4 * NV], v[R];
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) {
      kv[i] = to_f32(kn[i]);
      qv[i] = to_f32(qn[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = to_f32(vn[i]);
    const float dv = to_f32(dn), beta = to_f32(bn);
    if (t + 1 < L) load(t + 1);
    const float decay = fast_exp2(step_size(dv, bias, a.dt_softplus) * A2);
    float rk = 1.f, rq = a.scale;
    if (a.qk_norm) {
      float sk = 0.f, sq = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) {
        sk = fmaf(kv[i], kv[i], sk);
        sq = fmaf(qv[i], qv[i], sq);
      }
      rk = 1.f / sqrtf(row_sum<LPC>(sk) + kQkNormEps);
      rq = a.scale * (1.f / sqrtf(row_sum<LPC>(sq) + kQkNormEps));
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float y = gdr_token<LPC, NV>(S[i], kv, qv, v[i], decay, beta, rk, rq);
      const int64_t p = p0 + kRows * i;
      if (p < P && lq == 0) static_cast<T *>(a.y)[((b * L + t) * H + h) * P + p] = from_f32<T>(y);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (p0 + kRows * i < P) store_row<VEC, LPC, NV>(st + (p0 + kRows * i) * N, lq, N, S[i]);
}

bool aligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

template <typename T, int LPC, int NV>
hipError_t launch_shape(const GdrArgs &a, bool step, hipStream_t s) {
  constexpr int kRows = kThreads / LPC;
  const dim3 grid(static_cast<unsigned>((a.P + kRows - 1) / kRows), static_cast<unsigned>(a.H),
                  static_cast<unsigned>(a.B));
  // 16-byte pieces of the state, 4 elements of q and k at once
  bool vec = a.N % 4 == 0 && aligned(a.h0, 16) && aligned(a.h_final, 16) && aligned(a.h_ckpt, 16);
  if (step) vec = vec && aligned(a.q, 4 * sizeof(T)) && aligned(a.k, 4 * sizeof(T));
  if (step) {
    // R = 4 rows a lane group where blocks of one row each would come to 8 per
    // CU or more: in flight then is what counts, and 4 rows share k, q and the
    // norms.  Below that the one row's shorter chain: 16384 one-row blocks of
    // 16 x 128 states 59.3 (R = 1) against 49.5 us (R = 4), 2048 of them 8.9
    // against 7.5, 1024 5.6 against 5.8, 128 3.4 against 4.6.
    constexpr int R = 4;
    if (vec && a.P > 2 * kRows && static_cast<int64_t>(grid.x) * grid.y * grid.z >= 8 * kCus) {
      const dim3 tall(static_cast<unsigned>((a.P + kRows * R - 1) / (kRows * R)), grid.y, grid.z);
      gdr_step_kernel<T, LPC, NV, R, true><<<tall, kThreads, 0, s>>>(a);
    } else if (vec) {
      gdr_step_kernel<T, LPC, NV, 1, true><<<grid, kThreads, 0, s>>>(a);
    } else {
      gdr_step_kernel<T, LPC, NV, 1, false><<<grid, kThreads, 0, s>>>(a);
    }
  } else {
    if (vec) gdr_seq_kernel<T, LPC, NV, true><<<grid, kThreads, 0, s>>>(a);
    else gdr_seq_kernel<T, LPC, NV, false><<<grid, kThreads, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const GdrArgs &a, bool step, hipStream_t s) {
  if (a.N <= 16) return launch_shape<T, 4, 1>(a, step, s);
  if (a.N <= 32) return launch_shape<T, 8, 1>(a, step, s);
  if (a.N <= 64) return launch_shape<T, 16, 1>(a, step, s);
  if (a.N <= 128) return launch_shape<T, 16, 2>(a, step, s);
  if (a.N <= 192) return launch_shape<T, 16, 3>(a, step, s);
  return launch_shape<T, 16, 4>(a, step, s);
}

}  // namespace

hipError_t launch_gdr_seq(const GdrArgs &a, hipStream_t s) {
  return a.dt_type == DType::BF16 ? launch_t<bf16_t>(a, false, s) : launch_t<float>(a, false, s);
}
hipError_t launch_gdr_step(const GdrArgs &a, hipStream_t s) {
  return a.dt_type == DType::BF16 ? launch_t<bf16_t>(a, true, s) : launch_t<float>(a, true, s);
}

}  // namespace ssm
