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
// contractions end in log2(LPC) steps between lanes.  All state is fp32 in
// registers from the first token to the last.  A workgroup holds 256 / LPC rows of
// one head.
//
// Bound: the prefill by the chain of one token (two sums over lanes, whose DPP
// steps take 13 cycles each one behind the other, 7 beside others): fp32, 2048
// tokens, 24 heads of 64 x 128 0.30 ms, 146 ns a token; with many rows by the
// VALU: 16 x 512 tokens, 32 heads of 128 x 128 in 16 groups, states in and out, 0.77
// ms, 39 TFLOP/s.  The decode
// step by the state's bytes, read and written once: 256 sequences of 80 heads of
// 64 x 128 0.270 ms, 5.0 TB/s, what a copy reaches.
#include "device_common.h"
#include "gdr.h"
#include "gdr_common.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
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

// Rows of a (L, ..) tensor of one sequence, `pitch` bytes apart, from a token on
// that steps by 8; `width` bytes of the last row count.
struct Rows {
  uint64_t at;
  int64_t rest, step;
  __device__ __forceinline__ Rows(const void *first, int64_t L, int64_t pitch, int64_t width)
      : at(reinterpret_cast<uint64_t>(first)), rest((L - 1) * pitch + width), step(8 * pitch) {}
  // of the 8 tokens that have come; the next ones come
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t next() {
    constexpr int64_t kMost = 0x7fffffff;
    const __amdgpu_buffer_rsrc_t r = buffer_of(reinterpret_cast<const void *>(at),
                                               static_cast<uint32_t>(rest < 0 ? 0 : rest < kMost ? rest : kMost));
    at += step;
    rest -= step;
    return r;
  }
};

// Prefill, in groups of 8 tokens.  k and q of a group go through LDS, 16 lanes a
// row, which form the norms on the way: loaded 3 groups ahead, staged one ahead,
// one barrier a group.  What is one number a token (decay, beta, the norms, a
// row's v and y) is held by the lanes, lane j of 8 that of token j, and taken from
// there by DPP.  Tokens behind the last read as zeros and leave the state as it
// is.  Y false: the states alone, entering every kGdrSeg tokens (h_ckpt).
template <typename T, int LPC, int NV, bool Y, bool VEC>
__global__ __launch_bounds__(kThreads) void gdr_seq_kernel(GdrArgs a) {
  constexpr int kRows = kThreads / LPC, NP = 4 * LPC * NV, kFours = NP / 64;
  constexpr uint32_t kSize = sizeof(T);
  static_assert(kGdrSeg == 8 && kThreads == 16 * 16 && NP % 64 == 0, "16 lanes for each of 8 rows of k and q");
  __shared__ __attribute__((aligned(16))) float s_x[2][2][8][NP];  // k, q
  __shared__ float s_norm[2][2][8];                                // and 1 / |k|, scale / |q|
  const int64_t L = a.L, H = a.H, P = a.P, G = a.G, N = a.N;
  const int tid = threadIdx.x, lq = tid % LPC, mine = tid % 8;
  const int64_t h = blockIdx.y, b = blockIdx.z, g = h / (H / G);
  const int64_t p_raw = static_cast<int64_t>(blockIdx.x) * kRows + tid / LPC;
  int64_t row;
  if (!state_row(a, b, row)) return;  // the same for the whole workgroup
  const bool active = p_raw < P;
  const int64_t p = active ? p_raw : P - 1;
  const float A2 = a.A[h] * kLog2e, bias = a.dt_bias ? a.dt_bias[h] : 0.f;

  float S[4 * NV];
  if (a.h0 != nullptr)
    load_row<VEC, LPC, NV>(a.h0 + ((row * H + h) * P + p) * N, lq, N, S);
  else
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) S[i] = 0.f;

  const int wave = __builtin_amdgcn_readfirstlane(tid / 64), tok = 4 * (wave % 2) + tid % 64 / 16;
  const uint32_t row_at = static_cast<uint32_t>(tok * G * N) * kSize;
  const uint32_t gate_at = static_cast<uint32_t>(mine * H) * kSize, v_at = static_cast<uint32_t>(mine * H * P + p) * kSize;
  Four<VEC, T> x[2][kFours];
  T dn[2], bn[2], vn[2];
  auto rows = [&](const void *base, int64_t inner, int64_t first, int64_t width) {
    return Rows(static_cast<const T *>(base) + b * L * inner + first, L, inner * kSize, width * kSize);
  };
  Rows rows_x = rows(wave < 2 ? a.k : a.q, G * N, g * N, N), rows_dt = rows(a.dt, H, h, 1),
       rows_beta = rows(a.beta, H, h, 1), rows_v = rows(a.v, H * P, h * P, P), rows_y = rows(a.y, H * P, h * P, P);
  auto load_x = [&](int w) {
    const __amdgpu_buffer_rsrc_t r = rows_x.next();
#pragma unroll
    for (int j = 0; j < kFours; ++j) {
      const int n = 4 * (tid % 16 + 16 * j);
      x[w][j].load(r, n < N ? row_at + n * kSize : kNowhere, n, N);
    }
  };
  auto load_gates = [&](int w) {
    dn[w] = load_one<T>(rows_dt.next(), gate_at);
    bn[w] = load_one<T>(rows_beta.next(), gate_at);
    vn[w] = load_one<T>(rows_v.next(), v_at);
  };
  auto stage = [&](int w) {
    float ss = kQkNormEps / 16;
#pragma unroll
    for (int j = 0; j < kFours; ++j) {
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = to_f32(x[w][j].v[e]);
        ss = fmaf(f[e], f[e], ss);
      }
      *reinterpret_cast<float4 *>(&s_x[w][wave / 2][tok][4 * (tid % 16 + 16 * j)]) = make_float4(f[0], f[1], f[2], f[3]);
    }
    float r = 1.f;
    if (a.qk_norm) r = inverse_root(row_sum<16>(ss));
    if (tid % 16 == 0) s_norm[w][wave / 2][tok] = wave < 2 ? r : a.scale * r;
  };
  load_x(0);
  load_x(1);
  load_gates(0);
  load_gates(1);
  stage(0);
  load_x(0);
  meet_in_lds();
  auto group = [&](int64_t t0, auto parity) {
    constexpr int w = decltype(parity)::value;
    if (a.h_ckpt != nullptr && active)
      store_row<VEC, LPC, NV>(a.h_ckpt + (((b * H + h) * ((L + 7) / 8) + t0 / 8) * P + p) * N, lq, N, S);
    const float rk = s_norm[w][0][mine], rq = s_norm[w][1][mine], v = to_f32(vn[w]);
    const float decay = t0 + mine < L ? fast_exp2(step_size(to_f32(dn[w]), bias, a.dt_softplus) * A2) : 1.f;
    const float ar = -(decay * rk), br = to_f32(bn[w]) * rk;  // e = v + ar (S k), u = br e
    stage(1 - w);
    load_x(1 - w);
    load_gates(w);
    float y = 0.f, kv[2][4 * NV], qv[2][4 * NV];
    lds_row<LPC, NV>(s_x[w][0][0], lq, kv[0]);
    each<8>([&](auto number) {
      constexpr int i = decltype(number)::value;
      // what the next token's sums take is on its way while this one's are formed
      if constexpr (i < 7) lds_row<LPC, NV>(s_x[w][0][i + 1], lq, kv[1 - i % 2]);
      if constexpr (Y) lds_row<LPC, NV>(s_x[w][1][i], lq, qv[i % 2]);
      __builtin_amdgcn_sched_barrier(0);
      // y of the token before beside this one's S k
      if constexpr (Y && i > 0) {
        const float yt = row_dot<LPC, NV>(S, qv[1 - i % 2]);
        if (mine == i - 1) y = yt;
      }
      const float al = row_lane<i>(decay);
      const float u = row_lane<i>(br) * fmaf(row_lane<i>(ar), row_dot<LPC, NV>(S, kv[i % 2]), row_lane<i>(v));
#pragma unroll
      for (int n = 0; n < 4 * NV; ++n) S[n] = fmaf(al, S[n], u * kv[i % 2][n]);
    });
    if constexpr (Y) {
      const float yt = row_dot<LPC, NV>(S, qv[1]);
      if (mine == 7) y = yt;
    }
    if constexpr (Y)
      store_one(from_f32<T>(rq * y), rows_y.next(), active && lq < 8 ? v_at : kNowhere);
    meet_in_lds();
  };
  for (int64_t t0 = 0; t0 < L; t0 += 16) {
    group(t0, std::integral_constant<int, 0>());
    if (t0 + 8 < L) group(t0 + 8, std::integral_constant<int, 1>());
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
      rk = inverse_root(row_sum<LPC>(sk) + kQkNormEps);
      rq = a.scale * inverse_root(row_sum<LPC>(sq) + kQkNormEps);
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
hipError_t launch_seq_shape(const GdrArgs &a, bool vec, hipStream_t s) {
  constexpr int kRows = kThreads / LPC;
  const dim3 grid(static_cast<unsigned>((a.P + kRows - 1) / kRows), static_cast<unsigned>(a.H),
                  static_cast<unsigned>(a.B));
  if (a.y != nullptr) {
    if (vec) gdr_seq_kernel<T, LPC, NV, true, true><<<grid, kThreads, 0, s>>>(a);
    else gdr_seq_kernel<T, LPC, NV, true, false><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (vec) gdr_seq_kernel<T, LPC, NV, false, true><<<grid, kThreads, 0, s>>>(a);
    else gdr_seq_kernel<T, LPC, NV, false, false><<<grid, kThreads, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <typename T, int LPC, int NV>
hipError_t launch_step_shape(const GdrArgs &a, bool vec, hipStream_t s) {
  constexpr int kRows = kThreads / LPC;
  const dim3 grid(static_cast<unsigned>((a.P + kRows - 1) / kRows), static_cast<unsigned>(a.H),
                  static_cast<unsigned>(a.B));
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
  return hipGetLastError();
}

// 16-byte pieces of the state, 4 elements of q and k at once
template <typename T>
bool fours(const GdrArgs &a) {
  return a.N % 4 == 0 && aligned(a.h0, 16) && aligned(a.h_final, 16) && aligned(a.h_ckpt, 16) &&
         aligned(a.q, 4 * sizeof(T)) && aligned(a.k, 4 * sizeof(T));
}
template <typename T>
hipError_t launch_step(const GdrArgs &a, hipStream_t s) {
  const bool vec = fours<T>(a);
  if (a.N <= 16) return launch_step_shape<T, 4, 1>(a, vec, s);
  if (a.N <= 32) return launch_step_shape<T, 8, 1>(a, vec, s);
  if (a.N <= 64) return launch_step_shape<T, 16, 1>(a, vec, s);
  if (a.N <= 128) return launch_step_shape<T, 16, 2>(a, vec, s);
  if (a.N <= 192) return launch_step_shape<T, 16, 3>(a, vec, s);
  return launch_step_shape<T, 16, 4>(a, vec, s);
}
template <typename T>
hipError_t launch_seq(const GdrArgs &a, hipStream_t s) {
  const bool vec = fours<T>(a);
  // 32 lanes a row where that leaves at most one wave per SIMD: half the work on
  // a token's chain, one step more to its sums.  24 heads of 64 x 128, 2048
  // tokens: 309 against 350 us with 16 lanes; 2048 rows x 256: 102 against 135;
  // but 8192 rows x 256 253 against 197, 16384 x 128 332 against 230.
  const bool wide = a.B * a.H * a.P * 32 / 64 <= 4 * kCus;
  if (a.N <= 64) return launch_seq_shape<T, 16, 1>(a, vec, s);
  if (a.N <= 128) return wide ? launch_seq_shape<T, 32, 1>(a, vec, s) : launch_seq_shape<T, 16, 2>(a, vec, s);
  if (wide) return launch_seq_shape<T, 32, 2>(a, vec, s);
  return a.N <= 192 ? launch_seq_shape<T, 16, 3>(a, vec, s) : launch_seq_shape<T, 16, 4>(a, vec, s);
}

}  // namespace

hipError_t launch_gdr_seq(const GdrArgs &a, hipStream_t s) {
  return a.dt_type == DType::BF16 ? launch_seq<bf16_t>(a, s) : launch_seq<float>(a, s);
}
hipError_t launch_gdr_step(const GdrArgs &a, hipStream_t s) {
  return a.dt_type == DType::BF16 ? launch_step<bf16_t>(a, s) : launch_step<float>(a, s);
}

}  // namespace ssm
