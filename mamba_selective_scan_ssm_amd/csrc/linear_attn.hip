// Linear attention with a decay for each head: how the sequences are cut, the
// decode step over a pool of states, and the sums of partial gradients.
//
// The step, per sequence, head h and row p of the state S (P, N), a = exp(log_decay[h]):
//   S <- a S + v[p] k;   y[p] = scale sum_n S[n] q[n]
// Rows never meet.  LPC adjacent lanes hold a row, NV groups of four consecutive
// states each, so the row moves in 16-byte pieces that are contiguous over the
// lanes; a lane group holds R rows.  Bound by the states' bytes, read and written once:
// 256 sequences of 80 heads of 64 x 128 0.262 ms, 5.1 TB/s, what a copy reaches; one
// sequence of 16 heads of 128 x 128 5 us of kernel in a call of 10.  R = 4 where blocks
// of one row a lane group would come to 8 a CU and more: those 256 sequences 269 us, with
// R = 1 289; the one sequence, 128 workgroups, 15 us with either.
#include "device_common.h"
#include "gdr_common.h"
#include "linear_attn.h"
#include "linear_attn_common.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kCus = 256;

template <typename T, int LPC, int NV, int R, bool VEC>
__global__ __launch_bounds__(kThreads) void la_step_kernel(LaStepArgs a, int64_t b0) {
  constexpr int kRows = kThreads / LPC;
  const int64_t H = a.H, P = a.P, G = a.G, N = a.N;
  const int tid = threadIdx.x, lq = tid % LPC, lr = tid / LPC;
  const int64_t h = blockIdx.y, b = b0 + blockIdx.z, gr = h / (H / G);
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * (kRows * R) + lr;
  int64_t row = b;
  if (a.slots != nullptr) {
    row = a.slots[b];
    if (row < 0 || row >= a.pool_rows) return;
  }
  const int64_t at = (row * H + h) * P * N;
  float S[R][4 * NV];
#pragma unroll
  for (int i = 0; i < R; ++i) {  // rows behind P: the last one's, never stored
    const int64_t p = p0 + kRows * i < P ? p0 + kRows * i : P - 1;
    if (a.s_in != nullptr) {
      load_row<VEC, LPC, NV>(a.s_in + at + p * N, lq, N, S[i]);
    } else {
#pragma unroll
      for (int n = 0; n < 4 * NV; ++n) S[i][n] = 0.f;
    }
  }
  T kn[4 * NV], qn[4 * NV], vn[R];
  auto load = [&](int64_t t) {
    const int64_t tok = b * a.T + t;
    load_raw<VEC, LPC, NV>(static_cast<const T *>(a.k) + (tok * G + gr) * N, lq, N, kn);
    load_raw<VEC, LPC, NV>(static_cast<const T *>(a.q) + (tok * G + gr) * N, lq, N, qn);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t p = p0 + kRows * i < P ? p0 + kRows * i : P - 1;
      vn[i] = static_cast<const T *>(a.v)[(tok * H + h) * P + p];
    }
  };
  load(0);
  const float la = a.log_decay[h];
  // as in LaCarry: what is rounded is the change
  const bool near = la > -0.6931f && la < 0.6931f;
  const float by = near ? expm1f(la) : expf(la), one = near ? 1.f : 0.f;
  for (int64_t t = 0; t < a.T; ++t) {
    float kv[4 * NV], qv[4 * NV], v[R];
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) {
      kv[i] = to_f32(kn[i]);
      qv[i] = to_f32(qn[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = to_f32(vn[i]);
    if (t + 1 < a.T) load(t + 1);
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int n = 0; n < 4 * NV; ++n) S[i][n] = fmaf(v[i], kv[n], fmaf(S[i][n], by, one * S[i][n]));
      const float y = a.scale * row_dot<LPC, NV>(S[i], qv);
      const int64_t p = p0 + kRows * i;
      if (p < P && lq == 0) static_cast<T *>(a.y)[((b * a.T + t) * H + h) * P + p] = from_f32<T>(y);
    }
  }
  if (a.s_out == nullptr) return;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (p0 + kRows * i < P) store_row<VEC, LPC, NV>(a.s_out + at + (p0 + kRows * i) * N, lq, N, S[i]);
}

template <typename T, int LPC, int NV>
hipError_t launch_step_shape(const LaStepArgs &a, bool vec, hipStream_t s) {
  constexpr int kRows = kThreads / LPC, R = 4;
  const int64_t one = (a.P + kRows - 1) / kRows, all = (a.P + kRows * R - 1) / (kRows * R);
  const bool tall = vec && a.P > 2 * kRows && one * a.H * a.S >= 8 * kCus;
  // a grid's second and third dimension hold 65535
  for (int64_t b = 0; b < a.S; b += 65535) {
    const int64_t n = a.S - b < 65535 ? a.S - b : 65535;
    const dim3 grid(static_cast<unsigned>(tall ? all : one), static_cast<unsigned>(a.H), static_cast<unsigned>(n));
    if (tall) la_step_kernel<T, LPC, NV, R, true><<<grid, kThreads, 0, s>>>(a, b);
    else if (vec) la_step_kernel<T, LPC, NV, 1, true><<<grid, kThreads, 0, s>>>(a, b);
    else la_step_kernel<T, LPC, NV, 1, false><<<grid, kThreads, 0, s>>>(a, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

bool aligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

template <typename T>
hipError_t launch_step(const LaStepArgs &a, hipStream_t s) {
  // 16-byte pieces of the state, 4 elements of q and k at once
  const bool vec = a.N % 4 == 0 && aligned(a.s_in, 16) && aligned(a.s_out, 16) && aligned(a.q, 4 * sizeof(T)) &&
                   aligned(a.k, 4 * sizeof(T));
  if (a.N <= 16) return launch_step_shape<T, 4, 1>(a, vec, s);
  if (a.N <= 32) return launch_step_shape<T, 8, 1>(a, vec, s);
  if (a.N <= 64) return launch_step_shape<T, 16, 1>(a, vec, s);
  if (a.N <= 128) return launch_step_shape<T, 16, 2>(a, vec, s);
  if (a.N <= 192) return launch_step_shape<T, 16, 3>(a, vec, s);
  return launch_step_shape<T, 16, 4>(a, vec, s);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void la_reduce_kernel(LaArgs a, const float *part, int64_t parts, int64_t G,
                                                             int64_t N, int64_t base, T *out) {
  // row = (token, group): its heads follow each other
  const int64_t i = base + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t rows = a.T * G, per = a.H / G;
  if (i >= rows * N) return;
  const int64_t row = i / N, n = i % N;
  if (a.cu != nullptr && (row / G < a.cu[0] || row / G >= a.cu[a.S])) return;  // of no sequence: left as it was
  float sum = 0.f;
  for (int64_t q = 0; q < parts; ++q)
    for (int64_t h = 0; h < per; ++h) sum += part[((q * rows + row) * per + h) * N + n];
  out[i] = from_f32<T>(sum);
}

// One workgroup a head: thread i sums every 256th, in 64 bits.
__global__ __launch_bounds__(kThreads) void la_reduce_dot_kernel(const double *part, int64_t slots, int64_t H,
                                                                 int64_t columns, float *out) {
  __shared__ double s[kThreads];
  const int64_t h = blockIdx.x;
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < slots * columns; i += kThreads)
    sum += part[(i / columns * H + h) * columns + i % columns];
  s[threadIdx.x] = sum;
  __syncthreads();
  for (int d = kThreads / 2; d > 0; d /= 2) {
    if (threadIdx.x < d) s[threadIdx.x] += s[threadIdx.x + d];
    __syncthreads();
  }
  if (threadIdx.x == 0) out[h] = static_cast<float>(s[0]);
}

}  // namespace

void la_plan(LaArgs &a, int64_t columns) {
  // As many segments as give each CU two workgroups of 64 columns (or one of 128), of
  // 64 tokens and more in fp32 and of 256 in bf16, whose kernel takes longer to begin.
  // At least 256 / 128 / 64 tokens: fp32, 2048 tokens of 24 heads of 64 x 64 86 / 69 / 69
  // us, gradients of 1031 tokens of 6 heads of 40 x 48 251 / 158 / 120; bf16, gradients
  // of 2048 tokens of 16 heads of 64 x 128 95 / 98 / 123.  Twice as many segments: bf16,
  // 2 x 8192 tokens, 64 heads of 128 x 128 403 -> 437 us, 4096 tokens, 32 heads 78 -> 111.
  // Left whole, the former: 413 -> 437 by eight waves, 128 workgroups, 413 -> 436 by four.
  constexpr int64_t kWanted = 2 * kCus;
  const int64_t least = a.dt_type == DType::F32 ? 64 : 256;
  const int64_t longest = a.L < 0 ? a.T : a.L;
  a.seg_len = longest > 0 ? longest : 1;
  a.slots = a.S;
  if (a.S <= 0 || (a.L >= 0 && a.S * a.H * columns * 4 >= kWanted * 3)) return;
  int64_t len = (a.T * a.H * columns + kWanted - 1) / kWanted;
  len = len < least ? least : (len + 63) / 64 * 64;
  if (len >= longest) return;
  a.seg_len = len;
  a.slots = a.L < 0 ? a.T / len + a.S : a.S * ((a.L + len - 1) / len);
}

hipError_t launch_la(const LaArgs &a, const LaPass *p, int n, hipStream_t s) {
  return a.dt_type == DType::BF16 ? launch_la_bf16(a, p, n, s) : launch_la_f32(a, p, n, s);
}

hipError_t launch_la_step(const LaStepArgs &a, hipStream_t s) {
  return a.dt_type == DType::BF16 ? launch_step<bf16_t>(a, s) : launch_step<float>(a, s);
}

hipError_t launch_la_reduce(const LaArgs &a, const float *part, int64_t parts, int64_t G, int64_t N, void *out,
                            hipStream_t s) {
  const int64_t all = a.T * G * N, most = int64_t{1} << 30;
  for (int64_t base = 0; base < all; base += most) {
    const int64_t n = all - base < most ? all - base : most;
    const unsigned grid = static_cast<unsigned>((n + kThreads - 1) / kThreads);
    if (a.dt_type == DType::BF16)
      la_reduce_kernel<bf16_t><<<grid, kThreads, 0, s>>>(a, part, parts, G, N, base, static_cast<bf16_t *>(out));
    else
      la_reduce_kernel<float><<<grid, kThreads, 0, s>>>(a, part, parts, G, N, base, static_cast<float *>(out));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_la_reduce_dot(const double *part, int64_t slots, int64_t H, int64_t columns, float *out,
                                hipStream_t s) {
  la_reduce_dot_kernel<<<static_cast<unsigned>(H), kThreads, 0, s>>>(part, slots, H, columns, out);
  return hipGetLastError();
}

}  // namespace ssm
