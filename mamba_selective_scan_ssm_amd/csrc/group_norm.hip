// Group norm with an activation, channels last, and its gradients.
//
// x (S, T, D), G groups of W = D / G channels; mean and variance over the T
// tokens and W channels of a group (T = 1: per token, the norm that follows a
// mixer; T = L: a whole sequence).  With u = x silu(z) (gate first) or x,
//   xh = (u - mean) rstd,  n = xh w + b,  y = (SiLU? n) (silu(z) where the gate comes last)
// and, with dn the gradient of n and g = dn w,
//   du = rstd (g - mean(g) - xh mean(g xh)),  dw = sum dn xh,  db = sum dn
// (no mean(g) and no mean where not centred).
//
// Two paths, by the sizes alone:
//  - rows (T = 1, W up to 256 lanes x 8 pieces): a group's channels lie in the
//    registers of LPG adjacent lanes, so the statistics (the mean first, then
//    the squares about it) and the result take one pass over memory.  The
//    backward keeps its channels over a block of rows and sums dw and db in
//    registers; the blocks' sums are added in order by a second kernel.
//  - columns (everything else): per-channel sums over slices of the tokens,
//    coalesced whatever W is; a kernel that joins the slices and the channels
//    of a group (mean and squares about it by Chan's formula, as within a slice; the backward's
//    group sums are sums of its per-channel ones weighted by w); and a pass
//    that applies them.
// All sums are fp32 and in a fixed order.
//
// Bound by HBM where there is work: forward of 8 x 4096 tokens, 5120 channels in 8
// groups, gate first: 0.200 ms, 5.0 TB/s, what a copy reaches; forward and backward
// of 2 x 4096 tokens in 80 groups, gate last: 0.157 ms (53 + 98 + 7 us by themselves;
// the backward, 16 waves a CU by its registers, 4.3 TB/s).  Small ones by their
// launches: 4 x 1003 tokens of 640 channels in 32 groups, fp32, over whole sequences
// 47 us in 7 kernels, two of which join what a workgroup of the next could join.
#include "device_common.h"
#include "group_norm.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}
// silu(v) and its derivative s + v s (1 - s)
__device__ __forceinline__ float silu_grad(float v, float &slope) {
  const float s = sigmoid(v);
  slope = s * fmaf(v, 1.f - s, 1.f);
  return v * s;
}

// A dimension of a grid holds fewer than 2^32 threads: more workgroups than kMostX
// are laid out over z as well, and the last row's surplus ends at once.
constexpr int64_t kMostX = int64_t(1) << 22;
constexpr int64_t kMostTokens = 16 * 65535;  // at a time, 16 for a workgroup
__device__ __forceinline__ int64_t flat_block() {
  return blockIdx.x + static_cast<int64_t>(blockIdx.z) * gridDim.x;
}

// rounding may leave a variance below 0; a NaN stays one
__device__ __forceinline__ float not_negative(float v) { return v < 0.f ? 0.f : v; }

// VE consecutive elements (16 bytes where VE > 1)
template <typename T, int VE>
struct Piece {
  T v[VE];
};
template <typename T, int VE>
__device__ __forceinline__ Piece<T, VE> load_piece(const T *p) {
  Piece<T, VE> r;
  if constexpr (VE == 1) {
    r.v[0] = *p;
  } else {
    static_assert(sizeof(T) * VE == 16, "16-byte pieces");
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    __builtin_memcpy(r.v, &u, 16);
  }
  return r;
}
template <typename T, int VE>
__device__ __forceinline__ void store_piece(T *p, const float *f) {
  if constexpr (VE == 1) {
    *p = from_f32<T>(f[0]);
  } else {
    T v[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = from_f32<T>(f[e]);
    uint4 u;
    __builtin_memcpy(&u, v, 16);
    *reinterpret_cast<uint4 *>(p) = u;
  }
}
template <int VE>
__device__ __forceinline__ void load_f32(const float *p, float *f) {
  if constexpr (VE == 1) {
    f[0] = *p;
  } else {
#pragma unroll
    for (int e = 0; e < VE; e += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(p + e);
      f[e] = q.x;
      f[e + 1] = q.y;
      f[e + 2] = q.z;
      f[e + 3] = q.w;
    }
  }
}

// Sum over LPG adjacent lanes, every lane getting it; LPG = 256: the workgroup
// (s_red: 4 floats; the barriers order repeated uses).
template <int kCtrl>
__device__ __forceinline__ float dpp_get(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kCtrl, 0xF, 0xF, true));
}
template <int LPG>
__device__ __forceinline__ float lanes_sum(float v, float *s_red) {
  if constexpr (LPG >= 2) v += dpp_get<0xB1>(v);
  if constexpr (LPG >= 4) v += dpp_get<0x4E>(v);
  if constexpr (LPG >= 8) v += dpp_get<0x141>(v);
  if constexpr (LPG >= 16) v += dpp_get<0x140>(v);
  if constexpr (LPG >= 32) v += __shfl_xor(v, 16);
  if constexpr (LPG >= 64) v += __shfl_xor(v, 32);
  if constexpr (LPG == 256) {
    __syncthreads();
    if (threadIdx.x % 64 == 0) s_red[threadIdx.x / 64] = v;
    __syncthreads();
    v = (s_red[0] + s_red[1]) + (s_red[2] + s_red[3]);
  }
  return v;
}

// ------------------------------------------------------------------ rows
// Unit u = s G + g covers the W elements from u W.  Lane l of the unit holds
// the pieces l, l + LPG, ...
template <typename T, int VE, int LPG, int NV>
__global__ __launch_bounds__(kThreads) void norm_rows_fwd_kernel(NormArgs a) {
  __shared__ float s_red[4];
  const int64_t W = a.D / a.G, units = a.S * a.G;
  const int l = threadIdx.x % LPG;
  const int64_t u_raw = static_cast<int64_t>(blockIdx.x) * (kThreads / LPG) + threadIdx.x / LPG;
  const bool live = u_raw < units;
  const int64_t u = live ? u_raw : units - 1;
  const int64_t g = u % a.G;
  const int pieces = static_cast<int>(W / VE);
  const T *xp = static_cast<const T *>(a.x) + u * W;
  const T *zp = a.z ? static_cast<const T *>(a.z) + u * W : xp;  // read alike; unused without a gate
  Piece<T, VE> xr[NV], zr[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int at = l + j * LPG < pieces ? l + j * LPG : 0;
    xr[j] = load_piece<T, VE>(xp + at * VE);
    if (a.z) zr[j] = load_piece<T, VE>(zp + at * VE);
  }
  float v[NV][VE];
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      float f = to_f32(xr[j].v[e]);
      if (a.z && a.gate_first) f *= silu(to_f32(zr[j].v[e]));
      if (l + j * LPG >= pieces) f = 0.f;
      v[j][e] = f;
      sum += f;
    }
  const float inv = 1.f / static_cast<float>(W);
  const float mean = a.center ? lanes_sum<LPG>(sum, s_red) * inv : 0.f;
  // the values about the mean, and what the rounded mean leaves of their sum
  float sq = 0.f, left = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      v[j][e] = l + j * LPG < pieces ? v[j][e] - mean : 0.f;
      left += v[j][e];
      sq = fmaf(v[j][e], v[j][e], sq);
    }
  const float delta = a.center ? lanes_sum<LPG>(left, s_red) * inv : 0.f;
  const float var = not_negative(fmaf(lanes_sum<LPG>(sq, s_red), inv, -delta * delta));
  const float rstd = 1.f / sqrtf(var + a.eps);
  if (!live) return;
  if (l == 0) {
    if (a.mean) a.mean[u] = mean + delta;
    if (a.rstd) a.rstd[u] = rstd;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int at = l + j * LPG;
    if (at < pieces) {
      float wv[VE], bv[VE], out[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        wv[e] = 1.f;
        bv[e] = 0.f;
      }
      if (a.w) load_f32<VE>(a.w + g * W + at * VE, wv);
      if (a.b) load_f32<VE>(a.b + g * W + at * VE, bv);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        float n = fmaf((v[j][e] - delta) * rstd, wv[e], bv[e]);
        if (a.act) n = silu(n);
        if (a.z && !a.gate_first) n *= silu(to_f32(zr[j].v[e]));
        out[e] = n;
      }
      store_piece<T, VE>(static_cast<T *>(a.y) + u * W + at * VE, out);
    }
  }
}

// One element of the backward up to its normalised value and the gradient dn
// of n; what the gate's gradient needs is formed again where it is stored.
__device__ __forceinline__ void norm_elem(const NormArgs &a, float x, float z, float dy, float w, float b, float mean,
                                          float rstd, float &xh, float &dn) {
  const float zs = a.z ? silu(z) : 1.f;
  xh = ((a.gate_first ? x * zs : x) - mean) * rstd;
  float slope = 1.f;
  if (a.act) silu_grad(fmaf(xh, w, b), slope);
  dn = (a.gate_first ? dy : dy * zs) * slope;
}
// dx and dz of one element, from du
__device__ __forceinline__ void norm_elem_out(const NormArgs &a, float x, float z, float dy, float w, float b, float xh,
                                              float du, float &dx, float &dz) {
  dx = du;
  if (!a.z) return;
  float zslope;
  const float zs = silu_grad(z, zslope);
  if (a.gate_first) {
    dx = du * zs;
    dz = du * x * zslope;
  } else {
    const float n = fmaf(xh, w, b);
    dz = dy * (a.act ? silu(n) : n) * zslope;
  }
}

// The unit of the forward, its group fixed, walks the rows r0, r0 + step, ...
// of a block: units of a workgroup are gsub groups by rsub rows.
template <typename T, int VE, int LPG, int NV>
__global__ __launch_bounds__(kThreads, NV == 1 ? 4 : 1) void norm_rows_bwd_kernel(NormArgs a, int gsub, int64_t rows, int64_t parts) {
  __shared__ float s_red[4];
  const int64_t W = a.D / a.G;
  const int l = threadIdx.x % LPG, ui = threadIdx.x / LPG;
  const int rsub = kThreads / LPG / gsub;
  const int64_t g_raw = static_cast<int64_t>(blockIdx.x) * gsub + ui % gsub;
  const bool glive = g_raw < a.G;
  const int64_t g = glive ? g_raw : a.G - 1;
  const int64_t s0 = static_cast<int64_t>(blockIdx.y) * rows, s1 = s0 + rows < a.S ? s0 + rows : a.S;
  const int pieces = static_cast<int>(W / VE);
  const float inv = 1.f / static_cast<float>(W);
  float wv[NV][VE], bv[NV][VE], dw[NV][VE], db[NV][VE];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int at = l + j * LPG < pieces ? l + j * LPG : 0;
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      wv[j][e] = 1.f;
      bv[j][e] = dw[j][e] = db[j][e] = 0.f;
    }
    if (a.w) load_f32<VE>(a.w + g * W + at * VE, wv[j]);
    if (a.b) load_f32<VE>(a.b + g * W + at * VE, bv[j]);
  }
  const int64_t steps = (s1 - s0 + rsub - 1) / rsub;  // the same for every lane of the workgroup
  for (int64_t i = 0; i < steps; ++i) {
    const int64_t s_raw = s0 + i * rsub + ui / gsub;
    const bool live = glive && s_raw < s1;
    const int64_t s = s_raw < s1 ? s_raw : s1 - 1;
    const int64_t base = (s * a.G + g) * W;
    const T *xp = static_cast<const T *>(a.x) + base, *yp = static_cast<const T *>(a.dy) + base;
    const T *zp = a.z ? static_cast<const T *>(a.z) + base : xp;
    Piece<T, VE> xr[NV], yr[NV], zr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = l + j * LPG < pieces ? l + j * LPG : 0;
      xr[j] = load_piece<T, VE>(xp + at * VE);
      yr[j] = load_piece<T, VE>(yp + at * VE);
      if (a.z) zr[j] = load_piece<T, VE>(zp + at * VE);
    }
    const float mean = a.center ? a.mean[s * a.G + g] : 0.f, rstd = a.rstd[s * a.G + g];
    float sg = 0.f, sgx = 0.f;
    float xh[NV][VE], dn[NV][VE];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = l + j * LPG < pieces;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        norm_elem(a, to_f32(xr[j].v[e]), a.z ? to_f32(zr[j].v[e]) : 0.f, to_f32(yr[j].v[e]), wv[j][e], bv[j][e],
                  mean, rstd, xh[j][e], dn[j][e]);
        if (in) {
          const float gr = dn[j][e] * wv[j][e];
          sg += gr;
          sgx = fmaf(gr, xh[j][e], sgx);
        }
        if (in && live) {
          dw[j][e] = fmaf(dn[j][e], xh[j][e], dw[j][e]);
          db[j][e] += dn[j][e];
        }
      }
    }
    const float mg = a.center ? lanes_sum<LPG>(sg, s_red) * inv : 0.f;
    const float mgx = lanes_sum<LPG>(sgx, s_red) * inv;
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int at = l + j * LPG;
        if (at < pieces) {
          float ox[VE], oz[VE];
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float du = rstd * (dn[j][e] * wv[j][e] - mg - xh[j][e] * mgx);
            norm_elem_out(a, to_f32(xr[j].v[e]), a.z ? to_f32(zr[j].v[e]) : 0.f, to_f32(yr[j].v[e]), wv[j][e],
                          bv[j][e], xh[j][e], du, ox[e], oz[e]);
          }
          store_piece<T, VE>(static_cast<T *>(a.dx) + base + at * VE, ox);
          if (a.z) store_piece<T, VE>(static_cast<T *>(a.dz) + base + at * VE, oz);
        }
      }
    }
  }
  if (!glive) return;
  const int64_t part = static_cast<int64_t>(blockIdx.y) * rsub + ui / gsub;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int at = l + j * LPG;
    if (at < pieces)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int64_t d = g * W + at * VE + e;
        a.ws[part * a.D + d] = dw[j][e];
        a.ws[(parts + part) * a.D + d] = db[j][e];
      }
  }
}

// dw and db: the partial sums of a channel, added in order.  A workgroup holds
// 16 channels; 16 threads a channel take every 16th part and meet in LDS.
constexpr int kParamChannels = 16;
__global__ __launch_bounds__(kThreads) void norm_params_kernel(NormArgs a, int64_t parts, const float *pw,
                                                               const float *pb) {
  constexpr int kSplit = kThreads / kParamChannels;
  __shared__ float s_w[kSplit][kParamChannels], s_b[kSplit][kParamChannels];
  const int c = threadIdx.x % kParamChannels, k = threadIdx.x / kParamChannels;
  const int64_t d = flat_block() * kParamChannels + c;
  float x = 0.f, y = 0.f;
  if (d < a.D)
#pragma unroll 8
    for (int64_t i = k; i < parts; i += kSplit) {
      x += pw[i * a.D + d];
      y += pb[i * a.D + d];
    }
  s_w[k][c] = x;
  s_b[k][c] = y;
  __syncthreads();
  if (k == 0 && d < a.D) {
    x = y = 0.f;
#pragma unroll
    for (int i = 0; i < kSplit; ++i) {
      x += s_w[i][c];
      y += s_b[i][c];
    }
    if (a.dw) a.dw[d] = x;
    if (a.db) a.db[d] = y;
  }
}

// ------------------------------------------------------------------ columns
// Slices of `rows` tokens; a wave holds 64 VE channels of one slice, a
// workgroup 4 slices.  fwd: per channel the mean (less the slice's first value) and
// the squares about it, of four tokens after another joined with those before them:
// differences of sums would lose what a token far from the others leaves of them.
template <typename T, int VE>
__global__ __launch_bounds__(kThreads) void norm_cols_sums_kernel(NormArgs a, int64_t rows, int64_t slices) {
  const int lane = threadIdx.x % 64;
  const int64_t cb = (a.D + 64 * VE - 1) / (64 * VE), block = flat_block(), s = block / cb;
  const int64_t slice = static_cast<int64_t>(blockIdx.y) * 4 + threadIdx.x / 64;
  const int64_t d = (block % cb * 64 + lane) * VE;
  if (s >= a.S || slice >= slices || d >= a.D) return;
  const int64_t t0 = slice * rows, t1 = t0 + rows < a.T ? t0 + rows : a.T;
  const bool gate = a.z && a.gate_first;
  constexpr int kAhead = 4;  // tokens loaded together
  float first[VE], mean[VE], sq[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) first[e] = mean[e] = sq[e] = 0.f;
  for (int64_t t = t0; t < t1; t += kAhead) {
    Piece<T, VE> xr[kAhead], zr[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = (s * a.T + (t + i < t1 ? t + i : t1 - 1)) * a.D + d;
      xr[i] = load_piece<T, VE>(static_cast<const T *>(a.x) + at);
      if (gate) zr[i] = load_piece<T, VE>(static_cast<const T *>(a.z) + at);
    }
    // the four tokens' share of those so far
    const float before = static_cast<float>(t - t0), n = t + kAhead < t1 ? kAhead : static_cast<float>(t1 - t);
    const float inv = 1.f / n, share = n / (before + n);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      float u[kAhead], sum = 0.f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        u[i] = to_f32(xr[i].v[e]);
        if (gate) u[i] *= silu(to_f32(zr[i].v[e]));
        if (i == 0 && t == t0 && a.center) first[e] = u[0];
        u[i] -= first[e];
        if (t + i < t1) sum += u[i];
      }
      const float m = a.center ? sum * inv : 0.f, off = m - mean[e];
      float about = 0.f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (t + i < t1) about = fmaf(u[i] - m, u[i] - m, about);
      sq[e] += fmaf(off * off, before * share, about);
      mean[e] = fmaf(off, share, mean[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const int64_t at = (s * slices + slice) * a.D + d + e;
    // not centred: the squares about 0, and no mean
    a.ws[at] = first[e] + mean[e];
    a.ws[a.S * slices * a.D + at] = sq[e];
  }
}

// f(slice, place of slice and channel, channel) for a thread's share of a group's
// partial sums, slice after slice; the division is by 32 bits where it can be.
template <typename F>
__device__ __forceinline__ void each_partial(int64_t slices, int64_t W, int64_t D, F &&f) {
  if (slices * W < int64_t{1} << 31) {
    const uint32_t w = static_cast<uint32_t>(W), all = static_cast<uint32_t>(slices * W);
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < all; i += kThreads) {
      const uint32_t slice = i / w, c = i - slice * w;
      f(slice, slice * D + c, c);
    }
  } else {
    for (int64_t i = threadIdx.x; i < slices * W; i += kThreads) f(i / W, i / W * D + i % W, i % W);
  }
}

// one workgroup per (s, g): joins slices and channels
__global__ __launch_bounds__(kThreads) void norm_cols_join_kernel(NormArgs a, int64_t rows, int64_t slices, float *stat) {
  __shared__ float s_red[4];
  const int64_t W = a.D / a.G, block = flat_block(), g = block % a.G, s = block / a.G;
  if (s >= a.S) return;
  const float *pm = a.ws + s * slices * a.D + g * W, *p2 = pm + a.S * slices * a.D;
  const float inv = 1.f / (static_cast<float>(a.T) * static_cast<float>(W));
  auto count = [&](int64_t slice) {
    return static_cast<float>(slice + 1 < slices ? rows : a.T - slice * rows);
  };
  float mean = 0.f;
  if (a.center) {
    float m = 0.f;
    each_partial(slices, W, a.D, [&](int64_t slice, int64_t at, int64_t) { m = fmaf(count(slice), pm[at], m); });
    mean = lanes_sum<256>(m, s_red) * inv;
  }
  float sq = 0.f, left = 0.f;
  each_partial(slices, W, a.D, [&](int64_t slice, int64_t at, int64_t) {
    const float d = pm[at] - mean, nd = count(slice) * d;
    left += nd;
    sq += fmaf(nd, d, p2[at]);
  });
  const float delta = a.center ? lanes_sum<256>(left, s_red) * inv : 0.f;
  const float var = not_negative(fmaf(lanes_sum<256>(sq, s_red), inv, -delta * delta));
  const float rstd = 1.f / sqrtf(var + a.eps);
  if (threadIdx.x == 0) {
    stat[3 * (s * a.G + g)] = mean;
    stat[3 * (s * a.G + g) + 1] = rstd;
    stat[3 * (s * a.G + g) + 2] = delta;
    if (a.mean) a.mean[s * a.G + g] = mean + delta;
    if (a.rstd) a.rstd[s * a.G + g] = rstd;
  }
}

// y; VE divides W or is 1.  A thread holds VE channels of 4 tokens.
template <typename T, int VE>
__global__ __launch_bounds__(kThreads) void norm_cols_apply_kernel(NormArgs a, const float *stat) {
  const int lane = threadIdx.x % 64;
  const int64_t cb = (a.D + 64 * VE - 1) / (64 * VE), block = flat_block(), s = block / cb;
  const int64_t W = a.D / a.G, d = (block % cb * 64 + lane) * VE;
  if (s >= a.S || d >= a.D) return;
  const int64_t g = d / W;
  const float mean = stat[3 * (s * a.G + g)], rstd = stat[3 * (s * a.G + g) + 1];
  const float delta = stat[3 * (s * a.G + g) + 2];  // the mean's part below its fp32 step
  float wv[VE], bv[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    wv[e] = a.w ? a.w[d + e] : 1.f;
    bv[e] = a.b ? a.b[d + e] : 0.f;
  }
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.y) * 4 + threadIdx.x / 64) * 4; t0 < a.T; t0 += 16 * gridDim.y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + i;
      if (t >= a.T) return;
      const int64_t at = (s * a.T + t) * a.D + d;
      const Piece<T, VE> xr = load_piece<T, VE>(static_cast<const T *>(a.x) + at);
      Piece<T, VE> zr;
      if (a.z) zr = load_piece<T, VE>(static_cast<const T *>(a.z) + at);
      float out[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float zs = a.z ? silu(to_f32(zr.v[e])) : 1.f;
        float u = to_f32(xr.v[e]);
        if (a.gate_first) u *= zs;
        float n = fmaf((u - mean - delta) * rstd, wv[e], bv[e]);
        if (a.act) n = silu(n);
        if (!a.gate_first) n *= zs;
        out[e] = n;
      }
      store_piece<T, VE>(static_cast<T *>(a.y) + at, out);
    }
  }
}

// bwd: per channel the sums of dn and dn xh over a slice
template <typename T, int VE>
__global__ __launch_bounds__(kThreads) void norm_cols_bsums_kernel(NormArgs a, int64_t rows, int64_t slices) {
  const int lane = threadIdx.x % 64;
  const int64_t cb = (a.D + 64 * VE - 1) / (64 * VE), block = flat_block(), s = block / cb;
  const int64_t slice = static_cast<int64_t>(blockIdx.y) * 4 + threadIdx.x / 64;
  const int64_t d = (block % cb * 64 + lane) * VE;
  if (s >= a.S || slice >= slices || d >= a.D) return;
  const int64_t g = d / (a.D / a.G);
  const float mean = a.center ? a.mean[s * a.G + g] : 0.f, rstd = a.rstd[s * a.G + g];
  const int64_t t0 = slice * rows, t1 = t0 + rows < a.T ? t0 + rows : a.T;
  float wv[VE], bv[VE], s1[VE], s2[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    wv[e] = a.w ? a.w[d + e] : 1.f;
    bv[e] = a.b ? a.b[d + e] : 0.f;
    s1[e] = s2[e] = 0.f;
  }
  constexpr int kAhead = 4;  // tokens loaded together
  for (int64_t t = t0; t < t1; t += kAhead) {
    Piece<T, VE> xr[kAhead], yr[kAhead], zr[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = (s * a.T + (t + i < t1 ? t + i : t1 - 1)) * a.D + d;
      xr[i] = load_piece<T, VE>(static_cast<const T *>(a.x) + at);
      yr[i] = load_piece<T, VE>(static_cast<const T *>(a.dy) + at);
      if (a.z) zr[i] = load_piece<T, VE>(static_cast<const T *>(a.z) + at);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (t + i < t1)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          float xh, dn;
          norm_elem(a, to_f32(xr[i].v[e]), a.z ? to_f32(zr[i].v[e]) : 0.f, to_f32(yr[i].v[e]), wv[e], bv[e], mean, rstd,
                    xh, dn);
          s1[e] += dn;
          s2[e] = fmaf(dn, xh, s2[e]);
        }
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const int64_t at = (s * slices + slice) * a.D + d + e;
    a.ws[at] = s2[e];
    a.ws[a.S * slices * a.D + at] = s1[e];
  }
}

// one workgroup per (s, g): mean(g) and mean(g xh)
__global__ __launch_bounds__(kThreads) void norm_cols_bjoin_kernel(NormArgs a, int64_t slices, float *stat) {
  __shared__ float s_red[4];
  const int64_t W = a.D / a.G, block = flat_block(), g = block % a.G, s = block / a.G;
  if (s >= a.S) return;
  const float *p2 = a.ws + s * slices * a.D + g * W, *p1 = p2 + a.S * slices * a.D;
  const float inv = 1.f / (static_cast<float>(a.T) * static_cast<float>(W));
  float x = 0.f, y = 0.f;
  each_partial(slices, W, a.D, [&](int64_t, int64_t at, int64_t c) {
    const float w = a.w ? a.w[g * W + c] : 1.f;
    x = fmaf(w, p1[at], x);
    y = fmaf(w, p2[at], y);
  });
  x = lanes_sum<256>(x, s_red);
  y = lanes_sum<256>(y, s_red);
  if (threadIdx.x == 0) {
    stat[2 * (s * a.G + g)] = a.center ? x * inv : 0.f;
    stat[2 * (s * a.G + g) + 1] = y * inv;
  }
}

template <typename T, int VE>
__global__ __launch_bounds__(kThreads) void norm_cols_bapply_kernel(NormArgs a, const float *stat) {
  const int lane = threadIdx.x % 64;
  const int64_t cb = (a.D + 64 * VE - 1) / (64 * VE), block = flat_block(), s = block / cb;
  const int64_t W = a.D / a.G, d = (block % cb * 64 + lane) * VE;
  if (s >= a.S || d >= a.D) return;
  const int64_t g = d / W;
  const float mean = a.center ? a.mean[s * a.G + g] : 0.f, rstd = a.rstd[s * a.G + g];
  const float mg = stat[2 * (s * a.G + g)], mgx = stat[2 * (s * a.G + g) + 1];
  float wv[VE], bv[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    wv[e] = a.w ? a.w[d + e] : 1.f;
    bv[e] = a.b ? a.b[d + e] : 0.f;
  }
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.y) * 4 + threadIdx.x / 64) * 4; t0 < a.T; t0 += 16 * gridDim.y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + i;
      if (t >= a.T) return;
      const int64_t at = (s * a.T + t) * a.D + d;
      const Piece<T, VE> xr = load_piece<T, VE>(static_cast<const T *>(a.x) + at);
      const Piece<T, VE> yr = load_piece<T, VE>(static_cast<const T *>(a.dy) + at);
      Piece<T, VE> zr;
      if (a.z) zr = load_piece<T, VE>(static_cast<const T *>(a.z) + at);
      float ox[VE], oz[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float x = to_f32(xr.v[e]), z = a.z ? to_f32(zr.v[e]) : 0.f, dy = to_f32(yr.v[e]);
        float xh, dn;
        norm_elem(a, x, z, dy, wv[e], bv[e], mean, rstd, xh, dn);
        const float du = rstd * (dn * wv[e] - mg - xh * mgx);
        norm_elem_out(a, x, z, dy, wv[e], bv[e], xh, du, ox[e], oz[e]);
      }
      store_piece<T, VE>(static_cast<T *>(a.dx) + at, ox);
      if (a.z) store_piece<T, VE>(static_cast<T *>(a.dz) + at, oz);
    }
  }
}

// ------------------------------------------------------------------ choice
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// n workgroups for flat_block(), each y times
dim3 flat_grid(int64_t n, int64_t y = 1) {
  const int64_t x = n < kMostX ? n : kMostX;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y), static_cast<unsigned>(ceil_div(n, x)));
}
bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int vector_width(const NormArgs &a) {
  const int ve = a.dt == DType::BF16 ? 8 : 4;
  const bool ok = (a.D / a.G) % ve == 0 && aligned16(a.x) && aligned16(a.z) && aligned16(a.y) && aligned16(a.dy) &&
                  aligned16(a.dx) && aligned16(a.dz) && aligned16(a.w) && aligned16(a.b);
  return ok ? ve : 1;
}

// Lanes and pieces per lane of a group of `pieces` pieces of ve elements: 8
// lanes (128 bytes in a row) and more, with at most 5 pieces per lane; then the
// workgroup.  The backward, which holds six values an element, takes at most 2
// (3 where the workgroup shares the group; 8 single elements).
struct RowPlan {
  int lpg, nv;  // nv 0: the columns path
};
RowPlan plan_rows(int64_t pieces, int ve, bool bwd) {
  if (pieces <= 1) return {1, 1};
  if (pieces <= 2) return {2, 1};
  if (pieces <= 4) return {4, 1};
  if (pieces <= 8) return {8, 1};
  if (pieces <= 16) return {8, 2};
  if (bwd) {
    if (pieces <= 32) return {16, 2};
    if (pieces <= 64) return {32, 2};
    if (pieces <= 128) return {64, 2};
    // single elements leave registers for more of them, and a wave needs no barrier:
    // 8 x 4096 tokens of 1001 channels in 7 groups 209 us, 541 by a workgroup a group,
    // of 1197 in 3 groups 166 and 248
    if (ve == 1 && pieces <= 256) return {64, 4};
    if (ve == 1 && pieces <= 512) return {64, 8};
  } else {
    if (pieces <= 40) return {8, 5};
    if (pieces <= 48) return {16, 3};
    if (pieces <= 80) return {16, 5};
    if (pieces <= 96) return {32, 3};
    if (pieces <= 160) return {32, 5};
    if (pieces <= 320) return {64, 5};
  }
  if (pieces <= 512) return {256, 2};
  if (pieces <= 768) return {256, 3};
  if (pieces <= 1280 && !(bwd && ve == 8)) return {256, 5};
  if (pieces <= 2048 && ve == 1) return {256, 8};
  return {0, 0};
}

// Blocks of rows of the backward: a workgroup's four waves find room four times a
// CU where a lane holds one piece (128 registers), twice where it holds more, and
// each writes its sums of dw and db, as much as 1.6 rows, so beyond one a CU there
// are 8 rows and more for each.  With one a CU, 512, 768, 1024, 1536 in all (us):
// 2 x 4096 tokens of 5120 channels in 80 groups (one piece) 124 (three a CU) and 151,
// 122, 121, 130, 8 x 4096 of 2048 in 128 309, 188, 167, 162, 177; of 4096 in 1 (two
// pieces) 149, 104, 136, 118, 135; of 1024 in 16 (one piece, 4 rows at 1024) 32, 29,
// 32, 36, 42.
struct RowBwd {
  int gsub, rsub;
  int64_t rows, blocks, parts;
};
RowBwd plan_rows_bwd(int64_t S, int64_t G, RowPlan p) {
  constexpr int64_t kCus = 256;
  RowBwd r;
  const int units = kThreads / p.lpg;
  r.gsub = 1;
  while (r.gsub < units && r.gsub < G) r.gsub *= 2;
  r.rsub = units / r.gsub;
  const int64_t passes = ceil_div(S, r.rsub);  // rows in steps of rsub
  const int64_t across = ceil_div(G, r.gsub), room = (p.nv == 1 ? 4 : 2) * kCus;
  int64_t blocks = passes / 8;
  if (blocks < ceil_div(kCus, across)) blocks = ceil_div(kCus, across);
  if (blocks > room / across) blocks = room / across > 0 ? room / across : 1;
  r.rows = ceil_div(passes, blocks) * r.rsub;
  r.blocks = ceil_div(S, r.rows > 0 ? r.rows : 1);
  r.parts = r.blocks * r.rsub;
  return r;
}
// Tokens per slice: at least 8 where there are that many, 128 slices where that is
// more, at most 256 (sums one behind the other stay short).
int64_t slice_rows(int64_t T) {
  const int64_t r = ceil_div(T, 128);
  return r < 8 ? 8 : r < 256 ? r : 256;
}
int64_t cols_ws_floats(int64_t S, int64_t T, int64_t D, int64_t G) {
  const int64_t slices = ceil_div(T, slice_rows(T));
  return 2 * S * slices * D + 3 * S * G;
}

template <typename T, int VE, int LPG, int NV>
void rows_fwd(const NormArgs &a, hipStream_t s) {
  const int64_t blocks = ceil_div(a.S * a.G, kThreads / LPG);
  norm_rows_fwd_kernel<T, VE, LPG, NV><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
}
template <typename T, int VE, int LPG, int NV>
void rows_bwd(const NormArgs &a, hipStream_t s) {
  const RowBwd r = plan_rows_bwd(a.S, a.G, RowPlan{LPG, NV});
  const dim3 grid(static_cast<unsigned>(ceil_div(a.G, r.gsub)), static_cast<unsigned>(r.blocks));
  norm_rows_bwd_kernel<T, VE, LPG, NV><<<grid, kThreads, 0, s>>>(a, r.gsub, r.rows, r.parts);
  norm_params_kernel<<<flat_grid(ceil_div(a.D, kParamChannels)), kThreads, 0, s>>>(a, r.parts, a.ws,
                                                                                   a.ws + r.parts * a.D);
}
template <typename T, int VE, bool BWD>
bool rows(const NormArgs &a, hipStream_t s) {
  const RowPlan p = plan_rows(a.D / a.G / VE, VE, BWD);
#define SSM_NORM_CASE(LPG, NV)                         \
  if (p.lpg == LPG && p.nv == NV) {                    \
    if constexpr (BWD) rows_bwd<T, VE, LPG, NV>(a, s); \
    else rows_fwd<T, VE, LPG, NV>(a, s);               \
    return true;                                       \
  }
  SSM_NORM_CASE(1, 1) SSM_NORM_CASE(2, 1) SSM_NORM_CASE(4, 1) SSM_NORM_CASE(8, 1) SSM_NORM_CASE(8, 2)
  if constexpr (BWD) {
    SSM_NORM_CASE(16, 2) SSM_NORM_CASE(32, 2) SSM_NORM_CASE(64, 2)
    if constexpr (VE == 1) { SSM_NORM_CASE(64, 4) SSM_NORM_CASE(64, 8) }
  } else {
    SSM_NORM_CASE(8, 5) SSM_NORM_CASE(16, 3) SSM_NORM_CASE(16, 5) SSM_NORM_CASE(32, 3) SSM_NORM_CASE(32, 5)
    SSM_NORM_CASE(64, 5)
  }
  if constexpr (!(BWD && VE == 1)) { SSM_NORM_CASE(256, 2) }
  SSM_NORM_CASE(256, 3)
  if constexpr (!(BWD && VE == 8)) { SSM_NORM_CASE(256, 5) }
  if constexpr (VE == 1) { SSM_NORM_CASE(256, 8) }
#undef SSM_NORM_CASE
  return false;
}

template <typename T, int VE, bool BWD>
void cols(const NormArgs &a, hipStream_t s) {
  const int64_t rows = slice_rows(a.T), slices = ceil_div(a.T, rows);
  const int64_t cb = ceil_div(a.D, 64 * VE) * a.S;
  const dim3 gs = flat_grid(cb, ceil_div(slices, 4)), ga = flat_grid(cb, a.T <= kMostTokens ? ceil_div(a.T, 16) : kMostTokens / 16),
             gj = flat_grid(a.G * a.S);
  float *stat = a.ws + 2 * a.S * slices * a.D;
  if constexpr (BWD) {
    norm_cols_bsums_kernel<T, VE><<<gs, kThreads, 0, s>>>(a, rows, slices);
    norm_cols_bjoin_kernel<<<gj, kThreads, 0, s>>>(a, slices, stat);
    norm_cols_bapply_kernel<T, VE><<<ga, kThreads, 0, s>>>(a, stat);
    norm_params_kernel<<<flat_grid(ceil_div(a.D, kParamChannels)), kThreads, 0, s>>>(a, a.S * slices, a.ws,
                                                                                     a.ws + a.S * slices * a.D);
  } else {
    norm_cols_sums_kernel<T, VE><<<gs, kThreads, 0, s>>>(a, rows, slices);
    norm_cols_join_kernel<<<gj, kThreads, 0, s>>>(a, rows, slices, stat);
    norm_cols_apply_kernel<T, VE><<<ga, kThreads, 0, s>>>(a, stat);
  }
}

template <typename T, int VE, bool BWD>
void launch_ve(const NormArgs &a, hipStream_t s) {
  if (a.T == 1 && rows<T, VE, BWD>(a, s)) return;
  cols<T, VE, BWD>(a, s);
}
template <bool BWD>
hipError_t launch(const NormArgs &a, hipStream_t s) {
  const bool vec = vector_width(a) > 1;
  if (a.dt == DType::BF16) {
    if (vec) launch_ve<bf16_t, 8, BWD>(a, s);
    else launch_ve<bf16_t, 1, BWD>(a, s);
  } else {
    if (vec) launch_ve<float, 4, BWD>(a, s);
    else launch_ve<float, 1, BWD>(a, s);
  }
  return hipGetLastError();
}

// Of these sizes in pieces of ve elements.
int64_t fwd_floats(int64_t S, int64_t T, int64_t D, int64_t G, int ve) {
  return T == 1 && plan_rows(D / G / ve, ve, false).nv != 0 ? 0 : cols_ws_floats(S, T, D, G);
}
int64_t bwd_floats(int64_t S, int64_t T, int64_t D, int64_t G, int ve) {
  const RowPlan p = T == 1 ? plan_rows(D / G / ve, ve, true) : RowPlan{0, 0};
  return p.nv != 0 ? 2 * plan_rows_bwd(S, G, p).parts * D : cols_ws_floats(S, T, D, G);
}
// The most over either type and any alignment.
template <typename F>
int64_t of_any_width(int64_t W, F f) {
  int64_t n = 0;
  for (int ve : {1, 4, 8})
    if (W % ve == 0 && f(ve) > n) n = f(ve);
  return n;
}

}  // namespace

int64_t group_norm_fwd_ws_floats(const NormArgs &a) { return fwd_floats(a.S, a.T, a.D, a.G, vector_width(a)); }
int64_t group_norm_bwd_ws_floats(const NormArgs &a) { return bwd_floats(a.S, a.T, a.D, a.G, vector_width(a)); }
int64_t group_norm_fwd_ws_floats(int64_t S, int64_t T, int64_t D, int64_t G) {
  return of_any_width(D / G, [&](int ve) { return fwd_floats(S, T, D, G, ve); });
}
int64_t group_norm_bwd_ws_floats(int64_t S, int64_t T, int64_t D, int64_t G) {
  return of_any_width(D / G, [&](int ve) { return bwd_floats(S, T, D, G, ve); });
}

hipError_t launch_group_norm_fwd(const NormArgs &a, hipStream_t s) { return launch<false>(a, s); }
hipError_t launch_group_norm_bwd(const NormArgs &a, hipStream_t s) {
  if (a.S == 0 || a.T == 0) {
    norm_params_kernel<<<flat_grid(ceil_div(a.D, kParamChannels)), kThreads, 0, s>>>(a, 0, nullptr, nullptr);
    return hipGetLastError();
  }
  return launch<true>(a, s);
}

}  // namespace ssm
