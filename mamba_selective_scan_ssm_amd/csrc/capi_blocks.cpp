// C ABI of linear attention and of the norm with the residual's addition:
// host-side validation and dispatch, as in capi.cpp (nothing is enqueued by a
// rejected call).
#include <cmath>

#include "add_rms_norm.h"
#include "capi_common.h"
#include "linear_attn.h"

namespace {

using ssm::DType;
using namespace ssm::capi;

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1 - 256;
// Tokens up to which the step kernel runs a prefill: 64 sequences of 32 heads of 64 x 128,
// 4 / 8 / 16 tokens: bf16 36 / 51 / 81 us against 55 / 56 / 57 by chunks, fp32 28 / 36 / 55
// against 92 / 91 / 91; one sequence of 16 heads 13 against 14.
constexpr int64_t kTokenStep = 8;
constexpr int64_t kPart = 256;        // widest contraction of a pass

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
int64_t up(int64_t n) { return (n + 255) / 256 * 256; }

struct AttnSizes {
  int64_t nQ, nV, nS, S;  // elements of q (k), v (y), all states; sequences
};

ssm_status attn_sizes(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype dt, bool packed,
                      int64_t n_seqs, AttnSizes *z) {
  if (B < 0 || L < 0 || H < 0 || P < 0 || G < 0 || N < 0 || n_seqs < 0 || !valid_dtype(dt)) return SSM_ERR_INVALID_ARG;
  if (packed ? B != 1 : n_seqs != 0) return SSM_ERR_INVALID_ARG;
  if (N < 1 || N > SSM_LINEAR_ATTN_MAX_N) return SSM_ERR_UNSUPPORTED;
  if (G <= 0 || H % G != 0) return SSM_ERR_UNSUPPORTED;
  z->S = packed ? n_seqs : B;
  int64_t tok, width;
  if (H > kMaxGridYZ || !product({H, P}, &width) || width > int64_t{1} << 24) return SSM_ERR_UNSUPPORTED;
  if (!product({B, L}, &tok) || tok > kMaxTokens || z->S > kMaxTokens) return SSM_ERR_UNSUPPORTED;
  if (!product({B, L, G, N}, &z->nQ) || !product({B, L, H, P}, &z->nV) || !product({z->S, H, P, N}, &z->nS))
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

ssm::LaArgs attn_args(int64_t B, int64_t L, int64_t H, int64_t P, int64_t N, ssm_dtype dt, const float *log_decay,
                      const int32_t *cu, bool packed, int64_t S) {
  ssm::LaArgs a{};
  a.S = S; a.L = packed ? -1 : L; a.T = B * L;
  a.cu = cu; a.H = H; a.state = P * N;
  a.log_decay = log_decay;
  a.dt_type = dt == SSM_BF16 ? DType::BF16 : DType::F32;
  return a;
}

// The roles of a pass: q, k (by group, N wide) and v, dy (by head, P wide).
struct Rows {
  const void *p;
  int64_t row, width;
  int32_t per;
};
ssm::LaPass attn_pass(Rows x, Rows key, Rows val, int64_t K, int64_t M) {
  ssm::LaPass p{};
  p.x = x.p; p.x_row = x.row; p.x_width = x.width; p.x_per = x.per;
  p.key = key.p; p.key_row = key.row; p.key_width = key.width; p.key_per = key.per;
  p.val = val.p; p.val_row = val.row; p.val_width = val.width; p.val_per = val.per;
  p.K = static_cast<int32_t>(K); p.M = static_cast<int32_t>(M);
  p.c_out = p.c_in = 1.f;
  return p;
}

bool by_step(int64_t L, bool packed) { return !packed && L > 0 && L <= kTokenStep; }

// The backward's workspace, in bytes from its start.
struct AttnBwdSpace {
  ssm::LaArgs qk, v, tan;              // how each of its launches is cut
  int64_t parts;                       // of P, of up to kPart
  int64_t dq, dk, dv, tan_s, tan_u;    // local states
  int64_t part_q, part_k, dot, bytes;  // partial gradients (0 wide: written at once)
  bool direct;
};
AttnBwdSpace attn_bwd_space(const ssm::LaArgs &a, int64_t H, int64_t P, int64_t G, int64_t N, bool decay) {
  AttnBwdSpace w{};
  const int64_t cN = ssm::la_columns(N), cP = ssm::la_columns(P);
  w.qk = w.v = w.tan = a;
  ssm::la_plan(w.qk, 2 * cN);
  ssm::la_plan(w.v, cP);
  ssm::la_plan(w.tan, cP);
  w.parts = (P + kPart - 1) / kPart;
  w.direct = G == H && w.parts == 1;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t from = at;
    at += up(bytes);
    return from;
  };
  auto local = [&](const ssm::LaArgs &a, int64_t K, int64_t M) {
    return ssm::la_cut(a) ? ssm::la_local_floats(a, K, M) * 4 : 0;
  };
  const int64_t qk = local(w.qk, P < kPart ? P : kPart, N), tan = decay ? local(w.tan, N, P) : 0;
  w.dq = take(qk);
  w.dk = take(qk);
  w.dv = take(local(w.v, N, P));
  w.tan_s = take(tan);
  w.tan_u = take(tan);
  const int64_t part = w.direct ? 0 : w.parts * a.T * H * N * 4;
  w.part_q = take(part);
  w.part_k = take(part);
  w.dot = take(decay ? w.tan.slots * H * cP * 8 : 0);
  w.bytes = at;
  return w;
}

}  // namespace

extern "C" {

size_t ssm_linear_attn_fwd_workspace_size(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N,
                                          ssm_dtype dt, int32_t packed, int64_t n_seqs) {
  AttnSizes z;
  if (packed != 0 && packed != 1) return 0;
  if (attn_sizes(B, L, H, P, G, N, dt, packed == 1, n_seqs, &z) != SSM_OK) return 0;
  if (z.S == 0 || H == 0 || P == 0 || by_step(L, packed == 1)) return 0;
  ssm::LaArgs a = attn_args(B, L, H, P, N, dt, nullptr, nullptr, packed == 1, z.S);
  ssm::la_plan(a, ssm::la_columns(P));
  return ssm::la_cut(a) ? static_cast<size_t>(ssm::la_local_floats(a, N, P)) * 4 : 0;
}

ssm_status ssm_linear_attn_fwd(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype dt,
                               const void *q, const void *k, const void *v, const float *log_decay, const float *h0,
                               const int32_t *cu_seqlens, int64_t n_seqs, float scale, void *y, float *h_final,
                               void *workspace, size_t workspace_bytes, void *stream) {
  AttnSizes z;
  const bool packed = cu_seqlens != nullptr;
  const ssm_status st = attn_sizes(B, L, H, P, G, N, dt, packed, n_seqs, &z);
  if (st != SSM_OK) return st;
  if (z.S == 0 || H == 0 || P == 0) return SSM_OK;
  if (!log_decay || (L > 0 && (!q || !k || !v || !y))) return SSM_ERR_INVALID_ARG;
  const int64_t es = esize(dt);
  ssm::LaArgs a = attn_args(B, L, H, P, N, dt, log_decay, cu_seqlens, packed, z.S);
  ssm::la_plan(a, ssm::la_columns(P));
  const int64_t need = static_cast<int64_t>(
      ssm_linear_attn_fwd_workspace_size(B, L, H, P, G, N, dt, packed ? 1 : 0, n_seqs));
  if (need > 0 && (!workspace || !aligned16(workspace) || static_cast<int64_t>(workspace_bytes) < need))
    return SSM_ERR_WORKSPACE;
  const Range ins[] = {{q, z.nQ * es},     {k, z.nQ * es}, {v, z.nV * es},
                       {log_decay, H * 4}, {h0, z.nS * 4}, {cu_seqlens, packed ? (n_seqs + 1) * 4 : 0}};
  const Range outs[] = {{y, z.nV * es}, {h_final, z.nS * 4}, {workspace, need}};
  for (const Range &r : outs)
    if (overlaps_any(r, ins)) return SSM_ERR_INVALID_ARG;
  if (any_pair(outs, sizeof(outs) / sizeof(outs[0]))) return SSM_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (by_step(L, packed)) {
    const ssm::LaStepArgs t{B, L, H, P, G, N, a.dt_type, q, k, v, log_decay, scale, y, h0, h_final, nullptr, B};
    return hip_status(ssm::launch_la_step(t, s));
  }
  const int32_t per = static_cast<int32_t>(H / G);
  const Rows rq{q, G * N, N, per}, rk{k, G * N, N, per}, rv{v, H * P, P, 1};
  ssm::LaPass p = attn_pass(rq, rk, rv, N, P);
  p.out = y; p.out_row = H * P; p.out_width = P;
  p.c_out = scale;
  p.s0 = h0; p.s_last = h_final;
  p.sm = N; p.sn = 1;
  p.local = static_cast<float *>(workspace);
  return hip_status(ssm::launch_la(a, &p, 1, s));
}

ssm_status ssm_linear_attn_decode_steps(int64_t S, int64_t T, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype dt,
                                        float *state_pool, int64_t pool_rows, const int32_t *slot_idx, const void *q,
                                        const void *k, const void *v, const float *log_decay, float scale, void *y,
                                        void *stream) {
  AttnSizes z;
  const ssm_status st = attn_sizes(S, T, H, P, G, N, dt, false, 0, &z);
  if (st != SSM_OK) return st;
  int64_t nPool;
  if (pool_rows < 0) return SSM_ERR_INVALID_ARG;
  if (!product({pool_rows, H, P, N}, &nPool)) return SSM_ERR_UNSUPPORTED;
  if (S == 0 || H == 0 || P == 0 || T == 0) return SSM_OK;
  if (slot_idx == nullptr && pool_rows < S) return SSM_ERR_INVALID_ARG;
  if (!q || !k || !v || !log_decay || !y) return SSM_ERR_INVALID_ARG;
  if (slot_idx != nullptr && pool_rows == 0) return SSM_OK;  // every slot lies outside: all are skipped
  if (!state_pool) return SSM_ERR_INVALID_ARG;
  const int64_t es = esize(dt);
  const Range ins[] = {{q, z.nQ * es}, {k, z.nQ * es}, {v, z.nV * es}, {log_decay, H * 4}, {slot_idx, S * 4}};
  const Range ry{y, z.nV * es}, rp{state_pool, nPool * 4};
  if (overlaps_any(ry, ins) || overlaps_any(rp, ins) || overlap(ry, rp)) return SSM_ERR_INVALID_ARG;
  const ssm::LaStepArgs t{S, T, H, P, G, N, dt == SSM_BF16 ? DType::BF16 : DType::F32, q, k, v, log_decay, scale, y,
                          state_pool, state_pool, slot_idx, pool_rows};
  return hip_status(ssm::launch_la_step(t, static_cast<hipStream_t>(stream)));
}

size_t ssm_linear_attn_bwd_workspace_size(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N,
                                          ssm_dtype dt, int32_t packed, int64_t n_seqs, int32_t decay) {
  AttnSizes z;
  if ((packed != 0 && packed != 1) || (decay != 0 && decay != 1)) return 0;
  if (attn_sizes(B, L, H, P, G, N, dt, packed == 1, n_seqs, &z) != SSM_OK || H < 1 || P < 1) return 0;
  const ssm::LaArgs a = attn_args(B, L, H, P, N, dt, nullptr, nullptr, packed == 1, z.S);
  return static_cast<size_t>(attn_bwd_space(a, H, P, G, N, decay == 1).bytes);
}

ssm_status ssm_linear_attn_bwd(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype dt,
                               const void *q, const void *k, const void *v, const float *log_decay, const float *h0,
                               const int32_t *cu_seqlens, int64_t n_seqs, const void *dy, const float *dh_final,
                               float scale, void *dq, void *dk, void *dv, float *dh0, float *dlog_decay,
                               void *workspace, size_t workspace_bytes, void *stream) {
  AttnSizes z;
  const bool packed = cu_seqlens != nullptr;
  const ssm_status st = attn_sizes(B, L, H, P, G, N, dt, packed, n_seqs, &z);
  if (st != SSM_OK) return st;
  // the fp32 rows of a chunk of 64 tokens within 32-bit offsets
  if (P < 1 || H < 1 || P > SSM_LINEAR_ATTN_BWD_MAX_P || H * N > int64_t{1} << 22) return SSM_ERR_UNSUPPORTED;
  if (!log_decay || (B * L > 0 && (!q || !k || !v || !dy || !dq || !dk || !dv))) return SSM_ERR_INVALID_ARG;
  const int64_t es = esize(dt);
  const AttnBwdSpace w =
      attn_bwd_space(attn_args(B, L, H, P, N, dt, log_decay, cu_seqlens, packed, z.S), H, P, G, N, dlog_decay != nullptr);
  if (w.bytes > 0 && (!workspace || !aligned16(workspace) || static_cast<int64_t>(workspace_bytes) < w.bytes))
    return SSM_ERR_WORKSPACE;
  const Range ins[] = {{q, z.nQ * es},     {k, z.nQ * es}, {v, z.nV * es},
                       {log_decay, H * 4}, {h0, z.nS * 4}, {cu_seqlens, packed ? (n_seqs + 1) * 4 : 0},
                       {dy, z.nV * es},    {dh_final, z.nS * 4}};
  const Range outs[] = {{dq, z.nQ * es},  {dk, z.nQ * es},       {dv, z.nV * es},
                        {dh0, z.nS * 4}, {dlog_decay, H * 4}, {workspace, w.bytes}};
  for (const Range &r : outs)
    if (overlaps_any(r, ins)) return SSM_ERR_INVALID_ARG;
  if (any_pair(outs, sizeof(outs) / sizeof(outs[0]))) return SSM_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  auto floats = [&](int64_t at) { return reinterpret_cast<float *>(ws + at); };
  const ssm::LaArgs &a = w.qk;
  if (z.S == 0) return hip_status(dlog_decay ? ssm::launch_la_reduce_dot(nullptr, 0, H, 1, dlog_decay, s) : hipSuccess);

  const int32_t per = static_cast<int32_t>(H / G);
  const Rows rq{q, G * N, N, per}, rk{k, G * N, N, per}, rv{v, H * P, P, 1}, rdy{dy, H * P, P, 1};
  hipError_t e = hipSuccess;
  // dq and dk, over a part of P at a time
  for (int64_t i = 0; i < w.parts && e == hipSuccess; ++i) {
    const int64_t p0 = i * kPart, wide = P - p0 < kPart ? P - p0 : kPart;
    auto from = [&](Rows r) {
      r.p = r.p == nullptr ? nullptr : static_cast<const char *>(r.p) + p0 * es;
      return r;
    };
    auto state = [&](const float *h) { return h == nullptr ? nullptr : h + p0 * N; };
    ssm::LaPass p[2] = {attn_pass(from(rdy), from(rv), rk, wide, N), attn_pass(from(rv), from(rdy), rq, wide, N)};
    p[0].c_out = scale;
    p[0].s0 = state(h0);
    p[0].local = floats(w.dq);
    p[0].out = w.direct ? dq : floats(w.part_q) + i * a.T * H * N;
    p[1].c_in = scale;
    p[1].reverse = true;
    p[1].s0 = state(dh_final);
    p[1].local = floats(w.dk);
    p[1].out = w.direct ? dk : floats(w.part_k) + i * a.T * H * N;
    for (ssm::LaPass &x : p) {
      x.sm = 1;
      x.sn = N;
      x.out_row = H * N;
      x.out_width = N;
      x.out_f32 = !w.direct;
    }
    e = ssm::launch_la(a, p, 2, s);
  }
  if (e != hipSuccess) return hip_status(e);
  ssm::LaPass p = attn_pass(rk, rq, rdy, N, P);
  p.c_in = scale;
  p.reverse = true;
  p.s0 = dh_final; p.s_last = dh0;
  p.sm = N; p.sn = 1;
  p.local = floats(w.dv);
  p.out = dv; p.out_row = H * P; p.out_width = P;
  e = ssm::launch_la(w.v, &p, 1, s);
  if (e != hipSuccess) return hip_status(e);
  if (dlog_decay != nullptr) {
    p = attn_pass(rq, rk, rv, N, P);
    p.c_out = scale;
    p.s0 = h0;
    p.sm = N; p.sn = 1;
    p.local = floats(w.tan_s); p.local_tan = floats(w.tan_u);
    p.dot = dy; p.s_dot = dh_final;
    p.dot_sum = reinterpret_cast<double *>(ws + w.dot);
    e = ssm::launch_la(w.tan, &p, 1, s);
    if (e == hipSuccess)
      e = ssm::launch_la_reduce_dot(p.dot_sum, w.tan.slots, H, ssm::la_columns(P), dlog_decay, s);
    if (e != hipSuccess) return hip_status(e);
  }
  if (!w.direct) {
    e = ssm::launch_la_reduce(a, floats(w.part_q), w.parts, G, N, dq, s);
    if (e == hipSuccess) e = ssm::launch_la_reduce(a, floats(w.part_k), w.parts, G, N, dk, s);
  }
  return hip_status(e);
}

// ---------------------------------------------------------------- add + norm

static ssm_status add_norm_sizes(int64_t rows, int64_t D, ssm_dtype dt, ssm_dtype stream_dt, int64_t *n) {
  if (rows < 0 || D < 0 || !valid_dtype(dt) || !valid_dtype(stream_dt)) return SSM_ERR_INVALID_ARG;
  if (stream_dt == SSM_BF16 && dt == SSM_F32) return SSM_ERR_UNSUPPORTED;
  if (D > SSM_ADD_RMS_NORM_MAX_D || !product({rows, D}, n)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}
static ssm::AddNormArgs add_norm_args(int64_t rows, int64_t D, ssm_dtype dt, ssm_dtype stream_dt, const float *w) {
  ssm::AddNormArgs a{};
  a.rows = rows; a.D = D; a.w = w;
  a.dt = dt == SSM_BF16 ? DType::BF16 : DType::F32;
  a.stream = stream_dt == SSM_BF16 ? DType::BF16 : DType::F32;
  return a;
}

ssm_status ssm_add_rms_norm_fwd(int64_t rows, int64_t D, ssm_dtype dt, ssm_dtype stream_dt, const void *x,
                                const void *residual, const float *weight, float eps, int32_t quant,
                                int64_t quant_group, void *h, void *y, float *scale, float *rstd, void *stream) {
  int64_t n;
  const ssm_status st = add_norm_sizes(rows, D, dt, stream_dt, &n);
  if (st != SSM_OK) return st;
  if (quant < 0 || quant > 2 || quant_group < 0 || !(eps >= 0.f) || !std::isfinite(eps)) return SSM_ERR_INVALID_ARG;
  if (quant == 0 && quant_group != 0) return SSM_ERR_INVALID_ARG;
  if ((residual != nullptr) != (h != nullptr) && n > 0) return SSM_ERR_INVALID_ARG;
  if (residual == nullptr && dt != stream_dt) return SSM_ERR_INVALID_ARG;
  const int64_t group = quant_group == 0 ? D : quant_group;
  if (group != D && (group < ssm::kAddNormLeastGroup || D % group != 0)) return SSM_ERR_UNSUPPORTED;
  if (n == 0) return SSM_OK;
  if (!x || !y || (quant != 0) != (scale != nullptr)) return SSM_ERR_INVALID_ARG;
  const int64_t es = esize(dt), hs = esize(stream_dt);
  const Range ins[] = {{x, n * es}, {residual, n * hs}, {weight, D * 4}};
  const Range outs[] = {{h, n * hs}, {y, n * (quant ? 1 : es)}, {scale, quant ? rows * (D / group) * 4 : 0},
                        {rstd, rows * 4}};
  for (const Range &r : outs) {
    if (r.p == h && h == residual) {  // the sum in place of the residual
      if (overlap(r, ins[0]) || overlap(r, ins[2])) return SSM_ERR_INVALID_ARG;
    } else if (overlaps_any(r, ins)) {
      return SSM_ERR_INVALID_ARG;
    }
  }
  if (any_pair(outs, sizeof(outs) / sizeof(outs[0]))) return SSM_ERR_INVALID_ARG;
  ssm::AddNormArgs a = add_norm_args(rows, D, dt, stream_dt, weight);
  a.x = x; a.residual = residual; a.eps = eps;
  a.quant = quant; a.group = group;
  a.h = h; a.y = y; a.scale = scale; a.rstd = rstd;
  return hip_status(ssm::launch_add_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_add_rms_norm_bwd_workspace_size(int64_t rows, int64_t D) {
  int64_t n;
  if (add_norm_sizes(rows, D, SSM_F32, SSM_F32, &n) != SSM_OK || n == 0) return 0;
  return static_cast<size_t>(ssm::add_norm_bwd_ws_floats(rows, D)) * 4;
}

ssm_status ssm_add_rms_norm_bwd(int64_t rows, int64_t D, ssm_dtype dt, ssm_dtype stream_dt, const void *h,
                                const float *weight, const void *dy, const void *dh, const float *rstd, void *dx,
                                void *dresidual, float *dweight, void *workspace, size_t workspace_bytes,
                                void *stream) {
  int64_t n;
  const ssm_status st = add_norm_sizes(rows, D, dt, stream_dt, &n);
  if (st != SSM_OK) return st;
  if (D == 0) return SSM_OK;
  if (n > 0 && (!h || !dy || !rstd)) return SSM_ERR_INVALID_ARG;
  const int64_t need = dweight ? static_cast<int64_t>(ssm_add_rms_norm_bwd_workspace_size(rows, D)) : 0;
  if (need > 0 && (!workspace || !aligned16(workspace) || static_cast<int64_t>(workspace_bytes) < need))
    return SSM_ERR_WORKSPACE;
  const int64_t es = esize(dt), hs = esize(stream_dt);
  const Range ins[] = {{h, n * hs}, {weight, D * 4}, {dy, n * es}, {dh, n * hs}, {rstd, rows * 4}};
  const Range outs[] = {{dx, n * es}, {dresidual, n * hs}, {dweight, D * 4}, {workspace, need}};
  for (const Range &r : outs)
    if (overlaps_any(r, ins)) return SSM_ERR_INVALID_ARG;
  if (any_pair(outs, sizeof(outs) / sizeof(outs[0]))) return SSM_ERR_INVALID_ARG;
  ssm::AddNormArgs a = add_norm_args(rows, D, dt, stream_dt, weight);
  a.h = const_cast<void *>(h); a.dy = dy; a.dh = dh; a.rstd = const_cast<float *>(rstd);
  a.dx = dx; a.dresidual = dresidual; a.dw = dweight;
  a.ws = static_cast<float *>(workspace);
  return hip_status(ssm::launch_add_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
