// C ABI of the gated delta rule and of the group norm: host-side validation
// and dispatch, as in capi.cpp (nothing is enqueued by a rejected call).
#include <cmath>

#include "capi_common.h"
#include "gdr.h"
#include "group_norm.h"

namespace {

using ssm::DType;
using namespace ssm::capi;

constexpr int64_t kMaxGridX = (int64_t(1) << 31) - 1;

struct GdrSizes {
  int64_t nQ, nV, nT, nS;  // elements of q (k), v (y), dt (beta), a state
};

// The checks of sizes that all entry points share.
ssm_status gdr_sizes(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype dt,
                     int32_t qk_norm, const ssm_delta_opts *dopts, GdrSizes *z) {
  if (B < 0 || L < 0 || H < 0 || P < 0 || G < 0 || N < 0 || !valid_dtype(dt) || !dopts_ok(dopts))
    return SSM_ERR_INVALID_ARG;
  if (qk_norm != 0 && qk_norm != 1) return SSM_ERR_INVALID_ARG;
  if (N < 1 || N > SSM_GDR_MAX_N) return SSM_ERR_UNSUPPORTED;
  if (G <= 0 || H % G != 0) return SSM_ERR_UNSUPPORTED;
  if (B > kMaxGridYZ || H > kMaxGridYZ) return SSM_ERR_UNSUPPORTED;
  int64_t tok, ckpt, chans;
  // the rows of a chunk of 64 tokens within 32-bit offsets
  if (!product({H, P}, &chans) || chans > int64_t{1} << 24) return SSM_ERR_UNSUPPORTED;
  if (!product({B, L, G, N}, &z->nQ) || !product({B, L, H, P}, &z->nV) || !product({B, L, H}, &z->nT) ||
      !product({B, H, P, N}, &z->nS) || !product({B, L, H, P, N}, &ckpt) || !product({B, L, G}, &tok) ||
      tok > kMaxGridX || P > kMaxGridX)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

ssm::GdrArgs gdr_args(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype dt, const void *q,
                      const void *k, const void *v, const void *dt_in, const float *A, const void *beta,
                      const float *h0, float scale, int32_t qk_norm, const ssm_delta_opts *dopts) {
  ssm::GdrArgs a{};
  a.B = B; a.L = L; a.H = H; a.P = P; a.G = G; a.N = N;
  a.dt_type = dt == SSM_BF16 ? DType::BF16 : DType::F32;
  a.q = q; a.k = k; a.v = v; a.dt = dt_in; a.A = A; a.beta = beta; a.h0 = h0;
  a.scale = scale; a.qk_norm = qk_norm != 0;
  a.dt_bias = dbias_of(dopts); a.dt_softplus = dsoft_of(dopts);
  return a;
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Whether two of the outputs share memory.
bool any_pair(const Range *r, size_t n) {
  for (size_t i = 0; i < n; ++i)
    for (size_t j = i + 1; j < n; ++j)
      if (overlap(r[i], r[j])) return true;
  return false;
}

}  // namespace

extern "C" {

// The prefill's kernels keep everything in registers and LDS.
size_t ssm_gdr_fwd_workspace_size(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, ssm_dtype) { return 0; }

ssm_status ssm_gdr_fwd(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype dt, const void *q,
                       const void *k, const void *v, const void *dt_in, const float *A, const void *beta,
                       const float *h0, float scale, int32_t qk_norm, void *y, float *h_final, void * /*workspace*/,
                       size_t /*workspace_bytes*/, const ssm_delta_opts *dopts, void *stream) {
  GdrSizes z;
  const ssm_status st = gdr_sizes(B, L, H, P, G, N, dt, qk_norm, dopts, &z);
  if (st != SSM_OK) return st;
  if (B == 0 || H == 0 || P == 0) return SSM_OK;
  if (!A || (L > 0 && (!q || !k || !v || !dt_in || !beta || !y))) return SSM_ERR_INVALID_ARG;
  const int64_t es = esize(dt);
  const Range ins[] = {{q, z.nQ * es},     {k, z.nQ * es}, {v, z.nV * es}, {dt_in, z.nT * es}, {A, H * 4},
                       {beta, z.nT * es}, {h0, z.nS * 4}, {dbias_of(dopts), H * 4}};
  const Range ry{y, z.nV * es}, rh{h_final, z.nS * 4};
  if (overlaps_any(ry, ins) || overlaps_any(rh, ins) || overlap(ry, rh)) return SSM_ERR_INVALID_ARG;
  ssm::GdrArgs a = gdr_args(B, L, H, P, G, N, dt, q, k, v, dt_in, A, beta, h0, scale, qk_norm, dopts);
  a.y = y;
  a.h_final = h_final;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return hip_status(ssm::gdr_chunk_applies(a) ? ssm::launch_gdr_chunk(a, s) : ssm::launch_gdr_seq(a, s));
}

ssm_status ssm_gdr_decode_steps(int64_t S, int64_t T, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype dt,
                                float *state_pool, int64_t pool_rows, const int32_t *slot_idx, const void *q,
                                const void *k, const void *v, const void *dt_in, const float *A, const void *beta,
                                float scale, int32_t qk_norm, void *y, const ssm_delta_opts *dopts, void *stream) {
  GdrSizes z;
  const ssm_status st = gdr_sizes(S, T, H, P, G, N, dt, qk_norm, dopts, &z);
  if (st != SSM_OK) return st;
  int64_t nPool;
  if (pool_rows < 0) return SSM_ERR_INVALID_ARG;
  if (!product({pool_rows, H, P, N}, &nPool)) return SSM_ERR_UNSUPPORTED;
  if (S == 0 || H == 0 || P == 0 || T == 0) return SSM_OK;
  if (slot_idx == nullptr && pool_rows < S) return SSM_ERR_INVALID_ARG;
  if (!q || !k || !v || !dt_in || !A || !beta || !y) return SSM_ERR_INVALID_ARG;
  if (slot_idx != nullptr && pool_rows == 0) return SSM_OK;  // every slot lies outside: all are skipped
  if (!state_pool) return SSM_ERR_INVALID_ARG;
  const int64_t es = esize(dt);
  const Range ins[] = {{q, z.nQ * es},     {k, z.nQ * es},    {v, z.nV * es},           {dt_in, z.nT * es}, {A, H * 4},
                       {beta, z.nT * es}, {slot_idx, S * 4}, {dbias_of(dopts), H * 4}};
  const Range ry{y, z.nV * es}, rp{state_pool, nPool * 4};
  if (overlaps_any(ry, ins) || overlaps_any(rp, ins) || overlap(ry, rp)) return SSM_ERR_INVALID_ARG;
  ssm::GdrArgs a = gdr_args(S, T, H, P, G, N, dt, q, k, v, dt_in, A, beta, state_pool, scale, qk_norm, dopts);
  a.y = y;
  a.h_final = state_pool;
  a.slots = slot_idx;
  a.pool_rows = pool_rows;
  return hip_status(ssm::launch_gdr_step(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_gdr_bwd_workspace_size(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype dt,
                                  int32_t aligned) {
  GdrSizes z;
  if (gdr_sizes(B, L, H, P, G, N, dt, 0, nullptr, &z) != SSM_OK || P < 1 || H < 1) return 0;
  if (aligned != 0 && aligned != 1) return 0;
  ssm::GdrBwdArgs a{};  // no pointers: all of them aligned
  a.f.B = B; a.f.L = L; a.f.H = H; a.f.P = P; a.f.G = G; a.f.N = N;
  a.f.dt_type = dt == SSM_BF16 ? DType::BF16 : DType::F32;
  const bool chunks = aligned == 1 && ssm::gdr_bwd_chunk_applies(a);
  return static_cast<size_t>(chunks ? ssm::gdr_bwd_chunk_ws_floats(B, L, H, P, G, N)
                                    : ssm::gdr_bwd_seq_ws_floats(B, L, H, P, G, N)) * 4;
}

ssm_status ssm_gdr_bwd(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype dt, const void *q,
                       const void *k, const void *v, const void *dt_in, const float *A, const void *beta,
                       const float *h0, const void *dy, const float *dh_final, float scale, int32_t qk_norm, void *dq,
                       void *dk, void *dv, void *ddt, void *dbeta, float *dA, float *dh0, float *d_dt_bias,
                       void *workspace, size_t workspace_bytes, const ssm_delta_opts *dopts, void *stream) {
  GdrSizes z;
  const ssm_status st = gdr_sizes(B, L, H, P, G, N, dt, qk_norm, dopts, &z);
  if (st != SSM_OK) return st;
  if (P < 1 || H < 1) return SSM_ERR_UNSUPPORTED;
  const bool data = B > 0 && L > 0;
  if (!A || !dA) return SSM_ERR_INVALID_ARG;
  if (data && (!q || !k || !v || !dt_in || !beta || !dy || !dq || !dk || !dv || !ddt || !dbeta))
    return SSM_ERR_INVALID_ARG;
  const int64_t es = esize(dt);
  const Range ins[] = {{q, z.nQ * es},     {k, z.nQ * es},         {v, z.nV * es}, {dt_in, z.nT * es},
                       {A, H * 4},         {beta, z.nT * es},      {h0, z.nS * 4}, {dy, z.nV * es},
                       {dh_final, z.nS * 4}, {dbias_of(dopts), H * 4}};
  ssm::GdrBwdArgs a{};
  a.f = gdr_args(B, L, H, P, G, N, dt, q, k, v, dt_in, A, beta, h0, scale, qk_norm, dopts);
  a.dy = dy; a.dh_final = dh_final;
  a.dq = dq; a.dk = dk; a.dv = dv; a.ddt = ddt; a.dbeta = dbeta;
  a.dA = dA; a.dbias = d_dt_bias; a.dh0 = dh0;
  a.ws = static_cast<float *>(workspace);
  const bool chunks = ssm::gdr_bwd_chunk_applies(a);
  const int64_t need = static_cast<int64_t>(ssm_gdr_bwd_workspace_size(B, L, H, P, G, N, dt, chunks ? 1 : 0));
  if (need > 0 && (!workspace || !aligned16(workspace) || static_cast<int64_t>(workspace_bytes) < need))
    return SSM_ERR_WORKSPACE;
  const Range outs[] = {{dq, z.nQ * es},    {dk, z.nQ * es}, {dv, z.nV * es},  {ddt, z.nT * es},
                        {dbeta, z.nT * es}, {dA, H * 4},     {dh0, z.nS * 4},  {d_dt_bias, H * 4},
                        {workspace, need}};
  for (const Range &r : outs)
    if (overlaps_any(r, ins)) return SSM_ERR_INVALID_ARG;
  if (any_pair(outs, sizeof(outs) / sizeof(outs[0]))) return SSM_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (B == 0) return hip_status(ssm::launch_gdr_reduce(a, 0, nullptr, nullptr, nullptr, nullptr, s));
  return hip_status(chunks ? ssm::launch_gdr_bwd_chunk(a, s) : ssm::launch_gdr_bwd_seq(a, s));
}

// ---------------------------------------------------------------- group norm

static ssm_status norm_sizes(int64_t S, int64_t T, int64_t D, int64_t G, ssm_dtype dt, float eps, int32_t center,
                             int32_t activation, int32_t gate_first, int64_t *n) {
  if (S < 0 || T < 0 || D < 0 || G < 0 || !valid_dtype(dt)) return SSM_ERR_INVALID_ARG;
  for (int32_t f : {center, activation, gate_first})
    if (f != 0 && f != 1) return SSM_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return SSM_ERR_INVALID_ARG;
  if (G < 1 || D % G != 0) return SSM_ERR_UNSUPPORTED;
  int64_t sd;
  if (!product({S, T, D}, n) || !product({S, D}, &sd) || sd > kMaxGridX || D > kMaxGridX || T > (int64_t(1) << 20))
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

size_t ssm_group_norm_fwd_workspace_size(int64_t S, int64_t T, int64_t D, int64_t G) {
  int64_t n;
  if (norm_sizes(S, T, D, G, SSM_F32, 0.f, 0, 0, 0, &n) != SSM_OK || n == 0) return 0;
  return static_cast<size_t>(ssm::group_norm_fwd_ws_floats(S, T, D, G)) * 4;
}
size_t ssm_group_norm_bwd_workspace_size(int64_t S, int64_t T, int64_t D, int64_t G) {
  int64_t n;
  if (norm_sizes(S, T, D, G, SSM_F32, 0.f, 0, 0, 0, &n) != SSM_OK || n == 0) return 0;
  return static_cast<size_t>(ssm::group_norm_bwd_ws_floats(S, T, D, G)) * 4;
}

// Sizes of a call whose tensors are all 16-byte aligned, or of one whose are not.
static ssm::NormArgs norm_of(int64_t S, int64_t T, int64_t D, int64_t G, ssm_dtype dt, int32_t aligned) {
  ssm::NormArgs a{};
  a.S = S; a.T = T; a.D = D; a.G = G;
  a.dt = dt == SSM_BF16 ? DType::BF16 : DType::F32;
  a.x = aligned ? nullptr : reinterpret_cast<const void *>(uintptr_t{1});
  return a;
}
size_t ssm_group_norm_fwd_workspace_size_ex(int64_t S, int64_t T, int64_t D, int64_t G, ssm_dtype dt,
                                            int32_t aligned) {
  int64_t n;
  if (norm_sizes(S, T, D, G, dt, 0.f, 0, 0, 0, &n) != SSM_OK || n == 0 || (aligned != 0 && aligned != 1)) return 0;
  return static_cast<size_t>(ssm::group_norm_fwd_ws_floats(norm_of(S, T, D, G, dt, aligned))) * 4;
}
size_t ssm_group_norm_bwd_workspace_size_ex(int64_t S, int64_t T, int64_t D, int64_t G, ssm_dtype dt,
                                            int32_t aligned) {
  int64_t n;
  if (norm_sizes(S, T, D, G, dt, 0.f, 0, 0, 0, &n) != SSM_OK || n == 0 || (aligned != 0 && aligned != 1)) return 0;
  return static_cast<size_t>(ssm::group_norm_bwd_ws_floats(norm_of(S, T, D, G, dt, aligned))) * 4;
}

ssm_status ssm_group_norm_fwd(int64_t S, int64_t T, int64_t D, int64_t G, ssm_dtype dt, const void *x, const void *z,
                              const float *weight, const float *bias, float eps, int32_t center, int32_t activation,
                              int32_t gate_first, void *y, float *mean, float *rstd, void *workspace,
                              size_t workspace_bytes, void *stream) {
  int64_t n;
  const ssm_status st = norm_sizes(S, T, D, G, dt, eps, center, activation, gate_first, &n);
  if (st != SSM_OK) return st;
  if (n == 0) return SSM_OK;
  if (!x || !y) return SSM_ERR_INVALID_ARG;
  if (mean && !center) return SSM_ERR_INVALID_ARG;
  const int64_t es = esize(dt);
  const Range ins[] = {{x, n * es}, {z, n * es}, {weight, D * 4}, {bias, D * 4}};
  ssm::NormArgs a{};
  a.S = S; a.T = T; a.D = D; a.G = G;
  a.dt = dt == SSM_BF16 ? DType::BF16 : DType::F32;
  a.x = x; a.z = z; a.w = weight; a.b = bias; a.eps = eps;
  a.center = center != 0; a.act = activation != 0; a.gate_first = gate_first != 0;
  a.y = y; a.mean = mean; a.rstd = rstd;
  a.ws = static_cast<float *>(workspace);
  const int64_t need = ssm::group_norm_fwd_ws_floats(a) * 4;
  if (need > 0 && (!workspace || !aligned16(workspace) || static_cast<int64_t>(workspace_bytes) < need))
    return SSM_ERR_WORKSPACE;
  const Range outs[] = {{y, n * es}, {mean, S * G * 4}, {rstd, S * G * 4}, {workspace, need}};
  for (const Range &r : outs)
    if (overlaps_any(r, ins)) return SSM_ERR_INVALID_ARG;
  if (any_pair(outs, sizeof(outs) / sizeof(outs[0]))) return SSM_ERR_INVALID_ARG;
  return hip_status(ssm::launch_group_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

ssm_status ssm_group_norm_bwd(int64_t S, int64_t T, int64_t D, int64_t G, ssm_dtype dt, const void *x, const void *z,
                              const float *weight, const float *bias, const void *dy, const float *mean,
                              const float *rstd, float eps, int32_t center, int32_t activation, int32_t gate_first,
                              void *dx, void *dz, float *dweight, float *dbias, void *workspace,
                              size_t workspace_bytes, void *stream) {
  int64_t n;
  const ssm_status st = norm_sizes(S, T, D, G, dt, eps, center, activation, gate_first, &n);
  if (st != SSM_OK) return st;
  if (D == 0) return SSM_OK;
  if (n > 0 && (!x || !dy || !rstd || !dx || (center && !mean))) return SSM_ERR_INVALID_ARG;
  if (n > 0 && ((z != nullptr) != (dz != nullptr))) return SSM_ERR_INVALID_ARG;
  const int64_t es = esize(dt);
  const Range ins[] = {{x, n * es},    {z, n * es},         {weight, D * 4},     {bias, D * 4},
                       {dy, n * es}, {mean, S * G * 4}, {rstd, S * G * 4}};
  ssm::NormArgs a{};
  a.S = S; a.T = T; a.D = D; a.G = G;
  a.dt = dt == SSM_BF16 ? DType::BF16 : DType::F32;
  a.x = x; a.z = z; a.w = weight; a.b = bias; a.eps = eps;
  a.center = center != 0; a.act = activation != 0; a.gate_first = gate_first != 0;
  a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
  a.dy = dy; a.dx = dx; a.dz = dz; a.dw = dweight; a.db = dbias;
  a.ws = static_cast<float *>(workspace);
  const int64_t need = n > 0 ? ssm::group_norm_bwd_ws_floats(a) * 4 : 0;
  if (need > 0 && (!workspace || !aligned16(workspace) || static_cast<int64_t>(workspace_bytes) < need))
    return SSM_ERR_WORKSPACE;
  const Range outs[] = {{dx, n * es}, {dz, n * es}, {dweight, D * 4}, {dbias, D * 4}, {workspace, need}};
  for (const Range &r : outs)
    if (overlaps_any(r, ins)) return SSM_ERR_INVALID_ARG;
  if (any_pair(outs, sizeof(outs) / sizeof(outs[0]))) return SSM_ERR_INVALID_ARG;
  return hip_status(ssm::launch_group_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
