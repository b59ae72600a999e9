// Launcher interface of the gated delta rule (gdr_seq.hip, gdr_chunk.hip,
// gdr_bwd.hip).  The arguments are validated by the C ABI before the launch.
#pragma once

#include "launch.h"

namespace ssm {

// 1 / sqrt(sum of squares + kQkNormEps): the norm of q and k.
constexpr float kQkNormEps = 1e-6f;

struct GdrArgs {
  int64_t B, L, H, P, G, N;
  DType dt_type;              // storage type of q, k, v, dt, beta and y
  const void *q, *k;          // (B, L, G, N)
  const void *v;              // (B, L, H, P)
  const void *dt;             // (B, L, H)
  const float *A;             // (H)
  const void *beta;           // (B, L, H)
  const float *h0;            // (B, H, P, N) or null
  float scale;                // of the output
  bool qk_norm;               // divide q and k by their 2-norms
  void *y;                    // (B, L, H, P)
  float *h_final;             // (B, H, P, N) or null
  const float *dt_bias;       // (H) or null: added to dt
  bool dt_softplus;           // softplus of (dt + bias)
  // Optional: sequence b reads h0 and writes h_final at row slots[b] of a
  // pool of pool_rows rows; a slot outside [0, pool_rows) skips it.
  const int32_t *slots;
  int64_t pool_rows;
  // Optional (token path): the state entering every kGdrSeg-token segment,
  // at (((b * H + h) * nseg + s) * P + p) * N + n.
  float *h_ckpt;
};

constexpr int kGdrSeg = 8;  // tokens per saved state of the token path

// Token by token on the vector ALU (gdr_seq.hip): any dtype, P, 1 <= N <= 256,
// any alignment, no workspace.  y may be null (states only).
hipError_t launch_gdr_seq(const GdrArgs &a, hipStream_t s);
// The same recurrence for a few tokens: the state goes from memory to
// registers and back once, nothing is staged.
hipError_t launch_gdr_step(const GdrArgs &a, hipStream_t s);

// By chunks of 64 tokens on the matrix cores (gdr_chunk.hip): bf16, N a
// multiple of 8 up to 128, L >= kGdrChunkMinL, q, k and the states 16-byte
// aligned; no workspace.  A chunk takes its time however few its tokens: 8
// sequences, 32 heads of 128 x 128: 29 to 30 us for 32 to 64 tokens, by tokens 26 for
// 24, 34 for 32, 57 for 64; gradients 109 to 115 us for 32 to 64 tokens, by tokens 137
// for 24, 167 for 32, 323 for 64.  2 sequences, 80 heads of 64 x 128: gradients 69 to
// 70, by tokens 75 for 16, 89 for 24, 151 for 64.
constexpr int64_t kGdrChunkMinL = 32;
bool gdr_chunk_applies(const GdrArgs &a);
// Columns of a state that a workgroup of a chain takes, 16 a wave: as few as leave
// each a CU of its own, where the waves that prepare the chunks are in the way of
// fewer of the chain's.  64 / 32 / 16: 4001 tokens, 32 heads of 128 x 128 297 / 279 /
// 260 us; 2048 tokens, 80 heads of 64 x 128 157 / 148 / (two on many CUs) 273;
// gradients of 4096 tokens, 16 heads of 64 x 128 674 / 599 / 578, of 2048 tokens, 32
// heads of 128 x 128 455 / 425 / 415.
inline int gdr_chain_columns(int64_t B, int64_t H, int64_t P) {
  constexpr int64_t kCus = 256;
  for (int cols = 16; cols < 64; cols *= 2)
    if (B * H * ((P + cols - 1) / cols) <= kCus) return cols;
  return 64;
}
hipError_t launch_gdr_chunk(const GdrArgs &a, hipStream_t s);

// What the chunked backward keeps of each (sequence, head, chunk), item
// (b H + h) ceil(L / 64) + chunk:
struct GdrSaved {
  float *S;    // (items, P, N): the state entering the chunk
  float *dS;   // (items, P, N): the gradient of the state leaving it
  float *E;    // (items, 64, P): the corrected values
  float *W;    // (items, 64, P): the gradient of v, before its rounding
  float *XM;   // (items, 20, 256): tiles of X, then of M, as the lanes hold them
  float *vec;  // (items, kGdrVec): a, b, w, 1 / |k|, 1 / |q|, and c in 64 bits
};
constexpr int64_t kGdrVec = 5 * 64 + 2 * 64;
// The prefill's chunks, kept (S, E, XM and vec) in place of y and h_final.
hipError_t launch_gdr_chunk_save(const GdrArgs &a, const GdrSaved &keep, hipStream_t s);

// Gradients by chunks (gdr_bwd_chunk.hip): where gdr_chunk_applies, and dy,
// dh_final, dh0 and the workspace 16-byte aligned.
struct GdrBwdArgs;
bool gdr_bwd_chunk_applies(const GdrBwdArgs &a);
int64_t gdr_bwd_chunk_ws_floats(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N);
hipError_t launch_gdr_bwd_chunk(const GdrBwdArgs &a, hipStream_t s);

struct GdrBwdArgs {
  GdrArgs f;                  // the forward's inputs (y, h_final unused)
  const void *dy;             // (B, L, H, P)
  const float *dh_final;      // (B, H, P, N) or null
  void *dq, *dk;              // (B, L, G, N), dtype
  void *dv, *ddt, *dbeta;     // dtype
  float *dA;                  // (H)
  float *dbias;               // (H) or null
  float *dh0;                 // (B, H, P, N) or null
  float *ws;
};

// Gradients token by token on the vector ALU: any dtype, P, 1 <= N <= 256.
int64_t gdr_bwd_seq_ws_floats(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N);
hipError_t launch_gdr_bwd_seq(const GdrBwdArgs &a, hipStream_t s);

// Sums of the per-head, per-tile partial gradients (gdr_bwd.hip), shared by
// the token path and the chunked path.  dq_part, dk_part: (tiles, B, L, H, N)
// of the normalised q and k; sc_part: (2, tiles, B, L, H), the gradients of
// beta and of the log decay; red: gdr_reduce_ws_floats floats.
int64_t gdr_reduce_ws_floats(int64_t B, int64_t L, int64_t H);
// Those of q and k alone, over `tiles` and each group's share of `parts` (H, or G
// where the heads are summed already); and dA and dbias alone, from nblk partial
// sums (2, H) each.
hipError_t launch_gdr_reduce_qk(const GdrBwdArgs &a, int64_t tiles, int64_t parts, const float *dq_part,
                                const float *dk_part, hipStream_t s);
hipError_t launch_gdr_reduce_params(const GdrBwdArgs &a, int64_t nblk, const float *red, hipStream_t s);
hipError_t launch_gdr_reduce(const GdrBwdArgs &a, int64_t tiles, const float *dq_part, const float *dk_part,
                             const float *sc_part, float *red, hipStream_t s);

}  // namespace ssm
