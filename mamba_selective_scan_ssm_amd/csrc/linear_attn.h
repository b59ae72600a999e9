// Launcher interface of linear attention with a decay for each head
// (linear_attn.hip, linear_attn_f32.hip, linear_attn_bf16.hip).  The arguments
// are validated by the C ABI before the launch.
#pragma once

#include "launch.h"

namespace ssm {

// One run of the recurrence over the tokens, per sequence and head:
//   S <- a S + c_in val_t key_t^T (M, K),   out_t = c_out S x_t,   a = exp(log_decay[h])
// The prefill is one (x = q, key = k, val = v) and so are the gradients, with the
// roles changed (dq: x = dy, key = v, val = k; dk: x = v, key = dy, val = q; dv:
// x = k, key = q, val = dy; the last two from the last token to the first, where
// the state passes to the next token already decayed).
struct LaPass {
  const void *x, *key, *val;            // row t of head h: t * row + (h / per) * width
  int64_t x_row, key_row, val_row, out_row;
  int32_t x_per, key_per, val_per;
  int64_t x_width, key_width, val_width, out_width;  // from head to head
  int32_t K, M;                         // widths that count
  void *out;                            // null: states alone
  bool out_f32;                         // out is fp32 whatever the inputs
  float c_out, c_in;                    // factors of out, and of what a token adds
  bool reverse;
  // State element (m, n), n < K, of sequence s and head h: (s H + h) state + m sm + n sn.
  const float *s0;                      // null: zeros
  float *s_last;                        // null: not returned
  int64_t sm, sn;
  // The tangent by log_decay in place of out: its product with dot (laid out as
  // val) is summed, and with s_dot at the end; a partial sum for each slot, head
  // and column block.
  const void *dot;
  const float *s_dot;
  double *dot_sum;
  // Workspace: what each segment adds to the state (and to its tangent), at
  // ((slot H + h) M + m) Kp + n, Kp = K rounded up to 16.
  float *local, *local_tan;
};

struct LaArgs {
  int64_t S, L, T;        // sequences; tokens of each, or -1: packed; of all
  const int32_t *cu;      // (S + 1) or null: first token of each sequence, and the end
  int64_t H, state;       // heads; elements of a head's state
  const float *log_decay; // (H)
  DType dt_type;
  // Segments: sequence s has ceil(length / seg_len) of them, whose slots begin at
  // floor(first token / seg_len) + s (s ceil(L / seg_len) where not packed).
  int64_t seg_len, slots;
};

// Tokens of a segment and the number of slots for these sizes.  A sequence is cut
// where there are too few chains to fill the GPU: each segment's own addition to
// the state is formed first (keys and values alone), then all segments run at once.
void la_plan(LaArgs &a, int64_t columns);
// Elements of one pass's local states.
inline int64_t la_local_floats(const LaArgs &a, int64_t K, int64_t M) {
  return a.slots * a.H * M * ((K + 15) / 16 * 16);
}
inline int64_t la_columns(int64_t M) { return (M + 63) / 64; }
inline bool la_cut(const LaArgs &a) { return a.slots > a.S; }

// By chunks, fp32 inputs, in fp32 matrix instructions (linear_attn_f32.hip): any size
// and alignment, K <= 256.  Passes of one number of columns run side by side.
hipError_t launch_la_f32(const LaArgs &a, const LaPass *p, int n, hipStream_t s);
// By chunks, bf16 inputs, on the bf16 matrix cores (linear_attn_bf16.hip).
hipError_t launch_la_bf16(const LaArgs &a, const LaPass *p, int n, hipStream_t s);
// The kernel that the type and the sizes choose.
hipError_t launch_la(const LaArgs &a, const LaPass *p, int n, hipStream_t s);

// A few tokens for each sequence, the state from memory to registers and back
// once (linear_attn.hip).
struct LaStepArgs {
  int64_t S, T, H, P, G, N;
  DType dt_type;
  const void *q, *k, *v;
  const float *log_decay;
  float scale;
  void *y;
  const float *s_in;      // (rows, H, P, N) or null: zeros
  float *s_out;           // the same pool, or one of its own, or null
  const int32_t *slots;   // null: row s for sequence s
  int64_t pool_rows;
};
hipError_t launch_la_step(const LaStepArgs &a, hipStream_t s);

// out[t][g][n] = sum over parts and over the heads of group g of part[.][t][h][n], for
// the tokens of the sequences.
hipError_t launch_la_reduce(const LaArgs &a, const float *part, int64_t parts, int64_t G, int64_t N, void *out,
                            hipStream_t s);
// out[h] = sum over slots and columns of part[(slot H + h) columns + column].
hipError_t launch_la_reduce_dot(const double *part, int64_t slots, int64_t H, int64_t columns, float *out,
                                hipStream_t s);

}  // namespace ssm
