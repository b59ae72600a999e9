// Linear attention by chunks of 64 tokens on the bf16 matrix cores.
//
// The formulas are those of linear_attn_f32.hip.  A workgroup of W waves runs 16 W
// columns m of one head's chain over a segment, 16 columns a wave, whose part of the
// state S (n down, m across) stays in its registers.  x, keys and values of a chunk lie
// in LDS, double-buffered, and come there straight from memory a chunk ahead.
//
// v_mfma_f32_16x16x32_bf16 on lane 16 g + r takes A[r][k], B[k][r] for the 8
// contraction indices k of slot g and gives C[4 g + e][r]; which index a slot stands
// for is free as long as both operands agree, so
//  - n: slot (g, 4 u + e) of block kb is n = 32 kb + 8 g + 4 u + e, 16 bytes of a row
//    as it lies in memory; rows 4 g + e of the state's tile 2 kb + u are these n (the
//    transposing reads of the keys choose them so), and S is an operand as it is;
//  - tokens: slot (g, 4 u + e) of block tb is token 32 tb + 16 u + 4 g + e, so two
//    score tiles key . x, one above the other, are the operand of the values'
//    product as they are.
// Outputs come out as C[m][token]: a lane's four channels are one store.
//
// Eight waves (128 columns, where M passes 64) form the ten score tiles below the
// diagonal once and share them through LDS, behind the chunk's second barrier.  Four
// waves (64 columns, two workgroups a CU) form them each for itself.  M = 128, 8 x 2048
// tokens, 64 heads, K = 128: 285 us with eight, 344 with four; M = 64, 4 x 4096 tokens, 64
// heads, K = 64: 214 with eight, half of them without a column, 171 with four.  K above 128
// takes 144 KB and one workgroup a CU.
//
// Precision: inputs are exact in bf16.  What is computed enters a product in bf16
// parts: the weighted values, from which the state is made, in three (all 24 bits),
// the scores and S, from which the outputs are made, in two (off by 2^-18 of each
// term; the output is rounded to 2^-9, or summed over heads in fp32 and then rounded),
// and in three where they make the decays' gradient, which stays in fp32.  Sums are fp32.
//
// Bound by the phases' latency and issue, not by a unit: 2 x 8192 tokens, 64 heads of
// 128 x 128 take 0.37 to 0.43 ms (by the card; 2.5 to 3.0 TB/s of inputs and outputs, 160 to
// 190 TFLOP/s of the recurrence's work).  A chunk takes 7.8 thousand cycles on its CU, of
// which the matrix cores are busy for 3.1, the vector units issue for about as many, the
// LDS for 2.6.  By a clock in each phase (8.2 with the clocks), thousand cycles of the first
// and the last four of the eight waves: asking for rows 0.4, checks 0.3, scores 0.7 to 1.3 /
// 0.7, the state's answers 1.5 / 2.2, the barrier and the scores' values 1.3 to 1.9 / 0.9 to
// 1.1, the state 1.7 / 2.7, stores 0.7 / 0.6, the last barrier 1.1 / 0.1.  The loop of eight
// waves with whole 16-byte rows holds no spill: its reload would wait for the rows on their
// way, which the same counter counts.  Other kernels have some: of whole rows, four waves with
// K from 65 to 128 7 registers; of rows that are no whole 16 bytes, whose next chunk is held in
// registers too, four waves with K from 65 to 128 291, the others up to 46.
//
// Measured and dropped: 32 columns a wave, four waves (14.3 thousand cycles for the same
// chunk: one wave a SIMD), three buffers (2 x 8192 tokens: 424 -> 428 us, a chunk hides its
// loads), a raised priority of the later four waves (no change), the weighted values
// before the barrier (8 x 2048 tokens: 291 -> 300 us).
#include "device_common.h"
#include "linear_attn.h"
#include "linear_attn_common.h"

namespace ssm {
namespace {

// Element offset of 16-byte piece c of row t.  The LDS has 64 banks; which exchange of
// a row's pieces meets fewest of them twice was measured for each kind of read, in
// cycles a wave: x, sixteen rows' one piece, 5.8 (rows without an exchange 33); keys,
// read transposing, four rows' four pieces and half of each, 5.6 (9.4 with x's); values,
// four rows by two whole pieces, 4.0.  Rows of 128 bytes: by t % 8 for all of them.
template <int PIECES>
__device__ __forceinline__ constexpr int x_at(int t, int c) {
  return t * PIECES * 8 + 8 * (c ^ t % (PIECES < 16 ? PIECES : 16));
}
template <int PIECES>
__device__ __forceinline__ constexpr int key_at(int t, int c) {
  return t * PIECES * 8 + 8 * (c ^ (PIECES < 16 ? t % PIECES : 4 * (t % 4) + t / 4 % 4));
}
template <int PIECES>
__device__ __forceinline__ constexpr int value_at(int t, int c) {
  return t * PIECES * 8 +
         8 * (c ^ (PIECES < 16 ? t % PIECES : 4 * (t % 2) + 2 * (t / 2 % 2) + 8 * (t / 4 % 2) + t / 8 % 2));
}

__device__ __forceinline__ float low_half(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_half(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

constexpr uint32_t kOutside = 0x80000000u;  // of every buffer, and so is what lies a little behind

// 16 bytes of a row from element n on; those from `width` on are 0
__device__ __forceinline__ u32x4 load_piece(__amdgpu_buffer_rsrc_t r, uint32_t at, int n, int width) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = n + 2 * i;
    const uint32_t lo = load_one<bf16_t>(r, e < width ? at + 2 * e : kOutside).bits;
    const uint32_t hi = load_one<bf16_t>(r, e + 1 < width ? at + 2 * e + 2 : kOutside).bits;
    v[i] = lo | hi << 16;
  }
  return v;
}

// 16 bytes of each lane's address into LDS at `to`, one lane's behind the other's.  In
// assembly: of the builtin the compiler does not know which LDS it writes, and waits for
// it before the next read of any; who reads it waits for it here (vmcnt).
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint64_t u = static_cast<uint64_t>(v);
  return static_cast<int64_t>(
      static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32)))) << 32 |
      static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u))));
}
// Whether a state's rows are whole pieces of four consecutive n.
__device__ __forceinline__ bool fours_of(const LaPass &p, const float *state) {
  return p.sn == 1 && p.sm % 4 == 0 && p.K % 4 == 0 && reinterpret_cast<uintptr_t>(state) % 16 == 0;
}
// A slot's numbers in scalar registers (bounds that are loaded come in vector ones).
__device__ __forceinline__ LaSlot la_uniform(const LaSlot &z) {
  LaSlot r;
  r.seq = uniform(z.seq);
  r.first = uniform(z.first);
  r.step = uniform(z.step);
  r.before = uniform(z.before);
  r.slot0 = uniform(z.slot0);
  r.len = __builtin_amdgcn_readfirstlane(z.len);
  r.last = __builtin_amdgcn_readfirstlane(static_cast<int>(z.last)) != 0;
  return r;
}
struct Rows {
  u32x4 words;
  __device__ __forceinline__ Rows(const void *base, uint32_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    words = u32x4{static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32) & 0xffffu, bytes, 0x00020000u};
  }
};
__device__ __forceinline__ void fetch_lds(const Rows &r, uint32_t to, uint32_t at, uint32_t more) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to), "v"(at), "s"(r.words),
               "s"(more)
               : "memory", "m0");
}

// fp32 as a sum of NP bf16 parts, as split4 of gdr_mfma.h, the rest by a shift (or a
// mask) and a subtraction: v_dot2c_f32_bf16 writes over its operand, which has to be
// copied where it is wanted again, and is waited for.
template <int NP>
__device__ __forceinline__ void split_four(f32x4 v, u32x2 *out) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    out[p] = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    if (p + 1 < NP)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] -= e % 2 ? high_half(out[p][e / 2]) : low_half(out[p][e / 2]);
  }
}
template <int NP>
__device__ __forceinline__ void split_parts(f32x4 top, f32x4 bottom, u32x4 *out) {
  u32x2 a[NP], b[NP];
  split_four<NP>(top, a);
  split_four<NP>(bottom, b);
#pragma unroll
  for (int p = 0; p < NP; ++p) out[p] = u32x4{a[p][0], a[p][1], b[p][0], b[p][1]};
}

template <int N>
using Number = std::integral_constant<int, N>;

// Weights from the log decay in units of log 2: a^n, 1 for n = 0 whatever a.
__device__ __forceinline__ float power_of(double log2_a, int n) {
  return n == 0 ? 1.f : fast_exp2(static_cast<float>(log2_a * n));
}

// KB: blocks of 32 that K is rounded up to; W waves of 16 columns each.  SHARE: the
// scores are formed once, by all waves, and shared through LDS; else by each wave.
template <int KB, int W, bool SHARE, bool Y, bool TAN, bool VEC>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(KB == 8 || TAN ? 1 : 2)))
void la_bf16_kernel(LaArgs a, LaPasses all, int64_t items, int64_t sub, int64_t base) {
  constexpr int kThreads = 64 * W, C = 64, KP = 4 * KB, kColumns = 16 * W, VP = kColumns / 8;
  constexpr int kRowsK = C * KP / kThreads, kRowsV = C * VP / kThreads;  // pieces a thread brings
  constexpr uint32_t kTile = 2 * C * KP * 8, kTileV = 2 * C * VP * 8;    // bytes
  constexpr int kParts = TAN ? 3 : 2;  // of S and of the scores
  // two buffers of keys, of values, of x, and (shared) two parts of the scores: one
  // array, so that two workgroups find room where these are 80 KB
  constexpr int kSizeK = C * KP * 8, kSizeV = C * VP * 8;
  __shared__ __attribute__((aligned(128))) uint16_t lds[2 * kSizeK + 2 * kSizeV + (Y ? 2 * kSizeK : 0) +
                                                        (Y && SHARE ? 2 * C * C : 0)];
  uint16_t *const s_k = lds, *const s_v = lds + 2 * kSizeK, *const s_x = s_v + 2 * kSizeV,
                  *const s_a = s_x + (Y ? 2 * kSizeK : 0);

  const LaPass &p = all.p[blockIdx.y];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64, r = lane % 16,
            g = lane / 16;
  int64_t unit, in;
  la_place(blockIdx.x, sub, unit, in);
  const int64_t item = base + unit * sub + in;
  if (item >= items) return;
  const int64_t cols = (p.M + kColumns - 1) / kColumns;
  const int64_t h = item / cols % a.H, slot = item / (cols * a.H);
  const int m0 = static_cast<int>(item % cols) * kColumns, mw = 16 * wave;  // this wave's columns: m0 + mw ..
  const LaSlot z = la_uniform(la_slot(a, slot, p.reverse));
  if constexpr (TAN && Y) {  // every partial sum is written
    if (z.len < 0 && tid == 0) p.dot_sum[item] = 0.0;
  }
  if (z.len < 0 || (!Y && z.last)) return;  // nothing follows the last segment
  const double log_a = a.log_decay[h], log2_a = log_a * 1.4426950408889634;
  const int f = z.step < 0 ? 0 : 1;

  // Elements from row to row; a row's byte offset within a chunk's rows stays below 2^31.
  const uint32_t x_row = uniform(static_cast<uint32_t>(p.x_row)), key_row = uniform(static_cast<uint32_t>(p.key_row)),
                 val_row = uniform(static_cast<uint32_t>(p.val_row)), out_row = uniform(static_cast<uint32_t>(p.out_row));
  const bool reverse = z.step < 0;
  auto start = [&](const void *q, int64_t from) {
    return reinterpret_cast<const uint16_t *>(
        uniform(static_cast<int64_t>(reinterpret_cast<uintptr_t>(static_cast<const uint16_t *>(q) + from))));
  };
  const uint16_t *const x = start(p.x, h / p.x_per * p.x_width), *const key = start(p.key, h / p.key_per * p.key_width),
                 *const val = start(p.val, h / p.val_per * p.val_width + m0);
  const int K = __builtin_amdgcn_readfirstlane(p.K);
  const int wide = __builtin_amdgcn_readfirstlane(p.M - m0 < kColumns ? p.M - m0 : kColumns);  // columns of this workgroup

  // ---- the next chunk's rows.  VEC: from memory into LDS, 16 bytes a lane, a wave's
  // 64 pieces one behind the other there (which piece of the row lands where is the
  // lane's choice of address); else by registers.
  u32x4 px[Y && !VEC ? kRowsK : 1], pk[VEC ? 1 : kRowsK], pv[VEC ? 1 : kRowsV];
  // Row in memory of the chunk's first row there, and byte offset of its token t;
  // behind the last token: outside every buffer.
  auto low_row = [&](int t0, int left) {
    return z.first + (reverse ? -static_cast<int64_t>(t0 + left - 1) : static_cast<int64_t>(t0));
  };
  auto at_row = [&](int t, int left, uint32_t row, uint32_t size) {
    const int i = reverse ? left - 1 - t : t;
    return t < left ? static_cast<uint32_t>(i) * row * size : kOutside;
  };
  // A thread's first piece of a whole chunk of a tensor of PIECES a row; the others are
  // whole steps of rows behind it (where their places in the row are the same).
  auto first_at = [&](uint32_t row, int width, auto pieces, auto place) {
    constexpr int PIECES = decltype(pieces)::value, kStep = kThreads / PIECES;
    const int t = tid / PIECES, n = place(t, tid % PIECES) - t * PIECES * 8;
    const uint32_t at = static_cast<uint32_t>(reverse ? kStep - 1 - t : t) * row * 2;
    return n < width ? at + 2 * n : kOutside;
  };
  // One tensor's rows of a chunk of `left` tokens to LDS address `to`.
  auto fetch = [&](const uint16_t *from, const uint16_t *to, int left, uint32_t first, uint32_t row, int width,
                   auto pieces, auto place) {
    constexpr int PIECES = decltype(pieces)::value, kAll = C * PIECES / kThreads;
    constexpr int kStep = kThreads / PIECES;  // rows from one load of the thread to its next
    const Rows rs(from, 2 * (static_cast<uint32_t>(left - 1) * row + static_cast<uint32_t>(width)));
    const uint32_t at_lds = lds_address(to) + 2 * 64 * wave * 8;
    if (left == C && kStep % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kAll; ++i)
        fetch_lds(rs, at_lds + 2 * kThreads * i * 8, first, static_cast<uint32_t>(kStep * (reverse ? kAll - 1 - i : i)) * row * 2);
    } else {
      const int own = static_cast<int>(hold(static_cast<uint32_t>(tid)));
#pragma unroll
      for (int i = 0; i < kAll; ++i) {
        const int t = own / PIECES + kStep * i, n = place(t, own % PIECES) - t * PIECES * 8;  // the element that belongs there
        fetch_lds(rs, at_lds + 2 * kThreads * i * 8, n < width ? at_row(t, left, row, 2) + 2 * n : kOutside, 0);
      }
    }
  };
  const uint32_t x_first = VEC && Y ? first_at(x_row, K, Number<KP>(), x_at<KP>) : 0,
                 key_first = VEC ? first_at(key_row, K, Number<KP>(), key_at<KP>) : 0,
                 val_first = VEC ? first_at(val_row, wide, Number<VP>(), value_at<VP>) : 0;
  const bool out_f32 = __builtin_amdgcn_readfirstlane(static_cast<int>(p.out_f32)) != 0;
  char *const out = reinterpret_cast<char *>(uniform(static_cast<int64_t>(
      reinterpret_cast<uintptr_t>(static_cast<char *>(p.out) + (out_f32 ? 4 : 2) * (h * p.out_width + m0)))));
  // which: 0 x, 1 keys, 2 values, 3 all.  (They are asked for in three places: a wave's
  // next instruction waits while more of them are issued than the memory pipeline takes.)
  auto load = [&](int t0, int buf, int which) {
    const int left = z.len - t0 < C ? z.len - t0 : C;
    if (left <= 0) return;
    const int64_t low = low_row(t0, left);
    if constexpr (VEC) {
      auto all = [&](int left) {
        if (Y && (which == 0 || which == 3)) fetch(x + low * x_row, s_x + buf * kSizeK, left, x_first, x_row, K, Number<KP>(), x_at<KP>);
        if (which == 1 || which == 3) fetch(key + low * key_row, s_k + buf * kSizeK, left, key_first, key_row, K, Number<KP>(), key_at<KP>);
        if (which == 2 || which == 3) fetch(val + low * val_row, s_v + buf * kSizeV, left, val_first, val_row, wide, Number<VP>(), value_at<VP>);
      };
      if (left == C) all(C);
      else all(left);
    } else if (which == 0 || which == 3) {
      auto rows = [&](const uint16_t *q, uint32_t row, int width) {
        return rows_of(q + low * row, left, row, static_cast<uint32_t>(width));
      };
      const __amdgpu_buffer_rsrc_t rk = rows(key, key_row, K), rv = rows(val, val_row, wide);
      if constexpr (Y) {
        const __amdgpu_buffer_rsrc_t rx = rows(x, x_row, K);
#pragma unroll
        for (int i = 0; i < kRowsK; ++i) {
          const int q = tid + kThreads * i;
          px[i] = load_piece(rx, at_row(q / KP, left, x_row, 2), 8 * (q % KP), K);
        }
      }
#pragma unroll
      for (int i = 0; i < kRowsK; ++i) {
        const int q = tid + kThreads * i;
        pk[i] = load_piece(rk, at_row(q / KP, left, key_row, 2), 8 * (q % KP), K);
      }
#pragma unroll
      for (int i = 0; i < kRowsV; ++i) {
        const int q = tid + kThreads * i;
        pv[i] = load_piece(rv, at_row(q / VP, left, val_row, 2), 8 * (q % VP), wide);
      }
    }
  };
  // What has been asked for is in LDS, as far as this wave is concerned.
  auto stage = [&](int buf) {
    if constexpr (VEC) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    } else {
#pragma unroll
      for (int i = 0; i < kRowsK; ++i) {
        const int q = tid + kThreads * i;
        if constexpr (Y) *reinterpret_cast<u32x4 *>(&s_x[buf * kSizeK + x_at<KP>(q / KP, q % KP)]) = px[i];
        *reinterpret_cast<u32x4 *>(&s_k[buf * kSizeK + key_at<KP>(q / KP, q % KP)]) = pk[i];
      }
#pragma unroll
      for (int i = 0; i < kRowsV; ++i) {
        const int q = tid + kThreads * i;
        *reinterpret_cast<u32x4 *>(&s_v[buf * kSizeV + value_at<VP>(q / VP, q % VP)]) = pv[i];
      }
    }
  };
  load(0, 0, 3);

  // ---- the state that enters the segment: tile 2 kb + u holds n = 32 kb + 8 g + 4 u + e.
  // Offsets within the workgroup's columns are small: 32 bits.
  f32x4 S[2 * KB], U[TAN ? 2 * KB : 1];
  const int64_t state0 = (z.seq * a.H + h) * a.state + static_cast<int64_t>(m0) * p.sm;
  const int Kp = (p.K + 15) / 16 * 16;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  const int mc = mw + r;  // this lane's column of the workgroup's
  const bool col = mc < wide;
#pragma unroll
  for (int j = 0; j < 2 * KB; ++j) {
    S[j] = zero;
    if constexpr (TAN) U[j] = zero;
  }
  if constexpr (Y) {
    if (p.s0 != nullptr && col) {
      const float *from = p.s0 + state0;
      const int sn = static_cast<int>(p.sn), at = mc * static_cast<int>(p.sm) + 8 * g * sn;
      if (fours_of(p, from)) {
#pragma unroll
        for (int j = 0; j < 2 * KB; ++j) {
          const int n = 32 * (j / 2) + 4 * (j % 2);
          if (n + 8 * g < p.K) S[j] = *reinterpret_cast<const f32x4 *>(from + at + n);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2 * KB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = 32 * (j / 2) + 4 * (j % 2) + e;
            if (n + 8 * g < p.K) S[j][e] = from[at + n * sn];
          }
      }
    }
    const LaWhole whole(log_a, a.seg_len);
    const float n_whole = static_cast<float>(a.seg_len);
    for (int64_t b = 0; b < z.before; ++b) {
      const int64_t from = (((z.slot0 + b) * a.H + h) * p.M + m0) * Kp;
      const float *local = p.local + from, *local_tan = TAN ? p.local_tan + from : nullptr;
      const int at = mc * Kp + 8 * g;
#pragma unroll
      for (int j = 0; j < 2 * KB; ++j) {
        const int n = 32 * (j / 2) + 4 * (j % 2);
        const bool there = col && n + 8 * g < Kp;
        const f32x4 own = there ? *reinterpret_cast<const f32x4 *>(local + at + n) : zero;
        if constexpr (TAN) {
          const f32x4 tan = there ? *reinterpret_cast<const f32x4 *>(local_tan + at + n) : zero;
#pragma unroll
          for (int e = 0; e < 4; ++e) U[j][e] = whole(U[j][e]) + fmaf(n_whole, whole(S[j][e]), tan[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][e] = whole(S[j][e]) + own[e];
      }
    }
  }

  // ---- LDS addresses: row r, block kb of x and keys; the transposing reads of the
  // keys' block kb and of this wave's values, tokens 4 g + r / 4
  uint32_t lx[Y ? KB : 1], lk[Y ? KB : 1], lt[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    if constexpr (Y) {
      lx[kb] = hold(lds_address(&s_x[x_at<KP>(r, 4 * kb + g)]));
      lk[kb] = hold(lds_address(&s_k[key_at<KP>(r, 4 * kb + g)]));
    }
    lt[kb] = hold(lds_address(&s_k[key_at<KP>(4 * g + r / 4, 4 * kb + r % 4)]));
  }
  uint32_t lv = hold(lds_address(&s_v[value_at<VP>(4 * g + r / 4, (mw + 4 * (r % 4)) / 8) + 4 * (r % 2)]));
  // shared scores: row t, piece 4 tb + g holds the keys 32 tb + 16 u + 4 g + e
  const uint32_t la[2] = {hold(lds_address(&s_a[SHARE ? C * r + 8 * (g ^ (r % 8)) : 0])),
                          hold(lds_address(&s_a[SHARE ? C * r + 8 * ((4 + g) ^ (r % 8)) : 0]))};

  // ---- weights: of scores (token less key 16 d + r - 4 g - e), of the state's
  // answers (token 16 i + r), of values in the state (tokens 16 j + 4 g + e)
  const float cc = p.c_in * p.c_out;
  auto score_weight = [&](int d, int e) {
    const int n = 16 * d + r - 4 * g - e;
    const float w = cc * power_of(log2_a, n < 0 ? 0 : n);
    return TAN ? w * static_cast<float>(n) : w;
  };
  f32x4 w_score[Y && !SHARE ? 4 : 1], w_val[4];
  float w_out[Y ? 4 : 1];
  if constexpr (Y) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if constexpr (!SHARE)
#pragma unroll
        for (int e = 0; e < 4; ++e) w_score[d][e] = score_weight(d, e);
      w_out[d] = p.c_out * power_of(log2_a, 16 * d + r + f);
    }
  }
  // Shared: this wave's tiles, key block bs of token block bt, two of the ten below
  // the diagonal for the first two waves of eight and one for the others.
  constexpr int kTiles = SHARE ? (10 + W - 1) / W : 1;
  int bt_of[kTiles], bs_of[kTiles];
  f32x4 w_tile[Y && SHARE ? kTiles : 1];
  if constexpr (Y && SHARE) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int n = wave + W * i;
      bt_of[i] = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3;
      bs_of[i] = n - bt_of[i] * (bt_of[i] + 1) / 2;
#pragma unroll
      for (int e = 0; e < 4; ++e) w_tile[i][e] = n < 10 ? score_weight(bt_of[i] - bs_of[i], e) : 0.f;
    }
  }
  // (What the last chunk alone needs is formed from a copy that `hold` hides, or it
  // would be formed before the loop and kept in registers over it.)
  auto weigh = [&](int left) {
    const int g = static_cast<int>(hold(static_cast<uint32_t>(lane))) / 16;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = left - 1 - (16 * j + 4 * g + e);
        w_val[j][e] = d < 0 ? 0.f : p.c_in * power_of(log2_a, d + 1 - f);
      }
  };
  weigh(C);
  float carry = 0.f;
  float n_left = static_cast<float>(C) * power_of(log2_a, C);
  double sum = 0.0;

  // A product of a key and an x tile: weighted, masked, in parts.
  auto split_scores = [&](f32x4 w, const f32x4 &weight, bool diagonal, u32x2 *half) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] *= weight[e];
      w[e] = diagonal && r < 4 * g + e ? 0.f : w[e];
    }
    split_four<kParts>(w, half);
  };
  // The weighted values of token block tb, in three parts.
  auto weighted = [&](const u32x4 &v, int tb, int left, u32x4 *out, bool tan) {
    f32x4 t[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t q = v[2 * u + e / 2];
        t[u][e] = (e % 2 ? high_half(q) : low_half(q)) * w_val[2 * tb + u][e];
        if (tan) t[u][e] *= static_cast<float>(max(left - 1 - (32 * tb + 16 * u + 4 * g + e), 0));
      }
    split_parts<3>(t[0], t[1], out);
  };

  // One chunk from buffer buf.
  auto chunk = [&](int t0, int left, int buf) {
    // ---- this wave's values, transposed: tokens 32 tb + 16 u + 4 g + e of column r
    u32x4 v[2], wv[2][3];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const u32x2 q = lds_transposed(lv + 2 * 8 * VP * (32 * tb + 16 * u));
        v[tb][2 * u] = q[0];
        v[tb][2 * u + 1] = q[1];
      }
    // Those that are not finite are left out of the products; their column's outputs and
    // state are set from their token `bad` on.
    int bad = C;
    bool dirty = false;
    auto check = [&] {
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 top = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, v[i / 4][i % 4] & 0x7fff7fffu));
      dirty = __ballot(top[0] >= 0x7f80 || top[1] >= 0x7f80) != 0;
      if (!dirty) return;
#pragma unroll
      for (int i = 7; i >= 0; --i) {
        uint32_t q = v[i / 4][i % 4];
        const int t = 32 * (i / 4) + 16 * (i % 4 / 2) + 4 * g + 2 * (i % 2);
        if ((q >> 16 & 0x7f80) == 0x7f80) {
          bad = min(bad, t + 1);
          q &= 0xffffu;
        }
        if ((q & 0x7f80) == 0x7f80) {
          bad = min(bad, t);
          q &= 0xffff0000u;
        }
        v[i / 4][i % 4] = q;
      }
      bad = min(bad, __shfl_xor(bad, 16));
      bad = min(bad, __shfl_xor(bad, 32));
    };
    if constexpr (Y && !SHARE) check();
    f32x4 y[Y ? 4 : 1], yu[TAN ? 4 : 1];
    if constexpr (Y) {
      if constexpr (SHARE) {
        // ---- scores, keys 16 bs + 4 g + e of token 16 bt + r, for all waves
#pragma unroll
        for (int i = kTiles - 1; i >= 0; --i) {
          if (wave + W * i >= 10) continue;
          f32x4 w = zero;
          const uint32_t at_k = 2 * 8 * KP * 16 * bs_of[i], at_x = 2 * 8 * KP * 16 * bt_of[i];
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) w = mma(lds_get<u32x4>(lk[kb] + at_k), lds_get<u32x4>(lx[kb] + at_x), w);
          u32x2 half[2];
          split_scores(w, w_tile[i], bt_of[i] == bs_of[i], half);
#pragma unroll
          for (int q = 0; q < 2; ++q)
            lds_put<u32x2>((bs_of[i] >= 2 ? la[1] : la[0]) + 2 * C * C * q + 2 * C * 16 * bt_of[i] + 8 * (bs_of[i] % 2), half[q]);
        }
        load(t0 + C, buf ^ 1, 1);
        // ---- what the state answers, the next block's x on its way
        u32x4 xq[2][4], part[2][2];
        auto read_x = [&](int kb) {
#pragma unroll
          for (int i = 0; i < 4; ++i) xq[kb % 2][i] = lds_get<u32x4>(lx[kb] + 2 * 8 * KP * 16 * i);
        };
        read_x(0);
        split_parts<2>(S[0], S[1], part[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = zero;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          __builtin_amdgcn_sched_barrier(0);
          if (kb + 1 < KB) {
            read_x(kb + 1);
            split_parts<2>(S[2 * kb + 2], S[2 * kb + 3], part[(kb + 1) % 2]);
          }
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = mma(part[kb % 2][q], xq[kb % 2][i], y[i]);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[i][e] *= w_out[i];
        load(t0 + C, buf ^ 1, 2);
        check();
        meet_in_lds();
        // ---- the values under the scores
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
          u32x4 sc[2][4];
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int bt = 2 * tb; bt < 4; ++bt) {
              sc[q][bt] = lds_get<u32x4>(la[tb] + 2 * C * C * q + 2 * C * 16 * bt);
              if (bt == 2 * tb) sc[q][bt][2] = sc[q][bt][3] = 0;  // above the diagonal
            }
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int bt = 2 * tb; bt < 4; ++bt) y[bt] = mma(v[tb], sc[q][bt], y[bt]);
        }
      } else {
        // ---- token block by token block: what the state answers, the scores and the
        // values under them
        load(t0 + C, buf ^ 1, 1);
        u32x4 part[TAN ? 1 : KB][2];
        if constexpr (TAN) {
          // what the state and the tangent answer goes first, a block of 32 of their rows
          // at a time: all blocks' parts would not fit into the registers
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = yu[i] = zero;
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            u32x4 xq[4], ps[kParts], pu[kParts];
#pragma unroll
            for (int i = 0; i < 4; ++i) xq[i] = lds_get<u32x4>(lx[kb] + 2 * 8 * KP * 16 * i);
            split_parts<kParts>(S[2 * kb], S[2 * kb + 1], ps);
            split_parts<kParts>(U[2 * kb], U[2 * kb + 1], pu);
#pragma unroll
            for (int q = 0; q < kParts; ++q)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                y[i] = mma(ps[q], xq[i], y[i]);
                yu[i] = mma(pu[q], xq[i], yu[i]);
              }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[i][e] = fmaf(static_cast<float>(16 * i + r + 1), y[i][e], yu[i][e]) * w_out[i];
        } else {
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) split_parts<2>(S[2 * kb], S[2 * kb + 1], part[kb]);
        }
#pragma unroll
        for (int bt = 0; bt < 4; ++bt) {
          if (bt == 2) load(t0 + C, buf ^ 1, 2);
          u32x4 xq[KB];
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) xq[kb] = lds_get<u32x4>(lx[kb] + 2 * 8 * KP * 16 * bt);
          f32x4 w[4];
#pragma unroll
          for (int bs = 0; bs <= bt; ++bs) {
            w[bs] = zero;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) w[bs] = mma(lds_get<u32x4>(lk[kb] + 2 * 8 * KP * 16 * bs), xq[kb], w[bs]);
          }
          if constexpr (!TAN) {
            y[bt] = zero;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int q = 0; q < 2; ++q) y[bt] = mma(part[kb][q], xq[kb], y[bt]);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[bt][e] *= w_out[bt];
          }
#pragma unroll
          for (int tb = 0; tb <= bt / 2; ++tb) {
            u32x2 half[2][kParts] = {};
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (2 * tb + u <= bt) split_scores(w[2 * tb + u], w_score[SHARE ? 0 : bt - 2 * tb - u], 2 * tb + u == bt, half[u]);
#pragma unroll
            for (int q = 0; q < kParts; ++q)
              y[bt] = mma(v[tb], u32x4{half[0][q][0], half[0][q][1], half[1][q][0], half[1][q][1]}, y[bt]);
          }
        }
      }
    }
    // ---- the state that leaves the chunk, the next keys on their way.  What the chunk adds
    // is summed from zero and joined with the state in one rounding: in products that
    // begin with a large state the matrix cores cut off what lies below it, always
    // towards zero (4096 chunks of positive terms, a memory of 800: states 3.6e-6 off on
    // the average and up to 1.5e-5, now none and 2.2e-6; 2 x 8192 tokens, 64 heads of 128 x
    // 128 407 -> 410 us).
    u32x4 kt[2][2];
    auto read_keys = [&](int i) {  // block kb, transposed: rows n of its two tiles, tokens of block tb
      const int kb = i / 2, tb = i % 2;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const u32x2 q = lds_transposed(lt[kb] + 2 * (8 * KP * (32 * tb + 16 * s) + 4 * u));
          kt[i % 2][u][2 * s] = q[0];
          kt[i % 2][u][2 * s + 1] = q[1];
        }
    };
    read_keys(0);
    u32x4 wu[TAN ? 2 : 1][3];
    f32x4 add[2][2], add_u[2][TAN ? 2 : 1];
    auto join = [&](int kb) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (TAN)
            U[2 * kb + u][e] = fmaf(n_left, S[2 * kb + u][e], fmaf(carry, U[2 * kb + u][e], add_u[kb % 2][u][e]));
          S[2 * kb + u][e] = fmaf(carry, S[2 * kb + u][e], add[kb % 2][u][e]);
        }
    };
#pragma unroll
    for (int i = 0; i < 2 * KB; ++i) {
      const int kb = i / 2, tb = i % 2;
      if (kb == 0) {
        weighted(v[tb], tb, left, wv[tb], false);
        if constexpr (TAN) weighted(v[tb], tb, left, wu[tb], true);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (i + 1 < 2 * KB) read_keys(i + 1);
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          f32x4 &to = add[kb % 2][u];
          to = mma(kt[i % 2][u], wv[tb][q], tb == 0 && q == 0 ? zero : to);
          if constexpr (TAN) {
            f32x4 &to = add_u[kb % 2][u];
            to = mma(kt[i % 2][u], wu[tb][q], tb == 0 && q == 0 ? zero : to);
          }
        }
      if (tb == 0 && kb > 0) join(kb - 1);
    }
    join(KB - 1);
    __builtin_amdgcn_sched_barrier(0);
    if (dirty) {
      if (bad < C) {
#pragma unroll
        for (int j = 0; j < 2 * KB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            S[j][e] = __builtin_nanf("");
            if constexpr (TAN) U[j][e] = __builtin_nanf("");
          }
      }
    }
    // the next chunk's loads, before anything that is stored after them has to be
    // waited for too
    if (t0 + C < z.len) stage(buf ^ 1);
    if constexpr (Y) {
      // ---- out: channels 4 g .. + 3 of token 16 i + r
      if (dirty) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int from = __shfl(bad, 4 * g + e);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * i + r >= from) y[i][e] = __builtin_nanf("");
        }
      }
      const int64_t low = low_row(t0, left);
      const int mo = mw + 4 * g;
      if constexpr (TAN) {
        const uint16_t *dot = static_cast<const uint16_t *>(p.dot) + h / p.val_per * p.val_width + m0;
        const __amdgpu_buffer_rsrc_t rd = rows_of(dot + low * val_row, left, val_row, static_cast<uint32_t>(wide));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = at_row(16 * i + r, left, val_row, 2);
          float d[4], s = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = to_f32(load_one<bf16_t>(rd, mo + e < wide ? at + 2 * (mo + e) : kOutside));
#pragma unroll
          for (int e = 0; e < 4; ++e) s = fmaf(mo + e < wide && 16 * i + r < left ? y[i][e] : 0.f, d[e], s);
          sum += static_cast<double>(s);
        }
      } else {
        auto store = [&](auto element, bool full) {
          constexpr int kSize = decltype(element)::value;  // bytes of it
          const __amdgpu_buffer_rsrc_t ro = buffer_of(
              out + kSize * (low * out_row), kSize * (static_cast<uint32_t>(left - 1) * out_row + static_cast<uint32_t>(wide)));
          const int row0 = static_cast<int>(full ? static_cast<uint32_t>(r) : hold(static_cast<uint32_t>(r)));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t at, more = 0;
            if (!full) {
              at = at_row(16 * i + row0, left, out_row, kSize);
            } else {  // one address a lane, and a step that all share
              at = static_cast<uint32_t>(reverse ? 15 - row0 : row0) * out_row * kSize;
              more = static_cast<uint32_t>(16 * (reverse ? 3 - i : i)) * out_row * kSize;
            }
            if constexpr (VEC && kSize == 4) {
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y[i]), ro,
                                                     static_cast<int>(mo < wide ? at + 4 * mo : kOutside),
                                                     static_cast<int>(more), 0);
            } else if constexpr (VEC) {
              __builtin_amdgcn_raw_buffer_store_b64(
                  u32x2{pack_bf16(y[i][0], y[i][1]), pack_bf16(y[i][2], y[i][3])}, ro,
                  static_cast<int>(mo < wide ? at + 2 * mo : kOutside), static_cast<int>(more), 0);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t to = mo + e < wide ? at + more + kSize * (mo + e) : kOutside;
                if constexpr (kSize == 4) store_one(y[i][e], ro, to);
                else store_one(from_f32<bf16_t>(y[i][e]), ro, to);
              }
            }
          }
        };
        auto sized = [&](bool full) {
          if (out_f32) store(Number<4>(), full);
          else store(Number<2>(), full);
        };
        if (left == C) sized(true);
        else sized(false);
      }
    }
  };

  // The factor of a chunk's decay, a^C = high + low (low no more than half a step of
  // high): high, and a step more or less now and then, so that their product over the
  // chunks so far is the decay's to 2^-24 (one rounded factor again and again drifts
  // off).  owed: what the product lacks, as a part of itself.
  const double decay = exp(log_a * C);
  const float high = uniform(static_cast<float>(decay)), low = uniform(static_cast<float>(decay - high)),
              inverse = uniform(high > 1e-30f ? 1.f / high : 0.f);
  float owed = 0.f;
  if (z.len > 0) stage(0);
  __syncthreads();

  for (int t0 = 0, buf = 0; t0 < z.len; t0 += C, buf ^= 1) {
    const int left = z.len - t0 < C ? z.len - t0 : C;
    load(t0 + C, buf ^ 1, Y ? 0 : 3);
    const float lack = fmaf(high, owed, low);
    carry = high + lack;
    owed = (lack - (carry - high)) * inverse;
    if (left < C) {
      weigh(left);
      carry = la_power(log_a, left);
      n_left = static_cast<float>(left) * carry;
    }
    chunk(t0, left, buf);
    meet_in_lds();
    const uint32_t step = buf ? -kTile : kTile;  // to the other buffer
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if constexpr (Y) {
        lx[kb] += step;
        lk[kb] += step;
      }
      lt[kb] += step;
    }
    lv += buf ? -kTileV : kTileV;
  }

  // ---- the state behind the segment (its offsets are formed anew: those of the one
  // that entered it would be kept in registers over the loop)
  const int g_end = static_cast<int>(hold(static_cast<uint32_t>(g)));
  if (col) {
    if constexpr (!Y) {
      const int64_t to = ((slot * a.H + h) * p.M + m0) * Kp;
      float *local = p.local + to, *local_tan = TAN ? p.local_tan + to : nullptr;
      const int at = mc * Kp + 8 * g_end;
#pragma unroll
      for (int j = 0; j < 2 * KB; ++j) {
        const int n = 32 * (j / 2) + 4 * (j % 2);
        if (n + 8 * g_end < Kp) {
          *reinterpret_cast<f32x4 *>(local + at + n) = S[j];
          if constexpr (TAN) *reinterpret_cast<f32x4 *>(local_tan + at + n) = U[j];
        }
      }
    } else if (z.last) {
      float *to = p.s_last != nullptr ? p.s_last + state0 : nullptr;
      const float *dot = TAN && p.s_dot != nullptr ? p.s_dot + state0 : nullptr;
      const int sn = static_cast<int>(p.sn), at = mc * static_cast<int>(p.sm) + 8 * g_end * sn;
      if (!TAN && to != nullptr && fours_of(p, to)) {
#pragma unroll
        for (int j = 0; j < 2 * KB; ++j) {
          const int n = 32 * (j / 2) + 4 * (j % 2);
          if (n + 8 * g_end < p.K) *reinterpret_cast<f32x4 *>(to + at + n) = S[j];
        }
        return;
      }
#pragma unroll
      for (int j = 0; j < 2 * KB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = 32 * (j / 2) + 4 * (j % 2) + e;
          if (n + 8 * g_end >= p.K) continue;
          if (to != nullptr) to[at + n * sn] = S[j][e];
          if constexpr (TAN)
            if (dot != nullptr) sum += static_cast<double>(U[j][e]) * dot[at + n * sn];
        }
    }
  }
  if constexpr (Y && TAN) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    double *s_sum = reinterpret_cast<double *>(lds);  // the last chunk has been read
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < W; ++i) sum += s_sum[i];
      p.dot_sum[item] = sum;
    }
  }
}

template <int KB, int W, bool SHARE, bool Y, bool TAN, bool VEC>
hipError_t launch_one(const LaArgs &a, const LaPasses &all, int n, hipStream_t s) {
  const int64_t cols = (all.p[0].M + 16 * W - 1) / (16 * W);
  const int64_t sub = la_sub(a, all.p[0].x_per, cols);
  return la_launches(a, cols, sub, n, [&](dim3 grid, int64_t items, int64_t base) {
    la_bf16_kernel<KB, W, SHARE, Y, TAN, VEC><<<grid, 64 * W, 0, s>>>(a, all, items, sub, base);
  });
}
// The segments' own additions where the sequences are cut, by workgroups of four waves
// whatever W is: no scores are shared there, and eight take the same time (2 x 8192 tokens,
// 64 heads of 128 x 128: 391 us against 390).
template <int KB, int W, bool SHARE, bool TAN, bool VEC>
hipError_t launch_kb(const LaArgs &a, const LaPasses &all, int n, hipStream_t s) {
  const hipError_t e = la_cut(a) ? launch_one<KB, 4, false, false, TAN, VEC>(a, all, n, s) : hipSuccess;
  return e != hipSuccess ? e : launch_one<KB, W, SHARE, true, TAN, VEC>(a, all, n, s);
}

// 16-byte pieces of every row, head and output
bool pieces(const LaPass &p) {
  for (const void *q : {p.x, p.key, p.val, static_cast<const void *>(p.out)})
    if (reinterpret_cast<uintptr_t>(q) % 16 != 0) return false;
  for (int64_t n : {p.x_row, p.key_row, p.val_row, p.x_width, p.key_width, p.val_width, p.out_row, p.out_width,
                    static_cast<int64_t>(p.K), static_cast<int64_t>(p.M)})
    if (n % 8 != 0) return false;
  return true;
}

template <bool TAN, bool VEC>
hipError_t launch_vec(const LaArgs &a, const LaPasses &all, int n, hipStream_t s) {
  const int64_t K = all.p[0].K, M = all.p[0].M;
  if constexpr (TAN) {
    if (K <= 64) return launch_kb<2, 4, false, TAN, VEC>(a, all, n, s);
    if (K <= 128) return launch_kb<4, 4, false, TAN, VEC>(a, all, n, s);
  } else if (M <= 64) {
    if (K <= 64) return launch_kb<2, 4, false, TAN, VEC>(a, all, n, s);
    if (K <= 128) return launch_kb<4, 4, false, TAN, VEC>(a, all, n, s);
  } else {
    if (K <= 64) return launch_kb<2, 8, true, TAN, VEC>(a, all, n, s);
    if (K <= 128) return launch_kb<4, 8, true, TAN, VEC>(a, all, n, s);
  }
  return launch_kb<8, 4, false, TAN, VEC>(a, all, n, s);
}

}  // namespace

hipError_t launch_la_bf16(const LaArgs &a, const LaPass *p, int n, hipStream_t s) {
  LaPasses all{};
  bool vec = true;
  for (int i = 0; i < n; ++i) {
    all.p[i] = p[i];
    vec = vec && pieces(p[i]);
  }
  if (p[0].dot_sum != nullptr) return vec ? launch_vec<true, true>(a, all, n, s) : launch_vec<true, false>(a, all, n, s);
  return vec ? launch_vec<false, true>(a, all, n, s) : launch_vec<false, false>(a, all, n, s);
}

}  // namespace ssm
