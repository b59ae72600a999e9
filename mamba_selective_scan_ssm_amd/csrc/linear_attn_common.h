// Device helpers shared by the chunked kernels of linear attention.
#pragma once

#include "gdr_mfma.h"
#include "linear_attn.h"

namespace ssm {

// Sequence and tokens of a slot.  Tokens are counted in the order in which the
// pass takes them: local token i of the slot is token first + i * step.
struct LaSlot {
  int64_t seq, first, step;
  int64_t before;   // segments of the sequence before this one
  int64_t slot0;    // the sequence's first slot
  int32_t len;      // tokens of the segment; -1: there is no such segment
  bool last;        // of its sequence
};
__device__ __forceinline__ void la_bounds(const LaArgs &a, int64_t s, int64_t &c0, int64_t &c1) {
  if (a.cu == nullptr) {
    c0 = s * a.L;
    c1 = c0 + a.L;
    return;
  }
  // whatever cu holds, tokens stay inside
  c0 = a.cu[s];
  c1 = a.cu[s + 1];
  c0 = c0 < 0 ? 0 : c0 > a.T ? a.T : c0;
  c1 = c1 < c0 ? c0 : c1 > a.T ? a.T : c1;
}
__device__ __forceinline__ LaSlot la_slot(const LaArgs &a, int64_t slot, bool reverse) {
  LaSlot r;
  const int64_t per = a.cu == nullptr ? a.slots / a.S : 0;
  if (a.slots == a.S) {
    r.seq = r.slot0 = slot;
  } else if (a.cu == nullptr) {
    r.seq = slot / per;
    r.slot0 = r.seq * per;
  } else {  // the last sequence whose slots begin at or before this one
    int64_t lo = 0, hi = a.S - 1;
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) / 2;
      int64_t c0, c1;
      la_bounds(a, mid, c0, c1);
      if (c0 / a.seg_len + mid <= slot) lo = mid;
      else hi = mid - 1;
    }
    int64_t c0, c1;
    la_bounds(a, lo, c0, c1);
    r.seq = lo;
    r.slot0 = c0 / a.seg_len + lo;
  }
  int64_t c0, c1;
  la_bounds(a, r.seq, c0, c1);
  r.before = slot - r.slot0;
  int64_t from = r.before * a.seg_len, to = from + a.seg_len;
  const int64_t len = c1 - c0;
  r.last = to >= len;
  if (r.last) to = len;
  r.len = r.before < 0 || (r.before > 0 && from >= len) ? -1 : static_cast<int32_t>(to - from);
  r.step = reverse ? -1 : 1;
  r.first = reverse ? c1 - 1 - from : c0 + from;
  return r;
}

// a^n S as m S + one S: with m = a^n - 1 where that is small, so that what is
// rounded is the change and a state that lasts long is not scaled by one rounded
// factor again and again (each time off by up to 2^-25 in the same direction).
struct LaCarry {
  float m, one;
  __device__ __forceinline__ LaCarry(double log_a, int64_t n) {
    const double e = log_a * static_cast<double>(n);
    const bool near = e > -0.6931 && e < 0.6931;
    m = n == 0 ? 0.f : static_cast<float>(near ? expm1(e) : exp(e));
    one = n == 0 || near ? 1.f : 0.f;
  }
  __device__ __forceinline__ float operator()(float s) const { return fmaf(s, m, s * one); }
  // and what is added to it: the change first, then one sum
  __device__ __forceinline__ float operator()(float s, float more) const { return fmaf(s, m, more) + s * one; }
};
// The same over a whole segment, thousands of tokens it may be: there the power of a decay
// above 1 passes fp32 where the state, zero or small, and the result do not, and is taken in
// two halves.
struct LaWhole {
  LaCarry first;
  float again;
  __device__ __forceinline__ LaWhole(double log_a, int64_t n) : first(log_a, n), again(1.f) {
    const double e = log_a * static_cast<double>(n);
    if (e > 88.0) {
      again = static_cast<float>(fmin(exp(0.5 * e), 3e38));
      first.m = again;
    }
  }
  __device__ __forceinline__ float operator()(float s) const { return first(s) * again; }
};
// a^n, 1 for n = 0 whatever a
__device__ __forceinline__ float la_power(double log_a, int64_t n) {
  return n == 0 ? 1.f : static_cast<float>(exp(log_a * static_cast<double>(n)));
}

// Unit (sequence's segment, group of heads) and the workgroup's place in it: the
// workgroups of a unit read the same keys, so they are 8 numbers apart, on one of
// the 8 XCDs and its L2, one after the other.
__device__ __forceinline__ void la_place(int64_t id, int64_t sub, int64_t &unit, int64_t &in) {
  unit = id / (8 * sub) * 8 + id % 8;
  in = id / 8 % sub;
}
// Workgroups of a unit: those of a group's heads, or of a head, or one alone, where
// there would be too few units for the XCDs.
inline int64_t la_sub(const LaArgs &a, int64_t per, int64_t cols) {
  const int64_t heads = a.slots * a.H;
  return heads / per >= 64 ? per * cols : heads >= 64 ? cols : 1;
}
// One or two passes over all workgroups of `cols` columns each, in grids below 2^32 threads.
struct LaPasses {
  LaPass p[2];
};
template <typename F>
hipError_t la_launches(const LaArgs &a, int64_t cols, int64_t sub, int n, F &&launch) {
  // at most 65535 heads, of 2^24 channels together: sub stays below 2^18 + 2^16
  const int64_t items = a.slots * a.H * cols, most = (int64_t{1} << 22) / (8 * sub) * (8 * sub);
  for (int64_t base = 0; base < items; base += most) {
    const int64_t now = items - base < most ? items - base : most, units = (now + sub - 1) / sub;
    launch(dim3(static_cast<unsigned>((units + 7) / 8 * 8 * sub), static_cast<unsigned>(n)), items, base);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace ssm
