// What the kernels that write and read paged caches share: the rotation's
// angles, the place of a packed row, and the scales of a cache in 4 bits' scores
// and weights.
#pragma once

#include <climits>
#include <cstdint>

#include "kernels.h"

namespace sdpa {

// freq / 2 pi as the sum of three floats, good to 2^-70 of itself.
struct Turns {
  float hi, mid, low;
};
__device__ __forceinline__ Turns turns_of(float freq) {
  // 1 / (2 pi) = 0.15915494309189533576888376..., rounded to fp32, then what that left, twice
  constexpr float kInvTwoPi0 = 0x1.45f306p-3f, kInvTwoPi1 = 0x1.b9391p-28f, kInvTwoPi2 = 0x1.529fc2p-54f;
  const float th = freq * kInvTwoPi0, e0 = fmaf(freq, kInvTwoPi0, -th);
  const float p1 = freq * kInvTwoPi1, e1 = fmaf(freq, kInvTwoPi1, -p1);
  const float tm = e0 + p1, back = tm - e0;
  return {th, tm, (e0 - (tm - back)) + (p1 - back) + fmaf(freq, kInvTwoPi2, e1)};
}

// cos and sin of pos * freq.  The angle in turns is formed from products whose
// rounding errors are kept (fma): the position in two parts of at most 19 bits,
// freq / 2 pi as a sum of three floats, good to 2^-70 of itself.  Whole turns are
// dropped after each sum of two parts of at most half a turn, which rounds off by
// 2^-25 at most; there are six such sums and a last one, so that the fraction is good
// to 7 2^-25 = 2.1e-7 of a turn, 1.3e-6 rad, while the angle is below 2^48.  (Against
// exact arithmetic, 300000 angles of positions up to 2^30 and frequencies up to 1e5
// were off by 4.6e-7 rad at most.)
__device__ __forceinline__ float2 cos_sin(int pos, float freq) {
  const Turns f = turns_of(freq);
  const float th = f.hi, tm = f.mid, tl = f.low;
  float t = 0.f, rest = 0.f;
  auto add = [&](float part) {
    const float x = t + (part - rintf(part));
    t = x - rintf(x);
  };
  auto add_product = [&](float x) {
    const float a = x * th, b = x * tm;
    add(a);
    add(fmaf(x, th, -a));
    add(b);
    rest += fmaf(x, tl, fmaf(x, tm, -b));
  };
  add_product(static_cast<float>(pos >> 12) * 4096.f);
  add_product(static_cast<float>(pos & 4095));
  add(rest);
  float2 r;
  sincospif(2.f * t, &r.y, &r.x);
  return r;
}

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Sequence of packed row t: the last s with q_starts[s] <= t, found by a warp
// with 32 probes a round.  Returns -1 for a row outside every sequence.
template <class Params>
__device__ __forceinline__ int find_seq(const Params& p, int t, int lane) {
  int lo = 0, hi = p.b + 1;                                   // q_starts[0 .. b]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int probe = lo + lane * step;
    const bool le = probe < hi && p.q_starts[probe] <= t;
    const uint32_t votes = __ballot_sync(0xffffffffu, le);
    if (votes == 0) return -1;                                // before the first sequence
    lo += (31 - __clz(votes)) * step;
    hi = min(hi, lo + step);
  }
  return lo < p.b ? lo : -1;
}

// Where packed row t lies: its position (INT_MIN: no sequence's row) and the
// page row of its first head, page * h_kv * P + position % P (-1: none; a page
// number outside the cache is reported).
struct RowPlace {
  int pos;
  long long row;
};
template <class Params>
__device__ __forceinline__ RowPlace place_in_seq(const Params& p, int t, int s, bool report) {
  RowPlace r{INT_MIN, -1};
  const int end = s >= 0 ? min(p.q_starts[s + 1], p.n_tokens) : 0;
  if (t >= end) return r;
  const int len = min(max(p.kv_lengths[s], 0), p.pages_per_seq << p.page_shift);
  r.pos = len - end + t;
  if (r.pos < 0) return r;
  const int page = p.page_table[static_cast<long long>(s) * p.pages_per_seq + (r.pos >> p.page_shift)];
  if (page >= 0 && page < p.n_pages)
    r.row = (static_cast<long long>(page) * p.h_kv << p.page_shift) + (r.pos & ((1 << p.page_shift) - 1));
  else if (report)
    atomicOr(p.status, kStatusBadPage);
  return r;
}
// One warp, every lane: one row's.
template <class Params>
__device__ __forceinline__ RowPlace place_of_row(const Params& p, int t, int lane) {
  return place_in_seq(p, t, find_seq(p, t, lane), lane == 0);
}
// One warp, t0 + lane's for each of the first `rows` lanes.  (A warp for each row in
// turn would wait four times for memory for each.)
template <class Params>
__device__ __forceinline__ RowPlace place_of_rows(const Params& p, int t0, int rows, int lane) {
  const int t = t0 + min(lane, rows - 1);
  int s = find_seq(p, t0, lane);
  const int last = find_seq(p, t0 + rows - 1, lane);
  if (s != last || s < 0) {
    int lo = 0, hi = p.b + 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.q_starts[mid] <= t) lo = mid;
      else hi = mid;
    }
    s = lo < p.b && p.q_starts[lo] <= t ? lo : -1;
  }
  return place_in_seq(p, t, s, lane < rows);
}

// The softmax weights of a cache in 4 bits enter the products as fp16, relative to what a
// row's largest scaled score was, times 2^kWeightUp: half a step is at most 2^-11 of a
// weight, and 2^-30 of the largest for those below 2^-19 of it.  (Times 1 it was 2^-25: one
// strong key made the weaker ones at 2^-25 of its weight drop out of O, but not out of the
// sum l, however many they were.)  bf16, of which half a step is up to 2^-8, would cost as
// much as the result's own rounding.
// What is kept and published is the reference itself, the largest score less kWeightUp: for
// scores from 2^24 on that is rounded, and weights of two references can be added all the
// same.  It moves when a score is more than kWeightMost above it.  For scores below 2^27 the
// sum and the difference are off by at most 3, and a score that is the difference of a fused
// product by half its step, 4: weights stay below fp16's 2^16.
// (So a reference lags by up to 6.  By 8, 6 and 4: 4 chunks of 512 tokens behind 7680
// positions 132.4, 132.2 and 134.6 us, with queries three times as large 143, 146 and 147, as
// it moves more often.)
constexpr float kWeightUp = 5.f, kWeightMost = 11.f;   // log2

// What turns a score of a cache in 4 bits, of a row that was scaled by 2^up, into log2
// units: score_scale 2^(score_exp - up).  The exponents are added before anything is
// multiplied: up goes from -114 to 120, k_exp from -32 to 32 and the scale over all
// floats, so that products of two of them may leave the range that the three's is in.
// Below 2^-126 all weights are one (scores are below 2^34), and a factor of zero would
// make a masked score of -infinity a NaN; up to 2^91 its products with scores are finite.
__device__ __forceinline__ float score_factor(const Paged4Params& p, int up) {
  return p.score_scale * __uint_as_float(static_cast<uint32_t>(127 + min(max(p.score_exp - up, -126), 90)) << 23);
}

}  // namespace sdpa
