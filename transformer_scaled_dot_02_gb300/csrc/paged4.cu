// A paged cache held in 4 bits: the append that fills it and the reading back.
//
// A row of d keys or values is held in blocks of 16 columns.  With u = 2^exp
// (a whole number the cache is kept with), a block x_0 .. x_15 is
//   s   = e4m3(max_i |x_i| / (6 u))     nearest, ties to even, at most 448
//   c_i = e2m1(x_i / (s u))             nearest, ties to even, at most 6; 0 where s = 0
// and stands for c_i s u: 4.5 bits a value, 6 the largest e2m1 number.  Codes
// have 2 significant bits and scales 4, so what a block stands for is exact in
// bf16.  A power of two as the unit moves the scales' range (2^-9 .. 448) to
// where the cache's values are and rounds nothing.
//
// A page of one key-value head has its rows' codes first (columns 2 i and
// 2 i + 1 in the low and the high half of byte i) and then their scales, both
// row by row: a run of rows is two runs of bytes, each aligned to 16.
#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace sdpa {
namespace {

constexpr int kThreads = 256;
constexpr int kReadTokens = 32;                               // of a block of the reading back

// Two floats as e2m1, `lo` in the low four bits.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint16_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u16.u8 %0, t;\n\t}"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}
// An e2m1 number.
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "r"(code));
  float f;
  asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(r));
  return f;
}
// Eight floats as e2m1, the first in the low four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {        // within an ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two floats as e4m3, `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// An e4m3 number (not NaN).
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(byte)));
  float f;
  asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(r));
  return f;
}

// -------------------------------------------------------------------- append
// Rotates the new queries and keys by their positions and stores keys and
// values in 4 bits: keys are quantised from the rotation itself, not from its
// rounding to bf16.
//
// It reads (h + 2 h_kv) d bf16 a token and writes h d bf16 and 9/16 h_kv d
// bytes.  An item is 16 columns of a head: of a query the two chunks of 8 whose
// columns pair up, of a key or value a block (the rotation reads its partners'
// columns beside it).  Blocks take kTokens tokens: their angles once, into shared
// memory, then every head of theirs.  16384 tokens (16 query heads, 4 of keys, d =
// 128, all columns rotated): 45 us, 4 TB/s.  10 of them are the rotation and the
// quantising (38 us where the queries were only copied, 35 where nothing was rotated or
// quantised; issue slots are 70 % busy).  What keeps those 35 above the bytes' 26 is not
// known; the next item's loads ahead of this one's work did not help.  For a few tokens the
// launch and three dependent reads: 2.9 us for 8.
//
// The rotation is in fp32 with angles good to 1.3e-6.  Where that leaves open
// which scale or code is the nearest, some element of a block lies within kSlack
// of a border between two (one block in 970 of normal numbers): the block is worked out
// again in 48 bits, so that the cache holds what the definition says.
// Of |a| + |b|: the angle, cos and sin's own rounding, and three roundings of products and sum,
// the sum or difference with it.
constexpr float kSlack = 2e-6f;

// A number as the sum of two floats, lo at most half a unit in hi's last place: 48
// bits in Dekker's and Knuth's exact sums and products.  (The card has few 64-bit units:
// with them a block in doubt took half as long again.)
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two quick_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fadd_rn(b, -__fadd_rn(s, -a))};
}
__device__ __forceinline__ Two exact_sum(float a, float b) {
  const float s = __fadd_rn(a, b), z = __fadd_rn(s, -a);
  return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -z)), __fadd_rn(b, -z))};
}
__device__ __forceinline__ Two exact_product(float a, float b) {
  const float x = __fmul_rn(a, b);
  return {x, fmaf(a, b, -x)};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  const Two s = exact_sum(a.hi, b.hi);
  return quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  const Two x = exact_product(a.hi, b.hi);
  return quick_sum(x.hi, __fadd_rn(x.lo, fmaf(a.hi, b.lo, __fmul_rn(a.lo, b.hi))));
}

// cos and sin of pos * freq, good to 2^-40 while the angle is below 2^30: the angle in
// turns as in cos_sin, with what its sums round off kept, less the nearest quarter,
// then Taylor's series up to an eighth of a turn.
__device__ __forceinline__ void cos_sin_in_48_bits(int pos, float freq, Two* cosine, Two* sine) {
  const Turns f = turns_of(freq);
  Two t{0.f, 0.f};
  auto add = [&](float part) {
    const Two x = exact_sum(t.hi, __fadd_rn(part, -rintf(part)));
    t = {x.hi, __fadd_rn(x.lo, t.lo)};
  };
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const float x = i == 0 ? static_cast<float>(pos >> 12) * 4096.f : static_cast<float>(pos & 4095);
    const Two a = exact_product(x, f.hi), b = exact_product(x, f.mid);
    add(a.hi);
    add(a.lo);
    add(b.hi);
    add(fmaf(x, f.low, b.lo));
  }
  t = quick_sum(t.hi, t.lo);
  const float k = rintf(4.f * t.hi);
  t = exact_sum(fmaf(k, -0.25f, t.hi), t.lo);
  t = t * Two{0x1.921fb6p+2f, -0x1.777a5cp-23f};              // 2 pi
  const Two z = t * t;
  // what of the series is below 2^-15 in one float
  const float s9 = fmaf(z.hi, fmaf(z.hi, 1.f / 6227020800.f, -1.f / 39916800.f), 1.f / 362880.f);
  const float c8 = fmaf(z.hi, fmaf(z.hi, fmaf(z.hi, -1.f / 87178291200.f, 1.f / 479001600.f), -1.f / 3628800.f), 1.f / 40320.f);
  // 1 / n! as two floats
  Two s = Two{s9, 0.f} * z + Two{-0x1.a01a02p-13f, 0x1.7f97fap-39f}; // -1 / 7!
  s = s * z + Two{0x1.111112p-7f, -0x1.dddddep-32f};          // 1 / 5!
  s = s * z + Two{-0x1.555556p-3f, 0x1.555556p-28f};          // -1 / 3!
  s = s * z * t + t;
  Two c = Two{c8, 0.f} * z + Two{-0x1.6c16c2p-10f, 0x1.27d27ep-35f}; // -1 / 6!
  c = c * z + Two{0x1.555556p-5f, -0x1.555556p-30f};          // 1 / 4!
  c = c * z + Two{-0.5f, 0.f};
  c = c * z + Two{1.f, 0.f};
  const int quarter = static_cast<int>(k) & 3;
  auto negated = [](Two x, bool negate) { return negate ? Two{-x.hi, -x.lo} : x; };
  *cosine = negated(quarter & 1 ? s : c, quarter == 1 || quarter == 2);
  *sine = negated(quarter & 1 ? c : s, quarter >= 2);
}

// Columns col .. col + 15 of key row `row` at position pos, in 48 bits, by all
// lanes of a warp: a lane for each column (one lane for the 16 took 30 us, ten times a
// short call).  Of the two scales or codes that 32 bits leave open the border between
// them decides, which is a float.
__device__ __noinline__ void block_in_48_bits(const Paged4AppendParams& p, const uint16_t* row, int col, int pos,
                                              int lane, uint2* codes, uint32_t* scale) {
  constexpr float kDown = 1.f - 0x1p-21f, kUp = 1.f + 0x1p-21f;
  const int half = p.d_rot / 2;
  auto value = [&](int x) { return __uint_as_float(static_cast<uint32_t>(row[x]) << 16); };
  auto more = [](Two a, Two b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); };
  const int i = lane & 15, x = col + i;
  const int pair = p.interleaved ? x / 2 : (x < half ? x : x - half);
  const bool second = p.interleaved ? (x & 1) : x >= half;
  const float own = value(x);
  float other = value(p.interleaved ? x ^ 1 : (second ? x - half : x + half));
  if (!second) other = -other;
  Two cs, sn;
  cos_sin_in_48_bits(pos, p.freqs[pair], &cs, &sn);
  const float plain = own * cs.hi + other * sn.hi;
  Two y{plain, 0.f};
  if (fabsf(plain) < INFINITY) {
    const Two a = exact_product(own, cs.hi), b = exact_product(other, sn.hi);
    y = Two{a.hi, fmaf(own, cs.lo, a.lo)} + Two{b.hi, fmaf(other, sn.lo, b.lo)};
  }
  y = {y.hi * p.k_unit, y.lo * p.k_unit};
  const bool negative = y.hi < 0.f;
  if (negative) y = {-y.hi, -y.lo};
  Two top = y.hi == y.hi ? y : Two{0.f, 0.f};
#pragma unroll
  for (int z = 8; z > 0; z >>= 1) {
    const Two o{__shfl_xor_sync(0xffffffffu, top.hi, z), __shfl_xor_sync(0xffffffffu, top.lo, z)};
    if (more(o, top)) top = o;
  }
  const float sixth = top.hi * (1.f / 6.f);
  const uint32_t s2 = e4m3x2(sixth * kDown, sixth * kUp);
  uint32_t s8 = s2 & 0xff;
  if (s8 != s2 >> 8) {
    const Two border{3.f * (e4m3_value(s8) + e4m3_value(s2 >> 8)), 0.f};
    if (more(top, border) || (!more(border, top) && (s8 & 1))) s8 = s2 >> 8;
  }
  const float s = e4m3_value(s8);
  // (a NaN has the largest code)
  const float a = fminf(y.hi * (s > 0.f ? rcp_approx(s) : 0.f), 8.f);
  const uint32_t c2 = e2m1x2(a * kDown, a * kUp);
  uint32_t c = c2 & 7u;
  if (c != c2 >> 4) {
    const Two border{0.5f * (e2m1_value(c) + e2m1_value(c2 >> 4)) * s, 0.f};
    if (more(y, border) || (!more(border, y) && (c & 1))) c = c2 >> 4;
  }
  c = (c | (negative ? 8u : 0u)) << (4 * (i & 7));
#pragma unroll
  for (int z = 1; z < 8; z <<= 1) c |= __shfl_xor_sync(0xffffffffu, c, z);
  *codes = make_uint2(__shfl_sync(0xffffffffu, c, 0), __shfl_sync(0xffffffffu, c, 8));
  *scale = s8;
}

// The codes and scale of y[16] (in units), which is off by at most `off` where
// kOff; false where that leaves one open.
template <bool kOff>
__device__ __forceinline__ bool quantise(const float (&y)[16], float off, uint2* codes, uint32_t* scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) top = fmax3(top, fabsf(y[i]), fabsf(y[i + 1]));
  uint32_t s8, open = 0;
  if constexpr (kOff) {
    s8 = e4m3x2((top + off) * 0x1.555558p-3f, (top - off) * 0x1.555552p-3f);   // 1/6 from above and below
    open = (s8 & 0xff) ^ (s8 >> 8);
  } else {
    // A bf16 number may be 6 times a border between two scales, but otherwise lies 2^-9 of
    // itself or more beside it, as both have at most 8 bits: the product with 1/6 (off by
    // 2^-23) is rounded to 13 bits.
    const uint32_t sixth = __float_as_uint(top * 0x1.555556p-3f);
    s8 = e4m3x2(__uint_as_float((sixth + 0x400u) & ~0x7ffu), 0.f);
  }
  s8 &= 0xff;
  const float s = e4m3_value(s8);
  const float inv = s > 0.f ? rcp_approx(s) : 0.f;
  auto near = [&](float* to, const float* from, float by) {
    const float2 v = __ffma2_rn(make_float2(from[0], from[1]), make_float2(inv, inv), make_float2(by, by));
    to[0] = v.x;
    to[1] = v.y;
  };
  uint32_t w[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float a[8];
    if constexpr (kOff) {
      const float d = fmaf(off, inv * 1.000001f, 2e-6f);     // (and what 1 / s and the products are off by)
#pragma unroll
      for (int i = 0; i < 8; i += 2) near(a + i, y + 8 * x + i, d);
      w[x] = e2m1x8(a);
#pragma unroll
      for (int i = 0; i < 8; i += 2) near(a + i, y + 8 * x + i, -d);
      open |= (w[x] ^ e2m1x8(a)) & 0x77777777u;              // (a zero's sign is nothing)
    } else {
      // Bf16 numbers may lie on a border itself, but none other lies nearer than 2^-10
      // to one: the product with 1 / s (off by 2^-20) is rounded to whole 2^-12.
      constexpr float kSnap = 0x1.8p11f;
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = __fadd_rn(fmaf(y[8 * x + i], inv, kSnap), -kSnap);
      w[x] = e2m1x8(a);
    }
  }
  *codes = make_uint2(w[0], w[1]);
  *scale = s8;
  return open == 0;
}

template <int kTokens, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) sdpa_paged4_append_kernel(const __grid_constant__ Paged4AppendParams p) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps % kTokens == 0, "a warp finds each token's place");
  // [kTokens][4][d_rot / 16]: (cos, cos, sin, sin) of two pairs, those of 8 pairs apart so that
  // lanes that read 16 bytes of neighbouring eights do not meet in a bank
  extern __shared__ __align__(16) float2 angles[];
  __shared__ long long row_of[kTokens];                       // page row of the token, head 0 (-1: not stored)
  __shared__ int pos_of[kTokens];                             // position (INT_MIN: no sequence's token)
  __shared__ uint8_t turned[kTokens][16];                     // of each eight pairs: some angle is not zero
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = static_cast<int>(blockIdx.x) * kTokens;
  const int half = p.d_rot / 2;
  const int heads = p.h + 2 * p.h_kv, warp_heads = 32 >> p.log_blocks;   // that a warp takes at a time
  const int tokens = min(kTokens, p.n_tokens - t0);
  const int page_rows_mask = (1 << p.page_shift) - 1;
  const int c = lane & ((1 << p.log_blocks) - 1);             // item of the head, in every head
  const bool rotates = c < p.d_rot / 16;
  const bool apart = rotates && !p.interleaved;
  const int q0 = apart ? c * 8 : c * 16, q1 = apart ? q0 + half : q0 + 8;   // columns of a query's chunks
  // a key's column x of a chunk of 8 pairs up with column x + partner
  auto partner = [&](int x) { return x < half ? half : -half; };
  auto source = [&](int token, int head) -> const uint16_t* {
    const long long t = t0 + token;
    if (head < p.h) return p.q == nullptr ? nullptr : p.q + t * p.q_stride + head * p.d;
    const int hk = head - p.h;
    return hk < p.h_kv ? p.k + t * p.k_stride + hk * p.d : p.v + t * p.v_stride + (hk - p.h_kv) * p.d;
  };
  uint4 a, b, pa, pb;
  auto load = [&](int token, int head) {
    if (head >= heads || token >= tokens) return;
    const uint16_t* src = source(token, head);
    if (src == nullptr) return;
    if (head < p.h) {
      a = *reinterpret_cast<const uint4*>(src + q0);
      b = *reinterpret_cast<const uint4*>(src + q1);
      return;
    }
    a = *reinterpret_cast<const uint4*>(src + c * 16);
    b = *reinterpret_cast<const uint4*>(src + c * 16 + 8);
    if (apart && head < p.h + p.h_kv) {
      pa = *reinterpret_cast<const uint4*>(src + c * 16 + partner(c * 16));
      pb = *reinterpret_cast<const uint4*>(src + c * 16 + 8 + partner(c * 16 + 8));
    }
  };
  // A warp takes warp_heads heads of a token, then the ones kWarps times as many further on.
  int token = 0, head0 = warp * warp_heads;
  auto carry = [&]() {
    for (; head0 >= heads && token < tokens; ++token) head0 -= (heads + warp_heads - 1) & -warp_heads;
  };
  carry();
  griddep_launch_dependents();
  griddep_wait();
  load(token, head0 + (lane >> p.log_blocks));
  if (warp < tokens) {
    const RowPlace at = place_of_row(p, t0 + warp, lane);
    if (lane == 0) {
      row_of[warp] = at.row;
      pos_of[warp] = at.pos;
    }
  }
  __syncthreads();
  {
    const int mine = warp % kTokens;                          // token
    if (mine < tokens && pos_of[mine] != INT_MIN)
      for (int i0 = warp / kTokens * 32; i0 < half; i0 += kWarps / kTokens * 32) {
        const int i = i0 + lane;
        bool turns_here = false;
        if (i < half) {
          const float freq = p.freqs[i];
          const float2 r = cos_sin(pos_of[mine], freq);
          turns_here = pos_of[mine] != 0 && freq != 0.f;     // (a sine may be rounded to zero)
          float* at = reinterpret_cast<float*>(angles + mine * half + (i >> 1 & 3) * (half >> 2) + (i >> 3) * 2) + (i & 1);
          at[0] = r.x;
          at[2] = r.y;
        }
        const uint32_t turns = __ballot_sync(0xffffffffu, turns_here);
        if ((lane & 7) == 0 && i < half) turned[mine][i >> 3] = (turns >> lane & 0xff) != 0;
      }
  }
  __syncthreads();
  // stores a key's or value's block
  auto store = [&](int token, int head, int c, uint2 codes, uint32_t scale) {
    // row_of: page h_kv P + r for page row r of head 0
    const long long row = row_of[token];
    const long long r = row & page_rows_mask;
    const int hk = head - p.h;
    const bool is_k = hk < p.h_kv;
    uint8_t* page = (is_k ? p.k_pages : p.v_pages) +
                    ((row >> p.page_shift) + (is_k ? hk : hk - p.h_kv)) * (static_cast<long long>(9 * p.d / 16) << p.page_shift);
    *reinterpret_cast<uint2*>(page + r * (p.d / 2) + c * 8) = codes;
    page[(static_cast<long long>(p.d / 2) << p.page_shift) + (r << p.log_blocks) + c] = static_cast<uint8_t>(scale);
  };
  // Does this lane's item of a head; true: its block has to be worked out in 48 bits.
  auto work = [&](int token, int head) -> bool {
    if (head >= heads || pos_of[token] == INT_MIN) return false;
    // of pairs 8 c + 2 e and 8 c + 2 e + 1: cos, cos, sin, sin
    auto turn = [&](int c, int e) { return reinterpret_cast<const float4*>(angles + token * half)[e * (half >> 3) + c]; };
    const uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ub[4] = {b.x, b.y, b.z, b.w};
    if (head < p.h) {
      if (p.q == nullptr) return false;
      uint16_t* dst = p.q_out + (static_cast<long long>(t0 + token) * p.h + head) * p.d;
      uint32_t ra[4], rb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ra[e] = ua[e];
        rb[e] = ub[e];
        if (!rotates) continue;
        const float2 x0 = unpack_bf16x2(ua[e]), x1 = unpack_bf16x2(ub[e]);
        if (p.interleaved) {
          const float4 r01 = turn(c, e / 2), r45 = turn(c, 2 + e / 2);
          const float2 r0 = e % 2 ? make_float2(r01.y, r01.w) : make_float2(r01.x, r01.z);
          const float2 r1 = e % 2 ? make_float2(r45.y, r45.w) : make_float2(r45.x, r45.z);
          ra[e] = pack_bf16x2(x0.x * r0.x - x0.y * r0.y, x0.y * r0.x + x0.x * r0.y);
          rb[e] = pack_bf16x2(x1.x * r1.x - x1.y * r1.y, x1.y * r1.x + x1.x * r1.y);
        } else {
          const float4 r = turn(c, e);
          const float2 cs = make_float2(r.x, r.y), sn = make_float2(r.z, r.w);
          const float2 p0 = __fmul2_rn(x1, sn), p1 = __fmul2_rn(x0, sn);
          const float2 y0 = __ffma2_rn(x0, cs, make_float2(-p0.x, -p0.y)), y1 = __ffma2_rn(x1, cs, p1);
          ra[e] = pack_bf16x2(y0.x, y0.y);
          rb[e] = pack_bf16x2(y1.x, y1.y);
        }
      }
      *reinterpret_cast<uint4*>(dst + q0) = make_uint4(ra[0], ra[1], ra[2], ra[3]);
      *reinterpret_cast<uint4*>(dst + q1) = make_uint4(rb[0], rb[1], rb[2], rb[3]);
      return false;
    }
    if (row_of[token] < 0) return false;
    const bool is_k = head < p.h + p.h_kv;
    const float unit = is_k ? p.k_unit : p.v_unit;
    float y[16];
    uint2 codes;
    uint32_t scale;
    // (Where every angle is zero, as at position 0, the rotation is exact, and ties are
    // frequent: half of such blocks would be in doubt, one after another in their warp, 8 us.)
    auto turns = [&]() {
      if (p.interleaved) return turned[token][c] != 0;
      const int eights = half >> 3, e0 = 2 * c < eights ? 2 * c : 2 * c - eights;
      const int e1 = 2 * c + 1 < eights ? 2 * c + 1 : 2 * c + 1 - eights;
      return (turned[token][e0] | turned[token][e1]) != 0;
    };
    if (rotates && is_k && turns()) {
      float off = 0.f;                                        // the largest |a| + |b|
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        const uint4 o4 = ch ? b : a, p4 = ch ? pb : pa;
        const uint32_t own[4] = {o4.x, o4.y, o4.z, o4.w}, other[4] = {p4.x, p4.y, p4.z, p4.w};
        const int x0 = c * 16 + ch * 8;
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 o = unpack_bf16x2(own[e]);
            const float4 r2 = turn(c, ch * 2 + e / 2);
            const float2 r = e % 2 ? make_float2(r2.y, r2.w) : make_float2(r2.x, r2.z);
            y[ch * 8 + 2 * e] = (o.x * r.x - o.y * r.y) * unit;
            y[ch * 8 + 2 * e + 1] = (o.y * r.x + o.x * r.y) * unit;
            off = fmaxf(off, fabsf(o.x) + fabsf(o.y));
          }
        } else {
          const bool second = x0 >= half;
          const int eight = (second ? x0 - half : x0) / 8;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 o = unpack_bf16x2(own[e]), t = unpack_bf16x2(other[e]);
            const float4 r = turn(eight, e);
            const float2 sn = second ? make_float2(r.z, r.w) : make_float2(-r.z, -r.w);
            const float2 v = __fmul2_rn(__ffma2_rn(o, make_float2(r.x, r.y), __fmul2_rn(t, sn)), make_float2(unit, unit));
            y[ch * 8 + 2 * e] = v.x;
            y[ch * 8 + 2 * e + 1] = v.y;
            off = fmax3(off, fabsf(o.x) + fabsf(t.x), fabsf(o.y) + fabsf(t.y));
          }
        }
      }
      if (!quantise<true>(y, off * kSlack * unit, &codes, &scale)) return true;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x0 = unpack_bf16x2(ua[e]), x1 = unpack_bf16x2(ub[e]);
        y[2 * e] = x0.x * unit;
        y[2 * e + 1] = x0.y * unit;
        y[8 + 2 * e] = x1.x * unit;
        y[8 + 2 * e + 1] = x1.y * unit;
      }
      quantise<false>(y, 0.f, &codes, &scale);
    }
    store(token, head, c, codes, scale);
    return false;
  };
  for (bool first = true; token < tokens; first = false) {
    const int head = head0 + (lane >> p.log_blocks);
    if (!first) load(token, head);
    const bool open = work(token, head);
    for (uint32_t left = __ballot_sync(0xffffffffu, open); left != 0; left &= left - 1) {
      const int from = __ffs(left) - 1, its_head = head0 + (from >> p.log_blocks);
      const int its_c = from & ((1 << p.log_blocks) - 1);
      uint2 codes;
      uint32_t scale;
      block_in_48_bits(p, source(token, its_head), its_c * 16, pos_of[token], lane, &codes, &scale);
      if (lane == 0) store(token, its_head, its_c, codes, scale);
    }
    head0 += kWarps * warp_heads;
    carry();
  }
}

template <int kTokens, int kBlocks>
cudaError_t launch_append_impl(const Paged4AppendParams& p, cudaStream_t stream) {
  const int blocks = (p.n_tokens + kTokens - 1) / kTokens;
  const size_t smem = static_cast<size_t>(kTokens) * (p.d_rot / 2) * sizeof(float2);
  return launch_kernel(sdpa_paged4_append_kernel<kTokens, kBlocks>, dim3(static_cast<unsigned>(blocks)),
                       dim3(kThreads), smem, stream, true, p);
}

// ---------------------------------------------------------------------- read
// An item is 8 columns of a row: 4 bytes of codes and a scale in, 16 bytes out.  Bound
// by HBM, four fifths of it the rows that are written (by the launch and the chain of
// loads to a token's page for a few tokens).
struct ReadPlace {
  long long codes, scales;                                    // of head 0; kZeros, kNone
};
constexpr long long kZeros = -1, kNone = -2;                  // no position; no sequence's row

__device__ __forceinline__ long long read_page_bytes(const Paged4ReadParams& p) {   // of one head
  return static_cast<long long>(9 * p.d / 16) << p.page_shift;
}
__device__ __forceinline__ ReadPlace read_place(const Paged4ReadParams& p, const RowPlace& at) {
  if (at.row < 0) return {at.pos == INT_MIN ? kNone : kZeros, 0};
  const long long page = (at.row >> p.page_shift) * read_page_bytes(p), r = at.row & ((1 << p.page_shift) - 1);
  return {page + r * (p.d / 2), page + (static_cast<long long>(p.d / 2) << p.page_shift) + r * (p.d / 16)};
}
// Eight columns: codes times scale times unit, exact in bf16.
__device__ __forceinline__ uint4 read_item(uint32_t codes, uint32_t scale, float unit) {
  const float f = e4m3_value(scale) * unit;
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t two;
    asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(two) : "r"(codes >> (8 * e)));
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(two));
    out[e] = pack_bf16x2(lo * f, hi * f);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// A block takes kTokens tokens, whose places a warp of it works out first, and a warp
// one head of K or V after another: consecutive rows of a page are consecutive bytes, a
// token's row goes out as 2 d consecutive bytes, and an item's addresses are two
// additions.  (With the items of all heads dealt out evenly an item costs two divisions:
// 122 us for 196608 tokens of 4 heads of d = 128, and 86 here, 6.1 TB/s.  Four items at
// once instead of eight 88 us, 16 tokens a block instead of 32 95 us.)
__global__ void __launch_bounds__(kThreads) sdpa_paged4_read_kernel(const __grid_constant__ Paged4ReadParams p) {
  constexpr int kWarps = kThreads / 32, kAtOnce = 8;
  __shared__ ReadPlace places[kReadTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = static_cast<int>(blockIdx.x) * kReadTokens;
  const int tokens = min(kReadTokens, p.n_tokens - t0);
  griddep_launch_dependents();
  griddep_wait();
  if (warp == 0) {
    const RowPlace at = place_of_rows(p, t0, tokens, lane);
    if (lane < tokens) places[lane] = read_place(p, at);
  }
  __syncthreads();
  const int c = lane & ((1 << p.log_items) - 1);              // item of the row
  const int first = lane >> p.log_items, step = 32 >> p.log_items;
  for (int head = warp; head < 2 * p.h_kv; head += kWarps) {
    const bool is_k = head < p.h_kv;
    const int hk = is_k ? head : head - p.h_kv;
    const uint8_t* from = (is_k ? p.k_pages : p.v_pages) + hk * read_page_bytes(p);
    uint16_t* to = (is_k ? p.k : p.v) + (static_cast<long long>(t0) * p.h_kv + hk) * p.d + c * 8;
    const float unit = is_k ? p.k_unit : p.v_unit;
    for (int i0 = first; i0 < tokens; i0 += kAtOnce * step) {
      uint32_t codes[kAtOnce], scales[kAtOnce];
      bool write[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = i0 + j * step;
        codes[j] = scales[j] = 0u;
        write[j] = i < tokens;
        if (!write[j]) continue;
        const ReadPlace at = places[i];
        write[j] = at.codes != kNone;
        if (at.codes < 0) continue;
        codes[j] = __ldcg(reinterpret_cast<const uint32_t*>(from + at.codes) + c);
        scales[j] = __ldcg(from + at.scales + (c >> 1));
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (write[j])
          *reinterpret_cast<uint4*>(to + static_cast<long long>(i0 + j * step) * p.h_kv * p.d) =
              read_item(codes[j], scales[j], unit);
    }
  }
}

// Few tokens: a block takes one, its threads its heads' items.
__global__ void __launch_bounds__(kThreads) sdpa_paged4_read_few_kernel(const __grid_constant__ Paged4ReadParams p) {
  __shared__ ReadPlace place;
  const int t = static_cast<int>(blockIdx.x), items = 2 * p.h_kv << p.log_items;
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x < 32) {
    const RowPlace at = place_of_row(p, t, threadIdx.x);
    if (threadIdx.x == 0) place = read_place(p, at);
  }
  __syncthreads();
  const ReadPlace at = place;
  if (at.codes == kNone) return;
  for (int x = threadIdx.x; x < items; x += kThreads) {
    const int head = x >> p.log_items, c = x & ((1 << p.log_items) - 1);
    const bool is_k = head < p.h_kv;
    const int hk = is_k ? head : head - p.h_kv;
    const uint8_t* from = (is_k ? p.k_pages : p.v_pages) + hk * read_page_bytes(p);
    uint32_t codes = 0, scale = 0;
    if (at.codes >= 0) {
      codes = __ldcg(reinterpret_cast<const uint32_t*>(from + at.codes) + c);
      scale = __ldcg(from + at.scales + (c >> 1));
    }
    *reinterpret_cast<uint4*>((is_k ? p.k : p.v) + (static_cast<long long>(t) * p.h_kv + hk) * p.d + c * 8) =
        read_item(codes, scale, is_k ? p.k_unit : p.v_unit);
  }
}

}  // namespace

cudaError_t launch_sdpa_paged4_append(const Paged4AppendParams& p, cudaStream_t stream) {
  const int sms = device_sm_count();
  // (608, 1216 and 2432 tokens of 16 + 2 x 4 heads of d = 128: 5.0, 7.9 and 12.4 us with a
  // block for each token, 6.4, 8.9 and 10.6 with one for four.  Registers for five blocks on an SM:
  // 2258 and 16384 tokens 8.7 and 44.6 us, for six 9.5 and 44.0; eight tokens a block 11.5 and 44.2)
  if (p.n_tokens <= 8 * sms) return launch_append_impl<1, 4>(p, stream);
  return launch_append_impl<4, 5>(p, stream);
}

cudaError_t launch_sdpa_paged4_read(const Paged4ReadParams& p, cudaStream_t stream) {
  const int sms = device_sm_count();
  // (1216, 2432 and 4864 tokens of 4 heads of d = 128: 3.0, 4.4 and 6.8 us with a block
  // each, 4.8, 4.8 and 4.7 with one for 32)
  if (p.n_tokens <= 16 * sms)
    return launch_kernel(sdpa_paged4_read_few_kernel, dim3(static_cast<unsigned>(p.n_tokens)), dim3(kThreads), 0, stream,
                         true, p);
  const unsigned blocks = (static_cast<unsigned>(p.n_tokens) + kReadTokens - 1) / kReadTokens;
  return launch_kernel(sdpa_paged4_read_kernel, dim3(blocks), dim3(kThreads), 0, stream, true, p);
}

}  // namespace sdpa
