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
// bytes, and is bound by HBM (by the launch for a few tokens).  An item is 16
// columns of a head: of a query the two chunks of 8 whose columns pair up, of a
// key or value a block (the rotation reads its partners' columns beside it).
// Blocks take kTokens tokens: their angles once, into shared memory, then every
// head of theirs.
//
// The rotation is in fp32 with angles good to 1.3e-6.  Where that leaves open
// which scale or code is the nearest, some element of a block lies within kSlack
// of a border between two (about one block in 3000): the block is worked out
// again in 64 bits, so that the cache holds what the definition says.
// Of |a| + |b|: the angle, cos and sin's own rounding, and three roundings of products and sum.
constexpr float kSlack = 1.8e-6f;

// Columns col .. col + 15 of key row `row` at position pos, in 64 bits, by all
// lanes of a warp: a lane for each column, as a sine in 64 bits takes 2 us (one
// lane for the 16 took 30 us, ten times a short call).
__device__ __noinline__ void block_in_64_bits(const Paged4AppendParams& p, const uint16_t* row, int col, int pos,
                                              int lane, uint2* codes, uint32_t* scale) {
  const int half = p.d_rot / 2;
  auto value = [&](int x) { return static_cast<double>(__uint_as_float(static_cast<uint32_t>(row[x]) << 16)); };
  const int i = lane & 15, x = col + i;
  const int pair = p.interleaved ? x / 2 : (x < half ? x : x - half);
  const bool second = p.interleaved ? (x & 1) : x >= half;
  const double own = value(x), other = value(p.interleaved ? x ^ 1 : (second ? x - half : x + half));
  double sn, cs;
  sincos(static_cast<double>(pos) * static_cast<double>(p.freqs[pair]), &sn, &cs);
  const double y = (second ? own * cs + other * sn : own * cs - other * sn) * static_cast<double>(p.k_unit);
  double top = fabs(y);
#pragma unroll
  for (int z = 8; z > 0; z >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, z));
  // rounded to a float that is odd where it is not exact, a second rounding is as if it were the first
  auto odd = [](double v) {
    const float f = __double2float_rz(v);
    return static_cast<double>(f) != v && isfinite(f) ? __uint_as_float(__float_as_uint(f) | 1u) : f;
  };
  const uint32_t s8 = e4m3x2(odd(fmin(top / 6.0, 448.0)), 0.f) & 0xff;
  const float s = e4m3_value(s8);
  uint32_t c = s > 0.f ? e2m1x2(odd(fmin(fabs(y) / static_cast<double>(s), 8.0)), 0.f) & 7u : 0u;
  c = (c | (y < 0.0 ? 8u : 0u)) << (4 * (i & 7));
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
  // a division, as the quotient of a bf16 number may lie between two scales
  const uint32_t s8 = kOff ? e4m3x2(__fdiv_rn(top + off, 6.f), __fdiv_rn(top - off, 6.f))
                           : e4m3x2(__fdiv_rn(top, 6.f), 0.f);
  const float s = e4m3_value(s8 & 0xff);
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t w[2] = {0, 0}, open = kOff ? (s8 & 0xff) ^ (s8 >> 8) : 0u;
  if constexpr (kOff) {
    const float d = fmaf(off, inv * 1.000001f, 2e-6f);       // (and the product's rounding)
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float a = fabsf(y[i]) * inv, b = fabsf(y[i + 1]) * inv;
      const uint32_t hi = e2m1x2(a + d, b + d);
      open |= hi ^ e2m1x2(fmaxf(a - d, 0.f), fmaxf(b - d, 0.f));
      w[i >> 3] |= hi << (4 * (i & 7));
    }
  } else {
    // Bf16 numbers may lie on a border itself, but none other lies nearer than 2^-10
    // to one: the product with 1 / s (off by 2^-22) is rounded to whole 2^-12.
    constexpr float kSnap = 0x1.8p11f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float a = __fadd_rn(__fadd_rn(fabsf(y[i]) * inv, kSnap), -kSnap);
      const float b = __fadd_rn(__fadd_rn(fabsf(y[i + 1]) * inv, kSnap), -kSnap);
      w[i >> 3] |= e2m1x2(a, b) << (4 * (i & 7));
    }
  }
  uint32_t sign[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) sign[i >> 3] |= __float_as_uint(y[i]) >> 31 << (4 * (i & 7) + 3);
  *codes = make_uint2(w[0] | sign[0], w[1] | sign[1]);
  *scale = s8 & 0xff;
  return open == 0;
}

template <int kTokens, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) sdpa_paged4_append_kernel(const __grid_constant__ Paged4AppendParams p) {
  static_assert(kTokens <= kThreads / 32, "a warp finds each token's place");
  extern __shared__ __align__(16) float2 angles[];            // [kTokens][d_rot / 2]
  __shared__ long long row_of[kTokens];                       // page row of the token, head 0 (-1: not stored)
  __shared__ int pos_of[kTokens];                             // position (INT_MIN: no sequence's token)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = static_cast<int>(blockIdx.x) * kTokens;
  const int half = p.d_rot / 2, rotated_blocks = p.d_rot / 16;
  const int blocks_mask = (1 << p.log_blocks) - 1;            // items of a head, d / 16
  const int items = (p.h + 2 * p.h_kv) << p.log_blocks;       // of a token
  const int all = min(kTokens, p.n_tokens - t0) * items;
  const int page_rows_mask = (1 << p.page_shift) - 1;
  struct Item {
    int token, head, c;                                       // c: of the head's items
    bool rotated;
    int c0, c1;                                               // columns of its chunks
  };
  auto item_of = [&](int x) {
    Item it;
    it.token = kTokens == 1 ? 0 : (p.items_magic != 0 ? __umulhi(x, p.items_magic) : x / items);
    const int y = x - it.token * items;
    it.head = y >> p.log_blocks;
    it.c = y & blocks_mask;
    it.rotated = it.c < rotated_blocks && it.head < p.h + p.h_kv;
    const bool apart = it.rotated && !p.interleaved && it.head < p.h;
    it.c0 = apart ? it.c * 8 : it.c * 16;
    it.c1 = apart ? it.c0 + half : it.c0 + 8;
    return it;
  };
  auto source = [&](const Item& it) -> const uint16_t* {
    const long long t = t0 + it.token;
    if (it.head < p.h) return p.q == nullptr ? nullptr : p.q + t * p.q_stride + it.head * p.d;
    const int hk = it.head - p.h;
    return hk < p.h_kv ? p.k + t * p.k_stride + hk * p.d : p.v + t * p.v_stride + (hk - p.h_kv) * p.d;
  };
  // a key's column x of a chunk of 8 pairs up with column x + partner
  auto partner = [&](int x) { return x < half ? half : -half; };
  uint4 a, b, pa, pb;
  auto load = [&](int x) {
    if (x >= all) return;
    const Item it = item_of(x);
    const uint16_t* src = source(it);
    if (src == nullptr) return;
    a = *reinterpret_cast<const uint4*>(src + it.c0);
    b = *reinterpret_cast<const uint4*>(src + it.c1);
    if (it.rotated && it.head >= p.h && !p.interleaved) {
      pa = *reinterpret_cast<const uint4*>(src + it.c0 + partner(it.c0));
      pb = *reinterpret_cast<const uint4*>(src + it.c1 + partner(it.c1));
    }
  };
  griddep_launch_dependents();
  griddep_wait();
  load(threadIdx.x);
  if (warp < kTokens && t0 + warp < p.n_tokens) {
    const RowPlace at = place_of_row(p, t0 + warp, lane);
    if (lane == 0) {
      row_of[warp] = at.row;
      pos_of[warp] = at.pos;
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < kTokens * half; x += kThreads) {
    const int i = x / half;
    if (t0 + i < p.n_tokens && pos_of[i] != INT_MIN) angles[x] = cos_sin(pos_of[i], p.freqs[x - i * half]);
  }
  __syncthreads();
  // stores a key's or value's block
  auto store = [&](const Item& it, uint2 codes, uint32_t scale) {
    // row_of: page h_kv P + r for page row r of head 0
    const long long row = row_of[it.token];
    const long long r = row & page_rows_mask;
    const int hk = it.head - p.h;
    const bool is_k = hk < p.h_kv;
    uint8_t* page = (is_k ? p.k_pages : p.v_pages) +
                    ((row >> p.page_shift) + (is_k ? hk : hk - p.h_kv)) * (static_cast<long long>(9 * p.d / 16) << p.page_shift);
    *reinterpret_cast<uint2*>(page + r * (p.d / 2) + it.c * 8) = codes;
    page[(static_cast<long long>(p.d / 2) << p.page_shift) + (r << p.log_blocks) + it.c] = static_cast<uint8_t>(scale);
  };
  // Does an item; true: its block has to be worked out in 64 bits.
  auto work = [&](const Item& it) -> bool {
    if (pos_of[it.token] == INT_MIN) return false;
    const float4* turn = reinterpret_cast<const float4*>(angles + it.token * half);   // (cos, sin) of two pairs
    const uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ub[4] = {b.x, b.y, b.z, b.w};
    if (it.head < p.h) {
      if (p.q == nullptr) return false;
      uint16_t* dst = p.q_out + (static_cast<long long>(t0 + it.token) * p.h + it.head) * p.d;
      uint32_t ra[4], rb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ra[e] = ua[e];
        rb[e] = ub[e];
        if (!it.rotated) continue;
        const float2 x0 = unpack_bf16x2(ua[e]), x1 = unpack_bf16x2(ub[e]);
        if (p.interleaved) {
          const float4 r01 = turn[it.c * 4 + e / 2], r45 = turn[it.c * 4 + 2 + e / 2];
          const float2 r0 = e % 2 ? make_float2(r01.z, r01.w) : make_float2(r01.x, r01.y);
          const float2 r1 = e % 2 ? make_float2(r45.z, r45.w) : make_float2(r45.x, r45.y);
          ra[e] = pack_bf16x2(x0.x * r0.x - x0.y * r0.y, x0.y * r0.x + x0.x * r0.y);
          rb[e] = pack_bf16x2(x1.x * r1.x - x1.y * r1.y, x1.y * r1.x + x1.x * r1.y);
        } else {
          const float4 r = turn[it.c * 4 + e];                // pairs 8 c + 2 e, 8 c + 2 e + 1
          ra[e] = pack_bf16x2(x0.x * r.x - x1.x * r.y, x0.y * r.z - x1.y * r.w);
          rb[e] = pack_bf16x2(x1.x * r.x + x0.x * r.y, x1.y * r.z + x0.y * r.w);
        }
      }
      *reinterpret_cast<uint4*>(dst + it.c0) = make_uint4(ra[0], ra[1], ra[2], ra[3]);
      *reinterpret_cast<uint4*>(dst + it.c1) = make_uint4(rb[0], rb[1], rb[2], rb[3]);
      return false;
    }
    if (row_of[it.token] < 0) return false;
    const float unit = it.head < p.h + p.h_kv ? p.k_unit : p.v_unit;
    float y[16];
    uint2 codes;
    uint32_t scale;
    if (it.rotated) {
      float off = 0.f;                                        // the largest |a| + |b|
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        const uint4 o4 = ch ? b : a, p4 = ch ? pb : pa;
        const uint32_t own[4] = {o4.x, o4.y, o4.z, o4.w}, other[4] = {p4.x, p4.y, p4.z, p4.w};
        const int x0 = it.c * 16 + ch * 8;
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 o = unpack_bf16x2(own[e]);
            const float4 r2 = turn[x0 / 4 + e / 2];
            const float2 r = e % 2 ? make_float2(r2.z, r2.w) : make_float2(r2.x, r2.y);
            y[ch * 8 + 2 * e] = (o.x * r.x - o.y * r.y) * unit;
            y[ch * 8 + 2 * e + 1] = (o.y * r.x + o.x * r.y) * unit;
            off = fmaxf(off, fabsf(o.x) + fabsf(o.y));
          }
        } else {
          const bool second = x0 >= half;
          const int base = (second ? x0 - half : x0) / 2;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 o = unpack_bf16x2(own[e]), t = unpack_bf16x2(other[e]);
            float4 r = turn[base + e];
            if (!second) {
              r.y = -r.y;
              r.w = -r.w;
            }
            y[ch * 8 + 2 * e] = (o.x * r.x + t.x * r.y) * unit;
            y[ch * 8 + 2 * e + 1] = (o.y * r.z + t.y * r.w) * unit;
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
    store(it, codes, scale);
    return false;
  };
  for (int x0 = warp * 32; x0 < all; x0 += kThreads) {
    const int x = x0 + lane;
    if (x0 != warp * 32) load(x);
    const Item it = item_of(min(x, all - 1));
    const bool open = x < all && work(it);
    for (uint32_t left = __ballot_sync(0xffffffffu, open); left != 0; left &= left - 1) {
      const Item its = item_of(x0 + __ffs(left) - 1);
      uint2 codes;
      uint32_t scale;
      block_in_64_bits(p, source(its), its.c * 16, pos_of[its.token], lane, &codes, &scale);
      if (lane == 0) store(its, codes, scale);
    }
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
  if (p.n_tokens <= 4 * sms) return launch_append_impl<1, 4>(p, stream);
  return launch_append_impl<4, 4>(p, stream);
}

cudaError_t launch_sdpa_paged4_read(const Paged4ReadParams& p, cudaStream_t stream) {
  const int sms = device_sm_count();
  // (2258 tokens of 8 heads of d = 64: 4.2 us with a block each, 5.0 with one for 32)
  if (p.n_tokens <= 16 * sms)
    return launch_kernel(sdpa_paged4_read_few_kernel, dim3(static_cast<unsigned>(p.n_tokens)), dim3(kThreads), 0, stream,
                         true, p);
  const unsigned blocks = (static_cast<unsigned>(p.n_tokens) + kReadTokens - 1) / kReadTokens;
  return launch_kernel(sdpa_paged4_read_kernel, dim3(blocks), dim3(kThreads), 0, stream, true, p);
}

}  // namespace sdpa
