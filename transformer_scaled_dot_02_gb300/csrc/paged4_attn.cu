// Attention of packed new tokens over a paged cache held in 4 bits (paged4.cu
// gives the format): the token at position p sees keys j <= p, with a window
// those with p - window < j or j < sinks.
//
// A UNIT is (sequence, key-value head, row tile): up to 8 NT rows, a row being
// a new token's query head of the group.  Its walk is the key tiles of 32 that
// some row sees.  All units' walks laid end to end are cut into equal runs, one
// for each CTA; the cut is worked out on the device from the lengths.  A piece
// of a unit that is cut is published as fp32 (O, m, l), and the run that
// publishes the last piece merges all of a unit's in the order of their keys,
// so that results repeat bit by bit and no run waits for another:
//   O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, M = max_s m_s.
//
// Every warp takes key tiles of its own (every kWarps'th of a piece), with a
// ring of bulk copies ahead of it, and keeps O, m and l of its own until the
// piece ends.  A step for single tokens is bound by reading the cache, so what
// counts is that few instructions stand between a byte and its products.  They
// are mma.sync on registers: tcgen05 takes its operands from shared memory (or A
// from tensor memory), where the expanded numbers, 4 bytes for each byte of the
// cache, would be written and read again, more than an SM's shared memory moves
// in the time that HBM brings the bytes.
//   S^T = K Q^T   A = 16 keys x 16 columns: a lane's columns are d / 4 consecutive
//                 ones of a row (the same order for Q: sums do not care), so a row
//                 is one wide load of four lanes, 16 bytes each at d = 128
//   O^T = V^T P   A = 16 columns x 16 keys: a register pairs two keys' codes of one
//                 column, so two keys' words are interleaved nibble by nibble
//                 (2 operations for 8 codes) before they are expanded
// Codes become fp16 in pairs (cvt.f16x2.e2m1x2) and are multiplied by the block's
// scale, which is exact.  Q is bf16, whose range fp16 has not: each row is scaled
// by a power of two to a largest element of 2^13 and more, which keeps every bit
// of elements down to 2^-27 of it.  The softmax weights are rounded to fp16
// (2^-12), P of S^T turned by movmatrix.
#include <algorithm>
#include <atomic>
#include <climits>

#include "kernels.h"
#include "ptx.cuh"

namespace sdpa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 32;                  // per tile
constexpr int kKeysShift = 5;
constexpr int kStages = 2;                 // tiles of a warp's ring
constexpr float kRescaleThreshold = 8.0f;  // log2 units, as in the other forward kernels
// What a unit costs beside its key tiles, in key tiles.
constexpr int kStart = 8;
constexpr int kMinRun = 16;                // items of a run, at least
constexpr int kRadix = 16;                 // pieces that one run merges

// ------------------------------------------------------------------ schedule
struct Seq {
  int start, n, len, tiles;                // tiles: row tiles
};

// The key tiles that rows of positions lo .. hi see (lo > hi or hi < 0: none):
// tiles [0, head), then those from `first` on.
struct Tiles {
  int head, first, count;
  __device__ __forceinline__ int at(int i) const { return i < head ? i : first + i - head; }
};

template <int R>
struct Plan {
  const Paged4Params& p;
  __device__ explicit Plan(const Paged4Params& params) : p(params) {}

  __device__ __forceinline__ Seq seq(int s) const {
    Seq q;
    const int cap = p.pages_per_seq << p.page_shift;
    q.start = min(max(p.q_starts[s], 0), p.n_tokens);
    q.n = min(max(p.q_starts[s + 1], q.start), p.n_tokens) - q.start;
    q.len = min(max(p.kv_lengths[s], 0), cap);
    q.tiles = static_cast<int>((1ll * q.n * p.group + R - 1) / R);
    return q;
  }
  __device__ __forceinline__ Tiles walk(int lo, int hi) const {
    Tiles t{0, 0, 0};
    if (hi < 0) return t;
    const int last = hi >> kKeysShift;
    if (p.window < INT_MAX) {
      const int from = max(max(lo, 0) - p.window + 1, 0);    // the first position of the window
      t.first = from >> kKeysShift;
      t.head = min((min(p.sinks, hi + 1) + kKeys - 1) >> kKeysShift, t.first);
    }
    t.count = t.head + last - t.first + 1;
    return t;
  }
  // positions of the first and the last row of a row tile
  __device__ __forceinline__ int first_pos(const Seq& q, int r) const { return q.len - q.n + r * R / p.group; }
  __device__ __forceinline__ int last_pos(const Seq& q, int r) const {
    return q.len - q.n + static_cast<int>((min((r + 1ll) * R, 1ll * q.n * p.group) - 1) / p.group);
  }
  // items of a unit: no walk of the sequence is longer
  __device__ __forceinline__ long long cost(const Seq& q) const {
    if (q.len <= 0) return kStart;
    int tiles = ((q.len - 1) >> kKeysShift) + 1;
    if (p.window < INT_MAX) {
      const long long span = 1ll * p.window + R / p.group + 1;
      tiles = static_cast<int>(min(1ll * tiles, (span >> kKeysShift) + 2 + ((min(p.sinks, q.len) + kKeys - 1) >> kKeysShift)));
    }
    return kStart + tiles;
  }
};

struct Place {
  int s, hk, r;
  long long begin;                         // the unit's first item
  Seq q;
};

struct ScheduleShared {
  long long warp_sum[kWarps];
  Place at;
};

// The runs: [begin(c), begin(c + 1)) of all items.
struct Cut {
  long long each;
  int over, runs;
  __device__ void set(long long work, int most) {
    runs = static_cast<int>(min(static_cast<long long>(most), max(1ll, work / kMinRun)));
    each = work / runs;
    over = static_cast<int>(work - each * runs);
  }
  __device__ long long begin(int c) const { return each * c + min(c, over); }
  __device__ int run_of(long long x) const {
    const long long longer = over * (each + 1);
    return static_cast<int>(x < longer ? x / (each + 1) : over + (x - longer) / each);
  }
};

// The whole block: the cut, and the unit in which run c begins.  Returns false
// when there is no such run.
template <int R>
__device__ bool find_place(const Plan<R>& plan, ScheduleShared* sh, int c, Cut* cut, Place* at) {
  const Paged4Params& p = plan.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (p.b + kThreads - 1) / kThreads;
  const int s0 = min(tid * per, p.b), s1 = min(s0 + per, p.b);
  long long mine = 0;
  for (int s = s0; s < s1; ++s) {
    const Seq q = plan.seq(s);
    mine += plan.cost(q) * q.tiles * p.h_kv;
  }
  long long incl = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, x);
    if (lane >= x) incl += o;
  }
  if (lane == 31) sh->warp_sum[warp] = incl;
  if (tid == 0) sh->at.begin = LLONG_MAX;                    // (no unit, should the lengths change meanwhile)
  __syncthreads();
  long long before = incl - mine, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const long long v = sh->warp_sum[w];
    if (w < warp) before += v;
    sum += v;
  }
  if (sum == 0) return false;
  cut->set(sum, p.runs);
  if (c >= cut->runs) return false;
  const long long x = cut->begin(c);
  if (mine > 0 && before <= x && x < before + mine) {
    Place pl;
    for (pl.s = s0; pl.s < s1; ++pl.s) {
      pl.q = plan.seq(pl.s);
      const long long unit = plan.cost(pl.q), all = unit * pl.q.tiles * p.h_kv;
      if (x < before + all) {
        const long long i = (x - before) / unit;
        pl.hk = static_cast<int>(i / pl.q.tiles);
        pl.r = static_cast<int>(i - 1ll * pl.hk * pl.q.tiles);
        pl.begin = before + i * unit;
        sh->at = pl;
        break;
      }
      before += all;
    }
  }
  __syncthreads();
  *at = sh->at;
  return true;
}

// ---------------------------------------------------------------- arithmetic
// 2 x 2 fp16 numbers of the codes in bytes 2 i and 2 i + 1 of a word (low half of
// a byte in the low half of the register).
__device__ __forceinline__ void expand4(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// two e4m3 numbers as fp16
__device__ __forceinline__ uint32_t scales_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float weight(float m, float sub) { return ex2_approx(m - sub); }

// N bytes of shared memory (aligned to N) as words; N < 4 in the low bytes of one.
template <int N>
__device__ __forceinline__ void load_bytes(const uint8_t* at, uint32_t (&w)[N < 4 ? 1 : N / 4]) {
  if constexpr (N == 1) {
    w[0] = *at;
  } else if constexpr (N == 2) {
    w[0] = *reinterpret_cast<const uint16_t*>(at);
  } else if constexpr (N == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  } else if constexpr (N == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(at)[i];
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
}

template <int D, int NT>
struct NCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kCodes = kKeys * D / 2, kScales = kKeys * D / 16;
  static constexpr int kHalf = kCodes + kScales;             // K or V of a tile
  static constexpr int kTile = 2 * kHalf;
  static constexpr int kRing = kWarps * kStages * kTile;
  // O of all warps is exchanged in kPasses parts of the columns
  static constexpr int kPasses = D * NT > 128 ? D * NT / 128 : 1;
  static constexpr int kPassCols = D / kPasses;
  static constexpr int kExchange = kWarps * kRows * kPassCols * 4;
  static constexpr int kMlOff = kRing + kExchange;
  static constexpr int kQOff = kMlOff + kWarps * kRows * 8;
  static constexpr int kBarOff = kQOff;
  static constexpr int kSmemBytes = kBarOff + kWarps * kStages * 8 + 16;
  static constexpr int kCtas = D * NT <= 128 ? 2 : 1;
  static_assert(kTile % 16 == 0 && kHalf % 16 == 0, "bulk copies");
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NCfg<D, NT>::kCtas) sdpa_paged4_few(const __grid_constant__ Paged4Params p) {
  using C = NCfg<D, NT>;
  constexpr int R = C::kRows;
  constexpr int KS = D / 16;                                 // steps of 16 columns
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ScheduleShared sched;
  __shared__ int last_one;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kWarps * kStages);
  const AbortState ab{abort_flag, p.status};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint64_t* full = bars + warp * kStages;
  uint8_t* ring = smem + warp * kStages * C::kTile;
  if (tid < kWarps * kStages) mbar_init(bars + tid, 1);
  if (tid == 0) {
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();

  const Plan<R> plan(p);
  Cut cut;
  Place at;
  const int cta = static_cast<int>(blockIdx.x);
  if (!find_place<R>(plan, &sched, cta, &cut, &at)) return;
  const long long x0 = cut.begin(cta), x1 = cut.begin(cta + 1);

  const int box_shift = min(p.page_shift, kKeysShift);       // rows of a page in a tile
  const long long page_bytes = static_cast<long long>(9 * D / 16) << p.page_shift;
  const int page_mask = (1 << p.page_shift) - 1;
  auto slot = [&](int i) { return p.slots + static_cast<long long>(i) * p.slot_bytes; };

  int used = 0, issued = 0;                                  // tiles that this warp has consumed, asked for
  bool ok = true;
  while (at.begin < x1) {
    const long long unit_items = plan.cost(at.q);
    const int first_pos = plan.first_pos(at.q, at.r), hi_pos = plan.last_pos(at.q, at.r);
    const int lo_pos = max(first_pos, 0);
    const Tiles tiles = plan.walk(lo_pos, hi_pos);
    const long long items0 = at.begin + kStart;              // the first key tile's item
    // this run's key tiles of the unit
    const int kt0 = static_cast<int>(min(1ll * tiles.count, max(0ll, x0 - items0)));
    const int kt1 = static_cast<int>(min(1ll * tiles.count, max(0ll, x1 - items0)));
    const int first_row = at.r * R, rows = static_cast<int>(min(1ll * R, 1ll * at.q.n * p.group - first_row));
    // where row x's output begins
    auto out_of = [&](int x) {
      const int token = (first_row + x) / p.group, head = first_row + x - token * p.group;
      return p.out + (static_cast<long long>(at.q.start + token) * p.h + at.hk * p.group + head) * D;
    };
    if (tiles.count == 0 && at.begin >= x0) {
      // nothing to see: rows of zeros
      for (int x = tid; x < rows * (D / 4); x += kThreads)
        *reinterpret_cast<uint2*>(out_of(x / (D / 4)) + x % (D / 4) * 4) = make_uint2(0u, 0u);
    }
    if (kt1 > kt0) {
      const int32_t* pages = p.page_table + static_cast<long long>(at.s) * p.pages_per_seq;
      const int mine = kt0 + warp < kt1 ? (kt1 - kt0 - warp + kWarps - 1) / kWarps : 0;
      // ---- copies: lane x & 3 of a page's part takes K's codes, K's scales, V's, V's
      const int part = lane >> 2, what = lane & 3;
      const bool copies = part << box_shift < kKeys;
      const uint32_t part_bytes = static_cast<uint32_t>((what & 1 ? D / 16 : D / 2) << box_shift);
      auto page_of = [&](int i) -> int {
        if (!copies || i >= mine) return -2;
        const int key = (tiles.at(kt0 + warp + i * kWarps) << kKeysShift) + (part << box_shift);
        // a page of which no row sees anything is not looked at
        const int end = key + (1 << box_shift) - 1;
        if (key > hi_pos || (p.window < INT_MAX && key >= p.sinks && end <= lo_pos - p.window)) return -2;
        const int page = pages[key >> p.page_shift];
        if (page >= 0 && page < p.n_pages) return page;
        atomicOr(p.status, kStatusBadPage);
        return -1;
      };
      auto issue = [&](int i, int page) {
        if (i >= mine) return;
        issued = used + i + 1;
        const int st = (used + i) % kStages;
        uint8_t* stage = ring + st * C::kTile;
        const int key = (tiles.at(kt0 + warp + i * kWarps) << kKeysShift) + (part << box_shift);
        const bool get = copies && page >= 0;
        uint8_t* dst = stage + (what >> 1) * C::kHalf + (what & 1 ? C::kCodes + (part << box_shift) * (D / 16)
                                                                  : (part << box_shift) * (D / 2));
        const uint32_t bytes = __reduce_add_sync(0xffffffffu, get ? part_bytes : 0u);
        if (lane == 0) mbar_arrive_expect_tx(full + st, bytes);
        if (copies && page == -1 && (what & 1)) {
          // a page outside the cache: scales of zero
          for (uint32_t x = 0; x < part_bytes; x += 4) *reinterpret_cast<uint32_t*>(dst + x) = 0u;
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (get) {
          const uint8_t* src = (what >> 1 ? p.v_pages : p.k_pages) +
                               (static_cast<long long>(page) * p.h_kv + at.hk) * page_bytes;
          const int r = key & page_mask;
          src += what & 1 ? (static_cast<long long>(D / 2) << p.page_shift) + r * (D / 16) : static_cast<long long>(r) * (D / 2);
          tma_load_1d(dst, src, part_bytes, full + st);
        }
      };
      int page_next = page_of(0);
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) {
        const int page = page_next;
        page_next = page_of(i + 1);
        issue(i, page);
      }
      // ---- Q: row 8 nt + g, columns [t D / 4, + D / 4)
      uint32_t qf[KS][NT][2];
      float sc[NT][2];                                       // of columns 2 t, 2 t + 1: score to log2 units
      int pos[NT][2];                                        // their positions (-1: no row)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int x = nt * 8 + g;
        const bool valid = x < rows;
        const int token = (first_row + (valid ? x : 0)) / p.group, head = first_row + (valid ? x : 0) - token * p.group;
        const uint2* src = reinterpret_cast<const uint2*>(
            p.q + static_cast<long long>(at.q.start + token) * p.q_stride + (at.hk * p.group + head) * D + t * (D / 4));
        uint2 raw[KS];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          raw[k] = valid ? src[k] : make_uint2(0u, 0u);
          top = max(max(top, max(raw[k].x & 0x7fffu, raw[k].y & 0x7fffu)), max(raw[k].x >> 16 & 0x7fffu, raw[k].y >> 16 & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = static_cast<int>(top >> 7);           // biased; rows of zeros, infinities and NaN stay
        const int up = top == 0 || ex == 255 ? 0 : max(-120, min(120, 13 + 127 - ex));
        const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        const float back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[k][nt][0] = pack_f16x2(__uint_as_float(raw[k].x << 16) * f, __uint_as_float(raw[k].x & 0xffff0000u) * f);
          qf[k][nt][1] = pack_f16x2(__uint_as_float(raw[k].y << 16) * f, __uint_as_float(raw[k].y & 0xffff0000u) * f);
        }
        const int row_pos = valid ? at.q.len - at.q.n + token : -1;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          sc[nt][c] = __shfl_sync(0xffffffffu, back, (2 * t + c) * 4) * p.k_unit * p.scale_log2;
          pos[nt][c] = __shfl_sync(0xffffffffu, row_pos, (2 * t + c) * 4);
        }
      }
      float o[KS][NT][4], m[NT][2], l[NT][2];
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][nt][e] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          m[nt][c] = -INFINITY;
          l[nt][c] = 0.f;
        }

      for (int i = 0; i < mine && ok; ++i) {
        {
          const int page = page_next;
          page_next = page_of(i + kStages);
          __syncwarp();                                      // (the stage has been read by all lanes)
          issue(i + kStages - 1, page);
        }
        const int st = (used + i) % kStages;
        ok = mbar_wait_warp(full + st, static_cast<uint32_t>((used + i) / kStages) & 1u, ab);
        if (!ok) break;
        const uint8_t* ks = ring + st * C::kTile;
        const uint8_t* vs = ks + C::kHalf;
        const int key0 = tiles.at(kt0 + warp + i * kWarps) << kKeysShift;
        const bool edge = key0 + kKeys - 1 > first_pos || (p.window < INT_MAX && key0 <= hi_pos - p.window);
        // ---- scores
        float s[2][NT][4];
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          constexpr int kB = D / 8, kW = kB < 4 ? 1 : kB / 4;   // bytes, words of a lane's columns
          uint32_t w[2][kW], sw[2];
          constexpr int kSB = D >= 64 ? D / 64 : 1;             // scales of a lane's columns
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int row = mb * 16 + hh * 8 + g;
            load_bytes<kB>(ks + row * (D / 2) + t * kB, w[hh]);
            uint32_t sb[1];
            load_bytes<kSB>(ks + C::kCodes + row * (D / 16) + (D >= 64 ? t * kSB : t * D / 64), sb);
            sw[hh] = sb[0];
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mb][nt][e] = 0.f;
#pragma unroll
          for (int wi = 0; wi < kW; ++wi) {
            uint32_t a[2][4];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              expand4(w[hh][wi], a[hh]);
              // columns t D / 4 + 8 wi ..: block wi / 2 of the lane's
              const uint32_t b = sw[hh] >> (8 * (wi / 2)) & 0xffu;
              const uint32_t sc2 = scales_f16x2(b | b << 8);
#pragma unroll
              for (int e = 0; e < 4; ++e) a[hh][e] = mul_f16x2(a[hh][e], sc2);
            }
            constexpr int kSteps = kB < 4 ? 1 : 2;
#pragma unroll
            for (int e = 0; e < kSteps; ++e)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(s[mb][nt], a[0][2 * e], a[1][2 * e], a[0][2 * e + 1], a[1][2 * e + 1], qf[wi * 2 + e][nt][0],
                        qf[wi * 2 + e][nt][1]);
          }
        }
        if (edge) {
#pragma unroll
          for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = key0 + mb * 16 + (e >> 1) * 8 + g;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const int pp = pos[nt][e & 1];
                if (j > pp || (j <= pp - p.window && j >= p.sinks)) s[mb][nt][e] = -INFINITY;
              }
            }
        }
        // ---- the running maxima: they move when one grew by more than the threshold
        bool need = false;
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            top[nt][c] = fmaxf(fmaxf(s[0][nt][c], s[0][nt][2 + c]), fmaxf(s[1][nt][c], s[1][nt][2 + c])) * sc[nt][c];
            need |= top[nt][c] > m[nt][c] + kRescaleThreshold;
          }
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float x = top[nt][c];
#pragma unroll
              for (int y = 4; y < 32; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
              x = fmaxf(x, m[nt][c]);
              const float f = x == -INFINITY ? 1.f : ex2_approx(m[nt][c] - x);
              m[nt][c] = x;
              l[nt][c] *= f;
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                o[k][nt][c] *= f;
                o[k][nt][2 + c] *= f;
              }
            }
        }
        // ---- weights, turned so that a lane holds two keys of a row
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
          for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float p0 = ex2_approx(fmaf(s[mb][nt][2 * hh], sc[nt][0], -m0));
              const float p1 = ex2_approx(fmaf(s[mb][nt][2 * hh + 1], sc[nt][1], -m1));
              l[nt][0] += p0;
              l[nt][1] += p1;
              pb[mb][nt][hh] = transpose8x8(pack_f16x2(p0, p1));
            }
        }
        // ---- O^T += V^T P
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          constexpr int kB = D / 16, kW = kB < 4 ? 1 : kB / 4;
          constexpr int kSB = D >= 128 ? D / 128 : 1;
          uint32_t w[4][kW], sw[4];                          // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = mb * 16 + 2 * t + (x & 1) + (x >> 1) * 8;
            load_bytes<kB>(vs + row * (D / 2) + g * kB, w[x]);
            uint32_t sb[1];
            load_bytes<kSB>(vs + C::kCodes + row * (D / 16) + (D >= 128 ? g * kSB : g * D / 128), sb);
            sw[x] = sb[0];
            if (edge) {
              // what no row sees may be anything: its weight is zero, zero times a NaN is not
              const int j = key0 + row;
              if (j > hi_pos || (p.window < INT_MAX && j <= lo_pos - p.window && j >= p.sinks)) sw[x] = 0;
            }
          }
#pragma unroll
          for (int wi = 0; wi < kW; ++wi) {
            uint32_t a[4][4];                                // [a0 .. a3][column pair]
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t w0 = w[2 * y][wi], w1 = w[2 * y + 1][wi];
              expand4((w0 & 0x0f0f0f0fu) | (w1 << 4 & 0xf0f0f0f0u), a[2 * y]);
              expand4((w0 >> 4 & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u), a[2 * y + 1]);
              const int blk = wi / 2;                         // 8 columns a word
              const uint32_t sc2 = scales_f16x2((sw[2 * y] >> (8 * blk) & 0xffu) | (sw[2 * y + 1] >> (8 * blk) & 0xffu) << 8);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                a[2 * y][e] = mul_f16x2(a[2 * y][e], sc2);
                a[2 * y + 1][e] = mul_f16x2(a[2 * y + 1][e], sc2);
              }
            }
#pragma unroll
            for (int e = 0; e < (kB < 4 ? kB : 4); ++e)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[wi * 4 + e][nt], a[0][e], a[1][e], a[2][e], a[3][e], pb[mb][nt][0], pb[mb][nt][1]);
          }
        }
      }
      used += mine;
      // ---- the piece's end: the warps' (O, m, l) are merged
      float2* ml = reinterpret_cast<float2*>(smem + C::kMlOff);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int y = 4; y < 32; y <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], y);
          if (g == 0) ml[warp * R + nt * 8 + 2 * t + c] = make_float2(m[nt][c], l[nt][c]);
        }
      const int first_run = cut.run_of(items0), last_run = cut.run_of(items0 + tiles.count - 1);
      const bool whole = first_run == last_run;
      const int of = last_run - first_run + 1;
      float* xo = reinterpret_cast<float*>(smem + C::kRing);
      uint8_t* own = whole ? nullptr : slot(2 * cta + (cta == first_run ? 1 : 0));
      constexpr int kPC = C::kPassCols, kPer = kPC / 8;      // columns of a lane group g in a pass
#pragma unroll
      for (int pass = 0; pass < C::kPasses; ++pass) {
        if (pass > 0) __syncthreads();
#pragma unroll
        for (int k = 0; k < KS / C::kPasses; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              *reinterpret_cast<float2*>(xo + (warp * R + nt * 8 + 2 * t + c) * kPC + g * kPer + 2 * k) =
                  make_float2(o[pass * (KS / C::kPasses) + k][nt][c], o[pass * (KS / C::kPasses) + k][nt][2 + c]);
        // (also the decision whether to go on, the same for all)
        if (__syncthreads_or(!ok)) {
          ok = false;
          break;
        }
        constexpr int kVec = kPer % 4 == 0 ? 4 : 2;          // columns that lie together
        for (int x = tid; x < rows * (kPC / kVec); x += kThreads) {
          const int row = x / (kPC / kVec), c0 = x % (kPC / kVec) * kVec;
          float2 mls[kWarps];
          float mm = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            mls[w] = ml[w * R + row];
            mm = fmaxf(mm, mls[w].x);
          }
          const float sub = mm == -INFINITY ? 0.f : mm;
          float acc[kVec], ll = 0.f;
#pragma unroll
          for (int e = 0; e < kVec; ++e) acc[e] = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float f = weight(mls[w].x, sub);
            ll += mls[w].y * f;
            const float* v = xo + (w * R + row) * kPC + c0;
#pragma unroll
            for (int e = 0; e < kVec; e += 2) {
              const float2 vv = *reinterpret_cast<const float2*>(v + e);
              acc[e] = fmaf(vv.x, f, acc[e]);
              acc[e + 1] = fmaf(vv.y, f, acc[e + 1]);
            }
          }
          // column c0 of the pass: group c0 / kPer's, of the row
          const int col = c0 / kPer * (D / 8) + pass * kPer + c0 % kPer;
          if (whole) {
            const float f = ll > 0.f ? p.v_unit / ll : 0.f;
            uint32_t* dst = reinterpret_cast<uint32_t*>(out_of(row) + col);
#pragma unroll
            for (int e = 0; e < kVec; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * f, acc[e + 1] * f);
          } else {
            float* dst = reinterpret_cast<float*>(own) + row * D + col;
#pragma unroll
            for (int e = 0; e < kVec; e += 2) *reinterpret_cast<float2*>(dst + e) = make_float2(acc[e], acc[e + 1]);
            if (col == 0) reinterpret_cast<float2*>(own + R * D * 4)[row] = make_float2(mm, ll);
          }
        }
      }
      if (!ok) break;
      if (!whole) {
        // ---- published; the last of a group of pieces merges it, the last
        // group's all groups
        const int j = cta - first_run, group = j / kRadix, groups = (of + kRadix - 1) / kRadix;
        auto place = [&](int i) { return 2 * (first_run + i) + (i == 0 ? 1 : 0); };   // of piece i
        // counts `count` up and tells everybody whether this was the last of `all`
        auto arrive = [&](unsigned long long* count, int all) -> bool {
          __threadfence();
          __syncthreads();
          if (tid == 0) {
            unsigned long long old = __ldcg(count), seen;
            while (true) {
              const unsigned long long base = (old & ~0xffffull) == p.call ? old : p.call;
              const bool last = static_cast<int>(base & 0xffff) + 1 >= all;
              seen = atomicCAS(count, old, last ? 0ull : base + 1);
              if (seen == old) {
                last_one = last;
                break;
              }
              old = seen;
            }
            __threadfence();
          }
          __syncthreads();
          return last_one != 0;
        };
        // pieces i0, i0 + step, .. of n, into the output or piece i0's place
        auto merge = [&](int i0, int step, int n, bool final) {
          for (int x = tid; x < rows * (D / 4); x += kThreads) {
            const int row = x / (D / 4), col = x % (D / 4) * 4;
            float mm = -INFINITY;
            for (int i = 0; i < n; ++i)
              mm = fmaxf(mm, __ldcg(reinterpret_cast<const float2*>(slot(place(i0 + i * step)) + R * D * 4) + row).x);
            const float sub = mm == -INFINITY ? 0.f : mm;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float ll = 0.f;
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
              const uint8_t* src = slot(place(i0 + i * step));
              const float2 one = __ldcg(reinterpret_cast<const float2*>(src + R * D * 4) + row);
              const float4 v = __ldcg(reinterpret_cast<const float4*>(src) + row * (D / 4) + col / 4);
              const float f = weight(one.x, sub);
              ll = fmaf(one.y, f, ll);
              acc.x = fmaf(v.x, f, acc.x);
              acc.y = fmaf(v.y, f, acc.y);
              acc.z = fmaf(v.z, f, acc.z);
              acc.w = fmaf(v.w, f, acc.w);
            }
            if (final) {
              const float f = ll > 0.f ? p.v_unit / ll : 0.f;
              *reinterpret_cast<uint2*>(out_of(row) + col) =
                  make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
            } else {
              // (this thread alone reads and writes these columns; the statistics are
              // in a place of their own, behind those that others still read)
              uint8_t* dst = slot(place(i0));
              reinterpret_cast<float4*>(dst)[row * (D / 4) + col / 4] = acc;
              if (col == 0) reinterpret_cast<float2*>(dst + R * D * 4)[R + row] = make_float2(mm, ll);
            }
          }
        };
        if (groups == 1) {
          if (arrive(p.counts + place(0), of)) merge(0, 1, of, true);
        } else {
          const int i0 = group * kRadix, n = min(kRadix, of - i0);
          if (arrive(p.counts + place(i0), n)) {
            merge(i0, 1, n, false);
            __syncthreads();
            // the merged statistics take the piece's place
            if (tid < rows) {
              float2* at_ml = reinterpret_cast<float2*>(slot(place(i0)) + R * D * 4);
              at_ml[tid] = at_ml[R + tid];
            }
            if (arrive(p.counts + 2 * p.runs + first_run, groups)) merge(0, kRadix, groups, true);
          }
        }
      }
      __syncthreads();                                       // (the exchange memory has been read)
    }
    // ---- the next unit
    at.begin += unit_items;
    if (++at.r == at.q.tiles) {
      at.r = 0;
      if (++at.hk == p.h_kv) {
        at.hk = 0;
        do {
          if (++at.s == p.b) break;
          at.q = plan.seq(at.s);
        } while (at.q.n == 0);
        if (at.s == p.b) break;
      }
    }
  }
  // let every copy land before the CTA can exit (a wait may have run out above)
  for (int u = max(0, issued - kStages); u < issued; ++u)
    mbar_wait_drain(full + u % kStages, static_cast<uint32_t>(u / kStages) & 1u);
}

template <int D, int NT>
cudaError_t launch_few_impl(const Paged4Params& p, cudaStream_t stream) {
  constexpr int smem = NCfg<D, NT>::kSmemBytes;
  // the kernel's shared-memory limit is set once on each device
  static std::atomic<unsigned long long> prepared{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev > 63 || !(prepared.load(std::memory_order_acquire) & bit)) {
    err = cudaFuncSetAttribute(sdpa_paged4_few<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    if (dev <= 63) prepared.fetch_or(bit, std::memory_order_release);
  }
  return launch_kernel(sdpa_paged4_few<D, NT>, dim3(static_cast<unsigned>(p.runs)), dim3(kThreads), smem, stream, true, p);
}

template <int D>
cudaError_t launch_d(const Paged4Params& p, cudaStream_t stream) {
  return paged4_rows(p.group, p.n_tokens, p.b) == 8 ? launch_few_impl<D, 1>(p, stream) : launch_few_impl<D, 2>(p, stream);
}

}  // namespace

int paged4_rows(int group, int n_tokens, int b) {
  return 1ll * group * n_tokens <= 8ll * b ? 8 : 16;
}

int paged4_resident_ctas(int d, int rows) { return d * rows <= 1024 ? 2 : 1; }

long long paged4_most_runs(long long units, long long max_len) {
  return std::max(1ll, units * (kStart + max_len / kKeys + 2) / kMinRun);
}

cudaError_t launch_sdpa_paged4(const Paged4Params& p, int d, cudaStream_t stream) {
  switch (d) {
    case 16: return launch_d<16>(p, stream);
    case 32: return launch_d<32>(p, stream);
    case 64: return launch_d<64>(p, stream);
    case 128: return launch_d<128>(p, stream);
    case 256: return launch_d<256>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sdpa
