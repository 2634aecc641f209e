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
// Every warp takes key tiles of its own (every kWarps'th of a piece), copies them
// some tiles ahead into a ring of its own and keeps O, m and l of its own until
// the piece ends.  CTAs are small, so that others on the SM work while one's
// warps meet.  The copies are cp.async, 16 bytes a lane, 9 instructions a tile at
// d = 128: as bulk copies, four for the codes and scales of K and V, a tile took
// the SM's copy engine 600 clock cycles (41 us instead of 38 for 32 sequences of
// 4096 to 8192 positions).  What bounds a step for single tokens is how long a tile's chain
// of loads, conversions, products and exponentials is for the few warps that registers
// leave room for (12 on an SM: issue slots 43 % busy, HBM 38 %), so what counts is that few
// instructions stand between a byte and its products.  They
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
// of elements down to 2^-27 of it.  The softmax weights are taken against a
// reference that lags and rounded to fp16 (paged.cuh), P of S^T turned by movmatrix.
#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace sdpa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 32;                  // per tile
constexpr int kKeysShift = 5;
// What a unit costs beside its key tiles, in key tiles.
// (32 single tokens of 4096 to 8192 positions: 39.3, 37.9 and 37.3 us with 8, 14 and 20;
// 32 of 2000 to 4000 with one key-value head: 25.2, 21.9 and 20.5)
constexpr int kStart = 20;
constexpr int kMinRun = 16;                // items of a run, at least
// How the work is cut.  At a level every unit is cut into pieces of its own, a run for
// each, of up to 8 << level key tiles, where that many runs fit the GPU; a walk of up to
// kWhole tiles is one piece, and at the last level one of more than 64 is cut as at the first.
// kItems: into equal runs, which end and begin inside units.
// Level 0: 8 sequences of 300 to 500 positions, 8 heads of keys, d = 128: 10.6 us with kWhole = 16,
// 11.5 with 12 or 8; 4 of 1000: 11.4 us with pieces of 8, 13.3 of 6, 11.9 of 12.
// Levels 1 to 3 instead of equal runs (sequences of single tokens, 4 heads of d = 128): 28 of 2000
// 17.5 us instead of 19.0, 28 of 4000 24.2 instead of 25.5, 100 of 800 18.2 instead of 25.4, 96 with a
// window of 1000 22.6 instead of 28.7.  With more runs left without work they lose: 27.9 instead of
// 26.9 for 16 sequences of 16 rows (level 2, a third of the runs), 31.4 instead of 29.7 for 64 of 2000
// (whole walks, 62 key tiles where an equal run has 46).
constexpr int kItems = -1, kLevels = 4, kWhole = 16;
constexpr int kMergeItems = 12;            // what publishing and merging a piece takes, in key tiles
constexpr int kTogether = 16;              // pieces that one run merges, at most (more in two steps)

// ------------------------------------------------------------------ schedule
struct Seq {
  int start, n, len, tiles;                // tiles: row tiles
};

// The key tiles that rows of positions lo .. hi see (lo > hi or hi < 0: none):
// tiles [0, head), then those from `first` on.
struct Tiles {
  int head, first, count;
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
    const long long rows = 1ll * q.n * p.group;
    q.tiles = rows <= p.few_rows ? static_cast<int>((rows + R - 1) / R) : 0;
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
  // (rows of a head: up to 2^31, as unsigned numbers; one tile of rows, the usual case, needs no division)
  __device__ __forceinline__ int first_pos(const Seq& q, int r) const {
    return q.len - q.n + (r == 0 ? 0 : static_cast<int>(static_cast<unsigned>(r) * R / static_cast<unsigned>(p.group)));
  }
  __device__ __forceinline__ int last_pos(const Seq& q, int r) const {
    if (r + 1 == q.tiles) return q.len - 1;
    return q.len - q.n + static_cast<int>((static_cast<unsigned>(r + 1) * R - 1u) / static_cast<unsigned>(p.group));
  }
  // key tiles that no walk of the sequence is longer than
  __device__ __forceinline__ int most_tiles(const Seq& q) const {
    if (q.len <= 0) return 0;
    int tiles = ((q.len - 1) >> kKeysShift) + 1;
    if (p.window < INT_MAX) {
      const long long span = 1ll * p.window + R / p.group + 1;
      tiles = static_cast<int>(min(1ll * tiles, (span >> kKeysShift) + 2 + ((min(p.sinks, q.len) + kKeys - 1) >> kKeysShift)));
    }
    return tiles;
  }
  __device__ __forceinline__ int pieces(int tiles, int level) const {
    if (tiles <= kWhole) return 1;
    const int shift = level == kLevels - 1 && tiles > 8 << level ? 3 : 3 + level;
    return (tiles + (1 << shift) - 1) >> shift;
  }
  // items of a unit
  __device__ __forceinline__ int cost(const Seq& q, int level) const {
    return level != kItems ? pieces(most_tiles(q), level) : kStart + most_tiles(q);
  }
};

// Most counts fit 32 bits, where a division costs a tenth of one in 64.
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// A run's place: a unit and the piece of it that is the run's.
struct Unit {
  Seq q;
  int s, hk, r;
  long long begin;                         // the unit's first item
  Tiles tiles;
  int kt0, kt1;                            // the piece, of tiles.count key tiles
  int first_run, of;                       // the unit's pieces are those of runs first_run .. first_run + of - 1
  int first_pos, hi_pos;                   // positions of the first and the last row
  int first_row, rows;                     // of the sequence's rows for this head (no rows: no further unit)
};

// The runs: [begin(c), begin(c + 1)) of all items.
struct Cut {
  long long each;
  int over, runs;
  int level;                               // or kItems
  __device__ void set(long long work, int most, int at_level) {
    level = at_level;
    if (level != kItems) {
      runs = static_cast<int>(work);
      each = 1;
      over = 0;
      return;
    }
    runs = static_cast<int>(min(static_cast<long long>(most), max(1ll, work / kMinRun)));
    each = divide(work, runs);
    over = static_cast<int>(work - each * runs);
  }
  __device__ long long begin(int c) const { return each * c + min(c, over); }
  __device__ int run_of(long long x) const {
    const long long longer = over * (each + 1);
    return static_cast<int>(x < longer ? divide(x, each + 1) : over + divide(x - longer, each));
  }
};

// The piece of run c of the unit *u.
template <int R>
__device__ __forceinline__ void set_piece(const Plan<R>& plan, const Cut& cut, int c, Unit* u) {
  const Paged4Params& p = plan.p;
  const long long x0 = cut.begin(c), x1 = cut.begin(c + 1);
  u->first_pos = plan.first_pos(u->q, u->r);
  u->hi_pos = plan.last_pos(u->q, u->r);
  const Tiles tiles = plan.walk(u->first_pos, u->hi_pos);
  u->tiles = tiles;
  u->first_row = u->r * R;
  u->rows = static_cast<int>(min(1ll * R, 1ll * u->q.n * p.group - u->first_row));
  u->kt0 = u->kt1 = 0;
  u->first_run = c;
  u->of = 1;
  if (cut.level != kItems) {
    // (as many as the sequence's longest walk is worth: this one may have fewer key tiles)
    const int j = static_cast<int>(x0 - u->begin);
    u->of = min(plan.cost(u->q, cut.level), max(tiles.count, 1));
    u->first_run = c - j;
    if (j < u->of) {
      u->kt0 = static_cast<int>(divide(1ll * j * tiles.count, u->of));
      u->kt1 = static_cast<int>(divide((j + 1ll) * tiles.count, u->of));
    }
  } else {
    const long long items0 = u->begin + kStart;              // the first key tile's item
    u->kt0 = static_cast<int>(min(1ll * tiles.count, max(0ll, x0 - items0)));
    u->kt1 = static_cast<int>(min(1ll * tiles.count, max(0ll, x1 - items0)));
    if (u->kt1 > u->kt0 && u->kt1 - u->kt0 < tiles.count) {
      u->first_run = cut.run_of(items0);
      u->of = cut.run_of(items0 + tiles.count - 1) - u->first_run + 1;
    }
  }
}

// The whole block: the cut, and the unit in which run c begins.  Returns false
// when there is no such run.
struct Schedule {
  long long mine[kWarps];
  uint32_t pieces[kWarps][kLevels + 1];
  Cut cut;
};

template <int R>
__device__ bool find_place(const Plan<R>& plan, Schedule* sh, Unit* first, int c) {
  const Paged4Params& p = plan.p;
  // (up to 32 sequences every warp looks at all of them, and none waits for another)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool alone = p.b <= 32;
  const int per = alone ? 1 : (p.b + kThreads - 1) / kThreads;
  const int s0 = min((alone ? lane : tid) * per, p.b), s1 = min(s0 + per, p.b);
  long long items = 0;
  uint32_t pieces[kLevels] = {};                             // (as good as too many from 2^20 on)
  Seq q;
  for (int s = s0; s < s1; ++s) {
    q = plan.seq(s);
    const int tiles = plan.most_tiles(q);
    const long long units = 1ll * q.tiles * p.h_kv;
    items += (kStart + tiles) * units;
#pragma unroll
    for (int x = 0; x < kLevels; ++x)
      pieces[x] = static_cast<uint32_t>(min(1ll << 20, pieces[x] + plan.pieces(tiles, x) * units));
  }
  if (tid == 0) first->begin = LLONG_MAX;                    // (no unit, should the lengths change meanwhile)
  __syncwarp();                                              // (another lane's unit comes after it)
  uint32_t all[kLevels + 1];                                 // the last: items
#pragma unroll
  for (int x = 0; x < kLevels; ++x) all[x] = __reduce_add_sync(0xffffffffu, pieces[x]);
  all[kLevels] = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(min(1ll << 20, items)));
  if (!alone) {
    if (lane == 0) {
#pragma unroll
      for (int x = 0; x <= kLevels; ++x) sh->pieces[warp][x] = all[x];
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x <= kLevels; ++x) {
      all[x] = 0;
      for (int w = 0; w < kWarps; ++w) all[x] += sh->pieces[w][x];
    }
  }
  if (all[0] == 0) return false;
  // The finest level that fits, if it leaves few runs without work.  Whole walks: if they are
  // not longer on average than an equal run, by more than what merging takes.
  int level = kItems;
  const uint32_t runs = static_cast<uint32_t>(p.runs);
  if (all[3] <= runs && 1ull * (all[kLevels] - all[3] * kStart) * runs <= (all[kLevels] + kMergeItems * runs) * 1ull * all[3])
    level = 3;
  if (16 * all[2] >= 13 * runs && all[2] <= runs) level = 2;
  if (8 * all[1] >= 5 * runs && all[1] <= runs) level = 1;
  if (all[0] <= runs) level = 0;
  long long mine = items;
#pragma unroll
  for (int x = 0; x < kLevels; ++x)
    if (level == x) mine = pieces[x];
  long long to = mine;                                       // of the threads up to this one
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long i = __shfl_up_sync(0xffffffffu, to, x);
    if (lane >= x) to += i;
  }
  long long work = __shfl_sync(0xffffffffu, to, 31);
  if (!alone) {
    if (lane == 31) sh->mine[warp] = to;
    __syncthreads();
    work = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) to += work;
      work += sh->mine[w];
    }
  }
  Cut cut;
  cut.set(work, p.runs, level);
  if (c >= cut.runs) return false;
  const long long x = cut.begin(c);
  if (tid == 0) sh->cut = cut;
  long long before = to - mine;
  if (mine > 0 && before <= x && x < before + mine && (!alone || warp == 0)) {
    for (int s = s0; s < s1; ++s) {
      if (per > 1) q = plan.seq(s);
      const int unit = plan.cost(q, level);
      const long long all = 1ll * unit * q.tiles * p.h_kv;
      if (x < before + all) {
        const long long i = divide(x - before, unit);
        Unit u;
        u.q = q;
        u.s = s;
        u.hk = static_cast<int>(divide(i, q.tiles));
        u.r = static_cast<int>(i - 1ll * u.hk * q.tiles);
        u.begin = before + i * unit;
        set_piece(plan, cut, c, &u);
        *first = u;
        break;
      }
      before += all;
    }
  }
  __syncthreads();
  return true;
}

// One thread: the unit after *u, false if there is none of run c's.
template <int R>
__device__ __noinline__ bool next_unit(const Plan<R>& plan, const Cut& cut, int c, Unit* u) {
  u->begin += plan.cost(u->q, cut.level);
  if (u->begin >= cut.begin(c + 1)) return false;
  if (++u->r == u->q.tiles) {
    u->r = 0;
    if (++u->hk == plan.p.h_kv) {
      u->hk = 0;
      do {
        if (++u->s >= plan.p.b) return false;
        u->q = plan.seq(u->s);
      } while (u->q.tiles == 0);
    }
  }
  set_piece(plan, cut, c, u);
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
  // CTAs on an SM: with 168 registers a thread nothing is spilled in the loop for up
  // to 128 columns (of rows of 8), with 255 for twice as many.  (A fourth CTA: with 128
  // registers 58 us instead of 37 for 32 tokens of d = 128, spilled; for 64 columns,
  // where nothing is spilled, 27.3 instead of 27.8 for 16 sequences of four rows.)
  static constexpr int kCtas = D * NT <= 128 ? 3 : 2;
  static constexpr int kStages = D * NT <= 128 ? 3 : D == 128 ? 3 : 2;   // tiles of a warp's ring
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
  static constexpr int kSmemBytes = kMlOff + kWarps * kRows * 8;
  static_assert(kSmemBytes * kCtas <= 232448 - 1024 * kCtas, "CTAs per SM");
};

// Copies 16 bytes, or zeros.
__device__ __forceinline__ void cp_async16_or_zeros(uint32_t dst, const uint8_t* src, bool get) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(get ? 16 : 0) : "memory");
}

// Where row x of a unit begins in the output.
template <int D>
__device__ __forceinline__ uint16_t* out_row(const Paged4Params& p, const Unit& at, int x) {
  const int row = at.first_row + x, token = row / p.group;
  return p.out + (static_cast<long long>(at.q.start + token) * p.h + at.hk * p.group + row - token * p.group) * D;
}

// The slot of piece i of a unit.  A run has two: for the unit in which it ends, and
// for the one in which it begins.
__device__ __forceinline__ int slot_of(const Unit& at, int i) { return 2 * (at.first_run + i) + (i == 0 ? 1 : 0); }

// The whole block: pieces i0, i0 + step, .. (n of them) merged into the output, or
// into piece i0's slot.  A thread takes kVectors vectors of four columns, kAhead
// pieces at a time, the first asked for together with the statistics.  (A function of
// its own, or its registers cost the loop over the keys some.)
template <int D, int R>
__device__ __noinline__ void merge_pieces(const Paged4Params& p, const Unit& at, float2* stats, int i0, int step, int n,
                                          bool final) {
  constexpr int kAhead = 8, kVectors = R * (D / 4) >= 2 * kThreads ? 2 : 1;
  const int rows = at.rows, all = rows * (D / 4);
  auto slot = [&](int i) { return p.slots + static_cast<long long>(slot_of(at, i0 + i * step)) * p.slot_bytes; };
  for (int x0 = threadIdx.x; x0 < (all + kThreads - 1) / kThreads * kThreads; x0 += kVectors * kThreads) {
    float4 acc[kVectors], v[kVectors][kAhead];
    float mm[kVectors], ll[kVectors];
    int row[kVectors];
    auto ask = [&](int i1) {
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
#pragma unroll
        for (int y = 0; y < kVectors; ++y)
          if (i1 + e < n && x0 + y * kThreads < all)
            v[y][e] = __ldcg(reinterpret_cast<const float4*>(slot(i1 + e)) + x0 + y * kThreads);
    };
    ask(0);
    if (x0 == static_cast<int>(threadIdx.x)) {
      for (int x = threadIdx.x; x < n * R; x += kThreads)    // [piece][row]
        if (x % R < rows) stats[x] = __ldcg(reinterpret_cast<const float2*>(slot(x / R) + R * D * 4) + x % R);
      __syncthreads();
    }
#pragma unroll
    for (int y = 0; y < kVectors; ++y) {
      row[y] = min((x0 + y * kThreads) / (D / 4), rows - 1);
      acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
      mm[y] = -INFINITY;
      ll[y] = 0.f;
    }
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int y = 0; y < kVectors; ++y) mm[y] = fmaxf(mm[y], stats[i * R + row[y]].x);
    for (int i1 = 0; i1 < n; i1 += kAhead) {
      if (i1 > 0) ask(i1);
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        if (i1 + e >= n) continue;
#pragma unroll
        for (int y = 0; y < kVectors; ++y) {
          const float2 one = stats[(i1 + e) * R + row[y]];
          const float f = weight(one.x, mm[y] == -INFINITY ? 0.f : mm[y]);
          ll[y] = fmaf(one.y, f, ll[y]);
          acc[y].x = fmaf(v[y][e].x, f, acc[y].x);
          acc[y].y = fmaf(v[y][e].y, f, acc[y].y);
          acc[y].z = fmaf(v[y][e].z, f, acc[y].z);
          acc[y].w = fmaf(v[y][e].w, f, acc[y].w);
        }
      }
    }
#pragma unroll
    for (int y = 0; y < kVectors; ++y) {
      const int x = x0 + y * kThreads, col = x % (D / 4) * 4;
      if (x >= all) continue;
      if (final) {
        const float f = ll[y] > 0.f ? p.v_unit / ll[y] : 0.f;
        *reinterpret_cast<uint2*>(out_row<D>(p, at, row[y]) + col) =
            make_uint2(pack_bf16x2(acc[y].x * f, acc[y].y * f), pack_bf16x2(acc[y].z * f, acc[y].w * f));
      } else {
        // (this thread alone reads and writes these columns)
        uint8_t* dst = slot(0);
        reinterpret_cast<float4*>(dst)[x] = acc[y];
        if (col == 0) reinterpret_cast<float2*>(dst + R * D * 4)[row[y]] = make_float2(mm[y], ll[y]);
      }
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NCfg<D, NT>::kCtas) sdpa_paged4_few(const __grid_constant__ Paged4Params p) {
  using C = NCfg<D, NT>;
  constexpr int R = C::kRows;
  constexpr int KS = D / 16;                                 // steps of 16 columns
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Schedule sched;
  __shared__ Unit at;                                        // (what is wanted at the ends of pieces only is no register's)
  __shared__ int last_one, more;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::kStages * C::kTile;
  // With a second kernel for the other sequences, which begins beside this one, the
  // kernel before has to be over first.
  if (p.few_rows == INT_MAX) griddep_launch_dependents();
  griddep_wait();
  if (p.few_rows != INT_MAX) griddep_launch_dependents();

  const Plan<R> plan(p);
  const int cta = static_cast<int>(blockIdx.x);
  if (!find_place<R>(plan, &sched, &at, cta) || at.begin == LLONG_MAX) return;

  const bool windowed = p.window < INT_MAX;
  // A word that counts published pieces: this call's number and the count.  Every
  // run that has a piece puts the number there long before the piece is done, so
  // that counting is one addition (counting from whatever was there took a
  // compare-and-swap for each of the pieces that come at once, 13 us for 16).
  auto open_count = [&](unsigned long long* count) {
    unsigned long long old = 0, seen;
    while ((seen = atomicCAS(count, old, p.call)) != old && (seen & ~0xffffull) != p.call) old = seen;
  };
  while (true) {
    const int rows = at.rows, first_row = at.first_row;
    auto out_of = [&](int x) { return out_row<D>(p, at, x); };
    if (at.tiles.count == 0 && at.begin >= sched.cut.begin(cta)) {
      // nothing to see: rows of zeros
      for (int x = tid; x < rows * (D / 4); x += kThreads)
        *reinterpret_cast<uint2*>(out_of(x / (D / 4)) + x % (D / 4) * 4) = make_uint2(0u, 0u);
    }
    if (at.kt1 > at.kt0) {
      const int mine = (at.kt1 - at.kt0 - warp + kWarps - 1) / kWarps;   // tiles of this warp
      const int hi_pos = at.hi_pos;
      const int hidden = windowed ? max(at.first_pos, 0) - p.window : -1;   // up to here nobody sees what is no sink
      auto key_of = [&](int i) {                             // of tile i
        const int kt = at.kt0 + warp + i * kWarps;
        return (kt < at.tiles.head ? kt : kt + at.tiles.first - at.tiles.head) << kKeysShift;
      };
      // pieces in groups, those of a group merged first where there are many
      auto radix_of = [&]() {
        int radix = at.of;
        if (radix > kTogether)
          for (radix = 4; radix * radix < at.of;) ++radix;
        return radix;
      };
      // ---- Q: row 8 nt + g, columns [t D / 4, + D / 4)
      uint2 raw[NT][KS];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int x = nt * 8 + g;
        const int token = (first_row + (x < rows ? x : 0)) / p.group;
        const int head = first_row + (x < rows ? x : 0) - token * p.group;
        const uint2* src = reinterpret_cast<const uint2*>(
            p.q + static_cast<long long>(at.q.start + token) * p.q_stride + (at.hk * p.group + head) * D + t * (D / 4));
#pragma unroll
        for (int k = 0; k < KS; ++k) raw[nt][k] = x < rows ? src[k] : make_uint2(0u, 0u);
      }
      // ---- copies.  A lane holds the page of one of this warp's next 32 tiles (of rows
      // 0 .. 15 and 16 .. 31 of it, with pages of 16): -1 where nothing is copied.
      const int32_t* pages = p.page_table + static_cast<long long>(at.s) * p.pages_per_seq;
      int page0 = -1, page1 = -1;
      auto page_at = [&](int key) -> int {
        // a page of which no row sees anything is not looked at
        if (key > hi_pos || (key + min(1 << p.page_shift, kKeys) - 1 <= hidden && key >= p.sinks)) return -1;
        const int page = pages[key >> p.page_shift];
        if (page >= 0 && page < p.n_pages) return page;
        // one outside the cache is reported and read as zeros
        atomicOr(p.status, kStatusBadPage);
        return -1;
      };
      auto ask = [&](int i) {                                // for tiles i .. i + 31
        page0 = page1 = -1;
        if (i + lane < mine) {
          const int key = key_of(i + lane);
          page0 = page_at(key);
          if (p.page_shift < kKeysShift) page1 = page_at(key + 16);
        }
        __syncwarp();
      };
      const uint32_t dst_lane = smem_u32(ring) + lane * 16;
      const uint8_t *k_head = p.k_pages + at.hk * p.page_bytes, *v_head = p.v_pages + at.hk * p.page_bytes;
      auto issue = [&](int i) {
        if (i < mine) {
          if ((i & 31) == 0 && i > 0) ask(i);
          const uint32_t dst = dst_lane + i % C::kStages * C::kTile;
          auto copy = [&](uint32_t to, const uint8_t* from, auto chunks, bool get) {
            constexpr int n = decltype(chunks)::value;       // of 16 bytes
#pragma unroll
            for (int y = 0; y < n; y += 32)
              if (n >= 32 || lane < n) cp_async16_or_zeros(to + y * 16, from + y * 16, get);
          };
          // (the scales of K and V by one instruction where 32 lanes do)
          auto rows = [&](auto share, int page, long long r, uint32_t codes_to, uint32_t scales_to) {
            constexpr int n = decltype(share)::value;         // of the tile's rows, one in n
            std::integral_constant<int, C::kCodes / 16 / n> codes;
            std::integral_constant<int, C::kScales / 16 / n> scales;
            const bool get = page >= 0;
            const long long off = get ? page * p.page_stride : 0;
            const uint8_t *k = k_head + off + lane * 16, *v = v_head + off + lane * 16;
            const long long at_codes = r * (D / 2), at_scales = r * (D / 16);
            copy(dst + codes_to, k + at_codes, codes, get);
            copy(dst + C::kHalf + codes_to, v + at_codes, codes, get);
            const long long skip = (static_cast<long long>(D / 2) << p.page_shift) + at_scales;
            if constexpr (scales <= 16) {
              const bool second = lane >= 16;
              const uint8_t* from = (second ? v - 256 : k) + skip;
              if ((lane & 15) < scales)
                cp_async16_or_zeros(dst + C::kCodes + scales_to + (second ? C::kHalf - 256 : 0), from, get);
            } else {
              copy(dst + C::kCodes + scales_to, k + skip, scales, get);
              copy(dst + C::kHalf + C::kCodes + scales_to, v + skip, scales, get);
            }
          };
          const int first = __shfl_sync(0xffffffffu, page0, i & 31);
          if (p.page_shift >= kKeysShift) {
            rows(std::integral_constant<int, 1>{}, first, key_of(i) & ((1 << p.page_shift) - 1), 0, 0);
          } else {
            const int second = __shfl_sync(0xffffffffu, page1, i & 31);
            rows(std::integral_constant<int, 2>{}, first, 0, 0, 0);
            rows(std::integral_constant<int, 2>{}, second, 0, C::kCodes / 2, C::kScales / 2);
          }
        }
        cp_async_commit();
      };
      ask(0);
#pragma unroll
      for (int i = 0; i < C::kStages - 1; ++i) issue(i);
      if (at.of > 1 && tid == kThreads - 1) {
        const int radix = radix_of();
        open_count(p.counts + slot_of(at, (cta - at.first_run) / radix * radix));
        if (radix < at.of) open_count(p.counts + 2 * p.runs + at.first_run);
      }
      uint32_t qf[KS][NT][2];
      float sc[NT][2];                                       // of columns 2 t, 2 t + 1: score to log2 units
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint2 v = raw[nt][k];
          top = max(max(top, max(v.x & 0x7fffu, v.y & 0x7fffu)), max(v.x >> 16 & 0x7fffu, v.y >> 16 & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = static_cast<int>(top >> 7);           // biased; rows of zeros, infinities and NaN stay
        const int up = top == 0 || ex == 255 ? 0 : max(-120, min(120, 13 + 127 - ex));
        const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint2 v = raw[nt][k];
          qf[k][nt][0] = pack_f16x2(__uint_as_float(v.x << 16) * f, __uint_as_float(v.x & 0xffff0000u) * f);
          qf[k][nt][1] = pack_f16x2(__uint_as_float(v.y << 16) * f, __uint_as_float(v.y & 0xffff0000u) * f);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) sc[nt][c] = score_factor(p, __shfl_sync(0xffffffffu, up, (2 * t + c) * 4));
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

      for (int i = 0; i < mine; ++i) {
        cp_async_wait<C::kStages - 2>();
        __syncwarp();                                        // (for all lanes; and the stage before has been read)
        issue(i + C::kStages - 1);
        uint8_t* ks = ring + i % C::kStages * C::kTile;
        const int key0 = key_of(i);
        const bool edge = key0 + kKeys - 1 > at.first_pos || (windowed && key0 <= hi_pos - p.window);
        if (edge) {
          // what no row sees may be anything: its weight is zero, but zero times a NaN
          // is not, so its scales are cleared (a lane for each key)
          const int j = key0 + lane;
          if (j > hi_pos || (j <= hidden && j >= p.sinks)) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x) ks[C::kHalf + C::kCodes + lane * (D / 16) + x] = 0;
          }
          __syncwarp();
        }
        // ---- scores of keys g and g + 8 of each half in rows 2 t, 2 t + 1
        float s[2][NT][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          {
            const uint8_t* kh = ks + half * (16 * (D / 2));
            constexpr int kB = D / 8, kW = kB < 4 ? 1 : kB / 4;   // bytes, words of a lane's columns
            constexpr int kSB = D >= 64 ? D / 64 : 1;             // scales of a lane's columns
            const uint8_t* scales = kh + C::kCodes - half * (16 * (D / 2 - D / 16)) + (D >= 64 ? t * kSB : t * D / 64);
            uint32_t w[2][kW], sw[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const int row = hh * 8 + g;
              load_bytes<kB>(kh + row * (D / 2) + t * kB, w[hh]);
              uint32_t sb[1];
              load_bytes<kSB>(scales + row * (D / 16), sb);
              sw[hh] = sb[0];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[half][nt][e] = 0.f;
#pragma unroll
            for (int wi = 0; wi < kW; ++wi) {
              uint32_t a[2][4];
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                expand4(w[hh][wi], a[hh]);
                // columns t D / 4 + 8 wi ..: block wi / 2 of the lane's
                const uint32_t sc2 = scales_f16x2(__byte_perm(sw[hh], 0, 0x11 * (wi / 2)));
#pragma unroll
                for (int e = 0; e < 4; ++e) a[hh][e] = mul_f16x2(a[hh][e], sc2);
              }
              constexpr int kSteps = kB < 4 ? 1 : 2;
#pragma unroll
              for (int e = 0; e < kSteps; ++e)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16(s[half][nt], a[0][2 * e], a[1][2 * e], a[0][2 * e + 1], a[1][2 * e + 1], qf[wi * 2 + e][nt][0],
                          qf[wi * 2 + e][nt][1]);
            }
          }
          if (edge) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int x = nt * 8 + 2 * t + c;            // this row's position (-1: no row)
                const int pp = x < rows ? at.q.len - at.q.n + (first_row + x) / p.group : -1;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  const int j = key0 + half * 16 + hh * 8 + g;
                  if (j > pp || (j <= pp - p.window && j >= p.sinks)) s[half][nt][2 * hh + c] = -INFINITY;
                }
              }
          }
        }
        {
          // ---- the references (m): they move when a score is too far above one
          bool need = false;
          float top[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              top[nt][c] = fmaxf(fmax3(s[0][nt][c], s[0][nt][2 + c], s[1][nt][c]), s[1][nt][2 + c]) * sc[nt][c];
              need |= top[nt][c] > m[nt][c] + kWeightMost;
            }
          if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float x = top[nt][c];
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
                x = fmaxf(x - kWeightUp, m[nt][c]);
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
        }
        // ---- weights, turned so that a lane holds two keys of a row
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float p0 = ex2_approx(fmaf(s[x >> 1][nt][2 * (x & 1)], sc[nt][0], -m0));
            const float p1 = ex2_approx(fmaf(s[x >> 1][nt][2 * (x & 1) + 1], sc[nt][1], -m1));
            l[nt][0] += p0;
            l[nt][1] += p1;
            pb[x >> 1][nt][x & 1] = transpose8x8(pack_f16x2(p0, p1));
          }
        }
        const uint8_t* vs = ks + C::kHalf;
#pragma unroll
        for (int half = 0; half < 2; ++half, vs += 16 * (D / 2)) {
          // ---- O^T += V^T P: keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
          constexpr int kB = D / 16, kW = kB < 4 ? 1 : kB / 4;
          constexpr int kSB = D >= 128 ? D / 128 : 1;
          const uint8_t* scales = vs + C::kCodes - half * (16 * (D / 2 - D / 16)) + (D >= 128 ? g * kSB : g * D / 128);
          uint32_t w[4][kW], sw[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = 2 * t + (x & 1) + (x >> 1) * 8;
            load_bytes<kB>(vs + row * (D / 2) + g * kB, w[x]);
            uint32_t sb[1];
            load_bytes<kSB>(scales + row * (D / 16), sb);
            sw[x] = sb[0];
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
              const uint32_t sc2 = scales_f16x2(__byte_perm(sw[2 * y], sw[2 * y + 1], blk | (4 + blk) << 4));
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
                mma_f16(o[wi * 4 + e][nt], a[0][e], a[1][e], a[2][e], a[3][e], pb[half][nt][0], pb[half][nt][1]);
          }
        }
      }
      cp_async_wait<0>();                                    // (groups without copies)
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
      const bool whole = at.of == 1;
      float* xo = reinterpret_cast<float*>(smem + C::kRing);
      uint8_t* own = whole ? nullptr : p.slots + static_cast<long long>(slot_of(at, cta - at.first_run)) * p.slot_bytes;
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
        __syncthreads();
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
      if (!whole) {
        // ---- published; the last of a group of pieces merges it, the last
        // group's all groups
        const int radix = radix_of(), of = at.of;
        const int group = (cta - at.first_run) / radix, groups = (of + radix - 1) / radix;
        // counts up and tells everybody whether this was the last of `all`
        auto arrive = [&](unsigned long long* count, int all) -> bool {
          __threadfence();
          __syncthreads();
          if (tid == 0) {
            last_one = static_cast<int>(atomicAdd(count, 1ull) & 0xffff) + 1 == all;
            __threadfence();
            if (last_one) *count = 0;
          }
          __syncthreads();
          return last_one != 0;
        };
        const int i0 = group * radix, n = min(radix, of - i0);
        if (arrive(p.counts + slot_of(at, i0), n)) {
          float2* stats = reinterpret_cast<float2*>(smem + C::kRing);   // (the exchange memory)
          merge_pieces<D, R>(p, at, stats, i0, 1, n, groups == 1);
          if (groups > 1 && arrive(p.counts + 2 * p.runs + at.first_run, groups))
            merge_pieces<D, R>(p, at, stats, 0, radix, groups, true);
        }
      }
    }
    __syncthreads();                                         // (the unit and the exchange memory have been read)
    if (tid == 0) more = next_unit<R>(plan, sched.cut, cta, &at);
    __syncthreads();
    if (more == 0) break;
  }
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

// Rows of a row tile: 8 where the sequences have that many on average.  (16 sequences of
// 4 rows: 28 us, and 34 with tiles of 16; of 16 rows: 26.9 with 16, 27.5 with 8.)
int paged4_rows(int group, int n_tokens, int b) {
  return 1ll * group * n_tokens <= 8ll * b ? 8 : 16;
}

int paged4_resident_ctas(int d, int rows) { return d * rows <= 1024 ? 3 : 2; }

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
