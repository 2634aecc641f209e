// Attention over a paged cache held in 4 bits (paged4.cu gives the format) for
// sequences with many rows: chunks of a prompt and whole prompts.  paged4_attn.cu
// has the few-rows kernel, which takes the other sequences.
//
// sdpa_paged4_many<D>: a UNIT is (sequence, key-value head, row tile), a row being
// a new token's query head of the group; a row tile has kSub times 128 rows, so that
// a key tile is expanded once for all of them.  All units' walks laid end to end are
// cut into equal runs, one for each CTA (one on an SM), by the keys that the rows
// see; the cut is worked out on the device.  A piece of a unit that is cut is
// published as fp32 (O, m, l), and the run that publishes the last piece merges them
// in the order of their keys: results repeat bit by bit, no run waits for another.
//
// Roles: two warps copy K's and V's pages as they are held (cp.async, 16 bytes a
// lane), the first works out the units too; four expand codes and scales to fp16
// (exact) into the tensor core's swizzled operands; one for each 128 rows issues the
// products (tcgen05.mma, kind::f16: S = Q K^T into tensor memory, O += P V with P
// from there); four for each 128 rows do the softmax, a row a thread.  Queries are
// scaled by a power of two for each row to fit fp16, the softmax weights are taken
// against a reference that lags and rounded to fp16 (paged.cuh).
//
// What bounds it: a key tile (128 keys, 256 rows, d = 128) takes 2048 clock cycles of
// the tensor core, and 3800 here.  Of the chain of each half of the rows a row's
// softmax takes 1500 from S to P (128 exponentials, maximum, sum, tensor memory to
// registers and back) and its products 1500 instead of 1024, as they share the shared
// memory with the warps that expand; the rest is waiting for the other half's
// products.  To the tiles come a run's beginning (place, Q, the first tile: 10 us) and
// its end (pieces out and merged: up to 15 us).  4 chunks of 512 tokens behind 7680
// positions (16 query heads, 4 of keys, d = 128): 132 us, half of the tensor core's
// peak rate.  One chunk of 500 tokens over 8000: 70 us, 229 in the few-rows kernel.
#include <algorithm>
#include <atomic>
#include <climits>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace sdpa {
namespace {

// What a unit costs beside its keys (loading Q, storing O), in keys.  (A prompt of 4096: 99, 90 and
// 94 us with 256, 512 and 1024; 16 sequences of 128 rows 54, 50 and 52.)
constexpr int kStartKeys = 512;
// Of a run, at least.  (3 chunks of 200 tokens of d = 256: 60.5, 60.8 and 62.3 us with 256, 512 and 1024.)
constexpr int kMinRunKeys = 512;

// ------------------------------------------------------------------ schedule
struct Seq {
  int start, n, len, tiles;                // tiles: row tiles
};

// Most counts fit 32 bits, where a division costs a tenth of one in 64.
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// Items are keys x group.  A unit is start items and then those of the keys that its
// last row sees, were the tile full: group (len - n) + (r + 1) R, or what a window
// holds of them.  So the sum over row tiles has a closed form.
template <int R, int kBNShift>
struct Plan {
  static constexpr int kBN = 1 << kBNShift;                  // keys of a tile
  const Paged4Params& p;
  __device__ explicit Plan(const Paged4Params& params) : p(params) {}
  // (What the caller's kernels wrote is read past L1, here and below: this kernel does not
  // wait for them itself, the one before it has.)
  __device__ __forceinline__ int start_of(int s) const { return __ldcg(p.q_starts + s); }
  // rows of a head
  __device__ __forceinline__ long long rows(int s) const {
    const int start = min(max(start_of(s), 0), p.n_tokens);
    return 1ll * (min(max(start_of(s + 1), start), p.n_tokens) - start) * p.group;
  }
  __device__ __forceinline__ Seq seq(int s) const {
    Seq q;
    const int cap = p.pages_per_seq << p.page_shift;
    q.start = min(max(start_of(s), 0), p.n_tokens);
    q.n = min(max(start_of(s + 1), q.start), p.n_tokens) - q.start;
    q.len = min(max(__ldcg(p.kv_lengths + s), 0), cap);
    const long long rows = 1ll * q.n * p.group;
    q.tiles = rows > p.few_rows ? static_cast<int>((rows + R - 1) / R) : 0;
    return q;
  }
  __device__ __forceinline__ long long start() const { return 1ll * kStartKeys * p.group; }
  __device__ __forceinline__ long long most() const {
    return p.window < INT_MAX ? (1ll * p.window + p.sinks + 2 * kBN) * p.group + R : LLONG_MAX / 4;
  }
  // row tiles that see no more than a window holds
  __device__ __forceinline__ long long growing(const Seq& q, long long a) const {
    const long long m = most() - a;
    return m <= 0 ? 0 : min(static_cast<long long>(q.tiles), m / R);   // (R: a power of two)
  }
  __device__ __forceinline__ long long base(const Seq& q) const { return 1ll * max(q.len - q.n, 0) * p.group; }
  __device__ __forceinline__ long long cost(const Seq& q, int r) const {
    return start() + min(base(q) + (r + 1ll) * R, most());
  }
  // of row tiles 0 .. f - 1
  __device__ __forceinline__ long long before(const Seq& q, long long f) const {
    const long long a = base(q), g = min(f, growing(q, a));
    return start() * f + a * g + R * (g * (g + 1) / 2) + (f - g) * (f > g ? most() : 0);
  }
};

// The key tiles that rows of positions lo .. hi see: tiles [0, head), then those
// from `first` on.
struct Tiles {
  int head, first, count;
};

struct Unit {
  Seq q;
  int s, hk, r;
  long long begin;                         // the unit's first item
  Tiles tiles;
  int kt0, kt1;                            // the piece, of tiles.count key tiles
  int first_run, of;                       // the unit's pieces are those of runs first_run .. first_run + of - 1
  int first_pos, hi_pos;                   // positions of the first and the last row
  int first_row, rows;                     // of the sequence's rows for this head (no rows: no further unit)
  bool zeros;                              // nothing to see, and this run's
  // which key tile the piece's tile i is
  __device__ __forceinline__ int tile(int i) const {
    const int kt = kt0 + i;
    return kt < tiles.head ? kt : kt + tiles.first - tiles.head;
  }
};

// The runs: [begin(c), begin(c + 1)) of all items.
struct Cut {
  long long each;
  int over, runs;
  __device__ long long begin(int c) const { return each * c + min(c, over); }
  __device__ int run_of(long long x) const {
    const long long longer = over * (each + 1);
    return static_cast<int>(x < longer ? divide(x, each + 1) : over + divide(x - longer, each));
  }
};

template <int R, int S>
__device__ void set_piece(const Plan<R, S>& plan, const Cut& cut, int c, Unit* u) {
  const Paged4Params& p = plan.p;
  constexpr int kBN = 1 << S;
  const Seq& q = u->q;
  const long long rows = 1ll * q.n * p.group, row0 = 1ll * u->r * R;
  u->first_row = static_cast<int>(row0);
  u->rows = static_cast<int>(min(static_cast<long long>(R), rows - row0));
  u->first_pos = q.len - q.n + static_cast<int>(divide(row0, p.group));
  u->hi_pos = q.len - q.n + static_cast<int>(divide(row0 + u->rows - 1, p.group));
  Tiles t{0, 0, 0};
  if (u->hi_pos >= 0) {
    if (p.window < INT_MAX) {
      t.first = max(max(u->first_pos, 0) - p.window + 1, 0) >> S;
      t.head = min((min(p.sinks, u->hi_pos + 1) + kBN - 1) >> S, t.first);
    }
    t.count = t.head + (u->hi_pos >> S) - t.first + 1;
  }
  u->tiles = t;
  // Key tiles before item y of the unit, in proportion; all of them at once where a tile
  // would be more than a run (rows at negative positions see less than they count for).
  const long long items = plan.cost(q, u->r) - plan.start();
  const bool single = items > t.count * cut.each;
  auto tile_at = [&](long long y) -> int {
    y -= plan.start();
    return y <= 0 ? 0 : single ? t.count : static_cast<int>(min(static_cast<long long>(t.count), divide(y * t.count, items)));
  };
  const long long y0 = cut.begin(c) - u->begin, y1 = cut.begin(c + 1) - u->begin;
  u->kt0 = tile_at(y0);
  u->kt1 = tile_at(y1);
  u->first_run = c;
  u->of = 1;
  u->zeros = t.count == 0 && y0 <= 0;
  if (u->kt1 > u->kt0 && u->kt1 - u->kt0 < t.count) {
    // (a run between the first and the last is longer than a tile, so it has one)
    int first = cut.run_of(u->begin), last = cut.run_of(u->begin + plan.cost(q, u->r) - 1);
    while (tile_at(cut.begin(first + 1) - u->begin) == 0) ++first;
    while (tile_at(cut.begin(last) - u->begin) == t.count) --last;
    u->first_run = first;
    u->of = last - first + 1;
  }
}

struct Schedule {
  long long items[16];
  Cut cut;
};

// The whole block: the cut, and the unit in which run c begins.  Returns false
// when there is no such run.
template <int R, int S>
__device__ bool find_place(const Plan<R, S>& plan, Schedule* sh, Unit* first, int c) {
  const Paged4Params& p = plan.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
  const int per = (p.b + threads - 1) / threads;
  const int s0 = min(tid * per, p.b), s1 = min(s0 + per, p.b);
  long long items = 0;
  for (int s = s0; s < s1; ++s) {
    const Seq q = plan.seq(s);
    items += plan.before(q, q.tiles) * p.h_kv;
  }
  long long to = items;                                      // of the threads up to this one
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long i = __shfl_up_sync(0xffffffffu, to, x);
    if (lane >= x) to += i;
  }
  if (lane == 31) sh->items[warp] = to;
  if (tid == 0) first->begin = LLONG_MAX;                    // (no unit, should the lengths change meanwhile)
  __syncthreads();
  long long all = 0;
  for (int w = 0; w < threads / 32; ++w) {
    if (w == warp) to += all;
    all += sh->items[w];
  }
  if (all == 0) return false;
  Cut cut;
  const long long least = 1ll * kMinRunKeys * p.group;
  cut.runs = static_cast<int>(min(static_cast<long long>(p.runs), max(1ll, divide(all, least))));
  cut.each = divide(all, cut.runs);
  cut.over = static_cast<int>(all - cut.each * cut.runs);
  if (c >= cut.runs) return false;
  if (tid == 0) sh->cut = cut;
  const long long x = cut.begin(c);
  long long before = to - items;
  if (items > 0 && before <= x && x < to) {
    for (int s = s0; s < s1; ++s) {
      const Seq q = plan.seq(s);
      const long long head = plan.before(q, q.tiles), here = head * p.h_kv;
      if (x < before + here) {
        Unit u;
        u.q = q;
        u.s = s;
        u.hk = static_cast<int>(divide(x - before, head));
        before += u.hk * head;
        int lo = 0, hi = q.tiles;                            // the last row tile that begins at or before x
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (before + plan.before(q, mid) <= x) lo = mid;
          else hi = mid;
        }
        u.r = lo;
        u.begin = before + plan.before(q, lo);
        set_piece(plan, cut, c, &u);
        *first = u;
        break;
      }
      before += here;
    }
  }
  __syncthreads();
  return true;
}

// One thread: the unit after *u, false if there is none of run c's.
template <int R, int S>
__device__ __forceinline__ bool next_unit(const Plan<R, S>& plan, const Cut& cut, int c, Unit* u) {
  u->begin += plan.cost(u->q, u->r);
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

// ---------------------------------------------------------------------- kernel
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t byte) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(byte * 0x101u)));
  return r;
}
// Eight codes times a scale, as fp16.
__device__ __forceinline__ uint4 expand8(uint32_t w, uint32_t scale2) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(r[i]) : "r"(scale2));
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// Copies 16 bytes, or zeros.
__device__ __forceinline__ void cp_async16_or_zeros(uint32_t dst, const uint8_t* src, bool get) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(get ? 16 : 0) : "memory");
}
// This thread's arrival on `bar` once the copies that it has asked for are done.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Instruction descriptor, kind::f16: fp16 A and B (formats 0), fp32 D.
constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((static_cast<uint32_t>(N) >> 3) << 17) |
         ((static_cast<uint32_t>(M) >> 4) << 24);
}
__device__ __forceinline__ float weight(float m, float sub) { return ex2_approx(m - sub); }

template <int D>
struct WCfg {
  static constexpr int kSub = D <= 128 ? 2 : 1;              // 128 rows each
  // Keys of a tile and score buffers: with two times 128 rows one's softmax runs beside
  // the other's products, and a tile of 128 keys costs the tensor core 2048 clock cycles
  // (d = 128) where two of 64 cost 2560, as a product of 64 columns is bound by reading A.
  static constexpr int kBNShift = kSub == 2 ? 7 : 6, kBN = 1 << kBNShift, kBufs = kSub == 2 ? 1 : 2;
  static constexpr int kRows = 128 * kSub;
  static constexpr int kSoftmaxWarps = 4 * kSub;
  static constexpr int kExpandWarp = kSoftmaxWarps;          // the first of four
  static constexpr int kMmaWarp = kExpandWarp + 4;           // one for each 128 rows
  static constexpr int kCopyWarp = kMmaWarp + 2;             // K's, and V's; K's works out the units too
  static constexpr int kThreads = 32 * (kMmaWarp + 4);       // whole warpgroups, for the registers' split
  static constexpr int kBoxCols = D < 64 ? D : 64;
  static constexpr int kBoxes = D / kBoxCols;
  static constexpr int kRowBytes = kBoxCols * 2;
  static constexpr uint32_t kLayout = kRowBytes == 128 ? 2u : (kRowBytes == 64 ? 4u : 6u);
  static constexpr uint32_t kSBO = 8 * kRowBytes;
  static constexpr int kStepsPerRow = kRowBytes / 32;
  static constexpr int kQBox = 128 * kRowBytes;
  static constexpr int kQBytes = kBoxes * kQBox;             // of 128 rows
  static constexpr int kKVBytes = kBN * D * 2;               // a tile of K or of V
  // a tile lies as [8 rows][column block][row of the eight]
  static constexpr int kGroupBytes = kBoxes * kSBO;
  static constexpr int kRing = D <= 64 ? 3 : 2;
  static constexpr int kKOff = kSub * kQBytes;
  static constexpr int kVOff = kKOff + kRing * kKVBytes;
  // A tile as it is held, on its way to be expanded: K's codes and scales, V's
  static constexpr int kCodes = kBN * D / 2, kScales = kBN * D / 16;
  static constexpr int kRawOff = kVOff + kRing * kKVBytes;
  static constexpr int kRawHalf = kCodes + kScales;
  static constexpr int kRawSlots = D == 256 ? 2 : 3;         // halves (K or V of a tile) under way, in turn
  static constexpr int kBarOff = kRawOff + kRawSlots * kRawHalf;
  // A warp's rows on their way to the output lie over its own rows of Q, where they fit:
  // the other warps of the 128 rows may be at the next unit's Q already.
  static constexpr int kTurnRow = 64 + 16;
  static constexpr int kTurnSlot = 32 * kTurnRow;
  static constexpr int kWarpQ = 32 * kRowBytes;              // of a column block
  static constexpr bool kTurns = kTurnSlot <= kWarpQ;
  // q_full, o_full, o_last, o_free, s_full, p_full [2]; k_full, v_full, k_empty, v_empty [R];
  // ready, done [2]; meet, drain; raw_full, raw_empty [3]; turn [2]
  static constexpr int kNumBars = 12 + 4 * kRing + 4 + 2 + 6 + 2;
  static constexpr int kSmemBytes = kBarOff + kNumBars * 8 + 16 + 1024;
  static constexpr int kOChunk = D < 32 ? D : 32;
  static constexpr uint32_t kSubCols = 128 + (D < 32 ? 32 : D);
  static constexpr uint32_t kOCol = 128;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kSub * kSubCols <= kTmemCols, "tensor memory");
  static_assert(kSmemBytes <= 232448 - 1024, "shared memory");
  static_assert(kKOff % 1024 == 0 && kVOff % 1024 == 0 && kKVBytes % 512 == 0, "alignment");
  static constexpr uint32_t kIdescS = idesc_f16(128, kBN, false);
  static constexpr uint32_t kIdescPV = idesc_f16(128, D, true);
  static constexpr uint32_t kDescHi = (kSBO >> 4) | (1u << 14) | (kLayout << 29);
  static constexpr uint32_t kDescHiKV = (kGroupBytes >> 4) | (1u << 14) | (kLayout << 29);
  // registers a thread: the launch's 128 (kSub == 2) are split, a row's scores being 128 of them
  // (4 chunks of 512 tokens: 134 us; with 192, 72, 56 136, with 176, 96, 64 139, with 208, 32, 64 138)
  static constexpr int kSoftmaxRegs = 200, kExpandRegs = 48, kRestRegs = 64;
  static_assert(kSub == 1 || 2 * kSoftmaxRegs + kExpandRegs + kRestRegs <= 512, "registers");
};

// The slot of piece i of a unit.  A run has two: for the unit in which it ends, and
// for the one in which it begins.
__device__ __forceinline__ int slot_of(const Unit& at, int i) { return 2 * (at.first_run + i) + (i == 0 ? 1 : 0); }

// O columns [c kOChunk, + kOChunk) of a warp's rows (`rows` of the 32), a lane for each,
// times f into the output: turned through shared memory, four lanes write 64 bytes of a row.
template <int D>
__device__ __forceinline__ void store_rows(uint8_t* turn, uint16_t* out, int rows, int c,
                                           const uint32_t (&o)[WCfg<D>::kOChunk], float f) {
  using C = WCfg<D>;
  const int lane = threadIdx.x & 31;
  if constexpr (!C::kTurns) {
    if (lane < rows)
      for (int e = 0; e < C::kOChunk / 2; ++e)
        reinterpret_cast<uint32_t*>(out)[c * (C::kOChunk / 2) + e] =
            pack_bf16x2(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
  } else {
    uint4* mine = reinterpret_cast<uint4*>(turn + lane * C::kTurnRow);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      mine[e] = make_uint4(pack_bf16x2(__uint_as_float(o[e * 8 + 0]) * f, __uint_as_float(o[e * 8 + 1]) * f),
                           pack_bf16x2(__uint_as_float(o[e * 8 + 2]) * f, __uint_as_float(o[e * 8 + 3]) * f),
                           pack_bf16x2(__uint_as_float(o[e * 8 + 4]) * f, __uint_as_float(o[e * 8 + 5]) * f),
                           pack_bf16x2(__uint_as_float(o[e * 8 + 6]) * f, __uint_as_float(o[e * 8 + 7]) * f));
    __syncwarp();
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int x = (lane >> 2) + 8 * y;                     // row of this warp (its lane knows where it goes)
      const long long at_out = __shfl_sync(0xffffffffu, reinterpret_cast<long long>(out), x);
      const uint4 v = *reinterpret_cast<const uint4*>(turn + x * C::kTurnRow + (lane & 3) * 16);
      if (x < rows) *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(at_out) + c * 32 + (lane & 3) * 8) = v;
    }
    __syncwarp();
  }
}

// A warp's rows of all pieces of a unit, in their order, into the output: a lane for
// each row, the next piece's columns under way while one's are summed.  (A function
// of its own, or its registers cost the loop over the keys some.)
template <int D>
__device__ __noinline__ void merge_rows(const Paged4Params& p, const Unit& at, uint8_t* turn, uint16_t* out, int rows,
                                        int row) {
  using C = WCfg<D>;
  constexpr int kVec = C::kOChunk / 4;
  const int of = at.of;
  const int rw = min(row, at.rows - 1);
  auto slot = [&](int i) { return p.slots + static_cast<long long>(slot_of(at, i)) * p.slot_bytes; };
  auto ml_of = [&](int i) { return __ldcg(reinterpret_cast<const float2*>(slot(i) + C::kRows * D * 4) + rw); };
  float4 acc[kVec], v[2][kVec];
  float2 ml[2];
  auto fetch = [&](int c, int i, float4 (&x)[kVec], float2& w) {
    w = ml_of(i);
    const float4* src = reinterpret_cast<const float4*>(slot(i)) + rw;
#pragma unroll
    for (int e = 0; e < kVec; ++e) x[e] = __ldcg(src + (c * kVec + e) * C::kRows);
  };
  int fc = 0, fi = 0;                                        // of the step that is asked for
  auto next = [&]() {
    if (++fi == of) {
      fi = 0;
      ++fc;
    }
  };
  fetch(fc, fi, v[0], ml[0]);
  next();
  float mm = -INFINITY, sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < of; ++i) mm = fmaxf(mm, ml_of(i).x);
  const float base = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
  for (int i = 0; i < of; ++i) {
    const float2 one = ml_of(i);
    sum = fmaf(one.y, weight(one.x, base), sum);
  }
  const float f = sum > 0.f ? p.v_unit / sum : 0.f;
  int c = 0, i = 0;                                          // of the step that is summed
  auto sum_up = [&](const float4 (&x)[kVec], const float2& w) {
    const float g = weight(w.x, base);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if (i == 0) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      acc[e].x = fmaf(x[e].x, g, acc[e].x);
      acc[e].y = fmaf(x[e].y, g, acc[e].y);
      acc[e].z = fmaf(x[e].z, g, acc[e].z);
      acc[e].w = fmaf(x[e].w, g, acc[e].w);
    }
    if (++i < of) return;
    uint32_t o[C::kOChunk];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      o[4 * e] = __float_as_uint(acc[e].x);
      o[4 * e + 1] = __float_as_uint(acc[e].y);
      o[4 * e + 2] = __float_as_uint(acc[e].z);
      o[4 * e + 3] = __float_as_uint(acc[e].w);
    }
    store_rows<D>(turn, out, rows, c, o, f);
    i = 0;
    ++c;
  };
  const int steps = D / C::kOChunk * of;
#pragma unroll 1
  for (int x = 0; x < steps; x += 2) {
    if (x + 1 < steps) fetch(fc, fi, v[1], ml[1]);
    next();
    sum_up(v[0], ml[0]);
    if (x + 2 < steps) fetch(fc, fi, v[0], ml[0]);
    next();
    if (x + 1 < steps) sum_up(v[1], ml[1]);
  }
}

template <int D>
__global__ void __launch_bounds__(WCfg<D>::kThreads, 1) sdpa_paged4_many(const __grid_constant__ Paged4Params p) {
  using C = WCfg<D>;
  constexpr int R = C::kRing, kBN = C::kBN, kBNShift = C::kBNShift;
  const Plan<C::kRows, kBNShift> plan(p);
  // Drafts and other short rows beside single tokens leave this kernel nothing, which the
  // starts alone tell before anything is set up.  (Looked at where rows are few on average: 16
  // sequences of 16 rows 25.2 us instead of 26.9; looked at in any call a prompt of 4096 took 1.2 us more.)
  if (1ll * p.n_tokens * p.group <= 1ll * p.few_rows * p.b) {
    bool mine = false;
    for (int s = threadIdx.x; s < p.b; s += C::kThreads) mine |= plan.rows(s) > p.few_rows;
    if (__syncthreads_or(mine) == 0) {
      griddep_wait();
      return;
    }
  }
  extern __shared__ uint8_t smem_raw[];
  __shared__ Schedule sched;
  __shared__ Unit units[2];
  __shared__ int last_one;
  const uint32_t raw_u32 = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);
  const uint32_t smem_base = smem_u32(smem);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* o_full = q_full + 2;
  uint64_t* o_last = o_full + 2;           // once a piece, after its last O += P V
  uint64_t* o_free = o_last + 2;           // once a piece, when the softmax warps have read O
  uint64_t* s_full = o_free + 2;           // [sub], or [buffer]
  uint64_t* p_full = s_full + 2;
  uint64_t* k_full = p_full + 2;
  uint64_t* v_full = k_full + R;
  uint64_t* k_empty = v_full + R;
  uint64_t* v_empty = k_empty + R;
  uint64_t* ready = v_empty + R;
  uint64_t* done = ready + 2;
  uint64_t* meet_bar = done + 2;
  uint64_t* drain = meet_bar + 1;
  uint64_t* raw_full = drain + 1;          // half 2 u + y, y = 0 for K and 1 for V of tile u, is in slot (2 u + y) % kRawSlots
  uint64_t* raw_empty = raw_full + 3;
  uint64_t* turn = raw_empty + 3;          // of the warps that issue products
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(turn + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const AbortState ab{abort_flag, p.status};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 128);
      mbar_init(o_full + i, 1);
      mbar_init(o_last + i, 1);
      mbar_init(o_free + i, 128);
      mbar_init(ready + i, 1);
      mbar_init(turn + i, 1);
      mbar_init(done + i, C::kSoftmaxWarps + 4 + C::kSub + 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
    }
    for (int i = 0; i < R; ++i) {
      mbar_init(k_full + i, 128);
      mbar_init(v_full + i, 128);
      mbar_init(k_empty + i, C::kSub);
      mbar_init(v_empty + i, C::kSub);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(raw_full + i, 32);
      mbar_init(raw_empty + i, 4);
    }
    mbar_init(meet_bar, C::kSoftmaxWarps);
    mbar_init(drain, C::kSub);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  // (not before the block holds its tensor memory: the next kernel's block could be
  // given it, and then wait for this grid, which waits for the memory)
  griddep_launch_dependents();
  // The kernel before is the one for the other sequences: all of its blocks had waited for
  // the one before it before this one could begin, so everything that a call reads is in L2.
  // That kernel itself is waited for at the end only.

  const int cta = static_cast<int>(blockIdx.x);
  const bool any = find_place(plan, &sched, &units[0], cta) && units[0].begin != LLONG_MAX;
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (any && warp < C::kSoftmaxWarps) {
    // ------------------------------------------------------------- softmax
    if constexpr (C::kSub == 2) regs_increase<C::kSoftmaxRegs>();
    const int sub = warp >> 2, quarter = warp & 3;
    const int row = sub * 128 + quarter * 32 + lane;         // of the row tile
    const uint32_t lane_base = tmem + sub * C::kSubCols + (static_cast<uint32_t>(quarter * 32) << 16);
    const bool windowed = p.window < INT_MAX;
    auto open_count = [&](unsigned long long* count) {       // (see the few-rows kernel)
      unsigned long long old = 0, seen;
      while ((seen = atomicCAS(count, old, p.call)) != old && (seen & ~0xffffull) != p.call) old = seen;
    };
    int met = 0;
    // all softmax warps, each seeing what the others wrote before
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet_bar);
      return mbar_wait_warp(meet_bar, static_cast<uint32_t>(met++) & 1u, ab);
    };
    int u = 0, pieces = 0;                                   // tiles and pieces of this sub so far
    bool ok = true;
    for (int k = 0; ok; ++k) {
      ok = mbar_wait_warp(ready + (k & 1), static_cast<uint32_t>(k >> 1) & 1u, ab);
      if (!ok) break;
      const Unit& at = units[k & 1];
      const int rows = at.rows, n = at.kt1 - at.kt0;
      if (rows == 0) break;
      const bool active = sub * 128 < rows, valid = row < rows;
      const bool busy = sub * 128 + quarter * 32 < rows;     // some row of this warp is one
      const int token = (at.first_row + (valid ? row : 0)) / p.group;
      const int head = at.hk * p.group + at.first_row + (valid ? row : 0) - token * p.group;
      uint16_t* out = p.out + (static_cast<long long>(at.q.start + token) * p.h + head) * D;
      if (at.zeros && valid) {
        for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(out)[c] = make_uint4(0, 0, 0, 0);
      }
      if (n > 0) {
        const int pos = valid ? at.q.len - at.q.n + token : -1;
        float m_used = -INFINITY, l = 0.f, sc = 0.f;
        if (active) {
          // ---- Q: rows scaled by powers of two, as fp16 (the last scores are done with the ones before);
          // kLanes lanes read a row (rows apart by thread touch 32 lines with each load: 7 us)
          const long long mine = reinterpret_cast<long long>(p.q + static_cast<long long>(at.q.start + token) * p.q_stride + head * D);
          constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes, kLoads = 32 / kRowsAtOnce, kAtOnce = 4;
          uint8_t* q_smem = smem + sub * C::kQBytes;
          const int row0 = sub * 128 + quarter * 32;
          int up_here = 0;                                   // of this lane's row
#pragma unroll 1
          for (int x0 = 0; x0 < kLoads; x0 += kAtOnce) {
            uint4 v[kAtOnce];
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
              const int r = ((x0 + x) * kRowsAtOnce + lane / kLanes) & 31;
              const long long src = __shfl_sync(0xffffffffu, mine, r);
              v[x] = make_uint4(0, 0, 0, 0);
              if (row0 + r < rows && x0 + x < kLoads) v[x] = __ldcg(reinterpret_cast<const uint4*>(src) + lane % kLanes);
            }
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
              if (x0 + x >= kLoads) continue;
              const int r = (x0 + x) * kRowsAtOnce + lane / kLanes;
              const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
              uint32_t top = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, w[e] >> 16 & 0x7fffu));
#pragma unroll
              for (int y = 1; y < kLanes; y <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, y));
              const int ex = static_cast<int>(top >> 7);     // biased; rows of zeros, infinities and NaN stay
              const int up = top == 0 || ex == 255 ? 0 : max(-120, min(120, 13 + 127 - ex));
              const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                h[e] = pack_f16x2(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
              constexpr int kChunks = C::kRowBytes / 16;
              const int c = lane % kLanes;
              *reinterpret_cast<uint4*>(q_smem + (c / kChunks) * C::kQBox +
                                        swizzle_offset<C::kRowBytes>(quarter * 32 + r, c % kChunks)) =
                  make_uint4(h[0], h[1], h[2], h[3]);
              // to the lane whose row it is
              const int its = __shfl_sync(0xffffffffu, up, (lane % kRowsAtOnce) * kLanes);
              if (lane / kRowsAtOnce == x0 + x) up_here = its;
            }
          }
          sc = score_factor(p, up_here);
          fence_proxy_async_smem();
          mbar_arrive(q_full + sub);
          if (at.of > 1 && tid == 0) open_count(p.counts + slot_of(at, 0));
          const float2 sc2 = make_float2(sc, sc);
          // ---- key tiles
          for (int i = 0; i < n; ++i, ++u) {
            // (two buffers: tile u's phases come every second tile)
            const int buf = C::kBufs == 2 ? u & 1 : 0;
            const uint32_t phase = static_cast<uint32_t>(C::kBufs == 2 ? u >> 1 : u) & 1u;
            const uint32_t s_col = static_cast<uint32_t>(buf * kBN);
            const int bar = C::kBufs == 2 ? buf : sub;       // of s_full and p_full
            const int key0 = at.tile(i) << kBNShift;
            ok = mbar_wait_warp(s_full + bar, phase, ab);
            if (!ok) break;
            tc_fence_after();
            if (busy) {
              float s[kBN];
              {
                uint32_t sr[kBN / 32][32];
#pragma unroll
                for (int c = 0; c < kBN / 32; ++c) tmem_ld32(lane_base + s_col + c * 32, sr[c]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < kBN / 32; ++c) {
                  reg_fence(sr[c]);
#pragma unroll
                  for (int e = 0; e < 32; ++e) s[c * 32 + e] = __uint_as_float(sr[c][e]);
                }
              }
              if (key0 + kBN - 1 > at.first_pos || (windowed && key0 <= at.hi_pos - p.window)) {
                const int hi_c = pos - key0;                 // visible columns: up to hi_c, and
                const int lo_c = windowed ? pos - p.window - key0 : -1, sink_c = p.sinks - key0;   // beyond lo_c or below sink_c
#pragma unroll
                for (int c = 0; c < kBN; ++c)
                  if (c > hi_c || (c <= lo_c && c >= sink_c)) s[c] = -INFINITY;
              }
              float mx8[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) mx8[x] = s[x];
#pragma unroll
              for (int c = 8; c < kBN; c += 16)
#pragma unroll
                for (int x = 0; x < 8; ++x) mx8[x] = fmax3(mx8[x], s[c + x], c + 8 + x < kBN ? s[c + 8 + x] : s[c + x]);
              const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
              // the reference moves when a score is too far above it
              const float top = mx * sc, m_new = top - kWeightUp;
              float alpha = 1.f;
              bool rescale = false;
              if (i == 0) {
                m_used = m_new;
              } else {
                const bool need = valid && top > m_used + kWeightMost;
                rescale = __any_sync(0xffffffffu, need);
                if (need) {
                  alpha = ex2_approx(m_used - m_new);
                  m_used = m_new;
                  l *= alpha;
                }
              }
              if (rescale) {
                // With one buffer these scores were issued behind O += P V of the tile before, which
                // is done then; with two it is waited for (of the one before that it is done, and
                // the next needs this tile's P).
                if constexpr (C::kBufs == 2) {
                  ok = mbar_wait_warp(o_full, static_cast<uint32_t>(u - 1) & 1u, ab);
                  if (!ok) break;
                  tc_fence_after();
                }
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {           // (rare)
                  uint32_t o[16];
                  tmem_ld_chunk(lane_base + C::kOCol + c * 16, o);
                  tmem_ld_wait();
                  reg_fence(o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                  tmem_st_chunk(lane_base + C::kOCol + c * 16, o);
                }
              }
              const float m_sub = m_used == -INFINITY ? 0.f : m_used;
              const float2 neg2 = make_float2(-m_sub, -m_sub);
              float2 acc[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) acc[x] = make_float2(0.f, 0.f);
              // (P is handed over whole: in two or four parts the warps that issue the products
              // wait for each, 143 and 160 us instead of 140 for 4 chunks of 512 tokens behind
              // 7680 positions)
#pragma unroll
              for (int y = 0; y < kBN / 32; ++y) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const int c = y * 32 + 2 * e;
                  const float2 x = __ffma2_rn(make_float2(s[c], s[c + 1]), sc2, neg2);
                  const float2 pe = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                  acc[e & 3] = __fadd2_rn(acc[e & 3], pe);
                  pk[e] = pack_f16x2(pe.x, pe.y);
                }
                tmem_st16(lane_base + s_col + y * 16, pk);
              }
              const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
              l += a.x + a.y;
              tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive(p_full + bar);
          }
          if (!ok) break;
          // (a barrier of its own: o_full may still be two tiles behind)
          ok = mbar_wait_warp(o_last + sub, static_cast<uint32_t>(pieces++) & 1u, ab);
          if (!ok) break;
          tc_fence_after();
        }
        // ---- the piece's end.  Slots: O as [D / 4][rows] vectors of four columns, (m, l) as [rows].
        const bool whole = at.of == 1;
        uint8_t* own = p.slots + static_cast<long long>(whole ? 0 : slot_of(at, cta - at.first_run)) * p.slot_bytes;
        float ll = l;
        // O columns [c kOChunk, + kOChunk) of this row
        auto load_o = [&](int c, uint32_t (&o)[C::kOChunk]) {
          __syncwarp();
          tmem_ld_chunk(lane_base + C::kOCol + c * C::kOChunk, o);
          tmem_ld_wait();
          reg_fence(o);
        };
        uint8_t* turn = smem + sub * C::kQBytes + quarter * C::kWarpQ;   // (the products are done with Q)
        const int rows_here = rows - (sub * 128 + quarter * 32);
        if (busy && active) {
          const float f = ll > 0.f ? p.v_unit / ll : 0.f;
#pragma unroll 1
          for (int c = 0; c < D / C::kOChunk; ++c) {
            uint32_t o[C::kOChunk];
            load_o(c, o);
            if (whole) {
              store_rows<D>(turn, out, rows_here, c, o, f);
            } else if (valid) {
              float4* dst = reinterpret_cast<float4*>(own) + row;
#pragma unroll
              for (int e = 0; e < C::kOChunk / 4; ++e)
                dst[(c * (C::kOChunk / 4) + e) * C::kRows] =
                    make_float4(__uint_as_float(o[e * 4]), __uint_as_float(o[e * 4 + 1]), __uint_as_float(o[e * 4 + 2]),
                                __uint_as_float(o[e * 4 + 3]));
            }
          }
          if (!whole && valid) reinterpret_cast<float2*>(own + C::kRows * D * 4)[row] = make_float2(m_used, ll);
        }
        auto release_o = [&]() {
          if (!active) return;
          tc_fence_before();
          mbar_arrive(o_free + sub);
        };
        // This run's piece of two is merged from tensor memory, if no unit comes after it (a
        // prompt of 4096 takes 90 us so, and 98 with both pieces read back; with d = 256 the
        // code costs the loop over the keys registers, 65 us instead of 61 for 3 chunks of 200)
        bool keep = D <= 128 && at.of == 2;
        if (keep) {
          if (!(ok = mbar_wait_warp(ready + ((k + 1) & 1), static_cast<uint32_t>((k + 1) >> 1) & 1u, ab))) break;
          keep = units[(k + 1) & 1].rows == 0;
        }
        if (!keep) release_o();
        if (!whole) {
          unsigned long long* count = p.counts + slot_of(at, 0);
          __threadfence();
          if (!(ok = meet())) break;
          if (tid == 0) {
            last_one = static_cast<int>(atomicAdd(count, 1ull) & 0xffff) + 1 == at.of;
            __threadfence();
            if (last_one) *count = 0;
          }
          if (!(ok = meet())) break;
          if (last_one != 0 && busy && active) {
            if (!keep) {
              merge_rows<D>(p, at, turn, out, rows_here, row);
            } else {
              // the most frequent case: this run's piece from tensor memory, half the reading
              const int mine = cta - at.first_run;
              const uint8_t* slot = p.slots + static_cast<long long>(slot_of(at, 1 - mine)) * p.slot_bytes;
              const int rw = min(row, rows - 1);
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(slot + C::kRows * D * 4) + rw);
              const float4* src = reinterpret_cast<const float4*>(slot) + rw;
              const float mm = fmaxf(m_used, ml.x), base = mm == -INFINITY ? 0.f : mm;
              const float g = weight(m_used, base), g2 = weight(ml.x, base);
              // (rounded as merge_rows does it, which merges this unit where the other run is the
              // last: the first piece's product, then the second's added with one rounding)
              auto sum_of = [&](float own, float other) {
                return mine == 0 ? fmaf(other, g2, __fmul_rn(own, g)) : fmaf(own, g, __fmul_rn(other, g2));
              };
              const float sum = sum_of(ll, ml.y), f = sum > 0.f ? p.v_unit / sum : 0.f;
              constexpr int kVec = C::kOChunk / 4, kChunks = D / C::kOChunk;
              float4 x[kVec], x2[kVec];
              auto fetch = [&](int c, float4 (&to)[kVec]) {
                if (c >= kChunks) return;
#pragma unroll
                for (int e = 0; e < kVec; ++e) to[e] = __ldcg(src + (c * kVec + e) * C::kRows);
              };
              fetch(0, x);
              auto step = [&](int c, const float4 (&x)[kVec]) {
                uint32_t o[C::kOChunk];
                load_o(c, o);
                auto both = [&](uint32_t& a, float b) { a = __float_as_uint(sum_of(__uint_as_float(a), b)); };
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                  both(o[4 * e], x[e].x);
                  both(o[4 * e + 1], x[e].y);
                  both(o[4 * e + 2], x[e].z);
                  both(o[4 * e + 3], x[e].w);
                }
                store_rows<D>(turn, out, rows_here, c, o, f);
              };
#pragma unroll 1
              for (int c = 0; c < kChunks; c += 2) {
                fetch(c + 1, x2);
                step(c, x);
                fetch(c + 2, x);
                if (c + 1 < kChunks) step(c + 1, x2);
              }
            }
          }
          if (keep) release_o();
          // (last_one has been read)
          if (!(ok = meet())) break;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(done + (k & 1));
    }
  } else if (any && warp < C::kMmaWarp) {
    // -------------------------------------------------------------- expand
    if constexpr (C::kSub == 2) regs_decrease<C::kExpandRegs>();
    // (Loops are short for the instruction cache's sake, which all roles share: with two
    // tiles' loads and products unrolled every role waited for instructions, and 4 chunks of
    // 512 tokens behind 7680 positions took 250 us instead of 160.)
    const int tid_e = tid - C::kExpandWarp * 32;
    // A thread expands blocks of 16 columns: the same place in every kStep-th row.
    constexpr int kBlocks = D / 16, kStep = 128 / kBlocks, kTimes = kBN / kStep;
    static_assert(kStep % 8 == 0 && kBN % kStep == 0, "the swizzle is the same in all of a thread's rows");
    const int row0 = tid_e / kBlocks, chunk = 2 * (tid_e % kBlocks);
    constexpr int kRowChunks = C::kRowBytes / 16;
    const int at_row = (row0 >> 3) * C::kGroupBytes + (chunk / kRowChunks) * C::kSBO;
    const int dst0 = at_row + swizzle_offset<C::kRowBytes>(row0 & 7, chunk % kRowChunks);
    const int dst1 = at_row + swizzle_offset<C::kRowBytes>(row0 & 7, chunk % kRowChunks + 1);
    int u = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      ok = mbar_wait_warp(ready + (k & 1), static_cast<uint32_t>(k >> 1) & 1u, ab);
      if (!ok) break;
      const Unit& at = units[k & 1];
      if (at.rows == 0) break;
      const int n = at.kt1 - at.kt0, hi_pos = at.hi_pos;
      const int hidden = p.window < INT_MAX ? max(at.first_pos, 0) - p.window : -1;
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i, ++u) {
        const int st = u % R, key0 = at.tile(i) << kBNShift;
        const bool edge = key0 + kBN - 1 > hi_pos || key0 <= hidden;
#pragma unroll 1
        for (int y = 0; y < 2; ++y) {                        // K, V
          const int half = 2 * u + y, slot = half % C::kRawSlots;
          ok = mbar_wait_warp(raw_full + slot, static_cast<uint32_t>(half / C::kRawSlots) & 1u, ab) &&
               (u < R || mbar_wait_warp((y == 0 ? k_empty : v_empty) + st, static_cast<uint32_t>(u / R - 1) & 1u, ab));
          if (!ok) break;
          uint8_t* raw = smem + C::kRawOff + slot * C::kRawHalf;
          uint8_t* scales = raw + C::kCodes + tid_e;
          if (edge) {
            // what no row sees may be anything: its scale could be a NaN
            for (int x = 0; x < kTimes; ++x) {
              const int key = key0 + row0 + x * kStep;
              if (key > hi_pos || (key <= hidden && key >= p.sinks)) scales[x * 128] = 0;
            }
          }
          uint8_t* stage = smem + (y == 0 ? C::kKOff : C::kVOff) + st * C::kKVBytes;
#pragma unroll
          for (int x = 0; x < kTimes; ++x) {
            const uint2 w = *reinterpret_cast<const uint2*>(raw + tid_e * 8 + x * (128 * 8));
            const uint32_t sc2 = scale_f16x2(scales[x * 128]);
            uint8_t* dst = stage + x * (kStep / 8 * C::kGroupBytes);
            *reinterpret_cast<uint4*>(dst + dst0) = expand8(w.x, sc2);
            *reinterpret_cast<uint4*>(dst + dst1) = expand8(w.y, sc2);
          }
          fence_proxy_async_smem();
          mbar_arrive((y == 0 ? k_full : v_full) + st);
          __syncwarp();
          if (lane == 0) mbar_arrive(raw_empty + slot);
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(done + (k & 1));
    }
  } else if (any) {
    if constexpr (C::kSub == 2) regs_decrease<C::kRestRegs>();
    if (warp < C::kMmaWarp + C::kSub) {
      // ---------------------------------------------------------- products
      // A warp for each 128 rows, which take turns: while one's products are under way the
      // other's P is waited for, and one's softmax runs beside the other's products.  (One warp
      // for both takes 0.9 us for each one's share of a tile, 2.1 us a tile; without turns both
      // do the same at the same time, 2.4 us.)
      const int sub = warp - C::kMmaWarp;
      auto lo = [](uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); };
      const uint32_t q_lo = lo(smem_base + sub * C::kQBytes, 16);
      const uint32_t t_sub = tmem + sub * C::kSubCols;
      // scores of tile u (us: of this sub's)
      auto issue_s = [&](int u, int us) {
        const int buf = C::kBufs == 2 ? us & 1 : 0;
        const uint32_t d = t_sub + static_cast<uint32_t>(buf * kBN);
        const uint32_t b0 = lo(smem_base + C::kKOff + (u % R) * C::kKVBytes, 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          constexpr int kS = C::kStepsPerRow;
          mma_bf16_ss_warp(d, q_lo + static_cast<uint32_t>(((k / kS) * C::kQBox + (k % kS) * 32) >> 4), C::kDescHi,
                           b0 + static_cast<uint32_t>(((k / kS) * C::kSBO + (k % kS) * 32) >> 4), C::kDescHiKV, C::kIdescS,
                           k > 0 ? 1u : 0u);
        }
#ifdef SDPA_TEST_WITHHOLD_FIRST_S_COMMIT
        if (us > 0)                                          // failure injection for the timeout test
#endif
        mma_commit_warp(s_full + (C::kBufs == 2 ? buf : sub));
        mma_commit_warp(k_empty + u % R);
      };
      // O += P V of tile u
      auto issue_pv = [&](int u, int us, bool accumulate) -> bool {
        const int buf = C::kBufs == 2 ? us & 1 : 0;
        const uint32_t phase = static_cast<uint32_t>(C::kBufs == 2 ? us >> 1 : us) & 1u;
        if (!mbar_wait_warp(p_full + (C::kBufs == 2 ? buf : sub), phase, ab)) return false;
        tc_fence_after();
        const uint32_t pa = t_sub + static_cast<uint32_t>(buf * kBN);
        const uint32_t b0 = lo(smem_base + C::kVOff + (u % R) * C::kKVBytes, C::kSBO);
#pragma unroll
        for (int k = 0; k < kBN / 16; ++k)
          mma_bf16_ts_warp(t_sub + C::kOCol, pa + static_cast<uint32_t>(k * 8),
                           b0 + static_cast<uint32_t>((k * 2 * C::kGroupBytes) >> 4), C::kDescHiKV, C::kIdescPV,
                           (accumulate || k > 0) ? 1u : 0u);
        if (C::kBufs == 2) mma_commit_warp(o_full);
        return true;
      };
      auto k_ready = [&](int v) { return mbar_wait_warp(k_full + v % R, static_cast<uint32_t>(v / R) & 1u, ab); };
      auto v_ready = [&](int v) { return mbar_wait_warp(v_full + v % R, static_cast<uint32_t>(v / R) & 1u, ab); };
      int u = 0, us = 0, pieces = 0, turns = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        ok = mbar_wait_warp(ready + (k & 1), static_cast<uint32_t>(k >> 1) & 1u, ab);
        if (!ok) break;
        const int rows = units[k & 1].rows, n = units[k & 1].kt1 - units[k & 1].kt0;
        if (rows == 0) break;
        const bool both = rows > 128;
        // waits for this warp's turn; gives it away
        auto take = [&]() -> bool {
          if (!both) return true;
          const int t = turns++ - (sub == 0 ? 1 : 0);        // (the first is sub 0's)
          return t < 0 || mbar_wait_warp(turn + sub, static_cast<uint32_t>(t) & 1u, ab);
        };
        auto pass = [&]() {
          if (both && lane == 0) mbar_arrive(turn + (sub ^ 1));
        };
        if (sub * 128 >= rows) {
          // no rows: the tiles are released as they come
#pragma unroll 1
          for (int i = 0; i < n && ok; ++i, ++u) {
            if (!(ok = k_ready(u))) break;
            if (lane == 0) mbar_arrive(k_empty + u % R);
            if (!(ok = v_ready(u))) break;
            if (lane == 0) mbar_arrive(v_empty + u % R);
          }
        } else if (n > 0) {
          ok = k_ready(u) && mbar_wait_warp(q_full + sub, static_cast<uint32_t>(pieces) & 1u, ab) && take();
          if (!ok) break;
          tc_fence_after();
          issue_s(u, us);
          pass();
#pragma unroll 1
          for (int i = 0; i < n; ++i, ++u, ++us) {
            // With two buffers the next scores go ahead of this tile's O += P V (into the buffer
            // of the P before: its product was issued before), with one behind it, into P's place.
            auto next_s = [&]() -> bool {
              if (i + 1 >= n) return true;
              if (!k_ready(u + 1)) return false;
              tc_fence_after();
              issue_s(u + 1, us + 1);
              return true;
            };
            if (C::kBufs == 2 && !(ok = next_s())) break;
            // O of the piece before has been read out
            ok = take() && v_ready(u) &&
                 (i > 0 || pieces == 0 || mbar_wait_warp(o_free + sub, static_cast<uint32_t>(pieces - 1) & 1u, ab)) &&
                 issue_pv(u, us, i > 0);
            if (!ok) break;
            if (i + 1 == n) mma_commit_warp(o_last + sub);
            mma_commit_warp(v_empty + u % R);
            if (C::kBufs == 1 && !(ok = next_s())) break;
            pass();
          }
          ++pieces;
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(done + (k & 1));
      }
      mma_commit_warp(drain);
      mbar_wait_drain(drain, 0);
    } else if (warp >= C::kCopyWarp) {
      // ------------------------------------------------------------- copies
      // One warp K's, one V's, 16 bytes a lane, by 16 rows: they are one page's.  A lane
      // looks up the page of one of a tile's 16 rows, a tile ahead of their copies.
      const int y = warp - C::kCopyWarp;
      constexpr int kGroups = kBN / 16, kChunks = D / 2, kScaleChunks = D / 16;   // of 16 rows
      int u = 0;
      bool ok = true;
      if (y == 0 && lane == 0) mbar_arrive(ready);           // (the first unit)
      for (int k = 0; ok; ++k) {
        ok = mbar_wait_warp(ready + (k & 1), static_cast<uint32_t>(k >> 1) & 1u, ab);
        if (!ok) break;
        const Unit& at = units[k & 1];
        if (at.rows == 0) break;
        const int n = at.kt1 - at.kt0, hi_pos = at.hi_pos;
        const int hidden = p.window < INT_MAX ? max(at.first_pos, 0) - p.window : -1;
        const int32_t* pages = p.page_table + static_cast<long long>(at.s) * p.pages_per_seq;
        const uint8_t* from = (y == 0 ? p.k_pages : p.v_pages) + at.hk * p.page_bytes + lane * 16;
        // what no row sees is not looked at (-1: zeros are copied)
        auto ask = [&](int i) -> int {
          const int key = (at.tile(i) << kBNShift) + lane * 16;
          const bool seen = i < n && lane < kGroups && key <= hi_pos && (key + 15 > hidden || key < p.sinks);
          return seen ? __ldcg(pages + (key >> p.page_shift)) : -1;
        };
        int page = ask(0), shown = page;
#pragma unroll 1
        for (int i = 0; i < n; ++i, ++u) {
          const int next = ask(i + 1);
          const int key0 = at.tile(i) << kBNShift;
          shown = page;
          if (page >= p.n_pages || page < -1) {
            atomicOr(p.status, kStatusBadPage);              // and zeros
            shown = -1;
          } else if (page == -1 && lane < kGroups) {
            // (-1 in the table is a bad page too, if it was asked for)
            const int key = key0 + lane * 16;
            if (key <= hi_pos && (key + 15 > hidden || key < p.sinks)) atomicOr(p.status, kStatusBadPage);
          }
          __syncwarp();
          const int half = 2 * u + y, slot = half % C::kRawSlots;
          ok = half < C::kRawSlots || mbar_wait_warp(raw_empty + slot, static_cast<uint32_t>(half / C::kRawSlots - 1) & 1u, ab);
          if (!ok) break;
          const uint32_t dst = smem_base + C::kRawOff + slot * C::kRawHalf + lane * 16;
#pragma unroll 2
          for (int g = 0; g < kGroups; ++g) {
            const int pg = __shfl_sync(0xffffffffu, shown, g);
            const long long r = (key0 + g * 16) & ((1 << p.page_shift) - 1);
            const uint8_t* src = from + (pg >= 0 ? pg * p.page_stride : 0);
            const uint8_t* codes = src + r * (D / 2);
#pragma unroll
            for (int c = 0; c < kChunks; c += 32)
              if (kChunks >= 32 || lane < kChunks) cp_async16_or_zeros(dst + g * (8 * D) + c * 16, codes + c * 16, pg >= 0);
            if (lane < kScaleChunks)
              cp_async16_or_zeros(dst + C::kCodes + g * D, src + (static_cast<long long>(D / 2) << p.page_shift) + r * (D / 16),
                                  pg >= 0);
          }
          cp_async_arrive(raw_full + slot);
          page = next;
        }
        if (!ok) break;
        if (y == 0) {
          // the next unit, once all are done with the one before this
          Unit next = at;
          const bool more = next_unit(plan, sched.cut, cta, &next);
          if (!more) next.rows = 0;
          ok = k == 0 || mbar_wait_warp(done + ((k + 1) & 1), static_cast<uint32_t>((k - 1) >> 1) & 1u, ab);
          if (!ok) break;
          if (lane == 0) {
            units[(k + 1) & 1] = next;
            mbar_arrive(ready + ((k + 1) & 1));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(done + (k & 1));
      }
      cp_async_wait<0>();                                    // (a wait may have run out above)
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  // what waits for this kernel waits for the one before it too
  griddep_wait();
}

template <int D>
cudaError_t launch_wide_impl(const Paged4Params& p, cudaStream_t stream) {
  constexpr int smem = WCfg<D>::kSmemBytes;
  // the kernel's shared-memory limit is set once on each device
  static std::atomic<unsigned long long> prepared{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev > 63 || !(prepared.load(std::memory_order_acquire) & bit)) {
    err = cudaFuncSetAttribute(sdpa_paged4_many<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    if (dev <= 63) prepared.fetch_or(bit, std::memory_order_release);
  }
  return launch_kernel(sdpa_paged4_many<D>, dim3(static_cast<unsigned>(p.runs)), dim3(WCfg<D>::kThreads), smem, stream,
                       true, p);
}

}  // namespace

int paged4_wide_rows(int d) { return d <= 128 ? 256 : 128; }

long long paged4_wide_most_runs(long long units, long long max_len) {
  return std::max(1ll, units * (kStartKeys + max_len + 128) / kMinRunKeys);
}

cudaError_t launch_sdpa_paged4_wide(const Paged4Params& p, int d, cudaStream_t stream) {
  switch (d) {
    case 16: return launch_wide_impl<16>(p, stream);
    case 32: return launch_wide_impl<32>(p, stream);
    case 64: return launch_wide_impl<64>(p, stream);
    case 128: return launch_wide_impl<128>(p, stream);
    case 256: return launch_wide_impl<256>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sdpa
