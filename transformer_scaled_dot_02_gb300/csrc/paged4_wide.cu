// Attention over a paged cache held in 4 bits (paged4.cu gives the format) for
// sequences with many rows: chunks of a prompt and whole prompts.  paged4_attn.cu
// has the few-rows kernel, which takes the other sequences.
//
// sdpa_paged4_many<D>: a UNIT is (sequence, key-value head, row tile), a row being
// a new token's query head of the group; a row tile has kSub times 128 rows, so that
// a key tile of 64 is expanded once for all of them.  All units' walks laid end to
// end are cut into equal runs, one for each CTA (one on an SM), by the keys that
// the rows see; the cut is worked out on the device.  A piece of a unit that is cut
// is published as fp32 (O, m, l), and the run that publishes the last piece merges
// them in the order of their keys: results repeat bit by bit, no run waits for another.
//
// Roles: four warps expand K and V, codes and scales to fp16 (exact), into shared
// memory as the tensor core's swizzled operands; one issues the products
// (tcgen05.mma, kind::f16: S = Q K^T into tensor memory, O += P V with P from
// there); four for each 128 rows do the softmax, a row a thread; one works out the
// units.  Queries are scaled by a power of two for each row to fit fp16, the softmax
// weights are rounded to fp16 (2^-12).
//
// What bounds it: the products of a key tile take 1024 clock cycles of the tensor
// core for 256 rows of 128 columns; beside them an SM issues about 760 instructions
// (a warp's) to expand the tile and 2600 for its softmax, 840 cycles' worth.
#include <algorithm>
#include <atomic>
#include <climits>

#include "kernels.h"
#include "ptx.cuh"

namespace sdpa {
namespace {

constexpr int kBN = 64;                    // keys of a tile
constexpr int kBNShift = 6;
constexpr float kRescaleThreshold = 8.0f;  // log2 units, as in the other forward kernels
// What a unit costs beside its keys (loading Q, storing O), in keys.
constexpr int kStartKeys = 512;
constexpr int kMinRunTiles = 8;            // key tiles of a run, at least

// ------------------------------------------------------------------ schedule
struct Seq {
  int start, n, len, tiles;                // tiles: row tiles
};

// Items are keys x group.  A unit is start items and then those of the keys that its
// last row sees, were the tile full: group (len - n) + (r + 1) R, or what a window
// holds of them.  So the sum over row tiles has a closed form.
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
    return m <= 0 ? 0 : min(static_cast<long long>(q.tiles), m / R);
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
};

// The runs: [begin(c), begin(c + 1)) of all items.
struct Cut {
  long long each;
  int over, runs;
  __device__ long long begin(int c) const { return each * c + min(c, over); }
  __device__ int run_of(long long x) const {
    const long long longer = over * (each + 1);
    return static_cast<int>(x < longer ? x / (each + 1) : over + (x - longer) / each);
  }
};

template <int R>
__device__ void set_piece(const Plan<R>& plan, const Cut& cut, int c, Unit* u) {
  const Paged4Params& p = plan.p;
  const Seq& q = u->q;
  const long long rows = 1ll * q.n * p.group, row0 = 1ll * u->r * R;
  u->first_row = static_cast<int>(row0);
  u->rows = static_cast<int>(min(static_cast<long long>(R), rows - row0));
  u->first_pos = q.len - q.n + static_cast<int>(row0 / p.group);
  u->hi_pos = q.len - q.n + static_cast<int>((row0 + u->rows - 1) / p.group);
  Tiles t{0, 0, 0};
  if (u->hi_pos >= 0) {
    if (p.window < INT_MAX) {
      t.first = max(max(u->first_pos, 0) - p.window + 1, 0) >> kBNShift;
      t.head = min((min(p.sinks, u->hi_pos + 1) + kBN - 1) >> kBNShift, t.first);
    }
    t.count = t.head + (u->hi_pos >> kBNShift) - t.first + 1;
  }
  u->tiles = t;
  // Key tiles before item y of the unit, in proportion; all of them at once where a tile
  // would be more than a run (rows at negative positions see less than they count for).
  const long long items = plan.cost(q, u->r) - plan.start();
  const bool single = items > t.count * cut.each;
  auto tile_at = [&](long long y) -> int {
    y -= plan.start();
    return y <= 0 ? 0 : single ? t.count : static_cast<int>(min(static_cast<long long>(t.count), y * t.count / items));
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
template <int R>
__device__ bool find_place(const Plan<R>& plan, Schedule* sh, Unit* first, int c) {
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
  const long long least = 1ll * kMinRunTiles * kBN * p.group;
  cut.runs = static_cast<int>(min(static_cast<long long>(p.runs), max(1ll, all / least)));
  cut.each = all / cut.runs;
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
        u.hk = static_cast<int>((x - before) / head);
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
template <int R>
__device__ __forceinline__ bool next_unit(const Plan<R>& plan, const Cut& cut, int c, Unit* u) {
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
// Instruction descriptor, kind::f16: fp16 A and B (formats 0), fp32 D.
constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((static_cast<uint32_t>(N) >> 3) << 17) |
         ((static_cast<uint32_t>(M) >> 4) << 24);
}
__device__ __forceinline__ float weight(float m, float sub) { return ex2_approx(m - sub); }

template <int D>
struct WCfg {
  static constexpr int kSub = D <= 128 ? 2 : 1;              // 128 rows each
  static constexpr int kRows = 128 * kSub;
  static constexpr int kSoftmaxWarps = 4 * kSub;
  static constexpr int kExpandWarp = kSoftmaxWarps;          // the first of four
  static constexpr int kMmaWarp = kExpandWarp + 4;
  static constexpr int kUnitWarp = kMmaWarp + 1;
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
  static constexpr int kRing = D <= 64 ? 4 : (D == 128 ? 3 : 2);
  static constexpr int kKOff = kSub * kQBytes;
  static constexpr int kVOff = kKOff + kRing * kKVBytes;
  static constexpr int kTurnOff = kVOff + kRing * kKVBytes;  // rows on their way to the output
  static constexpr int kTurnRow = 64 + 16;
  static constexpr int kTurnSlot = 32 * kTurnRow;
  static constexpr int kBarOff = kTurnOff + kSoftmaxWarps * kTurnSlot;
  // q_full, o_full, o_last, o_free [2]; s_full, p_full [2][2]; k_full, v_full, k_empty, v_empty [R];
  // ready, done [2]; meet, drain
  static constexpr int kNumBars = 8 + 8 + 4 * kRing + 4 + 2;
  static constexpr int kSmemBytes = kBarOff + kNumBars * 8 + 16 + 1024;
  static constexpr int kOChunk = D < 32 ? D : 32;
  static constexpr uint32_t kSubCols = 2 * kBN + (D < 32 ? 32 : D);
  static constexpr uint32_t kOCol = 2 * kBN;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kSub * kSubCols <= kTmemCols, "tensor memory");
  static_assert(kSmemBytes <= 232448 - 1024, "shared memory");
  static_assert(kKOff % 1024 == 0 && kVOff % 1024 == 0 && kKVBytes % 512 == 0, "alignment");
  static constexpr uint32_t kIdescS = idesc_f16(128, kBN, false);
  static constexpr uint32_t kIdescPV = idesc_f16(128, D, true);
  static constexpr uint32_t kDescHi = (kSBO >> 4) | (1u << 14) | (kLayout << 29);
  static constexpr uint32_t kDescHiKV = (kGroupBytes >> 4) | (1u << 14) | (kLayout << 29);
  // registers a thread: the launch's 128 (kSub == 2) are split
  static constexpr int kSoftmaxRegs = 160, kExpandRegs = 96, kRestRegs = 96;
  static_assert(kSub == 1 || 2 * kSoftmaxRegs + kExpandRegs + kRestRegs <= 512, "registers");
};

template <int D>
__global__ void __launch_bounds__(WCfg<D>::kThreads, 1) sdpa_paged4_many(const __grid_constant__ Paged4Params p) {
  using C = WCfg<D>;
  constexpr int R = C::kRing;
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
  uint64_t* s_full = o_free + 2;           // [sub][buffer]
  uint64_t* p_full = s_full + 4;
  uint64_t* k_full = p_full + 4;
  uint64_t* v_full = k_full + R;
  uint64_t* k_empty = v_full + R;
  uint64_t* v_empty = k_empty + R;
  uint64_t* ready = v_empty + R;
  uint64_t* done = ready + 2;
  uint64_t* meet_bar = done + 2;
  uint64_t* drain = meet_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
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
      mbar_init(done + i, C::kSoftmaxWarps + 4 + 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
    }
    for (int i = 0; i < R; ++i) {
      mbar_init(k_full + i, 128);
      mbar_init(v_full + i, 128);
      mbar_init(k_empty + i, 1);
      mbar_init(v_empty + i, 1);
    }
    mbar_init(meet_bar, C::kSoftmaxWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  // (not before the block holds its tensor memory: the next kernel's block could be
  // given it, and then wait for this grid, which waits for the memory)
  griddep_launch_dependents();
  // The kernel before is the one for the other sequences: it began when the one before
  // it was over, and is waited for at the end only.

  const Plan<C::kRows> plan(p);
  const int cta = static_cast<int>(blockIdx.x);
  const bool any = find_place<C::kRows>(plan, &sched, &units[0], cta) && units[0].begin != LLONG_MAX;
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (any && warp < C::kSoftmaxWarps) {
    // ------------------------------------------------------------- softmax
    if constexpr (C::kSub == 2) regs_increase<C::kSoftmaxRegs>();
    const int sub = warp >> 2, quarter = warp & 3;
    const int row = sub * 128 + quarter * 32 + lane;         // of the row tile
    const uint32_t lane_base = tmem + sub * C::kSubCols + (static_cast<uint32_t>(quarter * 32) << 16);
    const bool windowed = p.window < INT_MAX;
    auto slot = [&](int i) { return p.slots + static_cast<long long>(i) * p.slot_bytes; };
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
          // ---- Q: this row, scaled by a power of two, as fp16 (its last scores are done with the one before)
          const uint4* src = reinterpret_cast<const uint4*>(p.q + static_cast<long long>(at.q.start + token) * p.q_stride + head * D);
          uint32_t top = 0;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = valid ? src[c] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, w[e] >> 16 & 0x7fffu));
          }
          const int ex = static_cast<int>(top >> 7);         // biased; rows of zeros, infinities and NaN stay
          const int up = top == 0 || ex == 255 ? 0 : max(-120, min(120, 13 + 127 - ex));
          const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
          // (never 0, which a masked score of -infinity would make a NaN)
          sc = fmaxf(__uint_as_float(static_cast<uint32_t>(127 - up) << 23) * p.k_unit * p.scale_log2, 1e-37f);
          uint8_t* q_smem = smem + sub * C::kQBytes;
          const int r = quarter * 32 + lane;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = valid ? src[c] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              h[e] = pack_f16x2(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
            constexpr int kChunks = C::kRowBytes / 16;
            *reinterpret_cast<uint4*>(q_smem + (c / kChunks) * C::kQBox + swizzle_offset<C::kRowBytes>(r, c % kChunks)) =
                make_uint4(h[0], h[1], h[2], h[3]);
          }
          fence_proxy_async_smem();
          mbar_arrive(q_full + sub);
          const float2 sc2 = make_float2(sc, sc);
          // ---- key tiles
          for (int i = 0; i < n; ++i, ++u) {
            const int buf = u & 1;
            const uint32_t s_col = static_cast<uint32_t>(buf * kBN);
            int key0 = at.kt0 + i;
            if (key0 >= at.tiles.head) key0 += at.tiles.first - at.tiles.head;
            key0 <<= kBNShift;
            ok = mbar_wait_warp(s_full + sub * 2 + buf, static_cast<uint32_t>(u >> 1) & 1u, ab);
            if (!ok) break;
            tc_fence_after();
            if (busy) {
              float s[kBN];
              {
                uint32_t sr[2][32];
                tmem_ld32(lane_base + s_col, sr[0]);
                tmem_ld32(lane_base + s_col + 32, sr[1]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
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
              float mx4[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) mx4[x] = s[x];
#pragma unroll
              for (int c = 4; c < kBN; c += 8)
#pragma unroll
                for (int x = 0; x < 4; ++x) mx4[x] = fmax3(mx4[x], s[c + x], c + 4 + x < kBN ? s[c + 4 + x] : s[c + x]);
              const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
              // the running maximum moves when it grew by more than the threshold
              const float m_new = fmaxf(m_used, mx * sc);
              float alpha = 1.f;
              bool rescale = false;
              if (i == 0) {
                m_used = m_new;
              } else {
                const bool need = valid && m_new > m_used + kRescaleThreshold;
                rescale = __any_sync(0xffffffffu, need);
                if (need) {
                  alpha = ex2_approx(m_used - m_new);
                  m_used = m_new;
                  l *= alpha;
                }
                if (rescale) {
                  // (until O += P V of the tile before is done: of the one before that it is, its
                  // product was issued before these scores', and the next needs this tile's P)
                  ok = mbar_wait_warp(o_full + sub, static_cast<uint32_t>(u - 1) & 1u, ab);
                  if (!ok) break;
                  tc_fence_after();
                }
              }
              const float m_sub = m_used == -INFINITY ? 0.f : m_used;
              const float2 neg2 = make_float2(-m_sub, -m_sub);
              float2 acc[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) acc[x] = make_float2(0.f, 0.f);
              uint32_t pk[kBN / 2];
#pragma unroll
              for (int e = 0; e < kBN / 2; ++e) {
                const float2 x = __ffma2_rn(make_float2(s[2 * e], s[2 * e + 1]), sc2, neg2);
                const float2 pe = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                acc[e & 3] = __fadd2_rn(acc[e & 3], pe);
                pk[e] = pack_f16x2(pe.x, pe.y);
              }
              tmem_st32(lane_base + s_col, pk);
              const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
              if (rescale) {
#pragma unroll
                for (int c = 0; c < D / C::kOChunk; ++c) {
                  uint32_t o[C::kOChunk];
                  tmem_ld_chunk(lane_base + C::kOCol + c * C::kOChunk, o);
                  tmem_ld_wait();
                  reg_fence(o);
#pragma unroll
                  for (int e = 0; e < C::kOChunk; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                  tmem_st_chunk(lane_base + C::kOCol + c * C::kOChunk, o);
                }
              }
              l += a.x + a.y;
              tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive(p_full + sub * 2 + buf);
          }
          if (!ok) break;
          // (a barrier of its own: o_full may still be two tiles behind)
          ok = mbar_wait_warp(o_last + sub, static_cast<uint32_t>(pieces++) & 1u, ab);
          if (!ok) break;
          tc_fence_after();
        }
        // ---- the piece's end.  Slots: O as [D / 4][rows] vectors of four columns, (m, l) as [rows].
        const bool whole = at.of == 1;
        auto place = [&](int i) { return 2 * (at.first_run + i) + (i == 0 ? 1 : 0); };   // of piece i
        uint8_t* own = slot(whole ? 0 : place(cta - at.first_run));
        float ll = l;
        // O columns [c kOChunk, + kOChunk) of this row
        auto load_o = [&](int c, uint32_t (&o)[C::kOChunk]) {
          __syncwarp();
          tmem_ld_chunk(lane_base + C::kOCol + c * C::kOChunk, o);
          tmem_ld_wait();
          reg_fence(o);
        };
        // ... normalised into the output: four lanes write 64 bytes of a row
        auto store_out = [&](int c, const uint32_t (&o)[C::kOChunk], float f) {
          if constexpr (D < 32) {
            if (valid)
              for (int e = 0; e < C::kOChunk / 2; ++e)
                reinterpret_cast<uint32_t*>(out)[c * (C::kOChunk / 2) + e] =
                    pack_bf16x2(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
          } else {
            uint8_t* turn = smem + C::kTurnOff + warp * C::kTurnSlot;
            uint4* mine = reinterpret_cast<uint4*>(turn + lane * C::kTurnRow);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mine[e] = make_uint4(
                  pack_bf16x2(__uint_as_float(o[e * 8 + 0]) * f, __uint_as_float(o[e * 8 + 1]) * f),
                  pack_bf16x2(__uint_as_float(o[e * 8 + 2]) * f, __uint_as_float(o[e * 8 + 3]) * f),
                  pack_bf16x2(__uint_as_float(o[e * 8 + 4]) * f, __uint_as_float(o[e * 8 + 5]) * f),
                  pack_bf16x2(__uint_as_float(o[e * 8 + 6]) * f, __uint_as_float(o[e * 8 + 7]) * f));
            __syncwarp();
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int x = (lane >> 2) + 8 * y;             // row of this warp
              // (its output row: the lane that holds it knows)
              const long long at_out = __shfl_sync(0xffffffffu, reinterpret_cast<long long>(out), x);
              const uint4 v = *reinterpret_cast<const uint4*>(turn + x * C::kTurnRow + (lane & 3) * 16);
              if (sub * 128 + quarter * 32 + x < rows)
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(at_out) + c * 32 + (lane & 3) * 8) = v;
            }
            __syncwarp();
          }
        };
        if (busy && active) {
          const float f = ll > 0.f ? p.v_unit / ll : 0.f;
#pragma unroll 1
          for (int c = 0; c < D / C::kOChunk; ++c) {
            uint32_t o[C::kOChunk];
            load_o(c, o);
            if (whole) {
              store_out(c, o, f);
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
        if (active) {
          tc_fence_before();
          mbar_arrive(o_free + sub);
        }
        if (!whole) {
          unsigned long long* count = p.counts + place(0);
          __threadfence();
          if (!(ok = meet())) break;
          if (tid == 0) {
            open_count(count);
            last_one = static_cast<int>(atomicAdd(count, 1ull) & 0xffff) + 1 == at.of;
            if (last_one) *count = 0;
            __threadfence();
          }
          if (!(ok = meet())) break;
          if (last_one != 0 && busy) {
            // this row of all pieces, in their order
            const int of = at.of;
            const int rw = valid ? row : rows - 1;
            auto ml_of = [&](int i) {
              return __ldcg(reinterpret_cast<const float2*>(slot(place(i)) + C::kRows * D * 4) + rw);
            };
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
#pragma unroll 1
            for (int c = 0; c < D / C::kOChunk; ++c) {
              constexpr int kVec = C::kOChunk / 4;
              float4 acc[kVec];
#pragma unroll
              for (int e = 0; e < kVec; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
              for (int i = 0; i < of; ++i) {
                const float4* src = reinterpret_cast<const float4*>(slot(place(i))) + rw;
                float4 v[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) v[e] = __ldcg(src + (c * kVec + e) * C::kRows);
                const float g = weight(ml_of(i).x, base);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                  acc[e].x = fmaf(v[e].x, g, acc[e].x);
                  acc[e].y = fmaf(v[e].y, g, acc[e].y);
                  acc[e].z = fmaf(v[e].z, g, acc[e].z);
                  acc[e].w = fmaf(v[e].w, g, acc[e].w);
                }
              }
              uint32_t o[C::kOChunk];
#pragma unroll
              for (int e = 0; e < kVec; ++e) {
                o[4 * e] = __float_as_uint(acc[e].x);
                o[4 * e + 1] = __float_as_uint(acc[e].y);
                o[4 * e + 2] = __float_as_uint(acc[e].z);
                o[4 * e + 3] = __float_as_uint(acc[e].w);
              }
              store_out(c, o, f);
            }
          }
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
    const int tid_e = tid - C::kExpandWarp * 32;
    // An item is 32 columns of a row (16 at d = 16): 16 bytes of codes, two scales.
    constexpr int kCols = D < 32 ? 16 : 32, kPerRow = D / kCols, kAll = kBN * kPerRow;
    constexpr int kItems = (kAll + 127) / 128;
    struct Raw {
      uint4 codes;
      uint32_t scales;
    };
    Raw kr[kItems], vr[kItems];
    int page[kItems];                                        // of the next tile's items
    int u = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      ok = mbar_wait_warp(ready + (k & 1), static_cast<uint32_t>(k >> 1) & 1u, ab);
      if (!ok) break;
      const Unit& at = units[k & 1];
      if (at.rows == 0) break;
      const int n = at.kt1 - at.kt0, kt0 = at.kt0, head = at.tiles.head, skip = at.tiles.first - head;
      const int hi_pos = at.hi_pos, hidden = p.window < INT_MAX ? max(at.first_pos, 0) - p.window : -1;
      const int32_t* pages = p.page_table + static_cast<long long>(at.s) * p.pages_per_seq;
      const uint8_t *k_head = p.k_pages + at.hk * p.page_bytes, *v_head = p.v_pages + at.hk * p.page_bytes;
      auto key_of = [&](int i, int j) {
        const int kt = kt0 + i;
        return ((kt < head ? kt : kt + skip) << kBNShift) + (tid_e + 128 * j) / kPerRow;
      };
      // a position that no row sees is not looked at, and zero
      auto seen = [&](int key) { return key <= hi_pos && (key > hidden || key < p.sinks); };
      auto ask = [&](int i) {
        if (i >= n) return;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
          const int key = key_of(i, j);
          page[j] = tid_e + 128 * j < kAll && seen(key) ? pages[key >> p.page_shift] : 0;
        }
      };
      auto load = [&](int i) {
        if (i >= n) return;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
          const int key = key_of(i, j), part = (tid_e + 128 * j) % kPerRow;
          kr[j].codes = vr[j].codes = make_uint4(0, 0, 0, 0);
          kr[j].scales = vr[j].scales = 0;
          if (tid_e + 128 * j >= kAll || !seen(key)) continue;
          if (page[j] < 0 || page[j] >= p.n_pages) {
            atomicOr(p.status, kStatusBadPage);              // and zeros
            continue;
          }
          const int r = key & ((1 << p.page_shift) - 1);
          const long long off = page[j] * p.page_stride;
          const long long codes = off + static_cast<long long>(r) * (D / 2) + part * (kCols / 2);
          const long long scales = off + (static_cast<long long>(D / 2) << p.page_shift) + r * (D / 16) + part * (kCols / 16);
          if constexpr (kCols == 32) {
            kr[j].codes = __ldcg(reinterpret_cast<const uint4*>(k_head + codes));
            vr[j].codes = __ldcg(reinterpret_cast<const uint4*>(v_head + codes));
            kr[j].scales = __ldcg(reinterpret_cast<const uint16_t*>(k_head + scales));
            vr[j].scales = __ldcg(reinterpret_cast<const uint16_t*>(v_head + scales));
          } else {
            const uint2 a = __ldcg(reinterpret_cast<const uint2*>(k_head + codes));
            const uint2 b = __ldcg(reinterpret_cast<const uint2*>(v_head + codes));
            kr[j].codes = make_uint4(a.x, a.y, 0, 0);
            vr[j].codes = make_uint4(b.x, b.y, 0, 0);
            kr[j].scales = __ldcg(k_head + scales);
            vr[j].scales = __ldcg(v_head + scales);
          }
        }
      };
      auto store = [&](const Raw (&raw)[kItems], uint8_t* stage) {
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
          if (tid_e + 128 * j >= kAll) continue;
          const int row = (tid_e + 128 * j) / kPerRow, part = (tid_e + 128 * j) % kPerRow;
          const uint32_t w[4] = {raw[j].codes.x, raw[j].codes.y, raw[j].codes.z, raw[j].codes.w};
          uint8_t* dst = stage + (row >> 3) * C::kGroupBytes;
#pragma unroll
          for (int e = 0; e < kCols / 8; ++e) {
            constexpr int kChunks = C::kRowBytes / 16;
            const int c = part * (kCols / 8) + e;
            *reinterpret_cast<uint4*>(dst + (c / kChunks) * C::kSBO + swizzle_offset<C::kRowBytes>(row & 7, c % kChunks)) =
                expand8(w[e], scale_f16x2(raw[j].scales >> (8 * (e / 2)) & 0xffu));
          }
        }
        fence_proxy_async_smem();
      };
      ask(0);
      load(0);
      ask(1);
      for (int i = 0; i < n; ++i, ++u) {
        const int st = u % R;
        const uint32_t phase = static_cast<uint32_t>(u / R - 1) & 1u;
        if (u >= R && !(ok = mbar_wait_warp(k_empty + st, phase, ab))) break;
        store(kr, smem + C::kKOff + st * C::kKVBytes);
        mbar_arrive(k_full + st);
        if (u >= R && !(ok = mbar_wait_warp(v_empty + st, phase, ab))) break;
        store(vr, smem + C::kVOff + st * C::kKVBytes);
        mbar_arrive(v_full + st);
        load(i + 1);
        ask(i + 2);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(done + (k & 1));
    }
  } else if (any) {
    if constexpr (C::kSub == 2) regs_decrease<C::kRestRegs>();
    if (warp == C::kMmaWarp) {
      // ---------------------------------------------------------- products
      auto lo = [](uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); };
      auto issue_s = [&](int sub, int u, int us) {
        const uint32_t d = tmem + sub * C::kSubCols + static_cast<uint32_t>((us & 1) * kBN);
        const uint32_t a0 = lo(smem_base + sub * C::kQBytes, 16), b0 = lo(smem_base + C::kKOff + (u % R) * C::kKVBytes, 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          constexpr int kS = C::kStepsPerRow;
          mma_bf16_ss_warp(d, a0 + static_cast<uint32_t>(((k / kS) * C::kQBox + (k % kS) * 32) >> 4), C::kDescHi,
                           b0 + static_cast<uint32_t>(((k / kS) * C::kSBO + (k % kS) * 32) >> 4), C::kDescHiKV, C::kIdescS,
                           k > 0 ? 1u : 0u);
        }
        mma_commit_warp(s_full + sub * 2 + (us & 1));
      };
      auto issue_pv = [&](int sub, int u, int us, bool accumulate) {
        const uint32_t pa = tmem + sub * C::kSubCols + static_cast<uint32_t>((us & 1) * kBN);
        const uint32_t b0 = lo(smem_base + C::kVOff + (u % R) * C::kKVBytes, C::kSBO);
#pragma unroll
        for (int k = 0; k < kBN / 16; ++k)
          mma_bf16_ts_warp(tmem + sub * C::kSubCols + C::kOCol, pa + static_cast<uint32_t>(k * 8),
                           b0 + static_cast<uint32_t>((k * 2 * C::kGroupBytes) >> 4), C::kDescHiKV, C::kIdescPV,
                           (accumulate || k > 0) ? 1u : 0u);
        mma_commit_warp(o_full + sub);
      };
      int u = 0, us[2] = {0, 0}, pieces[2] = {0, 0};
      bool ok = true;
      for (int k = 0; ok; ++k) {
        ok = mbar_wait_warp(ready + (k & 1), static_cast<uint32_t>(k >> 1) & 1u, ab);
        if (!ok) break;
        const int rows = units[k & 1].rows, n = units[k & 1].kt1 - units[k & 1].kt0;
        if (rows == 0) break;
        if (n > 0) {
          const int subs = rows > 128 ? 2 : 1;
          auto k_ready = [&](int v) { return mbar_wait_warp(k_full + v % R, static_cast<uint32_t>(v / R) & 1u, ab); };
          if (!(ok = k_ready(u))) break;
#pragma unroll
          for (int sub = 0; sub < C::kSub; ++sub) {
            if (sub >= subs || !ok) continue;
            ok = mbar_wait_warp(q_full + sub, static_cast<uint32_t>(pieces[sub]) & 1u, ab);
            if (!ok) continue;
            tc_fence_after();
            issue_s(sub, u, us[sub]);
          }
          if (!ok) break;
          mma_commit_warp(k_empty + u % R);
          for (int i = 0; i < n && ok; ++i, ++u) {
            if (i + 1 < n && !(ok = k_ready(u + 1))) break;
            if (!(ok = mbar_wait_warp(v_full + u % R, static_cast<uint32_t>(u / R) & 1u, ab))) break;
#pragma unroll
            for (int sub = 0; sub < C::kSub; ++sub) {
              if (sub >= subs || !ok) continue;
              tc_fence_after();
              // S of the next tile into the buffer of P of the one before: its O += P V was issued before
              if (i + 1 < n) {
                issue_s(sub, u + 1, us[sub] + 1);
                if (sub + 1 == subs) mma_commit_warp(k_empty + (u + 1) % R);
              }
              // O of the piece before has been read out
              if (i == 0 && pieces[sub] > 0) {
                ok = mbar_wait_warp(o_free + sub, static_cast<uint32_t>(pieces[sub] - 1) & 1u, ab);
                if (!ok) continue;
              }
              ok = mbar_wait_warp(p_full + sub * 2 + (us[sub] & 1), static_cast<uint32_t>(us[sub] >> 1) & 1u, ab);
              if (!ok) continue;
              tc_fence_after();
              issue_pv(sub, u, us[sub], i > 0);
              if (i + 1 == n) mma_commit_warp(o_last + sub);
              ++us[sub];
            }
            if (ok) mma_commit_warp(v_empty + u % R);
          }
          if (!ok) break;
          ++pieces[0];
          if (subs > 1) ++pieces[1];
        }
        if (lane == 0) mbar_arrive(done + (k & 1));
      }
      mma_commit_warp(drain);
      mbar_wait_drain(drain, 0);
    } else if (warp == C::kUnitWarp && lane == 0) {
      // ------------------------------------------------------------- units
      mbar_arrive(ready);
      Unit next = units[0];
      for (int k = 1;; ++k) {
        const bool more = next_unit<C::kRows>(plan, sched.cut, cta, &next);
        if (k > 1 && !mbar_wait(done + (k & 1), static_cast<uint32_t>((k >> 1) - 1) & 1u, ab)) break;
        if (!more) next.rows = 0;
        units[k & 1] = next;
        mbar_arrive(ready + (k & 1));
        if (!more) break;
      }
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
  return std::max(1ll, units * (kStartKeys + max_len + kBN) / (kMinRunTiles * kBN));
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
