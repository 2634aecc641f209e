// Attention of new tokens over a paged K/V cache, and the append that fills
// the cache: the serving form of Eq. (1) of "Attention Is All You Need" with
// the decoder's mask of section 3.2.3 (position i sees keys j <= i).
//
// The new tokens of b sequences come packed, rows [q_starts[s],
// q_starts[s+1]) for sequence s; new token i of n sits at position
// len_s - n + i.  Positions lie in pages [n_pages, h_kv, P, d]; key j of
// sequence s is row j % P of page page_table[s][j / P].  Query head x reads
// key-value head x / (h / h_kv).
//
// sdpa_paged_split<D>: a UNIT is (sequence, key-value head, row tile); the
// rows of a tile are tile_tokens tokens x the group's heads (at most 128), so
// one walk over the keys serves every query head of the group.  A unit's walk
// is its visible keys in tiles of 64.  Where the GPU has a CTA for each piece
// that the units are worth cutting into, a CTA's run is one piece; else all
// units laid end to end, each as long as it is expected to take, are cut into
// equal runs, so that one long sequence, many short ones and any mixture load
// the SMs alike.  The cut is worked out on the device from the lengths, so a
// captured launch follows them.
//
// A CTA works its run from the end to the beginning.  If the run ends inside
// a unit, that piece comes first and its (O, m, l) is published in the
// workspace; if it begins inside a unit, that piece comes last, and the CTA
// merges the pieces that the runs before it published:
//   O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, M = max_s m_s.
// So a CTA waits for CTAs of lower index only.  GPUs start a launch's CTAs in the
// order of their index, which CUDA does not promise: with it the waits end however
// few CTAs run at a time, without it they run out and are reported.  Units cut into many pieces are
// merged in slices by several CTAs, which wait for one another, but not for long
// (see merge).  The pieces merge in an order fixed by the cut, so results repeat
// bit by bit.
//
// Row tiles of at most 16 rows (single tokens) would leave three of the four
// softmax warps idle and one with the whole row: they are NARROW, their queries
// are copied to all four quarters of the tile, each warp takes 16 of a tile's 64
// keys, and the quarters' (O, m, l) are merged when the piece ends.
//
// The roles of a split CTA are those of the one-tile forward kernel (TMA
// producer, MMA issuer, four softmax warps of one thread per row, S double
// buffered and O in tensor memory), kept running from piece to piece: tile
// and piece counters carry on, and two more barriers hand over Q (q_empty)
// and O (o_free).
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace sdpa {
namespace {

constexpr int kBlockM = 128;
constexpr int kBN = kPagedKeyTile;         // keys per tile
constexpr int kBNShift = 6;
static_assert(kBN == 1 << kBNShift, "key tile");
constexpr int kThreads = 192;
constexpr int kProducerWarp = 4;
constexpr int kMmaWarp = 5;
constexpr int kQuarter = 32;               // rows (tensor-memory lanes) of a softmax warp
// Rows of a tile that all four softmax warps hold, at most.  One walk of 16384
// positions, 4 key-value heads of 128, takes 18 / 21 / 28 us with 4 / 8 / 16 rows
// so and 39 with a warp for them; with 24 and 32 rows both take 36, and 128
// sequences of 200 to 1000 positions 41 and 44 us against 37.
constexpr int kNarrowRows = 16;
constexpr int kQuarterKeys = kBN / 4;
constexpr float kRescaleThreshold = 8.0f;  // log2 units, as in the other forward kernels

// ------------------------------------------------------------------ schedule
// One sequence, with everything the caller's device arrays say clamped into
// the buffers: rows inside [0, n_tokens), length inside the page table.
struct Seq {
  int start, n, len, tiles;
};

__device__ __forceinline__ Seq load_seq(const PagedParams& p, int s) {
  Seq q;
  const int cap = p.pages_per_seq << p.page_shift;
  q.start = min(max(p.q_starts[s], 0), p.n_tokens);
  q.n = min(max(p.q_starts[s + 1], q.start), p.n_tokens) - q.start;
  q.len = min(max(p.kv_lengths[s], 0), cap);
  q.tiles = q.n <= p.tile_tokens ? min(q.n, 1) : (q.n + p.tile_tokens - 1) / p.tile_tokens;
  return q;
}

// Keys that some row of row tile r sees, and the tile's walk in key tiles (at
// least one: a tile that sees nothing still writes its zeros).
__device__ __forceinline__ int tile_keys(const PagedParams& p, const Seq& q, int r) {
  return max(0, q.len - q.n + min((r + 1) * p.tile_tokens, q.n));
}
__device__ __forceinline__ int walk_tiles(int keys) { return max(1, (keys + kBN - 1) / kBN); }

// What a unit is expected to take: `start` (loading Q, storing O) and 2^log_tile
// for each key tile, in quarters of a key tile.  From least squares over the
// CTAs' times of two calls on GB300: two prompts of 8192 tokens (16 heads of 128) take
// 4.4 us a walk and 0.94 us a wide key tile, 16 x 4 drafted tokens (64 wide) 2.4 us
// and 0.67 us a narrow one.  So a start is worth 18 or 14 quarters; wide and narrow
// key tiles, and those of all head and page sizes, count alike, and a cut piece's
// publication and merge are left out.  Counting key tiles alone, the CTAs with a prompt's
// shortest walks finished 20 % after the others (514 us instead of 396).
struct Weight {
  int start, log_tile;
  __device__ long long of(long long tiles) const { return start + (tiles << log_tile); }
};
__device__ __forceinline__ Weight weight_of(bool narrow) { return narrow ? Weight{14, 2} : Weight{18, 2}; }
// How the work is cut.  kPieces: every unit into pieces of its own, a run for
// each, where that many runs fit the GPU.  kWeighed: into equal runs by weight.
enum Scheme { kWeighed, kPieces };
// kPieces: a piece of up to 8 KB has up to four key tiles, a larger one eight, one
// over 32 KB sixteen: a further cut saves time at the key tiles (0.5 to 0.9 us
// each), but there are more pieces to merge.  14 single tokens over 749 to 1147
// positions (2 key-value heads, 16 rows of 128: 8 KB) take 14.9 us with four, 20.3
// with one, 15.3 with eight; 128 tokens over 4096 positions of 4 key-value heads
// of 64 (32 KB) 18.4 us with eight, 20.3 with four, 19.2 with sixteen; 200 tokens over
// 8192 positions of 4 key-value heads of 128 (64 KB) 29.9 us with sixteen, 32.3
// with twelve, 31.7 with 24.  Pieces of up to 4 KB have two where the walk is short,
// but none is cut whose key tiles take less than a merge, six of up to 64 columns
// or four wider ones: single tokens over 500 positions take 8.8 us so and 9.8 with
// four (8 heads of 64), 9.6 and 11.6 (32 / 8 heads of 128), over 300 8.0 us uncut, 8.7 cut.
constexpr int kTinyPiece = 4 << 10, kSmallPiece = 8 << 10, kMiddlePiece = 32 << 10;
constexpr int kShortWalk = 32;

// The token that row `row` of a tile belongs to, row / group: rows are below 128, so
// the product's error stays below 2^16.
__device__ __forceinline__ int token_of(const PagedParams& p, int row) {
  return static_cast<int>(static_cast<unsigned>(row) * p.group_magic >> 16);
}
__device__ __forceinline__ int tile_rows(const PagedParams& p, const Seq& q, int r) {
  return min(p.tile_tokens, q.n - r * p.tile_tokens) * p.group;
}
// The pieces that a walk of `tiles` is worth with these rows.
__device__ __forceinline__ int pieces_of(const PagedParams& p, int rows, int tiles) {
  const int bytes = rows * p.row_bytes;
  const int shift = bytes <= kSmallPiece ? (bytes <= kTinyPiece && tiles <= kShortWalk ? 1 : 2)
                                         : (bytes <= kMiddlePiece ? 3 : 4);
  if (tiles <= (shift == 1 ? (p.row_bytes <= 256 ? 6 : 4) : 1 << shift)) return 1;
  return (tiles + (1 << shift) - 1) >> shift;
}
// Pieces of each full row tile of a sequence that has more than one: those of
// the longest walk, or as many as there are key tiles.
__device__ __forceinline__ int full_pieces(const PagedParams& p, const Seq& q) {
  return pieces_of(p, p.tile_tokens * p.group, walk_tiles(q.len));
}
__device__ __forceinline__ int unit_pieces(const PagedParams& p, const Seq& q, int r, int tiles) {
  return r + 1 < q.tiles ? min(full_pieces(p, q), tiles) : pieces_of(p, tile_rows(p, q, r), tiles);
}
__device__ __forceinline__ long long unit_cost(const PagedParams& p, const Seq& q, int r, Scheme scheme) {
  const int tiles = walk_tiles(tile_keys(p, q, r));
  if (scheme == kPieces) return unit_pieces(p, q, r, tiles);
  return weight_of(tile_rows(p, q, r) <= kNarrowRows).of(tiles);
}

// Key tiles of the first f row tiles, f < q.tiles.  They see A + (i + 1) t
// keys, A = len - n: z of them walk one tile, the others ceil((A + (i + 1) t)
// / 64).  With t = g t', 64 = g P, t' odd (or P = 1), the floor of (base + t i) / 64
// is that of (b + t' i) / P, b = base / g, so their sum is
//   (n b + t' n (n - 1) / 2 - sum_i (b + t' i) mod P) / P,
// and the residues are P's in steps of t' from place b / t' mod P on: p.residues
// holds the sums of the first k of them.
__device__ __noinline__ long long tiles_before(const PagedParams& p, const Seq& q, int f) {
  const int t = p.tile_tokens;
  const int a = q.len - q.n;
  const int z = kBN - a >= t ? min(f, (kBN - a) / t) : 0;
  const int cnt = f - z;
  if (cnt <= 0) return z;
  const int log_p = kBNShift - p.log_step, mask = (1 << log_p) - 1;
  const int b = (a + t * (z + 1) + kBN - 1) >> p.log_step;   // > 0
  const long long n = cnt;
  const int i0 = static_cast<int>(static_cast<unsigned>(b) * p.step_inverse) & mask, i1 = i0 + (cnt & mask);
  const int full = p.residues[mask + 1];
  const long long rest = (n >> log_p) * full + (i1 > mask ? full + p.residues[i1 - mask - 1] : p.residues[i1]) -
                         p.residues[i0];
  return z + ((n * b + (t >> p.log_step) * (n * (n - 1) / 2) - rest) >> log_p);
}

// Cost of row tiles 0 .. r-1 (r <= q.tiles) of one key-value head: all but
// the last are wide (a full tile has more than 64 rows).
__device__ __forceinline__ long long full_pieces_before(const PagedParams& p, const Seq& q, int f) {
  const int most = full_pieces(p, q);
  const int short_keys = kBN * (most - 1) - (q.len - q.n);   // row tiles with no more keys walk less
  const int z = most > 1 && short_keys >= p.tile_tokens ? min(f, short_keys / p.tile_tokens) : 0;
  return static_cast<long long>(most) * (f - z) + (z > 0 ? tiles_before(p, q, z) : 0);
}
__device__ __forceinline__ long long cost_before(const PagedParams& p, const Seq& q, int r, Scheme scheme) {
  const int f = min(r, q.tiles - 1);
  long long sum = 0;
  if (f > 0) {
    if (scheme == kPieces) {
      sum = full_pieces_before(p, q, f);
    } else {
      const Weight w = weight_of(false);
      sum = static_cast<long long>(w.start) * f + (tiles_before(p, q, f) << w.log_tile);
    }
  }
  if (r == q.tiles && r > 0) sum += unit_cost(p, q, r - 1, scheme);
  return sum;
}

// A place in the laid-out work: unit (s, hk, r), and the item of it that the
// place is behind.  kPieces: the unit's pieces, and the key tiles of the one
// that ends there.
struct Place {
  int s, hk, r;
  long long item;
  int pieces, kt0, kt1;
};

// What there is to do: the pieces that the units may be cut into, and their weights.
struct Work {
  long long pieces, cost;
  __device__ void add(const Work& o) {
    pieces += o.pieces;
    cost += o.cost;
  }
  __device__ long long of(Scheme scheme) const {
    return scheme == kPieces ? pieces : cost;
  }
};

struct ScheduleShared {
  Work warp_sum[kThreads / 32];
  long long rem;
  Place at;
  Seq q;
};

// Most work counts fit 32 bits, where a division costs a tenth of one in 64.
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// Work is cut into runs of `each` items, the first `over` of them one longer.
struct Cut {
  long long each, longer;                                    // longer: items in the longer runs
  int over;
  Scheme scheme;
  // kPieces: a run for each item.  `magic`: ceil(2^64 / ctas).
  __device__ Cut(long long work, int ctas, unsigned long long magic, Scheme how) : scheme(how) {
    each = how == kPieces ? 1 : ctas > 1 ? static_cast<long long>(__umul64hi(work, magic)) : work;
    over = static_cast<int>(work - each * ctas);
    longer = over * (each + 1);
  }
  __device__ long long begin(int c) const { return each * c + min(c, over); }
  // the run that holds item x
  __device__ int run_of(long long x) const {
    return static_cast<int>(x < longer ? divide(x, each + 1) : over + divide(x - longer, each));
  }
};

// The whole block: how the work is cut, and the place where run c ends.
// Returns false (everywhere) when there is no such run.  Up to 32 sequences every
// warp looks at all of them for itself, and no thread waits for another warp.
template <int D>
__device__ bool find_place(const PagedParams& p, ScheduleShared* sh, int c, int max_ctas, Cut* cut,
                           Place* at, Seq* seq) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool alone = p.b <= 32;
  const int per = alone ? 1 : (p.b + kThreads - 1) / kThreads;
  const int s0 = min((alone ? lane : tid) * per, p.b), s1 = min(s0 + per, p.b);
  Work mine = {0, 0}, one = {0, 0};                          // one: a head of the last sequence
  Seq q;
  for (int s = s0; s < s1; ++s) {
    q = load_seq(p, s);
    if (q.tiles == 0) continue;
    const int f = q.tiles - 1;                               // full tiles, the last one aside
    const int last = walk_tiles(q.len), rows = tile_rows(p, q, f);
    Work w = {pieces_of(p, rows, last), weight_of(rows <= kNarrowRows).of(last)};
    if (f > 0) {
      const Weight weight = weight_of(false);
      w.pieces += full_pieces_before(p, q, f);
      w.cost += static_cast<long long>(weight.start) * f + (tiles_before(p, q, f) << weight.log_tile);
    }
    one = w;
    w.pieces *= p.h_kv;
    w.cost *= p.h_kv;
    mine.add(w);
  }
  Work incl = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const Work o = {__shfl_up_sync(0xffffffffu, incl.pieces, x), __shfl_up_sync(0xffffffffu, incl.cost, x)};
    if (lane >= x) incl.add(o);
  }
  Work sum = {__shfl_sync(0xffffffffu, incl.pieces, 31), __shfl_sync(0xffffffffu, incl.cost, 31)};
  Work before = {incl.pieces - mine.pieces, incl.cost - mine.cost};
  if (!alone) {
    if (lane == 31) sh->warp_sum[warp] = incl;
    __syncthreads();
    sum = {0, 0};
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const Work v = sh->warp_sum[w];
      if (w < warp) before.add(v);
      sum.add(v);
    }
  }
  // (there are no more pieces than key tiles: no run is shorter than a key tile)
  const Scheme scheme = sum.pieces <= max_ctas ? kPieces : kWeighed;
  const int n = scheme == kPieces ? static_cast<int>(sum.pieces) : max_ctas;
  if (c >= n) return false;
  const long long own = mine.of(scheme), excl = before.of(scheme);
  *cut = Cut(sum.of(scheme), n, p.ctas_magic, scheme);
  const long long x = cut->begin(c + 1) - 1;                 // its last item
  const bool here = own > 0 && excl <= x && x < excl + own;
  long long rem = x - excl, head = one.of(scheme);
  Place pl;
  pl.s = s0;
  if (here && per > 1) {
    for (pl.s = s0; pl.s < s1; ++pl.s) {
      q = load_seq(p, pl.s);
      head = cost_before(p, q, q.tiles, scheme);
      if (rem < head * p.h_kv) break;
      rem -= head * p.h_kv;
    }
  }
  if (alone) {
    const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    pl.s = from;
    rem = __shfl_sync(0xffffffffu, rem, from);
    head = __shfl_sync(0xffffffffu, head, from);
    q.start = __shfl_sync(0xffffffffu, q.start, from);
    q.n = __shfl_sync(0xffffffffu, q.n, from);
    q.len = __shfl_sync(0xffffffffu, q.len, from);
    q.tiles = __shfl_sync(0xffffffffu, q.tiles, from);
  }
  if (alone || here) {
    pl.hk = static_cast<int>(divide(rem, head));
    rem -= pl.hk * head;
    pl.r = 0;
    pl.item = rem + 1;                                       // for a single row tile
  }
  if (!alone) {
    if (here) {
      sh->at = pl;
      sh->rem = rem;
      sh->q = q;
    }
    __syncthreads();
    pl = sh->at;
    rem = sh->rem;
    q = sh->q;
  }
  *at = pl;
  *seq = q;
  if (seq->tiles > 1) {
    // the last row tile that begins at or before rem: 32 probes a round (every
    // warp does it for itself)
    int lo = 0, hi = seq->tiles;
    long long before_lo = 0;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int probe = lo + lane * step;
      const long long cost = probe < hi ? cost_before(p, *seq, probe, scheme) : rem + 1;
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, cost <= rem));
      before_lo = __shfl_sync(0xffffffffu, cost, k);
      lo += k * step;
      hi = min(hi, lo + step);
    }
    at->r = lo;
    at->item = rem - before_lo + 1;
  }
  if (scheme == kPieces) {
    const unsigned tiles = walk_tiles(tile_keys(p, *seq, at->r)), i = static_cast<unsigned>(at->item);
    const unsigned pieces = unit_pieces(p, *seq, at->r, tiles);
    at->pieces = pieces;
    at->kt0 = i - 1;
    at->kt1 = i;
    if (pieces != tiles) {                                   // (a piece has up to 16: in 32 bits)
      at->kt0 = (i - 1) * tiles / pieces;
      at->kt1 = i * tiles / pieces;
    }
  }
  return true;
}

// The pieces of one run, from the last to the first; every role walks its
// own copy.  A key tile belongs to the run that its last item lies in.
struct Walk {
  int s, hk, r;                                              // the piece's unit
  Seq q;
  int kt0, kt1, tiles;                                       // its key tiles [kt0, kt1) of `tiles`
  int keys, rows;                                            // the unit's keys, rows that are queries
  Weight w;
  Scheme scheme;
  long long off;                                             // where the unit begins, seen from the run's begin

  // Key tiles that lie before item x of the unit.
  __device__ __forceinline__ int tiles_at(long long x) const {
    return x <= w.start ? 0 : static_cast<int>((x - w.start) >> w.log_tile);
  }
  __device__ __forceinline__ void load(const PagedParams& p) {
    keys = tile_keys(p, q, r);
    tiles = walk_tiles(keys);
    rows = tile_rows(p, q, r);
    w = weight_of(rows <= kNarrowRows);
  }
  // The first piece of a run of `run` items that ends at `end`; false: none.
  __device__ bool begin(const PagedParams& p, const Place& end, const Seq& seq, long long run, Scheme how) {
    scheme = how;
    s = end.s;
    hk = end.hk;
    r = end.r;
    q = seq;
    load(p);
    off = run - end.item;
    if (scheme == kPieces) {                                 // the whole run
      kt0 = end.kt0;
      kt1 = end.kt1;
      return true;
    }
    kt1 = tiles_at(end.item);
    kt0 = tiles_at(-off);
    return kt1 > kt0 || next(p);
  }
  __device__ bool next(const PagedParams& p) {
    if (off <= 0) return false;
    if (--r < 0) {
      if (--hk < 0) {
        do {
          if (--s < 0) return false;
          q = load_seq(p, s);
        } while (q.n == 0);
        hk = p.h_kv - 1;
      }
      r = q.tiles - 1;
    }
    load(p);
    off -= w.of(tiles);
    kt0 = tiles_at(-off);
    kt1 = tiles;
    return true;
  }
  // key tiles of the piece that hold keys (all, but for a unit that sees none)
  __device__ int count() const { return min(kt1, (keys + kBN - 1) / kBN) - kt0; }
};

// --------------------------------------------------------------------- merge
// Workspace slots: what run c publishes is slot c: O as [D / 4][rows] vectors
// of four columns and, right behind, (m, l) as [rows].  (A run that publishes a
// sliced unit's last piece, below, may publish the next one's first piece too:
// last pieces have slots of their own, split_ctas + c / 3, as they are three runs
// apart at least.)  A slot has a flag, which is the call's number once the slot
// is written and is put back to zero when everybody has seen it.  A run merges at its end, when its K and V stages
// are idle: the published pieces come into that memory by asynchronous copies.
//
// The pieces j = 0, 1, .. of a unit are runs c0 + j.  Few are merged by the last
// one, which keeps its own piece.  More are all published, and the runs that end
// with them (SLICERS) merge a slice each, a range of rows or, if there are more
// slicers than rows, of rows and columns: all of P pieces cost one SM P times a
// piece's bytes (64 KB take about a microsecond), a slice of them no more than
// one piece's, but publishing the last piece and asking for all others' takes 2 to
// 3 us.  One sequence of 26595 positions, 69 new tokens of 2 heads of 64 (52
// pieces of 18 KB a head) takes 17 us in slices and took 27 as a tree of radix 4.
// Of 8 pieces of 64 KB (32 tokens over 8192 positions, 16 / 4 heads of 128) the last
// run alone takes 23.8 us, slices 22.1; of 3 of 128 KB (3
// chunks of 200 tokens, 8 / 1 heads of 256) 28.8 and 33.2.  In a cut by weight,
// where every SM merges at once, 5 to 7 of 64 KB (2 chunks of 992 and 188 tokens, 20
// / 4 heads of 128) take 66.0 and 66.1 us, 4 69.1 in slices; of up to 16 narrow ones
// (single tokens, 32 / 8 heads of 128) 12.6 us, in slices 14.8.
//
// A slicer waits for pieces of later runs too, and those need not be running
// (with another kernel on the GPU): it waits so long and then leaves its slice
// to the unit's last run, whose own wait is for earlier ones alone.  A slicer's
// STATE says what became of its slice: kOpen while it waits, kTaken, kLeft.
// pieces that the last run merges alone, at most
constexpr int kTogether = 8, kTogetherPieces = 4, kTogetherNarrow = 16;
constexpr int kSliceVectors = 8;           // of a slice, at least (152 pieces of 8 rows: 34.7 us, 35.3 with 16, 41.8 with 32)
#ifndef SDPA_TEST_PATIENCE
#define SDPA_TEST_PATIENCE (1 << 17)       // (a test leaves slices at once)
#endif
constexpr long long kPatience = SDPA_TEST_PATIENCE;   // clock cycles, about 65 us: runs end within a few of each other
// The last run waits for the others' pieces as long as a CTA's warps wait for one
// another, and longer by what its run takes: an item, a quarter of a key tile, takes
// about 450 clock cycles.
#ifndef SDPA_TEST_ITEM_CYCLES
#define SDPA_TEST_ITEM_CYCLES 4096         // (a test waits longer)
#endif
constexpr long long kItemCycles = SDPA_TEST_ITEM_CYCLES;
enum State : unsigned long long { kOpen, kTaken, kLeft };

__device__ __forceinline__ unsigned long long load_acquire(const unsigned long long* x) {
  unsigned long long v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(x) : "memory");
  return v;
}

// Waits until the flag is this call's number (or the state is decided):
// false after `limit` clock cycles, or when another thread has given up.
template <class Ready>
__device__ __forceinline__ bool wait_word(const unsigned long long* x, Ready ready, long long limit,
                                          const AbortState& ab) {
  const long long t0 = clock64();
  while (!ready(load_acquire(x))) {
    if (*ab.flag || clock64() - t0 > limit) return false;
  }
  return true;
}

__device__ __forceinline__ void set_flag(unsigned long long* flag, unsigned long long call) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(flag), "l"(call) : "memory");
}

// 2^(m - sub), 0 for a piece that saw nothing
__device__ __forceinline__ float weight(float m, float sub) { return ex2_approx(m - sub); }

// --------------------------------------------------------------------- split
template <int D>
struct PCfg {
  static constexpr int kBoxCols = D < 64 ? D : 64;
  static constexpr int kBoxes = D / kBoxCols;
  static constexpr int kRowBytes = kBoxCols * 2;
  static constexpr uint32_t kLayout = kRowBytes == 128 ? 2u : (kRowBytes == 64 ? 4u : 6u);
  static constexpr uint32_t kSBO = 8 * kRowBytes;
  static constexpr int kStepsPerRow = kRowBytes / 32;
  static constexpr int kQBox = kBlockM * kRowBytes;
  static constexpr int kKVBox = kBN * kRowBytes;
  static constexpr int kQBytes = kBoxes * kQBox;
  static constexpr int kKVBytes = kBoxes * kKVBox;           // one tile of K or of V
  // K and V stages: what fits next to Q with two CTAs per SM (one at d = 256)
  static constexpr int kRing = D >= 128 ? 2 : 4;
  // With four stages K and V of a tile come together, on one barrier (k_full),
  // and are free together: the producer's wait and its announcement of the
  // bytes take as long as the copies of a small tile.  With two, K's stage is
  // worth having back before V's.
  static constexpr bool kJoint = kRing >= 4;
  static constexpr int kKOff = kQBytes;
  static constexpr int kVOff = kKOff + kRing * kKVBytes;
  // O columns of a tensor-memory load
  static constexpr int kOChunk = D < 32 ? D : 32;
  // Exchange memory: a narrow tile's quarters lay their rows here to be summed
  // (16 columns of 16 rows at least), a wide tile's warps turn theirs, 64 bytes
  // of each at a time (rows padded by 16).
  static constexpr int kXOff = kVOff + kRing * kKVBytes;
  static constexpr int kTurnRow = 64 + 16;
  static constexpr int kTurnSlot = 32 * kTurnRow;
  static constexpr int kXBytes = 4 * kTurnSlot;
  static_assert(4 * kNarrowRows * 16 * 4 <= kXBytes, "quarters");
  static constexpr int kXmlOff = kXOff + kXBytes;            // the quarters' (m, l)
  // merging: the idle K and V stages hold a wide piece's O, or with the exchange
  // memory behind them two of a narrow tile's, or of every piece a vector and
  // its (m, l) beside what the threads that share a vector exchange
  static constexpr int kMergeBytes = 2 * kRing * kKVBytes + kXBytes;
  static constexpr int kPartBytes = kBlockM * (16 + 8);
  static_assert(2 * kRing * kKVBytes >= kBlockM * D * 4 && kMergeBytes >= 2 * kNarrowRows * (D * 4 + 8) &&
                    kMergeBytes - kPartBytes >= kPagedMaxRuns * (16 + 8), "pieces");
  static constexpr int kBarOff = kXmlOff + 4 * kQuarter * 8;
  // q_full, q_empty, k_full[R], v_full[R], s_full[R], o_full[R], p_full[2], o_last, o_free,
  // merge, drain
  static constexpr int kNumBars = 2 + 4 * kRing + 2 + 4;
  // A tile of K or V lies as [8 rows][column block][row of the eight]: groups of eight
  // rows are equally far apart, as the operands' descriptors want them, however
  // many copies the tile came in, one for each page that it spans: a copy costs its
  // issue (100 clk and more) before its bytes, and copying each column block of a
  // page by itself took 136 us instead of 112 for 4 chunks of 512 tokens behind 7680
  // positions (heads of 128, pages of 16).
  static constexpr int kGroupBytes = kBoxes * kSBO;
  static constexpr int kSmemBytes = kBarOff + kNumBars * 8 + 16 + 1024;
  static constexpr uint32_t kOCol = 2 * kBN;
  static constexpr uint32_t kTmemCols = kOCol + D <= 256 ? 256u : 512u;
  static constexpr int kMinBlocks = static_cast<int>(512u / kTmemCols);
  static constexpr uint32_t kIdescS = idesc_bf16(kBlockM, kBN, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16(kBlockM, D, false, true);
  static constexpr uint32_t kDescHi = (kSBO >> 4) | (1u << 14) | (kLayout << 29);
  static constexpr uint32_t kDescHiKV = (kGroupBytes >> 4) | (1u << 14) | (kLayout << 29);
  static_assert(kSmemBytes * kMinBlocks <= 232448 - 1024 * kMinBlocks, "CTAs per SM");
  static_assert(kKOff % 1024 == 0 && kVOff % 1024 == 0 && kKVBox % 1024 == 0, "alignment");
  static_assert(kBN / kPagedMinPage <= 8 && kPagedMinPage % 8 == 0, "a lane of the producer warp for each copy");
};

// Where row rw of a tile begins in the output (row0: the tile's first token, head0:
// the group's first head), and four columns into the output.
template <int D>
__device__ __forceinline__ long long out_begin(const PagedParams& p, int row0, int head0, int rw) {
  const int tok = token_of(p, rw);
  return (static_cast<long long>(row0 + tok) * p.h + head0 + rw - tok * p.group) * D;
}
__device__ __forceinline__ void write_four(uint16_t* at, const float4& v, float f) {
  *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
}

// Where the parts of a unit are: piece j of `of` (this run's) is run cta.
struct Pieces {
  int rows, row0, head0, cta, j, of;
  bool sliced;
  __device__ __forceinline__ int place(const PagedParams& p, int i) const {
    const int c = cta - j + i;
    return sliced && i == of - 1 ? p.split_ctas + c / 3 : c;
  }
};

// All softmax threads meet at `bar` and see what each wrote before; `met`
// counts the times.
struct Meeting {
  uint64_t* bar;
  int met;
  AbortState ab;
  __device__ __forceinline__ bool operator()() { return within<kWaitLimitCycles>(); }
  // Where some of them come from a wait for other runs, which has a limit of its
  // own: when that is over the abort flag ends the others' wait here too.  (A limit
  // worked out here would cost registers in the loops: 8 bytes spilled at d = 128.)
  __device__ __forceinline__ bool after_waits() { return within<(kWaitLimitCycles << 10)>(); }

 private:
  template <long long kLimit>
  __device__ __forceinline__ bool within() {
    mbar_arrive(bar);
    return mbar_wait_warp(bar, static_cast<uint32_t>(met++) & 1u, ab, kLimit);
  }
};

__device__ __forceinline__ void time_out(const AbortState& ab) {
  *ab.flag = 1;
  atomicOr(ab.status, kStatusTimeout);
}

// Slice k of a unit's pieces, merged into the output: rows block k % row_blocks,
// columns block k / row_blocks.  `ring`: kMergeBytes of idle memory.  There is one
// warp on each of the SM's schedulers here, so every instruction's latency shows:
// the rows' weights are worked out first, places move on without divisions.
template <int D>
__device__ __forceinline__ bool merge_slice(const PagedParams& p, const Pieces& u, uint8_t* ring, int k, int row_blocks,
                                            int col_blocks, Meeting& meet) {
  const int tid = threadIdx.x, rows = u.rows, of = u.of;
  auto slot = [&](int i) { return p.slots + static_cast<long long>(u.place(p, i)) * p.slot_bytes; };
  const int rb = k % row_blocks, cb = k / row_blocks;
  const int r_begin = rb * rows / row_blocks, r_end = (rb + 1) * rows / row_blocks;
  const int c_begin = cb * (D / 4) / col_blocks, c_end = (cb + 1) * (D / 4) / col_blocks;
  // as many rows, and then columns, at a time as the memory holds of all pieces
  constexpr int kRoom = PCfg<D>::kMergeBytes - PCfg<D>::kPartBytes;
  const int room = kRoom / of;
  const int most_rows = min(r_end - r_begin, room / 24);
  const int most_cols = min(c_end - c_begin, (room / most_rows - 8) / 16);
  float4* o = reinterpret_cast<float4*>(ring);
  float4* part_o = reinterpret_cast<float4*>(ring + kRoom);
  long long* begin = reinterpret_cast<long long*>(part_o + kBlockM);   // of the rows in the output
  for (int r0 = r_begin; r0 < r_end; r0 += most_rows) {
    for (int c0 = c_begin; c0 < c_end; c0 += most_cols) {
      const int nr = min(most_rows, r_end - r0), nc = min(most_cols, c_end - c0), nv = nr * nc;
      float2* ml = reinterpret_cast<float2*>(o + of * nv);
      if ((r0 > r_begin || c0 > c_begin) && !meet()) return false;
      // a thread takes vectors of every piece, or if there are few a warp takes
      // those of every fourth piece
      const bool many = nv >= kBlockM;
      const int v0 = many ? tid : tid & 31, step = many ? kBlockM : 32;
      const int i0 = many ? 0 : tid >> 5, i_step = many ? 1 : 4;
      const int dc = step / nr, dr = step - dc * nr;
      int c = v0 / nr, r = v0 - c * nr;
      for (int v = v0; v < nv; v += step) {
        const int at = ((c0 + c) * rows + r0 + r) * 16;
#pragma unroll 4
        for (int i = i0; i < of; i += i_step) cp_async16(o + i * nv + v, slot(i) + at);
        c += dc;
        r += dr;
        if (r >= nr) {
          r -= nr;
          ++c;
        }
      }
#pragma unroll 4
      for (int x = tid; x < of * nr; x += kBlockM) {
        const int i = x / nr;
        ml[x] = __ldcg(reinterpret_cast<const float2*>(slot(i) + rows * D * 4) + r0 + x - i * nr);
      }
      if (tid < nr) begin[tid] = out_begin<D>(p, u.row0, u.head0, r0 + tid);
      cp_async_wait<0>();
      if (!meet()) return false;
      // what each piece weighs in each row, in the place of m: 2^(m - M) / l of all;
      // `lanes` lanes for a row
      int lanes = 32;
      while (lanes * nr > kBlockM) lanes >>= 1;
      const int row = tid / lanes;
      float top = -INFINITY, sum = 0.f;
      if (row < nr)
        for (int i = tid & (lanes - 1); i < of; i += lanes) top = fmaxf(top, ml[i * nr + row].x);
      for (int x = lanes >> 1; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float base = top == -INFINITY ? 0.f : top;
      if (row < nr)
        for (int i = tid & (lanes - 1); i < of; i += lanes) sum += ml[i * nr + row].y * weight(ml[i * nr + row].x, base);
      for (int x = lanes >> 1; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      if (row < nr)
        for (int i = tid & (lanes - 1); i < of; i += lanes) ml[i * nr + row].x = weight(ml[i * nr + row].x, base) * inv;
      if (!meet()) return false;
      // the sums; `parts` threads for a vector, each summing every parts'th piece
      auto sum_of = [&](int v, int rw, int from, int by) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = from; i < of; i += by) {
          const float4 x = o[i * nv + v];
          const float f = ml[i * nr + rw].x;
          acc.x = fmaf(x.x, f, acc.x);
          acc.y = fmaf(x.y, f, acc.y);
          acc.z = fmaf(x.z, f, acc.z);
          acc.w = fmaf(x.w, f, acc.w);
        }
        return acc;
      };
      if (many) {
        c = v0 / nr;
        r = v0 - c * nr;
        for (int v = v0; v < nv; v += kBlockM) {
          write_four(p.out + begin[r] + (c0 + c) * 4, sum_of(v, r, 0, 1), 1.f);
          c += dc;
          r += dr;
          if (r >= nr) {
            r -= nr;
            ++c;
          }
        }
      } else {
        const int parts = kBlockM / nv, part = tid / nv, v = tid - part * nv;
        if (part < parts) part_o[tid] = sum_of(v, v % nr, part, parts);
        if (!meet()) return false;
        if (part == 0) {
          float4 acc = part_o[v];
          for (int i = 1; i < parts; ++i) {
            const float4 x = part_o[i * nv + v];
            acc.x += x.x;
            acc.y += x.y;
            acc.z += x.z;
            acc.w += x.w;
          }
          write_four(p.out + begin[v % nr] + (c0 + v / nr) * 4, acc, 1.f);
        }
      }
    }
  }
  return true;
}

// All softmax threads of a run that has published its piece of a sliced unit: its
// slice, if it takes one.  `most`: runs that can take one, the unit's last ones;
// `left`: two words of shared memory, zero.  Returns how often the threads have
// met, -1 if they gave up.
template <int D>
__device__ __forceinline__ int merge_slices(const PagedParams& p, const Pieces& u, uint8_t* ring, int most, uint64_t* bar,
                                         int met, long long limit, volatile int* left, AbortState ab) {
  Meeting meet{bar, met, ab};
  most = min(most, max(1, u.rows * (D / 4) / kSliceVectors));
  const int row_blocks = min(most, u.rows), col_blocks = most / row_blocks;
  const int slicers = row_blocks * col_blocks;
  const int first = u.cta - u.j + u.of - slicers;            // the first slice's run
  const bool final = u.j == u.of - 1;
  if (u.cta < first) return met;
  bool got = true;
  for (int x = threadIdx.x; x < u.of && got; x += kBlockM)
    got = wait_word(p.flags + u.place(p, x), [&](unsigned long long v) { return v == p.call; },
                    final ? limit : kPatience, ab);
  if (!got) {
    if (final) time_out(ab);
    else left[0] = 1;
  }
  if (!meet.after_waits() || *ab.flag != 0) return -1;
  const bool taken = left[0] == 0;
  if (threadIdx.x == 0)
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p.states + u.cta),
                 "l"(static_cast<unsigned long long>(taken ? kTaken : kLeft)) : "memory");
  if (!taken) return meet.met;
  int k = u.cta - first;
  while (true) {
    if (!merge_slice<D>(p, u, ring, k, row_blocks, col_blocks, meet)) return -1;
    if (!final) return meet.met;
    if (k == slicers - 1) {
      // what became of the others'?  Then nobody waits for the flags any more.
      for (int x = threadIdx.x; x < slicers - 1; x += kBlockM) {
        if (!wait_word(p.states + first + x, [](unsigned long long v) { return v != kOpen; }, limit, ab)) time_out(ab);
        else if (load_acquire(p.states + first + x) == kLeft) left[1] = 1;
      }
      if (!meet.after_waits() || *ab.flag != 0) return -1;
      for (int x = threadIdx.x; x < u.of; x += kBlockM) p.flags[u.place(p, x)] = 0;
      if (left[1] == 0) return meet.met;
      k = -1;
    } else if (!meet()) {                                    // (the memory has been read)
      return -1;
    }
    do ++k; while (k < slicers - 1 && load_acquire(p.states + first + k) != kLeft);
    if (k == slicers - 1) return meet.met;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, PCfg<D>::kMinBlocks)
    sdpa_paged_split(const __grid_constant__ PagedParams p) {
  using C = PCfg<D>;
  constexpr int R = C::kRing;
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScheduleShared sched;
  __shared__ int left[2];                                    // slices left to the unit's last run: this one's, others'
  const uint32_t raw_u32 = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);
  const uint32_t smem_base = smem_u32(smem);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* q_empty = q_full + 1;     // the last scores of a piece are done with Q
  uint64_t* k_full = q_empty + 1;
  uint64_t* v_full = k_full + R;
  uint64_t* s_full = v_full + R;      // scores of tile u done (stage u % R of K is free)
  uint64_t* o_full = s_full + R;      // O += P V of tile u done (stage u % R of V is free)
  uint64_t* p_full = o_full + R;
  uint64_t* o_last = p_full + 2;      // once a piece, after its last O += P V
  uint64_t* o_free = o_last + 1;      // once a piece, when the softmax warps have read O
  uint64_t* merge = o_free + 1;       // steps of exchanging, publishing and merging
  uint64_t* drain = merge + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const AbortState ab{abort_flag, p.status};
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    left[0] = left[1] = 0;
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < R; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(v_full + s, 1);
      mbar_init(s_full + s, 1);
      mbar_init(o_full + s, 1);
    }
    for (int s = 0; s < 2; ++s) mbar_init(p_full + s, kBlockM);
    mbar_init(o_last, 1);
    mbar_init(o_free, kBlockM);
    mbar_init(merge, kBlockM);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  if (threadIdx.x == kProducerWarp * 32) {
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_q_narrow);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  tc_fence_before();
  __syncthreads();                                           // the set-up above, for all
  // not before the block has met: the next kernel's block could be given this
  // one's tensor memory, and then wait for this grid, which waits for the memory
  griddep_launch_dependents();
  griddep_wait();

  Cut cut(0, 1, 0, kWeighed);
  Place last;
  Seq last_seq;
  const int cta = static_cast<int>(blockIdx.x);
  const bool any = find_place<D>(p, &sched, cta, static_cast<int>(gridDim.x), &cut, &last, &last_seq);
  const long long run = any ? cut.begin(cta + 1) - cut.begin(cta) : 0;
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (run > 0 && warp == kProducerWarp) {
    // ---------------------------------------------------------- producer
    // Pages smaller than a tile are `parts` of it, each copied by a lane, all at
    // once (one lane doing them one after the other took 270 clk for each).  A
    // lane reads the page of its part two tiles ahead and looks at it only when it
    // uses it: waiting for each read took 700 clk a tile.
    const int box_shift = min(p.page_shift, kBNShift);
    const int box_rows = 1 << box_shift;
    const int row_mask = (1 << p.page_shift) - 1;
    // (together: lanes 0 - 7 copy K, lanes 8 - 15 V)
    const int part = C::kJoint ? lane & 7 : lane;
    const bool copies = part << box_shift < kBN && (!C::kJoint || lane < 16);
    const uint32_t dst = static_cast<uint32_t>((part << box_shift) * C::kRowBytes * C::kBoxes);
    Walk w;
    int u0 = 0, pieces = 0, k_issued = 0, v_issued = 0;
    bool go = true;
    for (bool more = w.begin(p, last, last_seq, run, cut.scheme); more; more = go && w.next(p)) {
      const int n = w.count();
      if (n <= 0) continue;
      const int kt0 = w.kt0;
      const int32_t* pages = p.page_table + static_cast<long long>(w.s) * p.pages_per_seq;
      const int key_lane = kt0 * kBN + (part << box_shift);
      // this lane's part of tile i: does it hold keys, and in which page
      auto holds = [&](int i) { return copies && i < n && key_lane + i * kBN < w.q.len; };
      auto page_of = [&](int i) -> int { return holds(i) ? pages[(key_lane + i * kBN) >> p.page_shift] : 0; };
      auto load = [&](const CUtensorMap* map, uint64_t* bar, uint8_t* stage, int i, int page) {
        const int rows = min(kBN, (w.q.len - (kt0 + i) * kBN + box_rows - 1) >> box_shift << box_shift);
        if (lane == 0)
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(rows) *
                                         (C::kRowBytes * C::kBoxes * (C::kJoint ? 2 : 1)));
        __syncwarp();
        if (holds(i)) {
          // page numbers outside the cache read as zeros and are reported
          if (page < 0 || page >= p.n_pages) {
            atomicOr(p.status, kStatusBadPage);
            page = p.n_pages;
          }
          tma_load_5d(map, bar, stage + dst, 0, 0, 0,
                      (w.hk << (p.page_shift - 3)) + (((key_lane + i * kBN) & row_mask) >> 3), page);
        }
      };
      int page_v = page_of(0), page_k = page_v, page_n = page_of(1);
      auto load_k = [&](int i) -> bool {
        const int u = u0 + i, s = u % R;
        if (u >= R && !mbar_wait_warp((C::kJoint ? o_full : s_full) + s, static_cast<uint32_t>(u / R - 1) & 1u, ab))
          return false;
        const bool v = C::kJoint && lane >= 8;
        load(v ? &p.tm_v : &p.tm_k, k_full + s, smem + (v ? C::kVOff : C::kKOff) + s * C::kKVBytes, i, page_k);
        k_issued = u + 1;
        return true;
      };
      if (!(go = load_k(0))) break;
      // Q, once the scores of the piece before are done with it
      if (pieces > 0 && !(go = mbar_wait_warp(q_empty, static_cast<uint32_t>(pieces - 1) & 1u, ab))) break;
      {
        // lane c * 4 + y: column box c, for a narrow tile into quarter y
        const bool narrow = w.rows <= kNarrowRows;
        const int rows = (narrow ? kNarrowRows / p.group : p.tile_tokens) * p.group;   // of the box
        if (lane == 0)
          mbar_arrive_expect_tx(q_full, static_cast<uint32_t>((narrow ? 4 : 1) * rows * C::kRowBytes * C::kBoxes));
        __syncwarp();
        const int c = lane >> 2, y = lane & 3;
        if (c < C::kBoxes && (narrow || y == 0))
          tma_load_3d(narrow ? &p.tm_q_narrow : &p.tm_q, q_full,
                      smem + c * C::kQBox + y * kQuarter * C::kRowBytes, c * C::kBoxCols,
                      w.hk * p.group, w.q.start + w.r * p.tile_tokens);
      }
      ++pieces;
      for (int i = 0; go && i < n; ++i) {
        // K of the next tile goes ahead of V of this one: its stage is free earlier
        page_k = page_n;
        page_n = page_of(i + 2);
        if (i + 1 < n && !(go = load_k(i + 1))) break;
        if constexpr (C::kJoint) continue;
        const int u = u0 + i, s = u % R;
        if (u >= R && !(go = mbar_wait_warp(o_full + s, static_cast<uint32_t>(u / R - 1) & 1u, ab))) break;
        load(&p.tm_v, v_full + s, smem + C::kVOff + s * C::kKVBytes, i, page_v);
        page_v = page_k;
        v_issued = u + 1;
      }
      u0 += n;
    }
    // let every copy land before the CTA can exit
    if (pieces > 0) mbar_wait_drain(q_full, static_cast<uint32_t>(pieces - 1) & 1u);
    for (int u = max(0, k_issued - R); u < k_issued; ++u)
      mbar_wait_drain(k_full + u % R, static_cast<uint32_t>(u / R) & 1u);
    for (int u = max(0, v_issued - R); u < v_issued; ++u)
      mbar_wait_drain(v_full + u % R, static_cast<uint32_t>(u / R) & 1u);
  } else if (run > 0 && warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    auto lo = [](uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); };
    const uint32_t q_lo = lo(smem_base, 16);
    auto issue_s = [&](int u) -> bool {
      const int ks = u % R;
      if (!mbar_wait_warp(k_full + ks, static_cast<uint32_t>(u / R) & 1u, ab)) return false;
      tc_fence_after();
      const uint32_t d = tmem + static_cast<uint32_t>((u & 1) * kBN);
      const uint32_t b0 = lo(smem_base + C::kKOff + ks * C::kKVBytes, 16);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        constexpr int kS = C::kStepsPerRow;
        mma_bf16_ss_warp(d, q_lo + static_cast<uint32_t>(((k / kS) * C::kQBox + (k % kS) * 32) >> 4),
                         C::kDescHi, b0 + static_cast<uint32_t>(((k / kS) * C::kSBO + (k % kS) * 32) >> 4),
                         C::kDescHiKV, C::kIdescS, k > 0 ? 1u : 0u);
      }
#ifdef SDPA_TEST_WITHHOLD_FIRST_S_COMMIT
      // (test builds only, never in libsdpa.so: the first score tile of a CTA
      // is never signalled, so the waits on it run out)
      if (u == 0) return true;
#endif
      mma_commit_warp(s_full + ks);
      return true;
    };
    auto issue_pv = [&](int u, bool accumulate) {
      const uint32_t pa = tmem + static_cast<uint32_t>((u & 1) * kBN);
      const uint32_t b0 = lo(smem_base + C::kVOff + (u % R) * C::kKVBytes, C::kSBO);
#pragma unroll
      for (int k = 0; k < kBN / 16; ++k)
        mma_bf16_ts_warp(tmem + C::kOCol, pa + static_cast<uint32_t>(k * 8),
                         b0 + static_cast<uint32_t>((k * 2 * C::kGroupBytes) >> 4), C::kDescHiKV, C::kIdescPV,
                         (accumulate || k > 0) ? 1u : 0u);
    };
    Walk w;
    int u = 0, pieces = 0;
    bool ok = true;
    for (bool more = w.begin(p, last, last_seq, run, cut.scheme); more; more = ok && w.next(p)) {
      const int n = w.count();
      if (n <= 0) continue;
      ok = mbar_wait_warp(q_full, static_cast<uint32_t>(pieces) & 1u, ab);
      if (!ok) break;
      tc_fence_after();
      if (!(ok = issue_s(u))) break;
      if (n == 1) mma_commit_warp(q_empty);
      for (int i = 0; i < n; ++i, ++u) {
        // S(u+1) into the buffer of P(u-1): PV(u-1) was issued before it
        if (i + 1 < n) {
          if (!(ok = issue_s(u + 1))) break;
          if (i + 2 == n) mma_commit_warp(q_empty);
        }
        // O of the piece before has been read out
        if (i == 0 && pieces > 0 &&
            !(ok = mbar_wait_warp(o_free, static_cast<uint32_t>(pieces - 1) & 1u, ab)))
          break;
        ok = mbar_wait_warp(p_full + (u & 1), static_cast<uint32_t>(u >> 1) & 1u, ab) &&
             (C::kJoint || mbar_wait_warp(v_full + u % R, static_cast<uint32_t>(u / R) & 1u, ab));
        if (!ok) break;
        tc_fence_after();
        issue_pv(u, i > 0);
        mma_commit_warp(o_full + u % R);
        if (i + 1 == n) mma_commit_warp(o_last);
      }
      ++pieces;
    }
    mma_commit_warp(drain);
    mbar_wait_drain(drain, 0);
  } else if (run > 0) {
    // ---------------------------------------------------------- softmax
    const int quarter = warp & 3;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float scale_log2 = p.scale_log2;
    const float2 sc2 = make_float2(scale_log2, scale_log2);
    Walk w;
    bool more = w.begin(p, last, last_seq, run, cut.scheme);
    int u = 0, pieces = 0;
    Meeting meet{merge, 0, ab};
    bool ok = true;

    // Rows of V past the length hold whatever the page held (or an older
    // tile): their weights are zero, but zero times an infinity or a NaN is a
    // NaN, so they are cleared.  (All four warps, before P is handed over.)
    auto clear_tail = [&](int key0) -> bool {
      if (key0 + kBN <= w.q.len) return true;
      if (!mbar_wait_warp((C::kJoint ? k_full : v_full) + u % R, static_cast<uint32_t>(u / R) & 1u, ab)) return false;
      uint8_t* v = smem + C::kVOff + (u % R) * C::kKVBytes;
      const int keep = w.q.len - key0;                       // in [1, kBN)
      constexpr int kPerRow = C::kRowBytes / 16;
      for (int x = threadIdx.x; x < (kBN - keep) * kPerRow; x += kBlockM) {
        const int r = keep + x / kPerRow;
        uint8_t* at = v + (r >> 3) * C::kGroupBytes + (r & 7) * C::kRowBytes + x % kPerRow * 16;
#pragma unroll
        for (int c = 0; c < C::kBoxes; ++c) *reinterpret_cast<uint4*>(at + c * C::kSBO) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      return true;
    };
    // The running maximum of a row, given this tile's: moves only when it
    // grew by more than the threshold (always on the first tile).  Returns
    // the factor for what was summed so far.  O is rescaled after O += P(u-1)
    // V(u-1): that barrier's previous phase is complete (S(u) was issued
    // after it) and its next one needs this softmax's next P, so the parity
    // wait is exact.  Rows that are no query hold leftovers and never ask.
    auto move_max = [&](int i, float mx, bool valid, float& m_used, float& l, float& alpha, bool& rescale) -> bool {
      const float m_new = fmaxf(m_used, mx * scale_log2);
      alpha = 1.f;
      rescale = false;
      if (i == 0) {
        m_used = m_new;
        return true;
      }
      const bool need = valid && m_new > m_used + kRescaleThreshold;
      rescale = __any_sync(0xffffffffu, need);
      if (need) {
        alpha = ex2_approx(m_used - m_new);
        m_used = m_new;
        l *= alpha;
      }
      if (rescale) {
        if (!mbar_wait_warp(o_full + (u - 1) % R, static_cast<uint32_t>((u - 1) / R) & 1u, ab)) return false;
        tc_fence_after();
      }
      return true;
    };
    auto rescale_o = [&](float alpha) {
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
    };

    for (; more; more = w.next(p)) {
      const int kt0 = w.kt0, n = w.count();
      const int rows = w.rows;
      const bool narrow = rows <= kNarrowRows;
      const int row = narrow ? lane : quarter * 32 + lane;   // row of the tile
      const int token = token_of(p, row), head = row - token * p.group;
      const int token0 = w.r * p.tile_tokens;
      const bool valid = row < rows;
      const int pos0 = w.q.len - w.q.n + token0;             // position of the tile's first row
      const int pos = pos0 + token;                          // this row sees keys 0 .. pos
      // a piece of a unit that later runs merge, or that this run merges with
      // what earlier runs published
      const bool open_above = w.kt1 < w.tiles, open_below = kt0 > 0;
      const bool whole = !open_above && !open_below;
      // its pieces, and which of them this is (the first key tile's last item says
      // which run it belongs to)
      int of = 1, j = 0;
      if (!whole) {
        j = static_cast<int>(last.item) - 1;
        of = last.pieces;
        if (cut.scheme != kPieces) {
          const long long begin = cut.begin(cta) + w.off;
          const int first = cut.run_of(begin + w.w.of(1) - 1);
          j = cta - first;
          of = cut.run_of(begin + w.w.of(w.tiles) - 1) - first + 1;
        }
      }
      const bool sliced = of > (narrow ? kTogetherNarrow : cut.scheme == kPieces ? kTogetherPieces : kTogether), publishes = open_above || sliced;
      const int sources = publishes ? 0 : of - 1;            // the runs before this one, merged here
      const Pieces unit{rows, w.q.start + token0, w.hk * p.group, cta, j, of, sliced};
      const int place = unit.place(p, j);                    // this piece's slot
      const long long out_row =
          static_cast<long long>(w.q.start + token0 + token) * p.h + w.hk * p.group + head;
      // a published piece of this unit: its bytes, run sl's slot, its (m, l)
      const int o_bytes = rows * D * 4, piece_bytes = o_bytes + (rows * 8 + 15) / 16 * 16;
      auto slot = [&](int sl) { return p.slots + static_cast<long long>(sl) * p.slot_bytes; };
      auto ml_of = [&](uint8_t* piece) { return reinterpret_cast<float2*>(piece + o_bytes); };
      uint8_t* ring = smem + C::kKOff;
      // The slot is written: its flag, released after everybody's writes.
      auto publish = [&]() -> bool {
#ifdef SDPA_TEST_LATE_PUBLISH
        // (test builds only, never in libsdpa.so: a piece that is all of its run,
        // and not the unit's last, is published this many clock cycles late)
        if (open_above && w.off <= 0)
          for (const long long t0 = clock64(); clock64() - t0 < SDPA_TEST_LATE_PUBLISH;) {}
#endif
        if (!meet()) return false;
        if (threadIdx.x == 0) set_flag(p.flags + place, p.call);
        return true;
      };
      const long long patience = kWaitLimitCycles + kItemCycles * run;
      // What this run merges alone has been published.
      auto wait_sources = [&]() -> bool {
        bool got = true;
        if (static_cast<int>(threadIdx.x) < sources) {
          unsigned long long* flag = p.flags + cta - 1 - static_cast<int>(threadIdx.x);
          got = wait_word(flag, [&](unsigned long long v) { return v == p.call; }, patience, ab);
          if (got) *flag = 0;
          else time_out(ab);
        }
        return __all_sync(0xffffffffu, got) && meet.after_waits();
      };
      // O columns [c kOChunk, +kOChunk) of this row, normalised into the output
      auto store = [&](int c, const uint32_t (&o)[C::kOChunk], float inv_l) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + out_row * D + c * C::kOChunk);
#pragma unroll
        for (int e = 0; e < C::kOChunk / 8; ++e) {
          uint4 x;
          x.x = pack_bf16x2(__uint_as_float(o[e * 8 + 0]) * inv_l, __uint_as_float(o[e * 8 + 1]) * inv_l);
          x.y = pack_bf16x2(__uint_as_float(o[e * 8 + 2]) * inv_l, __uint_as_float(o[e * 8 + 3]) * inv_l);
          x.z = pack_bf16x2(__uint_as_float(o[e * 8 + 4]) * inv_l, __uint_as_float(o[e * 8 + 5]) * inv_l);
          x.w = pack_bf16x2(__uint_as_float(o[e * 8 + 6]) * inv_l, __uint_as_float(o[e * 8 + 7]) * inv_l);
          dst[e] = x;
        }
      };
      if (n <= 0) {
        // nothing to see: rows of zeros
        if (valid) {
          uint32_t o[C::kOChunk];
#pragma unroll
          for (int e = 0; e < C::kOChunk; ++e) o[e] = 0u;
          for (int c = narrow ? quarter : 0; c < D / C::kOChunk; c += narrow ? 4 : 1) store(c, o, 0.f);
        }
        continue;
      }
      float m_used = -INFINITY, l = 0.f, alpha;
      bool rescale;
      if (narrow) {
        // ---- each warp: all rows, keys [16 quarter, +16) of a tile
        for (int i = 0; i < n; ++i, ++u) {
          const uint32_t s_col = static_cast<uint32_t>((u & 1) * kBN);
          const int key0 = (kt0 + i) * kBN;
          ok = mbar_wait_warp(s_full + u % R, static_cast<uint32_t>(u / R) & 1u, ab);
          if (!ok) break;
          tc_fence_after();
          if (!(ok = clear_tail(key0))) break;
          uint32_t sr[kQuarterKeys];
          tmem_ld_chunk(lane_base + s_col + quarter * kQuarterKeys, sr);
          tmem_ld_wait();
          reg_fence(sr);
          float s[kQuarterKeys];
#pragma unroll
          for (int c = 0; c < kQuarterKeys; ++c) s[c] = __uint_as_float(sr[c]);
          if (key0 + kBN - 1 > pos0) {
            const int hi_c = pos - key0 - quarter * kQuarterKeys;
#pragma unroll
            for (int c = 0; c < kQuarterKeys; ++c)
              if (c > hi_c) s[c] = -INFINITY;
          }
          float mx = fmax3(s[0], s[1], s[2]);
          float mx1 = fmax3(s[3], s[4], s[5]);
#pragma unroll
          for (int c = 6; c + 4 <= kQuarterKeys; c += 4) {
            mx = fmax3(mx, s[c], s[c + 1]);
            mx1 = fmax3(mx1, s[c + 2], s[c + 3]);
          }
          mx = fmax3(mx, mx1, fmaxf(s[kQuarterKeys - 2], s[kQuarterKeys - 1]));
          if (!(ok = move_max(i, mx, valid, m_used, l, alpha, rescale))) break;
          const float m_sub = (m_used == -INFINITY) ? 0.f : m_used;
          const float2 neg2 = make_float2(-m_sub, -m_sub);
          float2 acc = make_float2(0.f, 0.f);
          uint32_t pq[kQuarterKeys / 2];
#pragma unroll
          for (int e = 0; e < kQuarterKeys / 2; ++e) {
            const float2 x = __ffma2_rn(make_float2(s[2 * e], s[2 * e + 1]), sc2, neg2);
            const float2 pe = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            acc = __fadd2_rn(acc, pe);
            pq[e] = pack_bf16x2(pe.x, pe.y);
          }
          // the other quarters' keys weigh nothing in this quarter's rows
          uint32_t pk[kBN / 2];
#pragma unroll
          for (int e = 0; e < kBN / 2; ++e)
            pk[e] = e / (kQuarterKeys / 2) == quarter ? pq[e % (kQuarterKeys / 2)] : 0u;
          tmem_st32(lane_base + s_col, pk);
          if (rescale) rescale_o(alpha);
          l += acc.x + acc.y;
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(p_full + (u & 1));
        }
        if (!ok) break;
        ok = mbar_wait_warp(o_last, static_cast<uint32_t>(pieces) & 1u, ab);
        if (!ok) break;
        tc_fence_after();
        // x / rows, for the at most 16 rows and 1024 vectors of a narrow piece
        const unsigned rows_magic = ((1u << 16) + rows - 1) / rows;
        auto column_of = [&](int x) { return static_cast<int>(static_cast<unsigned>(x) * rows_magic >> 16); };
        // ---- sum the quarters: (m, l) and as many columns at a time as the
        // exchange memory holds of the rows there are (at the end of the run the
        // idle K and V stages serve, behind the place of the own piece)
        float2* xml = reinterpret_cast<float2*>(smem + C::kXmlOff);
        xml[quarter * kQuarter + lane] = make_float2(m_used, l);
        uint8_t* own = publishes ? slot(place) : ring;       // where the piece is kept while it is not whole
        const bool at_end = w.off <= 0;
        float4* lay = reinterpret_cast<float4*>(at_end ? ring + piece_bytes : smem + C::kXOff);
        const int room = at_end ? C::kMergeBytes - piece_bytes : C::kXBytes;
        int cols = 16;                                       // lay: [quarter][cols / 4][rows]
        while (cols < D && 2 * cols * rows * 16 <= room) cols *= 2;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += cols) {
          if (c0 > 0 && !(ok = meet())) break;               // the columns before are summed
          auto lay_columns = [&](int c, auto width) {
            constexpr int kWidth = decltype(width)::value;
            uint32_t o[kWidth];
            __syncwarp();
            tmem_ld_chunk(lane_base + C::kOCol + c0 + c, o);
            tmem_ld_wait();
            reg_fence(o);
            if (valid) {
#pragma unroll
              for (int e = 0; e < kWidth / 4; ++e)
                lay[(quarter * (cols / 4) + c / 4 + e) * rows + row] =
                    make_float4(__uint_as_float(o[e * 4]), __uint_as_float(o[e * 4 + 1]),
                                __uint_as_float(o[e * 4 + 2]), __uint_as_float(o[e * 4 + 3]));
            }
          };
          if (cols == 16) {
            lay_columns(0, std::integral_constant<int, 16>{});
          } else {
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) lay_columns(c, std::integral_constant<int, 32>{});
          }
          if (!(ok = meet())) break;
          const int items = rows * (cols / 4);
          for (int x = threadIdx.x; x < items; x += kBlockM) {
            const int col = column_of(x), rw = x - col * rows;
            float2 ml[4];
            float4 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              ml[y] = xml[y * kQuarter + rw];
              v[y] = lay[y * items + x];
            }
            const float mm = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
            const float sub = mm == -INFINITY ? 0.f : mm;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float ll = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float f = weight(ml[y].x, sub);
              ll += ml[y].y * f;
              sum.x += v[y].x * f;
              sum.y += v[y].y * f;
              sum.z += v[y].z * f;
              sum.w += v[y].w * f;
            }
            if (whole) {
              write_four(p.out + out_begin<D>(p, unit.row0, unit.head0, rw) + c0 + col * 4, sum,
                         ll > 0.f ? 1.f / ll : 0.f);
            } else {
              reinterpret_cast<float4*>(own)[c0 / 4 * rows + x] = sum;
              if (c0 == 0 && x < rows) ml_of(own)[x] = make_float2(mm, ll);
            }
          }
        }
        if (!ok) break;
        if (sources > 0) {
          // ---- merge: this run's own piece lies at the front, `fit` others
          // at a time come in behind it
          const int fit = C::kMergeBytes / piece_bytes - 1;
          if (!(ok = wait_sources())) break;
          for (int i0 = 0; i0 < sources; i0 += fit) {
            const int count = min(fit, sources - i0);
            const bool further = i0 + count < sources;
            for (int i = quarter; i < count; i += 4) {       // a warp for a piece
              const uint8_t* src = slot(cta - 1 - i0 - i);
              uint8_t* dst = ring + (1 + i) * piece_bytes;
#pragma unroll 8
              for (int x = lane * 16; x < piece_bytes; x += 32 * 16) cp_async16(dst + x, src + x);
            }
            cp_async_wait<0>();
            if (!(ok = meet())) break;
            float2 ml_row = make_float2(0.f, 0.f);
            for (int x = threadIdx.x; x < rows * (D / 4); x += kBlockM) {
              const int col = column_of(x), rw = x - col * rows;
              float4 acc = reinterpret_cast<float4*>(ring)[x];
              const float2 ml = ml_of(ring)[rw];
              float top = ml.x;
#pragma unroll 8
              for (int i = 1; i <= count; ++i) top = fmaxf(top, ml_of(ring + i * piece_bytes)[rw].x);
              const float base = top == -INFINITY ? 0.f : top;
              const float fo = weight(ml.x, base);
              float sum = ml.y * fo;
              acc.x *= fo; acc.y *= fo; acc.z *= fo; acc.w *= fo;
#pragma unroll 8
              for (int i = 1; i <= count; ++i) {
                const float2 mi = ml_of(ring + i * piece_bytes)[rw];
                const float4 v = reinterpret_cast<float4*>(ring + i * piece_bytes)[x];
                const float fi = weight(mi.x, base);
                sum += mi.y * fi;
                acc.x += v.x * fi;
                acc.y += v.y * fi;
                acc.z += v.z * fi;
                acc.w += v.w * fi;
              }
              if (x < rows) ml_row = make_float2(top, sum);
              if (further) {
                reinterpret_cast<float4*>(ring)[x] = acc;
              } else {
                write_four(p.out + out_begin<D>(p, unit.row0, unit.head0, rw) + col * 4, acc, sum > 0.f ? 1.f / sum : 0.f);
              }
            }
            if (further) {
              // (every row's own (m, l) has been read: they move on)
              if (!(ok = meet())) break;
              if (static_cast<int>(threadIdx.x) < rows) ml_of(ring)[threadIdx.x] = ml_row;
              if (!(ok = meet())) break;
            }
          }
          if (!ok) break;
        }
      } else {
        const bool busy = quarter * 32 < rows;               // some row of this warp is a query
        for (int i = 0; i < n; ++i, ++u) {
          const uint32_t s_col = static_cast<uint32_t>((u & 1) * kBN);
          const int key0 = (kt0 + i) * kBN;
          ok = mbar_wait_warp(s_full + u % R, static_cast<uint32_t>(u / R) & 1u, ab);
          if (!ok) break;
          tc_fence_after();
          if (!(ok = clear_tail(key0))) break;
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
            if (key0 + kBN - 1 > pos0) {
              const int hi_c = pos - key0;                   // visible columns [0, hi_c]
#pragma unroll
              for (int c = 0; c < kBN; ++c)
                if (c > hi_c) s[c] = -INFINITY;
            }
            float mx4[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) mx4[x] = s[x];
#pragma unroll
            for (int c = 4; c < kBN; c += 8)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                mx4[x] = fmax3(mx4[x], s[c + x], c + 4 + x < kBN ? s[c + 4 + x] : s[c + x]);
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            if (!(ok = move_max(i, mx, valid, m_used, l, alpha, rescale))) break;
            const float m_sub = (m_used == -INFINITY) ? 0.f : m_used;
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
              pk[e] = pack_bf16x2(pe.x, pe.y);
            }
            tmem_st32(lane_base + s_col, pk);
            const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
            if (rescale) rescale_o(alpha);
            l += a.x + a.y;
            tmem_st_wait();
          }
          tc_fence_before();
          mbar_arrive(p_full + (u & 1));
        }
        if (!ok) break;
        ok = mbar_wait_warp(o_last, static_cast<uint32_t>(pieces) & 1u, ab);
        if (!ok) break;
        tc_fence_after();
        float mm = m_used, ll = l;                           // of this piece and the ones merged into it
        if (sources > 0) {
          // Merge: O stays in tensor memory, the published pieces come into the
          // ring, every thread fetching its own row's vectors, the columns of
          // one load at a time: those of the next piece follow as soon as
          // these are summed.
          if (!(ok = wait_sources())) break;
          if (busy) {
            constexpr int kSteps = D / C::kOChunk, kVec = C::kOChunk / 4;
            const int rw = min(row, rows - 1);
            auto fetch = [&](int i, int c) {
              if (i < sources) {
                const float4* src = reinterpret_cast<const float4*>(slot(cta - 1 - i)) + rw;
                float4* dst = reinterpret_cast<float4*>(ring) + row;
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                  cp_async16(dst + (c * kVec + e) * kBlockM, src + (c * kVec + e) * rows);
              }
              cp_async_commit();
            };
#pragma unroll 1
            for (int c = 0; c < kSteps; ++c) fetch(0, c);
            float2 ml = __ldcg(ml_of(slot(cta - 1)) + rw);
#pragma unroll 1
            for (int i = 0; i < sources; ++i) {
              const float top = fmaxf(mm, ml.x), base = top == -INFINITY ? 0.f : top;
              const float fo = weight(mm, base), fi = weight(ml.x, base);
              mm = top;
              ll = ll * fo + ml.y * fi;
              if (i + 1 < sources) ml = __ldcg(ml_of(slot(cta - 2 - i)) + rw);
#pragma unroll 1
              for (int c = 0; c < kSteps; ++c) {
                uint32_t o[C::kOChunk];
                __syncwarp();
                tmem_ld_chunk(lane_base + C::kOCol + c * C::kOChunk, o);
                cp_async_wait<kSteps - 1>();
                tmem_ld_wait();
                reg_fence(o);
                const float4* src = reinterpret_cast<const float4*>(ring) + row;
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                  const float4 v = src[(c * kVec + e) * kBlockM];
                  o[e * 4] = __float_as_uint(fmaf(v.x, fi, __uint_as_float(o[e * 4]) * fo));
                  o[e * 4 + 1] = __float_as_uint(fmaf(v.y, fi, __uint_as_float(o[e * 4 + 1]) * fo));
                  o[e * 4 + 2] = __float_as_uint(fmaf(v.z, fi, __uint_as_float(o[e * 4 + 2]) * fo));
                  o[e * 4 + 3] = __float_as_uint(fmaf(v.w, fi, __uint_as_float(o[e * 4 + 3]) * fo));
                }
                tmem_st_chunk(lane_base + C::kOCol + c * C::kOChunk, o);
                fetch(i + 1, c);
              }
            }
            tmem_st_wait();
          }
        }
        if (busy) {
          const float inv_l = ll > 0.f ? 1.f / ll : 0.f;
          const int rows_here = min(32, rows - quarter * 32);
          uint8_t* turn = smem + C::kXOff + quarter * C::kTurnSlot;
          // where this lane's 16 bytes of rows lane / 4 + 8 k go
          const int r0 = lane >> 2, piece = lane & 3;
          uint16_t* dst[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rr = quarter * 32 + r0 + 8 * k, tok = token_of(p, rr);
            dst[k] = p.out + (static_cast<long long>(w.q.start + token0 + tok) * p.h + w.hk * p.group + rr -
                              tok * p.group) * D + piece * 8;
          }
#pragma unroll 1
          for (int c = 0; c < D / C::kOChunk; ++c) {
            uint32_t o[C::kOChunk];
            __syncwarp();
            tmem_ld_chunk(lane_base + C::kOCol + c * C::kOChunk, o);
            tmem_ld_wait();
            reg_fence(o);
            if (publishes) {
              if (valid) {
                float4* dst = reinterpret_cast<float4*>(slot(place)) + row;
#pragma unroll
                for (int e = 0; e < C::kOChunk / 4; ++e)
                  dst[(c * (C::kOChunk / 4) + e) * rows] =
                      make_float4(__uint_as_float(o[e * 4]), __uint_as_float(o[e * 4 + 1]),
                                  __uint_as_float(o[e * 4 + 2]), __uint_as_float(o[e * 4 + 3]));
              }
            } else if constexpr (D < 32) {
              if (valid) store(c, o, inv_l);
            } else {
              // Stores straight from the rows' owners would touch 32 lines
              // with 16 bytes each; turned through shared memory, four lanes
              // write 64 bytes of a row.
              uint4* mine = reinterpret_cast<uint4*>(turn + lane * C::kTurnRow);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint4 x;
                x.x = pack_bf16x2(__uint_as_float(o[e * 8 + 0]) * inv_l, __uint_as_float(o[e * 8 + 1]) * inv_l);
                x.y = pack_bf16x2(__uint_as_float(o[e * 8 + 2]) * inv_l, __uint_as_float(o[e * 8 + 3]) * inv_l);
                x.z = pack_bf16x2(__uint_as_float(o[e * 8 + 4]) * inv_l, __uint_as_float(o[e * 8 + 5]) * inv_l);
                x.w = pack_bf16x2(__uint_as_float(o[e * 8 + 6]) * inv_l, __uint_as_float(o[e * 8 + 7]) * inv_l);
                mine[e] = x;
              }
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int x = r0 + 8 * k;                    // row of this warp
                const uint4 v = *reinterpret_cast<const uint4*>(turn + x * C::kTurnRow + piece * 16);
                if (x < rows_here) *reinterpret_cast<uint4*>(dst[k] + c * 32) = v;
              }
            }
          }
          if (publishes && valid) ml_of(slot(place))[row] = make_float2(mm, ll);
        }
      }
      if (publishes) {
        if (sliced && threadIdx.x == 0) p.states[cta] = kOpen;
        if (!(ok = publish())) break;
        if (sliced) {
          // (a run's first piece, unless it is all of the run, is followed by
          // others, and takes no slice)
          const int most = of - (cut.scheme == kPieces ? 0 : 1);
          meet.met = merge_slices<D>(p, unit, ring, most, merge, meet.met, patience, left, ab);
          if (!(ok = meet.met >= 0)) break;
        }
      }
      __syncwarp();
      tc_fence_before();
      mbar_arrive(o_free);
      ++pieces;
    }
    cp_async_wait<0>();                                      // (a wait may have run out above)
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D>
cudaError_t launch_paged_impl(const PagedParams& p, cudaStream_t stream) {
  constexpr int smem = PCfg<D>::kSmemBytes;
  // the kernel's shared-memory limit is set once on each device
  static std::atomic<unsigned long long> prepared{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev > 63 || !(prepared.load(std::memory_order_acquire) & bit)) {
    err = cudaFuncSetAttribute(sdpa_paged_split<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    if (dev <= 63) prepared.fetch_or(bit, std::memory_order_release);
  }
  return launch_kernel(sdpa_paged_split<D>, dim3(static_cast<unsigned>(p.split_ctas)), dim3(kThreads), smem,
                       stream, true, p);
}

// -------------------------------------------------------------------- append
// Rotates the new queries and keys by their positions and stores keys and
// values into their pages.  The pair (a, b) of frequency f at position p
// becomes (a cos(p f) - b sin(p f), b cos(p f) + a sin(p f)).
//
// It moves (h + 2 h_kv) d bf16 a token in and out and is bound by HBM (by the
// launch for a few tokens).  A block takes kTokens tokens: their angles once,
// into shared memory, then every head of theirs, a thread handling two
// 16-byte chunks at a time (an item): the two whose columns pair up.  A block
// needs three dependent reads (sequence, length, page) before it can store, so
// each thread loads its first kAhead items before them.
constexpr int kAppendThreads = 256;

// cos and sin of pos * freq.  The angle in turns is formed from products whose
// rounding errors are kept (fma): the position in two parts of at most 19 bits,
// freq / 2 pi as a sum of three floats, good to 2^-70 of itself.  Whole turns are
// dropped after each sum of two parts of at most half a turn, which rounds off by
// 2^-25 at most; there are six such sums and a last one, so that the fraction is good
// to 7 2^-25 = 2.1e-7 of a turn, 1.3e-6 rad, while the angle is below 2^48.  (Against
// exact arithmetic, 300000 angles of positions up to 2^30 and frequencies up to 1e5
// were off by 4.6e-7 rad at most.)
__device__ __forceinline__ float2 cos_sin(int pos, float freq) {
  // 1 / (2 pi) = 0.15915494309189533576888376..., rounded to fp32, then what that left, twice
  constexpr float kInvTwoPi0 = 0x1.45f306p-3f, kInvTwoPi1 = 0x1.b9391p-28f, kInvTwoPi2 = 0x1.529fc2p-54f;
  const float th = freq * kInvTwoPi0, e0 = fmaf(freq, kInvTwoPi0, -th);
  const float p1 = freq * kInvTwoPi1, e1 = fmaf(freq, kInvTwoPi1, -p1);
  const float tm = e0 + p1, back = tm - e0;
  const float tl = (e0 - (tm - back)) + (p1 - back) + fmaf(freq, kInvTwoPi2, e1);
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
__device__ int find_seq(const PagedAppendParams& p, int t, int lane) {
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

template <int kTokens, int kAhead, int kBlocks>
__global__ void __launch_bounds__(kAppendThreads, kBlocks) sdpa_paged_append_kernel(const PagedAppendParams p) {
  static_assert(kTokens <= kAppendThreads / 32, "a warp finds each token's place");
  extern __shared__ __align__(16) float2 angles[];            // [kTokens][d_rot / 2]
  __shared__ long long row_of[kTokens];                       // page row of the token, head 0 (-1: not stored)
  __shared__ int pos_of[kTokens];                             // position (INT_MIN: no sequence's token)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = static_cast<int>(blockIdx.x) * kTokens;
  const int half = p.d_rot / 2, rotated_pairs = p.d_rot / 16;
  const int pairs_mask = (1 << p.log_pairs) - 1;              // items of a head, d / 16
  const int items = (p.h + 2 * p.h_kv) << p.log_pairs;        // of a token
  const int all = min(kTokens, p.n_tokens - t0) * items;
  struct Item {
    int token, head, c0, c1;                                  // c0, c1: columns of its chunks
    bool rotated;
  };
  auto item_of = [&](int x) {
    Item it;
    it.token = kTokens == 1 ? 0 : (p.items_magic != 0 ? __umulhi(x, p.items_magic) : x / items);
    const int y = x - it.token * items;
    it.head = y >> p.log_pairs;
    const int c = y & pairs_mask;
    it.rotated = c < rotated_pairs && it.head < p.h + p.h_kv;
    // columns 8 c and 8 c + d_rot / 2 of rotated halves, else neighbours
    it.c0 = (it.rotated && !p.interleaved) ? c * 8 : c * 16;
    it.c1 = (it.rotated && !p.interleaved) ? it.c0 + half : it.c0 + 8;
    return it;
  };
  auto source = [&](const Item& it) -> const uint16_t* {
    const long long t = t0 + it.token;
    if (it.head < p.h) return p.q == nullptr ? nullptr : p.q + t * p.q_stride + it.head * p.d;
    const int hk = it.head - p.h;
    return hk < p.h_kv ? p.k + t * p.k_stride + hk * p.d : p.v + t * p.v_stride + (hk - p.h_kv) * p.d;
  };
  uint4 a[kAhead], b[kAhead];
  auto load = [&](int x0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int x = x0 + j * kAppendThreads;
      if (x >= all) continue;
      const Item it = item_of(x);
      const uint16_t* src = source(it);
      if (src == nullptr) continue;
      a[j] = *reinterpret_cast<const uint4*>(src + it.c0);
      b[j] = *reinterpret_cast<const uint4*>(src + it.c1);
    }
  };
  griddep_launch_dependents();
  griddep_wait();
  load(threadIdx.x);
  if (warp < kTokens && t0 + warp < p.n_tokens) {
    const int t = t0 + warp;
    const int s = find_seq(p, t, lane);
    if (lane == 0) {
      long long row = -1;
      int pos = INT_MIN;
      const int end = s >= 0 ? min(p.q_starts[s + 1], p.n_tokens) : 0;
      if (t < end) {
        const int len = min(max(p.kv_lengths[s], 0), p.pages_per_seq << p.page_shift);
        pos = len - end + t;
        if (pos >= 0) {
          const int page = p.page_table[static_cast<long long>(s) * p.pages_per_seq + (pos >> p.page_shift)];
          if (page < 0 || page >= p.n_pages)
            atomicOr(p.status, kStatusBadPage);
          else
            row = (static_cast<long long>(page) * p.h_kv << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        }
      }
      row_of[warp] = row;
      pos_of[warp] = pos;
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < kTokens * half; x += kAppendThreads) {
    const int i = x / half;
    if (t0 + i < p.n_tokens && pos_of[i] != INT_MIN) angles[x] = cos_sin(pos_of[i], p.freqs[x - i * half]);
  }
  __syncthreads();
  for (int x0 = threadIdx.x; x0 < all; x0 += kAhead * kAppendThreads) {
    if (x0 != static_cast<int>(threadIdx.x)) load(x0);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int x = x0 + j * kAppendThreads;
      if (x >= all) break;
      const Item it = item_of(x);
      if (pos_of[it.token] == INT_MIN) continue;
      uint16_t* dst;
      if (it.head < p.h) {
        if (p.q == nullptr) continue;
        dst = p.q_out + (static_cast<long long>(t0 + it.token) * p.h + it.head) * p.d;
      } else {
        const long long row = row_of[it.token];
        if (row < 0) continue;
        const int hk = it.head - p.h;
        const bool is_k = hk < p.h_kv;
        dst = (is_k ? p.k_pages : p.v_pages) +
              (row + (static_cast<long long>(is_k ? hk : hk - p.h_kv) << p.page_shift)) * p.d;
      }
      if (it.rotated) {
        const int c = p.interleaved ? it.c0 / 16 : it.c0 / 8;
        const float4* cs = reinterpret_cast<const float4*>(angles + it.token * half + c * 8);   // pairs 8 c .. 8 c + 7
        uint32_t* ua = reinterpret_cast<uint32_t*>(&a[j]);
        uint32_t* ub = reinterpret_cast<uint32_t*>(&b[j]);
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x0v = unpack_bf16x2(ua[e]), x1v = unpack_bf16x2(ub[e]);
            const float4 r01 = cs[e / 2], r45 = cs[2 + e / 2];
            const float2 r0 = e % 2 ? make_float2(r01.z, r01.w) : make_float2(r01.x, r01.y);
            const float2 r1 = e % 2 ? make_float2(r45.z, r45.w) : make_float2(r45.x, r45.y);
            ua[e] = pack_bf16x2(x0v.x * r0.x - x0v.y * r0.y, x0v.y * r0.x + x0v.x * r0.y);
            ub[e] = pack_bf16x2(x1v.x * r1.x - x1v.y * r1.y, x1v.y * r1.x + x1v.x * r1.y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 xa = unpack_bf16x2(ua[e]), xb = unpack_bf16x2(ub[e]);
            const float4 r = cs[e];                           // (cos, sin) of pairs 2 e and 2 e + 1
            ua[e] = pack_bf16x2(xa.x * r.x - xb.x * r.y, xa.y * r.z - xb.y * r.w);
            ub[e] = pack_bf16x2(xb.x * r.x + xa.x * r.y, xb.y * r.z + xa.y * r.w);
          }
        }
      }
      *reinterpret_cast<uint4*>(dst + it.c0) = a[j];
      *reinterpret_cast<uint4*>(dst + it.c1) = b[j];
    }
  }
}

template <int kTokens, int kAhead, int kBlocks>
cudaError_t launch_append_impl(const PagedAppendParams& p, cudaStream_t stream) {
  const int blocks = (p.n_tokens + kTokens - 1) / kTokens;
  const size_t smem = static_cast<size_t>(kTokens) * (p.d_rot / 2) * sizeof(float2);
  return launch_kernel(sdpa_paged_append_kernel<kTokens, kAhead, kBlocks>, dim3(static_cast<unsigned>(blocks)),
                       dim3(kAppendThreads), smem, stream, true, p);
}

}  // namespace

bool paged_supports(int d) { return d == 16 || d == 32 || d == 64 || d == 128 || d == 256; }

int paged_resident_ctas(int d) { return d <= 128 ? 2 : 1; }

cudaError_t launch_sdpa_paged(const PagedParams& p, int d, cudaStream_t stream) {
  switch (d) {
    case 16: return launch_paged_impl<16>(p, stream);
    case 32: return launch_paged_impl<32>(p, stream);
    case 64: return launch_paged_impl<64>(p, stream);
    case 128: return launch_paged_impl<128>(p, stream);
    case 256: return launch_paged_impl<256>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_sdpa_paged_append(const PagedAppendParams& p, cudaStream_t stream) {
  // While all blocks run at once (four of four tokens on an SM), what counts is
  // a block's chain of reads: items loaded ahead of it take 6.0 us instead of
  // 7.6 for 2200 tokens of 16 + 32 heads of 64.  Beyond, blocks on an SM count:
  // eight with one item ahead take 34.3 us for 16384 tokens of 16 + 8 heads of
  // 128 (5.9 TB/s), four with three 39.7.  Up to four tokens an SM, one block
  // for each.
  const int sms = device_sm_count();
  if (p.n_tokens <= 4 * sms) return launch_append_impl<1, 2, 4>(p, stream);
  if (p.n_tokens <= 16 * sms) return launch_append_impl<4, 3, 4>(p, stream);
  return launch_append_impl<4, 1, 8>(p, stream);
}

}  // namespace sdpa
