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
// sdpa_paged_split<D>     A UNIT is (sequence, key-value head, row tile): the
//   rows of a tile are tile_tokens tokens x the group's heads (at most 128),
//   so one walk over the keys serves every query head of the group.  A
//   unit's walk is its visible keys in tiles of 64; all walks laid end to
//   end are cut into equal runs of tiles, one per CTA, so that one long
//   sequence, many short ones and any mixture load the SMs alike.  A CTA
//   whose run begins or ends inside a unit leaves that piece's (O, m, l) in
//   the workspace.  The cut is worked out on the device from the lengths, so
//   a captured launch follows them.
// sdpa_paged_combine<D>   merges the pieces of each unit that was cut:
//   O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, M = max_s m_s.
//
// The roles of a split CTA are those of the one-tile forward kernel (TMA
// producer, MMA issuer, four softmax warps of one thread per row, S double
// buffered and O in tensor memory), kept running from piece to piece: tile
// and piece counters carry on, and two more barriers hand over Q (q_empty)
// and O (o_free).
#include <climits>
#include <cmath>

#include "kernels.h"
#include "ptx.cuh"

namespace sdpa {
namespace {

constexpr int kBlockM = 128;
constexpr int kBN = kPagedKeyTile;         // keys per tile
constexpr int kThreads = 192;
constexpr int kProducerWarp = 4;
constexpr int kMmaWarp = 5;
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
  q.tiles = (q.n + p.tile_tokens - 1) / p.tile_tokens;
  return q;
}

// Keys that some row of row tile r sees, and the tile's cost in key tiles
// (at least one: a tile that sees nothing still writes its zeros).
__device__ __forceinline__ int tile_keys(const PagedParams& p, const Seq& q, int r) {
  return max(0, q.len - q.n + min((r + 1) * p.tile_tokens, q.n));
}
__device__ __forceinline__ int tile_cost(int keys) { return max(1, (keys + kBN - 1) / kBN); }

// Cost of row tiles 0 .. r-1 (r <= q.tiles) of one key-value head.  All but
// the last tile see A + (i + 1) t keys, A = len - n: z of them cost one, the
// others ceil((A + (i + 1) t) / 64), whose sum over 64 consecutive i grows by
// 64 t from one such block to the next.
__device__ long long cost_before(const PagedParams& p, const Seq& q, int r) {
  const int t = p.tile_tokens;
  const int f = min(r, q.tiles - 1);
  long long sum = 0;
  if (f > 0) {
    const int a = q.len - q.n;
    const int z = kBN - a >= t ? min(f, (kBN - a) / t) : 0;
    sum = z;
    const int cnt = f - z;
    if (cnt > 0) {
      const int base = a + t * (z + 1) + kBN - 1;   // > kBN
      const int blocks = cnt / kBN, rest = cnt % kBN;
      long long head = 0, full = 0;                  // the first `rest` terms; the first 64
      const int walk = blocks > 0 ? kBN : rest;
      for (int i = 0; i < walk; ++i) {
        const int c = (base + t * i) / kBN;
        full += c;
        if (i < rest) head += c;
      }
      const long long m = blocks;
      sum += m * full + static_cast<long long>(kBN) * t * (m * (m - 1) / 2) + head +
             static_cast<long long>(rest) * t * m;
    }
  }
  if (r == q.tiles && r > 0) sum += tile_cost(q.len);
  return sum;
}

// A place in the laid-out work: key tile kt of row tile r of head hk of
// sequence s.
struct Place {
  int s, hk, r, kt;
};

struct ScheduleShared {
  long long warp_sum[8];
  long long rem;
  int s;
  Place at;
};

__device__ __forceinline__ long long run_begin(long long work, int c, int ctas) {
  return work / ctas * c + work % ctas * c / ctas;
}

// The whole block: total work, and the place of work item `work * c / ctas`
// for the number of runs `ctas` that follows from the total.  Returns false
// (everywhere) when there is no such run.
template <int NT>
__device__ bool find_place(const PagedParams& p, ScheduleShared* sh, int c, int max_ctas,
                           long long* work, int* ctas, Place* at) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (p.b + NT - 1) / NT;
  const int s0 = min(tid * per, p.b), s1 = min(s0 + per, p.b);
  long long mine = 0;
  for (int s = s0; s < s1; ++s) {
    const Seq q = load_seq(p, s);
    mine += cost_before(p, q, q.tiles) * p.h_kv;
  }
  long long incl = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, x);
    if (lane >= x) incl += o;
  }
  if (lane == 31) sh->warp_sum[warp] = incl;
  __syncthreads();
  long long total = 0, excl = incl - mine;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) excl += sh->warp_sum[w];
    total += sh->warp_sum[w];
  }
  const long long want = (total + p.min_tiles - 1) / p.min_tiles;
  const int n = static_cast<int>(min(static_cast<long long>(max_ctas), want));
  *work = total;
  *ctas = n;
  if (c >= n) return false;
  const long long x = run_begin(total, c, n);
  if (mine > 0 && excl <= x && x < excl + mine) {
    long long rem = x - excl;
    for (int s = s0; s < s1; ++s) {
      const Seq q = load_seq(p, s);
      const long long w = cost_before(p, q, q.tiles) * p.h_kv;
      if (rem < w) {
        sh->s = s;
        sh->rem = rem;
        break;
      }
      rem -= w;
    }
  }
  __syncthreads();
  if (warp == 0) {
    Place pl;
    pl.s = sh->s;
    const Seq q = load_seq(p, pl.s);
    const long long head = cost_before(p, q, q.tiles);
    long long rem = sh->rem;
    pl.hk = static_cast<int>(rem / head);
    rem -= pl.hk * head;
    // the last row tile that begins at or before rem: 32 probes a round
    int lo = 0, hi = q.tiles;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int probe = lo + lane * step;
      const bool le = probe < hi && cost_before(p, q, probe) <= rem;
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));
      lo += k * step;
      hi = min(hi, lo + step);
    }
    pl.r = lo;
    pl.kt = static_cast<int>(rem - cost_before(p, q, lo));
    if (lane == 0) sh->at = pl;
  }
  __syncthreads();
  *at = sh->at;
  return true;
}

// The pieces of one run, in order; every role walks its own copy.
struct Walk {
  Place at;
  Seq q;
  int keys, cost;
  long long left;

  __device__ void begin(const PagedParams& p, const Place& a, long long run) {
    at = a;
    left = run;
    q = load_seq(p, at.s);
    keys = tile_keys(p, q, at.r);
    cost = tile_cost(keys);
  }
  // key tiles of this piece: [at.kt, end()); those with keys: [at.kt, real_end())
  __device__ int end() const {
    return static_cast<int>(min(static_cast<long long>(cost), at.kt + left));
  }
  __device__ int real_end() const { return min(end(), (keys + kBN - 1) / kBN); }
  __device__ bool next(const PagedParams& p) {
    const int e = end();
    left -= e - at.kt;
    if (left <= 0) return false;
    at.kt = 0;
    if (++at.r == q.tiles) {
      at.r = 0;
      if (++at.hk == p.h_kv) {
        at.hk = 0;
        do {
          if (++at.s >= p.b) return false;
          q = load_seq(p, at.s);
        } while (q.n == 0);
      }
    }
    keys = tile_keys(p, q, at.r);
    cost = tile_cost(keys);
    return true;
  }
};

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
  static constexpr int kKOff = kQBytes;
  static constexpr int kVOff = kKOff + kRing * kKVBytes;
  static constexpr int kBarOff = kVOff + kRing * kKVBytes;
  // q_full, q_empty, k_full[R], v_full[R], s_full[R], o_full[R], p_full[2], o_last, o_free, drain
  static constexpr int kNumBars = 2 + 4 * kRing + 2 + 3;
  static constexpr int kSmemBytes = kBarOff + kNumBars * 8 + 16 + 1024;
  static constexpr uint32_t kOCol = 2 * kBN;
  static constexpr int kOChunk = D < 32 ? D : 32;
  static constexpr uint32_t kTmemCols = kOCol + D <= 256 ? 256u : 512u;
  static constexpr int kMinBlocks = static_cast<int>(512u / kTmemCols);
  static constexpr uint32_t kIdescS = idesc_bf16(kBlockM, kBN, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16(kBlockM, D, false, true);
  static constexpr uint32_t kDescHi = (kSBO >> 4) | (1u << 14) | (kLayout << 29);
  static_assert(kSmemBytes * kMinBlocks <= 232448 - 1024 * kMinBlocks, "CTAs per SM");
  static_assert(kKOff % 1024 == 0 && kVOff % 1024 == 0 && kKVBox % 1024 == 0, "alignment");
  // one lane of the producer warp per TMA box of a tile (pages of 8 rows at least)
  static_assert(kBoxes * (kBN / kPagedMinPage) <= 32, "boxes of a tile");
};

template <int D>
__global__ void __launch_bounds__(kThreads, PCfg<D>::kMinBlocks)
    sdpa_paged_split(const __grid_constant__ PagedParams p) {
  using C = PCfg<D>;
  constexpr int R = C::kRing;
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScheduleShared sched;
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
  uint64_t* drain = o_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const AbortState ab{abort_flag, p.status};
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
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
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  // After the wait: the combine kernel may then read the lengths as soon as
  // it starts, the kernels that wrote them having completed.
  griddep_launch_dependents();

  long long work = 0;
  int ctas = 0;
  Place first;
  const int cta = static_cast<int>(blockIdx.x);
  const bool any = find_place<kThreads>(p, &sched, cta, static_cast<int>(gridDim.x), &work, &ctas, &first);
  const long long run = any ? run_begin(work, cta + 1, ctas) - run_begin(work, cta, ctas) : 0;

  if (run > 0 && warp == kProducerWarp) {
    // ---------------------------------------------------------- producer
    // Lane i < boxes copies column box i % kBoxes of the page part i / kBoxes
    // of a tile; it reads its page of the tile after next ahead of time.
    const int page_rows = 1 << p.page_shift;
    const int box_rows = min(page_rows, kBN);
    const int part = lane / C::kBoxes, col = lane % C::kBoxes;
    const bool copies = part < kBN / box_rows;
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_q);
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
    }
    const uint32_t dst = static_cast<uint32_t>(col * C::kKVBox + part * box_rows * C::kRowBytes);
    Walk w;
    w.begin(p, first, run);
    int u0 = 0, pieces = 0, k_issued = 0, v_issued = 0;
    bool go = true;
    do {
      const int n = w.real_end() - w.at.kt;
      if (n <= 0) continue;
      const int32_t* pages = p.page_table + static_cast<long long>(w.at.s) * p.pages_per_seq;
      const int key_first = w.at.kt * kBN + part * box_rows;
      // page of this lane's part of tile i; -1: no position there holds a key
      auto page_of = [&](int i) -> int {
        const int key = key_first + i * kBN;
        return (copies && i < n && key < w.q.len) ? pages[key >> p.page_shift] : -1;
      };
      // page numbers outside the cache read as zeros and are reported
      auto has = [&](int i) { return copies && key_first + i * kBN < w.q.len; };
      auto load = [&](const CUtensorMap* map, uint64_t* bar, uint8_t* stage, int i, int page) {
        const int key = w.at.kt * kBN + i * kBN;
        const int parts = min(kBN / box_rows, (w.q.len - key + box_rows - 1) / box_rows);
        if (lane == 0)
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(parts * box_rows * C::kRowBytes * C::kBoxes));
        __syncwarp();
        if (has(i)) {
          if (page < 0 || page >= p.n_pages) {
            atomicOr(p.status, kStatusBadPage);
            page = p.n_pages;
          }
          tma_load_4d(map, bar, stage + dst, col * C::kBoxCols,
                      (key_first + i * kBN) & (page_rows - 1), w.at.hk, page);
        }
      };
      int page_v = page_of(0);
      int page_k = page_v;
      // Q, once the scores of the piece before are done with it
      if (pieces > 0 && !(go = mbar_wait_warp(q_empty, static_cast<uint32_t>(pieces - 1) & 1u, ab))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(p.tile_tokens * p.group * C::kRowBytes * C::kBoxes));
        for (int c = 0; c < C::kBoxes; ++c)
          tma_load_3d(&p.tm_q, q_full, smem + c * C::kQBox, c * C::kBoxCols, w.at.hk * p.group,
                      w.q.start + w.at.r * p.tile_tokens);
      }
      ++pieces;
      auto load_k = [&](int i) -> bool {
        const int u = u0 + i, s = u % R;
        if (u >= R && !mbar_wait_warp(s_full + s, static_cast<uint32_t>(u / R - 1) & 1u, ab)) return false;
        load(&p.tm_k, k_full + s, smem + C::kKOff + s * C::kKVBytes, i, page_k);
        k_issued = u + 1;
        return true;
      };
      go = load_k(0);
      for (int i = 0; go && i < n; ++i) {
        // K of the next tile goes ahead of V of this one: its stage is free earlier
        page_k = page_of(i + 1);
        if (i + 1 < n && !(go = load_k(i + 1))) break;
        const int u = u0 + i, s = u % R;
        if (u >= R && !(go = mbar_wait_warp(o_full + s, static_cast<uint32_t>(u / R - 1) & 1u, ab))) break;
        load(&p.tm_v, v_full + s, smem + C::kVOff + s * C::kKVBytes, i, page_v);
        page_v = page_k;
        v_issued = u + 1;
      }
      u0 += n;
    } while (go && w.next(p));
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
                         C::kDescHi, b0 + static_cast<uint32_t>(((k / kS) * C::kKVBox + (k % kS) * 32) >> 4),
                         C::kDescHi, C::kIdescS, k > 0 ? 1u : 0u);
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
      const uint32_t b0 = lo(smem_base + C::kVOff + (u % R) * C::kKVBytes, C::kKVBox);
#pragma unroll
      for (int k = 0; k < kBN / 16; ++k)
        mma_bf16_ts_warp(tmem + C::kOCol, pa + static_cast<uint32_t>(k * 8),
                         b0 + static_cast<uint32_t>((k * 16 * C::kRowBytes) >> 4), C::kDescHi, C::kIdescPV,
                         (accumulate || k > 0) ? 1u : 0u);
    };
    Walk w;
    w.begin(p, first, run);
    int u = 0, pieces = 0;
    bool ok = true;
    do {
      const int n = w.real_end() - w.at.kt;
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
             mbar_wait_warp(v_full + u % R, static_cast<uint32_t>(u / R) & 1u, ab);
        if (!ok) break;
        tc_fence_after();
        issue_pv(u, i > 0);
        mma_commit_warp(o_full + u % R);
        if (i + 1 == n) mma_commit_warp(o_last);
      }
      ++pieces;
    } while (ok && w.next(p));
    mma_commit_warp(drain);
    mbar_wait_drain(drain, 0);
  } else if (run > 0) {
    // ---------------------------------------------------------- softmax
    const int row = (warp & 3) * 32 + lane;                  // row of the tile, tensor-memory lane
    const int token = row / p.group, head = row % p.group;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float scale_log2 = p.scale_log2;
    Walk w;
    w.begin(p, first, run);
    int u = 0, pieces = 0;
    bool ok = true;
    do {
      const int kt0 = w.at.kt, n = w.real_end() - kt0;
      const int token0 = w.at.r * p.tile_tokens;
      const bool valid = token < p.tile_tokens && token0 + token < w.q.n;
      const bool busy = __any_sync(0xffffffffu, valid);      // some row of this warp is a query
      const int pos0 = w.q.len - w.q.n + token0;             // position of the tile's first row
      const int pos = pos0 + token;                          // this row sees keys 0 .. pos
      float m_used = -INFINITY, l = 0.f;
      for (int i = 0; i < n; ++i, ++u) {
        const uint32_t s_col = static_cast<uint32_t>((u & 1) * kBN);
        const int key0 = (kt0 + i) * kBN;
        ok = mbar_wait_warp(s_full + u % R, static_cast<uint32_t>(u / R) & 1u, ab);
        if (!ok) break;
        tc_fence_after();
        if (key0 + kBN > w.q.len) {
          // Rows of V past the length hold whatever the page held (or an
          // older tile): their weights are zero, but zero times an infinity
          // or a NaN is a NaN, so they are cleared.
          ok = mbar_wait_warp(v_full + u % R, static_cast<uint32_t>(u / R) & 1u, ab);
          if (!ok) break;
          uint8_t* v = smem + C::kVOff + (u % R) * C::kKVBytes;
          const int keep = w.q.len - key0;                   // in [1, kBN)
          constexpr int kPerRow = C::kRowBytes / 16;
          for (int x = threadIdx.x; x < (kBN - keep) * kPerRow; x += kBlockM)
#pragma unroll
            for (int c = 0; c < C::kBoxes; ++c)
              *reinterpret_cast<uint4*>(v + c * C::kKVBox + keep * C::kRowBytes + x * 16) =
                  make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        if (busy) {
          float s[kBN];
          {
            uint32_t sr[32];
#pragma unroll
            for (int c = 0; c < kBN / 32; ++c) {
              tmem_ld32(lane_base + s_col + c * 32, sr);
              tmem_ld_wait();
              reg_fence(sr);
#pragma unroll
              for (int e = 0; e < 32; ++e) s[c * 32 + e] = __uint_as_float(sr[e]);
            }
          }
          if (key0 + kBN - 1 > pos0) {
            const int hi_c = pos - key0;                     // visible columns [0, hi_c]
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
          const float m_new = fmaxf(m_used, mx * scale_log2);
          float alpha = 1.f;
          bool rescale_warp = false;
          if (i == 0) {
            m_used = m_new;
          } else {
            // rows that are no query hold leftovers: they never ask for a rescale
            const bool need = valid && m_new > m_used + kRescaleThreshold;
            rescale_warp = __any_sync(0xffffffffu, need);
            if (need) {
              alpha = ex2_approx(m_used - m_new);
              m_used = m_new;
              l *= alpha;
            }
            // the rescale follows O += P(u-1) V(u-1): its barrier's previous
            // phase is complete (S(u) was issued after it) and its next one
            // needs this softmax's next P, so the parity wait is exact
            if (rescale_warp) {
              ok = mbar_wait_warp(o_full + (u - 1) % R, static_cast<uint32_t>((u - 1) / R) & 1u, ab);
              if (!ok) break;
              tc_fence_after();
            }
          }
          const float m_sub = (m_used == -INFINITY) ? 0.f : m_used;
          const float2 sc2 = make_float2(scale_log2, scale_log2);
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
          if (rescale_warp) {
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
        mbar_arrive(p_full + (u & 1));
      }
      if (!ok) break;
      // ---- end of the piece: a whole unit is normalised and stored, a part
      // goes to the workspace as it is
      const bool whole = kt0 == 0 && w.end() == w.cost;
      if (n > 0) {
        ok = mbar_wait_warp(o_last, static_cast<uint32_t>(pieces) & 1u, ab);
        if (!ok) break;
        tc_fence_after();
      }
      if (busy) {
        const float inv_l = (n > 0 && l > 0.f) ? 1.f / l : 0.f;
        const long long out_row =
            static_cast<long long>(w.q.start + token0 + token) * p.h + w.at.hk * p.group + head;
        const long long slot = static_cast<long long>(cta) * 2 + (kt0 > 0 ? 0 : 1);
        const long long part_row = slot * p.slot_rows + row;
#pragma unroll
        for (int c = 0; c < D / C::kOChunk; ++c) {
          uint32_t o[C::kOChunk];
          __syncwarp();
          if (n > 0) {
            tmem_ld_chunk(lane_base + C::kOCol + c * C::kOChunk, o);
            tmem_ld_wait();
            reg_fence(o);
          } else {
#pragma unroll
            for (int e = 0; e < C::kOChunk; ++e) o[e] = 0u;
          }
          if (valid && whole) {
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
          } else if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(p.part_o + part_row * D + c * C::kOChunk);
#pragma unroll
            for (int e = 0; e < C::kOChunk / 4; ++e)
              dst[e] = make_uint4(o[e * 4], o[e * 4 + 1], o[e * 4 + 2], o[e * 4 + 3]);
          }
        }
        if (!whole && valid)
          *reinterpret_cast<float2*>(p.part_ml + part_row * 2) = make_float2(m_used, l);
      }
      if (n > 0) {
        __syncwarp();
        tc_fence_before();
        mbar_arrive(o_free);
        ++pieces;
      }
    } while (w.next(p));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------- combine
// Block c - 1 looks after run boundary c: if it is the first one inside its
// unit, the block merges the unit's pieces.  The unit's first piece is the
// last of run c - 1 (slot 1), the others begin runs c, c + 1, ... (slot 0).
constexpr int kCombineThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCombineThreads) sdpa_paged_combine(const __grid_constant__ PagedParams p) {
  __shared__ ScheduleShared sched;
  const int c = static_cast<int>(blockIdx.x) + 1;
  long long work = 0;
  int ctas = 0;
  Place at;
  // the lengths were complete before the split kernel passed its own wait
  const bool any = find_place<kCombineThreads>(p, &sched, c, p.split_ctas, &work, &ctas, &at);
  griddep_launch_dependents();
  griddep_wait();
  if (!any || at.kt == 0) return;
  const long long begin = run_begin(work, c, ctas) - at.kt;
  if (run_begin(work, c - 1, ctas) > begin) return;
  const Seq q = load_seq(p, at.s);
  const long long end = begin + tile_cost(tile_keys(p, q, at.r));
  int last = c;
  while (last + 1 < ctas && run_begin(work, last + 1, ctas) < end) ++last;
  const int token0 = at.r * p.tile_tokens;
  const int rows = min(p.tile_tokens, q.n - token0) * p.group;
  constexpr int kVec = D / 4;
  for (int x = threadIdx.x + blockIdx.y * kCombineThreads; x < rows * kVec;
       x += kCombineThreads * gridDim.y) {
    const int row = x / kVec, col = x % kVec * 4;
    auto part_row = [&](int run) {   // run c-1 .. last
      return (static_cast<long long>(run) * 2 + (run < c ? 1 : 0)) * p.slot_rows + row;
    };
    float mm = -INFINITY;
    for (int r = c - 1; r <= last; ++r) mm = fmaxf(mm, p.part_ml[part_row(r) * 2]);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = c - 1; r <= last; ++r) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + part_row(r) * 2);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + part_row(r) * D + col);
      const float sc = (ml.x == -INFINITY) ? 0.f : ex2_approx(ml.x - mm);
      l += ml.y * sc;
      o.x += v.x * sc;
      o.y += v.y * sc;
      o.z += v.z * sc;
      o.w += v.w * sc;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const long long out_row =
        static_cast<long long>(q.start + token0 + row / p.group) * p.h + at.hk * p.group + row % p.group;
    *reinterpret_cast<uint2*>(p.out + out_row * D + col) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

template <int D>
cudaError_t launch_paged_impl(const PagedParams& p, cudaStream_t stream) {
  constexpr int smem = PCfg<D>::kSmemBytes;
  cudaError_t err =
      cudaFuncSetAttribute(sdpa_paged_split<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  err = launch_kernel(sdpa_paged_split<D>, dim3(static_cast<unsigned>(p.split_ctas)), dim3(kThreads), smem,
                      stream, true, p);
  if (err != cudaSuccess || p.split_ctas == 1) return err;
  const int y = (p.slot_rows * (D / 4) + 4 * kCombineThreads - 1) / (4 * kCombineThreads);
  return launch_kernel(sdpa_paged_combine<D>,
                       dim3(static_cast<unsigned>(p.split_ctas - 1), static_cast<unsigned>(y)),
                       dim3(kCombineThreads), 0, stream, true, p);
}

// -------------------------------------------------------------------- append
// Rotates the new queries and keys by their positions and stores keys and
// values into their pages.  The pair (a, b) of frequency f at position p
// becomes (a cos(p f) - b sin(p f), b cos(p f) + a sin(p f)).
//
// It moves (h + 2 h_kv) d bf16 a token in and out and is bound by HBM (by the
// launch for a few tokens).  A block takes kTokens tokens: their angles once,
// into shared memory, then every head of theirs, a thread handling two
// 16-byte chunks at a time: the two whose columns pair up.
constexpr int kAppendThreads = 256;

// cos and sin of pos * freq.  The angle in turns is formed from products
// whose rounding errors are kept (fma), so that its fraction is good to about
// 2^-22 of a turn wherever the position lies: the position in two parts of
// at most 19 bits, freq / 2 pi as a sum of two floats.
__device__ __forceinline__ float2 cos_sin(int pos, float freq) {
  constexpr float kInvTwoPiHi = 0.15915494f;                 // 1 / (2 pi), and what its rounding left
  constexpr float kInvTwoPiLo = static_cast<float>(0.15915494309189533577 - static_cast<double>(0.15915494f));
  const float th = freq * kInvTwoPiHi;
  const float tl = fmaf(freq, kInvTwoPiHi, -th) + freq * kInvTwoPiLo;
  float t = 0.f;
  auto frac = [](float x) { return x - rintf(x); };
  auto add = [&](float x) {
    const float a = x * th;
    t += frac(a) + frac(fmaf(x, th, -a)) + frac(x * tl);
  };
  add(static_cast<float>(pos >> 12) * 4096.f);
  add(static_cast<float>(pos & 4095));
  t = frac(t);
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

template <int kTokens>
__global__ void __launch_bounds__(kAppendThreads) sdpa_paged_append_kernel(const PagedAppendParams p) {
  extern __shared__ float2 angles[];                          // [kTokens][d_rot / 2]
  __shared__ long long row_of[kTokens];                       // page row of the token, head 0 (-1: not stored)
  __shared__ int pos_of[kTokens];                             // position (INT_MIN: no sequence's token)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = static_cast<int>(blockIdx.x) * kTokens;
  griddep_launch_dependents();
  griddep_wait();
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
  const int half = p.d_rot / 2;
  for (int x = threadIdx.x; x < kTokens * half; x += kAppendThreads) {
    const int i = x / half;
    if (t0 + i < p.n_tokens && pos_of[i] != INT_MIN) angles[x] = cos_sin(pos_of[i], p.freqs[x - i * half]);
  }
  __syncthreads();
  const int pairs = p.d / 16;                                 // two 16-byte chunks each
  const int heads = p.h + 2 * p.h_kv;
  const int items = heads * pairs;
  for (int x = threadIdx.x; x < kTokens * items; x += kAppendThreads) {
    const int i = x / items, y = x - i * items;
    const int head = y / pairs, c = y - head * pairs;
    const int t = t0 + i;
    if (t >= p.n_tokens || pos_of[i] == INT_MIN) continue;
    const bool rotated = c < p.d_rot / 16 && head < p.h + p.h_kv;
    // the two chunks: columns 8 c and 8 c + d_rot / 2 of rotated halves, else neighbours
    const int c0 = (rotated && !p.interleaved) ? c * 8 : c * 16;
    const int c1 = (rotated && !p.interleaved) ? c0 + half : c0 + 8;
    const uint16_t* src;
    uint16_t* dst;
    if (head < p.h) {
      if (p.q == nullptr) continue;
      src = p.q + t * p.q_stride + head * p.d;
      dst = p.q_out + (static_cast<long long>(t) * p.h + head) * p.d;
    } else {
      if (row_of[i] < 0) continue;
      const bool is_k = head < p.h + p.h_kv;
      const int hk = head - p.h - (is_k ? 0 : p.h_kv);
      src = is_k ? p.k + t * p.k_stride + hk * p.d : p.v + t * p.v_stride + hk * p.d;
      dst = (is_k ? p.k_pages : p.v_pages) + (row_of[i] + (static_cast<long long>(hk) << p.page_shift)) * p.d;
    }
    uint4 a = *reinterpret_cast<const uint4*>(src + c0);
    uint4 b = *reinterpret_cast<const uint4*>(src + c1);
    if (rotated) {
      const float2* cs = angles + i * half + c * 8;           // pairs 8 c .. 8 c + 7
      uint32_t* ua = reinterpret_cast<uint32_t*>(&a);
      uint32_t* ub = reinterpret_cast<uint32_t*>(&b);
      if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x0 = unpack_bf16x2(ua[e]), x1 = unpack_bf16x2(ub[e]);
          const float2 r0 = cs[e], r1 = cs[4 + e];
          ua[e] = pack_bf16x2(x0.x * r0.x - x0.y * r0.y, x0.y * r0.x + x0.x * r0.y);
          ub[e] = pack_bf16x2(x1.x * r1.x - x1.y * r1.y, x1.y * r1.x + x1.x * r1.y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 xa = unpack_bf16x2(ua[e]), xb = unpack_bf16x2(ub[e]);
          const float2 r0 = cs[2 * e], r1 = cs[2 * e + 1];
          ua[e] = pack_bf16x2(xa.x * r0.x - xb.x * r0.y, xa.y * r1.x - xb.y * r1.y);
          ub[e] = pack_bf16x2(xb.x * r0.x + xa.x * r0.y, xb.y * r1.x + xa.y * r1.y);
        }
      }
    }
    *reinterpret_cast<uint4*>(dst + c0) = a;
    *reinterpret_cast<uint4*>(dst + c1) = b;
  }
}

template <int kTokens>
cudaError_t launch_append_impl(const PagedAppendParams& p, cudaStream_t stream) {
  const int blocks = (p.n_tokens + kTokens - 1) / kTokens;
  const size_t smem = static_cast<size_t>(kTokens) * (p.d_rot / 2) * sizeof(float2);
  return launch_kernel(sdpa_paged_append_kernel<kTokens>, dim3(static_cast<unsigned>(blocks)),
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
  // one token a block while that leaves SMs idle anyway, four beyond
  if (p.n_tokens <= 4 * device_sm_count()) return launch_append_impl<1>(p, stream);
  return launch_append_impl<4>(p, stream);
}

}  // namespace sdpa
