// Attention of a drafted tree over the paged cache, bf16, on the 5th-generation
// tensor cores (tcgen05, accumulators in tensor memory).
//
// The n * G query rows of a (sequence, kv head) unit -- row r = (node r / G,
// head r % G) -- are the 128 rows of one UMMA tile (m_tiles tiles of whole
// nodes where there are more), whatever the tree looks like: the tree is in the
// masks of the last keys only.  One 3-D TMA box (64 columns, G heads, the
// tile's nodes) lands them in that order; rows past them, of shared memory that
// holds something else, give results that nobody reads.  The unit's keys and
// values stream in 64-token tiles: S = Q K^T into TMEM, the softmax by one
// thread per row, P back into the columns S came from, O += P V in TMEM.
//
// One CTA per SM, two groups of softmax warps.
//   Not PAIR (one row tile): the groups take the tiles in turn.  They share O and
//     the running maximum, which is handed from tile to tile through shared
//     memory as soon as a tile's maximum is known, so that a group's exponentials
//     run beside the other's; each group sums its own weights.
//   PAIR (two row tiles, head_dim 64 and 128): each group has a row tile and an O
//     of its own, and both use every tile, so K and V come to the SM once for 256
//     rows.  (Two CTAs with a row tile each read them twice, every byte from DRAM:
//     8 trees of 64 over 16K-128K keys 655 us where pairs took 636, before the
//     steps below.)
//
// Split.  The units, in order, are one line of work: of each, a fixed cost (its Q,
// masks and rows, counted in tiles) and its tiles.  The line is cut into one range
// for each CTA (of a row tile or pair).  A range is a sequence of pieces of units;
// loads run on into the next piece while the softmax is still at the last one.  A
// unit that lies in one range is written as rows of `out`; the pieces of one that
// is cut are written as partials, at most two per range (the piece that comes
// from the range before, the one that goes on in the next), and joined by
// tree_combine_kernel.  (The line's last 3/16 in shorter ranges, claimed by CTAs that
// are done: 554 for 510 us on 8 trees of 64 over 16K-128K keys, 125 for 114 on 256 of
// 24: a claimed range costs its CTA more, some 5 us, than SMs differ.)
//
// Warps 0-7: softmax, one row per thread; they also write the rows.  Warp 11: MMA
// issue, and the load of a piece's Q as soon as the last S of the piece before
// is done.  Warp 10: the schedule (pieces go to the other warps through a ring in
// shared memory) and the TMA loads of K; warp 9: those of V (boxes of 64 columns and
// as many rows as lie together, a block's up to 64, all issued by one lane).  Warp
// 8: the mending of V in masked tiles, between its load and its product (by the
// softmax warps, which then waited for V three tiles early, a masked tile took
// twice as long).
// Every wait is bounded; a wait that gives up raises the abort flag, which ends all
// roles.
//
// Masks.  A tile is masked where it reaches before a row's window, into the
// tree or past the sequence's end, or where a block id is bad; there each
// thread applies a 64-bit word of its own.  In such a tile a weight of zero
// would still carry a NaN or an infinity of V into rows that do not attend it,
// so V rows that no row attends are zeroed in shared memory, and elements that
// are not finite are taken out and given back at the end, to the rows that
// attend them (a sum with an infinity or a NaN does not depend on its weight).
#pragma once

#include "decode_common.cuh"
#include "decode_dynamic.cuh"
#include "decode_tree_common.cuh"
#include "ptx.cuh"
#include "umma.cuh"

namespace pa {

constexpr int kTreeRows = 128;  // query rows per row tile (UMMA M)
constexpr int kTreeTile = 64;   // keys per tile
constexpr int kTreeWarps = 12;
constexpr int kTreeThreads = kTreeWarps * 32;
// The warps behind the eight of the softmax.  Warps w and w + 4 share a scheduler, and
// row tiles of up to 64 rows leave the last two schedulers without softmax: there
// the two warps that pace the others (B200: 128 trees of 16 nodes 242 us with
// these roles the other way round, 227 so; 7 of 39 nodes 30.5 and 29.3).
constexpr int kTreeMendWarp = 8, kTreeVWarp = 9, kTreeKWarp = 10, kTreeMmaWarp = 11;
constexpr int kTreeCombineRows = 8;  // rows of the partials that lie side by side
constexpr int kTreePieces = 4;      // ring of pieces between the roles
constexpr int kTreeMarks = 2 * kTreePieces;  // pieces whose marks of V are kept: those between the mender and the last epilogue

// QR: rows of Q that shared memory holds (64 or 128).
template <int D, int QR, bool PAIR>
struct TreeCfg {
  static constexpr int kPanels = D / 64;  // 64-element (128-byte) column panels
  static constexpr int kRowTiles = PAIR ? 2 : 1;
  static constexpr int kQPanelBytes = QR * 128;
  static constexpr int kQBytes = kPanels * kQPanelBytes;  // one row tile
  static constexpr int kKVPanelBytes = kTreeTile * 128;
  static constexpr int kKBytes = kPanels * kKVPanelBytes;
  static constexpr int kMaxSmem = 232448;
  static constexpr int kSharedBytes = D == 256 && QR == 64 ? 3 * 1024 : 4096;
  static constexpr int kFit = (kMaxSmem - kSharedBytes - kRowTiles * kQBytes) / kKBytes;
  static constexpr int kKStages = (kFit + 1) / 2 < 10 ? (kFit + 1) / 2 : 10;
  static constexpr int kVStages = kFit / 2 < 10 ? kFit / 2 : 10;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kRowTiles * kQBytes;
  static constexpr int kVOff = kKOff + kKStages * kKBytes;
  static constexpr int kBarOff = kVOff + kVStages * kKBytes;
  static constexpr int kSmemBytes = kBarOff + kSharedBytes;
  static constexpr int kRing = kKStages <= 4 ? 8 : 16;  // tiles whose rows are remembered: those loaded and not done
  // Tiles that S runs ahead of P V (three with two stages of V: 61.4 for 58.7 us on
  // 121 trees of 44 nodes, head_dim 256).
  static constexpr int kLag = PAIR || kVStages < 3 ? 2 : 3;
  // What a unit costs besides its tiles, in tiles: its Q, masks, last tile's latency and
  // rows.  None counted, 64 trees of 8 nodes at head_dim 64 take 34 us for 26; 2 and 1
  // instead of 4 and 3, 128 of 16 at 128 233 for 218, 256 of 24 at 256 114 for 106.
  static constexpr int kUnitCost = D == 64 ? 4 : PAIR ? 2 : D == 128 ? 4 : 3;
  static constexpr int kOCol = 0;                       // O (PAIR: a second one D columns on)
  static constexpr int kSCol = 256;                     // four S buffers, two per group
  static_assert(!PAIR || D <= 128, "tensor memory");
  static_assert(kKStages + kLag + 1 < kRing && kVStages + kLag + 1 < kRing, "ring");
};

// A piece: tiles [t0, t1) of the `tiles` tiles of unit (b, g).  b < 0: no more.
struct TreePiece {
  int b, g, t0, t1, tiles;
  int L, n, ulo;  // the sequence's lengths, first attended position
};

// What the CTA's threads share besides the tiles (behind them, at kBarOff).
template <int D, int QR, bool PAIR>
struct TreeShared {
  using C = TreeCfg<D, QR, PAIR>;
  uint64_t kfull[C::kKStages], kempty[C::kKStages], vfull[C::kVStages], vready[C::kVStages], vempty[C::kVStages];
  uint64_t sfull[2][2], pready[2][2], odone[2][2];  // [group][buffer]
  uint64_t mready[4][2];                            // [warp of the group][tile parity]
  uint64_t pfull[kTreePieces], pempty[kTreePieces];
  uint64_t rfull[C::kRing];                         // rows[] of a tile are written
  uint64_t qfull, epi, ofree, drain;
  uint64_t bad[kTreeMarks][4];  // by piece: rows of V with elements that are not finite, in each masked tile
  TreePiece pieces[kTreePieces];
  alignas(16) int rows[C::kRing][4];  // by tile: cache rows of its boxes (-1: not loaded; -2: no more tiles)
  uint8_t skip[C::kRing];  // by tile: 16-row slices whose block id is bad
  float m[PAIR ? 1 : 2][PAIR ? 1 : QR];  // running maximum, by tile parity
  float l[PAIR ? 1 : 2][PAIR ? 1 : QR];  // the groups' sums at a piece's end
  long long before[kTreeWarps + 1];      // the line before each warp's part of the batch
  long long rel0;                        // where the CTA's range starts: a sequence, and how far in
  int b0;
  uint32_t tmem;
  int abort;
};

// The line of work, in ranges of `per`.
struct TreeLine {
  long long total, per;

  __device__ __forceinline__ TreeLine(long long all, int n) : total(all), per(max((all + n - 1) / n, 1ll)) {}
  __device__ __forceinline__ long long start(int r) const { return min(r * per, total); }
  __device__ __forceinline__ int range_of(long long x) const { return (int)(x / per); }
};

// Tiles of a unit of this sequence.
__device__ __forceinline__ int tree_unit_tiles(const TreeParams& p, const TreeSeq& s) {
  return s.n > 0 ? (s.L - (tree_start(s, p.window) & ~(kTreeTile - 1)) + kTreeTile - 1) / kTreeTile : 0;
}

// Sequences a lane takes in a scan of the batch by all warps.
__device__ __forceinline__ int tree_scan_step(const TreeParams& p) {
  return (p.batch + kTreeThreads - 1) / kTreeThreads;
}

// What this lane's sequences in `warp`'s part of the batch take of the line, and what is before them in that part.
template <int COST>
__device__ __forceinline__ long long tree_lane_work(const TreeParams& p, int warp, int lane, bool report,
                                                    long long& before, long long& all) {
  const int step = tree_scan_step(p), b0 = (warp * 32 + lane) * step;
  long long v = 0;
  for (int b = b0; b < min(b0 + step, p.batch); ++b) {
    const int tiles = tree_unit_tiles(p, tree_seq(p, b, report));
    if (tiles > 0) v += (long long)p.hkv * (tiles + COST);
  }
  long long incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  all = __shfl_sync(0xffffffffu, incl, 31);
  before = incl - v;
  return v;
}

// Walks the pieces of a range (one warp, the same in all lanes).
template <int COST>
struct TreeWalk {
  long long w, w1;
  int b, off, tiles, ulo;
  TreeSeq s;
  int next_len, next_nodes;  // of sequence b + 1, loaded ahead

  __device__ __forceinline__ int seq_work(const TreeParams& p) const { return tiles > 0 ? p.hkv * (tiles + COST) : 0; }

  // Start at `from` on the line, to before `to`; sequences from b0 on, `rel` after their start, are there.
  __device__ __forceinline__ void start(const TreeParams& p, long long from, long long to, int b0, long long rel) {
    w = from;
    w1 = to;
    b = b0;
    load(p);
    while (rel >= seq_work(p) && b + 1 < p.batch) {
      rel -= seq_work(p);
      ++b;
      load_next(p);
    }
    off = (int)rel;
  }
  __device__ __forceinline__ void fit(const TreeParams& p, int len, int nodes) {
    s = tree_fit(p, len, nodes, false);
    const int after = min(b + 1, p.batch - 1);
    next_len = p.context_lens[after];
    next_nodes = p.tree_lens ? p.tree_lens[after] : p.tree_len;
    ulo = tree_start(s, p.window);
    tiles = tree_unit_tiles(p, s);
  }
  __device__ __forceinline__ void load(const TreeParams& p) {
    fit(p, p.context_lens[b], p.tree_lens ? p.tree_lens[b] : p.tree_len);
  }
  __device__ __forceinline__ void load_next(const TreeParams& p) { fit(p, next_len, next_nodes); }
  // The next piece that has rows from node `first_node` on; `at`: where its unit's tile 0 is on the line.
  __device__ __forceinline__ bool next(const TreeParams& p, int first_node, TreePiece& o, long long& at) {
    while (w < w1) {
      while (off >= seq_work(p)) {  // w < w1 <= total: a sequence with work left exists
        if (b + 1 >= p.batch) return false;
        ++b;
        off = 0;
        load_next(p);
      }
      const int unit = tiles + COST;
      o.g = off / unit;
      const int q = off - o.g * unit, n = (int)min((long long)(unit - q), w1 - w);
      o.t0 = max(q - COST, 0);
      o.t1 = q + n - COST;
      at = w - q + COST;
      w += n;
      off += n;
      if (o.t1 <= 0 || first_node >= s.n) continue;  // only of the unit's cost; no rows in these row tiles
      o.b = b;
      o.tiles = tiles;
      o.L = s.L;
      o.n = s.n;
      o.ulo = ulo;
      return true;
    }
    return false;
  }
};

// Partials: of range c and row tile t, slot 2 (c m_tiles + t) for the piece that
// comes from the range before, the next slot for the one that goes on in the
// next; element (row r, column d) of a slot at [d / 4][r][d % 4], so that a
// warp's rows are neighbours, and (m, l) of a row behind.
__device__ __forceinline__ int tree_row_stride(const TreeParams& p) {
  return (p.q_nodes * p.group + kTreeCombineRows - 1) & ~(kTreeCombineRows - 1);
}

// One lane: a tile's boxes, of `box_rows` cache rows from row0, row1, ... on (-1: none), into its panels at dst.
template <int PANELS>
__device__ __forceinline__ void tree_load_boxes(uint32_t dst, const CUtensorMap* map, uint32_t full, int row0, int row1,
                                                int row2, int row3, int box_rows) {
  const int rows[4] = {row0, row1, row2, row3};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (rows[k] < 0) continue;
#pragma unroll
    for (int pn = 0; pn < PANELS; ++pn)
      tma_load_2d(dst + pn * kTreeTile * 128 + k * box_rows * 128, map, full, pn * 64, rows[k]);
  }
}

template <int D, int QR, bool PAIR>
__global__ void __launch_bounds__(kTreeThreads, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using C = TreeCfg<D, QR, PAIR>;
  using Shared = TreeShared<D, QR, PAIR>;
  static_assert(sizeof(Shared) <= C::kSharedBytes, "shared area");
  constexpr uint32_t FULL = 0xffffffffu;
  constexpr int NK = C::kKStages, NV = C::kVStages, TILE = kTreeTile, LAG = C::kLag;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int G = p.group;
  const int pairs = (p.m_tiles + C::kRowTiles - 1) / C::kRowTiles;  // CTAs that share a range
  const int pair = blockIdx.x % pairs, grp = blockIdx.x / pairs, mt0 = pair * C::kRowTiles;

  pdl_launch_dependents();  // the combine may launch; it waits for this grid to finish
  if (smem_addr(smem) & 1023) {  // the swizzled tiles need 1024-byte alignment
    if (tid == 0) raise_error(PA_DEVERR_LAYOUT);
    return;
  }
  auto bar = [&](const uint64_t& b) { return smem_addr(&b); };
  if (tid == 0) {
    for (int s = 0; s < NK; ++s) mbar_init(bar(sh.kfull[s]), 1), mbar_init(bar(sh.kempty[s]), 1);
    for (int s = 0; s < NV; ++s) mbar_init(bar(sh.vfull[s]), 1), mbar_init(bar(sh.vready[s]), 1), mbar_init(bar(sh.vempty[s]), 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(sh.sfull[s >> 1][s & 1]), 1);
      mbar_init(bar(sh.pready[s >> 1][s & 1]), 4);
      mbar_init(bar(sh.odone[s >> 1][s & 1]), 1);
      mbar_init(bar(sh.mready[s][0]), 1);
      mbar_init(bar(sh.mready[s][1]), 1);
    }
    for (int s = 0; s < kTreePieces; ++s) {
      mbar_init(bar(sh.pfull[s]), 1);
      mbar_init(bar(sh.pempty[s]), 10);  // the MMA warp, the mending warp and the softmax warps
    }
    for (int s = 0; s < C::kRing; ++s) mbar_init(bar(sh.rfull[s]), 1);
    mbar_init(bar(sh.qfull), 1);
    mbar_init(bar(sh.epi), 8);
    mbar_init(bar(sh.ofree), 8);
    mbar_init(bar(sh.drain), 1);
    sh.abort = 0;
    mbar_init_fence();
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (warp == 0) umma::alloc(smem_addr(&sh.tmem), 512);
  pdl_wait();  // a programmatic dependent: nothing of global memory was touched before
  long long before, all;
  const long long mine = tree_lane_work<C::kUnitCost>(p, warp, lane, blockIdx.x == 0, before, all);
  if (lane == 0) sh.before[warp + 1] = all;
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  if (tid == 0) {
    sh.before[0] = 0;
    for (int i = 1; i <= kTreeWarps; ++i) sh.before[i] += sh.before[i - 1];
  }
  __syncthreads();
  const TreeLine line(sh.before[kTreeWarps], gridDim.x / pairs);
  before += sh.before[warp];
  const long long from = line.start(grp);
  if (mine > 0 && from >= before && from < before + mine) {
    sh.b0 = tid * tree_scan_step(p);
    sh.rel0 = from - before;
  }
  __syncthreads();
  const uint32_t tmem = sh.tmem;
  const uint32_t s_base = smem_addr(smem);
  const uint32_t q_s = s_base + C::kQOff, k_s = s_base + C::kKOff, v_s = s_base + C::kVOff;
  volatile int* abort_flag = &sh.abort;

  auto wait_use = [&](const uint64_t& b, int use) {  // completion number `use` of a barrier (completions alternate parity)
    return __all_sync(FULL, mbar_wait_bounded(bar(b), use & 1, kWaitLimitNs));
  };
  auto give_up = [&]() {
    if (lane == 0) raise_error(PA_DEVERR_TIMEOUT);
    *abort_flag = 1;
  };
  // Tile number x of the CTA belongs to group x & 1 (not PAIR), as its tile x >> 1.
  auto group_of = [&](int x) { return PAIR ? 0 : x & 1; };
  auto count_of = [&](int x) { return PAIR ? x : x >> 1; };

  if (warp == kTreeKWarp) {
    // ================= schedule, TMA loads of K =================
    // Block ids of a piece's boxes come in windows of 32, lane l holding box
    // wb + l (pages) and wb + 32 + l (pages2); the next piece, and the block ids
    // of its first window, are looked up a piece ahead, so that no load waits
    // for a length or a block table.
    TreeWalk<C::kUnitCost> walk;
    TreePiece cur, nxt;
    int u = 0, i = 0, wb = 0, pages = -1, pages2 = -1, first = -1;
    bool more = false, ok = true;
    int4 rec = make_int4(0, 0, 0, 0);  // the unit that starts in this range and goes on: pieces, b, g, nodes
    cur.t1 = 0;
    auto page_of = [&](const TreePiece& c, int q) {
      const int kt0 = c.ulo & ~(TILE - 1), t = kt0 + c.t0 * TILE + (q << p.log2_box);
      return t < min(c.L, kt0 + c.t1 * TILE) ? p.block_tables[(int64_t)c.b * p.max_blocks + (t >> p.log2_bs)] : -1;
    };
    auto find = [&]() {  // the next piece
      long long at = 0;
      const bool found = walk.next(p, mt0 * p.q_nodes, nxt, at);
      if (found && nxt.t0 == 0 && nxt.t1 < nxt.tiles)
        rec = make_int4(line.range_of(at + nxt.tiles - 1) - grp + 1, nxt.b, nxt.g, nxt.n);
      return found;
    };
    const int boxes = TILE >> p.log2_box, box_rows = 1 << p.log2_box;  // of a tile: 4, 2 or 1
    int issued = 0;
    walk.w = walk.w1 = 0;
    if (from < line.start(grp + 1)) walk.start(p, from, line.start(grp + 1), sh.b0, sh.rel0);
    while (!*abort_flag) {
      if (i >= cur.t1) {  // the next piece goes into the ring, and the one after it is looked up (at first: both)
        bool stop = false;
#pragma unroll 1
        for (int z = issued > 0 ? 1 : 0; z < 2; ++z) {
          if (z == 1) {
            ok = u < kTreePieces || wait_use(sh.pempty[u % kTreePieces], u / kTreePieces - 1);
            stop = !ok || !more;
            cur = nxt;
            if (!more) cur.b = -1;
            if (ok && lane == 0) {
              sh.pieces[u % kTreePieces] = cur;
              mbar_arrive(bar(sh.pfull[u % kTreePieces]));
            }
            __syncwarp();
            ++u;
            if (stop) break;
            i = cur.t0;
            wb = 0;
            pages = first;
            pages2 = page_of(cur, 32 + lane);
          }
          more = find();
          first = more ? page_of(nxt, lane) : -1;
        }
        if (stop) break;
      }
      // The cursor's tile, as tile number `issued`.
      const int n = issued, stage = n % NK, at = n % C::kRing;
      ok = n < NK || wait_use(sh.kempty[stage], n / NK - 1);
      if (!ok) break;
      const int rel = boxes * (i - cur.t0);
      if (rel >= wb + 32) {
        wb += 32;
        pages = pages2;
        pages2 = page_of(cur, wb + 32 + lane);
      }
      const int t = (cur.ulo & ~(TILE - 1)) + i * TILE + (lane << p.log2_box);  // lane: box
      const int phys = __shfl_sync(FULL, pages, (rel + (lane & (boxes - 1)) - wb) & 31);
      const bool wanted = lane < boxes && t + box_rows > cur.ulo && t < cur.L;
      const bool valid = wanted && phys >= 0 && phys < p.num_blocks;
      const int row = valid ? (phys * p.hkv + cur.g) * p.block_size + (t & (p.block_size - 1)) : -1;
      const uint32_t bad = __ballot_sync(FULL, wanted && !valid), good = __ballot_sync(FULL, valid);
      if (lane < 4) sh.rows[at][lane] = row;  // for V; read long before tile n + kRing is issued
      const int row0 = __shfl_sync(FULL, row, 0), row1 = __shfl_sync(FULL, row, 1);
      const int row2 = __shfl_sync(FULL, row, 2), row3 = __shfl_sync(FULL, row, 3);
      if (umma::elect()) {
        uint32_t slices = 0;
        for (int k = 0; k < 4; ++k) slices |= ((bad >> (k * kSliceTokens >> p.log2_box)) & 1u) << k;
        sh.skip[at] = (uint8_t)slices;
        if (bad) raise_error(PA_DEVERR_BLOCK);
        const uint32_t full = bar(sh.kfull[stage]), dst = k_s + stage * C::kKBytes;
        if (good) mbar_arrive_expect_tx(full, __popc(good) * C::kPanels * box_rows * 128);
        else mbar_arrive(full);
        tree_load_boxes<C::kPanels>(dst, &kmap, full, row0, row1, row2, row3, box_rows);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.rfull[at]));
      issued = n + 1;
      ++i;
    }
    if (lane < C::kRowTiles && mt0 + lane < p.m_tiles) {  // the range's record, for each row tile
      const bool has = rec.x > 0 && (mt0 + lane) * p.q_nodes < rec.w;
      p.ws_rec[(int64_t)grp * p.m_tiles + mt0 + lane] = has ? rec : make_int4(0, 0, 0, 0);
    }
    if (lane == 0) {  // no more tiles; the ring's place is free, as for a tile
      sh.rows[issued % C::kRing][0] = -2;
      mbar_arrive(bar(sh.rfull[issued % C::kRing]));
    }
    if (!ok) give_up();
    if (!ok || *abort_flag) {
      // Before the CTA releases its shared memory: give the last loads of the
      // ring a bounded time to land (earlier ones have, their stages were reused).
      for (int j = max(issued - NK, 0); j < issued; ++j)
        (void)mbar_wait_bounded(bar(sh.kfull[j % NK]), (j / NK) & 1, kDrainLimitNs);
    }
  } else if (warp == kTreeVWarp) {
    // ================= TMA loads of V (one elected lane) =================
    if (umma::elect()) {
      const int box_rows = 1 << p.log2_box;
      bool ok = true;
      int n = 0;
      for (;; ++n) {
        const int stage = n % NV, at = n % C::kRing;
        ok = mbar_wait_bounded(bar(sh.rfull[at]), (n / C::kRing) & 1, kWaitLimitNs);
        if (!ok || *abort_flag) break;
        const int4 row = *reinterpret_cast<const int4*>(sh.rows[at]);
        if (row.x == -2) break;
        ok = n < NV || mbar_wait_bounded(bar(sh.vempty[stage]), (n / NV - 1) & 1, kWaitLimitNs);
        if (!ok || *abort_flag) break;
        const uint32_t full = bar(sh.vfull[stage]), dst = v_s + stage * C::kKBytes;
        const int good = (row.x >= 0) + (row.y >= 0) + (row.z >= 0) + (row.w >= 0);
        if (good) mbar_arrive_expect_tx(full, good * C::kPanels * box_rows * 128);
        else mbar_arrive(full);
        tree_load_boxes<C::kPanels>(dst, &vmap, full, row.x, row.y, row.z, row.w, box_rows);
      }
      if (!ok) {
        raise_error(PA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      if (!ok || *abort_flag) {  // as for K
        for (int j = max(n - NV, 0); j < n; ++j)
          (void)mbar_wait_bounded(bar(sh.vfull[j % NV]), (j / NV) & 1, kDrainLimitNs);
      }
    }
  } else if (warp == kTreeMendWarp) {
    // ================= mending of V =================
    // Every tile of V passes through here between its load and its product.  Most
    // pass as they are.
    bool ok = true;
    int x = 0;
    for (int u = 0; ok && !*abort_flag; ++u) {
      ok = wait_use(sh.pfull[u % kTreePieces], u / kTreePieces);
      if (!ok) break;
      const TreePiece c = sh.pieces[u % kTreePieces];
      uint64_t* bad = sh.bad[u % kTreeMarks];
      if (lane < 4) bad[lane] = 0;  // every warp is past the piece kTreeMarks ago
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.pempty[u % kTreePieces]));
      if (c.b < 0) break;
      const int base = c.L - c.n, kt0 = c.ulo & ~(TILE - 1);
      const int w_end = p.window > 0 ? min(base, c.ulo + TILE - 1) : 0;  // rows' windows start before it
      for (int i = c.t0; i < c.t1; ++i, ++x) {
        ok = wait_use(sh.vfull[x % NV], x / NV);
        if (!ok) break;
        const int kt = kt0 + i * TILE;
        const uint32_t skip = *const_cast<volatile uint8_t*>(&sh.skip[x % C::kRing]);
        if (kt < w_end || kt + TILE > base || kt < c.ulo || skip != 0) {
          constexpr int CPR = C::kPanels * 8, RPI = 32 / CPR, UNROLL = 8;  // 16-byte chunks of a row, rows at a time
          const uint32_t vst = v_s + (x % NV) * C::kKBytes;
          // Rows of V that no row attends (they were not loaded, or hold what
          // stands behind the end): zero.  Rows that some may attend and some
          // not, the tree's and those at the windows' starts: see above.
          uint64_t none = low_bits(min(max(c.ulo - kt, 0), TILE)) | ~low_bits(min(max(c.L - kt, 0), TILE));
          for (int e = 0; e < 4; ++e)
            if ((skip >> e) & 1u) none |= 0xffffull << (16 * e);
          const bool tree = kt + TILE > base;
          uint64_t some = tree ? ~low_bits(max(base - kt, 0)) : 0ull;
          if (kt < w_end) some |= low_bits(min(w_end - kt, TILE));
          some &= ~none;
          const int slot = tree ? 2 + (kt - (base & ~(TILE - 1))) / TILE : i;
          auto chunk = [&](int at) {  // this lane's of row `at`
            return vst + (lane % CPR >> 3) * C::kKVPanelBytes + at * 128 + ((lane & 7) << 4);
          };
#pragma unroll 1
          for (int from = 0; from < TILE; from += UNROLL * RPI) {
            const uint64_t some_here = (some >> from) & low_bits(UNROLL * RPI);
            if (some_here) {
              uint32_t v[UNROLL][4], seen = 0;
#pragma unroll
              for (int j = 0; j < UNROLL; ++j) {
                const int at = from + j * RPI + lane / CPR;
                v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0;
                if ((some >> at) & 1ull)
                  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                               : "=r"(v[j][0]), "=r"(v[j][1]), "=r"(v[j][2]), "=r"(v[j][3])
                               : "r"(chunk(at)));
              }
              // Exponent bits all set (not finite): 0x7f80 and above without the sign.
#pragma unroll
              for (int j = 0; j < UNROLL; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) seen |= (v[j][k] & 0x7fff7fffu) + 0x00800080u;
              if (seen & 0x80008000u) {
#pragma unroll 1
                for (int j = 0; j < UNROLL; ++j) {
                  const int at = from + j * RPI + lane / CPR;
                  if (!((some >> at) & 1ull)) continue;
                  bool change = false;
#pragma unroll 1
                  for (int k = 0; k < 4; ++k) {
                    uint32_t w;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(chunk(at) + 4 * k));
                    uint32_t keep = w;
                    if ((w & 0x7f80u) == 0x7f80u) keep &= 0xffff0000u;
                    if ((w & 0x7f800000u) == 0x7f800000u) keep &= 0xffffu;
                    if (keep == w) continue;
                    change = true;
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(chunk(at) + 4 * k), "r"(keep) : "memory");
                  }
                  if (change) atomicOr(reinterpret_cast<unsigned long long*>(&bad[slot]), 1ull << at);
                }
              }
            }
            if ((none >> from) & low_bits(UNROLL * RPI)) {
#pragma unroll
              for (int j = 0; j < UNROLL; ++j) {
                const int at = from + j * RPI + lane / CPR;
                if ((none >> at) & 1ull)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(chunk(at)), "r"(0) : "memory");
              }
            }
          }
        }
        fence_proxy_async_smem();  // visible to the tensor core's reads
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.vready[x % NV]));
      }
    }
    if (!ok) give_up();
  } else if (warp == kTreeMmaWarp) {
    // ================= MMA issuer (one elected lane, from here to the end) =================
    // Everything this lane does between two products delays the next one, so
    // stages and parities are counted up, not divided out of a tile's number.
    if (umma::elect()) {
      const uint32_t idesc_s = umma::idesc_bf16(kTreeRows, TILE, 0, 0);
      const uint32_t idesc_o = umma::idesc_bf16(kTreeRows, D, 0, 1);
      // Descriptors of the first Q, K and V bytes; the others lie (bytes / 16) on.
      const uint64_t q_desc = umma::desc_sw128(q_s, 16, 1024), k_desc = umma::desc_sw128(k_s, 16, 1024);
      const uint64_t v_desc = umma::desc_sw128(v_s, C::kKVPanelBytes, 1024);
      const uint32_t kfull = bar(sh.kfull[0]), kempty = bar(sh.kempty[0]), vready = bar(sh.vready[0]);
      const uint32_t vempty = bar(sh.vempty[0]), sfull = bar(sh.sfull[0][0]), pready = bar(sh.pready[0][0]);
      const uint32_t odone = bar(sh.odone[0][0]);
      auto wait = [&](uint32_t b, uint32_t parity) { return mbar_wait_bounded(b, parity, kWaitLimitNs); };
      // S buffer (and its barriers) of tile x for row tile t, and its use's parity.
      auto buffer = [&](int x, int t) { return PAIR ? 2 * t + (x & 1) : 2 * (x & 1) + (x >> 1 & 1); };
      auto parity = [&](int x) { return (uint32_t)(PAIR ? x >> 1 : x >> 2) & 1u; };
      int x = 0, y = 0;                           // next tile of S, of P V
      uint32_t kst = 0, kph = 0, vst = 0, vph = 0;  // their stages, and the parities of these
      int asked = 0;                              // pieces whose Q load is issued
      TreePiece next;
      // Take piece number `asked` from the ring and load its Q.  The last piece's
      // last S is done, or not issued; false: not in the ring (yet), unless `block`.
      bool ok = true;
      auto ask = [&](bool block) {
        const uint32_t in = bar(sh.pfull[asked % kTreePieces]), par = (asked / kTreePieces) & 1;
        if (block ? !wait(in, par) : !mbar_try_wait(in, par)) return false;
        if (x > 0 && !wait(sfull + 8 * buffer(x - 1, PAIR ? 1 : 0), parity(x - 1))) return false;
        next = sh.pieces[asked % kTreePieces];
        mbar_arrive(bar(sh.pempty[asked % kTreePieces]));
        ++asked;
        if (next.b < 0) return true;
        const int tiles = min(C::kRowTiles, p.m_tiles - mt0);
        mbar_arrive_expect_tx(bar(sh.qfull), tiles * C::kPanels * p.q_nodes * G * 128);
#pragma unroll 1
        for (int k = 0; k < tiles * C::kPanels; ++k)
          tma_load_3d(q_s + k * C::kQPanelBytes, &qmap, bar(sh.qfull), k % C::kPanels * 64, next.g * G,
                      next.b * p.tree_len + (mt0 + k / C::kPanels) * p.q_nodes);
        return true;
      };
      for (int u = 0;; ++u) {
        ok = asked > u || ask(true);
        if (!ok || next.b < 0 || *abort_flag) break;
        // Step i: P V of the piece's tile i - LAG, then S of its tile i, whose buffer
        // is free by then.  (PAIR: row tile by row tile, so that the second
        // group's S comes when the first group has finished a tile: the groups, whose
        // warps share the special function units, run half a tile apart.)  The
        // last steps have no S: there the next piece's Q is asked for.
        const int len = next.t1 - next.t0;
#pragma unroll 1
        for (int i = 0; ok && i < len + LAG; ++i) {
          const bool s = i < len, o = i >= LAG;
          if (o) {
            if (i == LAG && u > 0) ok = wait(bar(sh.ofree), (u - 1) & 1);  // the last piece's O is read
            ok = ok && wait(vready + 8 * vst, vph);
          }
          if (s) ok = ok && (i > 0 || wait(bar(sh.qfull), u & 1)) && wait(kfull + 8 * kst, kph);
          else if (asked == u + 1) (void)ask(false);
          if (!ok) break;
#pragma unroll
          for (int t = 0; t < C::kRowTiles; ++t) {
            if (o) {
              const uint32_t at = buffer(y, t);
              if (!(ok = wait(pready + 8 * at, parity(y)))) break;
              umma::fence_after();
              const uint64_t vd = v_desc + vst * (C::kKBytes / 16);
              const uint32_t pcol = tmem + C::kSCol + at * TILE;
#pragma unroll
              for (int kk = 0; kk < TILE / 16; ++kk)
                umma::mma_f16_tmem_a(tmem + C::kOCol + t * D, pcol + kk * 8, vd + kk * 16 * 128 / 16, idesc_o,
                                     kk > 0 || i > LAG ? 1u : 0u);
              umma::commit(odone + 8 * at);
              if (t == C::kRowTiles - 1) umma::commit(vempty + 8 * vst);
            }
            if (s) {
              umma::fence_after();
              const uint32_t at = buffer(x, t), col = tmem + C::kSCol + at * TILE;
              const uint64_t qd = q_desc + t * (C::kQBytes / 16), kd = k_desc + kst * (C::kKBytes / 16);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma::mma_f16(col, qd + ((kk >> 2) * C::kQPanelBytes + (kk & 3) * 32) / 16,
                              kd + ((kk >> 2) * C::kKVPanelBytes + (kk & 3) * 32) / 16, idesc_s, kk > 0 ? 1u : 0u);
              umma::commit(sfull + 8 * at);
              if (t == C::kRowTiles - 1) umma::commit(kempty + 8 * kst);
            }
          }
          if (o) {
            ++y;
            if (++vst == NV) vst = 0, vph ^= 1;
          }
          if (s) {
            ++x;
            if (++kst == NK) kst = 0, kph ^= 1;
          }
        }
        if (!ok) break;
      }
      if (!ok) {
        raise_error(PA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      if (!ok || *abort_flag) {  // the MMAs and loads issued get a bounded time to finish before TMEM is freed
        umma::commit(bar(sh.drain));
        if (asked > 0) (void)mbar_wait_bounded(bar(sh.qfull), (asked - 1) & 1, kDrainLimitNs);
        (void)mbar_wait_bounded(bar(sh.drain), 0, kDrainLimitNs);
      }
    }
  } else {
    // ================= softmax warps 0-7: one query row per thread =================
    const int grp_w = warp >> 2, quad = warp & 3, r = quad * 32 + lane;  // TMEM lane = row
    const int mt = PAIR ? mt0 + grp_w : mt0;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t o_col = lane_base + C::kOCol + (PAIR ? grp_w * D : 0);
    const int row_stride = tree_row_stride(p);
    const bool sectors = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;  // out may be aligned to 16 bytes only
    const int node = mt * p.q_nodes + r / G;  // this thread's row: its node and its head
    const int64_t head = (int64_t)node * p.hq + r % G;
    // Scores in the base-2 domain: x * xs, or the capped score
    // cap tanh(s / cap) log2 e = cap_a - cap_b / (1 + 2^(x cap_c)), since tanh y = 1 - 2 / (1 + e^(2 y)).
    const float xs_all = p.scale * kLog2e;
    const bool pre = p.use_softcap || !(xs_all > 0.f);  // scores computed ahead of the maximum
    const float xs = pre ? 1.f : xs_all;
    const float cap_a = p.softcap * kLog2e, cap_b = 2.f * cap_a;
    const float cap_c = p.use_softcap ? 2.f * xs_all / p.softcap : 0.f;
    // Where a score is at most half of the cap, y = s / cap <= 0.5, the Taylor series
    // y - y^3 / 3 + 2 y^5 / 15 - ... to y^11 is within 5e-7 of tanh y, and takes
    // the place of two special function results by five packed operations.
    const float cap_y = p.use_softcap ? p.scale / p.softcap : 0.f;
    const float cap_lim = p.use_softcap ? 0.5f / fabsf(cap_y) : 0.f;
    const float2 cap_y2 = make_float2(cap_y, cap_y), cap_s2 = make_float2(xs_all, xs_all);

    // Rows of nodes that a tree does not have: no piece writes them.
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
      const TreeSeq s = tree_seq(p, b, false);
      const int done = s.n * G, per_head = (p.tree_len * G - done) * (D / 8);
      for (int g = 0; g < p.hkv && per_head > 0; ++g) {
        for (int i = tid; i < per_head; i += 256) {
          const int z = done + i / (D / 8);
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) +
                             (((int64_t)b * p.tree_len + z / G) * p.hq + (int64_t)g * G + z % G) * D + i % (D / 8) * 8;
          *reinterpret_cast<uint4*>(o) = make_uint4(0, 0, 0, 0);
        }
      }
    }

    bool ok = true;
    int x0 = 0;  // the CTA's tiles before this piece
    TreePiece c, nxt;
    uint64_t word = 0;  // this row's mask word in the next piece
    nxt.b = -1;
    // Turn u: the tiles of piece u - 1, the next piece's mask words (they come while
    // the last P V runs), then the rows of piece u - 1.
    for (int u = 0; ok; ++u) {
      c = nxt;
      const bool work = u > 0;
      const int rows = max(0, min(p.q_nodes, c.n - mt * p.q_nodes)) * G;
      const bool real = r < rows, active = 32 * quad < rows;
      const int L = c.L, base = L - c.n, kt0 = c.ulo & ~(TILE - 1), len = work ? c.t1 - c.t0 : 0;
      const TreeRow row = work ? tree_row(p, TreeSeq{L, c.n, base}, c.b, node, word) : TreeRow{0, 0};
      // Rows' windows start in [ulo, ulo + 63] (a depth is at most 63) and at most at base.
      const int w_end = p.window > 0 ? min(base, c.ulo + TILE - 1) : 0;
      const uint64_t* bad = sh.bad[(u + kTreeMarks - 1) % kTreeMarks];  // piece u - 1's
      float m = -CUDART_INF_F, l = 0.f;  // this group's last reference, its sum
      for (int i = PAIR ? 0 : (x0 + grp_w) & 1; i < len; i += PAIR ? 1 : 2) {
        const int x = x0 + i, k = count_of(x);
        ok = wait_use(sh.sfull[grp_w][k & 1], k >> 1);
        if (!ok) break;
        umma::fence_after();
        const int kt = kt0 + (c.t0 + i) * TILE;
        const uint32_t skip = *const_cast<volatile uint8_t*>(&sh.skip[x % C::kRing]);
        const bool edge = kt < w_end || kt + TILE > base;
        const bool masked = edge || kt < c.ulo || skip != 0;
        const uint32_t s_col = lane_base + C::kSCol + (2 * grp_w + (k & 1)) * TILE;
        if (active) {
          if (pre || masked) {
            // Cap and masks, in place and 16 columns at a time: this path is
            // rare or bound by its exponentials, and unrolled over the tile it
            // was most of the kernel's code (its first pass, from a cold
            // instruction cache, took 11,000 cycles).
            uint64_t see = ~0ull;
            if (masked) {  // bit e: this row attends position kt + e
              const int from = min(max(row.lo - kt, 0), TILE), to = min(max(base - kt, 0), TILE);
              see = low_bits(to) & ~low_bits(from);
              if (kt >= base) see |= row.nodes >> (kt - base);
              else if (base - kt < TILE) see |= row.nodes << (base - kt);
              for (int e = 0; e < 4; ++e)
                if ((skip >> e) & 1u) see &= ~(0xffffull << (16 * e));
            }
#pragma unroll 1
            for (int e = 0; e < TILE; e += 16) {
              float v[16];
              umma::ld16(s_col + e, v);
              if (p.use_softcap) {
                float big = 0.f;  // NaN: not at all within the bound
#pragma unroll
                for (int j = 0; j < 16; ++j) big = (fabsf(v[j]) <= cap_lim) ? big : 1.f;
                if (__any_sync(FULL, big != 0.f && real)) {
#pragma unroll
                  for (int j = 0; j < 16; ++j) {
                    float a, q;
                    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(v[j] * cap_c));
                    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.f + a));
                    v[j] = fmaf(-cap_b, q, cap_a);
                  }
                } else {
#pragma unroll
                  for (int j = 0; j < 16; j += 2) {
                    const float2 a = make_float2(v[j], v[j + 1]), y = mul_f32x2(a, cap_y2), z = mul_f32x2(y, y);
                    float2 t = make_float2(-1382.f / 155925.f, -1382.f / 155925.f);
                    t = fma_f32x2(t, z, make_float2(62.f / 2835.f, 62.f / 2835.f));
                    t = fma_f32x2(t, z, make_float2(-17.f / 315.f, -17.f / 315.f));
                    t = fma_f32x2(t, z, make_float2(2.f / 15.f, 2.f / 15.f));
                    t = fma_f32x2(t, z, make_float2(-1.f / 3.f, -1.f / 3.f));
                    t = fma_f32x2(t, z, make_float2(1.f, 1.f));
                    t = mul_f32x2(t, mul_f32x2(a, cap_s2));
                    v[j] = t.x, v[j + 1] = t.y;
                  }
                }
              } else if (pre) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] *= xs_all;
              }
              const uint32_t bits = (uint32_t)(see >> e);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = (bits >> j) & 1u ? v[j] : -CUDART_INF_F;
              umma::st16(s_col + e, v);
            }
          }
          float y[TILE];
          {
            uint32_t v[TILE / 32][32];
#pragma unroll
            for (int e = 0; e < TILE / 32; ++e) umma::ld32_nowait(s_col + e * 32, v[e]);
            umma::wait_ld();
#pragma unroll
            for (int e = 0; e < TILE; ++e) y[e] = __uint_as_float(v[e / 32][e % 32]);
          }
          float mx[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) mx[e] = max3(y[e], y[e + 8], y[e + 16]);
#pragma unroll
          for (int e = 24; e < 56; e += 16)
#pragma unroll
            for (int j = 0; j < 8; ++j) mx[j] = max3(mx[j], y[e + j], y[e + 8 + j]);
#pragma unroll
          for (int j = 0; j < 8; ++j) mx[j] = fmaxf(mx[j], y[56 + j]);
          const float top = fmaxf(max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[4]), max3(mx[5], mx[6], mx[7])) * xs;  // xs > 0
          // The reference so far: this group's, or (not PAIR) the tile's before, the other group's.
          float before = m;
          if (!PAIR) {
            before = -CUDART_INF_F;
            if (i > 0) {
              ok = wait_use(sh.mready[quad][(x - 1) & 1], (x - 1) >> 1);
              if (!ok) break;
              before = sh.m[(x - 1) & 1][r];
            }
          }
          // Lazy rescaling, as in the prefill: the reference moves when the
          // tile's maximum exceeds it by more than 8 (base 2), so weights stay
          // below 256 and share the reference of the sum and of O.
          const float now = (before == -CUDART_INF_F || top > before + 8.f) ? top : before;
          if (!PAIR) {
            sh.m[x & 1][r] = now;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(sh.mready[quad][x & 1]));
          }
          const float ref = now == -CUDART_INF_F ? 0.f : now;
          float fade;  // of this group's sum so far
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(fade) : "f"(m - ref));
          m = now;
          // Weights in fp32 for the sum, rounded to bf16 for the second product
          // (a relative 2^-8 at most on each weight, what the output's own
          // rounding allows; the tensor cores take both operands in one type).
          float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 xs2 = make_float2(xs, xs), ref2 = make_float2(-ref, -ref);
          uint32_t pk[TILE / 2];
#pragma unroll
          for (int e = 0; e < TILE / 2; ++e) {
            const float2 a = fma_f32x2(make_float2(y[2 * e], y[2 * e + 1]), xs2, ref2);
            float2 w;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w.x) : "f"(a.x));
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w.y) : "f"(a.y));
            ps[e & 1] = add_f32x2(ps[e & 1], w);
            pk[e] = pack_bf16x2(w.x, w.y);
          }
          l = fmaf(l, fade, (ps[0].x + ps[1].x) + (ps[0].y + ps[1].y));
          umma::st16_nowait(s_col, *reinterpret_cast<uint32_t(*)[16]>(&pk[0]));
          umma::st16_nowait(s_col + 16, *reinterpret_cast<uint32_t(*)[16]>(&pk[16]));
          // (The first tile's P V overwrites O; rows that nobody reads move nothing.)
          if (i > 0 && __any_sync(FULL, now != before && real)) {
            const float alpha = exp2f(before - ref);
            const int w = PAIR ? grp_w : group_of(x - 1), kb = count_of(x - 1);
            ok = wait_use(sh.odone[w][kb & 1], kb >> 1);
            if (!ok) break;
            umma::fence_after();
#pragma unroll 1
            for (int e = 0; e < D / 16; ++e) {
              float v[16];
              umma::ld16(o_col + e * 16, v);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] *= alpha;
              umma::st16(o_col + e * 16, v);
            }
          }
          umma::wait_st();
        } else if (!PAIR && lane == 0) {
          mbar_arrive(bar(sh.mready[quad][x & 1]));  // one arrival a tile, whoever reads
        }
        umma::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.pready[grp_w][k & 1]));
      }
      if (!ok || *abort_flag) break;
      // The piece after is in the ring by now, or comes without this warp's help.
      ok = wait_use(sh.pfull[u % kTreePieces], u / kTreePieces);
      if (!ok) break;
      nxt = sh.pieces[u % kTreePieces];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.pempty[u % kTreePieces]));
      word = nxt.b >= 0 ? tree_word(p, nxt.b, nxt.n, node) : 0ull;  // used at the next turn
      if (!work) {
        if (nxt.b < 0) break;
        continue;
      }

      // ---- write the piece's rows -------------------------------------------------------
      const int last = x0 + len - 1, kl = count_of(last);
      x0 += len;
      float fin = m;  // the reference of the piece's last tile
      if (!PAIR && active && group_of(last) != grp_w) {
        ok = wait_use(sh.mready[quad][last & 1], last >> 1);
        if (!ok) break;
        fin = sh.m[last & 1][r];
      }
      if (!PAIR) l *= exp2f(m - (fin == -CUDART_INF_F ? 0.f : fin));
      ok = wait_use(sh.odone[PAIR ? grp_w : group_of(last)][kl & 1], kl >> 1);
      if (!ok) break;
      umma::fence_after();
      if (!PAIR && active) sh.l[grp_w][r] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.epi));
      ok = wait_use(sh.epi, u - 1);
      if (!ok) break;
      if (!PAIR && active) l = sh.l[0][r] + sh.l[1][r];
      uint64_t marks = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) marks |= *const_cast<const volatile uint64_t*>(&bad[e]);
      const bool begins = c.t0 == 0, whole = begins && c.t1 == c.tiles;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int64_t slot = ((int64_t)grp * p.m_tiles + mt) * 2 + (begins ? 1 : 0);
      float* po = p.ws_o + slot * row_stride * D + r * 4;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) +
                            ((int64_t)c.b * p.tree_len * p.hq + (int64_t)c.g * G + head) * D;
      if (active) {
        // Not PAIR: each group writes half of the columns.
        constexpr int CH = PAIR ? D / 16 : D / 32;  // 16-column chunks
        const int e0 = PAIR ? 0 : grp_w * CH;
        if (marks) {  // give back what was taken out of V, to the rows that attend it
#pragma unroll 1
          for (int e = e0; e < e0 + CH; ++e) {
            float v[16];
            umma::ld16(o_col + e * 16, v);
            for (int z = 0; real && z < 4; ++z) {
              uint64_t rest = bad[z];
              const int kt = z < 2 ? kt0 + z * TILE : (base & ~(TILE - 1)) + (z - 2) * TILE;
              while (rest) {
                const int t = kt + __ffsll((long long)rest) - 1;
                rest &= rest - 1;
                if (t < base ? t < row.lo : !((row.nodes >> (t - base)) & 1ull)) continue;
                const int phys = p.block_tables[(int64_t)c.b * p.max_blocks + (t >> p.log2_bs)];
                const __nv_bfloat16* src =
                    static_cast<const __nv_bfloat16*>(p.v_cache) +
                    (((int64_t)phys * p.hkv + c.g) * p.block_size + (t & (p.block_size - 1))) * D + e * 16;
                for (int j = 0; j < 16; ++j) {
                  const float f = __bfloat162float(src[j]);
                  if (!isfinite(f)) v[j] += f;
                }
              }
            }
            __syncwarp();
            umma::st16(o_col + e * 16, v);
          }
        }
#pragma unroll 1
        for (int e = e0; e < e0 + CH; e += 2) {  // 32 columns
          uint32_t f[32];
          umma::ld32_nowait(o_col + e * 16, f);
          umma::wait_ld();
          if (!real) continue;
          if (whole) {
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              o[j] = pack_bf16x2(__uint_as_float(f[2 * j]) * inv, __uint_as_float(f[2 * j + 1]) * inv);
            if (sectors) {
              st_global_32(orow + e * 16, *reinterpret_cast<uint32_t(*)[8]>(&o[0]));
              st_global_32(orow + e * 16 + 16, *reinterpret_cast<uint32_t(*)[8]>(&o[8]));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                reinterpret_cast<uint4*>(orow + e * 16)[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
          } else {
            uint4* at = reinterpret_cast<uint4*>(po + (int64_t)e * 4 * row_stride * 4);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              at[(int64_t)j * row_stride] = make_uint4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
          }
        }
        if (real && !whole && (PAIR || grp_w == 0))
          *reinterpret_cast<float2*>(p.ws_ml + (slot * row_stride + r) * 2) = make_float2(fin, l);
      }
      umma::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.ofree));
      if (nxt.b < 0) break;
    }
    if (!ok) give_up();
  }
  // Every tcgen05 access is complete (waited); free the tensor memory.
  umma::fence_before();
  __syncthreads();
  if (warp == 0) {
    umma::fence_after();
    umma::dealloc(tmem, 512);
  }
}

// Joins the pieces of each unit that was cut.  blockIdx.x: a record, of range c
// and row tile t: the unit whose first piece is in c (slot 1) and that goes on;
// the other pieces are in slot 0 of the next ranges.  With M = max m_p:
//   out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,
// in piece order.  blockIdx.y: 8 EACH rows; a thread has four columns of EACH of
// them, and neighbouring threads neighbouring rows, as the partials lie.  M runs
// along, and DEPTH pieces are loaded at a time (two of 74 on one unit: 62 us, four
// 56, eight 55; but eight cost registers: 256 trees of 24 nodes 108 for 106).
template <int D, int EACH>
__global__ void __launch_bounds__(2 * D) tree_combine_kernel(const TreeParams p) {
  constexpr int kRows = kTreeCombineRows, DEPTH = EACH == 1 ? 4 : 2;
  pdl_wait();  // the partials come from the attention grid
  const int c = blockIdx.x / p.m_tiles, t = blockIdx.x - c * p.m_tiles;
  const int ranges = gridDim.x / p.m_tiles;
  const int4 rec = p.ws_rec[blockIdx.x];
  if (rec.x < 2 || c + rec.x > ranges) return;
  if ((unsigned)rec.y >= (unsigned)p.batch || (unsigned)rec.z >= (unsigned)p.hkv) return;  // left by a call that gave up
  const int G = p.group, row_stride = tree_row_stride(p);
  const int r0 = blockIdx.y * EACH * kRows + (threadIdx.x & (kRows - 1)), col4 = threadIdx.x / kRows;
  const int rows = min(p.q_nodes, min(rec.w, p.tree_len) - t * p.q_nodes) * G;  // the unit's in this row tile
  if (r0 >= rows) return;
  auto slot = [&](int k) { return ((int64_t)(c + k) * p.m_tiles + t) * 2 + (k == 0 ? 1 : 0); };
  float M[EACH], den[EACH];
  float4 acc[EACH];
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    M[j] = -CUDART_INF_F;
    den[j] = 0.f;
    acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int k0 = 0; k0 < rec.x; k0 += DEPTH) {
    float2 ml[DEPTH][EACH];
    float4 o[DEPTH][EACH];
#pragma unroll
    for (int k = 0; k < DEPTH; ++k)
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        const int r = r0 + j * kRows;
        ml[k][j] = make_float2(-CUDART_INF_F, 0.f);
        o[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && k0 + k < rec.x) {
          const int64_t at = slot(k0 + k);
          ml[k][j] = *reinterpret_cast<const float2*>(p.ws_ml + (at * row_stride + r) * 2);
          o[k][j] = *reinterpret_cast<const float4*>(p.ws_o + (at * (D / 4) + col4) * row_stride * 4 + r * 4);
        }
      }
#pragma unroll
    for (int k = 0; k < DEPTH; ++k)
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        const float top = fmaxf(M[j], ml[k][j].x), ref = top == -CUDART_INF_F ? 0.f : top;
        const float old = exp2f(M[j] - ref), w = exp2f(ml[k][j].x - ref);
        M[j] = top;
        den[j] = fmaf(w, ml[k][j].y, old * den[j]);
        acc[j].x = fmaf(w, o[k][j].x, old * acc[j].x);
        acc[j].y = fmaf(w, o[k][j].y, old * acc[j].y);
        acc[j].z = fmaf(w, o[k][j].z, old * acc[j].z);
        acc[j].w = fmaf(w, o[k][j].w, old * acc[j].w);
      }
  }
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int r = r0 + j * kRows;
    if (r >= rows) continue;
    const float inv = den[j] > 0.f ? 1.f / den[j] : 0.f;  // a row that attends nothing is zero
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + col4 * 4 +
                         (((int64_t)rec.y * p.tree_len + t * p.q_nodes + r / G) * p.hq + (int64_t)rec.z * G + r % G) * D;
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack_bf16x2(acc[j].x * inv, acc[j].y * inv), pack_bf16x2(acc[j].z * inv, acc[j].w * inv));
  }
}

}  // namespace pa
