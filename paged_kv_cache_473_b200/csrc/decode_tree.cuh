// Attention of a drafted tree over the paged cache, bf16, on the 5th-generation
// tensor cores (tcgen05, accumulators in tensor memory).
//
// The n * G query rows of a (sequence, kv head) unit -- row r = (node r / G,
// head r % G) -- are the 128 rows of one UMMA tile (m_tiles tiles of whole
// nodes where there are more), whatever the tree looks like: the tree is in the
// masks of the last keys only.  One 3-D TMA box (64 columns, G heads, the
// tile's nodes) lands them in that order; rows past them, of shared memory that
// holds something else, give results that nobody reads.  The unit's keys and values stream in 64-token tiles, as in the
// prefill kernel: S = Q K^T into one of two TMEM buffers, the softmax by one
// thread per row, P back into the columns S came from, O += P V in TMEM.
//
// Split.  The tiles of all units, in order, are one line of work that is cut
// into equal ranges, one for each group of m_tiles CTAs (as many CTAs as are
// resident at once; the CTAs of a group take the same keys for another 128 rows
// at about the same time, so that these are read from DRAM once).  A CTA runs
// the pieces of units in its range one after the other; its loads run on into
// the next piece while the softmax is still at the last one.  A unit that lies
// in one range is written as rows of `out`; the pieces of one that is cut are
// written as partials, at most two per CTA (the piece that comes from the range
// before, the one that goes on in the next), and joined by tree_combine_kernel.
// So every CTA streams the same number of tiles whatever the lengths, and the
// workspace does not grow with the batch.
//
// Warps 0-3: softmax, one row per thread; they also write the rows.  Warp 4:
// MMA issue, and the load of a piece's Q as soon as the last S of the piece
// before is done.  Warp 5: TMA loads of K and V (16-row boxes, one per lane).
// What a role reads of the next piece (lengths, mask words, block ids) it reads
// one piece ahead.  Every wait is bounded; a wait that gives up raises the abort
// flag, which ends all roles.
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

constexpr int kTreeRows = 128;     // query rows per CTA (UMMA M)
constexpr int kTreeTile = 64;      // keys per tile
constexpr int kTreeMinTiles = 2;   // shortest range of a CTA: below, a piece's fixed cost outweighs its tiles
constexpr int kTreeThreads = 192;
constexpr int kTreeCombineRows = 8;

// QR: rows of Q that shared memory holds (64 or 128).  At head_dim 128 and 256
// the 64 rows that smaller trees leave free are one more V stage.
template <int D, int QR>
struct TreeCfg {
  static constexpr int kPanels = D / 64;  // 64-element (128-byte) column panels
  static constexpr int kKStages = D <= 64 ? 6 : 3;
  static constexpr int kVStages = D <= 64 ? 6 : (QR <= 64 ? 3 : 2);
  static constexpr int kQPanelBytes = QR * 128;
  static constexpr int kKVPanelBytes = kTreeTile * 128;
  static constexpr int kKBytes = kPanels * kKVPanelBytes;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kPanels * kQPanelBytes;
  static constexpr int kVOff = kKOff + kKStages * kKBytes;
  static constexpr int kBarOff = kVOff + kVStages * kKBytes;
  static constexpr int kSmemBytes = kBarOff + 768;
  static constexpr int kSCol = 0;              // two S buffers
  static constexpr int kOCol = 2 * kTreeTile;  // O: D columns
  static constexpr int kTmemCols = (2 * kTreeTile + D) <= 256 ? 256 : 512;
  static constexpr int kMinBlocks = D <= 128 ? 2 : 1;  // resident CTAs per SM: TMEM columns and shared memory allow these
};

// What the CTA's threads share besides the tiles (behind them, at kBarOff).
template <int D, int QR>
struct TreeShared {
  using C = TreeCfg<D, QR>;
  uint64_t kfull[C::kKStages], kempty[C::kKStages], vfull[C::kVStages], vempty[C::kVStages];
  uint64_t sfull[2], pready[2], odone[2], qfull, drain;
  uint64_t bad[3][4];      // by piece: rows of V with elements that are not finite, in each masked tile
  long long scan[8];
  long long w0, w1, per;   // the CTA's range of tiles
  int b0, off0;            // where it starts: sequence, tile within the sequence
  uint32_t skip[16];       // by tile: slices whose block id is bad
  uint32_t tmem;
  int abort;
};

// A piece: tiles [t0, t1) of the `tiles` tiles of unit (b, g).
struct TreePiece {
  int b, g, t0, t1, tiles;
  TreeSeq s;
  int ulo, kt0;     // first attended position; its tile's start
  long long start;  // tile t0 on the line of all work
};

// Walks the pieces of a CTA's range.
struct TreeWalk {
  long long w, w1;
  int b, off, tiles, ulo;
  TreeSeq s;
  int next_len, next_nodes;  // of sequence b + 1, loaded ahead

  __device__ __forceinline__ void start(const TreeParams& p, long long from, long long to, int b0, int off0) {
    w = from;
    w1 = to;
    b = b0;
    off = off0;
    next_len = p.context_lens[b];
    next_nodes = p.tree_lens ? p.tree_lens[b] : p.tree_len;
    load(p);
  }
  __device__ __forceinline__ void load(const TreeParams& p) {  // sequence b, whose lengths are here
    s = tree_fit(p, next_len, next_nodes, false);
    const int after = min(b + 1, p.batch - 1);
    next_len = p.context_lens[after];
    next_nodes = p.tree_lens ? p.tree_lens[after] : p.tree_len;
    ulo = tree_start(s, p.window);
    tiles = s.n > 0 ? (s.L - (ulo & ~(kTreeTile - 1)) + kTreeTile - 1) / kTreeTile : 0;
  }
  __device__ __forceinline__ bool next(const TreeParams& p, int mt, TreePiece& o) {
    while (w < w1) {
      while (off >= p.hkv * tiles) {  // w < w1 <= total: a sequence with tiles left exists
        if (b + 1 >= p.batch) return false;
        ++b;
        off = 0;
        load(p);
      }
      o.g = off / tiles;
      o.t0 = off - o.g * tiles;
      const int n = (int)min((long long)(tiles - o.t0), w1 - w);
      o.t1 = o.t0 + n;
      o.start = w;
      w += n;
      off += n;
      if (mt * p.q_nodes >= s.n) continue;  // this tree has no rows in the CTA's row tile
      o.b = b;
      o.tiles = tiles;
      o.s = s;
      o.ulo = ulo;
      o.kt0 = ulo & ~(kTreeTile - 1);
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ long long tree_tiles(const TreeParams& p, int b, bool report) {
  const TreeSeq s = tree_seq(p, b, report);
  if (s.n == 0) return 0;
  return (long long)p.hkv * ((s.L - (tree_start(s, p.window) & ~(kTreeTile - 1)) + kTreeTile - 1) / kTreeTile);
}

// Exclusive scan over the CTA's threads (two barriers).
__device__ __forceinline__ long long tree_scan(long long v, long long* scratch, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kTreeThreads / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  return before + incl - v;
}

// The range of group grp: its tiles [w0, w1) on the line of all work, and the
// sequence and the tile within it where the range starts.
template <typename Shared>
__device__ __forceinline__ void tree_locate(const TreeParams& p, int grp, int groups, Shared& sh) {
  const int tid = threadIdx.x;
  const bool report = blockIdx.x == 0;
  long long v = tid < p.batch ? tree_tiles(p, tid, report) : 0, total, more = 0;
  long long before = tree_scan(v, sh.scan, total);
  if (p.batch > kTreeThreads) {
    for (int b = tid + kTreeThreads; b < p.batch; b += kTreeThreads) more += tree_tiles(p, b, report);
    long long rest;
    tree_scan(more, sh.scan, rest);
    more = total;  // tiles before the next chunk of sequences
    total += rest;
  }
  const long long per = max((total + groups - 1) / groups, (long long)kTreeMinTiles);
  const long long w0 = min(grp * per, total);
  if (tid == 0) {
    sh.w0 = w0;
    sh.w1 = min(w0 + per, total);
    sh.per = per;
  }
  if (v > 0 && w0 >= before && w0 < before + v) {
    sh.b0 = tid;
    sh.off0 = (int)(w0 - before);
  }
  for (int c = kTreeThreads; c < p.batch && w0 >= more; c += kTreeThreads) {  // w0 and `more`: the same in all threads
    long long chunk;
    v = c + tid < p.batch ? tree_tiles(p, c + tid, false) : 0;
    before = more + tree_scan(v, sh.scan, chunk);
    if (v > 0 && w0 >= before && w0 < before + v) {
      sh.b0 = c + tid;
      sh.off0 = (int)(w0 - before);
    }
    more += chunk;
  }
  __syncthreads();
}

// Partials: slot 2 c of CTA c for the piece that comes from the range before,
// 2 c + 1 for the one that goes on in the next; element (row r, column d) of a
// slot at [d / 4][r][d % 4], so that a warp's rows are neighbours, and (m, l)
// of a row behind.
__device__ __forceinline__ int tree_row_stride(const TreeParams& p) {
  return (p.q_nodes * p.group + kTreeCombineRows - 1) & ~(kTreeCombineRows - 1);
}

template <int D, int QR>
__global__ void __launch_bounds__(kTreeThreads, TreeCfg<D, QR>::kMinBlocks)
    decode_tree_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using C = TreeCfg<D, QR>;
  using Shared = TreeShared<D, QR>;
  static_assert(sizeof(Shared) <= C::kSmemBytes - C::kBarOff, "shared area");
  constexpr uint32_t FULL = 0xffffffffu;
  constexpr int NK = C::kKStages, NV = C::kVStages, TILE = kTreeTile;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int G = p.group, mt = blockIdx.x % p.m_tiles, grp = blockIdx.x / p.m_tiles;

  pdl_launch_dependents();  // the combine may launch; it waits for this grid to finish
  if (smem_addr(smem) & 1023) {  // the swizzled tiles need 1024-byte alignment
    if (tid == 0) raise_error(PA_DEVERR_LAYOUT);
    return;
  }
  auto bar = [&](const uint64_t& b) { return smem_addr(&b); };
  if (tid == 0) {
    for (int s = 0; s < NK; ++s) mbar_init(bar(sh.kfull[s]), 1), mbar_init(bar(sh.kempty[s]), 1);
    for (int s = 0; s < NV; ++s) mbar_init(bar(sh.vfull[s]), 1), mbar_init(bar(sh.vempty[s]), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(sh.sfull[s]), 1);
      mbar_init(bar(sh.pready[s]), 4);
      mbar_init(bar(sh.odone[s]), 1);
    }
    mbar_init(bar(sh.qfull), 1);
    mbar_init(bar(sh.drain), 1);
    sh.abort = 0;
    mbar_init_fence();
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (tid < 12) sh.bad[tid / 4][tid % 4] = 0;
  pdl_wait();  // a programmatic dependent: nothing of global memory was touched before
  tree_locate(p, grp, gridDim.x / p.m_tiles, sh);

  // ---- rows that no piece writes: those of nodes that a tree does not have ------------------
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    const TreeSeq s = tree_seq(p, b, false);
    const int done = s.n * G, all = p.tree_len * G;
    const int per_head = (all - done) * (D / 8);
    for (int g = 0; g < p.hkv && per_head > 0; ++g) {
      for (int i = tid; i < per_head; i += kTreeThreads) {
        const int r = done + i / (D / 8);
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) +
                           (((int64_t)b * p.tree_len + r / G) * p.hq + (int64_t)g * G + r % G) * D + i % (D / 8) * 8;
        *reinterpret_cast<uint4*>(o) = make_uint4(0, 0, 0, 0);
      }
    }
  }
  if (sh.w0 >= sh.w1) {  // the same in all threads
    if (tid == 0) p.ws_rec[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  TreeWalk walk;
  walk.start(p, sh.w0, sh.w1, sh.b0, sh.off0);

  if (warp == 0) umma::alloc(smem_addr(&sh.tmem), C::kTmemCols);
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
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

  if (warp == 5) {
    // ================= TMA producer =================
    // One cursor per ring.  Block ids of a piece's 16-token slices come in
    // windows of 32, lane l holding slice wb + l (cur) and wb + 32 + l (nxt),
    // and those of the next piece's first window are loaded a piece ahead, so
    // that no load waits for a block table.
    struct Cursor {
      TreeWalk walk;
      TreePiece cur, nxt;
      bool more;  // nxt holds a piece
      bool live;  // cur holds a tile to load
      int i, wb, pages, pages2, first;
    };
    auto page_of = [&](const TreePiece& c, int q) {
      const int t = c.kt0 + c.t0 * TILE + q * kSliceTokens;
      return t < min(c.s.L, c.kt0 + c.t1 * TILE) ? p.block_tables[(int64_t)c.b * p.max_blocks + (t >> p.log2_bs)] : -1;
    };
    auto advance = [&](Cursor& c) {  // to the next piece
      c.cur = c.nxt;
      c.live = c.more;
      c.pages = c.first;
      c.i = c.live ? c.cur.t0 : 0;
      c.wb = 0;
      c.pages2 = c.live ? page_of(c.cur, 32 + lane) : -1;
      c.more = c.more && c.walk.next(p, mt, c.nxt);
      c.first = c.more ? page_of(c.nxt, lane) : -1;
    };
    auto start = [&](Cursor& c) {
      c.walk = walk;
      c.more = c.walk.next(p, mt, c.nxt);
      c.first = c.more ? page_of(c.nxt, lane) : -1;
      advance(c);
    };
    int issued[2] = {0, 0};
    auto issue = [&](Cursor& c, int kv) {  // the cursor's tile into its ring, as tile number issued[kv]
      const int n = issued[kv], stage = n % (kv ? NV : NK);
      const uint32_t full = kv ? bar(sh.vfull[stage]) : bar(sh.kfull[stage]);
      const int rel = 4 * (c.i - c.cur.t0);
      if (rel >= c.wb + 32) {
        c.wb += 32;
        c.pages = c.pages2;
        c.pages2 = page_of(c.cur, c.wb + 32 + lane);
      }
      const int s = lane / C::kPanels, pn = lane % C::kPanels;  // this lane's box: slice, panel
      const int t = c.cur.kt0 + c.i * TILE + s * kSliceTokens;
      const int phys = __shfl_sync(FULL, c.pages, (rel + (s & 3) - c.wb) & 31);
      const bool wanted = lane < 4 * C::kPanels && t + kSliceTokens > c.cur.ulo && t < c.cur.s.L;
      const bool valid = wanted && phys >= 0 && phys < p.num_blocks;
      if (kv == 0) {
        const uint32_t bad = __ballot_sync(FULL, wanted && !valid && pn == 0);
        if (lane == 0) {
          uint32_t slices = 0;
          for (int k = 0; k < 4; ++k) slices |= ((bad >> (k * C::kPanels)) & 1u) << k;
          sh.skip[n & 15] = slices;  // read behind this tile's S, long before tile n + 16 is issued
          if (bad) raise_error(PA_DEVERR_BLOCK);
        }
      }
      const uint32_t boxes = __popc(__ballot_sync(FULL, valid));
      if (lane == 0) {
        if (boxes) mbar_arrive_expect_tx(full, boxes * kSliceTokens * 128);
        else mbar_arrive(full);
      }
      __syncwarp();
      if (valid) {
        const uint32_t dst = (kv ? v_s : k_s) + stage * C::kKBytes + pn * C::kKVPanelBytes + s * kSliceTokens * 128;
        const int row = (phys * p.hkv + c.cur.g) * p.block_size + (t & (p.block_size - 1));
        tma_load_2d(dst, kv ? &vmap : &kmap, full, pn * 64, row);
      }
      issued[kv] = n + 1;
      if (++c.i >= c.cur.t1) advance(c);
    };
    // A K stage frees when the S that read it is done, a V stage when its P V
    // is.  The MMAs complete in issue order, S(m + 1) before P V(m) within a
    // piece, so the refills go in that order: K(m + 1 + NK), then V(m + NV).
    auto refill = [&](Cursor& c, int kv) {
      const int u = issued[kv] - (kv ? NV : NK);
      if (!wait_use(kv ? sh.vempty[u % NV] : sh.kempty[u % NK], u / (kv ? NV : NK))) return false;
      issue(c, kv);
      return true;
    };
    Cursor k, v;
    start(k);
    start(v);
    for (int i = 0; i < NK && k.live; ++i) issue(k, 0);
    for (int i = 0; i < NV && v.live; ++i) issue(v, 1);
    bool ok = true;
    if (k.live) ok = refill(k, 0);
    while (ok && (k.live || v.live) && !*abort_flag) {
      if (k.live) ok = refill(k, 0);
      if (ok && v.live) ok = refill(v, 1);
    }
    if (!ok) give_up();
    if (!ok || *abort_flag) {
      // Before the CTA releases its shared memory: give the last loads of each
      // ring a bounded time to land (earlier ones have, their stages were reused).
      for (int kv = 0; kv < 2; ++kv) {
        const int n = kv ? NV : NK;
        for (int j = max(issued[kv] - n, 0); j < issued[kv]; ++j)
          (void)mbar_wait_bounded(kv ? bar(sh.vfull[j % n]) : bar(sh.kfull[j % n]), (j / n) & 1, kDrainLimitNs);
      }
    }
  } else if (warp == 4) {
    // ================= MMA issuer (one elected lane) =================
    const uint32_t idesc_s = umma::idesc_bf16(kTreeRows, TILE, 0, 0);
    const uint32_t idesc_o = umma::idesc_bf16(kTreeRows, D, 0, 1);
    auto s_mma = [&](int n) {  // S(n) = Q K(n)^T into buffer n % 2
      if (!wait_use(sh.kfull[n % NK], n / NK)) return false;
      umma::fence_after();
      if (umma::elect()) {
        const uint32_t kst = k_s + (n % NK) * C::kKBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t ad = umma::desc_sw128(q_s + (kk >> 2) * C::kQPanelBytes + (kk & 3) * 32, 16, 1024);
          const uint64_t bd = umma::desc_sw128(kst + (kk >> 2) * C::kKVPanelBytes + (kk & 3) * 32, 16, 1024);
          umma::mma_f16(tmem + C::kSCol + (n & 1) * TILE, ad, bd, idesc_s, kk > 0 ? 1u : 0u);
        }
        umma::commit(bar(sh.sfull[n & 1]));
        umma::commit(bar(sh.kempty[n % NK]));
      }
      __syncwarp();
      return true;
    };
    auto o_mma = [&](int n, bool first) {  // O (+)= P V(n), P in the columns of S buffer n % 2
      if (!wait_use(sh.pready[n & 1], n >> 1) || *abort_flag) return false;
      if (!wait_use(sh.vfull[n % NV], n / NV)) return false;
      umma::fence_after();
      if (umma::elect()) {
        const uint32_t vst = v_s + (n % NV) * C::kKBytes;
        const uint32_t pcol = tmem + C::kSCol + (n & 1) * TILE;
#pragma unroll
        for (int k = 0; k < TILE / 16; ++k) {
          const uint64_t bd = umma::desc_sw128(vst + k * 16 * 128, C::kKVPanelBytes, 1024);
          umma::mma_f16_tmem_a(tmem + C::kOCol, pcol + k * 8, bd, idesc_o, (!first || k > 0) ? 1u : 0u);
        }
        umma::commit(bar(sh.odone[n & 1]));
        umma::commit(bar(sh.vempty[n % NV]));
      }
      __syncwarp();
      return true;
    };
    int q_issued = 0;  // Q loads issued, in the lane that issues them
    // S of a tile goes out before P V of the tile before, except where a piece
    // starts: its Q takes the place of the last piece's, so its first S waits
    // for that load, and P V of the tile before does not wait for it.
    bool ok = true, before_first = false;
    int n = 0;
    TreePiece c, nxt;
    bool more = walk.next(p, mt, nxt);
    for (int u = 0; ok && more; ++u) {
      c = nxt;
      for (int i = c.t0; ok && i < c.t1; ++i, ++n) {
        if (i == c.t0) {
          ok = n == 0 || wait_use(sh.sfull[(n - 1) & 1], (n - 1) >> 1);
          if (!ok) break;
          if (umma::elect()) {
            mbar_arrive_expect_tx(bar(sh.qfull), C::kPanels * p.q_nodes * G * 128);
            for (int k = 0; k < C::kPanels; ++k)
              tma_load_3d(q_s + k * C::kQPanelBytes, &qmap, bar(sh.qfull), k * 64, c.g * G,
                          c.b * p.tree_len + mt * p.q_nodes);
            q_issued = u + 1;
          }
          __syncwarp();
          ok = (n == 0 || o_mma(n - 1, before_first)) && wait_use(sh.qfull, u) && s_mma(n);
          more = ok && walk.next(p, mt, nxt);
        } else {
          ok = s_mma(n) && o_mma(n - 1, before_first);
        }
        before_first = i == c.t0;
      }
    }
    if (ok && n > 0) ok = o_mma(n - 1, before_first);
    if (!ok) give_up();
    if (!ok || *abort_flag) {  // the MMAs issued get a bounded time to finish before TMEM is freed
      if (umma::elect()) {
        umma::commit(bar(sh.drain));
        if (q_issued > 0) (void)mbar_wait_bounded(bar(sh.qfull), (q_issued - 1) & 1, kDrainLimitNs);
      }
      (void)mbar_wait_bounded(bar(sh.drain), 0, kDrainLimitNs);
    }
  } else {
    // ================= softmax warps 0-3: one query row per thread =================
    const int r = tid;  // TMEM lane = row
    const uint32_t lane_base = tmem + ((uint32_t)(32 * warp) << 16);
    const int row_stride = tree_row_stride(p);
    // Scores in the base-2 domain: x * xs, or the capped score
    // cap tanh(s / cap) log2 e = cap_a - cap_b / (1 + 2^(x cap_c)), since tanh y = 1 - 2 / (1 + e^(2 y)).
    const float xs_all = p.scale * kLog2e;
    const bool pre = p.use_softcap || !(xs_all > 0.f);  // scores computed ahead of the maximum
    const float xs = pre ? 1.f : xs_all;
    const float cap_a = p.softcap * kLog2e, cap_b = 2.f * cap_a;
    const float cap_c = p.use_softcap ? 2.f * xs_all / p.softcap : 0.f;

    TreePiece c, nxt;
    TreeRow row, row_nxt;
    const int node = mt * p.q_nodes + r / G;  // this thread's row: its node and its head
    const int64_t head = (int64_t)node * p.hq + r % G;
    bool ok = true, more = walk.next(p, mt, nxt);
    if (more) row_nxt = tree_row(p, nxt.s, nxt.b, node);
    int4 rec = make_int4(0, 0, 0, 0);
    int n = 0;
    for (int u = 0; ok && more; ++u) {
      c = nxt;
      row = row_nxt;
      const int rows = min(p.q_nodes, c.s.n - mt * p.q_nodes) * G;
      const bool real = r < rows, active = 32 * warp < rows;
      const int L = c.s.L, base = c.s.base;
      // Rows' windows start in [ulo, ulo + 63] (a depth is at most 63) and at most at base.
      const int w_end = p.window > 0 ? min(base, c.ulo + TILE - 1) : 0;
      uint64_t* bad = sh.bad[u % 3];
      float m = -CUDART_INF_F, l = 0.f;
      for (int i = c.t0; i < c.t1; ++i, ++n) {
        ok = wait_use(sh.sfull[n & 1], n >> 1);
        if (!ok || *abort_flag) break;
        umma::fence_after();
        const int kt = c.kt0 + i * TILE;
        const uint32_t skip = *const_cast<volatile uint32_t*>(&sh.skip[n & 15]);
        const bool edge = kt < w_end || kt + TILE > base;
        const bool masked = edge || kt < c.ulo || skip != 0;
        const uint32_t s_col = lane_base + C::kSCol + (n & 1) * TILE;
        if (active) {
          float x[TILE];
          {
            uint32_t w[TILE / 16][16];
#pragma unroll
            for (int k = 0; k < TILE / 16; ++k) umma::ld16_nowait(s_col + k * 16, w[k]);
            umma::wait_ld();
#pragma unroll
            for (int k = 0; k < TILE; ++k) x[k] = __uint_as_float(w[k / 16][k % 16]);
          }
          if (pre) {
            if (p.use_softcap) {
#pragma unroll
              for (int k = 0; k < TILE; ++k) {
                float e, q;
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x[k] * cap_c));
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.f + e));
                x[k] = fmaf(-cap_b, q, cap_a);
              }
            } else {
#pragma unroll
              for (int k = 0; k < TILE; ++k) x[k] *= xs_all;
            }
          }
          if (masked) {
            // Bit k: this row attends position kt + k.
            const int from = min(max(row.lo - kt, 0), TILE), to = min(max(base - kt, 0), TILE);
            uint64_t see = low_bits(to) & ~low_bits(from);
            if (kt >= base) see |= row.nodes >> (kt - base);
            else if (base - kt < TILE) see |= row.nodes << (base - kt);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if ((skip >> k) & 1u) see &= ~(0xffffull << (16 * k));
            const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
            for (int k = 0; k < TILE; ++k) x[k] = ((k < 32 ? lo >> k : hi >> (k - 32)) & 1u) ? x[k] : -CUDART_INF_F;
          }
          float mx[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx[k] = x[k];
#pragma unroll
          for (int k = 8; k < TILE; ++k) mx[k & 7] = fmaxf(mx[k & 7], x[k]);
          const float mt_ = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                  fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * xs;  // xs > 0
          // Lazy rescaling, as in the prefill: the reference m moves when the
          // tile's maximum exceeds it by more than 8 (base 2), so weights stay
          // below 256 and share the reference of the sum and of O.
          const float mn = (m == -CUDART_INF_F || mt_ > m + 8.f) ? mt_ : m;
          const float ref = mn == -CUDART_INF_F ? 0.f : mn;
          const float alpha = exp2f(m - ref);
          const bool moved = mn != m;
          m = mn;
          // Weights in fp32 for the sum, rounded to bf16 for the second product
          // (a relative 2^-8 at most on each weight, what the output's own
          // rounding allows; the tensor cores take both operands in one type).
          float ps[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[TILE / 2];
#pragma unroll
          for (int k = 0; k < TILE / 2; ++k) {
            float e0, e1;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(fmaf(x[2 * k], xs, -ref)));
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(fmaf(x[2 * k + 1], xs, -ref)));
            ps[k & 3] += e0 + e1;
            pk[k] = pack_bf16x2(e0, e1);
          }
          l = l * alpha + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
          umma::st16_nowait(s_col, *reinterpret_cast<uint32_t(*)[16]>(&pk[0]));
          umma::st16_nowait(s_col + 16, *reinterpret_cast<uint32_t(*)[16]>(&pk[16]));
          // (The first tile's P V overwrites O; rows that nobody reads move nothing.)
          if (i > c.t0 && __any_sync(FULL, moved && real)) {
            ok = wait_use(sh.odone[(n - 1) & 1], (n - 1) >> 1);
            if (!ok) break;
            umma::fence_after();
#pragma unroll 1
            for (int k = 0; k < D / 16; ++k) {
              float v[16];
              umma::ld16(lane_base + C::kOCol + k * 16, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] *= alpha;
              umma::st16(lane_base + C::kOCol + k * 16, v);
            }
          }
          umma::wait_st();
        }
        if (masked) {
          ok = wait_use(sh.vfull[n % NV], n / NV);
          if (!ok) break;
          const uint32_t vst = v_s + (n % NV) * C::kKBytes;
          constexpr int CPR = C::kPanels * 8;  // 16-byte chunks of a row
          auto chunk = [&](int idx) {          // row idx / CPR; where a row's chunks are does not matter
            const int k = idx / CPR, rem = idx % CPR;
            return vst + (rem >> 3) * C::kKVPanelBytes + k * 128 + ((rem & 7) << 4);
          };
          // Rows of V that no row attends: zero (they were not loaded, or hold what stands behind the end).
          uint64_t none = low_bits(min(max(c.ulo - kt, 0), TILE)) | ~low_bits(min(max(L - kt, 0), TILE));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if ((skip >> k) & 1u) none |= 0xffffull << (16 * k);
          if (none) {
            for (int idx = tid; idx < TILE * CPR; idx += 128)
              if ((none >> (idx / CPR)) & 1ull)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(chunk(idx)), "r"(0u) : "memory");
          }
          if (edge) {
            const int slot = kt + TILE > base ? 2 + (kt - (base & ~(TILE - 1))) / TILE : (kt - c.kt0) / TILE;
            constexpr int U = 4;
#pragma unroll 1
            for (int i0 = tid; i0 < TILE * CPR; i0 += 128 * U) {
              uint32_t w[U][4], top = 0;
#pragma unroll
              for (int e = 0; e < U; ++e)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[e][0]), "=r"(w[e][1]), "=r"(w[e][2]), "=r"(w[e][3])
                             : "r"(chunk(i0 + 128 * e)));
#pragma unroll
              for (int e = 0; e < U; ++e)
#pragma unroll
                for (int j = 0; j < 4; ++j) top = __vmaxu2(top, w[e][j] & 0x7f807f80u);
              // Exponent bits all set in some element: not finite.  (Rows just
              // zeroed by another thread may still read as what stood there.)
              if ((top & 0xffffu) != 0x7f80u && (top >> 16) != 0x7f80u) continue;
              for (int e = 0; e < U; ++e) {
                const int idx = i0 + 128 * e, k = idx / CPR;
                if ((none >> k) & 1ull) continue;
                bool found = false;
                for (int j = 0; j < 4; ++j) {
                  if ((w[e][j] & 0x7f80u) == 0x7f80u) w[e][j] &= 0xffff0000u, found = true;
                  if ((w[e][j] & 0x7f800000u) == 0x7f800000u) w[e][j] &= 0xffffu, found = true;
                }
                if (!found) continue;
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(chunk(idx)), "r"(w[e][0]),
                             "r"(w[e][1]), "r"(w[e][2]), "r"(w[e][3])
                             : "memory");
                atomicOr(reinterpret_cast<unsigned long long*>(&bad[slot]), 1ull << k);
              }
            }
          }
          fence_proxy_async_smem();  // visible to the tensor core's reads
        }
        // The next piece's marks, clear before any warp can be at that piece
        // and after every warp is past the piece that used them (three ago).
        if (i == c.t1 - 1 && tid < 4) sh.bad[(u + 1) % 3][tid] = 0;
        umma::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.pready[n & 1]));
        if (i == c.t0) {  // the next piece, while the tensor core is at this one
          more = walk.next(p, mt, nxt);
          if (more) row_nxt = tree_row(p, nxt.s, nxt.b, node);
        }
      }
      if (!ok || *abort_flag) break;

      // ---- write the piece's rows -------------------------------------------------------
      const bool begins = c.t0 == 0, ends = c.t1 == c.tiles;
      ok = wait_use(sh.odone[(n - 1) & 1], (n - 1) >> 1);
      if (!ok) break;
      umma::fence_after();
      uint64_t marks = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) marks |= *const_cast<volatile uint64_t*>(&bad[k]);
      const bool fin = begins && ends;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
      float* po = p.ws_o + (int64_t)slot * row_stride * D + r * 4;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) +
                            ((int64_t)c.b * p.tree_len * p.hq + (int64_t)c.g * G + head) * D;
      if (active) {
#pragma unroll 2
        for (int k = 0; k < D / 16; ++k) {
          float v[16];
          umma::ld16(lane_base + C::kOCol + k * 16, v);
          if (marks && real) {  // give back what was taken out of V, to a row that attends it
            for (int e = 0; e < 4; ++e) {
              uint64_t b = bad[e];
              const int kt = e < 2 ? c.kt0 + e * TILE : (base & ~(TILE - 1)) + (e - 2) * TILE;
              while (b) {
                const int t = kt + __ffsll((long long)b) - 1;
                b &= b - 1;
                if (t < base ? t < row.lo : !((row.nodes >> (t - base)) & 1ull)) continue;
                const int phys = p.block_tables[(int64_t)c.b * p.max_blocks + (t >> p.log2_bs)];
                const __nv_bfloat16* src =
                    static_cast<const __nv_bfloat16*>(p.v_cache) +
                    (((int64_t)phys * p.hkv + c.g) * p.block_size + (t & (p.block_size - 1))) * D + k * 16;
                for (int j = 0; j < 16; ++j) {
                  const float y = __bfloat162float(src[j]);
                  if (!isfinite(y)) v[j] += y;
                }
              }
            }
          }
          if (!real) continue;
          if (fin) {
            uint4 a, b;
            a.x = pack_bf16x2(v[0] * inv, v[1] * inv);
            a.y = pack_bf16x2(v[2] * inv, v[3] * inv);
            a.z = pack_bf16x2(v[4] * inv, v[5] * inv);
            a.w = pack_bf16x2(v[6] * inv, v[7] * inv);
            b.x = pack_bf16x2(v[8] * inv, v[9] * inv);
            b.y = pack_bf16x2(v[10] * inv, v[11] * inv);
            b.z = pack_bf16x2(v[12] * inv, v[13] * inv);
            b.w = pack_bf16x2(v[14] * inv, v[15] * inv);
            reinterpret_cast<uint4*>(orow + k * 16)[0] = a;
            reinterpret_cast<uint4*>(orow + k * 16)[1] = b;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float4*>(po + (int64_t)(k * 4 + e) * row_stride * 4) =
                  make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          }
        }
        if (real && !fin) *reinterpret_cast<float2*>(p.ws_ml + ((int64_t)slot * row_stride + r) * 2) = make_float2(m, l);
      }
      if (begins && !ends)  // goes on in the next ranges: joined by the combine
        rec = make_int4((int)((c.start + c.tiles - 1) / sh.per) - grp + 1, c.b, c.g, rows);
    }
    if (!ok) give_up();
    if (tid == 0) p.ws_rec[blockIdx.x] = ok && !*abort_flag ? rec : make_int4(0, 0, 0, 0);
  }
  // Every tcgen05 access is complete (waited); free the tensor memory.
  umma::fence_before();
  __syncthreads();
  if (warp == 0) {
    umma::fence_after();
    umma::dealloc(tmem, C::kTmemCols);
  }
}

// Joins the pieces of each unit that was cut: CTA blockIdx.x of the attention
// grid holds its first piece (slot 1) and says how many there are; the others
// are in slot 0 of the next CTAs of the same row tile.  With M = max m_p:
//   out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,
// in piece order.  blockIdx.y: 8 rows; a thread has four columns of one row,
// and neighbouring threads neighbouring rows, as the partials lie.
template <int D>
__global__ void __launch_bounds__(2 * D) tree_combine_kernel(const TreeParams p) {
  pdl_wait();  // the partials come from the attention grid
  const int c = blockIdx.x;
  const int4 rec = p.ws_rec[c];
  const int r = blockIdx.y * kTreeCombineRows + (threadIdx.x & (kTreeCombineRows - 1));
  const int col4 = threadIdx.x / kTreeCombineRows;
  if (rec.x == 0 || r >= rec.w) return;
  const int row_stride = tree_row_stride(p), G = p.group, node = c % p.m_tiles * p.q_nodes + r / G;
  auto slot = [&](int k) { return (int64_t)(k == 0 ? 2 * c + 1 : 2 * (c + k * p.m_tiles)); };
  float M = -CUDART_INF_F;
  for (int k = 0; k < rec.x; ++k) M = fmaxf(M, p.ws_ml[(slot(k) * row_stride + r) * 2]);
  const float ref = M == -CUDART_INF_F ? 0.f : M;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
#pragma unroll 4
  for (int k = 0; k < rec.x; ++k) {
    const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + (slot(k) * row_stride + r) * 2);
    const float4 o = *reinterpret_cast<const float4*>(p.ws_o + (slot(k) * (D / 4) + col4) * row_stride * 4 + r * 4);
    const float w = exp2f(ml.x - ref);
    den = fmaf(w, ml.y, den);
    acc.x = fmaf(w, o.x, acc.x);
    acc.y = fmaf(w, o.y, acc.y);
    acc.z = fmaf(w, o.z, acc.z);
    acc.w = fmaf(w, o.w, acc.w);
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;  // a row that attends nothing is zero
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) +
                       (((int64_t)rec.y * p.tree_len + node) * p.hq + (int64_t)rec.z * G + r % G) * D + col4 * 4;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace pa
