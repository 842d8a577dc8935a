// What the kernels of a drafted tree share: a sequence's lengths, a node's
// ancestors and the range it attends.
//
// Sequence b's tree has n nodes, whose rows are the last n of its L positions:
// node j at position base + j, base = L - n.  Bit i of node j's mask word says
// that j attends node i (itself included).  depth(j) is the number of nodes
// that j attends besides itself, and the logical position of j is
// p_j = base + depth(j): j attends the positions t < base and the nodes i of
// its mask, those with t, or p_i, above p_j - window where a window is set.
#pragma once

#include <stdint.h>

#include "decode_common.cuh"

namespace pa {

constexpr int kMaxTreeNodes = 64;  // one mask word

struct TreeParams {
  const void* q;                // [batch][tree_len][hq][D]
  void* out;                    // like q
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;  // [batch][max_blocks]
  const int32_t* context_lens;  // [batch], the tree's nodes included
  const int32_t* tree_lens;     // [batch], or null: tree_len nodes each
  const int64_t* tree_mask;     // [batch or 1][tree_len], rows mask_stride apart
  int64_t mask_stride;          // 0: every sequence has the same tree
  float* ws_o;                  // partials (decode_tree.cuh)
  float* ws_ml;
  int4* ws_rec;                 // one record per (range, row tile)
  int batch, tree_len, hq, hkv, group;
  int block_size, log2_bs, max_blocks, num_blocks;
  int log2_box;                 // rows of a K/V box: a block's, up to a tile's 64
  int window, max_context;
  int split;                    // CTAs of a cluster that share a range (decode_tree_simt.cuh)
  int q_nodes, m_tiles;         // nodes per row tile of at most 128 query rows, row tiles of a tree_len tree
  float scale, softcap;
  int use_softcap;
};

// A sequence's lengths.  n = 0: nothing to attend, all of its rows are zero
// (an empty sequence, L = 0, or lengths that do not fit, which raise
// PA_DEVERR_CONTEXT when `report`).
struct TreeSeq {
  int L, n, base;
};

__device__ __forceinline__ TreeSeq tree_fit(const TreeParams& p, int len, int nodes, bool report) {
  TreeSeq s;
  s.L = len;
  s.n = nodes;
  const int cap = min(p.max_context, p.max_blocks << p.log2_bs);
  if (s.L != 0 && (s.L < 0 || s.L > cap || s.n < 0 || s.n > p.tree_len || s.L < s.n)) {
    if (report) raise_error(PA_DEVERR_CONTEXT);
    s.L = 0;
  }
  if (s.L == 0) s.n = 0;
  s.base = s.L - s.n;
  return s;
}

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b, bool report) {
  return tree_fit(p, p.context_lens[b], p.tree_lens ? p.tree_lens[b] : p.tree_len, report);
}

// First position that any node of the tree may attend (the root's window start).
__device__ __forceinline__ int tree_start(const TreeSeq& s, int window) {
  return window > 0 ? max(0, s.base + 1 - window) : 0;
}

__device__ __forceinline__ uint64_t low_bits(int n) { return n >= 64 ? ~0ull : (1ull << n) - 1; }

__device__ __forceinline__ int tree_depth(const int64_t* mask, int j, int n) {
  return __popcll((uint64_t)mask[j] & low_bits(n) & ~(1ull << j));
}

// What node j attends: the positions [lo, base) and the nodes of `nodes`.
struct TreeRow {
  int lo;
  uint64_t nodes;
};

// Node j's mask word as it lies in memory (0 for a node that the tree does not have).
__device__ __forceinline__ uint64_t tree_word(const TreeParams& p, int b, int n, int j) {
  return j < n ? (uint64_t)p.tree_mask[b * p.mask_stride + j] : 0ull;
}

__device__ __forceinline__ TreeRow tree_row(const TreeParams& p, const TreeSeq& s, int b, int j, uint64_t word) {
  TreeRow r;
  if (j >= s.n) {
    r.lo = s.base;
    r.nodes = 0;
    return r;
  }
  r.nodes = word & low_bits(s.n);
  r.lo = 0;
  if (p.window > 0) {
    const int depth = __popcll(r.nodes & ~(1ull << j));
    r.lo = max(0, s.base + 1 - p.window + depth);
    if (r.lo > s.base) r.lo = s.base;
    if (p.window < kMaxTreeNodes) {  // a depth is below kMaxTreeNodes: wider windows reach every node
      const int64_t* mask = p.tree_mask + b * p.mask_stride;
      for (int i = 0; i < s.n; ++i)
        if (tree_depth(mask, i, s.n) + p.window <= depth) r.nodes &= ~(1ull << i);
    }
  }
  return r;
}

}  // namespace pa
