// Move the rows of an accepted path to the places it ends up in: node path[i]
// of sequence b's tree, at position base + path[i], becomes position base + i,
// in the key and the value cache of every layer; new_lens[b] = base + (number
// of accepted nodes), base = context_lens[b] - (nodes of b's tree).
//
// One CTA takes a sequence and up to kCommitThreads of the 16-byte chunks that
// make up one token in all layers (layer, K or V, kv head, chunk); a thread
// moves its chunk of every path row, in path order.  A path is strictly
// increasing, so path[i] >= i: no place i is the source of a later row, and a
// thread that loads some rows before it stores them, in order, overwrites
// nothing that it has yet to read.  Threads share nothing but the path.
// A few rows a sequence: the time is the chain of dependent loads (lengths and
// path, block ids, rows), each a trip to L2 or DRAM, and the launch.
#pragma once

#include "decode_common.cuh"
#include "decode_tree_common.cuh"
#include "ptx.cuh"

namespace pa {

constexpr int kCommitThreads = 128;

struct CommitParams {
  uint4 *k_cache, *v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* tree_lens;   // or null: tree_len nodes each
  const int32_t* accepted;    // [batch][max_accept]
  const int32_t* accept_lens;
  int32_t* new_lens;          // or null
  int64_t layer_chunks;       // 16-byte chunks of one layer's K (or V) cache
  int layers, hkv, chunks_per_row;
  int max_accept, tree_len;
  int log2_bs, max_blocks, num_blocks;
};

__global__ void __launch_bounds__(kCommitThreads) commit_tree_kernel(const CommitParams p) {
  __shared__ int src[kMaxTreeNodes], dst[kMaxTreeNodes];  // rows as slots, -1: no move
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.y, tid = threadIdx.x;
  const bool first = blockIdx.x == 0;
  const int L = p.context_lens[b];
  const int a = p.accept_lens[b];
  const int n = p.tree_lens ? p.tree_lens[b] : p.tree_len;
  const int cap = p.max_blocks << p.log2_bs;
  const int base = L - n;
  // L = 0: an empty (padding) sequence, nothing else of which is looked at.
  bool bad = L != 0 && (L < 0 || L > cap || n < 0 || n > p.tree_len || base < 0 || a < 0 || a > min(p.max_accept, n));
  if (!bad && L > 0 && tid < a) {
    const int32_t* path = p.accepted + (int64_t)b * p.max_accept;
    const int node = path[tid], before = tid ? path[tid - 1] : -1;
    int s = -1, d = -1;
    if (node <= before || node >= n) {
      bad = true;
    } else if (node != tid) {
      const int32_t* table = p.block_tables + (int64_t)b * p.max_blocks;
      const int mask = (1 << p.log2_bs) - 1, from = base + node, to = base + tid;
      const int fb = table[from >> p.log2_bs], tb = table[to >> p.log2_bs];
      if (fb >= 0 && fb < p.num_blocks && tb >= 0 && tb < p.num_blocks) {
        s = (fb << p.log2_bs) | (from & mask);
        d = (tb << p.log2_bs) | (to & mask);
      } else if (first) {
        raise_error(PA_DEVERR_BLOCK);
      }
    }
    src[tid] = s;
    dst[tid] = d;
  }
  bad = __syncthreads_or(bad);
  if (first && tid == 0) {
    if (bad) raise_error(PA_DEVERR_CONTEXT);
    if (p.new_lens) p.new_lens[b] = bad || L == 0 ? L : base + a;
  }
  if (bad || L == 0) return;

  const int64_t c = (int64_t)blockIdx.x * kCommitThreads + tid;
  const int per_head = p.chunks_per_row, per_cache = per_head * p.hkv;
  if (c >= (int64_t)p.layers * 2 * per_cache) return;
  const int64_t layer = c / (2 * per_cache);
  const int rem = (int)(c - layer * 2 * per_cache);
  const int in_cache = rem % per_cache, h = in_cache / per_head, part = in_cache % per_head;
  uint4* cache = (rem < per_cache ? p.k_cache : p.v_cache) + layer * p.layer_chunks;
  const int bs_mask = (1 << p.log2_bs) - 1;
  auto row = [&](int slot) {
    return cache + ((((int64_t)(slot >> p.log2_bs) * p.hkv + h) << p.log2_bs) + (slot & bs_mask)) * per_head + part;
  };
  constexpr int U = 8;  // rows in flight
  for (int i0 = 0; i0 < a; i0 += U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < a && src[i0 + u] >= 0) x[u] = *row(src[i0 + u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < a && src[i0 + u] >= 0) *row(dst[i0 + u]) = x[u];
  }
}

}  // namespace pa
