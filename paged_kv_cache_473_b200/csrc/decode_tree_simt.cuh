// Attention of a drafted tree over the paged cache on CUDA cores (fp32 caches).
//
// One CTA per (RT query rows, kv head, sequence): row r = (node r / G, head
// r % G) of the kv head's n * G rows.  As in the CUDA-core decode kernel, warp
// w takes every NW-th 16-token slice of the attended range, each lane owns
// D / 32 consecutive dims, reads the matching dims of a K and a V row with one
// vector load and the warp sums the partial dot products with shuffles; every
// key and value read serves the CTA's RT rows.  Which rows attend a position is
// the same for all lanes, so a masked weight is skipped, not multiplied by
// zero: what stands in a masked place (a NaN, an infinity) reaches no row.
// fp32 caches serve checks and small models; the bf16 kernel is decode_tree.cuh.
#pragma once

#include "decode_simt.cuh"
#include "decode_tree_common.cuh"

namespace pa {

constexpr int kTreeSimtRows = 8;
constexpr int kTreeSimtWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kTreeSimtWarps * 32) decode_tree_simt_kernel(const TreeParams p) {
  constexpr int VEC = D / 32, RT = kTreeSimtRows, NW = kTreeSimtWarps;
  constexpr int U = 2;  // tokens per inner step
  constexpr uint32_t FULL = 0xffffffffu;
  __shared__ int row_lo[RT];
  __shared__ uint64_t row_nodes[RT];
  __shared__ float sm[NW][RT], sl[NW][RT];
  extern __shared__ __align__(16) float so[];  // [NW][RT][D]

  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * RT, g = blockIdx.y, b = blockIdx.z, G = p.group;
  const TreeSeq s = tree_seq(p, b, blockIdx.x == 0 && g == 0 && tid == 0);
  const int all_rows = p.tree_len * G, rows = s.n * G;
  auto out_row = [&](int r) {  // row r of the kv head, in q and out
    return (((int64_t)b * p.tree_len + r / G) * p.hq + (int64_t)g * G + r % G) * D;
  };
  if (r0 >= rows) {  // no node in this tile: zero rows
    for (int i = tid; i < RT * D; i += NW * 32)
      if (r0 + i / D < all_rows) store_out<T>(static_cast<T*>(p.out) + out_row(r0 + i / D) + i % D, 0.f);
    return;
  }
  if (tid < RT) {
    TreeRow t;
    t.lo = s.base;
    t.nodes = 0;
    if (r0 + tid < rows) t = tree_row(p, s, b, (r0 + tid) / G);
    row_lo[tid] = t.lo;
    row_nodes[tid] = t.nodes;
  }
  __syncthreads();
  int lo = s.base;
#pragma unroll
  for (int r = 0; r < RT; ++r) lo = min(lo, row_lo[r]);

  float q[RT][VEC], m[RT], l[RT], o[RT][VEC];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = -CUDART_INF_F;
    l[r] = 0.f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) q[r][v] = o[r][v] = 0.f;
    if (r0 + r < rows) VecLoad<T, VEC>::load(static_cast<const T*>(p.q) + out_row(r0 + r) + lane * VEC, q[r]);
  }

  const float qk_scale = p.use_softcap ? p.scale : p.scale * kLog2e;
  const float inv_cap = p.use_softcap ? 1.f / p.softcap : 0.f;
  const int32_t* table = p.block_tables + (int64_t)b * p.max_blocks;
  const T* kc = static_cast<const T*>(p.k_cache);
  const T* vc = static_cast<const T*>(p.v_cache);
  for (int j = lo / kSliceTokens + warp; j * kSliceTokens < s.L; j += NW) {
    const int t0 = j * kSliceTokens;
    const int phys = table[t0 >> p.log2_bs];
    if (phys < 0 || phys >= p.num_blocks) {
      if (lane == 0) raise_error(PA_DEVERR_BLOCK);
      continue;
    }
    const int64_t row0 = ((int64_t)phys * p.hkv + g) * p.block_size + (t0 & (p.block_size - 1));
    for (int u0 = 0; u0 < kSliceTokens; u0 += U) {
      float kr[U][VEC], vr[U][VEC];
      uint32_t sees[U];  // rows that attend the token
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u0 + u;
        sees[u] = 0;
        if (t >= lo && t < s.L) {
#pragma unroll
          for (int r = 0; r < RT; ++r)
            sees[u] |= (t < s.base ? (uint32_t)(t >= row_lo[r]) : (uint32_t)(row_nodes[r] >> (t - s.base)) & 1u) << r;
        }
        if (sees[u]) {
          VecLoad<T, VEC>::load(kc + (row0 + u0 + u) * D + lane * VEC, kr[u]);
          VecLoad<T, VEC>::load(vc + (row0 + u0 + u) * D + lane * VEC, vr[u]);
        } else {
#pragma unroll
          for (int v = 0; v < VEC; ++v) kr[u][v] = vr[u][v] = 0.f;
        }
      }
      float x[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float acc = 0.f;
#pragma unroll
          for (int v = 0; v < VEC; ++v) acc = fmaf(q[r][v], kr[u][v], acc);
          x[u][r] = acc;
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int r = 0; r < RT; ++r) x[u][r] += __shfl_xor_sync(FULL, x[u][r], off);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float mx = m[r];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float y = x[u][r] * qk_scale;
          if (p.use_softcap) y = p.softcap * tanhf(y * inv_cap) * kLog2e;
          x[u][r] = y;
          if ((sees[u] >> r) & 1u) mx = fmaxf(mx, y);
        }
        const float ref = mx == -CUDART_INF_F ? 0.f : mx;
        const float al = exp2f(m[r] - ref);
        m[r] = mx;
        l[r] *= al;
#pragma unroll
        for (int v = 0; v < VEC; ++v) o[r][v] *= al;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (!((sees[u] >> r) & 1u)) continue;
          const float pw = exp2f(x[u][r] - ref);
          l[r] += pw;
#pragma unroll
          for (int v = 0; v < VEC; ++v) o[r][v] = fmaf(pw, vr[u][v], o[r][v]);
        }
      }
    }
  }

  // ---- join the warps' states, write the rows ---------------------------------------------
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (lane == 0) {
      sm[warp][r] = m[r];
      sl[warp][r] = l[r];
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) so[(warp * RT + r) * D + lane * VEC + v] = o[r][v];
  }
  __syncthreads();
  for (int i = tid; i < RT * D; i += NW * 32) {
    const int r = i / D, d = i % D;
    if (r0 + r >= all_rows) break;
    float M = -CUDART_INF_F, num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, sm[w][r]);
    const float ref = M == -CUDART_INF_F ? 0.f : M;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float c = exp2f(sm[w][r] - ref);
      num += c * so[(w * RT + r) * D + d];
      den += c * sl[w][r];
    }
    // den = 0: the row attends nothing (its sums are zero); a NaN stays one.
    store_out<T>(static_cast<T*>(p.out) + out_row(r0 + r) + d, den == 0.f ? 0.f : num / den);
  }
}

}  // namespace pa
