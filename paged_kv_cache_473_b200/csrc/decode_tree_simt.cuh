// Attention of a drafted tree over the paged cache on CUDA cores (fp32 caches).
//
// One CTA per (RT query rows, kv head, sequence): row r = (node r / G, head
// r % G) of the kv head's n * G rows.  D / 8 neighbouring lanes, 8 dims each, are a
// worker that takes a token at a time, every kWorkers-th of the attended range, with
// its own softmax state of the RT rows; the next token's key and value are
// loaded while it works on this one.  A dot product is 8 multiply-adds a lane and a
// shuffle over the worker's lanes, a key and value read serves RT rows, and the
// workers' states are joined once, at the end.  Which rows attend a token is
// the same for a worker's lanes, so a masked weight is skipped, not multiplied by
// zero: what stands in a masked place (a NaN, an infinity) reaches no row.
// fp32 caches serve checks and small models; the bf16 kernel is decode_tree.cuh.
#pragma once

#include "decode_tree_common.cuh"
#include "ptx.cuh"

namespace pa {

// Eight consecutive elements of a row.
struct Row8 {
  float4 a, b;
  __device__ __forceinline__ void load(const float* src) {
    a = reinterpret_cast<const float4*>(src)[0];
    b = reinterpret_cast<const float4*>(src)[1];
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

constexpr int kTreeSimtRows = 8;
constexpr int kTreeSimtWarps = 4;

template <int D>
__global__ void __launch_bounds__(kTreeSimtWarps * 32, 2) decode_tree_simt_kernel(const TreeParams p) {
  constexpr int RT = kTreeSimtRows, LPW = D / 8;          // lanes of a worker
  constexpr int kWorkers = kTreeSimtWarps * 32 / LPW;     // of the CTA
  constexpr uint32_t FULL = 0xffffffffu;
  __shared__ TreeRow row[RT];
  __shared__ float sm[kTreeSimtWarps][RT], sl[kTreeSimtWarps][RT];
  __shared__ float so[kTreeSimtWarps][RT][D];

  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int worker = tid / LPW, ch = tid % LPW;
  const int r0 = blockIdx.x * RT, g = blockIdx.y, b = blockIdx.z, G = p.group;
  const TreeSeq s = tree_seq(p, b, blockIdx.x == 0 && g == 0 && tid == 0);
  const int all_rows = p.tree_len * G, rows = s.n * G;
  auto out_row = [&](int r) {  // row r of the kv head, in q and out
    return (((int64_t)b * p.tree_len + r / G) * p.hq + (int64_t)g * G + r % G) * D;
  };
  float* out = static_cast<float*>(p.out);
  if (r0 >= rows) {  // no node in this tile: zero rows
    for (int i = tid; i < RT * D; i += kTreeSimtWarps * 32)
      if (r0 + i / D < all_rows) out[out_row(r0 + i / D) + i % D] = 0.f;
    return;
  }
  if (tid < RT) {
    const int node = r0 + tid < rows ? (r0 + tid) / G : s.n;
    row[tid] = tree_row(p, s, b, node, tree_word(p, b, s.n, node));
  }
  float q[RT][8], m[RT], l[RT], o[RT][8];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = -CUDART_INF_F;
    l[r] = 0.f;
    Row8 x;
    x.a = x.b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < rows) x.load(static_cast<const float*>(p.q) + out_row(r0 + r) + ch * 8);
    x.widen(q[r]);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[r][e] = 0.f;
  }
  __syncthreads();
  int lo = s.base;
#pragma unroll
  for (int r = 0; r < RT; ++r) lo = min(lo, row[r].lo);

  const float qk_scale = p.use_softcap ? p.scale : p.scale * kLog2e;
  const float inv_cap = p.use_softcap ? 1.f / p.softcap : 0.f;
  const int32_t* table = p.block_tables + (int64_t)b * p.max_blocks;
  const float* kc = static_cast<const float*>(p.k_cache);
  const float* vc = static_cast<const float*>(p.v_cache);
  // Rows that attend token t, and its key and value (zero when none does).
  auto fetch = [&](int t, Row8& k, Row8& v) -> uint32_t {
    uint32_t sees = 0;
    if (t < s.L) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
        sees |= (t < s.base ? (uint32_t)(t >= row[r].lo) : (uint32_t)(row[r].nodes >> (t - s.base)) & 1u) << r;
    }
    if (sees) {
      const int phys = table[t >> p.log2_bs];
      if (phys >= 0 && phys < p.num_blocks) {
        const int64_t at = (((int64_t)phys * p.hkv + g) * p.block_size + (t & (p.block_size - 1))) * D + ch * 8;
        k.load(kc + at);
        v.load(vc + at);
      } else {
        if (ch == 0) raise_error(PA_DEVERR_BLOCK);
        sees = 0;
      }
    }
    if (!sees) k.a = k.b = v.a = v.b = make_float4(0.f, 0.f, 0.f, 0.f);
    return sees;
  };
  Row8 k0, v0, k1, v1;
  uint32_t sees = fetch(lo + worker, k0, v0);
  // Every lane makes the same number of turns (the shuffles are warp-wide).
  for (int t0 = lo; t0 < s.L; t0 += kWorkers) {
    const uint32_t next = fetch(t0 + kWorkers + worker, k1, v1);
    float kx[8], vx[8];
    k0.widen(kx);
    v0.widen(vx);
    float x[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      x[r] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[r] = fmaf(q[r][e], kx[e], x[r]);
    }
#pragma unroll
    for (int off = LPW / 2; off > 0; off >>= 1)
#pragma unroll
      for (int r = 0; r < RT; ++r) x[r] += __shfl_xor_sync(FULL, x[r], off);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float y = x[r] * qk_scale;
      if (p.use_softcap) y = p.softcap * tanhf(y * inv_cap) * kLog2e;
      if (!((sees >> r) & 1u)) continue;
      if (y > m[r]) {  // the reference moves (a NaN does not move it: its weight is one)
        const float al = exp2f(m[r] - y);
        m[r] = y;
        l[r] *= al;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[r][e] *= al;
      }
      const float w = exp2f(y - (m[r] == -CUDART_INF_F ? 0.f : m[r]));
      l[r] += w;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[r][e] = fmaf(w, vx[e], o[r][e]);
    }
    k0 = k1;
    v0 = v1;
    sees = next;
  }

  // ---- join the workers: those of a warp by shuffles, the warps through shared memory ---------
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int off = LPW; off < 32; off <<= 1) {
      const float mo = __shfl_xor_sync(FULL, m[r], off), lo_ = __shfl_xor_sync(FULL, l[r], off);
      const float M = fmaxf(m[r], mo), ref = M == -CUDART_INF_F ? 0.f : M;
      const float c0 = exp2f(m[r] - ref), c1 = exp2f(mo - ref);
      m[r] = M;
      l[r] = c0 * l[r] + c1 * lo_;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[r][e] = c0 * o[r][e] + c1 * __shfl_xor_sync(FULL, o[r][e], off);
    }
    if (lane < LPW) {
      if (lane == 0) sm[warp][r] = m[r], sl[warp][r] = l[r];
#pragma unroll
      for (int e = 0; e < 8; ++e) so[warp][r][ch * 8 + e] = o[r][e];
    }
  }
  __syncthreads();
  for (int i = tid; i < RT * D; i += kTreeSimtWarps * 32) {
    const int r = i / D, d = i % D;
    if (r0 + r >= all_rows) break;
    float M = -CUDART_INF_F, num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kTreeSimtWarps; ++w) M = fmaxf(M, sm[w][r]);
    const float ref = M == -CUDART_INF_F ? 0.f : M;
#pragma unroll
    for (int w = 0; w < kTreeSimtWarps; ++w) {
      const float c = exp2f(sm[w][r] - ref);
      num += c * so[w][r][d];
      den += c * sl[w][r];
    }
    // den = 0: the row attends nothing (its sums are zero); a NaN stays one.
    out[out_row(r0 + r) + d] = den == 0.f ? 0.f : num / den;
  }
}

}  // namespace pa
