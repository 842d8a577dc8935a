// Attention of a drafted tree over the paged cache on CUDA cores (fp32 caches).
//
// A cluster of up to 8 CTAs per (RT query rows, kv head, sequence): row r = (node
// r / G, head r % G) of the kv head's n * G rows.  D / 8 neighbouring lanes, 8 dims
// each, are a worker that takes two tokens at a time, every (workers of the
// cluster)-th pair of the attended range; the next pair's keys are asked for when
// this one's are used up, and so are its values.  The 2 RT dot products of a pair
// are summed over the worker's lanes by halving what a lane holds at each
// shuffle, so that a lane ends with one row of one token (two tokens' at D = 64),
// whose row's running maximum and sum it keeps: one exponential a lane, and the
// weights go back by shuffles.  The workers' states are joined once, at the end,
// those of a warp by shuffles, the others through the cluster's shared memory.
// Which rows attend a token is the same for a worker's lanes, so a masked weight
// is skipped, not multiplied by zero: what stands in a masked place (a NaN, an
// infinity) reaches no row.
// Issue and latency of the ~190 instructions that a pair's half costs bound it, not
// bytes (B200: 63 nodes x 4 heads on 1.8K tokens of 8 kv heads, D = 128: 122 us,
// a fifth of the rate of the multiply-adds alone).  A token at a time costs 134 us;
// 4 rows a worker on twice the warps 164; row tiles of one CTA that share their
// tokens through the L1 124 there, and 1.2 - 1.4x as much where there are few rows.
// fp32 caches serve checks and small models; the bf16 kernel is decode_tree.cuh.
#pragma once

#include "decode_tree_common.cuh"
#include "ptx.cuh"

namespace pa {

constexpr int kTreeSimtRows = 8;
constexpr int kTreeSimtWarps = 4;
constexpr int kTreeSimtCluster = 8;  // CTAs that share a range at most (what every device takes)

// A lane's eight elements of a row, in pairs: four of each half, so that
// neighbouring lanes read neighbouring 16 bytes.
template <int D>
struct Row8 {
  float2 x[4];
  __device__ __forceinline__ void load(const float* src) {
    const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + D / 2);
    x[0] = make_float2(a.x, a.y), x[1] = make_float2(a.z, a.w);
    x[2] = make_float2(b.x, b.y), x[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void zero() { x[0] = x[1] = x[2] = x[3] = make_float2(0.f, 0.f); }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();  // the aligned forms take a warp as a whole
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What lies at `p` of this CTA's shared memory in that of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ float cluster_load(const float* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_load4(const float* p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr(p, rank))
               : "memory");
  return v;
}

template <int D>
__global__ void __launch_bounds__(kTreeSimtWarps * 32, 2) decode_tree_simt_kernel(const TreeParams p) {
  constexpr int RT = kTreeSimtRows, LPW = D / 8;          // lanes of a worker
  constexpr int kThreads = kTreeSimtWarps * 32, kWorkers = kThreads / LPW;
  constexpr uint32_t FULL = 0xffffffffu;
  static_assert(RT == 8 && LPW >= RT, "a lane for each row");
  __shared__ TreeRow row[RT];
  __shared__ float sm[kTreeSimtWarps][RT], sl[kTreeSimtWarps][RT];
  __shared__ alignas(16) float so[kTreeSimtWarps][RT][D];
  // The join: a state (CTA, warp) of each row's, and what it weighs there.
  __shared__ float jm[kTreeSimtCluster * kTreeSimtWarps * RT], jl[kTreeSimtCluster * kTreeSimtWarps * RT];

  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = p.split, rank = split > 1 ? (int)cluster_rank() : 0;
  const int worker = tid / LPW, ch = tid % LPW;
  const int g = blockIdx.y, b = blockIdx.z, G = p.group;
  const int r0 = blockIdx.x / split * RT;  // the CTA's first row
  const TreeSeq s = tree_seq(p, b, blockIdx.x == 0 && g == 0 && tid == 0);
  const int all_rows = p.tree_len * G, rows = s.n * G;
  auto out_row = [&](int r) {  // row r of the kv head, in q and out
    return (((int64_t)b * p.tree_len + r / G) * p.hq + (int64_t)g * G + r % G) * D;
  };
  float* out = static_cast<float*>(p.out);
  if (r0 >= rows) {  // no node in these rows: zero (for the whole cluster)
    for (int i = rank * kThreads + tid; i < RT * D; i += split * kThreads)
      if (r0 + i / D < all_rows) out[out_row(r0 + i / D) + i % D] = 0.f;
    return;
  }
  if (tid < RT) {
    const int node = r0 + tid < rows ? (r0 + tid) / G : s.n;
    row[tid] = tree_row(p, s, b, node, tree_word(p, b, s.n, node));
  }
  Row8<D> q[RT], o[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    q[r].zero();
    o[r].zero();
    if (r0 + r < rows) q[r].load(static_cast<const float*>(p.q) + out_row(r0 + r) + ch * 4);
  }
  const int mine = ch % RT;  // the row whose maximum and sum the lane keeps
  float m = -CUDART_INF_F, l = 0.f;
  __syncthreads();
  const int live = min(RT, rows - r0);  // rows of the tile that are nodes'
  int lo = s.base, whole = 0;           // positions [whole, base): every live row attends them
  for (int r = 0; r < live; ++r) {
    lo = min(lo, row[r].lo);
    whole = max(whole, row[r].lo);
  }

  const float qk_scale = p.use_softcap ? p.scale : p.scale * kLog2e;
  const float inv_cap = p.use_softcap ? 1.f / p.softcap : 0.f;
  const int32_t* table = p.block_tables + (int64_t)b * p.max_blocks;
  const float* kc = static_cast<const float*>(p.k_cache);
  const float* vc = static_cast<const float*>(p.v_cache);
  const int step = 2 * split * kWorkers;  // tokens between two of a worker's pairs
  const uint32_t full = (1u << live) - 1;
  // Rows that attend token t of block `phys`.
  auto attended = [&](int t, int phys) -> uint32_t {
    uint32_t sees = 0;
    if (t >= whole && t < s.base) {
      sees = full;
    } else if (t < s.L) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
        sees |= (t < s.base ? (uint32_t)(t >= row[r].lo) : (uint32_t)(row[r].nodes >> (t - s.base)) & 1u) << r;
    }
    if (sees && (phys < 0 || phys >= p.num_blocks)) {
      if (ch == 0) raise_error(PA_DEVERR_BLOCK);
      sees = 0;
    }
    return sees;
  };
  auto block = [&](int t) { return t < s.L ? table[t >> p.log2_bs] : 0; };
  // A pair of tokens: where they lie (asked for a pair ahead), who attends them, their keys and values.
  uint32_t sees[2], ahead[2];
  int phys[2];
  int64_t at_ahead[2];
  Row8<D> k[2], v[2];
  auto locate = [&](int t) {  // from phys[]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ahead[i] = attended(t + i, phys[i]);
      at_ahead[i] = (((int64_t)phys[i] * p.hkv + g) * p.block_size + ((t + i) & (p.block_size - 1))) * D + ch * 4;
    }
  };
  auto load = [&](Row8<D>(&x)[2], const float* cache, const uint32_t(&who)[2], const int64_t(&where)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (who[i])
        x[i].load(cache + where[i]);
      else
        x[i].zero();
    }
  };
  const int first = lo + 2 * rank * kWorkers, own = 2 * worker;
  phys[0] = block(first + own), phys[1] = block(first + own + 1);
  locate(first + own);
  load(k, kc, ahead, at_ahead);
  load(v, vc, ahead, at_ahead);
  phys[0] = block(first + step + own), phys[1] = block(first + step + own + 1);
  // Every lane of a warp makes the same number of turns (the shuffles are warp-wide).
#pragma unroll 1
  for (int t0 = first; t0 < s.L; t0 += step) {
    sees[0] = ahead[0], sees[1] = ahead[1];
    float x[2][RT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float2 a = mul_f32x2(q[r].x[0], k[i].x[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) a = fma_f32x2(q[r].x[e], k[i].x[e], a);
        x[i][r] = a.x + a.y;
      }
    locate(t0 + step + own);
    load(k, kc, ahead, at_ahead);
    phys[0] = block(t0 + 2 * step + own), phys[1] = block(t0 + 2 * step + own + 1);
    // Sum over the lanes, halving what a lane holds: the pair (16 lanes or more), then the rows.
    constexpr int kHeld = LPW >= 16 ? 1 : 2;  // tokens of the pair whose weight a lane makes
    if (kHeld == 1) {
      const bool up = (ch & 8) != 0;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float give = up ? x[0][r] : x[1][r], keep = up ? x[1][r] : x[0][r];
        x[0][r] = keep + __shfl_xor_sync(FULL, give, 8);
      }
    }
#pragma unroll
    for (int half = RT / 2; half > 0; half >>= 1)
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
#pragma unroll
        for (int r = 0; r < half; ++r) {
          const bool up = (ch & half) != 0;
          const float give = up ? x[i][r] : x[i][r + half], keep = up ? x[i][r + half] : x[i][r];
          x[i][r] = keep + __shfl_xor_sync(FULL, give, half);
        }
    if (LPW == 32) x[0][0] += __shfl_xor_sync(FULL, x[0][0], 16);
    float y[kHeld], top = -CUDART_INF_F;
    bool on[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      on[i] = ((kHeld == 1 && (ch & 8) ? sees[1] : sees[i]) >> mine) & 1u;
      y[i] = x[i][0] * qk_scale;
      if (p.use_softcap) y[i] = p.softcap * tanhf(y[i] * inv_cap) * kLog2e;
      if (on[i]) top = fmaxf(top, y[i]);  // (a NaN is not a maximum: its weight is one)
    }
    if (kHeld == 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, 8));
    const bool moved = top > m;
    if (__any_sync(FULL, moved)) {
      const float al = moved ? exp2f(m - top) : 1.f;
      if (moved) m = top;
      l *= al;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float a = __shfl_sync(FULL, al, (lane & ~(LPW - 1)) | r);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r].x[e] = mul_f32x2(o[r].x[e], make_float2(a, a));
      }
    }
    float w[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      w[i] = on[i] ? exp2f(y[i] - (m == -CUDART_INF_F ? 0.f : m)) : 0.f;
      l += w[i];
    }
    auto weight = [&](int i, int r) {
      return __shfl_sync(FULL, w[kHeld == 1 ? 0 : i], (lane & ~(LPW - 1)) | r | (kHeld == 1 ? 8 * i : 0));
    };
    if (__all_sync(FULL, sees[0] == full && sees[1] == full)) {
      // (rows behind the live ones have no weight and are not written from o)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = weight(i, r);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[r].x[e] = fma_f32x2(make_float2(a, a), v[i].x[e], o[r].x[e]);
        }
    } else {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = weight(i, r);
          if ((sees[i] >> r) & 1u) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r].x[e] = fma_f32x2(make_float2(a, a), v[i].x[e], o[r].x[e]);
          }
        }
    }
    load(v, vc, ahead, at_ahead);
  }
  if (LPW >= 16) l += __shfl_xor_sync(FULL, l, 8);

  // ---- join the workers: those of a warp by shuffles, the others through shared memory ---------
  {
    float M = m;
#pragma unroll
    for (int off = LPW; off < 32; off <<= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, off));
    const float c = exp2f(m - (M == -CUDART_INF_F ? 0.f : M));
    l *= c;
#pragma unroll
    for (int off = LPW; off < 32; off <<= 1) l += __shfl_xor_sync(FULL, l, off);
    if (lane < RT) sm[warp][mine] = M, sl[warp][mine] = l;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float a = __shfl_sync(FULL, c, (lane & ~(LPW - 1)) | r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 v = mul_f32x2(o[r].x[e], make_float2(a, a));
#pragma unroll
        for (int off = LPW; off < 32; off <<= 1) {
          v.x += __shfl_xor_sync(FULL, v.x, off);
          v.y += __shfl_xor_sync(FULL, v.y, off);
        }
        if (lane < LPW) *reinterpret_cast<float2*>(&so[warp][r][e / 2 * (D / 2) + ch * 4 + e % 2 * 2]) = v;
      }
    }
  }
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  const int states = split * kTreeSimtWarps;  // of each row; state j of row r at [r * states + j]
  for (int i = tid; i < RT * states; i += kThreads) {
    const int r = i / states, j = i % states;
    jm[i] = cluster_load(&sm[j % kTreeSimtWarps][r], j / kTreeSimtWarps);
    jl[i] = cluster_load(&sl[j % kTreeSimtWarps][r], j / kTreeSimtWarps);
  }
  __syncthreads();
  if (tid < RT) {
    float M = -CUDART_INF_F, den = 0.f;
    for (int j = 0; j < states; ++j) M = fmaxf(M, jm[tid * states + j]);
    if (M == -CUDART_INF_F) M = 0.f;
    for (int j = 0; j < states; ++j) {
      const float f = exp2f(jm[tid * states + j] - M);
      jm[tid * states + j] = f;
      den += f * jl[tid * states + j];
    }
    jl[tid * states] = den;
  }
  __syncthreads();
  for (int i = rank * kThreads + tid; i < RT * (D / 4); i += split * kThreads) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    if (r0 + r >= all_rows) break;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int j = 0; j < states; ++j) {
      const float f = jm[r * states + j];
      const float4 o4 = cluster_load4(&so[j % kTreeSimtWarps][r][d], j / kTreeSimtWarps);
      num.x += f * o4.x, num.y += f * o4.y, num.z += f * o4.z, num.w += f * o4.w;
    }
    // den = 0: the row attends nothing (its sums are zero); a NaN stays one.
    const float den = jl[r * states];
    if (den != 0.f) num.x /= den, num.y /= den, num.z /= den, num.w /= den;
    else num = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4*>(out + out_row(r0 + r) + d) = num;
  }
  if (split > 1) cluster_sync();  // the others read this CTA's shared memory
}

}  // namespace pa
