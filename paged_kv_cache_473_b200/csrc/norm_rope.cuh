// Per-head RMS norm and rotary position embedding of one step's queries and
// keys in one pass, with the append of keys and values to the paged cache
// (APPEND) or with the keys written to a plain tensor.
//
//   y = x / sqrt(mean(x^2) + eps) * w           (a weight vector given; fp32)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq[i],
//
// for pair i < rotary / 2 of each head: elements i and i + rotary / 2, or 2 i
// and 2 i + 1 (interleaved); elements from `rotary` on are only normed.  Values
// are held in fp32 from the load to the one rounding at the store.
//
// The angle.  t is taken modulo one turn in 64 bits: position * (inv_freq / 2 pi)
// minus its nearest integer, then sincospif in fp32.  (In fp32 the product
// alone is off by up to half a unit of its last place, 0.004 rad at position
// 131072.)
//
// The work is one read and one write of every row, so DRAM bounds it, and for
// a decode step's few tokens the launch.  A warp takes one token, or a part of
// its rows where there are few tokens, on its own: no barrier joins warps, and
// each has several rows in flight ahead of the one it works on.  A head's row is
// held by D / 8 neighbouring lanes, each with four pairs: two chunks of four
// elements (8-byte accesses for bf16), so that nothing but the norm's sum
// passes between lanes, and a lane reads and writes only its own elements
// (which makes in-place calls safe).  Issue slots come next to DRAM (72 % of them
// used before the arithmetic was packed), so it goes two elements to an instruction.
// B200, append of 16384 tokens of 48 rows of 128, bf16: 68 us on the machine of the
// comparisons below, 0.90 of the copy rate (72, 0.86, on another);
// 74 one element at a time; with 6, 9 or 10 CTAs an SM 72, 70 and 78; three rows in
// flight 71, six (at 6 CTAs) 69; the sums of four rows taken together, with fewer
// shuffles, 84 (a row then waits for the others); with eight neighbouring elements
// a lane and the pairs' other halves by shuffles 83.  The token's rotary / 2 angles
// are computed by each warp that has rows of it, two or so a lane, and pass through
// shared memory; a lane sits at the same place of each of its rows and keeps the
// four it needs in registers.
#pragma once

#include "decode_common.cuh"
#include "ptx.cuh"

namespace pa {

struct NormRopeParams {
  const void *q, *k, *v;                  // rows [token][heads][D], token strides in elements
  int64_t q_stride, k_stride, v_stride;
  const float *q_weight, *k_weight;       // [D], or null: no norm
  float eps;
  const float* inv_freq;                  // [rotary / 2]
  int rotary, interleaved;
  const int32_t* positions;               // [tokens]
  const int64_t* slots;                   // APPEND: [tokens]
  int hq, hkv;
  void *q_out, *k_out;
  int64_t q_out_stride, k_out_stride;
  void *k_cache, *v_cache;                // APPEND: [blocks][hkv][block_size][D]
  int64_t num_slots;
  int block_size;
  int tokens;
  int parts, part_rows;                   // warps per token, rows of each (a multiple of the rows a warp holds)
};

constexpr int kNormRopeWarps = 4;

// CTAs an SM: eight where the rows in flight fit the 64 registers a thread that this
// leaves, else seven (8192 tokens of 40 rows of 128, bf16, not appended: 55 us with eight, 36
// with seven; D = 256: 23 and 24).
template <typename T, int D, bool APPEND>
constexpr int norm_rope_ctas() {
  return sizeof(T) == 2 && (APPEND || D == 256) ? 8 : 7;
}

// Four consecutive elements in fp32, in pairs for packed arithmetic.
struct Wide4 {
  float2 a, b;
};

// Four consecutive elements, as they lie in memory.
template <typename T>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
  uint2 a;
  __device__ __forceinline__ void load(const void* src) { a = *static_cast<const uint2*>(src); }
  __device__ __forceinline__ void store(void* dst) const { *static_cast<uint2*>(dst) = a; }
  __device__ __forceinline__ Wide4 wide() const {
    return {make_float2(bf16_lo(a.x), bf16_hi(a.x)), make_float2(bf16_lo(a.y), bf16_hi(a.y))};
  }
  __device__ __forceinline__ void round(Wide4 x) {  // to nearest even
    a = make_uint2(pack_bf16x2(x.a.x, x.a.y), pack_bf16x2(x.b.x, x.b.y));
  }
};
template <>
struct Raw4<float> {
  float4 a;
  __device__ __forceinline__ void load(const void* src) { a = *static_cast<const float4*>(src); }
  __device__ __forceinline__ void store(void* dst) const { *static_cast<float4*>(dst) = a; }
  __device__ __forceinline__ Wide4 wide() const { return {make_float2(a.x, a.y), make_float2(a.z, a.w)}; }
  __device__ __forceinline__ void round(Wide4 x) { a = make_float4(x.a.x, x.a.y, x.b.x, x.b.y); }
};

__device__ __forceinline__ Wide4 wide4(const float* x) {
  const float4 v = *reinterpret_cast<const float4*>(x);
  return {make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
__device__ __forceinline__ Wide4 scale4(Wide4 x, float s, Wide4 w) {
  const float2 s2 = make_float2(s, s);
  return {mul_f32x2(mul_f32x2(x.a, s2), w.a), mul_f32x2(mul_f32x2(x.b, s2), w.b)};
}
// x u + y v.
__device__ __forceinline__ Wide4 turn4(Wide4 x, Wide4 u, Wide4 y, Wide4 v) {
  return {fma_f32x2(y.a, v.a, mul_f32x2(x.a, u.a)), fma_f32x2(y.b, v.b, mul_f32x2(x.b, u.b))};
}
// (a cos - b sin, b cos + a sin) of a pair in (x, y).
__device__ __forceinline__ float2 turn_pair(float2 x, float c, float s) {
  return make_float2(fmaf(-x.y, s, x.x * c), fmaf(x.x, s, x.y * c));
}

template <typename T, int D, bool APPEND>
__global__ void __launch_bounds__(kNormRopeWarps * 32, (norm_rope_ctas<T, D, APPEND>())) norm_rope_kernel(const NormRopeParams p) {
  constexpr uint32_t FULL = 0xffffffffu;
  constexpr int LPR = D / 8;                 // lanes per row
  constexpr int RPW = 32 / LPR;              // rows a warp holds at a time
  constexpr int U = sizeof(T) == 2 ? 4 : 3;  // of those, in flight
  __shared__ __align__(16) float cosines[kNormRopeWarps][D / 2], sines[kNormRopeWarps][D / 2];  // of a warp's token

  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, ch = lane % LPR, warp = threadIdx.x >> 5;
  const int64_t task = (int64_t)blockIdx.x * kNormRopeWarps + warp;
  const int64_t token = task / p.parts;
  if (token >= p.tokens) return;
  const int half = p.rotary >> 1;
  pdl_wait();  // a programmatic dependent: nothing of global memory is touched before

  // This lane's two chunks: the first and second elements of the pairs 4 ch .. 4 ch + 3
  // (half-split; behind `rotary` the halves of what is left), or (interleaved) two
  // pairs of each half of the row.  Neighbouring lanes' chunks are neighbours.
  const int split = p.interleaved ? D : half, rest = ch * 4 - split;
  const int lo = rest < 0 ? ch * 4 : p.rotary + rest;
  const int hi = p.interleaved ? lo + D / 2 : rest < 0 ? lo + half : lo + ((D - p.rotary) >> 1);
  const bool lo_turns = p.interleaved ? lo < p.rotary : rest < 0, hi_turns = p.interleaved ? hi < p.rotary : rest < 0;

  // ---- this warp's rows: q heads, then k heads, then (APPEND) v heads -----------------------
  const int64_t slot = APPEND ? p.slots[token] : 0;
  const double position = p.rotary > 0 ? (double)p.positions[token] : 0.0;
  const int rows = p.hq + (APPEND ? 2 : 1) * p.hkv;
  const int begin = (int)(task - token * p.parts) * p.part_rows;  // the same in all lanes
  const int end = min(rows, begin + p.part_rows);
  const T* q = static_cast<const T*>(p.q) + token * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + token * p.k_stride;
  const T* v = APPEND ? static_cast<const T*>(p.v) + token * p.v_stride : nullptr;
  auto source = [&](int r) -> const T* {
    if (r < p.hq) return q + (int64_t)r * D;
    if (!APPEND || r < p.hq + p.hkv) return k + (int64_t)(r - p.hq) * D;
    return v + (int64_t)(r - p.hq - p.hkv) * D;
  };
  Raw4<T> a[U], b[U];
  const int mine = lane / LPR;  // which of the warp's rows
  auto load = [&](int u, int r) {
    const T* x = source(r);
    a[u].load(x + lo);
    b[u].load(x + hi);
  };
#pragma unroll
  for (int u = 0; u < U; ++u)  // in flight while the angles are computed
    if (begin + u * RPW + mine < end) load(u, begin + u * RPW + mine);

  for (int i = lane; i < half; i += 32) {
    const double t = position * ((double)p.inv_freq[i] * 0.15915494309189535);  // turns: 1 / (2 pi)
    sincospif(2.f * (float)(t - rint(t)), &sines[warp][i], &cosines[warp][i]);
  }
  __syncwarp();
  if (APPEND && slot < 0) return;  // a padding token: none of its rows is written
  const bool in_pool = !APPEND || slot < p.num_slots;
  if (APPEND && !in_pool && lane == 0 && begin == 0) raise_error(PA_DEVERR_SLOT);
  const int64_t blk = APPEND ? slot / p.block_size : 0;
  const int64_t off = APPEND ? slot - blk * p.block_size : 0;
  auto target = [&](int r) -> T* {
    if (r < p.hq) return static_cast<T*>(p.q_out) + token * p.q_out_stride + (int64_t)r * D;
    if (!APPEND) return static_cast<T*>(p.k_out) + token * p.k_out_stride + (int64_t)(r - p.hq) * D;
    const bool is_k = r < p.hq + p.hkv;
    const int64_t h = r - p.hq - (is_k ? 0 : p.hkv);
    return static_cast<T*>(is_k ? p.k_cache : p.v_cache) + ((blk * p.hkv + h) * p.block_size + off) * D;
  };

  // This lane's angles: four pairs, or (interleaved) two of each chunk.
  Wide4 c = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, sn = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const int pair0 = p.interleaved ? lo / 2 : lo, pair1 = p.interleaved ? hi / 2 : lo + 2;
  if (lo_turns) {
    c.a = *reinterpret_cast<const float2*>(&cosines[warp][pair0]);
    sn.a = *reinterpret_cast<const float2*>(&sines[warp][pair0]);
  }
  if (hi_turns) {
    c.b = *reinterpret_cast<const float2*>(&cosines[warp][pair1]);
    sn.b = *reinterpret_cast<const float2*>(&sines[warp][pair1]);
  }
  const Wide4 minus = {make_float2(-sn.a.x, -sn.a.y), make_float2(-sn.b.x, -sn.b.y)};
  const int turned_rows = p.hq + p.hkv;  // of q and k; v rows are copied as they are
  const bool normed = p.q_weight || p.k_weight;

  for (int r0 = begin; r0 < end; r0 += U * RPW) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int first = r0 + u * RPW, r = first + mine;  // `first`: the same in all lanes
      if (first >= end) break;
      const bool real = r < end;
      if (first < turned_rows) {
        const bool turned = r < turned_rows;
        Wide4 x = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, y = x;
        if (real) x = a[u].wide(), y = b[u].wide();
        if (normed) {
          const float2 t = fma_f32x2(x.a, x.a, fma_f32x2(x.b, x.b, fma_f32x2(y.a, y.a, mul_f32x2(y.b, y.b))));
          float ss = t.x + t.y;
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
          const float* w = r < p.hq ? p.q_weight : p.k_weight;
          if (turned && w) {
            const float inv = rsqrtf(ss * (1.f / D) + p.eps);  // within 2 units of the last place
            x = scale4(x, inv, wide4(w + lo));
            y = scale4(y, inv, wide4(w + hi));
          }
        }
        if (turned) {
          // (What does not turn stays as it is: 0 times an infinity is not nothing.)
          if (p.interleaved) {
            if (lo_turns) x = {turn_pair(x.a, c.a.x, sn.a.x), turn_pair(x.b, c.a.y, sn.a.y)};
            if (hi_turns) y = {turn_pair(y.a, c.b.x, sn.b.x), turn_pair(y.b, c.b.y, sn.b.y)};
          } else if (lo_turns) {
            const Wide4 z = turn4(x, c, y, minus);
            y = turn4(y, c, x, sn);
            x = z;
          }
          a[u].round(x);
          b[u].round(y);
        }
      }
      if (real && (in_pool || r < p.hq)) {
        T* out = target(r);
        a[u].store(out + lo);
        b[u].store(out + hi);
      }
      if (r + U * RPW < end) load(u, r + U * RPW);
    }
  }
}

}  // namespace pa
