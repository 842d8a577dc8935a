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
// a decode step's few tokens the launch.  A head's row is held by D / 8
// neighbouring lanes, 8 elements each (16-byte accesses for bf16): the norm's
// sum is a shuffle over those lanes, and the half-split pair's other element
// comes by a shuffle from the lane that holds it, so that every lane reads and
// writes only its own 8 elements (which makes in-place calls safe).  A CTA
// takes one token: its rotary / 2 angles are computed once, by as many
// threads, into shared memory, and each lane keeps the eight it needs in
// registers over all of its rows, since a lane sits at the same place of each.
// Few tokens: the rows of a token are split over several CTAs.
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
  int rows_per_cta;
};

constexpr int kNormRopeThreads = 256;

// Eight consecutive elements of a row, as loaded (one 16-byte word for bf16, two for fp32).
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const void* src) { a = *static_cast<const uint4*>(src); }
  __device__ __forceinline__ void store(void* dst) const { *static_cast<uint4*>(dst) = a; }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  __device__ __forceinline__ void round(const float (&x)[8]) {  // to nearest even
    a = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* src) {
    a = static_cast<const float4*>(src)[0];
    b = static_cast<const float4*>(src)[1];
  }
  __device__ __forceinline__ void store(void* dst) const {
    static_cast<float4*>(dst)[0] = a;
    static_cast<float4*>(dst)[1] = b;
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void round(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

template <typename T, int D, bool APPEND>
__global__ void __launch_bounds__(kNormRopeThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr uint32_t FULL = 0xffffffffu;
  constexpr int LPR = D / 8;                        // lanes per row
  constexpr int RPI = kNormRopeThreads / LPR;       // rows per iteration of the CTA
  constexpr int U = sizeof(T) == 2 ? 4 : 2;         // rows a lane loads before it works on the first
  __shared__ float2 turn[D / 2];                    // (cos, sin) of the token's angles

  pdl_launch_dependents();
  pdl_wait();  // a programmatic dependent: nothing of global memory is touched before
  const int64_t token = blockIdx.x;
  const int tid = threadIdx.x, ch = tid % LPR;
  const int half = p.rotary >> 1;

  int64_t slot = 0;
  if (APPEND) {
    slot = p.slots[token];
    if (slot < 0) return;  // a padding token: none of its rows is written
  }
  const bool in_pool = !APPEND || slot < p.num_slots;
  if (APPEND && !in_pool && tid == 0 && blockIdx.y == 0) raise_error(PA_DEVERR_SLOT);

  // ---- this CTA's rows: q heads, then k heads, then (APPEND) v heads -----------------------
  const int rows = p.hq + (APPEND ? 2 : 1) * p.hkv;
  const int r_begin = blockIdx.y * p.rows_per_cta + tid / LPR;
  const int r_end = min(rows, ((int)blockIdx.y + 1) * p.rows_per_cta);
  const T* q = static_cast<const T*>(p.q) + token * p.q_stride + ch * 8;
  const T* k = static_cast<const T*>(p.k) + token * p.k_stride + ch * 8;
  const T* v = APPEND ? static_cast<const T*>(p.v) + token * p.v_stride + ch * 8 : nullptr;
  auto source = [&](int r) -> const T* {
    if (r < p.hq) return q + (int64_t)r * D;
    if (!APPEND || r < p.hq + p.hkv) return k + (int64_t)(r - p.hq) * D;
    return v + (int64_t)(r - p.hq - p.hkv) * D;
  };
  const int64_t blk = APPEND ? slot / p.block_size : 0;
  const int64_t off = APPEND ? slot - blk * p.block_size : 0;
  auto target = [&](int r) -> T* {
    if (r < p.hq) return static_cast<T*>(p.q_out) + token * p.q_out_stride + (int64_t)r * D + ch * 8;
    if (!APPEND) return static_cast<T*>(p.k_out) + token * p.k_out_stride + (int64_t)(r - p.hq) * D + ch * 8;
    const bool is_k = r < p.hq + p.hkv;
    const int64_t h = r - p.hq - (is_k ? 0 : p.hkv);
    return static_cast<T*>(is_k ? p.k_cache : p.v_cache) + ((blk * p.hkv + h) * p.block_size + off) * D + ch * 8;
  };

  Raw8<T> raw[U];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r0 + u * RPI < r_end) raw[u].load(source(r0 + u * RPI));
  };
  load(r_begin);  // in flight while the angles are computed

  if (tid < half) {
    const double turns = (double)p.positions[token] * ((double)p.inv_freq[tid] * 0.15915494309189535);  // 1 / (2 pi)
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    turn[tid] = make_float2(c, s);
  }
  __syncthreads();

  // This lane's eight elements: their angles, and the lane that holds their pairs.
  const bool rotated = ch * 8 < p.rotary;
  const bool second = !p.interleaved && ch * 8 >= half;  // second elements of half-split pairs
  int mate = tid & 31;
  float c8[8], s8[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) c8[e] = 1.f, s8[e] = 0.f;
  if (rotated) {
    if (!p.interleaved) mate += second ? -(half >> 3) : (half >> 3);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 t = turn[p.interleaved ? ch * 4 + e / 2 : ch * 8 + e - (second ? half : 0)];
      c8[e] = t.x;
      s8[e] = (p.interleaved ? (e & 1) != 0 : second) ? t.y : -t.y;
    }
  }

  // Every lane of a warp makes the same number of iterations (the shuffles are warp-wide).
  for (int r0 = r_begin; __any_sync(FULL, r0 < r_end); r0 += U * RPI) {
    if (r0 != r_begin) load(r0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPI;
      const bool real = r < r_end;
      const bool turned = r < p.hq + p.hkv;  // v rows are copied as they are
      if (!__any_sync(FULL, real)) break;
      if (__any_sync(FULL, real && turned)) {
        float x[8], y[8];
        if (real) {
          raw[u].widen(x);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = 0.f;
        }
        const float* w = r < p.hq ? p.q_weight : p.k_weight;
        const bool norm = turned && w;
        if (__any_sync(FULL, norm)) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
          if (norm) {
            const float inv = 1.f / sqrtf(ss * (1.f / D) + p.eps);
            const float4 wa = *reinterpret_cast<const float4*>(w + ch * 8);
            const float4 wb = *reinterpret_cast<const float4*>(w + ch * 8 + 4);
            const float wv[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * wv[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = p.interleaved ? x[e ^ 1] : __shfl_sync(FULL, x[e], mate);
          y[e] = rotated ? fmaf(other, s8[e], x[e] * c8[e]) : x[e];
        }
        if (turned) raw[u].round(y);
      }
      if (real && (in_pool || r < p.hq)) raw[u].store(target(r));
    }
  }
}

}  // namespace pa
