// Host-side pieces shared by the translation units of the C ABI: argument
// checks, tensor-map set-up, launch helpers and per-thread accounting.  Each
// unit gets its own copy of the helpers and of their small caches; the
// accounting and the device error word are the library's (one definition,
// reached through the functions declared here).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <utility>

#include "../../include/pagedattn.h"
#include "decode_common.cuh"

namespace pa_host {

// Launches of the calling thread's last successful call (pa_last_launch_count).
void set_last_launches(int32_t n);

// The device error word of tree_ops.cu's kernels on the current device: read
// into *bits, then zeroed when clear.  (Without relocatable device code each
// translation unit has a word of its own; pa_device_errors joins them.)
cudaError_t tree_ops_errors(unsigned int* bits, bool clear);

}  // namespace pa_host

namespace {

using pa::DecodeParams;

constexpr int kNoSplitPartition = 1 << 30;
constexpr int kMaxGridYZ = 65535;

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
inline int ilog2(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}

// ---- tensor maps ---------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

inline bool tensor_map_encoder() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

// The cache viewed as a 2-D bf16 tensor [rows = num_blocks*Hkv*bs][head_dim];
// a box is 64 columns (128 B) x 16 rows (or box_rows), landed with 128-byte swizzle.
inline bool encode_cache_map(CUtensorMap* map, const void* base, int head_dim, long long rows,
                             int box_rows = pa::kSliceTokens) {
  cuuint64_t dims[2] = {(cuuint64_t)head_dim, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)head_dim * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Tensor maps of the K and V caches, encoded once per (base addresses, rows,
// head_dim) and reused: a map holds only the address, the shape and the fixed
// box / swizzle, so a cached one is exactly what a fresh encode would give.
// A small per-thread table (no lock); the oldest entry is replaced.
inline bool cache_maps(const void* kbase, const void* vbase, int head_dim, long long rows, CUtensorMap* kmap,
                CUtensorMap* vmap) {
  struct Entry {
    const void* k;
    const void* v;
    long long rows;
    int d;
    CUtensorMap kmap, vmap;
  };
  constexpr int kEntries = 16;
  thread_local Entry table[kEntries] = {};
  thread_local int next = 0;
  for (const Entry& e : table) {
    if (e.k == kbase && e.v == vbase && e.rows == rows && e.d == head_dim && kbase) {
      *kmap = e.kmap;
      *vmap = e.vmap;
      return true;
    }
  }
  if (!tensor_map_encoder()) return false;
  if (!encode_cache_map(kmap, kbase, head_dim, rows) || !encode_cache_map(vmap, vbase, head_dim, rows)) return false;
  Entry& e = table[next];
  next = (next + 1) % kEntries;
  e.k = kbase;
  e.v = vbase;
  e.rows = rows;
  e.d = head_dim;
  e.kmap = *kmap;
  e.vmap = *vmap;
  return true;
}

// ---- argument checks -------------------------------------------------------------

struct Shape {
  int batch, hq, hkv, d, bs, max_blocks, num_blocks;
};

inline pa_status_t check_decode_args(const void* q, const void* kc, const void* vc, const int32_t* bt, const int32_t* cl,
                              const Shape& s, float softcap, const void* out, pa_dtype_t dt, pa_kernel_t kernel) {
  if (s.batch < 0 || s.hq <= 0 || s.hkv <= 0 || s.d <= 0 || s.bs <= 0 || s.max_blocks <= 0 || s.num_blocks <= 0)
    return PA_ERR_INVALID;
  if (s.hq % s.hkv != 0) return PA_ERR_INVALID;
  if (dt != PA_F32 && dt != PA_BF16) return PA_ERR_INVALID;
  if (kernel != PA_KERNEL_AUTO && kernel != PA_KERNEL_CUDA_CORE && kernel != PA_KERNEL_MMA) return PA_ERR_INVALID;
  if (std::isnan(softcap)) return PA_ERR_INVALID;
  if (s.batch > 0) {
    if (!q || !kc || !vc || !bt || !cl || !out) return PA_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(kc, 16) || !aligned(vc, 16) || !aligned(out, 16) || !aligned(bt, 4) ||
        !aligned(cl, 4))
      return PA_ERR_INVALID;
  }
  if (s.d != 64 && s.d != 128 && s.d != 256) return PA_ERR_UNSUPPORTED;
  if (!pow2(s.bs) || s.bs < 16 || s.bs > 256) return PA_ERR_UNSUPPORTED;
  if (s.hq / s.hkv > pa::kMaxGroup) return PA_ERR_UNSUPPORTED;
  if (s.batch > kMaxGridYZ || s.hkv > kMaxGridYZ) return PA_ERR_UNSUPPORTED;
  if ((long long)s.num_blocks * s.hkv * s.bs >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
  if ((long long)s.max_blocks * s.bs >= (1LL << 30)) return PA_ERR_UNSUPPORTED;
  if (kernel == PA_KERNEL_MMA && dt != PA_BF16) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

inline DecodeParams make_params(const void* q, const void* kc, const void* vc, const int32_t* bt, const int32_t* cl,
                         const Shape& s, float scale, float softcap, int32_t window, void* out) {
  DecodeParams p{};
  p.q = q;
  p.out = out;
  p.k_cache = kc;
  p.v_cache = vc;
  p.block_tables = bt;
  p.context_lens = cl;
  p.batch = s.batch;
  p.hq = s.hq;
  p.hkv = s.hkv;
  p.group = s.hq / s.hkv;
  p.head_dim = s.d;
  p.block_size = s.bs;
  p.log2_bs = ilog2(s.bs);
  p.max_blocks = s.max_blocks;
  p.num_blocks = s.num_blocks;
  p.window = window;
  p.partition = kNoSplitPartition;
  p.max_parts = 1;
  p.max_context = s.max_blocks * s.bs;
  p.scale = scale;
  p.use_softcap = (softcap > 0.f && std::isfinite(softcap)) ? 1 : 0;
  p.softcap = p.use_softcap ? softcap : 0.f;
  p.inv_softcap = p.use_softcap ? 1.f / softcap : 0.f;
  p.q_len = 1;
  return p;
}

// ---- launch helpers ---------------------------------------------------------------

// Opt a kernel in to more than 48 KB of dynamic shared memory, once per device
// (the flag word is per kernel instantiation: one bit per device ordinal < 64).
template <typename Kernel>
cudaError_t set_smem(Kernel k, int bytes, std::atomic<uint64_t>& done) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// Launch `kern` with cudaLaunchKernelEx; `pdl` lets it start while the
// preceding kernel on the stream finishes (it must call griddepcontrol.wait
// before reading that kernel's output).  `cluster` neighbouring CTAs of the
// grid's x form a cluster where it is above one.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, int cluster, dim3 block, int smem, cudaStream_t st,
                           bool pdl, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (pdl) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_ex(void (*kern)(KArgs...), dim3 grid, dim3 block, int smem, cudaStream_t st, bool pdl,
                      Args&&... args) {
  return launch_cluster(kern, grid, 1, block, smem, st, pdl, std::forward<Args>(args)...);
}

inline int sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64) {
    const int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Opt in to `bytes` of dynamic shared memory (growing only), once per device
// and size, for kernels whose size depends on the launch.
template <typename Kernel>
cudaError_t set_smem_at_least(Kernel k, int bytes, std::atomic<int>* done /* [64] */) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) {
    int cur = done[dev].load(std::memory_order_acquire);
    while (cur < bytes && !done[dev].compare_exchange_weak(cur, bytes)) {
    }
  }
  return e;
}

// Resident CTAs per SM of `kern` at `threads` x `smem`, on the current device:
// queried once per (kernel, shared-memory size, device) and remembered (one
// entry per device for each kernel instantiation; `cache` is that kernel's).
template <typename Kernel>
cudaError_t occupancy(Kernel kern, int threads, int smem, std::atomic<long long>* cache /* [64] */, int* occ) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64) {
    const long long v = cache[dev].load(std::memory_order_acquire);
    if (v > 0 && (v >> 16) == smem) {
      *occ = (int)(v & 0xffff);
      return cudaSuccess;
    }
  }
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(occ, kern, threads, smem);
  if (e == cudaSuccess && dev < 64 && *occ > 0 && *occ < 0x10000)
    cache[dev].store(((long long)smem << 16) | *occ, std::memory_order_release);
  return e;
}

}  // namespace
