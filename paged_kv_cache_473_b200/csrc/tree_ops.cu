// C ABI of the drafting step's operators: norm and rotation of queries and
// keys (with the paged append), attention of a drafted tree over the cache and
// the move of its accepted path.  See include/pagedattn.h.
#include <algorithm>

#include "../../include/pagedattn.h"
#include "commit_tree.cuh"
#include "decode_common.cuh"
#include "decode_tree.cuh"
#include "decode_tree_common.cuh"
#include "decode_tree_simt.cuh"
#include "host_common.cuh"
#include "norm_rope.cuh"

namespace {

using pa::NormRopeParams;
using pa::TreeParams;

// ---- norm, rotation, append ---------------------------------------------------------

template <typename T, int D, bool APPEND>
cudaError_t launch_norm_rope_t(NormRopeParams& p, int32_t tokens, cudaStream_t st) {
  constexpr int kRowsPerIter = pa::kNormRopeThreads / (D / 8);
  const int rows = p.hq + (APPEND ? 2 : 1) * p.hkv;
  const int iters = (rows + kRowsPerIter - 1) / kRowsPerIter;
  // One CTA per token; the rows of a token over several CTAs while there are
  // fewer than two CTAs per SM.
  const int split = (int)std::min<long long>(iters, (2LL * sm_count() + tokens - 1) / tokens);
  const int per = (iters + split - 1) / split;
  p.rows_per_cta = per * kRowsPerIter;
  const dim3 grid((unsigned)tokens, (unsigned)((iters + per - 1) / per));
  return launch_ex(pa::norm_rope_kernel<T, D, APPEND>, grid, dim3(pa::kNormRopeThreads), 0, st, true, p);
}

template <bool APPEND>
cudaError_t launch_norm_rope(NormRopeParams& p, int32_t tokens, int32_t head_dim, pa_dtype_t dt, cudaStream_t st) {
  if (dt == PA_F32) {
    switch (head_dim) {
      case 64:
        return launch_norm_rope_t<float, 64, APPEND>(p, tokens, st);
      case 128:
        return launch_norm_rope_t<float, 128, APPEND>(p, tokens, st);
      default:
        return launch_norm_rope_t<float, 256, APPEND>(p, tokens, st);
    }
  }
  switch (head_dim) {
    case 64:
      return launch_norm_rope_t<__nv_bfloat16, 64, APPEND>(p, tokens, st);
    case 128:
      return launch_norm_rope_t<__nv_bfloat16, 128, APPEND>(p, tokens, st);
    default:
      return launch_norm_rope_t<__nv_bfloat16, 256, APPEND>(p, tokens, st);
  }
}

// The checks both calls share; PA_OK with *empty set when there is no token.
pa_status_t check_norm_rope(const NormRopeParams& p, int32_t num_tokens, int32_t head_dim, pa_dtype_t dtype,
                            bool* empty) {
  *empty = false;
  if (num_tokens < 0 || p.hq <= 0 || p.hkv <= 0 || head_dim <= 0 || p.rotary < 0) return PA_ERR_INVALID;
  if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_INVALID;
  if (!(p.eps >= 0.f) || !std::isfinite(p.eps)) return PA_ERR_INVALID;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (p.rotary > head_dim) return PA_ERR_INVALID;
  if (p.rotary % 16 != 0) return PA_ERR_UNSUPPORTED;
  if ((long long)p.hq + 2LL * p.hkv > kMaxGridYZ) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) {
    *empty = true;
    return PA_OK;
  }
  const int64_t step = dtype == PA_F32 ? 4 : 8;  // elements of 16 bytes
  if (!p.q || !p.k || !p.q_out || !aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.q_out, 16)) return PA_ERR_INVALID;
  if (p.q_stride < 0 || p.k_stride < 0 || p.q_stride % step || p.k_stride % step) return PA_ERR_INVALID;
  if (p.q_out_stride < (int64_t)p.hq * head_dim || p.q_out_stride % step) return PA_ERR_INVALID;
  if (!aligned(p.q_weight, 16) || !aligned(p.k_weight, 16)) return PA_ERR_INVALID;
  if (p.rotary > 0 && (!p.positions || !p.inv_freq)) return PA_ERR_INVALID;
  if (!aligned(p.positions, 4) || !aligned(p.inv_freq, 4)) return PA_ERR_INVALID;
  return PA_OK;
}

// ---- tree attention -------------------------------------------------------------------

template <typename T, int D>
cudaError_t launch_tree_simt_t(const TreeParams& p, cudaStream_t st) {
  constexpr int RT = pa::kTreeSimtRows, NW = pa::kTreeSimtWarps;
  const dim3 grid((unsigned)((p.tree_len * p.group + RT - 1) / RT), p.hkv, p.batch);
  return launch_ex(pa::decode_tree_simt_kernel<T, D>, grid, dim3(NW * 32), NW * RT * D * 4, st, true, p);
}

cudaError_t launch_tree_simt(const TreeParams& p, int head_dim, cudaStream_t st) {
  switch (head_dim) {
    case 64:
      return launch_tree_simt_t<float, 64>(p, st);
    case 128:
      return launch_tree_simt_t<float, 128>(p, st);
    default:
      return launch_tree_simt_t<float, 256>(p, st);
  }
}

// CTAs of the tensor-core kernel: all that are resident at once, a whole number
// of groups of m_tiles.
int tree_grid(int head_dim, int m_tiles) {
  const int resident = sm_count() * (head_dim <= 128 ? pa::TreeCfg<128>::kMinBlocks : pa::TreeCfg<256>::kMinBlocks);
  return std::max(1, resident / m_tiles) * m_tiles;
}

int tree_m_tiles(int tree_len, int group) { return (tree_len * group + pa::kTreeRows - 1) / pa::kTreeRows; }

// Workspace of the tensor-core kernel: the counter region of the split-K calls
// (untouched), one record per CTA, two partials per CTA.
struct TreeWorkspace {
  size_t rec, o, ml, bytes;
};
TreeWorkspace tree_workspace(int grid, int head_dim, int tree_len, int group) {
  const size_t rows = std::min(pa::kTreeRows, (tree_len * group + pa::kTreeCombineRows - 1) / pa::kTreeCombineRows *
                                                  pa::kTreeCombineRows);
  TreeWorkspace w;
  w.rec = pa::kCounterBytes;
  w.o = w.rec + align256((size_t)grid * sizeof(int4));
  w.ml = w.o + align256(2 * (size_t)grid * rows * head_dim * 4);
  w.bytes = w.ml + align256(2 * (size_t)grid * rows * 2 * 4);
  return w;
}

template <int D>
cudaError_t launch_tree_t(const TreeParams& p, int grid, cudaStream_t st) {
  using Cfg = pa::TreeCfg<D>;
  CUtensorMap kmap, vmap;
  const long long rows = (long long)p.num_blocks * p.hkv * p.block_size;
  if (!cache_maps(p.k_cache, p.v_cache, D, rows, &kmap, &vmap)) return cudaErrorInvalidValue;
  auto kern = pa::decode_tree_kernel<D>;
  static std::atomic<uint64_t> smem_done{0};
  cudaError_t e = set_smem(kern, Cfg::kSmemBytes, smem_done);
  if (e != cudaSuccess) return e;
  e = launch_ex(kern, dim3(grid), dim3(pa::kTreeThreads), Cfg::kSmemBytes, st, true, kmap, vmap, p);
  if (e != cudaSuccess) return e;
  const int chunks = (std::min(pa::kTreeRows, p.tree_len * p.group) + pa::kTreeCombineRows - 1) / pa::kTreeCombineRows;
  return launch_ex(pa::tree_combine_kernel<D>, dim3(grid, chunks), dim3(2 * D), 0, st, true, p);
}

cudaError_t launch_tree(const TreeParams& p, int head_dim, int grid, cudaStream_t st) {
  switch (head_dim) {
    case 64:
      return launch_tree_t<64>(p, grid, st);
    case 128:
      return launch_tree_t<128>(p, grid, st);
    default:
      return launch_tree_t<256>(p, grid, st);
  }
}

}  // namespace

cudaError_t pa_host::tree_ops_errors(unsigned int* bits, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, pa::g_device_errors, sizeof *bits);
  if (e != cudaSuccess || !clear) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(pa::g_device_errors, &zero, sizeof zero);
}

extern "C" {

pa_status_t pa_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* q_weight,
                            const float* k_weight, float eps, const float* inv_freq, int32_t rotary_dim,
                            int32_t interleaved, const int32_t* positions, int32_t num_tokens, int32_t num_q_heads,
                            int32_t num_kv_heads, int32_t head_dim, void* q_out, int64_t q_out_stride, void* k_out,
                            int64_t k_out_stride, pa_dtype_t dtype, pa_stream_t stream) {
  pa_host::set_last_launches(0);
  NormRopeParams p{};
  p.q = q;
  p.k = k;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.inv_freq = inv_freq;
  p.rotary = rotary_dim;
  p.interleaved = interleaved != 0;
  p.positions = positions;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.q_out = q_out;
  p.q_out_stride = q_out_stride;
  p.k_out = k_out;
  p.k_out_stride = k_out_stride;
  bool empty;
  const pa_status_t st = check_norm_rope(p, num_tokens, head_dim, dtype, &empty);
  if (st != PA_OK || empty) return st;
  if (!k_out || !aligned(k_out, 16) || k_out_stride < (int64_t)num_kv_heads * head_dim ||
      k_out_stride % (dtype == PA_F32 ? 4 : 8))
    return PA_ERR_INVALID;
  if (launch_norm_rope<false>(p, num_tokens, head_dim, dtype, stream) != cudaSuccess) return PA_ERR_CUDA;
  pa_host::set_last_launches(1);
  return PA_OK;
}

pa_status_t pa_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const float* q_weight, const float* k_weight, float eps,
                           const float* inv_freq, int32_t rotary_dim, int32_t interleaved, const int32_t* positions,
                           const int64_t* slot_mapping, int32_t num_tokens, int32_t num_q_heads,
                           int32_t num_kv_heads, int32_t head_dim, void* q_out, void* k_cache, void* v_cache,
                           int32_t num_blocks, int32_t block_size, pa_dtype_t dtype, pa_stream_t stream) {
  pa_host::set_last_launches(0);
  if (num_blocks <= 0 || block_size <= 0) return PA_ERR_INVALID;
  NormRopeParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.inv_freq = inv_freq;
  p.rotary = rotary_dim;
  p.interleaved = interleaved != 0;
  p.positions = positions;
  p.slots = slot_mapping;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.q_out = q_out;
  p.q_out_stride = (int64_t)num_q_heads * head_dim;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.block_size = block_size;
  bool empty;
  const pa_status_t st = check_norm_rope(p, num_tokens, head_dim, dtype, &empty);
  if (st != PA_OK || empty) return st;
  if (!v || !k_cache || !v_cache || !slot_mapping || !aligned(v, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(slot_mapping, 8) || v_stride < 0 || v_stride % (dtype == PA_F32 ? 4 : 8))
    return PA_ERR_INVALID;
  if (launch_norm_rope<true>(p, num_tokens, head_dim, dtype, stream) != cudaSuccess) return PA_ERR_CUDA;
  pa_host::set_last_launches(1);
  return PA_OK;
}

size_t pa_decode_tree_workspace_size(int32_t batch, int32_t tree_len, int32_t num_q_heads, int32_t head_dim,
                                     int32_t max_context_len, int32_t num_kv_heads) {
  (void)max_context_len;  // the partials are two per CTA, however long the contexts are
  if (batch <= 0 || tree_len <= 0 || num_q_heads <= 0 || head_dim <= 0 || num_kv_heads <= 0) return 0;
  if (tree_len > pa::kMaxTreeNodes || num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > pa::kMaxGroup)
    return 0;
  const int group = num_q_heads / num_kv_heads;
  return tree_workspace(tree_grid(head_dim, tree_m_tiles(tree_len, group)), head_dim, tree_len, group).bytes;
}

pa_status_t pa_decode_tree(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                           const int32_t* context_lens, const int32_t* tree_lens, const int64_t* tree_mask,
                           int64_t mask_stride, int32_t batch, int32_t tree_len, int32_t num_q_heads,
                           int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t max_blocks_per_seq,
                           int32_t num_blocks, float scale, float softcap, int32_t window, void* out,
                           pa_dtype_t dtype, int32_t max_context_len, void* workspace, size_t workspace_bytes,
                           pa_stream_t stream) {
  pa_host::set_last_launches(0);
  const Shape s{batch, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks};
  const pa_status_t st = check_decode_args(q, k_cache, v_cache, block_tables, context_lens, s, softcap, out, dtype,
                                           PA_KERNEL_AUTO);
  if (st != PA_OK) return st;
  if (tree_len <= 0 || max_context_len <= 0) return PA_ERR_INVALID;
  if (tree_len > pa::kMaxTreeNodes) return PA_ERR_UNSUPPORTED;
  if (mask_stride != 0 && mask_stride < tree_len) return PA_ERR_INVALID;
  const long long longest = std::min<long long>(max_context_len, (long long)max_blocks_per_seq * block_size);
  const int group = num_q_heads / num_kv_heads, m_tiles = tree_m_tiles(tree_len, group);
  if ((longest / pa::kTreeTile + 1) * num_kv_heads >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
  if (batch == 0) return PA_OK;
  if (!tree_mask || !aligned(tree_mask, 8) || !aligned(tree_lens, 4)) return PA_ERR_INVALID;
  const bool tensor_cores = dtype == PA_BF16;
  const int grid = tree_grid(head_dim, m_tiles);
  const TreeWorkspace w = tree_workspace(grid, head_dim, tree_len, group);
  if (tensor_cores && (!workspace || !aligned(workspace, 16) || workspace_bytes < w.bytes)) return PA_ERR_WORKSPACE;

  TreeParams p{};
  p.q = q;
  p.out = out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.tree_lens = tree_lens;
  p.tree_mask = tree_mask;
  p.mask_stride = mask_stride;
  p.batch = batch;
  p.tree_len = tree_len;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.group = group;
  p.block_size = block_size;
  p.log2_bs = ilog2(block_size);
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.window = window;
  p.max_context = max_context_len;
  p.m_tiles = m_tiles;
  p.scale = scale;
  p.use_softcap = (softcap > 0.f && std::isfinite(softcap)) ? 1 : 0;
  p.softcap = p.use_softcap ? softcap : 0.f;
  if (!tensor_cores) {
    if (launch_tree_simt(p, head_dim, stream) != cudaSuccess) return PA_ERR_CUDA;
    pa_host::set_last_launches(1);
    return PA_OK;
  }
  char* ws = static_cast<char*>(workspace);
  p.ws_rec = reinterpret_cast<int4*>(ws + w.rec);
  p.ws_o = reinterpret_cast<float*>(ws + w.o);
  p.ws_ml = reinterpret_cast<float*>(ws + w.ml);
  if (launch_tree(p, head_dim, grid, stream) != cudaSuccess) return PA_ERR_CUDA;
  pa_host::set_last_launches(2);
  return PA_OK;
}

pa_status_t pa_commit_tree(void* k_cache, void* v_cache, int32_t num_layers, const int32_t* block_tables,
                           const int32_t* context_lens, const int32_t* tree_lens, int32_t tree_len,
                           const int32_t* accepted, int32_t max_accept, const int32_t* accept_lens, int32_t batch,
                           int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t max_blocks_per_seq,
                           int32_t num_blocks, int32_t* new_lens, pa_dtype_t dtype, pa_stream_t stream) {
  pa_host::set_last_launches(0);
  if (batch < 0 || num_layers <= 0 || tree_len <= 0 || max_accept <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
    return PA_ERR_INVALID;
  if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_INVALID;
  const int elt = dtype == PA_F32 ? 4 : 2;
  if ((long long)head_dim * elt % 16 != 0 || !pow2(block_size)) return PA_ERR_UNSUPPORTED;
  if (tree_len > pa::kMaxTreeNodes || batch > kMaxGridYZ) return PA_ERR_UNSUPPORTED;
  if ((long long)num_blocks * block_size >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
  if ((long long)max_blocks_per_seq * block_size >= (1LL << 30)) return PA_ERR_UNSUPPORTED;
  const long long token_chunks = (long long)num_kv_heads * (head_dim * elt / 16);  // one token in one cache
  if (token_chunks >= (1LL << 30)) return PA_ERR_UNSUPPORTED;
  if (batch == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !accepted || !accept_lens) return PA_ERR_INVALID;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
      !aligned(tree_lens, 4) || !aligned(accepted, 4) || !aligned(accept_lens, 4) || !aligned(new_lens, 4))
    return PA_ERR_INVALID;
  if (new_lens == context_lens) return PA_ERR_INVALID;
  const long long blocks = (2LL * num_layers * token_chunks + pa::kCommitThreads - 1) / pa::kCommitThreads;
  if (blocks > INT_MAX) return PA_ERR_UNSUPPORTED;

  pa::CommitParams p{};
  p.k_cache = static_cast<uint4*>(k_cache);
  p.v_cache = static_cast<uint4*>(v_cache);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.tree_lens = tree_lens;
  p.accepted = accepted;
  p.accept_lens = accept_lens;
  p.new_lens = new_lens;
  p.layer_chunks = (int64_t)num_blocks * block_size * token_chunks;
  p.layers = num_layers;
  p.hkv = num_kv_heads;
  p.chunks_per_row = head_dim * elt / 16;
  p.max_accept = max_accept;
  p.tree_len = tree_len;
  p.log2_bs = ilog2(block_size);
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  const cudaError_t e = launch_ex(pa::commit_tree_kernel, dim3((unsigned)blocks, batch), dim3(pa::kCommitThreads), 0,
                                  static_cast<cudaStream_t>(stream), true, p);
  if (e != cudaSuccess) return PA_ERR_CUDA;
  pa_host::set_last_launches(1);
  return PA_OK;
}

}  // extern "C"
