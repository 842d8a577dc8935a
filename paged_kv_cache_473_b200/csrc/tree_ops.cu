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

static_assert(PA_COUNTER_BYTES == pa::kCounterBytes, "the header's size of the counter region");

using pa::NormRopeParams;
using pa::TreeParams;

// ---- norm, rotation, append ---------------------------------------------------------

template <typename T, int D, bool APPEND>
cudaError_t launch_norm_rope_t(NormRopeParams& p, int32_t tokens, cudaStream_t st) {
  constexpr int kRows = 32 / (D / 8);  // that a warp holds at a time
  const int rows = p.hq + (APPEND ? 2 : 1) * p.hkv;
  const int iters = (rows + kRows - 1) / kRows;
  // A warp per token; a token's rows over several warps while there are fewer
  // than 64 per SM, two for each place (a few tokens: a warp for each 32 lanes' rows).
  const int split = (int)std::min<long long>(iters, (64LL * sm_count() + tokens - 1) / tokens);
  const int per = (iters + split - 1) / split;
  p.tokens = tokens;
  p.part_rows = per * kRows;
  p.parts = (iters + per - 1) / per;
  const long long tasks = (long long)tokens * p.parts;
  const dim3 grid((unsigned)((tasks + pa::kNormRopeWarps - 1) / pa::kNormRopeWarps));
  return launch_ex(pa::norm_rope_kernel<T, D, APPEND>, grid, dim3(pa::kNormRopeWarps * 32), 0, st, true, p);
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
  if (p.q_out == p.q && p.q_out_stride != p.q_stride && num_tokens > 1) return PA_ERR_INVALID;
  if (!aligned(p.q_weight, 16) || !aligned(p.k_weight, 16)) return PA_ERR_INVALID;
  if (p.rotary > 0 && (!p.positions || !p.inv_freq)) return PA_ERR_INVALID;
  if (!aligned(p.positions, 4) || !aligned(p.inv_freq, 4)) return PA_ERR_INVALID;
  return PA_OK;
}

// ---- commit ---------------------------------------------------------------------------

bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// ---- tree attention -------------------------------------------------------------------

template <int D>
cudaError_t launch_tree_simt_t(TreeParams& p, cudaStream_t st) {
  constexpr int RT = pa::kTreeSimtRows, kWorkers = pa::kTreeSimtWarps * 32 / (D / 8);
  const int tiles = (p.tree_len * p.group + RT - 1) / RT;
  // Two CTAs fit on an SM: a range is split while some would have none, and every
  // worker keeps 4 tokens.  B200, 5 nodes x 4 heads x 8 kv heads of one 776-token
  // sequence: 20 us split in 8, 143 whole; 4 sequences of 200 tokens x 2 kv heads:
  // 12.0 split in 4 or 8, 13.7 split to one token a worker.  Above two CTAs an SM a
  // split loses (60 nodes x 8 heads x 4 kv heads x 2 of 822 tokens: 63 against 77 us).
  const long long ctas = (long long)tiles * p.hkv * p.batch;
  p.split = 1;
  while (p.split < pa::kTreeSimtCluster && ctas * p.split < 2LL * sm_count() && p.max_context >= 8LL * p.split * kWorkers)
    p.split *= 2;
  return launch_cluster(pa::decode_tree_simt_kernel<D>, dim3((unsigned)(tiles * p.split), p.hkv, p.batch), p.split,
                        dim3(pa::kTreeSimtWarps * 32), 0, st, true, p);
}

cudaError_t launch_tree_simt(TreeParams& p, int head_dim, cudaStream_t st) {
  switch (head_dim) {
    case 64:
      return launch_tree_simt_t<64>(p, st);
    case 128:
      return launch_tree_simt_t<128>(p, st);
    default:
      return launch_tree_simt_t<256>(p, st);
  }
}

// How the tensor-core kernel takes a call: one CTA per SM, for one row tile of
// whole nodes or (head_dim 64 and 128, where tensor memory holds two outputs)
// for two of them.  Workspace: behind the counter region of the split-K calls, which
// stays as it is, one record per (range, row tile) and two partials of `rows` rows
// for each.
struct TreePlan {
  int q_nodes, m_tiles, grid, rows, records;
  bool pair;
  size_t rec, o, ml, bytes;
};
TreePlan tree_plan(int head_dim, int tree_len, int group) {
  TreePlan w;
  w.q_nodes = std::min(tree_len, pa::kTreeRows / group);
  w.m_tiles = (tree_len + w.q_nodes - 1) / w.q_nodes;
  w.pair = w.m_tiles > 1 && head_dim <= 128;
  const int share = w.pair ? (w.m_tiles + 1) / 2 : w.m_tiles;  // CTAs that take the same range
  w.grid = std::max(1, sm_count() / share) * share;
  w.rows = (w.q_nodes * group + pa::kTreeCombineRows - 1) / pa::kTreeCombineRows * pa::kTreeCombineRows;
  w.records = w.grid / share * w.m_tiles;
  w.rec = pa::kCounterBytes;
  w.o = w.rec + align256((size_t)w.records * sizeof(int4));
  w.ml = w.o + align256(2 * (size_t)w.records * w.rows * head_dim * 4);
  w.bytes = w.ml + align256(2 * (size_t)w.records * w.rows * 2 * 4);
  return w;
}

// What a workspace for trees of tree_len nodes holds: what such a call needs, and every
// call with fewer nodes, heads per kv head or dims does, some of which have more
// records (32 nodes of 8 heads are two row tiles on every SM; 48 are three, and two
// CTAs share a range).  A call has at most one record an SM, or two with pairs of row tiles.
size_t tree_workspace_bytes(int head_dim, int tree_len, int group) {
  const size_t rows = (size_t)std::min(tree_len * group, pa::kTreeRows), sms = std::max(1, sm_count());
  const size_t padded = (rows + pa::kTreeCombineRows - 1) / pa::kTreeCombineRows * pa::kTreeCombineRows;
  const size_t records = tree_len * group > pa::kTreeRows ? 2 * sms : sms;
  const size_t columns = std::max(records * std::min(head_dim, 128), sms * head_dim);  // no pairs at head_dim 256
  return pa::kCounterBytes + align256(records * sizeof(int4)) + align256(2 * columns * padded * 4) +
         align256(2 * records * padded * 2 * 4);
}

// q as a 3-D tensor [batch * tree_len][num_q_heads][head_dim]; a box is 64
// columns (128 B) x one kv head's heads x the nodes of a row tile.
bool encode_q_map(CUtensorMap* map, const TreeParams& p, int head_dim) {
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)p.hq, (cuuint64_t)p.batch * p.tree_len};
  const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)p.hq * head_dim * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)p.q_nodes};
  const cuuint32_t estr[3] = {1, 1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int QR, bool PAIR>
cudaError_t launch_tree_t(const TreeParams& p, const TreePlan& w, cudaStream_t st) {
  using Cfg = pa::TreeCfg<D, QR, PAIR>;
  CUtensorMap qmap, kmap, vmap;
  const long long rows = (long long)p.num_blocks * p.hkv * p.block_size;
  if (!tensor_map_encoder() || !encode_q_map(&qmap, p, D) || !encode_cache_map(&kmap, p.k_cache, D, rows, 1 << p.log2_box) ||
      !encode_cache_map(&vmap, p.v_cache, D, rows, 1 << p.log2_box))
    return cudaErrorInvalidValue;
  auto kern = pa::decode_tree_kernel<D, QR, PAIR>;
  static std::atomic<uint64_t> smem_done{0};
  cudaError_t e = set_smem(kern, Cfg::kSmemBytes, smem_done);
  if (e != cudaSuccess) return e;
  e = launch_ex(kern, dim3(w.grid), dim3(pa::kTreeThreads), Cfg::kSmemBytes, st, true, qmap, kmap, vmap, p);
  if (e != cudaSuccess) return e;
  // 8 rows of a record a block, or 32 where the records that can be in use (one for
  // each unit at most) would make more than two waves of blocks so.  B200: 64 trees of
  // 8 nodes 26.4 us with 8 rows, 32.1 with 32; 7 trees of 39 nodes, with three times
  // the blocks, 32.2 with 8 and 25.8 with 32; one tree of 39 nodes on 22K keys (8 units of
  // 19 pieces) 42 with 8, 51 with 32.
  const long long cut = std::min<long long>(w.records, (long long)p.batch * p.hkv * w.m_tiles);
  const int row_blocks = w.rows / pa::kTreeCombineRows;
  const bool many = 2LL * D * cut * row_blocks > 2 * 2048LL * sm_count();
  const dim3 grid(w.records, many ? (row_blocks + 3) / 4 : row_blocks);
  return launch_ex(many ? pa::tree_combine_kernel<D, 4> : pa::tree_combine_kernel<D, 1>, grid, dim3(2 * D), 0, st, true, p);
}

cudaError_t launch_tree(const TreeParams& p, int head_dim, const TreePlan& w, cudaStream_t st) {
  switch (head_dim) {
    case 64:
      return w.pair ? launch_tree_t<64, 128, true>(p, w, st) : launch_tree_t<64, 128, false>(p, w, st);
    case 128:
      return w.pair ? launch_tree_t<128, 128, true>(p, w, st) : launch_tree_t<128, 128, false>(p, w, st);
    default:
      // Up to 64 rows of Q leave room for a third stage of K and of V (256 trees of 24
      // nodes 124 us, 131 with two; at head_dim 64 and 128 there are enough either way).
      return w.rows <= 64 ? launch_tree_t<256, 64, false>(p, w, st) : launch_tree_t<256, 128, false>(p, w, st);
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
      k_out_stride % (dtype == PA_F32 ? 4 : 8) || (k_out == k && k_out_stride != k_stride && num_tokens > 1))
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
  return tree_workspace_bytes(head_dim, tree_len, num_q_heads / num_kv_heads);
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
  if ((longest / pa::kTreeTile + 8) * num_kv_heads >= (1LL << 31)) return PA_ERR_UNSUPPORTED;  // a sequence's work in 32 bits
  if (batch == 0) return PA_OK;
  if (!tree_mask || !aligned(tree_mask, 8) || !aligned(tree_lens, 4)) return PA_ERR_INVALID;
  const bool tensor_cores = dtype == PA_BF16;
  const TreePlan w = tree_plan(head_dim, tree_len, num_q_heads / num_kv_heads);
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
  p.group = num_q_heads / num_kv_heads;
  p.block_size = block_size;
  p.log2_bs = ilog2(block_size);
  p.log2_box = std::min(p.log2_bs, ilog2(pa::kTreeTile));
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.window = window;
  p.max_context = max_context_len;
  p.q_nodes = w.q_nodes;
  p.m_tiles = w.m_tiles;
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
  if (launch_tree(p, head_dim, w, stream) != cudaSuccess) return PA_ERR_CUDA;
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
  // One CTA of a sequence writes its new length while the others may still read these.
  const size_t lens_bytes = 4 * (size_t)batch;
  if (new_lens && (overlap(new_lens, lens_bytes, context_lens, lens_bytes) ||
                   overlap(new_lens, lens_bytes, accept_lens, lens_bytes) ||
                   (tree_lens && overlap(new_lens, lens_bytes, tree_lens, lens_bytes)) ||
                   overlap(new_lens, lens_bytes, accepted, lens_bytes * max_accept) ||
                   overlap(new_lens, lens_bytes, block_tables, lens_bytes * max_blocks_per_seq)))
    return PA_ERR_INVALID;
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
