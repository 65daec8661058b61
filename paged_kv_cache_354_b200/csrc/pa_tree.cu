// pa_decode_tree: attention of a tree of drafted tokens over the paged cache.
//
//   out[b][t][j] = softmax_{p in A(t)}(scale q[b][t][j] . K[p]) V[p],
//   A(t) = [0, L - n) and the tree nodes whose bit is set in t's mask row
//
// One warp per (request, node, query head): lanes share the head dimension,
// the positions are walked one after the other with an online softmax.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

struct TreeArgs {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const __nv_bfloat16* pool;
  const uint32_t* mask;
  int64_t mask_stride;  // words from one request's rows to the next one's (0: shared)
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* tree_lens;
  int32_t* err;
  int batch, nodes, words, num_q_heads, num_kv_heads, group;
  int num_blocks, max_blocks, max_seq_len, block_size;
  float scale_log2;
};

// Length and node count of request b after the device checks; n = 0 where
// the request has no (valid) tree.
__device__ __forceinline__ void tree_lengths(const TreeArgs& a, int b, bool report, int& len, int& n) {
  const int raw = a.seq_lens[b];
  const long long cap = min(static_cast<long long>(a.max_blocks) * a.block_size, static_cast<long long>(a.max_seq_len));
  len = static_cast<int>(min(static_cast<long long>(max(raw, 0)), cap));
  if (len != raw && report) flag_error(a.err, PA_DEVERR_SEQ_LEN);
  n = a.tree_lens != nullptr ? a.tree_lens[b] : a.nodes;
  if (len == 0) {
    n = 0;
  } else if (n < 0 || n > a.nodes || n > len) {
    if (report) flag_error(a.err, PA_DEVERR_TREE);
    n = 0;
  }
}

constexpr int kTreeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kTreeWarps) tree_rows_kernel(const TreeArgs a) {
  constexpr int kPer = D / 32;  // elements per lane
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kTreeWarps + (threadIdx.x >> 5);
  const int64_t rows = static_cast<int64_t>(a.batch) * a.nodes * a.num_q_heads;
  if (row >= rows) return;
  const int j = static_cast<int>(row % a.num_q_heads);
  const int t = static_cast<int>(row / a.num_q_heads % a.nodes);
  const int b = static_cast<int>(row / a.num_q_heads / a.nodes);
  const int h = j / a.group;
  int len, n;
  tree_lengths(a, b, t == 0 && j == 0 && lane == 0, len, n);
  float q[kPer], o[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    q[e] = __bfloat162float(a.q[row * D + lane * kPer + e]) * a.scale_log2;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  if (t < n) {
    const uint32_t* mask = a.mask + b * a.mask_stride + static_cast<int64_t>(t) * a.words;
    const int base = len - n;
    for (int p = 0; p < len; ++p) {
      const int i = p - base;
      if (i >= 0 && !((mask[i >> 5] >> (i & 31)) & 1u)) continue;
      const int block = a.block_tables[static_cast<int64_t>(b) * a.max_blocks + p / a.block_size];
      const bool real = static_cast<unsigned>(block) < static_cast<unsigned>(a.num_blocks);
      if (!real && lane == 0) flag_error(a.err, PA_DEVERR_BLOCK_ID);
      const int64_t at =
          ((static_cast<int64_t>(block) * 2 * a.num_kv_heads + h) * a.block_size + p % a.block_size) * D + lane * kPer;
      const int64_t to_values = static_cast<int64_t>(a.num_kv_heads) * a.block_size * D;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) s += q[e] * (real ? __bfloat162float(a.pool[at + e]) : 0.f);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      const float mn = fmaxf(m, s);
      const float keep = m == -INFINITY ? 0.f : exp2f(m - mn);
      const float w = exp2f(s - mn);
      m = mn;
      l = l * keep + w;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] = o[e] * keep + w * (real ? __bfloat162float(a.pool[at + to_values + e]) : 0.f);
    }
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) a.out[row * D + lane * kPer + e] = __float2bfloat16_rn(o[e] * inv);
}

int check_tree_shape(const char* who, int batch, int nodes, int hq, int hkv, int d, int bs, int max_seq_len) {
  if (batch < 0 || nodes <= 0 || hq <= 0 || hkv <= 0 || max_seq_len < 0)
    return fail(PA_ERR_INVALID, "%s: non-positive size", who);
  if (hq % hkv != 0) return fail(PA_ERR_INVALID, "%s: %d query heads are no multiple of %d KV heads", who, hq, hkv);
  if (d != 64 && d != 128) return fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d", who, d);
  if (bs != 16 && bs != 32) return fail(PA_ERR_UNSUPPORTED, "%s: block_size %d", who, bs);
  if (hq / hkv > 64) return fail(PA_ERR_UNSUPPORTED, "%s: group size %d beyond 64", who, hq / hkv);
  if (nodes > 1024) return fail(PA_ERR_UNSUPPORTED, "%s: %d nodes beyond 1024", who, nodes);
  if (batch > 32768) return fail(PA_ERR_UNSUPPORTED, "%s: batch %d beyond 32768", who, batch);
  return PA_OK;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace
}  // namespace pa

extern "C" {

int pa_decode_tree_workspace_size(int batch, int num_nodes, int num_q_heads, int num_kv_heads, int head_dim,
                                  int block_size, int max_seq_len, size_t* bytes_out) {
  using namespace pa;
  if (bytes_out == nullptr) return fail(PA_ERR_INVALID, "pa_decode_tree_workspace_size: bytes_out is NULL");
  const int rc = check_tree_shape("pa_decode_tree_workspace_size", batch, num_nodes, num_q_heads, num_kv_heads,
                                  head_dim, block_size, max_seq_len);
  if (rc != PA_OK) return rc;
  *bytes_out = 256;
  return PA_OK;
}

int pa_decode_tree(pa_bf16* out, const pa_bf16* q, const pa_bf16* kv_pool, const uint32_t* tree_mask,
                   int mask_per_request, const int32_t* block_tables, const int32_t* seq_lens,
                   const int32_t* tree_lens, int batch, int num_nodes, int num_q_heads, int num_kv_heads,
                   int head_dim, int block_size, int num_blocks, int max_blocks_per_seq, int max_seq_len, float scale,
                   void* workspace, size_t workspace_bytes, void* stream) {
  using namespace pa;
  const char* who = "pa_decode_tree";
  int rc = check_tree_shape(who, batch, num_nodes, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len);
  if (rc != PA_OK) return rc;
  if (num_blocks <= 0 || max_blocks_per_seq <= 0) return fail(PA_ERR_INVALID, "%s: non-positive size", who);
  if (batch == 0) return PA_OK;
  if (!out || !q || !kv_pool || !tree_mask || !block_tables || !seq_lens || !workspace)
    return fail(PA_ERR_INVALID, "%s: NULL pointer", who);
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(kv_pool, 16) || !aligned(tree_mask, 4) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(tree_lens, 4) || !aligned(workspace, 256))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", who);
  size_t need = 0;
  rc = pa_decode_tree_workspace_size(batch, num_nodes, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len, &need);
  if (rc != PA_OK) return rc;
  if (workspace_bytes < need)
    return fail(PA_ERR_INVALID, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes, need);
  rc = check_output_pointer(out, who);
  if (rc != PA_OK) return rc;
  int32_t* err = device_error_word();
  if (err == nullptr) return PA_ERR_CUDA;
  TreeArgs a;
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.pool = reinterpret_cast<const __nv_bfloat16*>(kv_pool);
  a.mask = tree_mask;
  a.words = (num_nodes + 31) / 32;
  a.mask_stride = mask_per_request ? static_cast<int64_t>(num_nodes) * a.words : 0;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.tree_lens = tree_lens;
  a.err = err;
  a.batch = batch;
  a.nodes = num_nodes;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.group = num_q_heads / num_kv_heads;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.max_seq_len = max_seq_len;
  a.block_size = block_size;
  a.scale_log2 = scale * 1.4426950408889634f;
  const int64_t rows = static_cast<int64_t>(batch) * num_nodes * num_q_heads;
  const dim3 grid(static_cast<unsigned>((rows + kTreeWarps - 1) / kTreeWarps));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (head_dim == 128) PA_CUDA_TRY(launch_pdl(tree_rows_kernel<128>, grid, dim3(32 * kTreeWarps), 0, st, a));
  else PA_CUDA_TRY(launch_pdl(tree_rows_kernel<64>, grid, dim3(32 * kTreeWarps), 0, st, a));
  return PA_OK;
}

}  // extern "C"
