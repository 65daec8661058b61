// pa_plan_append and pa_tree_accept: the device-resident bookkeeping of a
// tree-speculation step.
//
// pa_plan_append is three exclusive sums over the requests -- blocks given
// back, blocks needed, tokens -- and index arithmetic on them: the k-th block
// handed out is entry F + R - 1 - k of the free stack (F free before, R given
// back), so no request waits for another one's pop.  One CTA does all of it.
//
// pa_tree_accept moves rows of the pool.  A thread owns one 16-byte column of
// the rows of one request and walks the path in order: step i writes row i
// and reads row path[i] >= i, so no row is written before it is read, without
// any barrier.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct PlanArgs {
  int32_t* block_tables;
  const int32_t* blocks_held;
  int32_t* free_blocks;
  const int32_t* num_free;
  const int32_t* seq_lens;
  const int32_t* new_tokens;
  const int32_t* depths;
  int depths_stride;
  int64_t* slots;
  int32_t* positions;
  int32_t* token_starts;
  int32_t* seq_lens_out;
  int32_t* blocks_held_out;
  int32_t* num_free_out;
  int32_t* appended_out;
  int32_t* status_out;
  int batch, max_new, num_slots, num_blocks, block_size, max_blocks;
  int32_t* err;
};

constexpr int kPlanThreads = 1024;

struct Sums {
  long long back, need, tokens;
};

// What request b gives back, needs and appends; `bad` collects its checks.
__device__ __forceinline__ Sums plan_request(const PlanArgs& a, int b, int& len, int& held, int& c, bool& bad) {
  len = a.seq_lens[b];
  held = a.blocks_held[b];
  c = a.new_tokens[b];
  Sums s{0, 0, 0};
  const long long end = static_cast<long long>(len) + max(c, 0);
  if (len < 0 || held < 0 || held > a.max_blocks || end > static_cast<long long>(a.max_blocks) * a.block_size ||
      (a.max_new > 0 && c > a.max_new)) {
    bad = true;
    return s;
  }
  if (c < 0) {
    s.back = held;
  } else {
    s.need = max(0ll, (end + a.block_size - 1) / a.block_size - held);
    s.tokens = c;
  }
  return s;
}

__device__ __forceinline__ long long warp_inclusive(long long v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(kFull, v, off);
    if (lane >= off) v += y;
  }
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) plan_append_kernel(const PlanArgs a) {
  __shared__ long long part[3][32];
  __shared__ int any_bad;
  pdl_trigger();
  if (threadIdx.x == 0) any_bad = 0;
  pdl_wait();
  __syncthreads();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int per = (a.batch + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(a.batch, t * per), hi = min(a.batch, lo + per);
  Sums mine{0, 0, 0};
  bool bad = false;
  for (int b = lo; b < hi; ++b) {
    int len, held, c;
    const Sums s = plan_request(a, b, len, held, c, bad);
    mine.back += s.back;
    mine.need += s.need;
    mine.tokens += s.tokens;
  }
  if (bad) any_bad = 1;
  Sums incl{warp_inclusive(mine.back, lane), warp_inclusive(mine.need, lane), warp_inclusive(mine.tokens, lane)};
  if (lane == 31) {
    part[0][warp] = incl.back;
    part[1][warp] = incl.need;
    part[2][warp] = incl.tokens;
  }
  __syncthreads();
  if (warp < 3) {
    const long long v = warp_inclusive(part[warp][lane], lane);
    part[warp][lane] = v;
  }
  __syncthreads();
  const long long back = part[0][31], need = part[1][31], tokens = part[2][31];
  const int first = a.num_free[0];
  int status = 0;
  if (any_bad || first < 0 || first + back > a.num_blocks || tokens > a.num_slots) status = PA_DEVERR_PLAN;
  else if (need > first + back) status = PA_DEVERR_NO_BLOCKS;
  Sums at{incl.back - mine.back, incl.need - mine.need, incl.tokens - mine.tokens};
  if (warp > 0) {
    at.back += part[0][warp - 1];
    at.need += part[1][warp - 1];
    at.tokens += part[2][warp - 1];
  }
  if (t == 0) {
    if (status != 0) flag_error(a.err, status);
    if (a.status_out != nullptr) *a.status_out = status;
    if (a.token_starts != nullptr) a.token_starts[a.batch] = status ? 0 : static_cast<int>(tokens);
  }
  // returned blocks go on the stack before any block is taken from it
  if (status == 0 && back > 0) {
    long long to = first + at.back;
    for (int b = lo; b < hi; ++b)
      if (a.new_tokens[b] < 0)
        for (int i = 0; i < a.blocks_held[b]; ++i) a.free_blocks[to++] = a.block_tables[static_cast<size_t>(b) * a.max_blocks + i];
  }
  __syncthreads();  // every input of the state has been read, the stack is complete
  long long from = first + back - 1 - at.need;
  long long start = at.tokens;
  for (int b = lo; b < hi; ++b) {
    int len, held, c;
    bool ignored = false;
    const Sums s = plan_request(a, b, len, held, c, ignored);
    if (status == 0) {
      for (int i = 0; i < s.need; ++i) a.block_tables[static_cast<size_t>(b) * a.max_blocks + held + i] = a.free_blocks[from--];
      len = c < 0 ? 0 : len + c;
      held = c < 0 ? 0 : held + static_cast<int>(s.need);
    }
    if (a.token_starts != nullptr) a.token_starts[b] = status ? 0 : static_cast<int>(start);
    start += s.tokens;
    a.seq_lens_out[b] = len;
    a.blocks_held_out[b] = held;
    if (a.appended_out != nullptr) a.appended_out[b] = status ? 0 : static_cast<int>(s.tokens);
  }
  if (t == 0) *a.num_free_out = status ? first : static_cast<int>(first + back - need);
  __syncthreads();
  // the slots: positions follow from the new length and the count
  for (int i = t; i < a.num_slots; i += kPlanThreads) {
    int b = 0, off = 0;
    bool inside;
    if (a.max_new > 0) {
      b = i / a.max_new;
      off = i - b * a.max_new;
      inside = off < a.new_tokens[b];
    } else {
      inside = i < a.token_starts[a.batch];
      int up = a.batch - 1;  // the largest b with token_starts[b] <= i
      while (b < up) {
        const int mid = (b + up + 1) >> 1;
        if (a.token_starts[mid] <= i) b = mid;
        else up = mid - 1;
      }
      off = i - a.token_starts[b];
    }
    long long slot = -1;
    int pos = -1;
    if (inside && status == 0) {
      const int base = a.seq_lens_out[b] - a.new_tokens[b];
      pos = base + off;
      const int block = a.block_tables[static_cast<size_t>(b) * a.max_blocks + pos / a.block_size];
      if (static_cast<unsigned>(block) < static_cast<unsigned>(a.num_blocks))
        slot = static_cast<long long>(block) * a.block_size + pos % a.block_size;
      else
        flag_error(a.err, PA_DEVERR_BLOCK_ID);
      if (a.depths != nullptr) pos = base + a.depths[static_cast<size_t>(b) * a.depths_stride + off];
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
}

constexpr int kAcceptThreads = 256;
constexpr int kAcceptBatch = 8;  // path steps in flight per thread

struct AcceptArgs {
  uint4* pool;
  const int32_t* path;
  const int32_t* accept_lens;
  const int32_t* tree_lens;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  int32_t* seq_lens_out;
  int num_nodes, max_path, num_blocks, num_kv_heads, block_size, chunks, max_blocks;
  int32_t* err;
};

// One CTA per request.
__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const AcceptArgs a) {
  extern __shared__ int64_t rows[];  // [max_path] source, [max_path] target: element offset of the key row of head 0
  __shared__ int bad;
  pdl_trigger();
  if (threadIdx.x == 0) bad = 0;
  pdl_wait();
  __syncthreads();
  const int b = blockIdx.x, t = threadIdx.x;
  const int len = a.seq_lens[b];
  const int n = a.tree_lens != nullptr ? a.tree_lens[b] : a.num_nodes;
  const int acc = a.accept_lens[b];
  if (len == 0) {  // an empty request
    if (t == 0 && a.seq_lens_out != nullptr) a.seq_lens_out[b] = 0;
    return;
  }
  int reason = 0;
  if (len < 0 || len > static_cast<long long>(a.max_blocks) * a.block_size || n < 0 || n > a.num_nodes || n > len ||
      acc < 0 || acc > n || acc > a.max_path) {
    reason = PA_DEVERR_TREE;
  } else {
    const int base = len - n;
    const int32_t* path = a.path + static_cast<size_t>(b) * a.max_path;
    const int32_t* table = a.block_tables + static_cast<size_t>(b) * a.max_blocks;
    for (int i = t; i < acc; i += kAcceptThreads) {
      const int from = path[i];
      const int before = i > 0 ? path[i - 1] : -1;
      if (from <= before || from >= n || from < 0) {
        reason = PA_DEVERR_TREE;
        break;
      }
      const int ends[2] = {base + from, base + i};
      for (int e = 0; e < 2; ++e) {
        const int block = table[ends[e] / a.block_size];
        if (static_cast<unsigned>(block) >= static_cast<unsigned>(a.num_blocks)) reason |= PA_DEVERR_BLOCK_ID;
        rows[e * a.max_path + i] = (static_cast<int64_t>(block) * 2 * a.num_kv_heads * a.block_size + ends[e] % a.block_size) * a.chunks;
      }
    }
  }
  if (reason) {
    flag_error(a.err, reason);
    bad = 1;
  }
  __syncthreads();
  if (!bad) {
    const int columns = 2 * a.num_kv_heads * a.chunks;
    for (int col = t; col < columns; col += kAcceptThreads) {
      // (k/v, head, chunk): heads and k/v planes are block_size rows apart
      const int64_t at = static_cast<int64_t>(col / a.chunks) * a.block_size * a.chunks + col % a.chunks;
      for (int i0 = 0; i0 < acc; i0 += kAcceptBatch) {
        uint4 v[kAcceptBatch];
#pragma unroll
        for (int i = 0; i < kAcceptBatch; ++i)
          if (i0 + i < acc) v[i] = a.pool[rows[i0 + i] + at];
#pragma unroll
        for (int i = 0; i < kAcceptBatch; ++i)
          if (i0 + i < acc && rows[i0 + i] != rows[a.max_path + i0 + i]) a.pool[rows[a.max_path + i0 + i] + at] = v[i];
      }
    }
  }
  if (t == 0 && a.seq_lens_out != nullptr) a.seq_lens_out[b] = bad ? len : len - n + acc;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace
}  // namespace pa

extern "C" {

int pa_plan_append(int32_t* block_tables, const int32_t* blocks_held, int32_t* free_blocks, const int32_t* num_free,
                   const int32_t* seq_lens, const int32_t* new_tokens, const int32_t* depths, int depths_stride,
                   int64_t* slot_mapping, int32_t* positions, int32_t* token_starts, int32_t* seq_lens_out,
                   int32_t* blocks_held_out, int32_t* num_free_out, int32_t* appended_out, int32_t* status_out,
                   int batch, int max_new_tokens, int num_slots, int num_blocks, int block_size, int max_blocks_per_seq,
                   void* stream) {
  using namespace pa;
  if (batch < 0 || max_new_tokens < 0 || num_slots < 0 || num_blocks <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || depths_stride < 0)
    return fail(PA_ERR_INVALID, "pa_plan_append: non-positive size");
  if (batch > (1 << 20) || num_slots > (1 << 30))
    return fail(PA_ERR_UNSUPPORTED, "pa_plan_append: batch %d beyond %d or num_slots %d beyond %d", batch, 1 << 20,
                num_slots, 1 << 30);
  if (static_cast<int64_t>(max_blocks_per_seq) * block_size > 0x7fffffffll)
    return fail(PA_ERR_UNSUPPORTED, "pa_plan_append: a table row of more than 2^31 - 1 positions");
  if (max_new_tokens > 0 && static_cast<int64_t>(batch) * max_new_tokens != num_slots)
    return fail(PA_ERR_INVALID, "pa_plan_append: the padded layout has batch * max_new_tokens = %lld slots, not %d",
                static_cast<long long>(batch) * max_new_tokens, num_slots);
  if (depths != nullptr && (max_new_tokens == 0 || (depths_stride != 0 && depths_stride < max_new_tokens)))
    return fail(PA_ERR_INVALID, "pa_plan_append: depths need the padded layout and a stride of 0 or >= max_new_tokens");
  if (batch == 0) return PA_OK;
  if (!block_tables || !blocks_held || !free_blocks || !num_free || !seq_lens || !new_tokens || !seq_lens_out ||
      !blocks_held_out || !num_free_out || (num_slots > 0 && (!slot_mapping || !positions)) ||
      (max_new_tokens == 0 && !token_starts))
    return fail(PA_ERR_INVALID, "pa_plan_append: NULL pointer");
  for (const void* p : {static_cast<const void*>(block_tables), static_cast<const void*>(blocks_held),
                        static_cast<const void*>(free_blocks), static_cast<const void*>(num_free),
                        static_cast<const void*>(seq_lens), static_cast<const void*>(new_tokens),
                        static_cast<const void*>(depths), static_cast<const void*>(positions),
                        static_cast<const void*>(token_starts), static_cast<const void*>(seq_lens_out),
                        static_cast<const void*>(blocks_held_out), static_cast<const void*>(num_free_out),
                        static_cast<const void*>(appended_out), static_cast<const void*>(status_out)})
    if (!aligned(p, 4)) return fail(PA_ERR_INVALID, "pa_plan_append: misaligned pointer");
  if (!aligned(slot_mapping, 8)) return fail(PA_ERR_INVALID, "pa_plan_append: misaligned pointer");
  int32_t* err = device_error_word();
  if (err == nullptr) return PA_ERR_CUDA;
  const PlanArgs a{block_tables, blocks_held,  free_blocks,     num_free,     seq_lens,   new_tokens, depths,
                   depths_stride, slot_mapping, positions,       token_starts, seq_lens_out, blocks_held_out,
                   num_free_out, appended_out, status_out, batch,           max_new_tokens, num_slots, num_blocks, block_size,
                   max_blocks_per_seq, err};
  PA_CUDA_TRY(launch_pdl(plan_append_kernel, dim3(1), dim3(kPlanThreads), 0, static_cast<cudaStream_t>(stream), a));
  return PA_OK;
}

int pa_tree_accept(pa_bf16* kv_pool, const int32_t* path, const int32_t* accept_lens, const int32_t* tree_lens,
                   const int32_t* block_tables, const int32_t* seq_lens, int32_t* seq_lens_out, int batch,
                   int num_nodes, int max_path, int num_blocks, int num_kv_heads, int block_size, int head_dim,
                   int max_blocks_per_seq, void* stream) {
  using namespace pa;
  if (batch < 0 || num_nodes < 0 || max_path < 0 || num_blocks <= 0 || num_kv_heads <= 0 || block_size <= 0 ||
      head_dim <= 0 || max_blocks_per_seq <= 0)
    return fail(PA_ERR_INVALID, "pa_tree_accept: non-positive size");
  if (head_dim % 8 != 0) return fail(PA_ERR_INVALID, "pa_tree_accept: head_dim %d not a multiple of 8", head_dim);
  if (max_path > 1024) return fail(PA_ERR_UNSUPPORTED, "pa_tree_accept: max_path %d beyond 1024", max_path);
  if (batch == 0) return PA_OK;
  if (!kv_pool || !accept_lens || !block_tables || !seq_lens || (max_path > 0 && !path))
    return fail(PA_ERR_INVALID, "pa_tree_accept: NULL pointer");
  if (!aligned(kv_pool, 16)) return fail(PA_ERR_INVALID, "pa_tree_accept: misaligned pointer");
  for (const int32_t* p : {path, accept_lens, tree_lens, block_tables, seq_lens, static_cast<const int32_t*>(seq_lens_out)})
    if (!aligned(p, 4)) return fail(PA_ERR_INVALID, "pa_tree_accept: misaligned pointer");
  int32_t* err = device_error_word();
  if (err == nullptr) return PA_ERR_CUDA;
  const AcceptArgs a{reinterpret_cast<uint4*>(kv_pool), path, accept_lens, tree_lens, block_tables, seq_lens,
                     seq_lens_out, num_nodes, max_path, num_blocks, num_kv_heads, block_size, head_dim / 8,
                     max_blocks_per_seq, err};
  const size_t smem = static_cast<size_t>(max_path) * 2 * sizeof(int64_t);
  PA_CUDA_TRY(launch_pdl(tree_accept_kernel, dim3(static_cast<unsigned>(batch)), dim3(kAcceptThreads), smem,
                         static_cast<cudaStream_t>(stream), a));
  return PA_OK;
}

}  // extern "C"
