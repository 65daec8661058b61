// pa_plan_append and pa_tree_accept: the device-resident bookkeeping of a
// tree-speculation step.
//
// pa_plan_append is three exclusive sums over the requests -- blocks given
// back, blocks needed, tokens -- and index arithmetic on them: the k-th block
// handed out is entry F + R - 1 - k of the free stack (F free before, R given
// back), so no request waits for another one's pop.  Latency is all the cost:
// a decoding step is one CTA, and its barriers and dependent loads take the
// time (64 requests of 16 tokens: 5.2 us, 15 KB).  From kPlanSpread slots or
// kPlanMany requests on a cluster of 8 shares the requests and exchanges its
// sums through distributed shared memory, and a packed call of that size
// leaves its slots to a second, wide launch (1000 requests, 256k slots: 328 us
// on one CTA, 66 us when the cluster wrote the slots, 13.2 us so; floor 0.6 us).
//
// pa_tree_accept moves rows of the pool.  A thread owns one 16-byte column of
// the rows of one request and walks the path in order: step i writes row i
// and reads row path[i] >= i, so no row is written before it is read, without
// any barrier.  Bytes bound it when there are many rows: kAcceptBatch steps of
// a thread are in flight at once, and 600 paths of up to 16 rows of 4 KB (39
// MB) move in 8.4 us, 4.6 TB/s; 64 paths of up to 6 take 2.6 us.
//
// Neither lets the next kernel start early.  The decodes and the cache write
// read tables, lengths and slots through the read-only path, so they must not
// be resident while these are written.  That costs nothing: a captured step of
// 4 trees of 8 takes 24.3 us (26.4 with early starts), of 64 of 16 126 us (126).
#include <cooperative_groups.h>
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
constexpr int kPlanCluster = 8;
constexpr int kPlanSpread = 4096;  // slots, or
constexpr int kPlanMany = 2048;    // requests, from which a cluster is used

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

// Every lane's run of `count` entries, from src on upwards (dir 1) or downwards
// (-1), to dst on: eight lanes to a run, four runs at a time, kRunDepth entries
// per lane in flight.  (A warp to a run waits for memory once per run: the
// whole call 16.8 us where this took 14.4 in the case above; all runs in one
// line, each lane looking up the owner of its entries, 15.9.)
constexpr int kRunDepth = 8;

__device__ __forceinline__ void copy_runs(int count, const int32_t* src, int dir, int32_t* dst, int lane) {
  unsigned any = __ballot_sync(kFull, count > 0);
  any |= any >> 16;
  any |= any >> 8;  // bit r: some owner is lane r, 8 + r, 16 + r or 24 + r
#pragma unroll 1
  for (any &= 0xffu; any != 0; any &= any - 1) {
    const int owner = (lane & 24) + __ffs(any) - 1;
    const unsigned n = __shfl_sync(kFull, count, owner);
    const int32_t* from = reinterpret_cast<const int32_t*>(__shfl_sync(kFull, reinterpret_cast<uintptr_t>(src), owner));
    int32_t* to = reinterpret_cast<int32_t*>(__shfl_sync(kFull, reinterpret_cast<uintptr_t>(dst), owner));
    for (unsigned x0 = lane & 7; x0 < n; x0 += 8 * kRunDepth) {
      int32_t v[kRunDepth];
#pragma unroll
      for (int u = 0; u < kRunDepth; ++u)
        if (x0 + 8 * u < n) v[u] = __ldcg(from + dir * static_cast<int64_t>(x0 + 8 * u));
#pragma unroll
      for (int u = 0; u < kRunDepth; ++u)
        if (x0 + 8 * u < n) to[x0 + 8 * u] = v[u];
    }
  }
}

// Entry of a slot: position p of a request whose tokens begin at `base`.
__device__ __forceinline__ void write_slot(const PlanArgs& a, int64_t i, int b, int base, int off) {
  const int p = base + off;
  const int block = __ldcg(a.block_tables + static_cast<int64_t>(b) * a.max_blocks + p / a.block_size);
  int64_t slot = -1;
  if (static_cast<unsigned>(block) < static_cast<unsigned>(a.num_blocks))
    slot = static_cast<int64_t>(block) * a.block_size + p % a.block_size;
  else
    flag_error(a.err, PA_DEVERR_BLOCK_ID);
  a.slots[i] = slot;
  a.positions[i] = a.depths != nullptr ? base + a.depths[static_cast<int64_t>(b) * a.depths_stride + off] : p;
}

// kRanks CTAs (a cluster when more than one); kSlots: this launch writes the slots.
template <int kRanks, bool kSlots>
__global__ void __launch_bounds__(kPlanThreads) plan_append_kernel(const PlanArgs a) {
  namespace cg = cooperative_groups;
  __shared__ long long part[3][32];
  __shared__ long long mine_total[4];  // of this CTA: back, need, tokens, bad
  __shared__ long long totals[kRanks][4];
  // a single CTA keeps what its slots follow from
  constexpr int kKept = kRanks == 1 ? kPlanMany : 1;
  __shared__ int kept_len[kKept], kept_count[kKept], kept_start[kKept];
  auto sync_all = []() {
    if constexpr (kRanks > 1) cg::this_cluster().sync();
    else __syncthreads();
  };
  int rank = 0;
  if constexpr (kRanks > 1) rank = static_cast<int>(cg::this_cluster().block_rank());
  if (!kSlots && a.num_slots > 0) pdl_trigger();  // for the slots kernel, which waits
  pdl_wait();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  // this thread's requests, a run of them; few requests are spread over all
  // warps, which take turns at the blocks of theirs
  const int share = (a.batch + kRanks - 1) / kRanks;  // of the CTA
  const int per = (share + kPlanThreads - 1) / kPlanThreads;
  const int spread = per > 1 ? 1 : kPlanThreads / max(share, 1);
  const int end = min(a.batch, (rank + 1) * share);
  const int lo = t % spread == 0 ? min(end, rank * share + t / spread * per) : end;
  const int hi = min(end, lo + per);
  Sums mine{0, 0, 0};
  bool bad = false;
  for (int b = lo; b < hi; ++b) {
    int len, held, c;
    const Sums s = plan_request(a, b, len, held, c, bad);
    mine.back += s.back;
    mine.need += s.need;
    mine.tokens += s.tokens;
  }
  const int first = a.num_free[0];
  const Sums incl{warp_inclusive(mine.back, lane), warp_inclusive(mine.need, lane), warp_inclusive(mine.tokens, lane)};
  if (lane == 31) {
    part[0][warp] = incl.back;
    part[1][warp] = incl.need;
    part[2][warp] = incl.tokens;
  }
  const int any_bad = __syncthreads_or(bad);
  if (warp < 3) {
    const long long v = warp_inclusive(part[warp][lane], lane);
    part[warp][lane] = v;
    if (lane == 31) mine_total[warp] = v;
  } else if (warp == 3 && lane == 0) {
    mine_total[3] = any_bad;
  }
  sync_all();
  Sums at{incl.back - mine.back, incl.need - mine.need, incl.tokens - mine.tokens};
  if (warp > 0) {
    at.back += part[0][warp - 1];
    at.need += part[1][warp - 1];
    at.tokens += part[2][warp - 1];
  }
  if constexpr (kRanks > 1) {  // one remote load per CTA and sum (one per thread: 18.0 us, so 16.8)
    if (t < 4 * kRanks) totals[t >> 2][t & 3] = cg::this_cluster().map_shared_rank(mine_total, t >> 2)[t & 3];
    __syncthreads();
  }
  long long back = 0, need = 0, tokens = 0, wrong = 0;
#pragma unroll
  for (int r = 0; r < kRanks; ++r) {
    const long long* other = kRanks > 1 ? totals[r] : mine_total;
    if (r < rank) {
      at.back += other[0];
      at.need += other[1];
      at.tokens += other[2];
    }
    back += other[0];
    need += other[1];
    tokens += other[2];
    wrong += other[3];
  }
  int status = 0;
  if (wrong || first < 0 || first + back > a.num_blocks || tokens > a.num_slots) status = PA_DEVERR_PLAN;
  else if (need > first + back) status = PA_DEVERR_NO_BLOCKS;
  // returned blocks go on the stack before any block is taken from it
  if (status == 0 && back > 0) {
    long long to = first + at.back;
    for (int i = 0; i < per; ++i) {
      const int b = lo + i;
      const int count = b < hi && a.new_tokens[b] < 0 ? a.blocks_held[b] : 0;
      copy_runs(count, a.block_tables + static_cast<int64_t>(b) * a.max_blocks, 1, a.free_blocks + to, lane);
      to += count;
    }
  }
  sync_all();  // every input of the state has been read, the stack is complete
  long long from = first + back - 1 - at.need;
  long long start = at.tokens;
  for (int i = 0; i < per; ++i) {
    const int b = lo + i;
    int len = 0, held = 0, c = 0;
    bool ignored = false;
    Sums s{0, 0, 0};
    if (b < hi) s = plan_request(a, b, len, held, c, ignored);
    const int count = status == 0 ? static_cast<int>(s.need) : 0;
    // a few blocks by the request's own thread (a step's), many by its warp
    constexpr int kFew = 4;
    if (count <= kFew) {
#pragma unroll
      for (int x = 0; x < kFew; ++x)
        if (x < count) a.block_tables[static_cast<int64_t>(b) * a.max_blocks + held + x] = __ldcg(a.free_blocks + from - x);
    }
    copy_runs(count > kFew ? count : 0, a.free_blocks + from, -1,
              a.block_tables + static_cast<int64_t>(b) * a.max_blocks + held, lane);
    from -= count;
    if (b < hi) {
      if constexpr (kRanks == 1) {
        kept_len[b] = len;
        kept_count[b] = status == 0 ? static_cast<int>(s.tokens) : 0;
        kept_start[b] = status == 0 ? static_cast<int>(start) : 0;
      }
      if (status == 0) {
        len = c < 0 ? 0 : len + c;
        held = c < 0 ? 0 : held + count;
      }
      if (a.token_starts != nullptr) a.token_starts[b] = status ? 0 : static_cast<int>(start);
      start += s.tokens;
      a.seq_lens_out[b] = len;
      a.blocks_held_out[b] = held;
      if (a.appended_out != nullptr) a.appended_out[b] = status ? 0 : static_cast<int>(s.tokens);
    }
  }
  if (rank == 0 && t == 0) {
    if (status != 0) flag_error(a.err, status);
    if (a.status_out != nullptr) *a.status_out = status;
    if (a.token_starts != nullptr) a.token_starts[a.batch] = status ? 0 : static_cast<int>(tokens);
    *a.num_free_out = status ? first : static_cast<int>(first + back - need);
  }
  if constexpr (kRanks > 1) cg::this_cluster().sync();  // no CTA leaves while its sums are read
  if constexpr (kSlots) {
    __syncthreads();  // tables and lengths are written
    for (int64_t i = rank * kPlanThreads + t; i < a.num_slots; i += kRanks * kPlanThreads) {
      int b = 0, off;
      if (a.max_new > 0) {
        b = static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(a.max_new));
        off = static_cast<int>(i - static_cast<int64_t>(b) * a.max_new);
      } else if constexpr (kRanks == 1) {
        int up = a.batch - 1;  // the largest b that begins at or before i
        while (b < up) {
          const int mid = (b + up + 1) >> 1;
          if (kept_start[mid] <= i) b = mid;
          else up = mid - 1;
        }
        off = static_cast<int>(i - kept_start[b]);
      } else {
        off = 0x7fffffff;  // (a large packed call has its own kernel)
      }
      int c, base;
      if constexpr (kRanks == 1) {
        c = kept_count[b];
        base = kept_len[b];
      } else {  // other CTAs wrote it: past the L1 cache
        c = status == 0 ? a.new_tokens[b] : 0;
        base = __ldcg(a.seq_lens_out + b) - c;
      }
      if (off < c) {
        write_slot(a, i, b, base, off);
      } else {
        a.slots[i] = -1;
        a.positions[i] = -1;
      }
    }
  }
}

// The slots of a large packed call, one per thread.  A refused call has no
// tokens: its starts are all 0.
constexpr int kSlotThreads = 256;

__global__ void __launch_bounds__(kSlotThreads) plan_slots_kernel(const PlanArgs a) {
  __shared__ int starts[kSlotThreads + 1];
  pdl_wait();
  const int t = threadIdx.x, lane = t & 31;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSlotThreads, i = i0 + t;
  const int tokens = a.token_starts[a.batch];
  if (i0 >= tokens) {
    if (i < a.num_slots) {
      a.slots[i] = -1;
      a.positions[i] = -1;
    }
    return;
  }
  // the request of slot i0, the last b with token_starts[b] <= i0: 32 ways at a time
  int lo = 0, count = a.batch;  // it is in [lo, lo + count)
  while (count > 1) {
    const int step = (count + 31) / 32;
    const int b = lo + lane * step;
    const unsigned below = __ballot_sync(kFull, lane * step < count && a.token_starts[b] <= i0);
    const int way = 31 - __clz(below);
    count = min(step, count - way * step);
    lo += way * step;
  }
  // the starts of the block's requests: at most one begins per slot, apart
  // from requests without tokens, which are walked over
  int b = lo, off = static_cast<int>(i - a.token_starts[lo]);
  for (int base = lo; base < a.batch; base += kSlotThreads) {
    __syncthreads();
    for (int x = t; x <= kSlotThreads; x += kSlotThreads) starts[x] = base + x <= a.batch ? a.token_starts[base + x] : 0x7fffffff;
    __syncthreads();
    const int n = min(kSlotThreads, a.batch - base);
    if (starts[0] <= i) {
      int x = 0, up = n - 1;  // the largest x with starts[x] <= i
      while (x < up) {
        const int mid = (x + up + 1) >> 1;
        if (starts[mid] <= i) x = mid;
        else up = mid - 1;
      }
      b = base + x;
      off = static_cast<int>(i - starts[x]);
    }
    if (starts[n] > i0 + kSlotThreads - 1) break;  // uniform
  }
  if (i >= a.num_slots) return;
  if (i < tokens) {
    write_slot(a, i, b, a.seq_lens_out[b] - a.new_tokens[b], off);
  } else {
    a.slots[i] = -1;
    a.positions[i] = -1;
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (num_slots < kPlanSpread && batch < kPlanMany) {
    PA_CUDA_TRY(launch_pdl(plan_append_kernel<1, true>, dim3(1), dim3(kPlanThreads), 0, st, a));
    return PA_OK;
  }
  // Padded slots need no search for their request, and the cluster writes them
  // with the sums at hand: 16,000 slots of 1000 requests in 8.8 us (packed, with
  // the second launch, 10.0), 32,000 of 2000 in 10.9 (10.1).  Beyond that eight
  // CTAs are too few: 128,000 of 2000 take 21.5 (10.9).
  const bool wide = max_new_tokens == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCluster);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPlanCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  PA_CUDA_TRY(wide ? cudaLaunchKernelEx(&cfg, plan_append_kernel<kPlanCluster, false>, a)
                   : cudaLaunchKernelEx(&cfg, plan_append_kernel<kPlanCluster, true>, a));
  if (wide && num_slots > 0)
    PA_CUDA_TRY(launch_pdl(plan_slots_kernel, dim3(static_cast<unsigned>((num_slots + kSlotThreads - 1) / kSlotThreads)),
                           dim3(kSlotThreads), 0, st, a));
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
