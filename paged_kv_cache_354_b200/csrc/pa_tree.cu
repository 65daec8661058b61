// pa_decode_tree: attention of a tree of drafted tokens over the paged cache.
//
//   out[b][t][j] = softmax_{p in A(t)}(scale q[b][t][j] . K[p]) V[p],
//   A(t) = [0, L - n) and the tree nodes whose bit is set in t's mask row
//
// The rows of a KV head -- (node, query head of its group) -- are the M of a
// flash attention on tcgen05: S = Q K^T (128 rows x 128 tokens) into tensor
// memory, an online softmax with one thread per row, P (bf16) back into
// tensor memory over S, O += P V with P as the tensor-memory A operand and O
// in tensor memory for a whole segment.  128 / group whole tokens make a row
// tile, two row tiles an item; an item's unit of work is a tile of 128
// positions.
//
// Two streams (S, P and O each, one softmax warpgroup each) hide the softmax
// behind the products: step g belongs to stream g & 1, and the issuing
// thread's order S(0) S(1) PV(0) S(2) PV(1) S(3) ... leaves the tensor cores
// the other stream's products while one stream is in its softmax.  An item of
// two row tiles gives one to each stream; an item of one row tile gives the
// even tiles to one stream and the odd ones to the other, and the streams'
// (m, l, O) are joined at the end of the segment, in tensor memory, where
// both warpgroups reach both accumulators.
//
// The work is split like the balanced decode: all (request, KV head, row-tile
// pair, tile) units in one line, an equal contiguous share per CTA, items cut
// between CTAs joined by the merge kernel, which also writes the zeros of the
// rows that have no node.
//
// What a node does not attend to may hold anything.  K: a masked logit is
// replaced by -inf whatever it was.  V: 0 * NaN would reach every row of the
// tile, so two warps look through the rows of tree nodes (and zero the rows
// past the request's end) before the product reads them; values that are not
// finite are zeroed there, and the epilogue adds them to the rows that do
// attend (P > 0, so p * inf = inf and p * NaN = NaN whatever p is).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"
#include "pa_tree_mma.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kTile = 128;     // positions per unit of work
constexpr int kRows = 128;     // rows of a row tile: TMEM lanes
constexpr int kThreads = 384;  // producer, MMA and two cleaning warps; two softmax warpgroups
constexpr int kMaxBatch = 32768;
constexpr float kSlack = 8.f;  // log2 units a row's kept maximum may lag: probabilities stay <= 256

struct TreeArgs {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const __nv_bfloat16* pool;
  const uint32_t* mask;
  int64_t mask_stride;  // words from one request's rows to the next one's (0: shared)
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* tree_lens;
  float* part_o;      // [CTAs][2][2 * kRows][D] unnormalised, at the row's kept maximum
  float2* part_ml;    // [CTAs][2][2 * kRows] (kept maximum, sum)
  int* prefix_out;    // [batch + 1] unit prefix sums, per KV head
  int32_t* err;
  int batch, nodes, words, num_q_heads, num_kv_heads, group;
  int tile_tokens;    // tokens per row tile
  int pairs;          // row-tile pairs of num_nodes tokens
  int num_blocks, max_blocks, max_seq_len;
  int extra, min_units;
  float scale_log2;   // |scale| * log2(e)
  int negative;       // scale < 0: logits change sign
};

// Length and node count of request b after the device checks; n = 0 where
// the request has no (valid) tree.
template <int BS>
__device__ __forceinline__ void tree_lengths(const TreeArgs& a, int b, bool report, int& len, int& n) {
  const int raw = a.seq_lens[b];
  const long long cap = min(static_cast<long long>(a.max_blocks) * BS, static_cast<long long>(a.max_seq_len));
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

// Row-tile pairs and tiles of a request; both 0 without nodes.
__device__ __forceinline__ int pairs_of(const TreeArgs& a, int n) {
  return (n + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// CTAs that share `total` units: at least min_units each.
__device__ __forceinline__ int ctas_for(const TreeArgs& a, long long total, int ctas) {
  return static_cast<int>(max(1ll, min(static_cast<long long>(ctas), total / max(a.min_units, 1))));
}
__device__ __forceinline__ long long range_begin(long long total, int c, int ctas) { return total * c / ctas; }
// The CTA whose range holds unit u.
__device__ __forceinline__ int cta_of(long long total, long long u, int ctas) {
  return static_cast<int>((static_cast<long long>(ctas) * (u + 1) + total - 1) / total - 1);
}

// prefix[b] = units per KV head of the requests before b, b in [0, batch].
template <int BS>
__device__ __forceinline__ void unit_prefix(int* prefix, int* scan, const TreeArgs& a, bool report) {
  const int t = threadIdx.x;
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int lo = min(a.batch, t * per), hi = min(a.batch, lo + per);
  int sum = 0;
  for (int b = lo; b < hi; ++b) {
    int len, n;
    tree_lengths<BS>(a, b, report, len, n);
    const int units = n > 0 ? pairs_of(a, n) * (tiles_of(len) + a.extra) : 0;
    prefix[b] = units;
    sum += units;
  }
  scan[t] = sum;
  __syncthreads();
  if (t < 32) {  // exclusive scan of the kThreads partial sums by one warp
    constexpr int kPer = kThreads / 32;
    int run = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) run += scan[t * kPer + e];
    int incl = run;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, off);
      if (t >= off) incl += y;
    }
    int excl = incl - run;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int v = scan[t * kPer + e];
      scan[t * kPer + e] = excl;
      excl += v;
    }
    if (t == 31) prefix[a.batch] = incl;
  }
  __syncthreads();
  int run = scan[t];
  for (int b = lo; b < hi; ++b) {
    const int units = prefix[b];
    prefix[b] = run;
    run += units;
  }
  __syncthreads();
}

// The largest b with hkv * prefix[b] <= u (requests without units are skipped).
__device__ __forceinline__ int request_of(const int* prefix, int batch, int hkv, long long u) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<long long>(hkv) * prefix[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One CTA's share of one item, published by the producer.
struct Segment {
  int b, h;
  int token0;    // first token of the item's first row tile
  int len, n;    // positions and nodes of the request
  int tile0;     // first tile
  int steps;     // products per (S, PV): tiles, or twice as many with two row tiles
  int flags;
  int slot;      // partial slot of the CTA
  int poison;    // set by the cleaning warps: a tree node's value is not finite
  int pad[2];
};
constexpr int kTwo = 1;        // two row tiles
constexpr int kComplete = 2;   // all tiles of the item

template <int D, int BS>
struct Geo {
  static constexpr int kSlabs = D / 64;
  static constexpr int kGroupStride = kSlabs * 1024;  // between 8-token groups of a K or V tile
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kBlockBytes = BS * D * 2;
  static constexpr int kTileBlocks = kTile / BS;
  static constexpr int kQSlab = kRows * 128;
  static constexpr int kQBytes = kSlabs * kQSlab;
  // two query tiles and the rings fill shared memory: 2 + 3 tiles at head
  // dim 128 (a key tile is released after its S, a value tile is held
  // through a softmax), 6 + 5 at 64
  static constexpr int kKStages = D == 128 ? 2 : 6;
  static constexpr int kVStages = D == 128 ? 3 : 5;
  static constexpr int kSegs = D == 128 ? 8 : 16;  // see the producer
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kQBytes;
  static constexpr int kV = kK + kKStages * kTileBytes;
  static constexpr int kBar = kV + kVStages * kTileBytes;
  static constexpr int kNumBars = 2 * kKStages + 3 * kVStages + 2 * 6 + 2 + kSegs;
  static constexpr int kSeg = (kBar + 8 * kNumBars + 15) & ~15;
  static constexpr int kXch = kSeg + kSegs * static_cast<int>(sizeof(Segment));  // float2 [2][kRows]
  static constexpr int kMisc = kXch + 2 * kRows * 8;  // tmem base, abort, issued k, v, q loads
  static constexpr int kTotal = kMisc + 32;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kS = 0;              // S / P of stream s at kS + 128 s
  static constexpr int kO = 2 * kTile;      // O of stream s at kO + D s
  // the prefix sums and their scan fit the idle rings at any batch
  static_assert(4 * (kMaxBatch + 8 + kThreads) <= (kKStages + kVStages) * kTileBytes, "prefix table");
  static_assert(kTotal <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A wait of a whole warp: true when every lane saw the phase complete.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  const bool ok = mbar_wait(bar, parity);
  return __all_sync(kFull, ok);
}

__device__ __forceinline__ bool not_finite(uint32_t pair) {
  return (pair & 0x7f80u) == 0x7f80u || (pair & 0x7f800000u) == 0x7f800000u;
}

// Which of the positions pos0 .. pos0 + 31 node t's row attends to, as bits.
__device__ __forceinline__ uint32_t attended32(const uint32_t* mask_row, int pos0, int base, int n) {
  const int i0 = pos0 - base;
  if (i0 <= -32) return kFull;
  if (i0 >= n) return 0u;
  const int words = (n + 31) >> 5;
  uint32_t bits;
  if (i0 < 0) {
    bits = (mask_row[0] << -i0) | ((1u << -i0) - 1u);
  } else {
    const int w = i0 >> 5;
    bits = __funnelshift_r(mask_row[w], w + 1 < words ? mask_row[w + 1] : 0u, i0 & 31);
  }
  if (n - i0 < 32) bits &= (1u << (n - i0)) - 1u;
  return bits;
}

template <int D, int BS>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
                          const TreeArgs a) {
  using G = Geo<D, BS>;
  constexpr int KS = G::kKStages, VS = G::kVStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  auto bar = [&](int i) -> uint32_t { return sbase + G::kBar + 8 * i; };
  auto k_full = [&](int s) { return bar(s); };
  auto k_empty = [&](int s) { return bar(KS + s); };
  auto v_full = [&](int s) { return bar(2 * KS + s); };
  auto v_empty = [&](int s) { return bar(2 * KS + VS + s); };
  auto v_clean = [&](int s) { return bar(2 * KS + 2 * VS + s); };
  constexpr int kPairBars = 2 * KS + 3 * VS;
  auto q_full = [&](int j) { return bar(kPairBars + j); };
  auto q_empty = [&](int j) { return bar(kPairBars + 2 + j); };
  auto s_full = [&](int s) { return bar(kPairBars + 4 + s); };
  auto p_full = [&](int s) { return bar(kPairBars + 6 + s); };
  auto pv_done = [&](int s) { return bar(kPairBars + 8 + s); };
  auto xch_full = [&](int s) { return bar(kPairBars + 10 + s); };
  const uint32_t o_free = bar(kPairBars + 12);
  const uint32_t drain = bar(kPairBars + 13);
  auto seg_full = [&](int j) { return bar(kPairBars + 14 + j); };
  volatile Segment* segs = reinterpret_cast<volatile Segment*>(smem + G::kSeg);
  float2* xch = reinterpret_cast<float2*>(smem + G::kXch);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + G::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + G::kMisc + 4);
  volatile int* issued = reinterpret_cast<volatile int*>(smem + G::kMisc + 8);  // k, v, q loads

  if (sbase & 1023u) {  // the swizzled tiles need it; uniform
    if (threadIdx.x == 0) flag_error(a.err, PA_DEVERR_WAIT_TIMEOUT);
    return;
  }
  if (threadIdx.x == 0) {  // shared memory only: may overlap the previous grid
    for (int s = 0; s < KS; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
      mbar_init(v_clean(s), 64);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 128);
      mbar_init(pv_done(s), 1);
      mbar_init(xch_full(s), 128);
    }
    mbar_init(o_free, 256);
    mbar_init(drain, 1);
    for (int j = 0; j < G::kSegs; ++j) mbar_init(seg_full(j), 1);
    *abort_flag = 0;
    issued[0] = issued[1] = issued[2] = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    __syncwarp();
    tc::tmem_alloc(smem_u32(tmem_slot), G::kTmemCols);
    tc::tmem_relinquish();
  }
  pdl_wait();  // every global access below comes after the previous grid
  pdl_trigger();

  // the unit prefix sums, in the still idle rings
  int* prefix = reinterpret_cast<int*>(smem + G::kK);
  unit_prefix<BS>(prefix, prefix + ((a.batch + 4) & ~3), a, blockIdx.x == 0);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.batch; i += kThreads) a.prefix_out[i] = prefix[i];
  const int hkv = a.num_kv_heads;
  const long long total = static_cast<long long>(hkv) * prefix[a.batch];
  const int ctas = ctas_for(a, total, gridDim.x);
  const bool idle = total == 0 || static_cast<int>(blockIdx.x) >= ctas;
  const long long u_begin = idle ? 0 : range_begin(total, blockIdx.x, ctas);
  const long long u_end = idle ? 0 : range_begin(total, blockIdx.x + 1, ctas);
  const int b_first = idle ? 0 : request_of(prefix, a.batch, hkv, u_begin);
  const long long r_first = idle ? 0 : u_begin - static_cast<long long>(hkv) * prefix[b_first];
  fence_proxy_async_smem();  // the rings' generic writes above, TMA writes below
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  auto give_up = [&]() {
    flag_error(a.err, PA_DEVERR_WAIT_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // walks the CTA's units; real segments are published in a ring of
    // records.  A record is overwritten kSegs segments later: by then at
    // least kSegs - 1 - kVStages >= 4 later segments' products are done, so
    // both warpgroups, which take turns, are past it.
    if (lane == 0) {
      prefetch_tensor_map(&kv_map);
      prefetch_tensor_map(&q_map);
    }
    int b = b_first;
    int len = 0, n = 0;
    if (!idle) tree_lengths<BS>(a, b, false, len, n);
    int tiles = tiles_of(len), np = pairs_of(a, n);
    long long item = idle ? 0 : r_first / (tiles + a.extra);
    int k = idle ? 0 : static_cast<int>(r_first - item * (tiles + a.extra));
    int h = np > 0 ? static_cast<int>(item / np) : 0;
    int rp = np > 0 ? static_cast<int>(item - static_cast<long long>(h) * np) : 0;
    long long u = u_begin;
    int seg = 0, first = 1, kc = 0, vc = 0, qc = 0;
    bool ok = true;
    while (u < u_end && ok) {
      const int span = static_cast<int>(min(static_cast<long long>(tiles + a.extra - k), u_end - u));
      const int cnt = max(0, min(k + span, tiles) - k);  // real tiles
      if (cnt > 0) {
        const int token0 = rp * 2 * a.tile_tokens;
        const bool two = n - token0 > a.tile_tokens;
        if (lane == 0) {
          volatile Segment& s = segs[seg % G::kSegs];
          s.b = b;
          s.h = h;
          s.token0 = token0;
          s.len = len;
          s.n = n;
          s.tile0 = k;
          s.steps = two ? 2 * cnt : cnt;
          s.flags = (two ? kTwo : 0) | (k == 0 && cnt == tiles ? kComplete : 0);
          s.slot = first ? 0 : 1;
          s.poison = 0;
          mbar_arrive(seg_full(seg % G::kSegs));  // release: the record is visible
        }
        ++seg;
        const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks;
        const int blocks = (len + BS - 1) / BS;
        constexpr int kAhead = 32 / G::kTileBlocks;  // tiles per warp load of table entries
        int next = 0;
        auto fetch = [&](int tile) -> int {
          const int e = tile * G::kTileBlocks + lane;
          int block = 0;
          if (e < blocks) {
            block = __ldg(table + e);
            if (static_cast<unsigned>(block) >= static_cast<unsigned>(a.num_blocks)) {
              flag_error(a.err, PA_DEVERR_BLOCK_ID);
              block = a.num_blocks;  // past the tensor map: TMA fills with zeros
            }
          }
          return block;
        };
        next = fetch(k);
        int entries = 0;
        for (int i = 0; i < cnt && ok; ++i) {
          if (i % kAhead == 0) {
            entries = next;
            if (i + kAhead < cnt) next = fetch(k + i + kAhead);
          }
          const int mine = __shfl_sync(kFull, entries, (i % kAhead) * G::kTileBlocks + lane % G::kTileBlocks);
          const int live = min(G::kTileBlocks, blocks - (k + i) * G::kTileBlocks);  // blocks in the tile
          const int ks = kc % KS, vs = vc % VS;
          ok = warp_wait(k_empty(ks), ((kc / KS) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(k_full(ks), live * G::kBlockBytes);
            issued[0] = kc + 1;
          }
          __syncwarp();
          if (lane < live)
            tma_load_5d(sbase + G::kK + ks * G::kTileBytes + lane * G::kBlockBytes, &kv_map, k_full(ks), 0, 0, 0,
                        h * (BS / 8), 2 * mine);
          ++kc;
          // the queries, after the first keys: their buffer may still be in use
          for (int j = 0; i == 0 && j < (two ? 2 : 1) && ok; ++j) {
            const int qs = qc & 1;
            ok = warp_wait(q_empty(qs), ((qc >> 1) & 1) ^ 1);
            if (!ok) break;
            ++qc;
            if (lane == 0) {
              mbar_arrive_expect_tx(q_full(qs), G::kSlabs * 128 * a.group * a.tile_tokens);
              issued[2] = qc;
#pragma unroll
              for (int x = 0; x < G::kSlabs; ++x)
                tma_load_4d(sbase + G::kQ + qs * G::kQBytes + x * G::kQSlab, &q_map, q_full(qs), 0, h * a.group,
                            b * a.nodes + token0 + j * a.tile_tokens, x);
            }
          }
          if (!ok) break;
          ok = warp_wait(v_empty(vs), ((vc / VS) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(v_full(vs), live * G::kBlockBytes);
            issued[1] = vc + 1;
          }
          __syncwarp();
          if (lane < live)
            tma_load_5d(sbase + G::kV + vs * G::kTileBytes + lane * G::kBlockBytes, &kv_map, v_full(vs), 0, 0, 0,
                        h * (BS / 8), 2 * mine + 1);
          ++vc;
        }
      }
      first = 0;
      u += span;
      k = 0;
      if (u < u_end && ++rp == np) {
        rp = 0;
        if (++h == hkv) {
          h = 0;
          do {  // units are left, so a later request has nodes
            ++b;
            tree_lengths<BS>(a, b, false, len, n);
          } while (n == 0);
          tiles = tiles_of(len);
          np = pairs_of(a, n);
        }
      }
    }
    // the end: a record without steps
    if (lane == 0) {
      if (ok) {
        segs[seg % G::kSegs].steps = 0;
        mbar_arrive(seg_full(seg % G::kSegs));
      } else {
        give_up();
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issue
    if (lane == 0) {
      struct Walk {
        int seg = 0;    // segment ordinal
        int g0 = 0;     // global step at its start
        int g = 0;      // next step
        int steps = 0;  // of the segment; 0 before the first
        bool two = false, end = false;
        int tail = 0;   // len - first position of the segment's first tile
      };
      Walk sw, pw;
      int qc = 0, q_seg = 0;     // query tiles used by earlier segments, by this one
      int kc = 0, vc = 0;        // K / V tiles used so far
      int q_commits[2] = {0, 0};
      bool ok = true;
      // the segment of step w.g; false on a time-out
      auto enter = [&](Walk& w) -> bool {
        while (!w.end && w.g == w.g0 + w.steps) {
          const int j = w.seg % G::kSegs;
          if (!mbar_wait(seg_full(j), (w.seg / G::kSegs) & 1)) return false;
          w.g0 = w.g;
          w.steps = segs[j].steps;
          w.two = (segs[j].flags & kTwo) != 0;
          w.tail = segs[j].len - segs[j].tile0 * kTile;
          ++w.seg;
          if (w.steps == 0) w.end = true;
        }
        return true;
      };
      auto width = [&](const Walk& w, int tile) {  // tokens of the tile, rounded up to 16
        return min(kTile, ((w.tail - tile * kTile) + 15) & ~15);
      };
      auto issue_s = [&]() -> bool {
        if (!enter(sw)) return false;
        if (sw.end) return true;
        const int local = sw.g - sw.g0;
        if (local == 0) {
          qc += q_seg;
          q_seg = sw.two ? 2 : 1;
        }
        const int tile = sw.two ? local >> 1 : local;
        const int rt = sw.two ? local & 1 : 0;
        const int ks = kc % KS;
        const int qi = qc + rt;
        if (!mbar_wait(k_full(ks), (kc / KS) & 1)) return false;
        if (tile == 0 && !mbar_wait(q_full(qi & 1), (qi >> 1) & 1)) return false;
        tc::fence_after_sync();
        const uint32_t kt = sbase + G::kK + ks * G::kTileBytes;
        const uint32_t qt = sbase + G::kQ + (qi & 1) * G::kQBytes;
        const uint32_t d = tmem + G::kS + (sw.g & 1) * kTile;
        const uint32_t id = tc::idesc_bf16(kRows, width(sw, tile), false, false);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int x = i >> 2, kk = i & 3;
          const uint64_t ad = tc::smem_desc(qt + x * G::kQSlab + kk * 32, 16, 1024, tc::kSwizzle128B);
          const uint64_t bd = tc::smem_desc(kt + x * 1024 + kk * 32, 16, G::kGroupStride, tc::kSwizzle128B);
          tc::mma_bf16(d, ad, bd, id, i > 0 ? 1u : 0u);
        }
        tc::commit(s_full(sw.g & 1));
        if (!sw.two || rt == 1) {
          tc::commit(k_empty(ks));
          ++kc;
        }
        const int last = sw.two ? sw.steps - 2 + rt : sw.steps - 1;
        if (local == last) {
          tc::commit(q_empty(qi & 1));
          ++q_commits[qi & 1];
        }
        ++sw.g;
        return true;
      };
      auto issue_pv = [&]() -> bool {
        const int local = pw.g - pw.g0;
        const int s = pw.g & 1;
        const int tile = pw.two ? local >> 1 : local;
        const int vs = vc % VS;
        if (!mbar_wait(p_full(s), (pw.g >> 1) & 1)) return false;
        // the accumulators were read by the segment before; waited for after
        // P, which bounds how far behind the other warpgroup can be
        if (local < 2 && pw.seg > 1 && !mbar_wait(o_free, (pw.seg - 2) & 1)) return false;
        if (!mbar_wait(v_full(vs), (vc / VS) & 1) || !mbar_wait(v_clean(vs), (vc / VS) & 1)) return false;
        tc::fence_after_sync();
        const uint32_t vt = sbase + G::kV + vs * G::kTileBytes;
        const uint32_t p = tmem + G::kS + s * kTile;
        const uint32_t d = tmem + G::kO + s * D;
        constexpr uint32_t id = tc::idesc_bf16(kRows, D, false, true);
        const int steps = width(pw, tile) / 16;
        for (int i = 0; i < steps; ++i) {
          const uint64_t bd = tc::smem_desc(vt + 2 * i * G::kGroupStride, G::kSlabs > 1 ? 1024 : 0, G::kGroupStride,
                                            tc::kSwizzle128B);
          tc::mma_bf16_ts(d, p + 8 * i, bd, id, local >= 2 || i > 0 ? 1u : 0u);
        }
        tc::commit(pv_done(s));
        if (!pw.two || (local & 1)) {
          tc::commit(v_empty(vs));
          ++vc;
        }
        ++pw.g;
        return true;
      };
      ok = issue_s() && issue_s();
      while (ok) {
        ok = enter(pw);
        if (!ok || pw.end) break;
        ok = issue_pv() && issue_s();
      }
      if (!ok) give_up();
      // every issued product has finished before tensor memory is released,
      // and every commit's arrival has landed before shared memory goes away
      tc::commit(drain);
      mbar_wait_bounded(drain, 0, kWaitLimitNs);
      auto wait_last = [&](uint32_t at, int commits) {
        if (commits > 0) mbar_wait_bounded(at, (commits - 1) & 1, kWaitLimitNs);
      };
      for (int st = 0; st < KS; ++st) wait_last(k_empty(st), kc > st ? (kc - st + KS - 1) / KS : 0);
      for (int st = 0; st < VS; ++st) wait_last(v_empty(st), vc > st ? (vc - st + VS - 1) / VS : 0);
      for (int j = 0; j < 2; ++j) {
        wait_last(q_empty(j), q_commits[j]);
        wait_last(pv_done(j), (pw.g + 1 - j) >> 1);
        wait_last(s_full(j), (sw.g + 1 - j) >> 1);
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------- cleaning value tiles
    int vc = 0;
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      const int j = seg % G::kSegs;
      ok = warp_wait(seg_full(j), (seg / G::kSegs) & 1);
      if (!ok) break;
      const int steps = segs[j].steps;
      if (steps == 0) break;
      const int tiles = (segs[j].flags & kTwo) ? steps >> 1 : steps;
      const int len = segs[j].len, base = len - segs[j].n;
      for (int i = 0; i < tiles && ok; ++i, ++vc) {
        const int vs = vc % VS;
        ok = warp_wait(v_full(vs), (vc / VS) & 1);
        if (!ok) break;
        const int pos0 = (segs[j].tile0 + i) * kTile;
        const int end = min(kTile, len - pos0);  // rows of the request
        const int pad = min(kTile, (end + 15) & ~15);
        const int from = max(0, base - pos0);
        if (from < pad) {
          const uint32_t vt = sbase + G::kV + vs * G::kTileBytes;
          constexpr int kChunks = D / 8;  // 16-byte chunks of a row
          bool found = false;
          for (int e = (threadIdx.x - 64) + from * kChunks; e < pad * kChunks; e += 64) {
            const int row = e / kChunks, c = e % kChunks;
            const uint32_t at = vt + (row >> 3) * G::kGroupStride + (c >> 3) * 1024 + (row & 7) * 128 + (c & 7) * 16;
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            bool write = row >= end;
            if (!write) {
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (not_finite(w[x])) {
                  if ((w[x] & 0x7f80u) == 0x7f80u) w[x] &= 0xffff0000u;
                  if ((w[x] & 0x7f800000u) == 0x7f800000u) w[x] &= 0x0000ffffu;
                  write = found = true;
                }
            }
            if (write)
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
          }
          if (found) segs[j].poison = 1;
          fence_proxy_async_smem();  // the rows are read by the MMA
        }
        mbar_arrive(v_clean(vs));
      }
    }
    if (!ok && lane == 0) give_up();
    __syncwarp();
  } else {
    // ------------------------------------------------- softmax and epilogue
    const int s = (warp - 4) >> 2;     // stream
    const int qd = warp & 3;           // TMEM lane quadrant
    const int row = 32 * qd + lane;    // of the row tile
    const uint32_t lanes = tc::tmem_addr(tmem, 32 * qd, 0);
    const int row_token = row / a.group, row_head = row - row_token * a.group;
    int g0 = 0;
    int xch_phase = 0;
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      const int j = seg % G::kSegs;
      ok = warp_wait(seg_full(j), (seg / G::kSegs) & 1);
      if (!ok) break;
      const int steps = segs[j].steps;
      if (steps == 0) break;
      const int flags = segs[j].flags;
      const bool two = (flags & kTwo) != 0;
      const int len = segs[j].len, n = segs[j].n, base = len - n;
      const int b = segs[j].b, h = segs[j].h, tile0 = segs[j].tile0;
      const int rt = two ? (s - g0) & 1 : 0;
      const int token = segs[j].token0 + rt * a.tile_tokens + row_token;
      const bool valid = row_token < a.tile_tokens && token < n;
      const bool work = __any_sync(kFull, valid);
      const uint32_t* mask_row = a.mask + b * a.mask_stride + static_cast<int64_t>(valid ? token : 0) * a.words;
      float m = -INFINITY, l = 0.f;  // kept maximum (log2 units) and sum at it
      bool fresh = true;             // no step of this stream yet
      for (int g = g0 + ((s - g0) & 1); g < g0 + steps; g += 2) {
        const int tile = tile0 + (two ? (g - g0) >> 1 : g - g0);
        ok = warp_wait(s_full(s), (g >> 1) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        if (work) {
          const int pos0 = tile * kTile;
          const bool open = pos0 + kTile <= base;  // nothing to mask
          const uint32_t sp = lanes + G::kS + s * kTile;
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t r[32];
            const uint32_t bits = open ? kFull : valid ? attended32(mask_row, pos0 + 32 * c, base, n) : 0u;
            __syncwarp();
            tc::tmem_ld_x32(sp + 32 * c, r);
            tc::wait_ld_x32(r);
            if (a.negative) {
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] ^= 0x80000000u;
            }
            if (open) {
#pragma unroll
              for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(r[e]));
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) top = fmaxf(top, (bits >> e) & 1u ? __uint_as_float(r[e]) : -INFINITY);
            }
          }
          top *= a.scale_log2;
          const bool over = valid && top > m + kSlack;  // true while m = -inf and something is attended
          if (__any_sync(kFull, over)) {
            const float mn = over ? top : m;
            const float alpha = m == -INFINITY ? 0.f : ex2(m - mn);
            l = m == mn ? l : l * alpha;
            if (!fresh) {
              // O holds the sum through this stream's step before, which is
              // done: the products complete in order, and S of this step is
              const float keep = m == mn ? 1.f : alpha;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                const uint32_t oa = lanes + G::kO + s * D + 32 * c;
                tc::tmem_ld_x32(oa, o);
                tc::wait_ld_x32(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tc::tmem_st_x32(oa, o);
              }
            }
            m = mn;
          }
          const float shift = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t r[32];
            const uint32_t bits = open ? kFull : valid ? attended32(mask_row, pos0 + 32 * c, base, n) : 0u;
            __syncwarp();
            tc::tmem_ld_x32(sp + 32 * c, r);
            tc::wait_ld_x32(r);
            if (a.negative) {
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] ^= 0x80000000u;
            }
            if (!open) {
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = (bits >> e) & 1u ? r[e] : 0xff800000u;
            }
            // probabilities, rounded to bf16; the sum takes the rounded values
            // that the product multiplies, so the weights stay a convex combination
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              p[e] = pack_bf16x2(ex2(fmaf(__uint_as_float(r[2 * e]), a.scale_log2, -shift)),
                                 ex2(fmaf(__uint_as_float(r[2 * e + 1]), a.scale_log2, -shift)));
              l += bf16lo_to_f32(p[e]);
              l += bf16hi_to_f32(p[e]);
            }
            tc::tmem_st_x16(sp + 16 * c, p);  // over columns of S that have been read
          }
          tc::wait_st();
          fresh = false;
        }
        tc::fence_before_sync();
        mbar_arrive(p_full(s));
      }
      if (!ok) break;

      // ---- end of the segment: the streams' last products
      const int g1 = g0 + steps;
      const int last_own = g1 - 1 - ((g1 - 1 - s) & 1);          // the largest g < g1 on this stream
      const int last_other = g1 - 1 - ((g1 - 1 - (s ^ 1)) & 1);  // ... on the other one
      if (last_own >= g0) ok = warp_wait(pv_done(s), (last_own >> 1) & 1);
      if (ok && !two && last_other >= g0) ok = warp_wait(pv_done(s ^ 1), (last_other >> 1) & 1);
      if (!ok) break;
      tc::fence_after_sync();
      float keep0 = 1.f, keep1 = 0.f;  // factors of the own and the other stream's O
      if (!two) {
        xch[s * kRows + row] = make_float2(m, l);
        mbar_arrive(xch_full(s));
        ok = warp_wait(xch_full(s ^ 1), xch_phase & 1);
        if (!ok) break;
        ++xch_phase;
        const float2 o = xch[(s ^ 1) * kRows + row];
        const float mn = fmaxf(m, o.x);
        keep0 = m == -INFINITY ? 0.f : ex2(m - mn);
        keep1 = o.x == -INFINITY ? 0.f : ex2(o.x - mn);
        l = l * keep0 + o.y * keep1;
        m = mn;
      }
      if (work) {
        const bool complete = (flags & kComplete) != 0;
        const bool poison = segs[j].poison != 0;
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // a row that attends to nothing gets 0
        const int64_t out_row = (static_cast<int64_t>(b) * a.nodes + token) * a.num_q_heads + h * a.group + row_head;
        const int64_t part_row = (static_cast<int64_t>(blockIdx.x) * 2 + segs[j].slot) * (2 * kRows) + rt * kRows + row;
        // with one row tile each warpgroup writes half of the columns
        const int c_begin = two ? 0 : s * (D / 64), c_end = two ? D / 32 : (s + 1) * (D / 64);
        for (int c = c_begin; c < c_end; ++c) {
          uint32_t o[32];
          __syncwarp();
          tc::tmem_ld_x32(lanes + G::kO + s * D + 32 * c, o);
          tc::wait_ld_x32(o);
          if (!two) {
            uint32_t x[32];
            tc::tmem_ld_x32(lanes + G::kO + (s ^ 1) * D + 32 * c, x);
            tc::wait_ld_x32(x);
            // an accumulator whose stream saw nothing of the row is not read
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint((keep0 > 0.f ? __uint_as_float(o[e]) * keep0 : 0.f) +
                                     (keep1 > 0.f ? __uint_as_float(x[e]) * keep1 : 0.f));
          }
          if (valid && poison) {
            // values of attended nodes that are not finite
            const int tiles = two ? steps >> 1 : steps;
            const int lo = max(base, tile0 * kTile), hi = min(len, (tile0 + tiles) * kTile);
            for (int p = lo; p < hi; ++p) {
              const int i = p - base;
              if (!((mask_row[i >> 5] >> (i & 31)) & 1u)) continue;
              const int block = a.block_tables[static_cast<int64_t>(b) * a.max_blocks + p / BS];
              if (static_cast<unsigned>(block) >= static_cast<unsigned>(a.num_blocks)) continue;
              const uint32_t* v = reinterpret_cast<const uint32_t*>(
                  a.pool + ((static_cast<int64_t>(block) * 2 + 1) * hkv + h) * BS * D + (p % BS) * D + 32 * c);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint32_t w = v[e];
                if ((w & 0x7f80u) == 0x7f80u) o[2 * e] = __float_as_uint(__uint_as_float(o[2 * e]) + bf16lo_to_f32(w));
                if ((w & 0x7f800000u) == 0x7f800000u)
                  o[2 * e + 1] = __float_as_uint(__uint_as_float(o[2 * e + 1]) + bf16hi_to_f32(w));
              }
            }
          }
          if (valid && complete) {
            uint4* to = reinterpret_cast<uint4*>(a.out + out_row * D + 32 * c);
            // a row that attends to nothing holds no product
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * x]) * inv, __uint_as_float(o[8 * e + 2 * x + 1]) * inv);
              to[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (valid) {
            float4* to = reinterpret_cast<float4*>(a.part_o + part_row * D + 32 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              to[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                  __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            if (c == 0) a.part_ml[part_row] = make_float2(m, l);
          }
        }
      }
      tc::fence_before_sync();  // the next segment's first products overwrite O
      mbar_arrive(o_free);
      g0 = g1;
    }
    if (!ok && lane == 0) give_up();
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // unwind: let every issued load land before the CTA's memory goes away
    for (int i = max(0, issued[0] - KS); i < issued[0]; ++i) mbar_wait_bounded(k_full(i % KS), (i / KS) & 1, kWaitLimitNs);
    for (int i = max(0, issued[1] - VS); i < issued[1]; ++i) mbar_wait_bounded(v_full(i % VS), (i / VS) & 1, kWaitLimitNs);
    for (int i = max(0, issued[2] - 2); i < issued[2]; ++i) mbar_wait_bounded(q_full(i & 1), (i >> 1) & 1, kWaitLimitNs);
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc::tmem_dealloc(tmem, G::kTmemCols);
  }
}

// Joins the partials of items cut between CTAs, in the order of the CTAs, and
// writes the zeros of rows without a node.  One warp per (token, head) row.
constexpr int kMergeWarps = 8;

template <int D, int BS>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const TreeArgs a, int ctas_launched) {
  constexpr int kPer = D / 32;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int rp = static_cast<int>(blockIdx.x % a.pairs);
  const int h = static_cast<int>(blockIdx.x / a.pairs % a.num_kv_heads);
  const int b = static_cast<int>(blockIdx.x / a.pairs / a.num_kv_heads);
  int len, n;
  tree_lengths<BS>(a, b, false, len, n);
  const int token0 = rp * 2 * a.tile_tokens;
  const int tokens = min(2 * a.tile_tokens, a.nodes - token0);
  const int tiles = tiles_of(len);
  const long long total = static_cast<long long>(a.num_kv_heads) * a.prefix_out[a.batch];
  int c0 = 0, c1 = 0;
  long long u0 = 0;
  int ctas = 1;
  if (token0 < n) {
    ctas = ctas_for(a, total, ctas_launched);
    u0 = static_cast<long long>(a.num_kv_heads) * a.prefix_out[b] +
         (static_cast<long long>(h) * pairs_of(a, n) + rp) * (tiles + a.extra);
    c0 = cta_of(total, u0, ctas);
    c1 = cta_of(total, u0 + tiles - 1, ctas);
  }
  for (int e = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); e < tokens * a.group; e += gridDim.y * kMergeWarps) {
    const int tl = e / a.group, head = e - tl * a.group;
    const int token = token0 + tl;
    const bool zero = token >= n;
    if (!zero && c0 == c1) continue;
    const int rt = tl / a.tile_tokens;
    const int row = rt * kRows + (tl - rt * a.tile_tokens) * a.group + head;
    float o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = 0.f;
    float inv = 0.f;
    if (!zero) {
      auto at = [&](int c) -> int64_t {
        const int slot = c > c0 || range_begin(total, c0, ctas) >= u0 ? 0 : 1;
        return (static_cast<int64_t>(c) * 2 + slot) * (2 * kRows) + row;
      };
      float top = -INFINITY;
      for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, a.part_ml[at(c)].x);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
      float l = 0.f;
      for (int c = c0; c <= c1; ++c) {
        const float2 ml = a.part_ml[at(c)];
        if (ml.x == -INFINITY && ml.y == 0.f) continue;  // saw nothing of the row
        const float w = ex2(ml.x - top);
        l += ml.y * w;
        const float* from = a.part_o + at(c) * D + lane * kPer;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] += from[i] * w;
      }
      inv = l > 0.f || l != l ? 1.f / l : 0.f;
    }
    __nv_bfloat16* to = a.out + ((static_cast<int64_t>(b) * a.nodes + token) * a.num_q_heads + h * a.group + head) * D + lane * kPer;
    if constexpr (kPer == 4) {
      *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    } else {
      *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(o[0] * inv, o[1] * inv);
    }
  }
}

int check_tree_shape(const char* who, int batch, int nodes, int hq, int hkv, int d, int bs, int max_seq_len) {
  if (batch < 0 || nodes <= 0 || hq <= 0 || hkv <= 0 || max_seq_len < 0)
    return fail(PA_ERR_INVALID, "%s: non-positive size", who);
  if (hq % hkv != 0) return fail(PA_ERR_INVALID, "%s: %d query heads are no multiple of %d KV heads", who, hq, hkv);
  if (d != 64 && d != 128) return fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d", who, d);
  if (bs != 16 && bs != 32) return fail(PA_ERR_UNSUPPORTED, "%s: block_size %d", who, bs);
  if (hq / hkv > 64) return fail(PA_ERR_UNSUPPORTED, "%s: group size %d beyond 64", who, hq / hkv);
  if (nodes > 1024) return fail(PA_ERR_UNSUPPORTED, "%s: %d nodes beyond 1024", who, nodes);
  if (batch > kMaxBatch) return fail(PA_ERR_UNSUPPORTED, "%s: batch %d beyond %d", who, batch, kMaxBatch);
  return PA_OK;
}

struct Workspace {
  size_t part_o, part_ml, prefix, bytes;
};

// Two partial slots of two row tiles per CTA, one CTA per SM.
Workspace workspace_layout(int batch, int d) {
  const size_t rows = static_cast<size_t>(std::max(sm_count(), 1)) * 2 * (2 * kRows);
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  Workspace w;
  w.part_o = 0;
  w.part_ml = up(rows * d * sizeof(float));
  w.prefix = w.part_ml + up(rows * sizeof(float2));
  w.bytes = w.prefix + up((static_cast<size_t>(batch) + 1) * sizeof(int));
  return w;
}

// Pool view, 5-D, as the tcgen05 decode's: x = dim within a 64-dim slab, y =
// row within an 8-row group, z = slab, w = (KV head, 8-row group), v = 2 *
// block + (0 keys | 1 values).  A box (64, 8, D/64, bs/8, 1) lands in shared
// memory as [group][slab][row][64].  Query view, 4-D over [B][T][Hq][D]: x =
// dim within a slab, y = query head, z = (request, node), w = slab; a box
// (64, group, tokens, 1) brings one slab of a row tile.
template <int D, int BS>
int launch_tree(const TreeArgs& a, const void* q, cudaStream_t st) {
  using G = Geo<D, BS>;
  alignas(64) CUtensorMap kv_map, q_map;
  {
    const uint64_t dims[5] = {64, 8, D / 64, static_cast<uint64_t>(a.num_kv_heads) * BS / 8,
                              2ull * static_cast<uint64_t>(a.num_blocks)};
    const uint64_t strides[4] = {D * 2, 128, 16ull * D, static_cast<uint64_t>(a.num_kv_heads) * BS * D * 2};
    const uint32_t box[5] = {64, 8, D / 64, BS / 8, 1};
    const int rc = encode_tensor_map(&kv_map, 5, const_cast<__nv_bfloat16*>(a.pool), dims, strides, box, 1);
    if (rc != PA_OK) return rc;
  }
  {
    const uint64_t dims[4] = {64, static_cast<uint64_t>(a.num_q_heads), static_cast<uint64_t>(a.batch) * a.nodes, D / 64};
    const uint64_t strides[3] = {D * 2, static_cast<uint64_t>(a.num_q_heads) * D * 2, 128};
    const uint32_t box[4] = {64, static_cast<uint32_t>(a.group), static_cast<uint32_t>(a.tile_tokens), 1};
    const int rc = encode_tensor_map(&q_map, 4, const_cast<void*>(q), dims, strides, box, 1);
    if (rc != PA_OK) return rc;
  }
  auto kernel = tree_attention_kernel<D, BS>;
  const int rc = set_smem_attr(reinterpret_cast<const void*>(kernel), G::kTotal);
  if (rc != PA_OK) return rc;
  const int ctas = std::max(sm_count(), 1);
  PA_CUDA_TRY(launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), G::kTotal, st, kv_map, q_map, a));
  const int64_t items = static_cast<int64_t>(a.batch) * a.num_kv_heads * a.pairs;
  const int rows = std::min(2 * a.tile_tokens, a.nodes) * a.group;
  const dim3 grid(static_cast<unsigned>(items), static_cast<unsigned>((rows + 4 * kMergeWarps - 1) / (4 * kMergeWarps)));
  PA_CUDA_TRY(launch_pdl(tree_merge_kernel<D, BS>, grid, dim3(32 * kMergeWarps), 0, st, a, ctas));
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
  *bytes_out = workspace_layout(batch, head_dim).bytes;
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
  // smallest normal for 0: masked logits stay -inf, the others vanish
  a.scale_log2 = scale == 0.f ? FLT_MIN : fabsf(scale) * 1.4426950408889634f;
  a.negative = scale < 0.f;
  a.tile_tokens = std::min(kRows / a.group, num_nodes);
  a.pairs = (num_nodes + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
  a.extra = 1;
  a.min_units = 1;
  const int64_t longest = std::min(static_cast<int64_t>(max_seq_len), static_cast<int64_t>(max_blocks_per_seq) * block_size);
  if (static_cast<int64_t>(batch) * a.pairs * ((longest + kTile - 1) / kTile + a.extra) > 0x7fffffffll)
    return fail(PA_ERR_UNSUPPORTED, "%s: batch * row tiles * tiles of max_seq_len beyond 2^31 - 1", who);
  const Workspace w = workspace_layout(batch, head_dim);
  char* ws = static_cast<char*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  a.prefix_out = reinterpret_cast<int*>(ws + w.prefix);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (head_dim == 128) return block_size == 16 ? launch_tree<128, 16>(a, q, st) : launch_tree<128, 32>(a, q, st);
  return block_size == 16 ? launch_tree<64, 16>(a, q, st) : launch_tree<64, 32>(a, q, st);
}

}  // extern "C"
