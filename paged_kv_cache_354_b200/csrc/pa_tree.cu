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
// The softmax passes over S twice, 64 columns at a time in a rolled loop: the
// maximum, then the weights.  The issuing warp's code must stay in the
// instruction cache beside it, and a row held whole in registers left it no
// room (64 trees of 16: 131 us, in two passes 125; one pass that weighs at the
// kept maximum and repeats when it rose: 114 where two take 112).
//
// The work is split like the balanced decode: all (request, KV head, row-tile
// pair, tile) units in one line, an equal contiguous share per CTA, items cut
// between CTAs joined by the merge kernel.
//
// Bounds and what it takes (times of the GPU alone; in long runs the power
// limit lowers the clock and adds the second figure):
//   64 requests of about 2250 positions, 16 nodes, 32 / 8 heads of 128: 625 MB,
//     95 us at copy rate; 110 us = 5.7 TB/s (120 to 132 us).  Memory, and per item
//     some 8000 cycles in which both streams end one item and begin the next
//   4 requests of 32768 positions, 32 nodes: 540 MB, 82 us; 98 to 100 us (109
//     to 115 us)
//   32 requests, 64 nodes, 64 / 8 heads: 155 GFLOP, 94 us; 192 to 200 us (207
//     to 212 us).  A tile costs a stream 2230 cycles of softmax (two warps share
//     a quarter's exponentials), 1024 of products and 600 of hand-over (clock
//     stamps in a copy of the kernel); the two streams keep the tensor cores at
//     40 %, the exponentials at 41 %
//   one request, 700 positions, 8 nodes: 12.4 us; start-up, one cold pass
//     through the code, the merge (4 us)
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
// Warps 0 and 1 clean value tiles.  The issuing and the loading warp sit on
// the quarters of the SM whose softmax warps own rows 64 to 127: with up to
// 64 rows those are idle, and nothing competes with the issue.
constexpr int kProducer = 2, kIssuer = 3;
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
  float4* part_o;     // [CTAs][2][D / 4][2 * kRows] unnormalised, at the row's kept maximum:
                      // a warp, one row per lane, writes 512 bytes in a row
  float2* part_ml;    // [CTAs][2][2 * kRows] (kept maximum, sum)
  int* shares;        // [CTAs][8]: where each CTA's share begins, for the merge kernel
  int32_t* err;
  int batch, nodes, words, num_q_heads, num_kv_heads, group;
  int tile_tokens;    // tokens per row tile
  int pairs;          // row-tile pairs of num_nodes tokens
  unsigned cta_factor;  // __umulhi(x, cta_factor) = x / CTAs launched for x < CTAs^2
  int pair_factor;    // (x * pair_factor) >> 20 = x / (2 * tile_tokens) for x < 2048
  int num_blocks, max_blocks, max_seq_len;
  int extra;          // units that the start and end of an item count for
  float scale_log2;   // |scale| * log2(e)
  int negative;       // scale < 0: logits change sign
  int wide_out;       // out is 32-byte aligned
};

// Length and node count of request b after the device checks; n = 0 where
// the request has no (valid) tree.
template <int BS>
__device__ __forceinline__ void tree_lengths(const TreeArgs& a, int b, bool report, int& len, int& n) {
  const int raw = a.seq_lens[b];
  const int given = a.tree_lens != nullptr ? a.tree_lens[b] : a.nodes;
  const long long cap = min(static_cast<long long>(a.max_blocks) * BS, static_cast<long long>(a.max_seq_len));
  len = static_cast<int>(min(static_cast<long long>(max(raw, 0)), cap));
  if (len != raw && report) flag_error(a.err, PA_DEVERR_SEQ_LEN);
  n = given;
  if (len == 0) {
    n = 0;
  } else if (n < 0 || n > a.nodes || n > len) {
    if (report) flag_error(a.err, PA_DEVERR_TREE);
    n = 0;
  }
}

// Row-tile pairs and tiles of a request; both 0 without nodes.
__device__ __forceinline__ int pairs_of(const TreeArgs& a, int n) {
  return ((n + 2 * a.tile_tokens - 1) * a.pair_factor) >> 20;
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// Equal shares of the line of units, at least a unit each: CTA c begins at
// floor(total c / ctas).  What is left over is spread evenly, so that the CTAs
// half a line apart stay together over the whole line (see `levels`).
struct Split {
  int total, ctas, each;
  unsigned more, factor;
  __device__ __forceinline__ Split(int total, int launched, unsigned factor) : total(total), factor(factor) {
    ctas = max(1, min(launched, total));
    each = total / ctas;
    more = total - each * ctas;  // 0 unless every launched CTA takes part
  }
  __device__ __forceinline__ int begin(int c) const { return each * c + static_cast<int>(__umulhi(more * c, factor)); }
  __device__ __forceinline__ int holder(int u) const {  // the CTA whose share holds unit u: a guess, then a step or two
    int c = min(ctas - 1, static_cast<int>(static_cast<float>(u) * static_cast<float>(ctas) / static_cast<float>(total)));
    while (begin(c) > u) --c;
    while (c + 1 < ctas && begin(c + 1) <= u) ++c;
    return c;
  }
};

// A request in the line of units (per KV head).
struct InLine {
  int before, units;  // units of the requests before it, its own
  int len, n;
};

// The sum of all requests' units per KV head.  `mine`: request threadIdx.x,
// when it exists; prefix[b], units of the requests before b, for batches
// beyond one request per thread (visible after the caller's barrier).
// `uniform`: every request with nodes has as many row-tile pairs as num_nodes
// has.
template <int BS>
__device__ __forceinline__ int unit_prefix(int* prefix, int* sums, const TreeArgs& a, bool report, bool& uniform,
                                           InLine& mine) {
  constexpr int kWarps = kThreads / 32;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int carry = 0;
  int same = 1;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + t;
    InLine x{0, 0, 0, 0};
    bool other = false;
    if (b < a.batch) {
      tree_lengths<BS>(a, b, report, x.len, x.n);
      const int pairs = pairs_of(a, x.n);
      if (x.n > 0) {
        x.units = pairs * (tiles_of(x.len) + a.extra);
        other = pairs != a.pairs;
      }
    }
    int incl = x.units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, off);
      if (lane >= off) incl += y;
    }
    const int warp_same = __all_sync(kFull, !other);
    if (lane == 31) {
      sums[warp] = incl;
      sums[kWarps + warp] = warp_same;
    }
    __syncthreads();
    const int of_warp = lane < kWarps ? sums[lane] : 0;
    const int same_warp = lane < kWarps ? sums[kWarps + lane] : 1;
    const int all = carry + __reduce_add_sync(kFull, of_warp);
    x.before = carry + __reduce_add_sync(kFull, lane < warp ? of_warp : 0) + incl - x.units;
    same &= __all_sync(kFull, same_warp);
    if (b0 == 0) mine = x;
    if (a.batch > kThreads) {
      if (b < a.batch) prefix[b] = x.before;
      __syncthreads();
    }
    carry = all;
  }
  uniform = same != 0;
  return carry;
}

// What the merge kernel reads of a CTA (kShare ints): the item that its share
// begins in, and where.
constexpr int kShare = 8;
enum ShareField { kShareB, kShareH, kSharePair, kShareTile, kShareTiles, kShareNodes, kShareTotal };

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
  static constexpr int kNumBars = 2 * kKStages + 3 * kVStages + 2 * 7 + 1 + kSegs;
  static constexpr int kSeg = (kBar + 8 * kNumBars + 15) & ~15;
  static constexpr int kXch = kSeg + kSegs * static_cast<int>(sizeof(Segment));  // float2 [2][kRows]
  static constexpr int kMisc = kXch + 2 * kRows * 8;  // tmem base, abort, issued k, v, q loads
  static constexpr int kTotal = kMisc + 32;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kS = 0;              // S / P of stream s at kS + 128 s
  static constexpr int kO = 2 * kTile;      // O of stream s at kO + D s
  // the prefix sums fit the idle rings at any batch
  static_assert(4 * (kMaxBatch + 1) <= (kKStages + kVStages) * kTileBytes, "prefix table");
  static_assert(kTotal <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^x, x <= 0, as the weight of a stream or a partial that is joined with
// others: never 0, since a value that is not finite keeps its effect however
// small the weight is
__device__ __forceinline__ float weight_of(float x) { return fmaxf(ex2(x), 0x1p-149f); }

__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}

// Two fp32 operations per instruction.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)), "l"(reinterpret_cast<uint64_t&>(z)));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)));
  return r;
}

// Bounded wait for a phase: the clock is read only once the wait has been
// long, so a short one costs no more than its polls.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
    if ((it & 127u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitLimitNs) return false;
    }
  }
  return true;
}
// ... of a whole warp: true when every lane saw the phase complete.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  const bool ok = wait(bar, parity);
  return __all_sync(kFull, ok);
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// 32 bytes of one row per thread: a whole sector where the alignment allows.
__device__ __forceinline__ void store_32_bytes(__nv_bfloat16* to, const uint32_t (&w)[8], int wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A ring's next stage and the parity of its round.
template <int N>
struct Ring {
  int stage = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++stage == N) {
      stage = 0;
      parity ^= 1;
    }
  }
};

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
  auto o_free = [&](int s) { return bar(kPairBars + 12 + s); };
  const uint32_t drain = bar(kPairBars + 14);
  auto seg_full = [&](int j) { return bar(kPairBars + 15 + j); };
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
      mbar_init(v_empty(s), 3);  // the product and the two cleaning warps
      mbar_init(v_clean(s), 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 4);  // one arrival per warp
      mbar_init(pv_done(s), 1);
      mbar_init(xch_full(s), 128);
      mbar_init(o_free(s), 256);
    }
    mbar_init(drain, 1);
    for (int j = 0; j < G::kSegs; ++j) mbar_init(seg_full(j), 1);
    *abort_flag = 0;
    issued[0] = issued[1] = issued[2] = 0;
    fence_barrier_init();
    prefetch_tensor_map(&kv_map);
    prefetch_tensor_map(&q_map);
  }
  if (warp == kIssuer) {
    __syncwarp();
    tc::tmem_alloc(smem_u32(tmem_slot), G::kTmemCols);
    tc::tmem_relinquish();
  }
  // query rows past a row tile's last one are never loaded: as zeros they cost
  // the tensor cores less power than whatever was there
  for (int i = threadIdx.x; i < 2 * G::kQBytes / 16; i += kThreads)
    *reinterpret_cast<uint4*>(smem + G::kQ + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
  pdl_wait();  // every global access below comes after the previous grid
  pdl_trigger();

  // the unit prefix sums (of a large batch in the still idle rings)
  int* prefix = reinterpret_cast<int*>(smem + G::kK);
  bool uniform;
  InLine mine{0, 0, 0, 0};
  const int hkv = a.num_kv_heads;
  const int sum = unit_prefix<BS>(prefix, reinterpret_cast<int*>(smem + G::kXch), a, blockIdx.x == 0, uniform, mine);
  const int total = hkv * sum;  // fits: checked on the host
  const Split split(total, gridDim.x, a.cta_factor);
  const bool idle = total == 0 || static_cast<int>(blockIdx.x) >= split.ctas;
  const int u_begin = idle ? 0 : split.begin(blockIdx.x);
  const int u_end = idle ? 0 : split.begin(blockIdx.x + 1);
  // The line of units: request, KV head, row-tile pair, tile.  When all
  // requests have the same number of pairs the pair comes first: the CTAs
  // that need the same keys and values are then at them at the same time, and
  // all but one find them in L2 (512 rows per KV head, 32 requests: 352
  // instead of 659 MB from memory)
  const int levels = uniform && total > 0 ? a.pairs : 1;
  int level = 0, in_level = u_begin;
  if (levels > 1) {
    level = u_begin / (total / levels);
    in_level -= level * (total / levels);
  }
  int* found = reinterpret_cast<int*>(smem + G::kXch) + 64;  // the request of the first unit
  auto look = [&](int b, const InLine& x) {
    const int lo = hkv * x.before;
    if (lo > in_level * levels || in_level * levels >= lo + hkv * x.units) return;
    found[0] = b;
    found[1] = levels > 1 ? in_level - lo / levels : in_level - lo;
    found[2] = x.len;
    found[3] = x.n;
  };
  if (a.batch <= kThreads) {
    look(threadIdx.x, mine);
  } else {
    for (int b = threadIdx.x; b < a.batch; b += kThreads) {
      const int lo = prefix[b], hi = b + 1 < a.batch ? prefix[b + 1] : sum;
      InLine x{lo, hi - lo, 0, 0};
      if (hkv * lo <= in_level * levels && in_level * levels < hkv * hi) tree_lengths<BS>(a, b, false, x.len, x.n);
      look(b, x);
    }
  }
  fence_proxy_async_smem();  // the rings' generic writes above, TMA writes below
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  auto give_up = [&]() {
    flag_error(a.err, PA_DEVERR_WAIT_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    // walks the CTA's units; real segments are published in a ring of
    // records.  A record is overwritten kSegs segments later: by then at
    // least kSegs - 1 - kVStages >= 4 later segments' products are done, so
    // both warpgroups, which take turns, are past it.
    struct Item {
      int b, h, rp, len, n, tiles, pairs;
    };
    auto load_request = [&](Item& it) {
      tree_lengths<BS>(a, it.b, false, it.len, it.n);
      it.tiles = tiles_of(it.len);
      it.pairs = pairs_of(a, it.n);
    };
    auto next_item = [&](Item it) -> Item {  // units are left, so there is one
      if (levels == 1 && ++it.rp < it.pairs) return it;
      if (levels == 1) it.rp = 0;
      if (++it.h < hkv) return it;
      it.h = 0;
      do {
        if (++it.b == a.batch) {
          it.b = 0;
          ++it.rp;
        }
        load_request(it);
      } while (it.n == 0);
      return it;
    };
    constexpr int kAhead = 32 / G::kTileBlocks;  // tiles per warp load of table entries
    // a warp's worth of entries as they are: they are checked when used, a
    // while after they were asked for
    auto fetch = [&](const Item& it, int tile) -> int {
      const unsigned e = static_cast<unsigned>(tile) * G::kTileBlocks + lane;
      return e * BS < static_cast<unsigned>(it.len)
                 ? a.block_tables[static_cast<int64_t>(it.b) * a.max_blocks + e]
                 : 0;
    };
    Item cur{0, 0, 0, 0, 0, 0, 0};
    int k = 0, ahead = 0;
    if (!idle) {
      cur.b = found[0];
      cur.len = found[2];
      cur.n = found[3];
      cur.tiles = tiles_of(cur.len);
      cur.pairs = pairs_of(a, cur.n);
      const int item = found[1] / (cur.tiles + a.extra);
      k = found[1] - item * (cur.tiles + a.extra);
      cur.h = levels > 1 || cur.pairs == 1 ? item : item / cur.pairs;
      cur.rp = levels > 1 ? level : item - cur.h * cur.pairs;
      ahead = fetch(cur, k);
    }
    if (lane == 0) {
      int* share = a.shares + blockIdx.x * kShare;
      share[kShareB] = cur.b;
      share[kShareH] = cur.h;
      share[kSharePair] = cur.rp;
      share[kShareTile] = idle ? -1 : k;
      share[kShareTiles] = cur.tiles;
      share[kShareNodes] = cur.n;
      share[kShareTotal] = total;
    }
    int u = u_begin;
    int seg = 0, first = 1, kc = 0, vc = 0, qc = 0;
    Ring<KS> kr;
    Ring<VS> vr;
    bool ok = true;
    while (u < u_end && ok) {
      const int span = min(cur.tiles + a.extra - k, u_end - u);
      const int cnt = max(0, min(k + span, cur.tiles) - k);  // real tiles
      Item after = cur;
      int after_entries = 0;
      const int token0 = cur.rp * 2 * a.tile_tokens;
      const bool two = cur.n - token0 > a.tile_tokens;
      const int blocks = (cur.len + BS - 1) / BS;
      int entries = 0;
      if (cnt > 0) {
        if (lane == 0) {
          volatile Segment& s = segs[seg % G::kSegs];
          s.b = cur.b;
          s.h = cur.h;
          s.token0 = token0;
          s.len = cur.len;
          s.n = cur.n;
          s.tile0 = k;
          s.steps = two ? 2 * cnt : cnt;
          s.flags = (two ? kTwo : 0) | (k == 0 && cnt == cur.tiles ? kComplete : 0);
          s.slot = first ? 0 : 1;
          s.poison = 0;
          mbar_arrive(seg_full(seg % G::kSegs));  // release: the record is visible
        }
        ++seg;
      }
      for (int i = 0; i < max(cnt, 1) && ok; ++i) {
        if (cnt > 0) {
          if (i % kAhead == 0) {
            entries = ahead;
            if (static_cast<unsigned>(entries) >= static_cast<unsigned>(a.num_blocks)) {
              flag_error(a.err, PA_DEVERR_BLOCK_ID);
              entries = a.num_blocks;  // past the tensor map: TMA fills with zeros
            }
            if (i + kAhead < cnt) ahead = fetch(cur, k + i + kAhead);
          }
          const int mine = __shfl_sync(kFull, entries, (i % kAhead) * G::kTileBlocks + lane % G::kTileBlocks);
          const int live = min(G::kTileBlocks, blocks - (k + i) * G::kTileBlocks);  // blocks in the tile
          ok = warp_wait(k_empty(kr.stage), kr.parity ^ 1);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(k_full(kr.stage), live * G::kBlockBytes);
            issued[0] = ++kc;
          }
          __syncwarp();
          if (lane < live)
            tma_load_5d(sbase + G::kK + kr.stage * G::kTileBytes + lane * G::kBlockBytes, &kv_map, k_full(kr.stage), 0,
                        0, 0, cur.h * (BS / 8), 2 * mine);
          kr.next();
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
                tma_load_4d(sbase + G::kQ + qs * G::kQBytes + x * G::kQSlab, &q_map, q_full(qs), 0, cur.h * a.group,
                            cur.b * a.nodes + token0 + j * a.tile_tokens, x);
            }
          }
          if (!ok) break;
          ok = warp_wait(v_empty(vr.stage), vr.parity ^ 1);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(v_full(vr.stage), live * G::kBlockBytes);
            issued[1] = ++vc;
          }
          __syncwarp();
          if (lane < live)
            tma_load_5d(sbase + G::kV + vr.stage * G::kTileBytes + lane * G::kBlockBytes, &kv_map, v_full(vr.stage), 0,
                        0, 0, cur.h * (BS / 8), 2 * mine + 1);
          vr.next();
        }
        // the next item and its first table entries: a segment ahead, but
        // after the first loads of this one
        if (i == 0 && u + span < u_end) {
          after = next_item(cur);
          after_entries = fetch(after, 0);
        }
      }
      first = 0;
      u += span;
      k = 0;
      cur = after;
      ahead = after_entries;
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
  } else if (warp == kIssuer) {
    // ----------------------------------------------------------- MMA issue
    const uint32_t lead = lane == 0;
    constexpr uint64_t kHigh = (static_cast<uint64_t>(tc::kSwizzle128B) << 61) | (1ull << 46);
    constexpr uint64_t kQDesc = kHigh | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 16);
    constexpr uint64_t kKDesc = kHigh | (static_cast<uint64_t>(G::kGroupStride >> 4) << 32) | (1ull << 16);
    constexpr uint64_t kVDesc = kHigh | (static_cast<uint64_t>(G::kGroupStride >> 4) << 32) |
                                (static_cast<uint64_t>(G::kSlabs > 1 ? 1024 >> 4 : 0) << 16);
    struct Walk {
      int seg = 0;    // segments entered
      int g0 = 0;     // global step at the segment's start
      int g = 0;      // next step
      int steps = 0;  // of the segment; 0 before the first
      bool two = false, end = false;
      int tail = 0;   // positions from the segment's first tile to the request's end
      int nodes = 0;
    };
    Walk sw, pw;
    Ring<KS> kr;
    Ring<VS> vr;
    int qc = 0, q_seg = 0;  // query tiles used by earlier segments, by this one
    int kc = 0, vc = 0, q_commits0 = 0, q_commits1 = 0;
    // the segment of step w.g; false on a time-out
    auto enter = [&](Walk& w) -> bool {
      while (!w.end && w.g == w.g0 + w.steps) {
        const int j = w.seg % G::kSegs;
        if (!warp_wait(seg_full(j), (w.seg / G::kSegs) & 1)) return false;
        w.g0 = w.g;
        w.steps = __shfl_sync(kFull, segs[j].steps, 0);
        w.two = (__shfl_sync(kFull, segs[j].flags, 0) & kTwo) != 0;
        w.tail = __shfl_sync(kFull, segs[j].len - segs[j].tile0 * kTile, 0);
        w.nodes = __shfl_sync(kFull, segs[j].n, 0);
        ++w.seg;
        if (w.steps == 0) w.end = true;
      }
      return true;
    };
    // S of step sw.g, whose segment has been entered; `k_there`: its keys were
    // seen to be there
    auto issue_s = [&](bool k_there) -> bool {
      const int local = sw.g - sw.g0;
      const int tile = sw.two ? local >> 1 : local;
      const int rt = sw.two ? local & 1 : 0;
      const int qi = qc + rt;
      if (!k_there && !warp_wait(k_full(kr.stage), kr.parity)) return false;
      if (tile == 0 && !warp_wait(q_full(qi & 1), (qi >> 1) & 1)) return false;
      tc::fence_after_sync();
      const uint64_t kd = kKDesc | ((sbase + G::kK + kr.stage * G::kTileBytes) >> 4);
      const uint64_t qd = kQDesc | ((sbase + G::kQ + (qi & 1) * G::kQBytes) >> 4);
      const uint32_t d = tmem + G::kS + (sw.g & 1) * kTile;
      // the tile's tokens, rounded up to 16
      const uint32_t id = tc::idesc_bf16(kRows, min(kTile, (sw.tail - tile * kTile + 15) & ~15), false, false);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int x = i >> 2, kk = i & 3;
        tc::mma_ss(lead, d, qd + ((x * G::kQSlab + kk * 32) >> 4), kd + ((x * 1024 + kk * 32) >> 4), id, i > 0 ? 1u : 0u);
      }
      tc::commit_by(lead, s_full(sw.g & 1));
      if (!sw.two || rt == 1) {
        tc::commit_by(lead, k_empty(kr.stage));
        kr.next();
        ++kc;
      }
      if (local >= sw.steps - (sw.two ? 2 : 1)) {  // the row tile's last S
        tc::commit_by(lead, q_empty(qi & 1));
        if (qi & 1) ++q_commits1;
        else ++q_commits0;
      }
      ++sw.g;
      return true;
    };
    // the segment of the next S; its query tiles follow those of the one before
    auto enter_s = [&]() -> bool {
      if (sw.g != sw.g0 + sw.steps || sw.end) return true;
      qc += q_seg;
      if (!enter(sw)) return false;
      q_seg = sw.end ? 0 : sw.two ? 2 : 1;
      return true;
    };
    bool ok = true;
    for (int i = 0; i < 2 && ok; ++i) ok = enter_s() && (sw.end || issue_s(false));
    while (ok) {
      ok = enter(pw);
      if (!ok || pw.end) break;
      // Steps in the middle of a segment, where both products are of whole
      // tiles that need nothing else: few instructions per step, because this
      // warp shares its quarter of the SM with softmax warps, and what it
      // spends between two products the tensor cores wait for
      if (pw.seg == sw.seg && sw.g == pw.g + 2 && pw.g - pw.g0 >= 2) {
        const int shift = pw.two ? 1 : 0;
        const int whole = pw.tail / kTile;                           // whole tiles
        const int clean = max(0, pw.tail - pw.nodes) / kTile;        // of these, without nodes
        // PV of steps below `clean`, S two steps later of a whole tile that is not the last
        int until = min(clean << shift, min((whole << shift) - 2, pw.steps - 3 - shift));
        until += pw.g0;
        while (pw.g < until) {
          const int s = pw.g & 1;
          const uint32_t kb = k_full(kr.stage), vb = v_full(vr.stage), pb = p_full(s);
          const bool k_polled = mbar_test_wait(kb, kr.parity);
          const bool v_there = mbar_test_wait(vb, vr.parity);
          const bool p_there = mbar_test_wait(pb, (pw.g >> 1) & 1);
          const uint64_t vd = kVDesc | ((sbase + G::kV + vr.stage * G::kTileBytes) >> 4);
          const uint64_t kd = kKDesc | ((sbase + G::kK + kr.stage * G::kTileBytes) >> 4);
          const int qi = qc + (pw.two ? (sw.g - sw.g0) & 1 : 0);
          const uint64_t qd = kQDesc | ((sbase + G::kQ + (qi & 1) * G::kQBytes) >> 4);
          const uint32_t p = tmem + G::kS + s * kTile;
          if (!__all_sync(kFull, v_there && p_there)) {
            ok = warp_wait(vb, vr.parity) && warp_wait(pb, (pw.g >> 1) & 1);
            if (!ok) break;
          }
          tc::fence_after_sync();
#pragma unroll
          for (int i = 0; i < kTile / 16; ++i)
            tc::mma_ts(lead, tmem + G::kO + s * D, p + 8 * i, vd + ((2 * i * G::kGroupStride) >> 4),
                       tc::idesc_bf16(kRows, D, false, true), 1u);
          if (!__all_sync(kFull, k_polled)) {
            ok = warp_wait(kb, kr.parity);
            if (!ok) break;
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int x = i >> 2, kk = i & 3;
            tc::mma_ss(lead, p, qd + ((x * G::kQSlab + kk * 32) >> 4), kd + ((x * 1024 + kk * 32) >> 4),
                       tc::idesc_bf16(kRows, kTile, false, false), i > 0 ? 1u : 0u);
          }
          tc::commit_by(lead, s_full(s));
          tc::commit_by(lead, pv_done(s));
          if (!pw.two || ((pw.g - pw.g0) & 1)) {
            tc::commit_by(lead, v_empty(vr.stage));
            tc::commit_by(lead, k_empty(kr.stage));
            vr.next();
            kr.next();
            ++vc;
            ++kc;
          }
          ++pw.g;
          ++sw.g;
        }
        if (!ok) break;
      }
      const int local = pw.g - pw.g0;
      const int s = pw.g & 1;
      const int tile = pw.two ? local >> 1 : local;
      const int left = pw.tail - tile * kTile;
      // a poll takes its time, so the three of a step are in flight together
      // (tests: a try may sleep, and the keys may never come)
      const bool v_there = mbar_test_wait(v_full(vr.stage), vr.parity);
      const bool p_there = mbar_test_wait(p_full(s), (pw.g >> 1) & 1);
      const bool k_polled = mbar_test_wait(k_full(kr.stage), kr.parity);
      const bool k_there = __all_sync(kFull, k_polled);
      if (!__all_sync(kFull, v_there && p_there))
        ok = warp_wait(v_full(vr.stage), vr.parity) && warp_wait(p_full(s), (pw.g >> 1) & 1);
      if (ok && left < pw.nodes + kTile) ok = warp_wait(v_clean(vr.stage), vr.parity);  // see the cleaning warps
      // the accumulator has been read at the end of the segment before;
      // waited for after P, which bounds how far behind its readers can be
      if (ok && local < 2 && pw.seg > 1) ok = warp_wait(o_free(s), (pw.seg - 2) & 1);
      if (!ok) break;
      tc::fence_after_sync();
      const uint64_t vd = kVDesc | ((sbase + G::kV + vr.stage * G::kTileBytes) >> 4);
      const uint32_t p = tmem + G::kS + s * kTile;
      const uint32_t d = tmem + G::kO + s * D;
      constexpr uint32_t id = tc::idesc_bf16(kRows, D, false, true);
      const uint32_t more = local >= 2;
      if (left > kTile - 16) {
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
          tc::mma_ts(lead, d, p + 8 * i, vd + ((2 * i * G::kGroupStride) >> 4), id, i > 0 ? 1u : more);
      } else {
#pragma unroll 1
        for (int i = 0; i < (left + 15) / 16; ++i)
          tc::mma_ts(lead, d, p + 8 * i, vd + ((2 * i * G::kGroupStride) >> 4), id, i > 0 ? 1u : more);
      }
      tc::commit_by(lead, pv_done(s));
      if (!pw.two || (local & 1)) {
        tc::commit_by(lead, v_empty(vr.stage));
        vr.next();
        ++vc;
      }
      ++pw.g;
      ok = enter_s();
      if (ok && !sw.end) ok = issue_s(k_there);
    }
    if (!ok && lane == 0) give_up();
    __syncwarp();
    // every issued product has finished before tensor memory is released,
    // and every commit's arrival has landed before shared memory goes away
    tc::commit_by(lead, drain);
    wait(drain, 0);
    auto wait_last = [&](uint32_t at, int commits) {
      if (commits > 0) wait(at, (commits - 1) & 1);
    };
    for (int st = 0; st < KS; ++st) wait_last(k_empty(st), kc > st ? (kc - st + KS - 1) / KS : 0);
    for (int st = 0; st < VS; ++st) wait_last(v_empty(st), vc > st ? (vc - st + VS - 1) / VS : 0);
    wait_last(q_empty(0), q_commits0);
    wait_last(q_empty(1), q_commits1);
    for (int j = 0; j < 2; ++j) {
      wait_last(pv_done(j), (pw.g + 1 - j) >> 1);
      wait_last(s_full(j), (sw.g + 1 - j) >> 1);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------- cleaning value tiles
    // first the rows that have no node: 0.  A request's are one piece of out
    {
      constexpr int kPiece = 8192;  // bytes per turn of a CTA
      const int64_t row_bytes = static_cast<int64_t>(a.num_q_heads) * D * 2;
      const int pieces = static_cast<int>((a.nodes * row_bytes + kPiece - 1) / kPiece);
      for (int64_t i = blockIdx.x; i < static_cast<int64_t>(a.batch) * pieces; i += gridDim.x) {
        const int b = static_cast<int>(i / pieces);
        int len, n;
        tree_lengths<BS>(a, b, false, len, n);
        const int64_t lo = max(n * row_bytes, (i - static_cast<int64_t>(b) * pieces) * kPiece);
        const int64_t hi = min(a.nodes * row_bytes, (i - static_cast<int64_t>(b) * pieces + 1) * kPiece);
        char* out = reinterpret_cast<char*>(a.out) + b * a.nodes * row_bytes;
        for (int64_t at = lo + threadIdx.x * 16; at < hi; at += 64 * 16)
          *reinterpret_cast<uint4*>(out + at) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    Ring<VS> vr;
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      const int j = seg % G::kSegs;
      ok = warp_wait(seg_full(j), (seg / G::kSegs) & 1);
      if (!ok) break;
      const int steps = segs[j].steps;
      if (steps == 0) break;
      const int tiles = (segs[j].flags & kTwo) ? steps >> 1 : steps;
      const int len = segs[j].len, base = len - segs[j].n;
      for (int i = 0; i < tiles && ok; ++i, vr.next()) {
        const int vs = vr.stage;
        ok = warp_wait(v_full(vs), vr.parity);
        if (!ok) break;
        const int pos0 = (segs[j].tile0 + i) * kTile;
        const int end = min(kTile, len - pos0);  // rows of the request
        const int pad = min(kTile, (end + 15) & ~15);
        const int from = max(0, base - pos0);
        if (from < pad) {
          const uint32_t vt = sbase + G::kV + vs * G::kTileBytes;
          constexpr int kChunks = D / 8;  // 16-byte chunks of a row
          bool found = false;
          for (int e = threadIdx.x + from * kChunks; e < pad * kChunks; e += 64) {
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
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(v_clean(vs));
          mbar_arrive(v_empty(vs));  // before the stage's next round there is no next v_clean
        }
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
        const int pos0 = (tile0 + (two ? (g - g0) >> 1 : g - g0)) * kTile;
        const bool open = pos0 + kTile <= base;  // nothing to mask
        uint32_t bits0 = kFull, bits1 = kFull, bits2 = kFull, bits3 = kFull;
        if (!open && valid) {  // asked for while S is under way
          bits0 = attended32(mask_row, pos0, base, n);
          bits1 = attended32(mask_row, pos0 + 32, base, n);
          bits2 = attended32(mask_row, pos0 + 64, base, n);
          bits3 = attended32(mask_row, pos0 + 96, base, n);
        }
        ok = warp_wait(s_full(s), (g >> 1) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        if (work) {
          const uint32_t sp = lanes + G::kS + s * kTile;
          if (!open || a.negative) {
            // masks and signs are settled in tensor memory, so that the code
            // below, which holds the whole row, is the same for every tile
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t bits = valid ? bits0 : 0u, sign = a.negative ? 0x80000000u : 0u;
              bits0 = bits1, bits1 = bits2, bits2 = bits3;
              uint32_t x[32];
              __syncwarp();
              tc::tmem_ld_x32(sp + 32 * c, x);
              tc::wait_ld_x32(x);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = (bits >> e) & 1u ? x[e] ^ sign : 0xff800000u;
              tc::tmem_st_x32(sp + 32 * c, x);
            }
            tc::wait_st();
          }
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // independent chains
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t r[2][32];
            tc::tmem_ld_x32(sp + 64 * c, r[0]);
            tc::tmem_ld_x32(sp + 64 * c + 32, r[1]);
            tc::wait_ld_x32(r[0]);
            tc::wait_ld_x32(r[1]);
#pragma unroll
            for (int e = 0; e < 64; e += 2)
              tops[(e >> 1) & 3] = max3(tops[(e >> 1) & 3], __uint_as_float(r[e >> 5][e & 31]), __uint_as_float(r[e >> 5][(e & 31) + 1]));
          }
          const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * a.scale_log2;
          const bool over = valid && top > m + kSlack;  // true while m = -inf and something is attended
          if (__any_sync(kFull, over)) {
            const float mn = over ? top : m;
            const float alpha = m == -INFINITY ? 0.f : ex2(m - mn);
            const float keep = m == mn ? 1.f : alpha;
            if (!fresh) {
              // O holds the sum through this stream's step before, which is
              // done: the products complete in order, and S of this step is
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                const uint32_t oa = lanes + G::kO + s * D + 16 * c;
                tc::tmem_ld_x16(oa, o);
                tc::wait_ld_x16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tc::tmem_st_x16(oa, o);
              }
            }
            l *= keep;
            m = mn;
          }
          const float shift = m == -INFINITY ? 0.f : m;
          const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), shift2 = make_float2(-shift, -shift);
          float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t r[2][32];
            tc::tmem_ld_x32(sp + 64 * c, r[0]);
            tc::tmem_ld_x32(sp + 64 * c + 32, r[1]);
            tc::wait_ld_x32(r[0]);
            tc::wait_ld_x32(r[1]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t p[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 x = fma2(make_float2(__uint_as_float(r[u][2 * e]), __uint_as_float(r[u][2 * e + 1])), scale2, shift2);
                p[e] = pack_bf16x2(ex2(x.x), ex2(x.y));
                sums[e & 1] = add2(sums[e & 1], make_float2(bf16lo_to_f32(p[e]), bf16hi_to_f32(p[e])));
              }
              tc::tmem_st_x16(sp + 32 * c + 16 * u, p);  // over S, which has been read
            }
          }
          l += (sums[0].x + sums[1].x) + (sums[0].y + sums[1].y);
          tc::wait_st();
          fresh = false;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(s));
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
      const bool none0 = m == -INFINITY && l == 0.f;  // the stream saw nothing of the row
      bool none1 = true;
      if (!two) {
        xch[s * kRows + row] = make_float2(m, l);
        mbar_arrive(xch_full(s));
        ok = warp_wait(xch_full(s ^ 1), xch_phase & 1);
        if (!ok) break;
        ++xch_phase;
        const float2 o = xch[(s ^ 1) * kRows + row];
        none1 = o.x == -INFINITY && o.y == 0.f;
        const float mn = fmaxf(m, o.x);
        keep0 = weight_of(m - mn);
        keep1 = weight_of(o.x - mn);
        l = l * keep0 + o.y * keep1;
        m = mn;
      }
      // with one row tile each warpgroup writes half of the columns
      __syncwarp();
      if (work) {
        const bool poison = segs[j].poison != 0;
        if (flags & kComplete) {
          const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // a row that attends to nothing gets 0
          keep0 *= inv;
          keep1 *= inv;
        }
        // an accumulator whose stream saw nothing of the row may hold anything
        const bool bare = __any_sync(kFull, none0 || (!two && none1));
        const int64_t out_row = (static_cast<int64_t>(b) * a.nodes + token) * a.num_q_heads + h * a.group + row_head;
        const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + segs[j].slot;
        const int part_row = rt * kRows + row;
        // 32 columns at a time: code that runs once per segment is short, or
        // fetching it would take longer than running it
        const int c_begin = two ? 0 : s * (D / 2), c_end = two ? D : (s + 1) * (D / 2);
#pragma unroll 1
        for (int col = c_begin; col < c_end; col += 32) {
          uint32_t own[32], other[32] = {};
          __syncwarp();
          tc::tmem_ld_x32(lanes + G::kO + s * D + col, own);
          if (!two) tc::tmem_ld_x32(lanes + G::kO + (s ^ 1) * D + col, other);
          tc::wait_ld_x32(own);
          tc::wait_ld_x32(other);
          if (!valid) continue;
          if (bare) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              own[e] = none0 ? 0u : own[e];
              other[e] = none1 ? 0u : other[e];
            }
          }
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2 x = mul2(make_float2(__uint_as_float(other[e]), __uint_as_float(other[e + 1])), make_float2(keep1, keep1));
            x = fma2(make_float2(__uint_as_float(own[e]), __uint_as_float(own[e + 1])), make_float2(keep0, keep0), x);
            o[e] = x.x;
            o[e + 1] = x.y;
          }
          if (poison) {
            // values of attended nodes that are not finite
            const int tiles = two ? steps >> 1 : steps;
            const int lo = max(base, tile0 * kTile), hi = min(len, (tile0 + tiles) * kTile);
            for (int p = lo; p < hi; ++p) {
              const int i = p - base;
              if (!((mask_row[i >> 5] >> (i & 31)) & 1u)) continue;
              const int block = a.block_tables[static_cast<int64_t>(b) * a.max_blocks + p / BS];
              if (static_cast<unsigned>(block) >= static_cast<unsigned>(a.num_blocks)) continue;
              const __nv_bfloat16* v = a.pool + ((static_cast<int64_t>(block) * 2 + 1) * hkv + h) * BS * D + (p % BS) * D + col;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float x = __bfloat162float(v[e]);
                o[e] += isfinite(x) ? 0.f : x;
              }
            }
          }
          if (flags & kComplete) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(o[16 * x + 2 * e], o[16 * x + 2 * e + 1]);
              store_32_bytes(a.out + out_row * D + col + 16 * x, w, a.wide_out);
            }
          } else {
            float4* to = a.part_o + (slot * (D / 4) + col / 4) * (2 * kRows) + part_row;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              to[e * (2 * kRows)] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (valid && !(flags & kComplete) && c_begin == 0) a.part_ml[slot * (2 * kRows) + part_row] = make_float2(m, l);
      }
      __syncwarp();
      tc::fence_before_sync();  // the next segment's first products overwrite O
      if (two) {
        mbar_arrive_n(o_free(s), 2);
      } else {
        mbar_arrive(o_free(0));
        mbar_arrive(o_free(1));
      }
      g0 = g1;
    }
    if (!ok && lane == 0) give_up();
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // unwind: let every issued load land before the CTA's memory goes away
    for (int i = max(0, issued[0] - KS); i < issued[0]; ++i) wait(k_full(i % KS), (i / KS) & 1);
    for (int i = max(0, issued[1] - VS); i < issued[1]; ++i) wait(v_full(i % VS), (i / VS) & 1);
    for (int i = max(0, issued[2] - 2); i < issued[2]; ++i) wait(q_full(i & 1), (i >> 1) & 1);
  }
  __syncthreads();
  if (warp == kIssuer) {
    __syncwarp();
    tc::tmem_dealloc(tmem, G::kTmemCols);
  }
}

// Joins the partials of items cut between CTAs, in the order of the CTAs.  An
// item is found by the first CTA that continues it; a block takes 32 rows of
// it: lane = row, a warp D / 32 column groups of four, so a partial is read
// 512 bytes at a time; the rows are written out through shared memory.  Its
// bytes bound it when many items are cut (32 requests of 512 rows per KV head:
// 33 MB, 16 us cold, 12 us of a call), else its start: 4 us of a call.
constexpr int kMergeWarps = 8;
constexpr int kMergeBatch = 4;  // partials in flight

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const TreeArgs a, int launched) {
  constexpr int kGroups = D / 4 / kMergeWarps;  // column groups per warp
  constexpr int kPitch = D / 2 + 4;             // 32-bit words of a staged row
  __shared__ uint32_t staged[32 * kPitch];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x + 1;  // the CTA that continues the item
  const int* share = a.shares + c * kShare;
  const int first_tile = share[kShareTile], tiles = share[kShareTiles], total = share[kShareTotal];
  if (first_tile <= 0 || first_tile >= tiles) return;  // it begins with an item, or is idle
  const Split split(total, launched, a.cta_factor);
  const int u0 = split.begin(c) - first_tile;
  const int before = split.begin(c - 1);
  if (before > u0) return;  // the CTA before continues it already
  const int c0 = c - 1;
  const int parts = split.holder(u0 + tiles - 1) - c0 + 1;
  const int b = share[kShareB], h = share[kShareH], n = share[kShareNodes];
  const int rt = blockIdx.y / (kRows / 32);
  const int token0 = (share[kSharePair] * 2 + rt) * a.tile_tokens;
  const int row0 = (blockIdx.y % (kRows / 32)) * 32;  // of the row tile
  const int rows = min(a.tile_tokens, n - token0) * a.group;
  if (row0 >= rows) return;
  float4 o[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row0 + lane < rows) {
    const int slot0 = 2 * c0 + (before == u0 ? 0 : 1);  // the later CTAs begin with this item
    const int part_row = rt * kRows + row0 + lane;
    float top = -INFINITY, l = 0.f;
    for (int f0 = 0; f0 < parts; f0 += kMergeBatch) {
      float2 ml[kMergeBatch];
      float4 v[kMergeBatch][kGroups];
      float mn = top;
#pragma unroll
      for (int y = 0; y < kMergeBatch; ++y) {
        const int f = min(f0 + y, parts - 1);
        const int64_t at = f == 0 ? slot0 : 2 * (c0 + f);
        ml[y] = a.part_ml[at * (2 * kRows) + part_row];
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
          v[y][i] = a.part_o[(at * (D / 4) + warp * kGroups + i) * (2 * kRows) + part_row];
      }
#pragma unroll
      for (int y = 0; y < kMergeBatch; ++y)
        if (f0 + y < parts) mn = fmaxf(mn, ml[y].x);
      const float keep = top == -INFINITY ? 0.f : weight_of(top - mn);
      l *= keep;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) o[i] = make_float4(o[i].x * keep, o[i].y * keep, o[i].z * keep, o[i].w * keep);
      top = mn;
#pragma unroll
      for (int y = 0; y < kMergeBatch; ++y) {
        // a partial that saw nothing of the row weighs nothing
        if (f0 + y >= parts || (ml[y].x == -INFINITY && ml[y].y == 0.f)) continue;
        const float w = weight_of(ml[y].x - mn);
        l += ml[y].y * w;
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
          o[i] = make_float4(fmaf(v[y][i].x, w, o[i].x), fmaf(v[y][i].y, w, o[i].y), fmaf(v[y][i].z, w, o[i].z),
                             fmaf(v[y][i].w, w, o[i].w));
      }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) o[i] = make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv);
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
    *reinterpret_cast<uint2*>(staged + lane * kPitch + 2 * (warp * kGroups + i)) =
        make_uint2(pack_bf16x2(o[i].x, o[i].y), pack_bf16x2(o[i].z, o[i].w));
  __syncthreads();
  constexpr int kLanes = D / 8;  // 16-byte pieces of a row
  for (int x = threadIdx.x; x < 32 * kLanes; x += 32 * kMergeWarps) {
    const int r = x / kLanes, piece = x % kLanes;
    if (row0 + r >= rows) break;
    const int tl = (row0 + r) / a.group;
    const int64_t out_row = (static_cast<int64_t>(b) * a.nodes + token0 + tl) * a.num_q_heads + h * a.group + (row0 + r - tl * a.group);
    *reinterpret_cast<uint4*>(a.out + out_row * D + 8 * piece) = *reinterpret_cast<const uint4*>(staged + r * kPitch + 4 * piece);
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
  size_t part_o, part_ml, shares, bytes;
};

// Two partial slots of two row tiles per CTA, one CTA per SM.
Workspace workspace_layout(int d) {
  const size_t ctas = std::max(sm_count(), 1);
  const size_t rows = ctas * 2 * (2 * kRows);
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  Workspace w;
  w.part_o = 0;
  w.part_ml = up(rows * d * sizeof(float));
  w.shares = w.part_ml + up(rows * sizeof(float2));
  w.bytes = w.shares + up(ctas * kShare * sizeof(int));
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
  if (ctas > 1) {
    const int chunks = a.nodes > a.tile_tokens ? 2 * kRows / 32 : (a.tile_tokens * a.group + 31) / 32;
    PA_CUDA_TRY(launch_pdl(tree_merge_kernel<D>, dim3(static_cast<unsigned>(ctas - 1), static_cast<unsigned>(chunks)),
                           dim3(32 * kMergeWarps), 0, st, a, ctas));
  }
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
  *bytes_out = workspace_layout(head_dim).bytes;
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
  // smallest normal for 0: masked logits stay -inf, the others vanish
  const float scale_log2 = scale == 0.f ? FLT_MIN : fabsf(scale) * 1.4426950408889634f;
  if (!std::isfinite(scale_log2)) return fail(PA_ERR_INVALID, "%s: scale is not finite, or not times log2(e)", who);
  if (batch == 0) return PA_OK;
  if (!out || !q || !kv_pool || !tree_mask || !block_tables || !seq_lens || !workspace)
    return fail(PA_ERR_INVALID, "%s: NULL pointer", who);
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(kv_pool, 16) || !aligned(tree_mask, 4) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(tree_lens, 4) || !aligned(workspace, 256))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", who);
  const uintptr_t bytes = static_cast<uintptr_t>(batch) * num_nodes * num_q_heads * head_dim * sizeof(pa_bf16);
  const uintptr_t out_at = reinterpret_cast<uintptr_t>(out), q_at = reinterpret_cast<uintptr_t>(q);
  if (out_at < q_at + bytes && q_at < out_at + bytes) return fail(PA_ERR_INVALID, "%s: out overlaps q", who);
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
  a.max_seq_len = std::min(max_seq_len, 0x7fffffff - 4096);  // positions of a tile stay in range
  a.scale_log2 = scale_log2;
  a.negative = scale < 0.f;
  a.tile_tokens = std::min(kRows / a.group, num_nodes);
  a.pairs = (num_nodes + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
  // exact: the factor is above 2^20 / d by less than 1, x d <= 1279 * 256 < 2^20
  a.pair_factor = ((1 << 20) + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
  // ending one item and beginning the next takes as long as some tiles.  With
  // 1, 2, 3, 4, 6: 64 trees of 16 116.0, 110.4, 109.8, 111.1, 112.9 us; 512 rows
  // per KV head 195.7, 195.2, 194.0, 194.6, 196.4; ragged short requests at head
  // dim 64 27.6, 25.6, 25.8, 26.5, 27.3; long contexts 97.8 to 98.8 with any
  a.extra = 3;
  const unsigned ctas = std::max(sm_count(), 1);
  a.cta_factor = ctas > 1 ? 0xffffffffu / ctas + 1 : 0;  // exact: x ctas < ctas^3 < 2^32
  const int64_t longest = std::min(static_cast<int64_t>(max_seq_len), static_cast<int64_t>(max_blocks_per_seq) * block_size);
  if (static_cast<int64_t>(batch) * num_kv_heads * a.pairs > 0x7fffffffll / ((longest + kTile - 1) / kTile + a.extra))
    return fail(PA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 tiles of work at these sizes", who);
  const Workspace w = workspace_layout(head_dim);
  char* ws = static_cast<char*>(workspace);
  a.wide_out = aligned(out, 32);
  a.part_o = reinterpret_cast<float4*>(ws + w.part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  a.shares = reinterpret_cast<int*>(ws + w.shares);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (head_dim == 128) return block_size == 16 ? launch_tree<128, 16>(a, q, st) : launch_tree<128, 32>(a, q, st);
  return block_size == 16 ? launch_tree<64, 16>(a, q, st) : launch_tree<64, 32>(a, q, st);
}

}  // extern "C"
