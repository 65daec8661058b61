// pa_norm_rope_and_cache: per-head RMS norms of queries and keys, the
// position rotation, and the cache write, in one pass over the projections.
//
//   y = x * rsqrt(mean(x^2) + eps) * w,  (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)
//
// Bytes bound it: every query, key and value row is read once and written
// once.  head_dim / 16 lanes share a row, 16 elements (two 16-byte chunks)
// each, placed so that both elements of every rotated pair are in one thread:
// with half-split pairs lane l holds chunks l and l + rotary_dim / 16, with
// interleaved pairs chunks 2l and 2l + 1; either way it rotates by the angles
// 8l .. 8l + 7.  The lanes past the rotated chunks take the rest, two by two.
// A thread takes kRows rows of a token, all their loads in flight at once and
// the cosines and sines fetched once.  Sums and products are fp32, rounded to
// bf16 once.
//
// 16384 tokens of 32 + 8 + 8 heads of 128 (411 MB): 78 us = 5.3 TB/s, 80 % of
// a copy.  Without resident blocks it took 96 us, with 4 rows and 6 blocks per
// SM 88 us (spills), with 8 rows and 3 blocks 92 us, with streaming loads 80
// us.  1024 tokens (25.7 MB): 6.4 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <numeric>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

struct RopeArgs {
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  uint4* pool;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t q_out_stride, k_out_stride, q_stride, k_stride, v_stride;
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* k_weight;
  float eps;
  const float* cos_sin;
  int max_position, rotary_dim, interleaved;
  const int32_t* positions;
  const int64_t* slots;
  int num_q_heads, num_kv_heads;
  int64_t num_tokens;
  int rows_stride;     // groups of lanes per token: ceil(rows_per_token / kRows)
  int rows_per_token;  // query heads, KV heads (keys), KV heads again (values) when cached
  int block_size;
  int64_t num_slots;
  int32_t* err;
};

constexpr int kRopeThreads = 128;
constexpr int kRows = 6;  // rows of a thread
constexpr int kRopeBlocks = 4;  // per SM, resident

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo_to_f32(w[i]);
    f[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) norm_rope_kernel(const RopeArgs a) {
  constexpr int kLanes = D / 16;  // per row
  // the cache write and the fused append read new keys through the read-only
  // path: they must not be resident while k_out is written
  if (a.k_out == nullptr) pdl_trigger();
  pdl_wait();
  const int l = threadIdx.x & (kLanes - 1);
  // the two chunks of this lane
  const int turned = a.rotary_dim / 16;  // lanes that rotate
  const bool turns = l < turned;
  const int c0 = turns && !a.interleaved ? l : 2 * l;
  const int c1 = turns && !a.interleaved ? l + turned : 2 * l + 1;
  // groups of lanes: (token, first row), the rows of a group `stride` apart
  const int stride = a.rows_stride;
  const int64_t groups = a.num_tokens * stride, step = static_cast<int64_t>(gridDim.x) * (kRopeThreads / kLanes);
  auto token_of = [&](int64_t group) -> int64_t {
    return group <= 0xffffffffll ? static_cast<unsigned>(group) / static_cast<unsigned>(stride) : group / stride;
  };
  int64_t group = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) / kLanes;
  int64_t token = 0, slot_next = -1;
  int pos_next = 0;
  auto fetch = [&](int64_t g) {  // the token's position and slot, a round ahead of its rows
    token = token_of(g);
    if (g < groups) {
      if (a.positions != nullptr) pos_next = a.positions[token];
      if (a.pool != nullptr) slot_next = a.slots[token];
    }
  };
  fetch(group);
  // every lane of a warp makes the same rounds: the shuffles need all of them
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / kLanes); first < groups; first += step, group += step) {
    const int64_t at = token;
    const int rows = group < groups ? a.rows_per_token : 0;
    const int r_first = static_cast<int>(group - at * stride);
    const int pos = pos_next;
    int64_t slot = slot_next;
    const __nv_bfloat16* q = a.q + at * a.q_stride;
    const __nv_bfloat16* k = a.k + at * a.k_stride;
    const __nv_bfloat16* v = a.v + at * a.v_stride;
    // rows: queries, keys, and the values when they are cached
    auto row_at = [&](int r) -> const uint4* {
      const __nv_bfloat16* p = r < a.num_q_heads ? q + r * D
                               : r < a.num_q_heads + a.num_kv_heads ? k + (r - a.num_q_heads) * D
                                                                    : v + (r - a.num_q_heads - a.num_kv_heads) * D;
      return reinterpret_cast<const uint4*>(p);
    };
    uint4 u0[kRows], u1[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r_first + i * stride;
      if (r < rows) {
        const uint4* from = row_at(r);
        u0[i] = from[c0];
        u1[i] = from[c1];
      } else {
        u0[i] = u1[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    const bool beyond = a.rotary_dim > 0 && pos >= a.max_position && rows > 0;
    const bool padding = pos < 0 || beyond;
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
    }
    if (turns && !padding && rows > 0) {
      const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim + 8 * l;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + i);
        *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(cs + a.rotary_dim / 2 + i);
      }
    }
    fetch(group + step);
    if (r_first == 0 && l == 0 && rows > 0) {
      if (beyond) flag_error(a.err, PA_DEVERR_POSITION);
      if (slot >= a.num_slots) flag_error(a.err, PA_DEVERR_SLOT);
    }
    if (slot >= a.num_slots || padding) slot = -1;
    // key row of head 0 in the pool, in 16-byte chunks
    const int64_t block = slot / a.block_size;
    const int64_t pool_row = (block * 2 * a.num_kv_heads) * a.block_size + (slot - block * a.block_size);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r_first + i * stride;
      const bool is_q = r < a.num_q_heads, is_v = r >= a.num_q_heads + a.num_kv_heads;
      float x0[8], x1[8];
      unpack8(u0[i], x0);
      unpack8(u1[i], x1);
      float sum = 0.f;  // of the row's squares; every lane takes part in the shuffles
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += x0[e] * x0[e] + x1[e] * x1[e];
#pragma unroll
      for (int off = kLanes / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (r >= rows) continue;
      if (!is_v) {
        const __nv_bfloat16* weight = is_q ? a.q_weight : a.k_weight;
        if (weight != nullptr) {
          const float scale = rsqrtf(sum * (1.f / D) + a.eps);
          float w0[8], w1[8];
          unpack8(__ldg(reinterpret_cast<const uint4*>(weight) + c0), w0);
          unpack8(__ldg(reinterpret_cast<const uint4*>(weight) + c1), w1);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x0[e] = x0[e] * scale * w0[e];
            x1[e] = x1[e] * scale * w1[e];
          }
        }
        if (turns) {
          if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p0 = x0[2 * e], p1 = x0[2 * e + 1], p2 = x1[2 * e], p3 = x1[2 * e + 1];
              x0[2 * e] = p0 * c[e] - p1 * s[e];
              x0[2 * e + 1] = p1 * c[e] + p0 * s[e];
              x1[2 * e] = p2 * c[4 + e] - p3 * s[4 + e];
              x1[2 * e + 1] = p3 * c[4 + e] + p2 * s[4 + e];
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float p0 = x0[e], p1 = x1[e];
              x0[e] = p0 * c[e] - p1 * s[e];
              x1[e] = p1 * c[e] + p0 * s[e];
            }
          }
        }
        u0[i] = padding ? make_uint4(0u, 0u, 0u, 0u) : pack8(x0);
        u1[i] = padding ? make_uint4(0u, 0u, 0u, 0u) : pack8(x1);
      }
      if (is_q || (!is_v && a.k_out != nullptr)) {
        uint4* to = reinterpret_cast<uint4*>(is_q ? a.q_out + at * a.q_out_stride + r * D
                                                  : a.k_out + at * a.k_out_stride + (r - a.num_q_heads) * D);
        to[c0] = u0[i];
        to[c1] = u1[i];
      }
      if (!is_q && slot >= 0) {
        // heads of keys, then of values: block_size rows apart
        uint4* to = a.pool + (pool_row + static_cast<int64_t>(r - a.num_q_heads) * a.block_size) * (D / 8);
        to[c0] = u0[i];
        to[c1] = u1[i];
      }
    }
  }
}

// `count` rows of `row` bytes, `stride` bytes apart; count 0: not used.
struct Rows {
  const void* at;
  int64_t count, stride, row;
};

// Whether two of them share a byte.  Exact for equal strides, where rows meet
// when they meet modulo the stride; of different ones the greatest common
// divisor takes that place, and rows may be taken to meet that do not.
bool overlap(const Rows& a, const Rows& b) {
  if (a.count == 0 || b.count == 0) return false;
  const int64_t from = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at));
  if (from >= (a.count - 1) * a.stride + a.row || -from >= (b.count - 1) * b.stride + b.row) return false;
  const int64_t g = std::gcd(a.count > 1 ? a.stride : 0, b.count > 1 ? b.stride : 0);
  if (g == 0) return true;
  const int64_t at = (from % g + g) % g;
  return at < a.row || g - at < b.row;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace pa

extern "C" int pa_norm_rope_and_cache(pa_bf16* q_out, int64_t q_out_stride, pa_bf16* k_out, int64_t k_out_stride,
                                      pa_bf16* kv_pool, const pa_bf16* q, int64_t q_stride, const pa_bf16* k,
                                      int64_t k_stride, const pa_bf16* v, int64_t v_stride, const pa_bf16* q_weight,
                                      const pa_bf16* k_weight, float eps, const float* cos_sin, int max_position,
                                      int rotary_dim, int interleaved, const int32_t* positions,
                                      const int64_t* slot_mapping, int num_tokens, int num_q_heads, int num_kv_heads,
                                      int head_dim, int num_blocks, int block_size, void* stream) {
  using namespace pa;
  const char* who = "pa_norm_rope_and_cache";
  if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 || num_q_heads + static_cast<int64_t>(num_kv_heads) == 0)
    return fail(PA_ERR_INVALID, "%s: non-positive size", who);
  if (num_q_heads > 65536 || num_kv_heads > 65536)
    return fail(PA_ERR_UNSUPPORTED, "%s: %d and %d heads, beyond 65536", who, num_q_heads, num_kv_heads);
  if (head_dim != 64 && head_dim != 128) return fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d", who, head_dim);
  if (rotary_dim < 0 || rotary_dim % 16 != 0 || rotary_dim > head_dim)
    return fail(PA_ERR_INVALID, "%s: rotary_dim %d is not a multiple of 16 up to head_dim", who, rotary_dim);
  if (!(eps >= 0.f)) return fail(PA_ERR_INVALID, "%s: eps must not be negative", who);
  if (rotary_dim > 0 && max_position <= 0) return fail(PA_ERR_INVALID, "%s: an empty rotation table", who);
  if (kv_pool != nullptr && (num_blocks <= 0 || block_size <= 0)) return fail(PA_ERR_INVALID, "%s: an empty pool", who);
  if (num_tokens == 0) return PA_OK;
  if ((num_q_heads > 0 && (!q || !q_out)) || (num_kv_heads > 0 && (!k || (!kv_pool && !k_out))) ||
      (kv_pool && num_kv_heads > 0 && (!v || !slot_mapping)) || (rotary_dim > 0 && (!cos_sin || !positions)))
    return fail(PA_ERR_INVALID, "%s: NULL pointer", who);
  for (const void* p : {static_cast<const void*>(q), static_cast<const void*>(k), static_cast<const void*>(v),
                        static_cast<const void*>(q_out), static_cast<const void*>(k_out),
                        static_cast<const void*>(kv_pool), static_cast<const void*>(q_weight),
                        static_cast<const void*>(k_weight), static_cast<const void*>(cos_sin)})
    if (!aligned16(p)) return fail(PA_ERR_INVALID, "%s: misaligned pointer", who);
  if ((reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", who);
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim, k_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  const struct {
    bool used;
    int64_t stride, row;
  } strides[] = {{num_q_heads > 0, q_stride, q_row}, {num_q_heads > 0, q_out_stride, q_row},
                 {num_kv_heads > 0, k_stride, k_row}, {num_kv_heads > 0 && k_out, k_out_stride, k_row},
                 {num_kv_heads > 0 && kv_pool, v_stride, k_row}};
  for (const auto& s : strides)
    if (s.used && (s.stride < s.row || s.stride % 8 != 0))
      return fail(PA_ERR_INVALID, "%s: token stride %lld is below the heads' %lld elements or not a multiple of 8", who,
                  static_cast<long long>(s.stride), static_cast<long long>(s.row));
  if ((q_out == q && q_out_stride != q_stride && num_q_heads > 0) || (k_out && k_out == k && k_out_stride != k_stride))
    return fail(PA_ERR_INVALID, "%s: in place needs equal strides", who);
  // another group of lanes reads what an output over its input overwrites
  const int64_t qn = num_q_heads > 0 ? num_tokens : 0, kn = num_kv_heads > 0 ? num_tokens : 0;
  const Rows in_q{q, qn, 2 * q_stride, 2 * q_row}, in_k{k, kn, 2 * k_stride, 2 * k_row},
      in_v{v, kv_pool ? kn : 0, 2 * v_stride, 2 * k_row}, to_q{q_out, qn, 2 * q_out_stride, 2 * q_row},
      to_k{k_out, k_out ? kn : 0, 2 * k_out_stride, 2 * k_row},
      to_pool{kv_pool, kv_pool && kn ? 1 : 0, 0, 4 * k_row * num_blocks * block_size};
  if ((q_out != q && overlap(to_q, in_q)) || overlap(to_q, in_k) || overlap(to_q, in_v) || overlap(to_k, in_q) ||
      (k_out != k && overlap(to_k, in_k)) || overlap(to_k, in_v) || overlap(to_k, to_q) || overlap(to_pool, in_q) ||
      overlap(to_pool, in_k) || overlap(to_pool, in_v) || overlap(to_pool, to_q) || overlap(to_pool, to_k))
    return fail(PA_ERR_INVALID, "%s: an output overlaps an input or another output", who);
  int32_t* err = device_error_word();
  if (err == nullptr) return PA_ERR_CUDA;
  RopeArgs a;
  a.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  a.k_out = reinterpret_cast<__nv_bfloat16*>(k_out);
  a.pool = reinterpret_cast<uint4*>(kv_pool);
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.k = reinterpret_cast<const __nv_bfloat16*>(k);
  a.v = reinterpret_cast<const __nv_bfloat16*>(v);
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_weight = reinterpret_cast<const __nv_bfloat16*>(q_weight);
  a.k_weight = reinterpret_cast<const __nv_bfloat16*>(k_weight);
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.max_position = max_position;
  a.rotary_dim = rotary_dim;
  a.interleaved = interleaved != 0;
  a.positions = positions;
  a.slots = slot_mapping;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.rows_per_token = num_q_heads + num_kv_heads * (kv_pool ? 2 : 1);
  a.block_size = block_size;
  a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  a.err = err;
  a.num_tokens = num_tokens;
  a.rows_stride = (a.rows_per_token + kRows - 1) / kRows;
  // as many blocks as are resident, each going round: the position of the next
  // round's token is there when its rows and angles are asked for
  const int64_t blocks = (a.num_tokens * a.rows_stride * (head_dim / 16) + kRopeThreads - 1) / kRopeThreads;
  const int64_t grid = std::min(blocks, static_cast<int64_t>(std::max(sm_count(), 1)) * kRopeBlocks);
  const dim3 g(static_cast<unsigned>(grid));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (head_dim == 128) PA_CUDA_TRY(launch_pdl(norm_rope_kernel<128>, g, dim3(kRopeThreads), 0, st, a));
  else PA_CUDA_TRY(launch_pdl(norm_rope_kernel<64>, g, dim3(kRopeThreads), 0, st, a));
  return PA_OK;
}
