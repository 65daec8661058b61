// pa_norm_rope_and_cache: per-head RMS norms of queries and keys, the
// position rotation, and the cache write, in one pass over the projections.
//
//   y = x * rsqrt(mean(x^2) + eps) * w,  (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)
//
// Bytes bound it: every query, key and value row is read once and written
// once.  head_dim / 16 lanes share a row, 16 elements (two 16-byte chunks)
// each, placed so that both elements of every rotated pair are in one
// thread: with half-split pairs lane l holds chunks l and l + rotary_dim / 16,
// with interleaved pairs chunks 2l and 2l + 1; either way it rotates by the
// angles 8l .. 8l + 7.  The lanes past the rotated chunks take the rest, two
// by two.  Sums and products are fp32, rounded to bf16 once.
#include <cuda_runtime.h>

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
  int64_t total;  // rows: tokens * (q heads + kv heads (k) + kv heads (v, when cached))
  int num_q_heads, num_kv_heads, rows_per_token;
  int block_size;
  int64_t num_slots;
  int32_t* err;
};

constexpr int kRopeThreads = 256;

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
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeArgs a) {
  constexpr int kLanes = D / 16;  // per row
  pdl_trigger();
  pdl_wait();
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) / kLanes;
  const int l = threadIdx.x & (kLanes - 1);
  const bool live = row < a.total;
  const int64_t token = live ? row / a.rows_per_token : 0;
  const int r = live ? static_cast<int>(row - token * a.rows_per_token) : 0;
  const bool is_q = r < a.num_q_heads;
  const bool is_v = r >= a.num_q_heads + a.num_kv_heads;
  const int head = is_q ? r : (r - a.num_q_heads) % max(a.num_kv_heads, 1);

  // the two chunks of this lane
  const int turned = a.rotary_dim / 16;  // lanes that rotate
  const bool turns = l < turned && !is_v;
  int c0, c1;
  if (l < turned && !a.interleaved) {
    c0 = l;
    c1 = l + turned;
  } else {
    c0 = 2 * l;
    c1 = 2 * l + 1;
  }
  const __nv_bfloat16* src = is_q ? a.q + token * a.q_stride : is_v ? a.v + token * a.v_stride : a.k + token * a.k_stride;
  const uint4* from = reinterpret_cast<const uint4*>(src + head * D);
  int pos = 0;
  int64_t slot = -1;
  uint4 u0 = {}, u1 = {};
  if (live) {
    u0 = from[c0];
    u1 = from[c1];
    if (a.rotary_dim > 0 || a.positions != nullptr) pos = a.positions[token];
    if (a.pool != nullptr && !is_q) slot = a.slots[token];
  }
  const bool beyond = a.rotary_dim > 0 && pos >= a.max_position;
  const bool padding = pos < 0 || beyond;
  if (live && l == 0 && r == 0) {
    if (beyond) flag_error(a.err, PA_DEVERR_POSITION);
  }
  if (slot >= a.num_slots) {
    if (live && l == 0 && !is_v && head == 0) flag_error(a.err, PA_DEVERR_SLOT);
    slot = -1;
  }
  float x0[8], x1[8];
  unpack8(u0, x0);
  unpack8(u1, x1);
  float sum = 0.f;  // of the row's squares; every lane takes part in the shuffles
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += x0[i] * x0[i] + x1[i] * x1[i];
#pragma unroll
  for (int off = kLanes / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (!is_v) {
    const __nv_bfloat16* weight = is_q ? a.q_weight : a.k_weight;
    if (weight != nullptr) {
      const float scale = rsqrtf(sum * (1.f / D) + a.eps);
      float w0[8], w1[8];
      unpack8(reinterpret_cast<const uint4*>(weight)[c0], w0);
      unpack8(reinterpret_cast<const uint4*>(weight)[c1], w1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x0[i] = x0[i] * scale * w0[i];
        x1[i] = x1[i] * scale * w1[i];
      }
    }
    if (turns && live && !padding) {
      const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim + 8 * l;
      float c[8], s[8];
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + i);
        *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(cs + a.rotary_dim / 2 + i);
      }
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p0 = x0[2 * i], q0 = x0[2 * i + 1], p1 = x1[2 * i], q1 = x1[2 * i + 1];
          x0[2 * i] = p0 * c[i] - q0 * s[i];
          x0[2 * i + 1] = q0 * c[i] + p0 * s[i];
          x1[2 * i] = p1 * c[4 + i] - q1 * s[4 + i];
          x1[2 * i + 1] = q1 * c[4 + i] + p1 * s[4 + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = x0[i], q = x1[i];
          x0[i] = p * c[i] - q * s[i];
          x1[i] = q * c[i] + p * s[i];
        }
      }
    }
    u0 = padding ? make_uint4(0, 0, 0, 0) : pack8(x0);
    u1 = padding ? make_uint4(0, 0, 0, 0) : pack8(x1);
  }
  if (!live) return;
  if (is_q || (!is_v && a.k_out != nullptr)) {
    uint4* to = reinterpret_cast<uint4*>((is_q ? a.q_out + token * a.q_out_stride : a.k_out + token * a.k_out_stride) + head * D);
    to[c0] = u0;
    to[c1] = u1;
  }
  if (!is_q && slot >= 0 && !padding) {
    const int64_t block = slot / a.block_size;
    const int64_t at = ((block * 2 + (is_v ? 1 : 0)) * a.num_kv_heads + head) * a.block_size + (slot - block * a.block_size);
    a.pool[at * (D / 8) + c0] = u0;
    a.pool[at * (D / 8) + c1] = u1;
  }
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
  a.total = static_cast<int64_t>(num_tokens) * a.rows_per_token;
  a.block_size = block_size;
  a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  a.err = err;
  const int64_t grid = (a.total * (head_dim / 16) + kRopeThreads - 1) / kRopeThreads;
  if (grid > 0x7fffffffll) return fail(PA_ERR_INVALID, "%s: too many tokens", who);
  const dim3 g(static_cast<unsigned>(grid));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (head_dim == 128) PA_CUDA_TRY(launch_pdl(norm_rope_kernel<128>, g, dim3(kRopeThreads), 0, st, a));
  else PA_CUDA_TRY(launch_pdl(norm_rope_kernel<64>, g, dim3(kRopeThreads), 0, st, a));
  return PA_OK;
}
