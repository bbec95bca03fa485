// RMS norm of every query and key head and the rotation by position, in one pass over q and k; K and
// V can go to the paged cache in the same pass.
//
// Per row x of d channels: y = x * rsqrt(mean(x^2) + eps) * w, then the first `rot` channels are
// rotated in pairs, (a, b) -> (a cos - b sin, b cos + a sin), with cos and sin of position and pair
// from a float32 table.  Everything is computed in float32 and rounded to bf16 once.
//
// Bound by HBM: 2 bytes in and 2 bytes out a value, a few flops each.  A thread holds 8 consecutive
// channels (16 bytes) of a row and d / 8 threads a row, so a row's sum of squares is a few shuffles.
// Such a group takes ROWS rows (heads) of one token, whose loads are all in flight before the first
// is used: one load a thread would leave 16 KB an SM in flight, a third of what HBM needs.  With
// a = w cos of its own channels and b = +-w' sin of their partners', both made once for the rows of a
// kind, an output is r (x a + y b), r the row's norm factor.  With pairs (i, i + rot / 2) the partners
// are 8 channels of another thread of the row, exchanged as four words of raw bf16 pairs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "prefill.h"  // FastDiv
#include "sm103.cuh"
#include "step.h"

namespace attn {

__device__ uint32_t g_qk_rope_status;

namespace {

// Measured on 32749 tokens of 16 + 2 heads, d = 256 (604 MB): 64 threads a CTA 103 us, 128 107 us, 256
// 122 us (fewer warps wait for the slowest of their CTA); 8 rows a group 103 us, 4 108 us, 2 133 us.
constexpr int THREADS = 64;
constexpr int ROWS = 8;  // rows a group of threads takes, their loads in flight together

// eight bf16 values as four pairs of floats
__device__ __forceinline__ void unpack8(const uint4& u, uint64_t (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint32_t pack2(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return pack_bf16x2(a, b);
}

__device__ __forceinline__ uint64_t f2_swap(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return f2_pack(b, a);
}

// Group gid (D / 8 threads) takes part gid % parts of token gid / parts: up to ROWS query heads in the
// first q_parts parts, key heads in the next k_parts, value heads (copied to the cache) in the rest.
// NORM: there is a weight for queries or keys.
template <int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(THREADS)
    qk_rope_kernel(const QkRopeParams p, int q_parts, int k_parts, uint32_t parts, FastDiv div_parts) {
  constexpr int LPR = D / 8;  // threads a row
  const int sub = threadIdx.x % LPR;
  const uint32_t gid = (blockIdx.x * THREADS + threadIdx.x) / LPR;
  const uint32_t token = div_parts.div(gid);
  if (token >= static_cast<uint32_t>(p.T)) return;  // whole groups fall out together
  const int64_t t = token;
  const int part = static_cast<int>(gid - token * parts);
  const int row_lane0 = threadIdx.x & 31 & ~(LPR - 1);
  const unsigned row_mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << row_lane0;
  const int c0 = sub * 8;
  const bool is_q = part < q_parts, is_v = part >= q_parts + k_parts;
  const int h0 = (is_q ? part : is_v ? part - q_parts - k_parts : part - q_parts) * ROWS;
  const int n = min(ROWS, (is_q ? p.Hq : p.Hkv) - h0);
  const __nv_bfloat16* src =
      (is_q ? p.q + t * p.q_stride : is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride) + h0 * D + c0;
  const bool turns = c0 < p.rot;
  int pos = turns && !is_v ? p.positions[t] : 0;
  int64_t slot = !is_q && p.k_cache != nullptr ? p.slots[t] : -1;

  uint4 raw[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (i < n) raw[i] = __ldcs(reinterpret_cast<const uint4*>(src + i * D));
  }
  if (slot >= p.num_slots) {
    if (h0 == 0 && sub == 0) set_error(&g_qk_rope_status, kDevBadSlot);
    slot = -1;
  }
  __nv_bfloat16* cache = nullptr;
  if (slot >= 0) cache = (is_v ? p.v_cache : p.k_cache) + (slot * p.Hkv + h0) * D + c0;
  if (is_v) {
    if (cache != nullptr) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        if (i < n) *reinterpret_cast<uint4*>(cache + i * D) = raw[i];
    }
    return;
  }
  __nv_bfloat16* out = is_q ? p.q_out + t * p.q_out_stride + h0 * D + c0
                            : p.k_out != nullptr ? p.k_out + t * p.k_out_stride + h0 * D + c0 : nullptr;

  // an output is r (x * own + y * other), y the partner channel's value
  const int half = p.rot / 2;
  const int partner = INTERLEAVED || !turns ? sub : (c0 < half ? sub + half / 8 : sub - half / 8);
  uint64_t own[4], other[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    own[j] = f2_pack(1.f, 1.f);
    other[j] = f2_pack(0.f, 0.f);
  }
  if (turns) {
    if (pos < 0 || pos >= p.max_positions) {
      if (h0 == 0 && sub == 0) set_error(&g_qk_rope_status, kDevBadPosition);
      pos = pos < 0 ? 0 : p.max_positions - 1;
    }
    const int pair = INTERLEAVED ? c0 / 2 : (c0 < half ? c0 : c0 - half);
    const float* row = p.table + static_cast<int64_t>(pos) * p.rot + pair;
    if constexpr (INTERLEAVED) {
      const float4 c = *reinterpret_cast<const float4*>(row), s = *reinterpret_cast<const float4*>(row + half);
      own[0] = f2_pack(c.x, c.x); own[1] = f2_pack(c.y, c.y); own[2] = f2_pack(c.z, c.z); own[3] = f2_pack(c.w, c.w);
      other[0] = f2_pack(-s.x, s.x); other[1] = f2_pack(-s.y, s.y);
      other[2] = f2_pack(-s.z, s.z); other[3] = f2_pack(-s.w, s.w);
    } else {
      const float sign = c0 < half ? -1.f : 1.f;
      const uint64_t sign2 = f2_pack(sign, sign);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 c = reinterpret_cast<const float4*>(row)[i], s = reinterpret_cast<const float4*>(row + half)[i];
        own[2 * i] = f2_pack(c.x, c.y); own[2 * i + 1] = f2_pack(c.z, c.w);
        other[2 * i] = f2_mul(f2_pack(s.x, s.y), sign2); other[2 * i + 1] = f2_mul(f2_pack(s.z, s.w), sign2);
      }
    }
  }
  const __nv_bfloat16* weight = is_q ? p.q_weight : p.k_weight;
  if (NORM && weight != nullptr) {
    uint64_t w[4], v[4];
    unpack8(*reinterpret_cast<const uint4*>(weight + c0), w);
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f2_swap(w[j]);
    } else {
      unpack8(*reinterpret_cast<const uint4*>(weight + partner * 8), v);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      own[j] = f2_mul(own[j], w[j]);
      other[j] = f2_mul(other[j], v[j]);
    }
  }

#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (i >= n) break;
    uint64_t x[4], y[4];
    unpack8(raw[i], x);
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = turns ? f2_swap(x[j]) : 0;  // not y * 0: an infinity would give NaN
    } else {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (p.rot > 0) {
        const int from = row_lane0 + partner;
        u.x = __shfl_sync(row_mask, raw[i].x, from);
        u.y = __shfl_sync(row_mask, raw[i].y, from);
        u.z = __shfl_sync(row_mask, raw[i].z, from);
        u.w = __shfl_sync(row_mask, raw[i].w, from);
        if (!turns) u = make_uint4(0, 0, 0, 0);
      }
      unpack8(u, y);
    }
    uint64_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = f2_fma(x[j], own[j], f2_mul(y[j], other[j]));
    if (NORM && weight != nullptr) {
      const uint64_t sq = f2_fma(x[3], x[3], f2_fma(x[2], x[2], f2_fma(x[1], x[1], f2_mul(x[0], x[0]))));
      float ss, ss_hi;
      f2_unpack(sq, ss, ss_hi);
      ss += ss_hi;
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(row_mask, ss, off);
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
      const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = f2_mul(r[j], inv2);
    }
    const uint4 packed = make_uint4(pack2(r[0]), pack2(r[1]), pack2(r[2]), pack2(r[3]));
    if (out != nullptr) *reinterpret_cast<uint4*>(out + i * D) = packed;
    if (cache != nullptr) *reinterpret_cast<uint4*>(cache + i * D) = packed;
  }
}

// cos and sin of position * theta^(-2 i / rot), the angle in double: a float32 angle at position 10^6
// would be off by 0.06
__global__ void rope_table_kernel(float* table, int max_positions, int rot, double log2_theta) {
  const int half = rot / 2;
  const int64_t total = static_cast<int64_t>(max_positions) * half;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t pos = i / half;
    const int pair = static_cast<int>(i % half);
    const double angle = pos * exp2(-log2_theta * (2.0 * pair / rot));
    double s, c;
    sincos(angle, &s, &c);
    table[pos * rot + pair] = static_cast<float>(c);
    table[pos * rot + half + pair] = static_cast<float>(s);
  }
}

template <int D>
cudaError_t launch(const QkRopeParams& p, cudaStream_t stream) {
  const int q_parts = (p.Hq + ROWS - 1) / ROWS, k_parts = (p.Hkv + ROWS - 1) / ROWS;
  const uint32_t parts = static_cast<uint32_t>(q_parts + k_parts * (p.v_cache != nullptr ? 2 : 1));
  const FastDiv div = FastDiv::make(parts);
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.T) * parts * (D / 8) + THREADS - 1) / THREADS);
  const bool norm = p.q_weight != nullptr || p.k_weight != nullptr;
  if (p.interleaved && norm)
    qk_rope_kernel<D, true, true><<<grid, THREADS, 0, stream>>>(p, q_parts, k_parts, parts, div);
  else if (p.interleaved)
    qk_rope_kernel<D, true, false><<<grid, THREADS, 0, stream>>>(p, q_parts, k_parts, parts, div);
  else if (norm)
    qk_rope_kernel<D, false, true><<<grid, THREADS, 0, stream>>>(p, q_parts, k_parts, parts, div);
  else
    qk_rope_kernel<D, false, false><<<grid, THREADS, 0, stream>>>(p, q_parts, k_parts, parts, div);
  return cudaGetLastError();
}

}  // namespace

cudaError_t qk_rope_launch(const QkRopeParams& p, cudaStream_t stream) {
  if (p.d == 64) return launch<64>(p, stream);
  if (p.d == 128) return launch<128>(p, stream);
  if (p.d == 256) return launch<256>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t rope_table_launch(float* table, int max_positions, int rot, double theta, cudaStream_t stream) {
  const int64_t total = static_cast<int64_t>(max_positions) * (rot / 2);
  const int64_t blocks = (total + 255) / 256;
  rope_table_kernel<<<static_cast<int>(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(table, max_positions, rot,
                                                                                       log2(theta));
  return cudaGetLastError();
}

cudaError_t qk_rope_status(uint32_t* out, bool clear) { return read_status(g_qk_rope_status, out, clear); }

}  // namespace attn
