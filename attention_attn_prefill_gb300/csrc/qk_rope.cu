// RMS norm of every query and key head and the rotation by position, in one pass over q and k; K and
// V can go to the paged cache in the same pass.
//
// Per row x of d channels: y = x * rsqrt(mean(x^2) + eps) * w, then the first `rot` channels are
// rotated in pairs, (a, b) -> (a cos - b sin, b cos + a sin), with cos and sin of position and pair
// from a float32 table.  Everything is computed in float32 and rounded to bf16 once.
//
// Bound by HBM: 2 bytes in and 2 bytes out a value, a few flops each.  A thread holds 8 consecutive
// channels (16 bytes), d / 8 threads a row, so a row's sum of squares is a few shuffles.  With pairs
// (i, i + rot / 2) a thread's partners are 8 channels of another thread of the row: the four words
// of raw bf16 pairs are exchanged, not eight float32 results, since the partner's norm factor is the
// row's.  A thread keeps its cosines and sines in registers over the rows (heads) of a token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm103.cuh"
#include "step.h"

namespace attn {

__device__ uint32_t g_qk_rope_status;

namespace {

constexpr int THREADS = 256;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// A CTA takes THREADS / (D / 8) / lanes tokens; `lanes` groups of D / 8 threads share a token and walk
// its rows (query heads, key heads, and value heads where they are copied to the cache).
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) qk_rope_kernel(const QkRopeParams p, int lanes) {
  constexpr int LPR = D / 8;  // threads a row
  const int sub = threadIdx.x % LPR;
  const int grp = threadIdx.x / LPR;
  const int tokens = THREADS / LPR / lanes;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * tokens + grp / lanes;
  // whole groups fall out together; the shuffles below name the LPR threads of a row only
  if (grp / lanes >= tokens || t >= p.T) return;
  const int row_lane0 = threadIdx.x & 31 & ~(LPR - 1);
  const unsigned row_mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << row_lane0;
  const int rows = p.Hq + p.Hkv * (p.v_cache != nullptr ? 2 : 1);

  int64_t slot = -1;
  if (p.k_cache != nullptr) {
    slot = p.slots[t];
    if (slot >= p.num_slots) {
      if (grp % lanes == 0 && sub == 0) set_error(&g_qk_rope_status, kDevBadSlot);
      slot = -1;
    }
  }
  const int c0 = sub * 8;
  const bool turns = c0 < p.rot;
  const int half = p.rot / 2;
  float cs[INTERLEAVED ? 4 : 8], sn[INTERLEAVED ? 4 : 8];
  if (turns) {
    int pos = p.positions[t];
    if (pos < 0 || pos >= p.max_positions) {
      if (grp % lanes == 0 && sub == 0) set_error(&g_qk_rope_status, kDevBadPosition);
      pos = pos < 0 ? 0 : p.max_positions - 1;
    }
    const int pair = INTERLEAVED ? c0 / 2 : (c0 < half ? c0 : c0 - half);
    const float* row = p.table + static_cast<int64_t>(pos) * p.rot + pair;
#pragma unroll
    for (int i = 0; i < (INTERLEAVED ? 1 : 2); ++i) {
      const float4 a = reinterpret_cast<const float4*>(row)[i];
      const float4 b = reinterpret_cast<const float4*>(row + half)[i];
      cs[4 * i] = a.x; cs[4 * i + 1] = a.y; cs[4 * i + 2] = a.z; cs[4 * i + 3] = a.w;
      sn[4 * i] = b.x; sn[4 * i + 1] = b.y; sn[4 * i + 2] = b.z; sn[4 * i + 3] = b.w;
    }
  }
  // the thread of the row that holds the other halves of this thread's pairs
  const int partner = !turns ? sub : (c0 < half ? sub + half / 8 : sub - half / 8);

  for (int r = grp % lanes; r < rows; r += lanes) {
    const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv;
    const int h = is_q ? r : (is_v ? r - p.Hq - p.Hkv : r - p.Hq);
    const __nv_bfloat16* src = is_q ? p.q + t * p.q_stride : (is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride);
    const uint4 raw = *reinterpret_cast<const uint4*>(src + h * D + c0);
    const int64_t cache_at = (slot * p.Hkv + h) * D + c0;
    if (is_v) {
      if (slot >= 0) *reinterpret_cast<uint4*>(p.v_cache + cache_at) = raw;
      continue;
    }
    float x[8];
    unpack8(raw, x);
    const __nv_bfloat16* weight = is_q ? p.q_weight : p.k_weight;
    float inv = 1.f;
    if (weight != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(row_mask, ss, off);
      inv = rsqrtf(ss * (1.f / D) + p.eps);
      float w[8];
      unpack8(*reinterpret_cast<const uint4*>(weight + c0), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= inv * w[i];
    }
    if constexpr (INTERLEAVED) {
      if (turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[2 * i], b = x[2 * i + 1];
          x[2 * i] = a * cs[i] - b * sn[i];
          x[2 * i + 1] = b * cs[i] + a * sn[i];
        }
      }
    } else if (p.rot > 0) {
      const int from = row_lane0 + partner;
      uint4 other;
      other.x = __shfl_sync(row_mask, raw.x, from);
      other.y = __shfl_sync(row_mask, raw.y, from);
      other.z = __shfl_sync(row_mask, raw.z, from);
      other.w = __shfl_sync(row_mask, raw.w, from);
      if (turns) {
        float y[8];
        unpack8(other, y);
        if (weight != nullptr) {
          float w[8];
          unpack8(*reinterpret_cast<const uint4*>(weight + partner * 8), w);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] *= inv * w[i];
        }
        const float sign = c0 < half ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * cs[i] + sign * (y[i] * sn[i]);
      }
    }
    const uint4 out = pack8(x);
    if (is_q) {
      *reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + h * D + c0) = out;
    } else {
      if (p.k_out != nullptr) *reinterpret_cast<uint4*>(p.k_out + t * p.k_out_stride + h * D + c0) = out;
      if (slot >= 0) *reinterpret_cast<uint4*>(p.k_cache + cache_at) = out;
    }
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
  constexpr int groups = THREADS / (D / 8);
  const int rows = p.Hq + p.Hkv * (p.v_cache != nullptr ? 2 : 1);
  const int lanes = rows < groups ? rows : groups;
  const int tokens = groups / lanes;
  const int grid = (p.T + tokens - 1) / tokens;
  if (p.interleaved)
    qk_rope_kernel<D, true><<<grid, THREADS, 0, stream>>>(p, lanes);
  else
    qk_rope_kernel<D, false><<<grid, THREADS, 0, stream>>>(p, lanes);
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
