// Writing new keys and values into the 4-bit paged cache, and reading sequences back as bf16.
//
// Format and layout: cache_q4.cuh.  Both are bound by HBM: the write reads 2 bytes a value and writes
// 17 / 32, the read-back the other way round.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache_q4.cuh"
#include "sm103.cuh"
#include "step.h"

namespace attn {

__device__ uint32_t g_cache_q4_status;

namespace {

using q4::Record;

// Eight channels of a row; the 8 threads of a group (neighbours, aligned to 8) hold its 64 channels.
// Returns the codes as nibbles, channel j in nibble j, and the group's parameter word.
__device__ __forceinline__ uint32_t quantise(const uint4& raw, unsigned mask, uint32_t& param) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
  float hi = 0.f, lo = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    hi = fmaxf(hi, fmaxf(x[2 * i], x[2 * i + 1]));
    lo = fminf(lo, fminf(x[2 * i], x[2 * i + 1]));
    finite = finite && (w[i] & 0x7f80u) != 0x7f80u && (w[i] & 0x7f800000u) != 0x7f800000u;
  }
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, off));
    lo = fminf(lo, __shfl_xor_sync(mask, lo, off));
  }
  finite = !(__ballot_sync(mask, !finite) & (0xffu << (threadIdx.x & 31 & ~7)));
  float scale, zero;
  param = q4::make_param(hi, lo, scale, zero);
  if (!finite || !(scale < INFINITY)) {
    param = q4::PARAM_NAN;
    return 0;
  }
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = scale > 0.f ? rintf(__fdiv_rn(x[i], scale)) + zero : 0.f;
    codes |= static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f)) << (4 * i);
  }
  return codes;
}

// D / 8 threads a (token, KV head, K or V) row
template <int D>
__global__ void __launch_bounds__(256) append_q4_kernel(const AppendQ4Params p) {
  using R = Record<D>;
  constexpr int LPR = D / 8;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / LPR;
  const int i = threadIdx.x % LPR;
  const int h = static_cast<int>(row / 2 % p.Hkv);
  const int64_t t = row / 2 / p.Hkv;
  const bool is_v = row & 1;
  if (t >= p.T) return;  // whole rows fall out together
  const unsigned mask =
      LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << (threadIdx.x & 31 & ~(LPR - 1));
  const int64_t slot = p.slots[t];
  if (slot >= p.num_slots && i == 0 && h == 0) set_error(&g_cache_q4_status, kDevBadSlot);
  if (slot < 0 || slot >= p.num_slots) return;
  const __nv_bfloat16* src = is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride;
  uint32_t param;
  const uint32_t codes = quantise(*reinterpret_cast<const uint4*>(src + h * D + i * 8), mask, param);
  const int token = static_cast<int>(slot % q4::PAGE);
  uint8_t* rec = p.cache + (slot / q4::PAGE * p.Hkv + h) * R::BYTES;
  if (is_v) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
      rec[R::V_OFF + R::v_byte(token, i * 4 + b)] = static_cast<uint8_t>(codes >> (8 * b));
  } else {
    reinterpret_cast<uint32_t*>(rec + R::K_OFF + token * (D / 2))[R::k_word(i)] = q4::rotl3(codes);
  }
  if (i % 8 == 0)
    reinterpret_cast<uint16_t*>(rec + (is_v ? R::VP_OFF : R::KP_OFF))[token * R::NG + i / 8] =
        static_cast<uint16_t>(param);
}

// One CTA a (sequence, page): 8 channels of a token and head at a time
template <int D>
__global__ void __launch_bounds__(256) gather_q4_kernel(const GatherQ4Params p) {
  using R = Record<D>;
  const int n = blockIdx.y, page = blockIdx.x;
  int len = p.seq_lens[n];
  if (len < 0 || len > p.max_blocks * q4::PAGE) {
    if (threadIdx.x == 0 && page == 0) set_error(&g_cache_q4_status, kDevBadSeqlens);
    len = len < 0 ? 0 : p.max_blocks * q4::PAGE;
  }
  const int64_t at = static_cast<int64_t>(n) * p.max_blocks + page;
  if (p.out_table != nullptr && threadIdx.x == 0) p.out_table[at] = static_cast<int32_t>(at);
  const int valid = len - page * q4::PAGE < q4::PAGE ? len - page * q4::PAGE : q4::PAGE;
  if (valid <= 0) return;
  int pid = p.block_table[at];
  if (pid < 0 || pid >= p.num_blocks) {
    if (threadIdx.x == 0) set_error(&g_cache_q4_status, kDevBadPage);
    pid = 0;
  }
  for (int w = threadIdx.x; w < p.Hkv * valid * (D / 8); w += 256) {
    const int i = w % (D / 8), h = w / (D / 8) % p.Hkv, token = w / (D / 8) / p.Hkv;
    const uint8_t* rec = p.cache + (static_cast<int64_t>(pid) * p.Hkv + h) * R::BYTES;
    const int64_t out = ((at * q4::PAGE + token) * p.Hkv + h) * D + i * 8;
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
      uint32_t codes = 0;
      if (is_v) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          codes |= static_cast<uint32_t>(rec[R::V_OFF + R::v_byte(token, i * 4 + b)]) << (8 * b);
      } else {
        codes = reinterpret_cast<const uint32_t*>(rec + R::K_OFF + token * (D / 2))[R::k_word(i)];
        codes = __funnelshift_r(codes, codes, 3);
      }
      const uint32_t param =
          reinterpret_cast<const uint16_t*>(rec + (is_v ? R::VP_OFF : R::KP_OFF))[token * R::NG + i / 8];
      const float scale = __uint_as_float((param & 0xfff0u) << 16);
      const int zero = param & 15;
      float x[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) x[b] = scale * static_cast<float>(static_cast<int>(codes >> (4 * b) & 15) - zero);
      *reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + out) =
          make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                     pack_bf16x2(x[6], x[7]));
    }
  }
}

template <int D>
cudaError_t append(const AppendQ4Params& p, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(p.T) * p.Hkv * 2 * (D / 8);
  append_q4_kernel<D><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t gather(const GatherQ4Params& p, cudaStream_t stream) {
  gather_q4_kernel<D><<<dim3(p.max_blocks, p.N), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t append_q4_launch(const AppendQ4Params& p, cudaStream_t stream) {
  if (p.d == 64) return append<64>(p, stream);
  if (p.d == 128) return append<128>(p, stream);
  if (p.d == 256) return append<256>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t gather_q4_launch(const GatherQ4Params& p, cudaStream_t stream) {
  if (p.d == 64) return gather<64>(p, stream);
  if (p.d == 128) return gather<128>(p, stream);
  if (p.d == 256) return gather<256>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t cache_q4_status(uint32_t* out, bool clear) { return read_status(g_cache_q4_status, out, clear); }

}  // namespace attn
