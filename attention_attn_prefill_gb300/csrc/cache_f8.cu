// Writing new keys and values into the 8-bit paged cache, and reading sequences back as bf16.
//
// Format and layout: cache_f8.cuh.  Both are bound by HBM: the write reads 2 bytes a value and writes 1, the
// read-back the other way round.
//
// Write: a page's scale belongs to all its tokens, so the tokens of a call that go to one page are one item: a run
// of neighbouring tokens with consecutive slots.  A warp takes the keys, or the values, of a run and head: its lanes
// hold the rows as the record has them, find the largest magnitude, and write the codes as 16-byte words.  Where the
// run does not begin the page, the rows before it stay; if the new rows need a larger scale, their codes are moved to
// it.  The keys' warp also keeps the smallest and largest key of the page in each channel, which block selection
// scores by; the reduction over tokens halves the channels a lane holds at each step, 7 exchanges for 16 channels.
// Read-back: a warp at a record.
//
// Measured (GB300, copy rate 6796 GB/s): the write of 32002 tokens, 8 heads, d = 128, and their read-back, 402 MB in
// all, 63.2 us in a captured graph, 6.4 TB/s.  Alone and from a cold L2 31 and 29 us: the write uses half of the
// issue slots, the read-back a third; both wait for memory.  64 tokens written and 64 sequences of up to 250 read
// back: 12.4 us (7.9 at the copy rate), two launches with their start and end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache_f8.cuh"
#include "sm103.cuh"
#include "step.h"

namespace attn {

__device__ uint32_t g_cache_f8_status;

namespace {

using f8::Record;

constexpr int WARPS = 4;
constexpr uint32_t FULL = 0xffffffffu;
constexpr uint32_t NOT_FINITE = 0x7f80;  // a bf16's magnitude bits from which on it is no finite number
// Up to this many values a call gives each token a warp of its own, which leaves at once if the token begins no run
constexpr int64_t TOKENWISE_VALUES = 1 << 20;
constexpr int64_t GATHER_CTAS = 152 * 64;  // CTAs of a read-back, about: a block table may be far wider than its sequences are long

__device__ __forceinline__ uint32_t lo_min(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hmin2_nan(reinterpret_cast<const __nv_bfloat162&>(a), reinterpret_cast<const __nv_bfloat162&>(b));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t hi_max(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hmax2_nan(reinterpret_cast<const __nv_bfloat162&>(a), reinterpret_cast<const __nv_bfloat162&>(b));
  return reinterpret_cast<const uint32_t&>(r);
}

// A pair of bf16 as codes: times `inv`, rounded
__device__ __forceinline__ uint32_t codes_of(uint32_t w, float inv) {
  return f8::codes2(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xffff0000u) * inv);
}
// Infinities of a pair become NaN
__device__ __forceinline__ uint32_t nan_for_inf(uint32_t w) {
  if ((w & 0x7fffu) >= NOT_FINITE) w |= 0x7fffu;
  if ((w >> 16 & 0x7fffu) >= NOT_FINITE) w |= 0x7fff0000u;
  return w;
}
// The magnitudes of a pair, 0 for what is not finite
__device__ __forceinline__ uint32_t finite_bits(uint32_t w) {
  w &= 0x7fff7fffu;
  if ((w & 0xffffu) >= NOT_FINITE) w &= 0xffff0000u;
  if (w >> 16 >= NOT_FINITE) w &= 0xffffu;
  return w;
}
// Four codes moved to another scale
__device__ __forceinline__ uint32_t moved(uint32_t w, float ratio) {
  const uint32_t a = f8::halves2(w), b = f8::halves2_upper(w);
  const float2 x = __half22float2(reinterpret_cast<const __half2&>(a)), y = __half22float2(reinterpret_cast<const __half2&>(b));
  return f8::codes2(x.x * ratio, x.y * ratio) | f8::codes2(y.x * ratio, y.y * ratio) << 16;
}

// The keys (or values) of one head of a run: `rows` tokens from `token` on, to rows r0 .. of a page, by a warp
template <int D, bool IS_V>
__device__ __forceinline__ void write_run(const AppendF8Params& p, int64_t page, int r0, int rows, int64_t token, int h,
                                          int lane) {
  using R = Record<D>;
  constexpr int CB = IS_V ? R::VB : 16;   // channels of a chunk: a token's that the lane holds next to each other
  constexpr int CPT = IS_V ? R::VH : R::KJ;  // chunks of a token
  constexpr int TOK = IS_V ? 4 : 2;          // tokens of a lane
  constexpr int W = CB / 2;                  // words of a chunk
  const int g = lane >> 2, t = lane & 3;
  uint8_t* rec = p.cache + (page * p.Hkv + h) * R::BYTES;
  float* scale_at = reinterpret_cast<float*>(rec + R::S_OFF) + (IS_V ? 1 : 0);
  const uint32_t was = r0 > 0 ? __float_as_uint(*scale_at) >> 23 : 0u;  // biased exponent of the page's scale
  const __nv_bfloat16* src = IS_V ? p.v + h * D : p.k + h * D;
  const int64_t stride = IS_V ? p.v_stride : p.k_stride;

  uint32_t raw[TOK][CPT][W];
  uint32_t most2 = 0;
  bool live[TOK];
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const int row = IS_V ? 8 * (i >> 1) + 2 * t + (i & 1) : 8 * i + g;
    live[i] = row >= r0 && row < r0 + rows;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int channel = IS_V ? 8 * CB * c + CB * g : 64 * c + 16 * t;
#pragma unroll
      for (int w = 0; w < W; w += 4) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (live[i]) x = __ldcs(reinterpret_cast<const uint4*>(src + (token + row - r0) * stride + channel + 2 * w));
        raw[i][c][w] = x.x; raw[i][c][w + 1] = x.y; raw[i][c][w + 2] = x.z; raw[i][c][w + 3] = x.w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TOK; ++i)
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
      for (int w = 0; w < W; ++w) most2 = __vmaxu2(most2, raw[i][c][w] & 0x7fff7fffu);
  uint32_t most = __reduce_max_sync(FULL, max(most2 & 0xffffu, most2 >> 16));

  if (!IS_V && p.bounds != nullptr) {
    // bounds of the page's keys: word g of a lane's 16 channels is the one it is left with
    uint32_t* out = reinterpret_cast<uint32_t*>(p.bounds + (page * p.Hkv + h) * 2 * D);
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      uint32_t lo[8], hi[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        lo[w] = live[0] ? raw[0][c][w] : 0x7f807f80u;  // infinities where there is no token
        hi[w] = live[0] ? raw[0][c][w] : 0xff80ff80u;
        if (live[1]) {
          lo[w] = lo_min(lo[w], raw[1][c][w]);
          hi[w] = hi_max(hi[w], raw[1][c][w]);
        }
      }
#pragma unroll
      for (int half = 4; half >= 1; half >>= 1) {
        const bool up = (g & half) != 0;
#pragma unroll
        for (int w = 0; w < half; ++w) {
          const uint32_t l = __shfl_xor_sync(FULL, up ? lo[w] : lo[w + half], 4 * half);
          const uint32_t x = __shfl_xor_sync(FULL, up ? hi[w] : hi[w + half], 4 * half);
          lo[w] = lo_min(up ? lo[w + half] : lo[w], l);
          hi[w] = hi_max(up ? hi[w + half] : hi[w], x);
        }
      }
      uint32_t* at = out + 32 * c + 8 * t + g;
      if (r0 > 0) {
        lo[0] = lo_min(lo[0], at[0]);
        hi[0] = hi_max(hi[0], at[D / 2]);
      }
      at[0] = lo[0];
      at[D / 2] = hi[0];
    }
  }

  if (most >= NOT_FINITE) {  // rare: what is not finite takes no part in the scale
    most2 = 0;
#pragma unroll
    for (int i = 0; i < TOK; ++i)
#pragma unroll
      for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int w = 0; w < W; ++w) {
          most2 = __vmaxu2(most2, finite_bits(raw[i][c][w]));
          raw[i][c][w] = nan_for_inf(raw[i][c][w]);
        }
    most = __reduce_max_sync(FULL, max(most2 & 0xffffu, most2 >> 16));
  }
  const uint32_t need = f8::scale_exponent(most);
  const uint32_t now = max(need, was);
  const float inv = f8::pow2(254u - now);
  uint8_t* codes = rec + (IS_V ? R::V_OFF : R::K_OFF) + lane * CB;
  if (r0 > 0 && now != was) {
    // the rows before the run, at the larger scale
    const float ratio = was == 0 ? 0.f : f8::pow2(was) * inv;
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      const int row = IS_V ? 8 * (i >> 1) + 2 * t + (i & 1) : 8 * i + g;
      if (row >= r0) continue;
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        uint32_t* at = reinterpret_cast<uint32_t*>(codes + (i * CPT + c) * 32 * CB);
#pragma unroll
        for (int w = 0; w < CB / 4; ++w) at[w] = moved(at[w], ratio);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    if (!live[i]) continue;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      uint32_t out[CB / 4];
#pragma unroll
      for (int w = 0; w < CB / 4; ++w)
        out[w] = codes_of(raw[i][c][2 * w], inv) | codes_of(raw[i][c][2 * w + 1], inv) << 16;
      uint8_t* at = codes + (i * CPT + c) * 32 * CB;
      if constexpr (CB == 16) *reinterpret_cast<uint4*>(at) = make_uint4(out[0], out[1], out[2], out[3]);
      else *reinterpret_cast<uint2*>(at) = make_uint2(out[0], out[1]);
    }
  }
  if (lane == 0) *scale_at = f8::pow2(now);
}

// A warp takes the runs that begin among `window` tokens (1 or 16), for the keys or values of one head
template <int D>
__global__ void __launch_bounds__(WARPS * 32) append_f8_kernel(const AppendF8Params p, int window) {
  const int lane = threadIdx.x & 31;
  const int hv = blockIdx.y * WARPS + (threadIdx.x >> 5);
  if (hv >= 2 * p.Hkv) return;
  const int h = hv >> 1;
  const int base = blockIdx.x * window;
  auto slot_at = [&](int t) { return t >= 0 && t < p.T ? p.slots[t] : -1; };
  const int slot = slot_at(base + lane);
  int before = __shfl_up_sync(FULL, slot, 1);
  if (lane == 0) before = slot_at(base - 1);
  // a token that goes behind its neighbour, into the same page
  const bool follows = slot > 0 && slot % 16 != 0 && before == slot - 1;
  const unsigned on = __ballot_sync(FULL, follows);
  unsigned starts = __ballot_sync(FULL, slot >= 0 && !follows && lane < window);
  for (; starts != 0; starts &= starts - 1) {
    const int k = __ffs(starts) - 1;
    const int s = __shfl_sync(FULL, slot, k);
    const int rows = __ffs(~(on >> 1 >> k));  // it and those that follow: at most 16, a page's
    if (s >= p.num_slots) {
      if (hv == 0 && lane == 0) set_error(&g_cache_f8_status, kDevBadSlot);
      continue;
    }
    if (hv & 1) write_run<D, true>(p, s / 16, s % 16, rows, base + k, h, lane);
    else write_run<D, false>(p, s / 16, s % 16, rows, base + k, h, lane);
  }
}

// Four codes times the scale, as two pairs of bf16: exact
__device__ __forceinline__ uint2 values(uint32_t w, float scale) {
  const uint32_t a = f8::halves2(w), b = f8::halves2_upper(w);
  const float2 x = __half22float2(reinterpret_cast<const __half2&>(a)), y = __half22float2(reinterpret_cast<const __half2&>(b));
  return make_uint2(pack_bf16x2(x.x * scale, x.y * scale), pack_bf16x2(y.x * scale, y.y * scale));
}

// The first `valid` tokens of a record's keys or values to rows row_stride apart, by a warp.  A lane takes 8 bytes at a
// time: neighbouring lanes then write neighbouring 16 bytes, whole sectors at once.
template <int D, bool IS_V>
__device__ __forceinline__ void gather_half(const uint8_t* rec, float scale, __nv_bfloat16* out, int64_t row_stride,
                                            int valid, int lane) {
  using R = Record<D>;
  constexpr int LOADS = D / 16;
  const uint8_t* codes = rec + (IS_V ? R::V_OFF : R::K_OFF) + lane * 8;
  uint2 raw[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) raw[i] = __ldcs(reinterpret_cast<const uint2*>(codes + i * 256));
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    constexpr int ROW = IS_V ? 32 * R::VB : 512;  // bytes of a row of the record
    const int row = i * 256 / ROW, at = i * 256 % ROW + lane * 8;
    int token, channel;
    if (IS_V) {
      const int k = row / R::VH, g = at / (4 * R::VB), t = at / R::VB % 4;
      token = 8 * (k >> 1) + 2 * t + (k & 1);
      channel = 8 * R::VB * (row % R::VH) + R::VB * g + at % R::VB;
    } else {
      token = 8 * (row / R::KJ) + at / 64;
      channel = 64 * (row % R::KJ) + at % 64;
    }
    if (token >= valid) continue;
    const uint2 a = values(raw[i].x, scale), b = values(raw[i].y, scale);
    *reinterpret_cast<uint4*>(out + token * row_stride + channel) = make_uint4(a.x, a.y, b.x, b.y);
  }
}

// A warp takes every gridDim.x * WARPS-th record of sequence blockIdx.y
template <int D>
__global__ void __launch_bounds__(WARPS * 32) gather_f8_kernel(const GatherF8Params p) {
  const int n = blockIdx.y, lane = threadIdx.x & 31;
  int len = p.seq_lens[n];
  if (len < 0 || len > p.max_blocks * f8::PAGE) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_error(&g_cache_f8_status, kDevBadSeqlens);
    len = len < 0 ? 0 : p.max_blocks * f8::PAGE;
  }
  const int64_t row_stride = static_cast<int64_t>(p.Hkv) * D;
  const unsigned items = static_cast<unsigned>((len + f8::PAGE - 1) / f8::PAGE) * p.Hkv;
  for (unsigned item = blockIdx.x * WARPS + (threadIdx.x >> 5); item < items; item += gridDim.x * WARPS) {
    const int page = item / p.Hkv, h = item - page * p.Hkv;
    const int64_t at = static_cast<int64_t>(n) * p.max_blocks + page;
    if (p.out_table != nullptr && h == 0 && lane == 0) p.out_table[at] = static_cast<int32_t>(at);
    int pid = p.block_table[at];
    if (pid < 0 || pid >= p.num_blocks) {
      if (lane == 0) set_error(&g_cache_f8_status, kDevBadPage);
      pid = 0;
    }
    const uint8_t* rec = p.cache + (static_cast<int64_t>(pid) * p.Hkv + h) * Record<D>::BYTES;
    const float2 scales = *reinterpret_cast<const float2*>(rec + Record<D>::S_OFF);
    const int64_t out0 = at * f8::PAGE * row_stride + static_cast<int64_t>(h) * D;
    gather_half<D, false>(rec, scales.x, p.k_out + out0, row_stride, len - page * f8::PAGE, lane);
    gather_half<D, true>(rec, scales.y, p.v_out + out0, row_stride, len - page * f8::PAGE, lane);
  }
}

template <int D>
cudaError_t append(const AppendF8Params& p, cudaStream_t stream) {
  const int window = static_cast<int64_t>(p.T) * p.Hkv * D <= TOKENWISE_VALUES ? 1 : 16;
  const dim3 grid((p.T + window - 1) / window, (2 * p.Hkv + WARPS - 1) / WARPS);
  append_f8_kernel<D><<<grid, WARPS * 32, 0, stream>>>(p, window);
  return cudaGetLastError();
}

template <int D>
cudaError_t gather(const GatherF8Params& p, cudaStream_t stream) {
  const int64_t items = (static_cast<int64_t>(p.max_blocks) * p.Hkv + WARPS - 1) / WARPS;
  const int64_t most = (GATHER_CTAS + p.N - 1) / p.N;
  const unsigned grid = static_cast<unsigned>(items < most ? items : most);
  gather_f8_kernel<D><<<dim3(grid, p.N), WARPS * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t append_f8_launch(const AppendF8Params& p, cudaStream_t stream) {
  if (p.d == 64) return append<64>(p, stream);
  if (p.d == 128) return append<128>(p, stream);
  if (p.d == 256) return append<256>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t gather_f8_launch(const GatherF8Params& p, cudaStream_t stream) {
  if (p.d == 64) return gather<64>(p, stream);
  if (p.d == 128) return gather<128>(p, stream);
  if (p.d == 256) return gather<256>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t cache_f8_status(uint32_t* out, bool clear) { return read_status(g_cache_f8_status, out, clear); }

}  // namespace attn
