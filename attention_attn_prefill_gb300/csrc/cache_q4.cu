// Writing new keys and values into the 4-bit paged cache, and reading sequences back as bf16.
//
// Format and layout: cache_q4.cuh.  Both are bound by HBM: the write reads 2 bytes a value and writes
// 17 / 32, the read-back the other way round.
//
// Write: a warp takes 16 tokens of a KV head, whose rows are all in flight before the first is used.  V
// codes of a page are spread over its record token by token, a byte each; where 16 tokens in a row fill
// a page (any prompt), they are put together through shared memory and written as 16-byte words, else
// byte by byte.  Quantising costs more than the memory allows for unless it is done in pairs: the range
// by packed bf16 minima and maxima, the division as a product with the reciprocal and one correction
// by the exact remainder (P. Markstein, IBM J. Res. Dev. 34, 1990) on pairs of floats, the codes as 16-bit pairs.
// 32002 tokens of 8 heads, d = 128, take 34 us, 24 at the rate of a copy; issue slots bound it (72% used).
// Read-back: a warp at a record; V words are exchanged between the four lanes that hold 8 neighbouring
// channels, so that each lane writes 16 bytes.  5.5 to 6.6 TB/s, HBM's rate.
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

constexpr int WARPS = 4;
// Up to this many values a call takes a row at a time.  Measured at 8 heads, d = 128, by rows and by pages:
// 512 tokens that fill pages 2.8 and 3.5 us, 1024 tokens 3.6 and 3.6, 2048 tokens 5.4 and 4.6, 8192 tokens
// 16.1 and 11.7; tokens on a page each 3.1 and 4.8, 3.7 and 5.3, 5.4 and 6.8, 19.1 and 18.8.
constexpr int64_t ROWWISE_VALUES = 1 << 20;
// CTAs of a read-back, about: a block table may be far wider than its sequences are long.  One warp for each
// of its records, 64 sequences of 1000 tokens, 8 heads, d = 128, take 138 us with 2048 pages a row and 53 us
// with 63; with this limit 54 us both.  64 sequences of 8000: 405 us, without a limit 396.
constexpr int64_t GATHER_CTAS = 152 * 64;

constexpr float MAGIC = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, which the lower bits then hold

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Codes of eight channels where the scale is 0, too small or too large for its reciprocal, or not finite.
// The parameter word is the result's upper half.
__device__ __noinline__ uint64_t quantise_odd(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, float hi, float lo) {
  if (!(hi - lo < INFINITY)) return static_cast<uint64_t>(q4::PARAM_NAN) << 32;
  const float s = q4::make_scale(hi, lo);
  const float zero = s > 0.f ? rintf(__fdiv_rn(-lo, s)) : 0.f;
  uint32_t codes = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 4 ? (i < 2 ? w0 : w1) : (i < 6 ? w2 : w3);
    const float x = __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
    const float c = s > 0.f ? rintf(__fdiv_rn(x, s)) + zero : 0.f;
    codes |= static_cast<uint32_t>(fminf(c, 15.f)) << (4 * i);
  }
  return static_cast<uint64_t>(__float_as_uint(s) >> 16 | static_cast<uint32_t>(zero)) << 32 | codes;
}

// Eight channels of a row; the 8 threads of a group (neighbours, aligned to 8) hold its 64 channels.
// Returns the codes as nibbles, channel j in nibble j, and the group's parameter word.
__device__ __forceinline__ uint32_t quantise(const uint4& raw, uint32_t& param) {
  const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&raw);
  // a NaN or infinity passes through
  __nv_bfloat162 hi2 = __hmax2_nan(__hmax2_nan(w[0], w[1]), __hmax2_nan(w[2], w[3]));
  __nv_bfloat162 lo2 = __hmin2_nan(__hmin2_nan(w[0], w[1]), __hmin2_nan(w[2], w[3]));
  // the maximum and minus the minimum share a word for the rest of the way
  const uint32_t h = reinterpret_cast<const uint32_t&>(hi2), l = reinterpret_cast<const uint32_t&>(lo2) ^ 0x80008000u;
  const uint32_t lower = __byte_perm(h, l, 0x5410), upper = __byte_perm(h, l, 0x7632);
  __nv_bfloat162 ext = __hmax2_nan(reinterpret_cast<const __nv_bfloat162&>(lower),
                                   reinterpret_cast<const __nv_bfloat162&>(upper));
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) ext = __hmax2_nan(ext, __shfl_xor_sync(0xffffffffu, ext, off));
  const float2 ef = __bfloat1622float2(ext);
  const float hi = max_nan(ef.x, 0.f), lo = fminf(-ef.y, 0.f);
  const float s = q4::make_scale(hi, lo);
  constexpr uint32_t LEAST = 0x1e3ce508u, MOST = 0x7e967699u;  // 1e-20, 1e38
  if (__float_as_uint(s) - LEAST >= MOST - LEAST) {  // NaN too: its bits are past all of these, with either sign
    const uint64_t odd = quantise_odd(raw.x, raw.y, raw.z, raw.w, hi, lo);
    param = static_cast<uint32_t>(odd >> 32);
    return static_cast<uint32_t>(odd);
  }
  // x / s by Markstein's correction: q = x inv is off by a few ulp, x - q s is exact as a fused product, and adding
  // its quotient leaves an error of the last rounding alone.  That is all rint asks for: a tie, j + 1/2, is a float,
  // so q lands on it; any other x / s keeps 1 / 960 from every tie, x having 8 significant bits and s 4.
  const float inv = rcp_approx(s);
  const float zq = -lo * inv;
  const float zt = fmaf(fmaf(-zq, s, -lo), inv, zq) + MAGIC;
  param = __float_as_uint(s) >> 16 | (__float_as_uint(zt) & 15u);
  // codes >= 0 without a clamp: x >= lo, and rint is odd.  Integers in 16-bit pairs, channels j and j + 4.
  const uint64_t inv2 = f2_pack(inv, inv), ns2 = f2_pack(-s, -s), magic2 = f2_pack(MAGIC, MAGIC);
  const uint64_t zero2 = f2_pack(zt - MAGIC, zt - MAGIC);
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t n[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = f2_pack(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    uint64_t q = f2_mul(x, inv2);
    q = f2_fma(f2_fma(q, ns2, x), inv2, q);
    float a, b;
    f2_unpack(f2_add(f2_add(q, magic2), zero2), a, b);
    n[2 * i] = __float_as_uint(a);
    n[2 * i + 1] = __float_as_uint(b);
  }
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    codes += __vminu2(__byte_perm(n[i], n[i + 4], 0x5410), 0x000f000fu) << (4 * i);
  return codes;
}

// One row's codes and parameters into the record of its page and head; V byte by byte
template <int D, bool IS_V>
__device__ __forceinline__ void store_row(uint8_t* rec, int row, int sub, uint32_t codes, uint32_t param) {
  using R = Record<D>;
  if (sub % 8 == 0)
    reinterpret_cast<uint16_t*>(rec + (IS_V ? R::VP_OFF : R::KP_OFF))[row * R::NG + sub / 8] =
        static_cast<uint16_t>(param);
  if constexpr (IS_V) {
#pragma unroll
    for (int b = 0; b < 4; ++b) rec[R::V_OFF + R::v_byte(row, sub * 4 + b)] = static_cast<uint8_t>(codes >> (8 * b));
  } else {
    reinterpret_cast<uint32_t*>(rec + R::K_OFF + row * (D / 2))[R::k_word(sub)] = q4::rotl3(codes);
  }
}

// Few tokens (a decode step): D / 8 threads a row of K or V of a token and head
template <int D>
__global__ void __launch_bounds__(128) append_rows_q4_kernel(const AppendQ4Params p) {
  constexpr int LPR = D / 8;
  const unsigned row = (blockIdx.x * 128 + threadIdx.x) / LPR;
  const int sub = threadIdx.x % LPR;
  const unsigned t = row / (2 * p.Hkv);
  const int rest = row - t * (2 * p.Hkv), h = rest >> 1;
  const bool is_v = rest & 1;
  const int slot = t < static_cast<unsigned>(p.T) ? p.slots[t] : -1;
  const bool live = slot >= 0 && slot < p.num_slots;
  if (slot >= p.num_slots && rest == 0 && sub == 0) set_error(&g_cache_q4_status, kDevBadSlot);
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (live)
    raw = *reinterpret_cast<const uint4*>((is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride) + h * D + sub * 8);
  uint32_t param;
  const uint32_t codes = quantise(raw, param);
  if (!live) return;
  uint8_t* rec = p.cache + (static_cast<int64_t>(slot / 16) * p.Hkv + h) * Record<D>::BYTES;
  if (is_v) store_row<D, true>(rec, slot % 16, sub, codes, param);
  else store_row<D, false>(rec, slot % 16, sub, codes, param);
}

// K or V of a head, for 16 tokens from 16 blockIdx.x on.  A run of 16 tokens that fills a page belongs to
// the warp of its first token, whatever tokens it reaches into; the others of a warp's tokens are
// written row by row, their loads in flight together too: the last, partly filled page of a prompt is what a
// call of few pages waits for (2049 tokens of 8 heads, d = 128: 4.7 us; 8.1 us with two rows in flight).  K
// and V in one warp take 46 us instead of 40 us for 32002 tokens, for want of registers (this form: 34 us).
template <int D>
__global__ void __launch_bounds__(WARPS * 32) append_q4_kernel(const AppendQ4Params p) {
  using R = Record<D>;
  constexpr int LPR = D / 8;          // lanes a row
  constexpr int RPI = 32 / LPR;       // rows a load
  constexpr int IT = 16 / RPI;        // loads of 16 rows
  constexpr int ROW_WORDS = LPR + 1;  // a token's code words in shared memory
  __shared__ uint32_t s_codes[WARPS][16 * ROW_WORDS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (blockIdx.y * WARPS + warp) >> 1;
  const bool is_v = warp & 1;
  if (h >= p.Hkv) return;
  const int chunk = blockIdx.x * 16;
  const int sub = lane % LPR, k0 = lane / LPR;

  // bit k of the masks: token chunk - 16 + k starts a page / has the slot behind its neighbour's
  uint64_t aligned = 0, follows = 0;
  int my_slot = -1;  // of token chunk + lane - 16
  auto slot_at = [&](int t) { return t >= 0 && t < p.T ? p.slots[t] : -1; };
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    const int t = chunk - 16 + part * 32 + lane;
    const int slot = slot_at(t), before = slot_at(t - 1);
    const uint64_t starts_page = __ballot_sync(0xffffffffu, slot >= 0 && slot % 16 == 0 && slot < p.num_slots);
    const uint64_t continues = __ballot_sync(0xffffffffu, slot > 0 && slot % 16 != 0 && before == slot - 1);
    aligned |= starts_page << (32 * part);
    follows |= continues << (32 * part);
    if (part == 0) my_slot = slot;
  }
  auto full = [&](int k) { return (aligned >> k & 1) != 0 && ((follows >> (k + 1)) & 0x7fff) == 0x7fff; };
  const int in_page = my_slot >= 0 ? my_slot % 16 : 0;
  const bool mine = lane >= 16 && my_slot >= 0;
  if (mine && my_slot >= p.num_slots && h == 0 && !is_v) set_error(&g_cache_q4_status, kDevBadSlot);
  // lane - in_page is the run's first token in the window, from which on the masks hold 16 tokens
  const bool in_run = mine && lane - in_page >= 0 && full(lane - in_page);
  const unsigned starts = __ballot_sync(0xffffffffu, in_run && in_page == 0);
  const unsigned singles = __ballot_sync(0xffffffffu, mine && !in_run && my_slot < p.num_slots) >> 16;

  const __nv_bfloat16* base = (is_v ? p.v : p.k) + h * D + sub * 8;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  if (starts != 0) {
    const int from = __ffs(starts) - 1;  // runs do not overlap: at most one starts among 16 tokens
    const __nv_bfloat16* src = base + (chunk - 16 + from + k0) * stride;
    const int64_t page = __shfl_sync(0xffffffffu, my_slot, from) / 16;
    uint8_t* rec = p.cache + (page * p.Hkv + h) * R::BYTES;
    uint4 raw[IT];
#pragma unroll
    for (int it = 0; it < IT; ++it) raw[it] = __ldcs(reinterpret_cast<const uint4*>(src + it * (RPI * stride)));
    uint16_t* params = reinterpret_cast<uint16_t*>(rec + (is_v ? R::VP_OFF : R::KP_OFF)) + k0 * R::NG + sub / 8;
    uint32_t* k_codes = reinterpret_cast<uint32_t*>(rec + R::K_OFF + k0 * (D / 2)) + R::k_word(sub);
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      uint32_t param;
      const uint32_t codes = quantise(raw[it], param);
      if (sub % 8 == 0) params[it * RPI * R::NG] = static_cast<uint16_t>(param);
      if (is_v) s_codes[warp][(it * RPI + k0) * ROW_WORDS + sub] = codes;
      else k_codes[it * RPI * (D / 8)] = q4::rotl3(codes);
    }
    if (is_v) {
      // the record's word (i, lane = 4 g + t, k) is byte g % 4 of word 2 (4 i + k) + g / 4 of four tokens
      __syncwarp();
      const int g = lane >> 2, t = lane & 3;
      const uint32_t pick = (g & 3) | (4 + (g & 3)) << 4;  // that byte of two words
      const uint32_t* at = s_codes[warp] + 2 * t * ROW_WORDS + (g >> 2);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint32_t out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t* w = at + 2 * (4 * i + k);
          const uint32_t even = __byte_perm(w[0], w[8 * ROW_WORDS], pick);
          const uint32_t odd = __byte_perm(w[ROW_WORDS], w[9 * ROW_WORDS], pick);
          out[k] = __byte_perm(even, odd, 0x5410);
        }
        *reinterpret_cast<uint4*>(rec + R::V_OFF + (i * 32 + lane) * 16) = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
  }
  if (singles != 0) {
    uint4 raw[IT];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int k = it * RPI + k0;
      raw[it] = make_uint4(0, 0, 0, 0);
      if (singles >> k & 1) raw[it] = __ldcs(reinterpret_cast<const uint4*>(base + (chunk + k) * stride));
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if ((singles >> (it * RPI) & ((1u << RPI) - 1)) == 0) continue;
      const int k = it * RPI + k0;
      const int slot = __shfl_sync(0xffffffffu, my_slot, 16 + k);
      const bool live = singles >> k & 1;
      uint32_t param;
      const uint32_t codes = quantise(raw[it], param);
      if (live) {
        uint8_t* rec = p.cache + (static_cast<int64_t>(slot / 16) * p.Hkv + h) * R::BYTES;
        if (is_v) store_row<D, true>(rec, slot % 16, sub, codes, param);
        else store_row<D, false>(rec, slot % 16, sub, codes, param);
      }
      __syncwarp();
    }
  }
}

// 8 channels from their codes (nibble j: channel j)
__device__ __forceinline__ uint4 values(uint32_t codes, uint32_t param) {
  // 16 + c of two neighbouring channels: the byte that holds both, times 2^15 + 2^3, puts their nibbles
  // on the two halves' upper mantissa bits; less 16 + z, times s: every step exact
  const uint32_t z = (param & 15u) << 3 | 0x4180u, s = param & 0xfff0u;
  const uint32_t z2 = z | z << 16, s2 = s | s << 16;
  uint32_t out[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t c = (__byte_perm(codes, 0, 0x4440 | b) * 0x8008u & 0x00780078u) | 0x41804180u;
    const __nv_bfloat162 d =
        __hsub2(reinterpret_cast<const __nv_bfloat162&>(c), reinterpret_cast<const __nv_bfloat162&>(z2));
    const __nv_bfloat162 v = __hmul2(d, reinterpret_cast<const __nv_bfloat162&>(s2));
    out[b] = reinterpret_cast<const uint32_t&>(v);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The first `valid` tokens of a record to page `at` of the output, by a warp
template <int D>
__device__ __forceinline__ void gather_record(const GatherQ4Params& p, const uint8_t* rec, int64_t at, int h, int valid,
                                              int lane) {
  using R = Record<D>;
  constexpr int WPR = D / 8;     // code words a K row
  constexpr int RPI = 32 / WPR;  // K rows a load
  constexpr int NG = R::NG;
  const int64_t row_stride = static_cast<int64_t>(p.Hkv) * D;
  const int64_t out0 = at * q4::PAGE * row_stride + static_cast<int64_t>(h) * D;

  // every load of the record before the first use
  uint32_t kw[16 / RPI], kp[16 / RPI];
  uint4 vw[D / 64];
  const int g = lane >> 2, t = lane & 3;
  // word w of a row: channels 8 c .. 8 c + 7
  const int w = lane % WPR;
  const int c =
      (w / (8 * R::PAIR) * R::PAIR + w % (2 * R::PAIR) / 2) * 8 + w % (8 * R::PAIR) / (2 * R::PAIR) * 2 + w % 2;
#pragma unroll
  for (int i = 0; i < 16 / RPI; ++i) {
    const int token = i * RPI + lane / WPR;
    kw[i] = __ldcs(reinterpret_cast<const uint32_t*>(rec + R::K_OFF) + i * 32 + lane);
    kp[i] = reinterpret_cast<const uint16_t*>(rec + R::KP_OFF)[token * NG + c / 8];
  }
#pragma unroll
  for (int i = 0; i < D / 64; ++i) vw[i] = __ldcs(reinterpret_cast<const uint4*>(rec + R::V_OFF) + i * 32 + lane);
  uint32_t vp[4][D / 64];  // of the four tokens in this lane's V words
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int e = 0; e < NG; ++e)
      vp[b][e] = reinterpret_cast<const uint16_t*>(rec + R::VP_OFF)[(2 * t + b / 2 + 8 * (b % 2)) * NG + e];

#pragma unroll
  for (int i = 0; i < 16 / RPI; ++i) {
    const int token = i * RPI + lane / WPR;
    if (token < valid)
      *reinterpret_cast<uint4*>(p.k_out + out0 + token * row_stride + c * 8) =
          values(__funnelshift_r(kw[i], kw[i], 3), kp[i]);
  }
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    // this lane holds channels 2 g, 2 g + 1 of blocks 0 .. 3; after two exchanges with the lanes 4 g apart
    // it holds channels 8 (g / 4) .. + 7 of block g % 4, a word (byte: token) for each two channels
    uint32_t x[4] = {vw[i].x, vw[i].y, vw[i].z, vw[i].w};
    const bool up = g & 1, up2 = g & 2;
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x[k] : x[k + 1], 4);
      if (up) x[k] = got; else x[k + 1] = got;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up2 ? x[k] : x[k + 2], 8);
      if (up2) x[k] = got; else x[k + 2] = got;
    }
    const int channel = 64 * i + 16 * (g & 3) + 8 * (g >> 2);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int token = 2 * t + b / 2 + 8 * (b % 2);
      const uint32_t pick = b | (4 + b) << 4;
      const uint32_t codes = __byte_perm(__byte_perm(x[0], x[1], pick), __byte_perm(x[2], x[3], pick), 0x5410);
      if (token < valid)
        *reinterpret_cast<uint4*>(p.v_out + out0 + token * row_stride + channel) = values(codes, vp[b][i]);
    }
  }
}

// A warp takes every gridDim.x * WARPS-th record of sequence blockIdx.y
template <int D>
__global__ void __launch_bounds__(WARPS * 32) gather_q4_kernel(const GatherQ4Params p) {
  const int n = blockIdx.y, lane = threadIdx.x & 31;
  int len = p.seq_lens[n];
  if (len < 0 || len > p.max_blocks * q4::PAGE) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_error(&g_cache_q4_status, kDevBadSeqlens);
    len = len < 0 ? 0 : p.max_blocks * q4::PAGE;
  }
  const unsigned items = static_cast<unsigned>((len + q4::PAGE - 1) / q4::PAGE) * p.Hkv;
  for (unsigned item = blockIdx.x * WARPS + (threadIdx.x >> 5); item < items; item += gridDim.x * WARPS) {
    const int page = item / p.Hkv, h = item - page * p.Hkv;
    const int64_t at = static_cast<int64_t>(n) * p.max_blocks + page;
    if (p.out_table != nullptr && h == 0 && lane == 0) p.out_table[at] = static_cast<int32_t>(at);
    int pid = p.block_table[at];
    if (pid < 0 || pid >= p.num_blocks) {
      if (lane == 0) set_error(&g_cache_q4_status, kDevBadPage);
      pid = 0;
    }
    const uint8_t* rec = p.cache + (static_cast<int64_t>(pid) * p.Hkv + h) * Record<D>::BYTES;
    gather_record<D>(p, rec, at, h, len - page * q4::PAGE, lane);
  }
}

template <int D>
cudaError_t append(const AppendQ4Params& p, cudaStream_t stream) {
  if (static_cast<int64_t>(p.T) * p.Hkv * D <= ROWWISE_VALUES) {
    const int64_t threads = static_cast<int64_t>(p.T) * p.Hkv * 2 * (D / 8);
    append_rows_q4_kernel<D><<<static_cast<unsigned>((threads + 127) / 128), 128, 0, stream>>>(p);
  } else {
    append_q4_kernel<D><<<dim3((p.T + 15) / 16, (2 * p.Hkv + WARPS - 1) / WARPS), WARPS * 32, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t gather(const GatherQ4Params& p, cudaStream_t stream) {
  const int64_t items = (static_cast<int64_t>(p.max_blocks) * p.Hkv + WARPS - 1) / WARPS;
  const int64_t most = (GATHER_CTAS + p.N - 1) / p.N;
  const unsigned grid = static_cast<unsigned>(items < most ? items : most);
  gather_q4_kernel<D><<<dim3(grid, p.N), WARPS * 32, 0, stream>>>(p);
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
