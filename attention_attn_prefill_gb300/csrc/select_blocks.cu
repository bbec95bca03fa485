// The blocks (pages) that each query token and KV head attends to: the first and the last ones, and of the others
// those with the highest scores.
//
// A block's score is the largest value that q . k could have, summed over the query heads of the KV head, for a key k
// within the bounds lo <= k <= hi that the cache keeps a block and channel:
//   score = sum_g sum_c max(q_gc lo_c, q_gc hi_c) = sum_c (Q-_c lo_c + Q+_c hi_c),
//   Q+_c = sum_g max(q_gc, 0),  Q-_c = sum_g min(q_gc, 0),
// one product of length 2 d whatever the number of query heads.  Which blocks are chosen does not depend on the
// order of summation: scores come from the tensor cores with an error bound, and those blocks that lie within the
// bound of the border are scored again in 64 bits.
//
// Score kernel: a warp holds the bounds of 16 blocks as the left operand, from HBM straight to registers, and
// multiplies them with up to 32 query rows; Q+- enter as two bf16 numbers each (16 bits), in two columns.
//   |score - exact| <= EPS ||Q|| ||b||,  b = (lo, hi) of a block, by Cauchy and Schwarz on the sum of |terms|:
//   2^-18 for the two roundings, G 2^-24 for the sums over heads, and for the 2 d / 16 products and their final
//   addition, of 16 terms each, 2^-22 apiece.
// Select kernel: a CTA finds the k-th largest score of its row and head by its bits, 8 at a time, then settles the
// border.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "decode_shares.cuh"
#include "sm103.cuh"
#include "step.h"

namespace attn {

__device__ uint32_t g_select_blocks_status;

namespace {

using shares::mma_16816;

constexpr uint32_t FULL = 0xffffffffu;
constexpr int PAGE = 16;
constexpr int SCORE_WARPS = 8;
constexpr int TILE_ROWS = 32;      // query rows a CTA scores
constexpr int SELECT_THREADS = 256;
constexpr int BORDER = 512;        // blocks at the border whose exact scores shared memory holds
// Norms below this count as this: squares of smaller numbers may vanish, and a bound that is too large does no harm
constexpr float LEAST_NORM = 1e-14f;
constexpr int64_t SCORE_CTAS = 152 * 32;  // of the grid, about: a block table may be far wider than its sequences

__host__ __device__ constexpr float eps_of(int d, int G) {
  return 1.f / (1 << 18) + static_cast<float>(G) / (1 << 24) + static_cast<float>(d / 8 + 2) / (1 << 22);
}

struct Scratch {
  float* scores;  // [T][Hkv][stride]
  float* q_norm;  // [T][Hkv]
  float* b_norm;  // [N][Hkv][tiles]: the largest norm among 16 blocks
  int64_t stride;
  int tiles;
};
size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
__host__ __device__ constexpr int64_t score_stride(int64_t max_blocks) { return (max_blocks + 7) / 8 * 8; }

// The query tokens of sequence n: rows first .. end - 1; the last of them sees all `len` tokens
struct Span {
  int first, end, len;
};
__device__ __forceinline__ Span span_of(const SelectBlocksParams& p, int n, bool report) {
  Span s{n, n + 1, p.seq_lens[n]};
  if (p.cu != nullptr) {
    s.first = p.cu[n];
    s.end = p.cu[n + 1];
  }
  const bool bad = s.first < 0 || s.end < s.first || s.end > p.T || s.end - s.first > p.max_q || s.len < 0 ||
                   s.len > p.max_blocks * PAGE;
  if (bad && report) set_error(&g_select_blocks_status, kDevBadSeqlens);
  if (s.first < 0 || s.end < s.first || s.end > p.T || s.end - s.first > p.max_q) s.end = s.first = 0;  // skipped
  s.len = s.len < 0 ? 0 : s.len > p.max_blocks * PAGE ? p.max_blocks * PAGE : s.len;
  return s;
}
// blocks that row r of a span sees
__device__ __forceinline__ int blocks_seen(const Span& s, int r) {
  const int seen = s.len - (s.end - 1 - r);
  return seen <= 0 ? 0 : (seen + PAGE - 1) / PAGE;
}

__device__ __forceinline__ float2 pair_of(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// CG: groups of four query rows that a CTA takes
template <int D, int CG>
__global__ void __launch_bounds__(SCORE_WARPS * 32) score_kernel(const SelectBlocksParams p, const Scratch ws, int row_tiles,
                                                                 int chunks) {
  constexpr int KK = 2 * D / 32;            // 32 of the 2 d terms at a time
  constexpr int PART = KK < 8 ? KK : 8;     // as many as registers hold
  extern __shared__ __align__(16) uint32_t s_q[];  // [CG][KK][8 columns][16 words]
  const int chunk = blockIdx.x % chunks;
  const int rest = blockIdx.x / chunks, rt = rest % row_tiles, nh = rest / row_tiles;
  const int n = nh / p.Hkv, h = nh % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Span s = span_of(p, n, chunk == 0 && rt == 0 && h == 0 && threadIdx.x == 0);
  const int r0 = s.first + rt * (4 * CG);
  const int rows = s.end - r0 < 4 * CG ? s.end - r0 : 4 * CG;
  if (rows <= 0) return;
  const int nb = blocks_seen(s, r0 + rows - 1);
  if (nb <= p.K || chunk * SCORE_WARPS * 16 >= nb) return;  // every block is chosen, or none is this CTA's
  const bool last_rows = r0 + rows == s.end;  // they see all that the others do: the blocks' norms are theirs to write

  // ---- Q-, Q+ of the rows, each as two bf16 numbers in neighbouring columns
  const int G = p.Hq / p.Hkv;
  for (int i = threadIdx.x; i < CG * 4 * (D / 2); i += SCORE_WARPS * 32) {
    const int row = i / (D / 2), c = i % (D / 2);  // channels 2 c, 2 c + 1
    float neg[2] = {0.f, 0.f}, pos[2] = {0.f, 0.f};
    if (row < rows) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(r0 + row) * p.Hq + h * G) * D) + c;
      for (int e = 0; e < G; ++e) {
        const float2 x = pair_of(q[e * (D / 2)]);
        // a NaN stays one in both sums
        neg[0] += x.x > 0.f ? 0.f : x.x; pos[0] += x.x < 0.f ? 0.f : x.x;
        neg[1] += x.y > 0.f ? 0.f : x.y; pos[1] += x.y < 0.f ? 0.f : x.y;
      }
    }
    uint32_t* at = s_q + ((row / 4) * KK + c / 16) * 128 + row % 4 * 32 + c % 16;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float* x = half ? pos : neg;
      const uint32_t hi = pack_bf16x2(x[0], x[1]);
      const float2 y = pair_of(hi);
      at[half * (KK / 2) * 128] = hi;
      at[half * (KK / 2) * 128 + 16] = pack_bf16x2(x[0] - y.x, x[1] - y.y);
    }
  }
  __syncthreads();
  if (chunk == 0)
    for (int row = warp; row < rows; row += SCORE_WARPS) {
      float sum = 0.f;
      uint32_t any = 0;
      for (int i = lane; i < KK * 16; i += 32) {
        const uint32_t* at = s_q + ((row / 4) * KK + i / 16) * 128 + row % 4 * 32 + i % 16;
        any |= at[0] & 0x7fff7fffu;
        const float2 hi = pair_of(at[0]), lo = pair_of(at[16]);
        sum = fmaf(hi.x + lo.x, hi.x + lo.x, fmaf(hi.y + lo.y, hi.y + lo.y, sum));
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(FULL, sum, off);
      any = __reduce_or_sync(FULL, any);
      // (a NaN passes the comparison)
      if (lane == 0)
        ws.q_norm[static_cast<int64_t>(r0 + row) * p.Hkv + h] = any == 0 ? 0.f : sum < LEAST_NORM * LEAST_NORM ? LEAST_NORM : sqrtf(sum);
    }

  for (int tile = chunk * SCORE_WARPS + warp; tile * 16 < nb; tile += chunks * SCORE_WARPS) {
    // this lane's part of blocks 16 tile + g and + 8: 16 bytes of each 64
    const __nv_bfloat16* from[2];
    bool there[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int blk = tile * 16 + g + 8 * e;
      there[e] = blk < nb;
      int id = there[e] ? p.block_table[static_cast<int64_t>(n) * p.max_blocks + blk] : 0;
      if (id < 0 || id >= p.num_blocks) {
        if (t == 0) set_error(&g_select_blocks_status, kDevBadPage);
        id = 0;
      }
      from[e] = p.bounds + (static_cast<int64_t>(id) * p.Hkv + h) * 2 * D + 8 * t;
    }
    float acc[CG][4];
#pragma unroll
    for (int c = 0; c < CG; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;
    float norm[2] = {0.f, 0.f};
    uint32_t any = 0;
#pragma unroll
    for (int k0 = 0; k0 < KK; k0 += PART) {
      uint32_t a[PART][2][4];
#pragma unroll
      for (int k = 0; k < PART; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (there[e]) x = *reinterpret_cast<const uint4*>(from[e] + 32 * (k0 + k));
          a[k][e][0] = x.x; a[k][e][1] = x.y; a[k][e][2] = x.z; a[k][e][3] = x.w;
        }
      if (last_rows) {
#pragma unroll
        for (int k = 0; k < PART; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float2 x = pair_of(a[k][e][w]);
              any |= a[k][e][w] & 0x7fff7fffu;
              norm[e] = fmaf(x.x, x.x, fmaf(x.y, x.y, norm[e]));
            }
      }
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        if (CG > 1 && 4 * c >= rows) break;
#pragma unroll
        for (int k = 0; k < PART; ++k) {
          const uint4 b = *reinterpret_cast<const uint4*>(s_q + (c * KK + k0 + k) * 128 + g * 16 + t * 4);
          mma_16816<false>(acc[c], a[k][0][0], a[k][1][0], a[k][0][1], a[k][1][1], b.x, b.y);
          mma_16816<false>(acc[c], a[k][0][2], a[k][1][2], a[k][0][3], a[k][1][3], b.z, b.w);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < CG; ++c) {
      const int row = 4 * c + t;
      if (row >= rows) continue;
      float* out = ws.scores + (static_cast<int64_t>(r0 + row) * p.Hkv + h) * ws.stride + tile * 16 + g;
      if (there[0]) out[0] = acc[c][0] + acc[c][1];
      if (there[1]) out[8] = acc[c][2] + acc[c][3];
    }
    if (last_rows) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        norm[e] += __shfl_xor_sync(FULL, norm[e], 1);
        norm[e] += __shfl_xor_sync(FULL, norm[e], 2);
        if (!(norm[e] < INFINITY)) norm[e] = INFINITY;  // NaN too
      }
      const float most = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(fmaxf(norm[0], norm[1]))));
      any = __reduce_or_sync(FULL, any);
      if (lane == 0) ws.b_norm[static_cast<int64_t>(nh) * ws.tiles + tile] = any == 0 ? 0.f : fmaxf(sqrtf(most), LEAST_NORM);
    }
  }
}

// A float's bits in an order of whole numbers
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_order(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ unsigned long long order_of(double x) {
  if (x != x) return ~0ull;  // NaN is the highest
  const unsigned long long u = __double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}

template <int D>
__global__ void __launch_bounds__(SELECT_THREADS, 4) select_kernel(const SelectBlocksParams p, const Scratch ws) {
  constexpr int T = SELECT_THREADS, NW = T / 32;
  extern __shared__ __align__(16) uint32_t s_bits[];  // [words] chosen blocks, [words] ties
  __shared__ int s_hist[256];
  __shared__ double s_q[2 * D];
  __shared__ unsigned long long s_key[BORDER];
  __shared__ int s_at[BORDER], s_sum[NW], s_count, s_in, s_digit, s_above;
  __shared__ float s_norm[NW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  int n = r;
  if (p.cu != nullptr) {
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= r) lo = mid;
      else hi = mid;
    }
    n = lo;
  }
  const Span s = span_of(p, n, false);
  if (r < s.first || r >= s.end) return;  // of no sequence: left as it was
  const int nb = blocks_seen(s, r), K = p.K;
  int32_t* out = p.blocks + static_cast<int64_t>(blockIdx.x) * K;
  if (nb <= K) {
    for (int i = threadIdx.x; i < K; i += T) out[i] = i < nb ? i : -1;
    return;
  }
  const int c0 = p.first, c1 = nb - p.last;  // the blocks that compete
  const int want = K - p.first - p.last;     // for so many places: fewer than they are
  const int words = (nb + 31) / 32;
  uint32_t* ties = s_bits + words;
  const float* sc = ws.scores + static_cast<int64_t>(blockIdx.x) * ws.stride;

  // ---- how far a score may be off
  float most = 0.f;
  {
    const float* norms = ws.b_norm + (static_cast<int64_t>(n) * p.Hkv + h) * ws.tiles;
    for (int i = threadIdx.x; i < (nb + 15) / 16; i += T) most = fmaxf(most, norms[i]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(FULL, most, off));
    if (lane == 0) s_norm[warp] = most;
    if (threadIdx.x == 0) s_count = s_in = 0;
    __syncthreads();
    most = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) most = fmaxf(most, s_norm[i]);
  }
  const float off = eps_of(D, p.Hq / p.Hkv) * ws.q_norm[blockIdx.x] * most;
  const bool known = off < INFINITY;  // else a NaN or infinity is about, and every score is taken again

  // ---- the want-th largest score: digit by digit, from the highest
  uint32_t border = 0;
  if (known && want > 0) {
    uint32_t mask = 0;
    int left = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += T) s_hist[i] = 0;
      __syncthreads();
      for (int i = c0 + threadIdx.x; i < c1; i += T) {
        const uint32_t u = order_of(sc[i]);
        if (((u ^ border) & mask) == 0) atomicAdd(&s_hist[u >> shift & 255], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // lane 0 holds the eight highest digits
        int c[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += c[j] = s_hist[255 - 8 * lane - j];
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(FULL, upto, o);
          if (lane >= o) upto += x;
        }
        int above = upto - sum;
        if (above < left && left <= upto) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (above < left && left <= above + c[j]) {
              s_digit = 255 - 8 * lane - j;
              s_above = above;
            }
            above += c[j];
          }
        }
      }
      __syncthreads();
      border |= static_cast<uint32_t>(s_digit) << shift;
      mask |= 255u << shift;
      left -= s_above;
    }
  }
  // a score above `high` is chosen, one below `low` is not; the twofold bound, since the border is off by as much
  const float at = from_order(border), high = known ? at + 2.f * off : INFINITY, low = known ? at - 2.f * off : -INFINITY;
  auto undecided = [&](int i) { return want > 0 && i >= c0 && i < c1 && (!known || (sc[i] <= high && sc[i] >= low)); };
  int in = 0;
  for (int w = warp; w < words; w += NW) {
    const int i = 32 * w + lane;
    const bool kept = i < nb && (i < c0 || i >= c1), over = known && want > 0 && i >= c0 && i < c1 && sc[i] > high;
    const bool open = undecided(i);
    const unsigned chosen = __ballot_sync(FULL, kept || over);
    in += __popc(__ballot_sync(FULL, over));
    if (lane == 0) s_bits[w] = chosen;
    if (open) {
      const int k = atomicAdd(&s_count, 1);
      if (k < BORDER) s_at[k] = i;
    }
  }
  if (lane == 0) atomicAdd(&s_in, in);
  __syncthreads();
  const int open = s_count, places = want - s_in;  // places <= open
  auto choose = [&](int i) { atomicOr(&s_bits[i >> 5], 1u << (i & 31)); };
  // the exact scores: the sums over heads, and a product with block i's bounds by a warp
  auto sum_heads = [&]() {
    const int G = p.Hq / p.Hkv;
    for (int c = threadIdx.x; c < D; c += T) {
      const __nv_bfloat16* q = p.q + (static_cast<int64_t>(r) * p.Hq + h * G) * D + c;
      double neg = 0.0, pos = 0.0;
      for (int e = 0; e < G; ++e) {
        const double x = __bfloat162float(q[e * D]);
        neg += x > 0.0 ? 0.0 : x;
        pos += x < 0.0 ? 0.0 : x;
      }
      s_q[c] = neg;
      s_q[D + c] = pos;
    }
    __syncthreads();
  };
  auto exact = [&](int i) {
    int id = p.block_table[static_cast<int64_t>(n) * p.max_blocks + i];
    if (id < 0 || id >= p.num_blocks) id = 0;
    const uint32_t* b = reinterpret_cast<const uint32_t*>(p.bounds + (static_cast<int64_t>(id) * p.Hkv + h) * 2 * D);
    double sum = 0.0;
#pragma unroll
    for (int c = lane; c < D; c += 32) {
      const float2 x = pair_of(b[c]);
      sum = fma(s_q[2 * c], static_cast<double>(x.x), fma(s_q[2 * c + 1], static_cast<double>(x.y), sum));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    return order_of(sum);
  };

  if (places > 0 && open <= BORDER) {
    const bool all = places == open;
    if (!all && off != 0.f) {
      sum_heads();
      for (int k = warp; k < open; k += NW) {
        const unsigned long long key = exact(s_at[k]);
        if (lane == 0) s_key[k] = key;
      }
    } else if (!all) {  // every score is 0
      for (int k = threadIdx.x; k < open; k += T) s_key[k] = 0;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < open; k += T) {
      int before = 0;  // that go before this one
      if (!all)
        for (int j = 0; j < open; ++j)
          before += s_key[j] > s_key[k] || (s_key[j] == s_key[k] && s_at[j] < s_at[k]) ? 1 : 0;
      if (before < places) choose(s_at[k]);
    }
  } else if (places > 0) {
    // Many: NaN or infinities, or pages that are alike.  The exact scores' border digit by digit; each is computed again
    // for every digit.
    unsigned long long key_at = 0, mask = 0;
    int left = places;
    const bool zeros = known && off == 0.f;  // every score is 0
    if (!zeros && places < open) {
      sum_heads();
      for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += T) s_hist[i] = 0;
        __syncthreads();
        for (int w = warp; w < words; w += NW)
          for (unsigned todo = __ballot_sync(FULL, undecided(32 * w + lane)); todo != 0; todo &= todo - 1) {
            const unsigned long long key = exact(32 * w + __ffs(todo) - 1);
            if (lane == 0 && ((key ^ key_at) & mask) == 0) atomicAdd(&s_hist[key >> shift & 255], 1);
          }
        __syncthreads();
        if (threadIdx.x == 0) {
          int above = 0, digit = 255;
          while (digit > 0 && above + s_hist[digit] < left) above += s_hist[digit--];
          s_digit = digit;
          s_above = above;
        }
        __syncthreads();
        key_at |= static_cast<unsigned long long>(s_digit) << shift;
        mask |= 255ull << shift;
        left -= s_above;
      }
    }
    for (int w = warp; w < words; w += NW) {
      const unsigned todo = __ballot_sync(FULL, undecided(32 * w + lane));
      unsigned over = 0, tie = todo;
      if (!zeros && places < open) {
        tie = 0;
        for (unsigned x = todo; x != 0; x &= x - 1) {
          const unsigned long long key = exact(32 * w + __ffs(x) - 1);
          if (key > key_at) over |= x & -x;
          else if (key == key_at) tie |= x & -x;
        }
      }
      if (lane == 0) {
        s_bits[w] |= over;
        ties[w] = tie;
      }
    }
    __syncthreads();
    if (warp == 0)  // the lowest of those that tie
      for (int w = 0; w < words && left > 0; ++w) {
        unsigned tie = ties[w];
        while (__popc(tie) > left) tie &= ~(0x80000000u >> __clz(tie));
        left -= __popc(tie);
        if (lane == 0) s_bits[w] |= tie;
      }
  }
  __syncthreads();

  // ---- in ascending order: each warp a run of words
  const int per = (words + NW - 1) / NW, w0 = warp * per < words ? warp * per : words;
  const int w1 = w0 + per < words ? w0 + per : words;
  int sum = 0;
  for (int w = w0 + lane; w < w1; w += 32) sum += __popc(s_bits[w]);
  sum = __reduce_add_sync(FULL, sum);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  int to = 0;
  for (int i = 0; i < warp; ++i) to += s_sum[i];
  for (int w = w0; w < w1; ++w) {
    const unsigned bits = s_bits[w];
    const int place = to + __popc(bits & ((1u << lane) - 1));
    if (bits >> lane & 1 && place < K) out[place] = 32 * w + lane;
    to += __popc(bits);
  }
}

template <int D, int CG>
cudaError_t launch(const SelectBlocksParams& p, const Scratch& ws, cudaStream_t stream) {
  const int row_tiles = (p.max_q + 4 * CG - 1) / (4 * CG);
  const int64_t pairs = static_cast<int64_t>(p.N) * p.Hkv * row_tiles;
  const int64_t all = (p.max_blocks + SCORE_WARPS * 16 - 1) / (SCORE_WARPS * 16), most = (SCORE_CTAS + pairs - 1) / pairs;
  const int chunks = static_cast<int>(all < most ? all : most);
  const int smem = CG * (2 * D / 32) * 512;
  cudaError_t e = cudaFuncSetAttribute(score_kernel<D, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  score_kernel<D, CG><<<static_cast<unsigned>(pairs * chunks), SCORE_WARPS * 32, smem, stream>>>(p, ws, row_tiles, chunks);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int bits = 2 * ((p.max_blocks + 31) / 32) * 4;
  e = cudaFuncSetAttribute(select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bits);
  if (e != cudaSuccess) return e;
  select_kernel<D><<<static_cast<unsigned>(static_cast<int64_t>(p.T) * p.Hkv), SELECT_THREADS, bits, stream>>>(p, ws);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_for(const SelectBlocksParams& p, const Scratch& ws, cudaStream_t stream) {
  return p.max_q <= 4 ? launch<D, 1>(p, ws, stream) : launch<D, TILE_ROWS / 4>(p, ws, stream);
}

}  // namespace

size_t select_blocks_workspace_bytes(int64_t T, int64_t N, int64_t Hkv, int64_t max_blocks) {
  return up256(T * Hkv * score_stride(max_blocks) * 4) + up256(T * Hkv * 4) + up256(N * Hkv * ((max_blocks + 15) / 16) * 4);
}

cudaError_t select_blocks_launch(const SelectBlocksParams& p, cudaStream_t stream) {
  Scratch ws;
  ws.stride = score_stride(p.max_blocks);
  ws.tiles = (p.max_blocks + 15) / 16;
  const size_t rows = static_cast<size_t>(p.T) * p.Hkv;
  uint8_t* at = static_cast<uint8_t*>(p.workspace);
  ws.scores = reinterpret_cast<float*>(at);
  at += up256(rows * ws.stride * 4);
  ws.q_norm = reinterpret_cast<float*>(at);
  at += up256(rows * 4);
  ws.b_norm = reinterpret_cast<float*>(at);
  if (p.d == 64) return launch_for<64>(p, ws, stream);
  if (p.d == 128) return launch_for<128>(p, ws, stream);
  if (p.d == 256) return launch_for<256>(p, ws, stream);
  return cudaErrorInvalidValue;
}

cudaError_t select_blocks_status(uint32_t* out, bool clear) { return read_status(g_select_blocks_status, out, clear); }

}  // namespace attn
