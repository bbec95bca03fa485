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
//   |score - exact| <= eps ||Q|| ||b||,  b = (lo, hi) of a block, by Cauchy and Schwarz on the sum of |terms|.
// Select kernel: a CTA puts the scores of its row and head into bins over their range, gathers the few in and about the
// bin that holds the border, and a warp settles the border among them.
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
constexpr int BINS = 512;          // of a window of scores
constexpr int CACHED = 12288;      // scores of a row that shared memory holds
constexpr int NARROW = 1024;       // columns of a block table, and ...
constexpr int64_t FEW_ROWS = 1024;  // ... rows times heads from which on a row has 128 threads
// Norms below this count as this: squares of smaller numbers may vanish, and a bound that is too large does no harm
constexpr float LEAST_NORM = 1e-14f;
constexpr int64_t SCORE_CTAS = 152 * 4;  // of the grid, about: a block table may be far wider than its sequences

struct Scratch {
  float* scores;  // [T][Hkv][stride]
  float* q_norm;  // [T][Hkv]
  float* b_norm;  // [N][Hkv][tiles]: a bound of the largest norm among 16 blocks
  int64_t stride;
  int tiles;
  float eps;
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

__device__ __forceinline__ int sequence_of(const SelectBlocksParams& p, int r) {
  int lo = 0, hi = p.N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float2 pair_of(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// sum + w * w for a pair, in bf16: 64 such additions are off by an eighth at most
__device__ __forceinline__ uint32_t add_squares(uint32_t w, uint32_t sum) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %1, %2;" : "=r"(d) : "r"(w), "r"(sum));
  return d;
}

// A piece of 16 bytes of row r of a tile in shared memory: rows are whole multiples of 128 bytes apart, and a quarter
// of a warp reads four pieces of two neighbouring rows
__device__ __forceinline__ int swizzled(int r, int piece) { return piece ^ ((r & 1) << 2 | (r >> 1 & 3)); }

template <int D>
struct FewCfg {
  static constexpr int PARTS = D == 256 ? 2 : 1;     // of a tile, a stage of the ring each
  static constexpr int ROW = 4 * D / PARTS;          // bytes of a block's bounds in a stage
  static constexpr int STAGE = 16 * ROW;
  static constexpr int DEPTH = 2;                    // stages a warp: a tile's arithmetic takes longer than HBM does
  static constexpr int TERMS = 2 * 2 * D * 2;        // bytes of Q- and Q+ of a row: two columns
  static constexpr int MOST_WARPS = D == 64 ? 16 : 13;
  static constexpr int warp_bytes(int rows) { return DEPTH * STAGE + rows * TERMS; }
  static int warps(int rows) {
    const int fit = 222 * 1024 / warp_bytes(rows);
    return fit < MOST_WARPS ? fit : MOST_WARPS;
  }
};

// Up to four query rows a sequence (a decode step): HBM's rate is what matters.  The list of (sequence, KV head, tile
// of 16 blocks) is cut into equal runs, one a warp of a grid that fills the device; each warp keeps DEPTH tiles in
// flight to shared memory, so that the chain from lengths to table to bounds is waited for once.
template <int D>
__global__ void __launch_bounds__(FewCfg<D>::MOST_WARPS * 32, 1) score_few_kernel(const SelectBlocksParams p, const Scratch ws) {
  using C = FewCfg<D>;
  constexpr int KK = 2 * D / 32, PART = KK / C::PARTS, PIECES = C::ROW / 16;  // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_before[C::MOST_WARPS * 32], s_sum[C::MOST_WARPS];
  const int NW = blockDim.x / 32, T = blockDim.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // every CTA of this grid is resident: the select kernel's may queue up behind them
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int N = p.N, Hkv = p.Hkv;
  struct Seq {
    int tiles, nb;  // of a KV head; no tiles where every block is chosen
  };
  auto seq_of = [&](int n, bool report) {
    const Span s = span_of(p, n, report);
    const int nb = s.end > s.first ? blocks_seen(s, s.end - 1) : 0;
    return Seq{nb <= p.K ? 0 : (nb + 15) / 16, nb};
  };
  const int chunk = (N + T - 1) / T;  // sequences a thread counts
  int mine = 0;
  for (int n = threadIdx.x * chunk, i = 0; i < chunk && n < N; ++n, ++i) mine += seq_of(n, blockIdx.x == 0).tiles;
  int upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(FULL, upto, off);
    if (lane >= off) upto += x;
  }
  s_before[threadIdx.x] = upto - mine;  // within the warp
  if (lane == 31) s_sum[warp] = upto;
  __syncthreads();
  const int sums = lane < NW ? s_sum[lane] : 0;
  int before = sums;
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) {
    const int x = __shfl_up_sync(FULL, before, off);
    if (lane >= off) before += x;
  }
  const unsigned W = static_cast<unsigned>(__shfl_sync(FULL, before, 15)) * Hkv;  // below 2^31
  before -= sums;
  const unsigned runs = gridDim.x * NW, per = (W + runs - 1) / runs, x0 = (blockIdx.x * NW + warp) * per;
  if (x0 >= W) return;
  const int count = min(per, W - x0);
  // the warp, then the thread, whose sequences hold tile x0
  const int v = 31 - __clz(__ballot_sync(FULL, lane < NW && static_cast<unsigned>(before) * Hkv <= x0));
  before = __shfl_sync(FULL, before, v);
  const int in_warp = before + s_before[v * 32 + lane];
  const int u = 31 - __clz(__ballot_sync(FULL, static_cast<unsigned>(in_warp) * Hkv <= x0));
  unsigned rest = x0 - static_cast<unsigned>(__shfl_sync(FULL, in_warp, u)) * Hkv;
  int n0 = (v * 32 + u) * chunk;
  Seq seq0 = seq_of(n0, false);
  while (rest >= static_cast<unsigned>(seq0.tiles) * Hkv) {
    rest -= static_cast<unsigned>(seq0.tiles) * Hkv;
    seq0 = seq_of(++n0, false);
  }

  struct Place {  // in the list
    int n, h, tile, tiles, nb;
  };
  auto advance = [&](Place& x) {
    if (++x.tile < x.tiles) return;
    x.tile = 0;
    if (++x.h < Hkv) return;
    x.h = 0;
    Seq y;
    do y = seq_of(++x.n, false);
    while (y.tiles == 0);
    x.tiles = y.tiles;
    x.nb = y.nb;
  };
  auto page_of = [&](const Place& x) {  // of block 16 tile + lane % 16; page 0 where there is none
    const int blk = x.tile * 16 + (lane & 15);
    int id = blk < x.nb ? p.block_table[static_cast<int64_t>(x.n) * p.max_blocks + blk] : 0;
    if (id < 0 || id >= p.num_blocks) {
      set_error(&g_select_blocks_status, kDevBadPage);
      id = 0;
    }
    return id;
  };
  const int rows_held = p.max_q;
  uint8_t* ring = smem + warp * C::warp_bytes(rows_held);
  // Q-, Q+ of the rows, each as two bf16 numbers in neighbouring columns: [2 rows_held columns][KK][16 words]
  uint32_t* s_q = reinterpret_cast<uint32_t*>(ring + C::DEPTH * C::STAGE);
  const uint32_t ring_at = smem_u32(ring);
  const uint32_t page_bytes = static_cast<uint32_t>(Hkv) * (4 * D);
  auto request = [&](int h, int id, int part, int stage) {
    // a lane's piece is the same in every row that it copies
    const uint8_t* base =
        reinterpret_cast<const uint8_t*>(p.bounds) + static_cast<int64_t>(h) * (4 * D) + part * C::ROW + lane % PIECES * 16;
#pragma unroll 8
    for (int i = 0; i < PIECES / 2; ++i) {
      const int r = i * (32 / PIECES) + lane / PIECES;
      const uint8_t* from = base + static_cast<uint64_t>(static_cast<uint32_t>(__shfl_sync(FULL, id, r))) * page_bytes;
      const uint32_t to = ring_at + stage * C::STAGE + r * C::ROW + swizzled(r, lane % PIECES) * 16;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // row `row`'s heads e0 .. e0 + 3 of a KV head, channels 2 lane + 64 x and the next; all loads in flight
  uint32_t heads[4][D / 64];
  const int G = p.Hq / Hkv;
  auto load_heads = [&](int row, int h, int e0) {
    const uint32_t* from = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(row) * p.Hq + h * G) * D) + lane;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int x = 0; x < D / 64; ++x) heads[e][x] = e0 + e < G ? from[(e0 + e) * (D / 2) + 32 * x] : 0u;
  };
  Place ahead{n0, static_cast<int>(rest / seq0.tiles), static_cast<int>(rest % seq0.tiles), seq0.tiles, seq0.nb};
  Place at = ahead;
  load_heads(p.cu == nullptr ? n0 : p.cu[n0], at.h, 0);  // before the bounds, behind which they would wait
  bool loaded = true;
  const int steps = count * C::PARTS;  // a part of a tile each
  // the next tile to request and the one behind it: table entries are read two tiles ahead, or they would wait behind
  // the bounds that are on their way
  int h_now = ahead.h, id_now = page_of(ahead), h_then = 0, id_then = 0, known = 1;
  auto look_ahead = [&]() {
    if (known == count) return;
    ++known;
    advance(ahead);
    h_then = ahead.h;
    id_then = page_of(ahead);
  };
  look_ahead();
  int asked = 0, asked_part = 0;
  auto request_next = [&](int stage) {
    if (asked >= steps) {
      asm volatile("cp.async.commit_group;" ::: "memory");  // an empty one: the count of groups stays in step
      return;
    }
    request(h_now, id_now, asked_part, stage);
    ++asked;
    if (++asked_part == C::PARTS) {
      asked_part = 0;
      h_now = h_then;
      id_now = id_then;
      look_ahead();
    }
  };
  request_next(0);
  int rows = 0, r0 = 0, stage = 0;
  bool fresh = true;
  float acc[2][4] = {};
  float norm[2] = {0.f, 0.f};
  for (int done = 0; done < steps; ++done) {
    const int part = C::PARTS == 1 ? 0 : done % C::PARTS;
    request_next(stage ^ 1);
    if (fresh) {  // another sequence or head
      fresh = false;
      const Span s = span_of(p, at.n, false);
      r0 = s.first;
      rows = s.end - s.first;
      for (int row = 0; row < rows; ++row) {
        float squares = 0.f;
        uint32_t any = 0;
        float neg[D / 32] = {}, pos[D / 32] = {};
        for (int e0 = 0; e0 < G; e0 += 4) {
          if (!loaded) load_heads(r0 + row, at.h, e0);
          loaded = false;
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
              const float2 y = pair_of(heads[e][x]);
              // a NaN stays one in both sums
              neg[2 * x] += y.x > 0.f ? 0.f : y.x;
              pos[2 * x] += y.x < 0.f ? 0.f : y.x;
              neg[2 * x + 1] += y.y > 0.f ? 0.f : y.y;
              pos[2 * x + 1] += y.y < 0.f ? 0.f : y.y;
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            const float a = half ? pos[2 * x] : neg[2 * x], b = half ? pos[2 * x + 1] : neg[2 * x + 1];
            const uint32_t hi = pack_bf16x2(a, b);
            const float2 z = pair_of(hi);
            const int word = half * (D / 2) + 32 * x + lane;  // of the 2 d terms
            uint32_t* to = s_q + (word / 16 * (2 * rows_held) + 2 * row) * 16 + word % 16;
            to[0] = hi;
            to[16] = pack_bf16x2(a - z.x, b - z.y);
            squares = fmaf(a, a, fmaf(b, b, squares));
            any |= hi & 0x7fff7fffu;
          }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) squares += __shfl_xor_sync(FULL, squares, off);
        any = __reduce_or_sync(FULL, any);
        // (a NaN passes the comparison)
        if (at.tile == 0 && lane == 0)
          ws.q_norm[static_cast<int64_t>(r0 + row) * Hkv + at.h] =
              any == 0 ? 0.f : squares < LEAST_NORM * LEAST_NORM ? LEAST_NORM : sqrtf(squares);
      }
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();

    const uint8_t* from = ring + stage * C::STAGE;
    uint32_t sum[2][2] = {};
    const bool column = g < 2 * rows;
    const uint32_t* q = s_q + (part * PART * (2 * rows_held) + g) * 16 + t * 4;
#pragma unroll 4
    for (int k = 0; k < PART; ++k) {
      uint32_t a[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint4 x = *reinterpret_cast<const uint4*>(from + (g + 8 * e) * C::ROW + swizzled(g, 4 * k + t) * 16);
        a[e][0] = x.x; a[e][1] = x.y; a[e][2] = x.z; a[e][3] = x.w;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum[e][w & 1] = add_squares(a[e][w], sum[e][w & 1]);
      }
      uint4 b = make_uint4(0, 0, 0, 0);
      if (column) b = *reinterpret_cast<const uint4*>(q + k * (2 * rows_held) * 16);
      mma_16816<false>(acc[0], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
      mma_16816<false>(acc[1], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
    }
    __syncwarp();  // every lane has read the stage
    stage ^= 1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 y = pair_of(sum[e][0]), z = pair_of(sum[e][1]);
      norm[e] += (y.x + y.y) + (z.x + z.y);
    }
    if (part + 1 < C::PARTS) continue;
    const int blk = at.tile * 16 + g;
    if (t < rows) {  // columns 2 t, 2 t + 1 are row t's
      float* out = ws.scores + (static_cast<int64_t>(r0 + t) * Hkv + at.h) * ws.stride + blk;
      if (blk < at.nb) out[0] = (acc[0][0] + acc[1][0]) + (acc[0][1] + acc[1][1]);
      if (blk + 8 < at.nb) out[8] = (acc[0][2] + acc[1][2]) + (acc[0][3] + acc[1][3]);
    }
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      norm[e] += __shfl_xor_sync(FULL, norm[e], 1);
      norm[e] += __shfl_xor_sync(FULL, norm[e], 2);
      if (!(norm[e] < INFINITY)) norm[e] = INFINITY;  // NaN too
      if (blk + 8 * e < at.nb) most = max(most, __float_as_uint(norm[e]));  // else page 0's
      norm[e] = 0.f;
    }
    most = __reduce_max_sync(FULL, most);
    // the sum of squares may have been an eighth too small
    if (lane == 0)
      ws.b_norm[(static_cast<int64_t>(at.n) * Hkv + at.h) * ws.tiles + at.tile] =
          fmaxf(1.1f * sqrtf(__uint_as_float(most)), LEAST_NORM);
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[0][x] = acc[1][x] = 0.f;
    if (done + 1 < steps) {
      const int n = at.n, h = at.h;
      advance(at);
      fresh = at.n != n || at.h != h;
    }
  }
}

// CG: groups of four query rows that a CTA takes
template <int D, int CG>
__global__ void __launch_bounds__(SCORE_WARPS * 32, D == 256 ? 1 : 2)
    score_kernel(const SelectBlocksParams p, const Scratch ws, int row_tiles, int chunks) {
  constexpr int KK = 2 * D / 32;            // 32 of the 2 d terms at a time
  constexpr int PART = KK < 8 ? KK : 8;     // as many as registers hold
  constexpr int PARTS = KK / PART;
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

  // page of block 16 tile + lane % 16
  auto page_of = [&](int tile) {
    const int blk = tile * 16 + (lane & 15);
    int id = blk < nb ? p.block_table[static_cast<int64_t>(n) * p.max_blocks + blk] : 0;
    if (id < 0 || id >= p.num_blocks) {
      set_error(&g_select_blocks_status, kDevBadPage);
      id = 0;
    }
    return id;
  };
  // terms 32 PART part .. of this lane's share of blocks 16 tile + g and + 8: 16 bytes of each 64
  uint32_t a[PART][2][4];
  auto load = [&](int tile, int id, int part) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t page = __shfl_sync(FULL, id, g + 8 * e);
      const bool there = tile * 16 + g + 8 * e < nb;
      const __nv_bfloat16* from = p.bounds + (page * p.Hkv + h) * 2 * D + 32 * PART * part + 8 * t;
#pragma unroll
      for (int k = 0; k < PART; ++k) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (there) x = *reinterpret_cast<const uint4*>(from + 32 * k);
        a[k][e][0] = x.x; a[k][e][1] = x.y; a[k][e][2] = x.z; a[k][e][3] = x.w;
      }
    }
  };
  int tile = chunk * SCORE_WARPS + warp;
  int id = 0;
  if (tile * 16 < nb) id = page_of(tile);

  // ---- Q-, Q+ of the rows, each as two bf16 numbers in neighbouring columns
  const int G = p.Hq / p.Hkv;
  for (int i = threadIdx.x; i < CG * 4 * (D / 2); i += SCORE_WARPS * 32) {
    const int row = i / (D / 2), c = i % (D / 2);  // channels 2 c, 2 c + 1
    float neg[2] = {0.f, 0.f}, pos[2] = {0.f, 0.f};
    if (row < rows) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(r0 + row) * p.Hq + h * G) * D) + c;
      for (int e0 = 0; e0 < G; e0 += 4) {  // four heads' loads in flight
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = e0 + e < G ? q[(e0 + e) * (D / 2)] : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = pair_of(w[e]);
          // a NaN stays one in both sums
          neg[0] += x.x > 0.f ? 0.f : x.x; pos[0] += x.x < 0.f ? 0.f : x.x;
          neg[1] += x.y > 0.f ? 0.f : x.y; pos[1] += x.y < 0.f ? 0.f : x.y;
        }
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

  if (tile * 16 < nb) load(tile, id, 0);
  while (tile * 16 < nb) {
    const int next = tile + chunks * SCORE_WARPS;
    int next_id = 0;
    if (next * 16 < nb) next_id = page_of(next);
    float* out = ws.scores + (static_cast<int64_t>(r0 + t) * p.Hkv + h) * ws.stride + tile * 16 + g;
    const int64_t four_rows = 4 * p.Hkv * ws.stride;
    auto write = [&](int c, const float (&acc)[4]) {  // columns 2 t, 2 t + 1 are row 4 c + t's
      if (4 * c + t >= rows) return;
      if (tile * 16 + g < nb) out[c * four_rows] = acc[0] + acc[1];
      if (tile * 16 + g + 8 < nb) out[c * four_rows + 8] = acc[2] + acc[3];
    };
    float acc[PARTS > 1 ? CG : 1][4];
#pragma unroll
    for (int c = 0; c < (PARTS > 1 ? CG : 1); ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;
    float norm[2] = {0.f, 0.f};
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      if (part > 0) load(tile, id, part);
      if (last_rows) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t sum[2] = {0u, 0u};
#pragma unroll
          for (int k = 0; k < PART; ++k)
#pragma unroll
            for (int w = 0; w < 4; ++w) sum[w & 1] = add_squares(a[k][e][w], sum[w & 1]);
          const float2 x = pair_of(sum[0]), y = pair_of(sum[1]);
          norm[e] += (x.x + x.y) + (y.x + y.y);
        }
      }
      auto multiply = [&](int c, float (&sum)[4]) {
#pragma unroll
        for (int k = 0; k < PART; ++k) {
          const uint4 b = *reinterpret_cast<const uint4*>(s_q + (c * KK + part * PART + k) * 128 + g * 16 + t * 4);
          mma_16816<false>(sum, a[k][0][0], a[k][1][0], a[k][0][1], a[k][1][1], b.x, b.y);
          mma_16816<false>(sum, a[k][0][2], a[k][1][2], a[k][0][3], a[k][1][3], b.z, b.w);
        }
      };
      if constexpr (PARTS > 1) {
#pragma unroll
        for (int c = 0; c < CG; ++c)
          if (4 * c < rows) multiply(c, acc[c]);
      } else {
#pragma unroll 2
        for (int c = 0; c < CG; ++c) {
          if (4 * c >= rows) break;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          multiply(c, sum);
          write(c, sum);
        }
      }
    }
    if constexpr (PARTS > 1) {
#pragma unroll
      for (int c = 0; c < CG; ++c) write(c, acc[c]);
    }
    if (last_rows) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        norm[e] += __shfl_xor_sync(FULL, norm[e], 1);
        norm[e] += __shfl_xor_sync(FULL, norm[e], 2);
        if (!(norm[e] < INFINITY)) norm[e] = INFINITY;  // NaN too
      }
      const float most = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(fmaxf(norm[0], norm[1]))));
      // the sum of squares may have been an eighth too small
      if (lane == 0) ws.b_norm[static_cast<int64_t>(nh) * ws.tiles + tile] = fmaxf(1.1f * sqrtf(most), LEAST_NORM);
    }
    tile = next;
    id = next_id;
    if (tile * 16 < nb) load(tile, id, 0);
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

template <int D, int T>
__global__ void __launch_bounds__(T) select_kernel(const SelectBlocksParams p, const Scratch ws, int cached) {
  constexpr int NW = T / 32;
  extern __shared__ __align__(16) uint32_t s_bits[];  // [words] chosen blocks, [words] ties; then [cached] scores
  __shared__ __align__(16) int s_hist[2][BINS];
  __shared__ double s_q[2 * D];
  __shared__ float s_score[32];
  __shared__ int s_at[32], s_open[2], s_over[2], s_digit, s_above;
  __shared__ unsigned s_among;
  __shared__ unsigned long long s_key[32];
  __shared__ uint4 s_red[NW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  const int n = p.cu == nullptr ? r : sequence_of(p, r);
  const Span s = span_of(p, n, false);
  for (int i = threadIdx.x; i < 2 * BINS; i += T) s_hist[0][i] = 0;
  if (threadIdx.x < 2) s_open[threadIdx.x] = s_over[threadIdx.x] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores are there
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

  // ---- how far a score may be off, and the scores' range
  const float* sc = ws.scores + static_cast<int64_t>(blockIdx.x) * ws.stride;
  float low, high, off;
  {
    const float* norms = ws.b_norm + (static_cast<int64_t>(n) * p.Hkv + h) * ws.tiles;
    const float q_norm = ws.q_norm[blockIdx.x];
    uint32_t most = 0, least = ~0u, top = 0;  // norms by their bits, scores by their order
    for (int i = threadIdx.x; i < (nb + 15) / 16; i += T) most = max(most, __float_as_uint(norms[i]));
    float* to = reinterpret_cast<float*>(s_bits + 2 * ((p.max_blocks + 31) / 32));
    const bool keep = nb <= cached;
#pragma unroll 4
    for (int i = threadIdx.x; i < c1; i += T) {
      const float x = sc[i];
      if (keep) to[i] = x;
      if (i >= c0) {
        least = min(least, order_of(x));
        top = max(top, order_of(x));
      }
    }
    if (keep) sc = to;
    most = __reduce_max_sync(FULL, most);
    least = __reduce_min_sync(FULL, least);
    top = __reduce_max_sync(FULL, top);
    if (lane == 0) s_red[warp] = make_uint4(most, least, top, 0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const uint4 x = s_red[i];
      most = max(most, x.x);
      least = min(least, x.y);
      top = max(top, x.z);
    }
    off = ws.eps * q_norm * __uint_as_float(most);
    low = from_order(least);
    high = from_order(top);
  }
  const bool known = off < INFINITY;  // else a NaN or infinity is about, and every score is taken again
  auto choose = [&](int i) { atomicOr(&s_bits[i >> 5], 1u << (i & 31)); };
  // the exact scores: the sums over heads, and a product with block i's bounds by a warp
  auto sum_heads = [&](int begin, int step) {
    const int G = p.Hq / p.Hkv;
    for (int c = begin; c < D; c += step) {
      const __nv_bfloat16* q = p.q + (static_cast<int64_t>(r) * p.Hq + h * G) * D + c;
      double neg = 0.0, pos = 0.0;
      for (int e0 = 0; e0 < G; e0 += 4) {  // four heads' loads in flight
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = e0 + e < G ? __bfloat162float(q[(e0 + e) * D]) : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          neg += x[e] > 0.f ? 0.f : x[e];
          pos += x[e] < 0.f ? 0.f : x[e];
        }
      }
      s_q[c] = neg;
      s_q[D + c] = pos;
    }
  };
  auto exact = [&](int i) {
    int id = p.block_table[static_cast<int64_t>(n) * p.max_blocks + i];
    if (id < 0 || id >= p.num_blocks) id = 0;
    const uint32_t* b = reinterpret_cast<const uint32_t*>(p.bounds + (static_cast<int64_t>(id) * p.Hkv + h) * 2 * D);
    double sum = 0.0;
#pragma unroll 4
    for (int c = lane; c < D; c += 32) {
      const float2 x = pair_of(b[c]);
      sum = fma(s_q[2 * c], static_cast<double>(x.x), fma(s_q[2 * c + 1], static_cast<double>(x.y), sum));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    return order_of(sum);
  };

  // ---- Narrow the window [low, high] about the border, a bin of BINS at a time, until 32 blocks at most are in it.
  // A score far from the others (a first page's, say) costs a round.
  bool few = false;
  int open = 0, over = 0;  // in the window; above it
  for (int round = 0; known && want > 0 && !few; ++round) {
    int* hist = s_hist[round & 1];
    const float range = high - low, per_bin = BINS / range;
    if (!(range < INFINITY && per_bin < INFINITY)) break;  // all alike, or past float32
#pragma unroll 2
    for (int i = threadIdx.x; i < c1; i += T) {
      const float x = sc[i];
      if (i >= c0 && x >= low && x <= high) {
        const int bin = static_cast<int>((x - low) * per_bin);
        atomicAdd(&hist[bin < BINS ? bin : BINS - 1], 1);
      }
    }
    __syncthreads();
    // every warp finds the bin of the border: lane 0 holds the highest
    constexpr int PER = BINS / 32;
    int c[PER], sum = 0, bin = -1;
#pragma unroll
    for (int j = 0; j < PER; j += 4) {
      const int4 x = *reinterpret_cast<const int4*>(hist + BINS - PER * (lane + 1) + j);
      c[j] = x.x; c[j + 1] = x.y; c[j + 2] = x.z; c[j + 3] = x.w;
      sum += x.x + x.y + x.z + x.w;
    }
    int above = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(FULL, above, o);
      if (lane >= o) above += x;
    }
    above += over - sum;
#pragma unroll
    for (int j = PER - 1; j >= 0; --j) {
      if (above < want && want <= above + c[j]) bin = BINS - PER * (lane + 1) + j;
      above += c[j];
    }
    bin = __reduce_max_sync(FULL, bin);
    // its blocks, and those within the twofold error (and a rounding of the bin's ends, 2^-6 of a bin) of it
    const float width = range / BINS, slack = 2.f * off + width * (1.f / 64);
    low = low + bin * width - slack;
    high = low + width + 2.f * slack;
    int above_high = 0;
#pragma unroll 2
    for (int i = threadIdx.x; i - lane < nb; i += T) {
      const bool competes = i >= c0 && i < c1;
      const float x = competes ? sc[i] : 0.f;
      const bool in = competes && x > high, here = competes && !in && x >= low;
      if (here) {
        const int k = atomicAdd(&s_open[round & 1], 1);
        if (k < 32) {
          s_at[k] = i;
          s_score[k] = x;
        }
      }
      const unsigned ins = __ballot_sync(FULL, in), kept = __ballot_sync(FULL, !competes && i < nb);
      above_high += __popc(ins);
      if (lane == 0) s_bits[i >> 5] = ins | kept;
    }
    if (lane == 0 && above_high > 0) atomicAdd(&s_over[round & 1], above_high);
    for (int i = threadIdx.x; i < BINS; i += T) s_hist[round & 1 ^ 1][i] = 0;  // for the round after this one
    __syncthreads();
    open = s_open[round & 1];
    over = s_over[round & 1];
    few = open <= 32;
    if (!few) {
      if (!(high - low < 0.5f * range)) break;  // the error's width: they may as well be alike
      __syncthreads();
      if (threadIdx.x == 0) s_open[round & 1] = s_over[round & 1] = 0;
    }
  }

  if (few) {
    // ---- a warp settles it, a lane a block
    const int places = want - over;  // 1 <= places <= open
    bool sure = false, close = false;
    int i = 0x7fffffff, rest = 0;
    unsigned among = 0;
    if (warp == 0) {
      const bool mine = lane < open;
      const float x = mine ? s_score[lane] : -INFINITY;
      if (mine) i = s_at[lane];
      int rank = 0;
      for (int j = 0; j < open; ++j) {
        const float y = __shfl_sync(FULL, x, j);
        const int k = __shfl_sync(FULL, i, j);
        rank += y > x || (y == x && k < i) ? 1 : 0;
      }
      const float border = __shfl_sync(FULL, x, __ffs(__ballot_sync(FULL, mine && rank == places - 1)) - 1);
      sure = mine && x > border + 2.f * off;
      close = mine && !sure && x >= border - 2.f * off;
      among = __ballot_sync(FULL, close);
      rest = places - __popc(__ballot_sync(FULL, sure));
      const bool all = __popc(among) == rest;
      if (lane == 0) s_among = all || off == 0.f ? 0u : among;
      if (all && (sure || close)) choose(i);
      close = close && !all;
      sure = sure && !all;
      if (all) among = 0;
    }
    __syncthreads();
    if (s_among != 0) {  // by the exact scores, a warp a block
      sum_heads(threadIdx.x, T);
      __syncthreads();
      unsigned todo = s_among;
      for (int k = 0; todo != 0; todo &= todo - 1, ++k) {
        if (k % NW != warp) continue;
        const int j = __ffs(todo) - 1;
        const unsigned long long key = exact(s_at[j]);
        if (lane == 0) s_key[j] = key;
      }
      __syncthreads();
    }
    if (among != 0) {
      const unsigned long long key = close && off != 0.f ? s_key[lane] : 0ull;  // where the bound is 0 every score is
      int before = 0;  // that go before this one
      for (unsigned todo = among; todo != 0; todo &= todo - 1) {
        const int j = __ffs(todo) - 1;
        const unsigned long long y = __shfl_sync(FULL, key, j);
        const int k = __shfl_sync(FULL, i, j);
        before += y > key || (y == key && k < i) ? 1 : 0;
      }
      if (sure || (close && before < rest)) choose(i);
    }
  } else {
    // ---- Many at the border, or none: NaN or infinities, pages that are alike, or no place but the kept ones'.  The
    // border digit by digit, of the scores and then, among those that they leave open, of the exact scores, each computed
    // again for every digit.
    int* hist = s_hist[0];
    auto digit = [&](int left) {  // the one that holds the left-th largest
      __syncthreads();
      if (threadIdx.x == 0) {
        int above = 0, at = 255;
        while (at > 0 && above + hist[at] < left) above += hist[at--];
        s_digit = at;
        s_above = above;
      }
      __syncthreads();
    };
    auto clear = [&]() {
      __syncthreads();
      for (int i = threadIdx.x; i < 256; i += T) hist[i] = 0;
      __syncthreads();
    };
    uint32_t border = 0;
    if (known && want > 0) {
      uint32_t mask = 0;
      int left = want;
      for (int shift = 24; shift >= 0; shift -= 8) {
        clear();
        for (int i = c0 + threadIdx.x; i < c1; i += T) {
          const uint32_t u = order_of(sc[i]);
          if (((u ^ border) & mask) == 0) atomicAdd(&hist[u >> shift & 255], 1);
        }
        digit(left);
        border |= static_cast<uint32_t>(s_digit) << shift;
        mask |= 255u << shift;
        left -= s_above;
      }
    }
    const float at = from_order(border), most = known ? at + 2.f * off : INFINITY, least = known ? at - 2.f * off : -INFINITY;
    auto undecided = [&](int i) { return want > 0 && i >= c0 && i < c1 && (!known || (sc[i] <= most && sc[i] >= least)); };
    __syncthreads();
    if (threadIdx.x == 0) s_open[0] = s_over[0] = 0;
    __syncthreads();
    int ins = 0, opens = 0;
    for (int w = warp; w < words; w += NW) {
      const int i = 32 * w + lane;
      const bool kept = i < nb && (i < c0 || i >= c1), in = known && want > 0 && i >= c0 && i < c1 && sc[i] > most;
      opens += __popc(__ballot_sync(FULL, undecided(i)));
      const unsigned in_bits = __ballot_sync(FULL, in), kept_bits = __ballot_sync(FULL, kept);
      ins += __popc(in_bits);
      if (lane == 0) s_bits[w] = in_bits | kept_bits;
    }
    if (lane == 0) {
      atomicAdd(&s_over[0], ins);
      atomicAdd(&s_open[0], opens);
    }
    __syncthreads();
    const int places = want - s_over[0];
    const bool score_again = places < s_open[0] && !(known && off == 0.f);  // with a bound of 0 every score is 0
    unsigned long long key_at = 0, mask = 0;
    int left = places;
    if (score_again) {
      sum_heads(threadIdx.x, T);
      for (int shift = 56; shift >= 0; shift -= 8) {
        clear();
        for (int w = warp; w < words; w += NW)
          for (unsigned todo = __ballot_sync(FULL, undecided(32 * w + lane)); todo != 0; todo &= todo - 1) {
            const unsigned long long key = exact(32 * w + __ffs(todo) - 1);
            if (lane == 0 && ((key ^ key_at) & mask) == 0) atomicAdd(&hist[key >> shift & 255], 1);
          }
        digit(left);
        key_at |= static_cast<unsigned long long>(s_digit) << shift;
        mask |= 255ull << shift;
        left -= s_above;
      }
    }
    for (int w = warp; w < words; w += NW) {
      const unsigned todo = __ballot_sync(FULL, undecided(32 * w + lane));
      unsigned above = 0, tie = todo;
      if (score_again) {
        tie = 0;
        for (unsigned x = todo; x != 0; x &= x - 1) {
          const unsigned long long key = exact(32 * w + __ffs(x) - 1);
          if (key > key_at) above |= x & -x;
          else if (key == key_at) tie |= x & -x;
        }
      }
      if (lane == 0) {
        s_bits[w] |= above;
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

  // ---- in ascending order: every warp counts, and writes its words
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += 32) {
    const unsigned bits = w0 + lane < words ? s_bits[w0 + lane] : 0u;
    int upto = __popc(bits);
    const int own = upto;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(FULL, upto, o);
      if (lane >= o) upto += x;
    }
    for (int j = warp; j < 32; j += NW) {
      const unsigned word = __shfl_sync(FULL, bits, j);
      const int place = base + __shfl_sync(FULL, upto - own, j) + __popc(word & ((1u << lane) - 1));
      if (word >> lane & 1 && place < K) out[place] = 32 * (w0 + j) + lane;
    }
    base += __shfl_sync(FULL, upto, 31);
  }
}

template <int D, int T>
cudaError_t select(const SelectBlocksParams& p, const Scratch& ws, cudaStream_t stream) {
  const int cached = p.max_blocks <= CACHED ? p.max_blocks : 0;
  const int bits = (2 * ((p.max_blocks + 31) / 32) + cached) * 4;
  const cudaError_t e = cudaFuncSetAttribute(select_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, bits);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(p.T) * p.Hkv));
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = bits;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<D, T>, p, ws, cached);
}

template <int D>
cudaError_t score_few(const SelectBlocksParams& p, const Scratch& ws, cudaStream_t stream) {
  using C = FewCfg<D>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int warps = C::warps(p.max_q), smem = warps * C::warp_bytes(p.max_q);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(score_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  score_few_kernel<D><<<sms, warps * 32, smem, stream>>>(p, ws);
  return cudaGetLastError();
}

template <int D, int CG>
cudaError_t score_rows(const SelectBlocksParams& p, const Scratch& ws, cudaStream_t stream) {
  const int row_tiles = (p.max_q + 4 * CG - 1) / (4 * CG);
  const int64_t pairs = static_cast<int64_t>(p.N) * p.Hkv * row_tiles;
  const int64_t all = (p.max_blocks + SCORE_WARPS * 16 - 1) / (SCORE_WARPS * 16), most = (SCORE_CTAS + pairs - 1) / pairs;
  const int chunks = static_cast<int>(all < most ? all : most);
  const int smem = CG * (2 * D / 32) * 512;
  const cudaError_t e = cudaFuncSetAttribute(score_kernel<D, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  score_kernel<D, CG><<<static_cast<unsigned>(pairs * chunks), SCORE_WARPS * 32, smem, stream>>>(p, ws, row_tiles, chunks);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(const SelectBlocksParams& p, Scratch& ws, cudaStream_t stream) {
  // the two roundings of Q+-, the sums over heads, and 2 d / 16 products of 16 terms with their final addition
  ws.eps = 1.f / (1 << 18) + static_cast<float>(p.Hq / p.Hkv) / (1 << 24) + static_cast<float>(D / 8 + 2) / (1 << 22);
  const cudaError_t e = p.max_q <= 4 ? score_few<D>(p, ws, stream) : score_rows<D, TILE_ROWS / 4>(p, ws, stream);
  if (e != cudaSuccess) return e;
  // few rows leave the latency of one to be shortened; many, the CTAs an SM holds
  const bool many = static_cast<int64_t>(p.T) * p.Hkv >= FEW_ROWS;
  return many || p.max_blocks <= NARROW ? select<D, 128>(p, ws, stream) : select<D, 512>(p, ws, stream);
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
  if (p.d == 64) return launch<64>(p, ws, stream);
  if (p.d == 128) return launch<128>(p, ws, stream);
  if (p.d == 256) return launch<256>(p, ws, stream);
  return cudaErrorInvalidValue;
}

cudaError_t select_blocks_status(uint32_t* out, bool clear) { return read_status(g_select_blocks_status, out, clear); }

}  // namespace attn
