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
// Scores: bounds are the left operand, Q+- enter as two bf16 numbers each (16 bits).  Up to FEW rows a sequence (a decode
// step) are bound by reading the bounds: score_few_kernel.  More (a prompt's chunk) by the products: score_many_kernel,
// 128 blocks by 64 rows a tcgen05 tile.  Either way
//   |score - exact| <= eps ||Q|| ||b||,  b = (lo, hi) of a block, by Cauchy and Schwarz on the sum of |terms| (score_error).
// Pick: a CTA, or where there are many a warp, puts the scores of its row and head into bins over their range, gathers
// the few in and about the bin that holds the border, and a warp settles the border among them.  Few short sequences of
// one row each take one launch, a CTA scoring and picking: select_one_kernel.  Pages whose bounds are no finite numbers, or
// far above the others', would make the bound too wide for the rest: they are scored in 64 bits and take part (tame).
//
// Measured (GB300, calls in a captured graph, copy rate 6796 GB/s): 64 rows over 512 to 8192 tokens, 32/8 heads, d = 128,
// 27.9 us, of which the scores take 17.5 (72 MB of bounds: 10.6 at the copy rate) and the pick's chain of dependent steps
// the rest; 8 rows over 6335 to 122863 tokens, 16/2 heads, d = 256, 29.5 (9.8), of which the scores 16.3; 512 rows of one
// sequence of 32768, 32/8 heads, 43.6, of which the scores 20.4 (4096 rows of 2048: 33 MB written) and the pick 23.
// One page of NaN beside the others: 129 us instead of 43 for the latter, 52 instead of 25 for 64 rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "decode_shares.cuh"
#include "sm103.cuh"
#include "step.h"

namespace attn {

__device__ uint32_t g_select_blocks_status;

#ifdef ATTN_TEST_DROP_COPY
// Test-only builds (never the product library): the first CTA of score_many_kernel leaves out its first row tile.  The
// waits for it run out after ATTN_WAIT_LIMIT_NS.
__device__ int g_test_drop_copy_select;
#endif

namespace {

using shares::mma_16816;
using shares::sequence_of;

constexpr uint32_t FULL = 0xffffffffu;
constexpr int PAGE = 16;
constexpr int FEW = 4;             // rows a sequence up to which score_few_kernel takes them
constexpr int BINS = 512;          // of a window of scores
constexpr int CACHED_BLOCKS = 12288;  // scores of a row that shared memory holds
constexpr int64_t WARP_ROWS = 1024;   // rows times heads from which on a warp takes each, if its registers hold the scores
constexpr int NARROW = 1024;       // columns of a block table up to which 128 threads take a row
constexpr int ONE_BLOCKS = 4096;   // columns up to which select_one_kernel may be taken
// Norms below this count as this: squares of smaller numbers may vanish, and a bound that is too large does no harm
constexpr float LEAST_NORM = 1e-14f;
// Squared norms of a block from here on count as infinite, so that no finite norm makes a score overflow
constexpr float MOST_SQUARES = 1e36f;
constexpr int64_t SCORE_CTAS = 152 * 4;  // of the grid, about: a block table may be far wider than its sequences

struct Scratch {
  float* scores;  // [T][Hkv][stride]
  float* q_norm;  // [T][Hkv]
  float* b_norm;  // [N][Hkv][tiles]: a bound of the largest norm among those of 16 blocks that compete
  uint8_t* images;  // [row tiles][Hkv]: the queries' sums, where a sequence has more than FEW rows
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
// whether block i of nb competes: the first and the last ones are chosen, whatever their scores
__device__ __forceinline__ bool competes(const SelectBlocksParams& p, int i, int nb) {
  return static_cast<unsigned>(i - p.first) < static_cast<unsigned>(nb - p.last - p.first);
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

// Adds a pair to its negative and positive sums; a NaN stays one in both
__device__ __forceinline__ void add_parts(uint32_t w, float* neg, float* pos) {
  const float2 y = pair_of(w);
  neg[0] += y.x > 0.f ? 0.f : y.x;
  pos[0] += y.x < 0.f ? 0.f : y.x;
  neg[1] += y.y > 0.f ? 0.f : y.y;
  pos[1] += y.y < 0.f ? 0.f : y.y;
}
// A row's norm, from the lanes' sums of squares and whether any of its numbers is not 0
__device__ __forceinline__ void write_norm(float* to, float squares, uint32_t any, int lane) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) squares += __shfl_xor_sync(FULL, squares, off);
  any = __reduce_or_sync(FULL, any);
  // (a NaN passes the comparison)
  if (lane == 0) *to = any == 0 ? 0.f : squares < LEAST_NORM * LEAST_NORM ? LEAST_NORM : sqrtf(squares);
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
  static constexpr int warps(int rows) {
    const int fit = 222 * 1024 / warp_bytes(rows);
    return fit < MOST_WARPS ? fit : MOST_WARPS;
  }
  static constexpr int most_bytes() {  // of a CTA, whatever the number of rows
    int most = 0;
    for (int rows = 1; rows <= FEW; ++rows) most = most > warps(rows) * warp_bytes(rows) ? most : warps(rows) * warp_bytes(rows);
    return most;
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
            for (int x = 0; x < D / 64; ++x) add_parts(heads[e][x], neg + 2 * x, pos + 2 * x);
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
        if (at.tile == 0) write_norm(ws.q_norm + static_cast<int64_t>(r0 + row) * Hkv + at.h, squares, any, lane);
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
      if (!(norm[e] < MOST_SQUARES)) norm[e] = INFINITY;  // NaN too
      if (competes(p, blk + 8 * e, at.nb)) most = max(most, __float_as_uint(norm[e]));
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

// ---- more rows: the tensor cores take 128 blocks by RT rows at a time
// What shared memory holds, in us: d = 128, 32 sequences of 4000 tokens with 64 rows, 8 KV heads, 36.2 with one CTA an SM and
// two tiles of 64 rows in flight, 28.9 with two CTAs and one tile of 32 (SMALL); a sequence of 65536 with 2048 rows 113 and
// 152.  d = 64, 64 rows either way: 26.2 with one CTA, 17.8 with two; 111 and 80.
template <int D, bool SMALL>
struct ManyCfg {
  static_assert(!SMALL || D == 128, "the others have one form");
  static constexpr int RT = D == 256 || SMALL ? 32 : 64;         // rows of a tile
  static constexpr int STAGES = D == 128 && !SMALL ? 2 : 1;      // row tiles in flight
  static constexpr int CTAS = D == 64 || SMALL ? 2 : 1;          // an SM
  static constexpr int PANELS = 2 * D / 64;         // 128-byte columns of the 2 d terms
  static constexpr int A_PANEL = 128 * 128, B_PANEL = RT * 128;
  static constexpr int A_BYTES = PANELS * A_PANEL;
  static constexpr int B_BYTES = 2 * PANELS * B_PANEL;  // a row tile: Q- and Q+, first and second bf16 parts
  static constexpr int B_OFF = A_BYTES;
  static constexpr int OUT_OFF = B_OFF + STAGES * B_BYTES;  // a tile's scores, [RT][128]
  static constexpr int SMEM = OUT_OFF + RT * 128 * 4;
  static constexpr uint32_t TMEM_COLS = 2 * RT;     // two accumulators
  static constexpr int EPILOGUE = 4, LOADER = 4, ISSUER = 5, WARPS = 6;
};
constexpr int SMALL_ROWS = 128;  // rows a sequence up to which the SMALL form may be taken
constexpr int SUM_ROWS = 16;  // rows a CTA of the kernel that sums the heads takes

// Place of row tile i of a sequence whose first row is `first`, among all tiles' images: no two share one
__host__ __device__ constexpr int64_t tile_place(int64_t first, int64_t n, int64_t i, int RT) { return first / RT + n + i; }

// Q-, Q+ of a row and KV head, each as two bf16 numbers, into the image of its row tile: [part][panel][row][128 bytes],
// as the tensor core reads it from shared memory (16-byte pieces exchanged within 128 bytes, by the row)
template <int D, bool SMALL>
__global__ void __launch_bounds__(SUM_ROWS / 2 * 32) sum_heads_kernel(const SelectBlocksParams p, const Scratch ws, int row_tiles) {
  using C = ManyCfg<D, SMALL>;
  const int rt = blockIdx.x % row_tiles, nh = blockIdx.x / row_tiles, n = nh / p.Hkv, h = nh % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.Hq / p.Hkv;
  // score_many_kernel gathers bounds meanwhile, and waits before it takes the images
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Span s = span_of(p, n, rt == 0 && h == 0 && threadIdx.x == 0);
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const int at = rt * SUM_ROWS + 2 * warp + e, row = s.first + at;  // at: within the sequence
    if (row >= s.end) return;
    const uint32_t* from = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(row) * p.Hq + h * G) * D) + lane;
    float neg[D / 32] = {}, pos[D / 32] = {};  // of channels 2 lane + 64 x and the next
    for (int e0 = 0; e0 < G; e0 += 4) {        // four heads' loads in flight
      uint32_t w[4][D / 64];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int x = 0; x < D / 64; ++x) w[k][x] = e0 + k < G ? from[(e0 + k) * (D / 2) + 32 * x] : 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int x = 0; x < D / 64; ++x) add_parts(w[k][x], neg + 2 * x, pos + 2 * x);
    }
    uint8_t* image = ws.images + (tile_place(s.first, n, at / C::RT, C::RT) * p.Hkv + h) * C::B_BYTES;
    float squares = 0.f;
    uint32_t any = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        const float a = half ? pos[2 * x] : neg[2 * x], b = half ? pos[2 * x + 1] : neg[2 * x + 1];
        const uint32_t hi = pack_bf16x2(a, b);
        const float2 z = pair_of(hi);
        const int word = half * (D / 2) + 32 * x + lane, r = at % C::RT;
        uint8_t* to = image + word / 32 * C::B_PANEL + r * 128 + ((word % 32 / 4) ^ (r & 7)) * 16 + word % 4 * 4;
        *reinterpret_cast<uint32_t*>(to) = hi;
        *reinterpret_cast<uint32_t*>(to + C::PANELS * C::B_PANEL) = pack_bf16x2(a - z.x, b - z.y);
        squares = fmaf(a, a, fmaf(b, b, squares));
        any |= hi & 0x7fff7fffu;
      }
    write_norm(ws.q_norm + static_cast<int64_t>(row) * p.Hkv + h, squares, any, lane);
  }
}

// A CTA takes every `chunks`-th tile of 128 blocks of a sequence and KV head: its bounds are gathered through the block
// table once and multiplied with one row tile after another, which arrive in bulk copies.  Where there are few tiles of
// blocks, `splits` CTAs take each, and every splits-th row tile.
template <int D, bool SMALL>
__global__ void __launch_bounds__(ManyCfg<D, SMALL>::WARPS * 32, ManyCfg<D, SMALL>::CTAS)
    score_many_kernel(const SelectBlocksParams p, const Scratch ws, int chunks, int splits) {
  using C = ManyCfg<D, SMALL>;
  constexpr int RT = C::RT, STAGES = C::STAGES, THREADS = C::WARPS * 32;
  extern __shared__ __align__(1024) uint8_t tiles[];
  __shared__ uint64_t bars[2 * STAGES + 2 * 2 + 1];
  __shared__ uint32_t s_tmem;
  __shared__ int s_page[128];
  uint64_t* b_full = bars;              // [STAGES]
  uint64_t* b_empty = b_full + STAGES;  // [STAGES]
  uint64_t* d_full = b_empty + STAGES;  // [2]: a row tile's products are done
  uint64_t* d_empty = d_full + 2;       // [2]: its scores have been read
  uint64_t* all_done = d_empty + 2;
  const int warp = __shfl_sync(FULL, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int split = blockIdx.x % splits, part = blockIdx.x / splits;
  const int chunk = part % chunks, nh = part / chunks, n = nh / p.Hkv, h = nh % p.Hkv;
  const Span s = span_of(p, n, false);
  const int rows = s.end - s.first, nb = rows > 0 ? blocks_seen(s, s.end - 1) : 0;
  const bool misaligned = (smem_u32(tiles) & 1023u) != 0;  // swizzled tiles need 1 KB alignment
  if (misaligned && threadIdx.x == 0) set_error(&g_select_blocks_status, kDevMisaligned);
  if (nb <= p.K || chunk * 128 >= nb || misaligned) {  // every block is chosen, or none is this CTA's
    asm volatile("griddepcontrol.wait;" ::: "memory");  // no CTA, and so not this kernel, ends before the one ahead of it
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], C::EPILOGUE);
    }
    mbar_init(all_done, 1);
    fence_mbar_init();
  }
  if (warp == C::ISSUER) {
    tmem_alloc(&s_tmem, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(FULL, s_tmem, 0);
  auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(FULL, mbar_wait(bar, parity)) != 0; };

  const int row_tiles = (rows + RT - 1) / RT;
  bool ok = true;
  int done = 0;    // row tiles so far, over all tiles of blocks
  int issued = 0;  // of them, those that the loading warp has asked for
  for (int tile = chunk; tile * 128 < nb; tile += chunks) {
    // ---- the bounds of 128 blocks, of page 0 where there is none
    if (threadIdx.x < 128) {
      const int blk = tile * 128 + threadIdx.x;
      int id = blk < nb ? p.block_table[static_cast<int64_t>(n) * p.max_blocks + blk] : 0;
      if (id < 0 || id >= p.num_blocks) {
        set_error(&g_select_blocks_status, kDevBadPage);
        id = 0;
      }
      s_page[threadIdx.x] = id;
    }
    __syncthreads();
#pragma unroll 8
    for (int i = threadIdx.x; i < 128 * (D / 4); i += THREADS) {
      const int r = i / (D / 4), piece = i % (D / 4);
      const __nv_bfloat16* from = p.bounds + (static_cast<int64_t>(s_page[r]) * p.Hkv + h) * 2 * D + piece * 8;
      const uint32_t to = smem_u32(tiles) + piece / 8 * C::A_PANEL + r * 128 + ((piece % 8) ^ (r & 7)) * 16;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the images are there
    // rows see more blocks the later they are: the first row tile with something to score here
    const int least = tile * 128 > p.K ? tile * 128 : p.K;
    int first = 0;
    while (blocks_seen(s, min(s.first + (first + 1) * RT, s.end) - 1) <= least) ++first;
    // every splits-th of them, the first one for this CTA
    const int mine = first + split, count = row_tiles > mine ? (row_tiles - mine + splits - 1) / splits : 0;

    if (warp == C::LOADER) {
      for (int i = 0; i < count && ok; ++i) {
        const int stage = (done + i) % STAGES;
        ok = wait(&b_empty[stage], ((done + i) / STAGES & 1) ^ 1);
        if (!ok) break;
        const int rt = mine + i * splits, left = rows - rt * RT;
        // eight rows at a time, as the exchange of pieces goes; what lies behind the last row is not looked at
        const uint32_t bytes = (left < RT ? (left + 7) / 8 * 8 : RT) * 128;
        if (lane == 0) mbar_arrive_expect_tx(&b_full[stage], 2 * C::PANELS * bytes);
        __syncwarp();
        const uint8_t* image = ws.images + (tile_place(s.first, n, rt, RT) * p.Hkv + h) * C::B_BYTES;
#ifdef ATTN_TEST_DROP_COPY
        if (blockIdx.x == 0 && done + i == 0 && g_test_drop_copy_select != 0) continue;
#endif
        if (lane < 2 * C::PANELS)
          bulk_load(tiles + C::B_OFF + stage * C::B_BYTES + lane * C::B_PANEL, image + lane * C::B_PANEL, bytes, &b_full[stage]);
        __syncwarp();
        issued = done + i + 1;
      }
    } else if (warp == C::ISSUER) {
      constexpr uint32_t IDESC = idesc_bf16_f32(128, RT, 0);  // bounds (K-major) x queries (K-major)
      for (int i = 0; i < count && ok; ++i) {
        const int stage = (done + i) % STAGES, buf = (done + i) & 1;
        ok = wait(&b_full[stage], (done + i) / STAGES & 1) && wait(&d_empty[buf], ((done + i) / 2 & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = smem_u32(tiles), b = smem_u32(tiles + C::B_OFF + stage * C::B_BYTES);
        // the second parts of Q first: their sum is small, and so is what the products round off it
#pragma unroll
        for (int part = 1; part >= 0; --part)
#pragma unroll
          for (int k = 0; k < 2 * D / 16; ++k)
            umma_ss_warp(tmem + buf * RT, smem_desc_sw128(a + (k >> 2) * C::A_PANEL + (k & 3) * 32, 16, 1024),
                         smem_desc_sw128(b + (part * C::PANELS + (k >> 2)) * C::B_PANEL + (k & 3) * 32, 16, 1024), IDESC,
                         part == 0 || k > 0 ? 1u : 0u);
        umma_commit_warp(&d_full[buf]);
        umma_commit_warp(&b_empty[stage]);
      }
    } else {
      // ---- norms of the blocks, a thread a block, then its scores of one row after another
      const int r = threadIdx.x, blk = tile * 128 + r;
      float norm = 0.f;
#pragma unroll 1
      for (int panel = 0; panel < C::PANELS; ++panel) {
        uint32_t sum[2] = {0u, 0u};
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(tiles + panel * C::A_PANEL + r * 128 + (c ^ (r & 7)) * 16);
          sum[0] = add_squares(x.x, sum[0]); sum[1] = add_squares(x.y, sum[1]);
          sum[0] = add_squares(x.z, sum[0]); sum[1] = add_squares(x.w, sum[1]);
        }
        const float2 y = pair_of(sum[0]), z = pair_of(sum[1]);
        norm += (y.x + y.y) + (z.x + z.y);
      }
      if (!(norm < MOST_SQUARES)) norm = INFINITY;  // NaN too
      uint32_t most = competes(p, blk, nb) ? __float_as_uint(norm) : 0u;
      for (int off = 8; off > 0; off >>= 1) most = max(most, __shfl_xor_sync(FULL, most, off));
      // the sum of squares may have been an eighth too small
      if (lane % 16 == 0 && blk < nb)
        ws.b_norm[static_cast<int64_t>(nh) * ws.tiles + blk / 16] = fmaxf(1.1f * sqrtf(__uint_as_float(most)), LEAST_NORM);
      // A thread has a block's scores in TMEM, a row of scores lies in one piece: through shared memory, and on in bulk
      // copies (stored by the threads themselves they took 5500 cycles a tile, three times the products).
      float* staging = reinterpret_cast<float*>(tiles + C::OUT_OFF);
      const int held = ws.stride - tile * 128 < 128 ? static_cast<int>(ws.stride) - tile * 128 : 128;  // a multiple of 8
      for (int i = 0; i < count; ++i) {
        const int buf = (done + i) & 1, row = (mine + i * splits) * RT + r;  // whose scores this thread sends off
        if (ok) ok = wait(&d_full[buf], (done + i) / 2 & 1);         // after a wait that ran out: none, all the same steps
        tc_fence_after();
        tma_store_wait_read0();
        named_barrier_sync(1, C::EPILOGUE * 32);
#pragma unroll
        for (int c = 0; c < RT; c += 32) {
          uint32_t x[32];
          tmem_ld32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + buf * RT + c, x);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) staging[(c + k) * 128 + r] = __uint_as_float(x[k]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_empty[buf]);
        fence_proxy_async_smem();
        named_barrier_sync(1, C::EPILOGUE * 32);
        if (r < RT && row < rows)
          bulk_store(ws.scores + (static_cast<int64_t>(s.first + row) * p.Hkv + h) * ws.stride + tile * 128,
                     staging + r * 128, held * 4);
        tma_store_commit();
      }
    }
    done += count;
    // the products that read these bounds are done where their scores have been read
    ok = __syncthreads_and(ok);
    if (!ok) break;
  }
  // nothing is on its way to this CTA's memory when it leaves, also after a wait that ran out
  if (warp == C::ISSUER) {
    umma_commit_warp(all_done);
    ok = wait(all_done, 0) && ok;
  }
  if (warp == C::LOADER)
    for (int k = issued > STAGES ? issued - STAGES : 0; k < issued; ++k) ok = wait(&b_full[k % STAGES], k / STAGES & 1) && ok;
  if (!ok && lane == 0) set_error(&g_select_blocks_status, kDevWaitTimeout);
  tma_store_wait0();
  tc_fence_before();
  __syncthreads();
  if (warp == C::ISSUER) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
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

// Words of shared memory before the scores: two bits a block, in whole 16 bytes
__host__ __device__ constexpr int cache_at(int max_blocks) { return (2 * ((max_blocks + 31) / 32) + 3) / 4 * 4; }
// Bytes of it that picking takes, with the scores or without
constexpr int pick_bytes(int max_blocks, bool cached) {
  return (cache_at(max_blocks) + (cached ? (max_blocks + 31) / 32 * 32 : 0)) * 4;
}

// Every block that a row sees, and -1 behind
template <int T>
__device__ __forceinline__ void choose_all(const SelectBlocksParams& p, int64_t at, int nb) {
  for (int i = threadIdx.x % T; i < p.K; i += T) p.blocks[at * p.K + i] = i < nb ? i : -1;
}

struct PickShared {
  union {
    __align__(16) int hist[2][BINS];
    double q[2 * 256];  // the sums over heads, once the bins are done with
  };
  int digits[256];
  unsigned long long key[32];
  uint4 red[32];
  float score[32];
  int at[32], open[2], over[2], digit, above;
  unsigned among;
};

// What picking needs of a row and KV head
struct Row {
  int r, h, n, nb;     // row, KV head, sequence; the blocks that it sees, more than it may choose
  float* scores;       // in global memory, rows of whole multiples of eight floats; null: in shared memory already
  const float* norms;  // of tiles of 16 blocks: infinite where the tile is wild
  float q_norm, b_norm;  // b_norm: this thread's share of the maximum of the others
  bool wild;             // this thread's share of whether there are wild ones
};
// A tile's norm counts
__device__ __forceinline__ void count_norm(Row& row, float norm) {
  if (norm < INFINITY) row.b_norm = fmaxf(row.b_norm, norm);
  else row.wild = true;
}
// ||Q|| as the bound takes it: not 0 beside wild tiles, whose scores may be anything all the same
__device__ __forceinline__ float norm_of_q(const Row& row, bool wild) {
  return wild && row.q_norm < LEAST_NORM ? LEAST_NORM : row.q_norm;
}

// All threads of a row: a warp of a CTA, or a CTA
template <int T>
__device__ __forceinline__ void sync_row() {
  if constexpr (T == 32) __syncwarp();
  else __syncthreads();
}

// Bit j of lane l goes to bit l of lane j
__device__ __forceinline__ unsigned transpose_32x32(unsigned w, int lane) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const unsigned keep = s == 16 ? 0xffffu : s == 8 ? 0xff00ffu : s == 4 ? 0xf0f0f0fu : s == 2 ? 0x33333333u : 0x55555555u;
    const unsigned y = __shfl_xor_sync(FULL, w, s);
    w = lane & s ? (w & ~keep) | (y >> s & keep) : (w & keep) | (y << s & ~keep);
  }
  return w;
}

// A bit for each number below n of a word's 32
__device__ __forceinline__ unsigned below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1; }

// Counts a score within [low, high]: 4 BINS - 1 steps, of which a bin takes four.  Adding 3 2^22 rounds a score's step to the
// nearest, and leaves it in the sum's last bits.
__device__ __forceinline__ void count_step(int* hist, float x, float low, float high, float per_step) {
  if (x >= low && x <= high) {
    const int step = __float_as_int(fmaf(x - low, per_step, 12582912.f));
    atomicAdd(&hist[(step & (4 * BINS - 1)) >> 2], 1);
  }
}
// The bin that holds the border, by a warp: lane 0 holds the highest
__device__ __forceinline__ int border_bin(const int* hist, int over, int want, int lane) {
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
  return __reduce_max_sync(FULL, bin);
}
// [low, high] becomes a bin of it, and what is within the twofold error (and a rounding of the bin's ends, 2^-6 of a bin)
__device__ __forceinline__ void narrow(int bin, float range, float off, float& low, float& high) {
  const float step = range / (4 * BINS - 1), slack = 2.f * off + step * (1.f / 16);
  low = low + (4 * bin - 0.5f) * step - slack;
  high = low + 4.f * step + 2.f * slack;
}

// The window's blocks, a lane each: those that are sure of one of `places`, and those close to the border
struct Border {
  int block, rest;     // this lane's; places that the sure ones leave
  bool sure, close;
  unsigned among;      // the close ones' lanes; 0 where they all have a place
};
__device__ __forceinline__ Border settle(const PickShared& sh, int open, int places, float off, int lane) {
  Border b;
  const bool mine = lane < open;
  const float x = mine ? sh.score[lane] : -INFINITY;
  b.block = mine ? sh.at[lane] : 0x7fffffff;
  int rank = 0;
  for (int j = 0; j < open; ++j) {
    const float y = __shfl_sync(FULL, x, j);
    const int k = __shfl_sync(FULL, b.block, j);
    rank += y > x || (y == x && k < b.block) ? 1 : 0;
  }
  const float border = __shfl_sync(FULL, x, __ffs(__ballot_sync(FULL, mine && rank == places - 1)) - 1);
  b.sure = mine && x > border + 2.f * off;
  b.close = mine && !b.sure && x >= border - 2.f * off;
  b.among = __ballot_sync(FULL, b.close);
  b.rest = places - __popc(__ballot_sync(FULL, b.sure));
  if (__popc(b.among) == b.rest) b.among = 0;
  return b;
}
// Whether this lane's block has a place, by the close ones' exact scores
__device__ __forceinline__ bool takes(const Border& b, unsigned long long key) {
  int before = 0;  // that go before this one
  for (unsigned todo = b.among; todo != 0; todo &= todo - 1) {
    const int j = __ffs(todo) - 1;
    const unsigned long long y = __shfl_sync(FULL, key, j);
    const int k = __shfl_sync(FULL, b.block, j);
    before += y > key || (y == key && k < b.block) ? 1 : 0;
  }
  return b.sure || (b.close && before < b.rest);
}

// hi + lo += x, with what the sum drops
__device__ __forceinline__ void add_exactly(float& hi, float& lo, float x) {
  const float s = hi + x, b = s - hi;
  lo += (hi - (s - b)) + (x - b);
  hi = s;
}

// The close blocks' scores to 40 bits, as sums of two floats (Dekker's and Knuth's exact sums and products): 64-bit arithmetic
// has a sixtieth of the rate here, and a warp that settled its row's border by it took 10 to 20 us.  What remains close is
// left to it.  By a warp: lane l has words 32 k + l of a block's bounds, of which D / 32 there are; norms: ||Q|| times the
// largest ||b||.  The loads go ahead of the sums: table entries, then the queries, four heads at a time, and the first
// block's bounds.
__device__ __forceinline__ void refine(const SelectBlocksParams& p, const Row& row, float norms, Border& at, int lane) {
  const int D = p.d, G = p.Hq / p.Hkv;
  int id = 0;
  if (at.close) id = p.block_table[static_cast<int64_t>(row.n) * p.max_blocks + at.block];
  if (id < 0 || id >= p.num_blocks) id = 0;
  uint32_t lo[4], hi[4];  // of channels 2 (32 x + lane) and the next
  auto load_bounds = [&](int lane_of) {
    const int64_t page = __shfl_sync(FULL, id, lane_of);
    const uint32_t* from = reinterpret_cast<const uint32_t*>(p.bounds + (page * p.Hkv + row.h) * 2 * D) + lane;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      lo[x] = 64 * x < D ? from[32 * x] : 0u;
      hi[x] = 64 * x < D ? from[D / 2 + 32 * x] : 0u;
    }
  };
  const uint32_t* heads = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(row.r) * p.Hq + row.h * G) * D) + lane;
  float neg[4][2][2] = {}, pos[4][2][2] = {};  // sums over heads: [x][channel][first and second float]
  for (int e0 = 0; e0 < G; e0 += 4) {
    uint32_t y[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int x = 0; x < 4; ++x) y[e][x] = e0 + e < G && 64 * x < D ? heads[(e0 + e) * (D / 2) + 32 * x] : 0u;
    if (e0 == 0) load_bounds(__ffs(at.among) - 1);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (64 * x >= D) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 z = pair_of(y[e][x]);
        add_exactly(neg[x][0][0], neg[x][0][1], fminf(z.x, 0.f));
        add_exactly(neg[x][1][0], neg[x][1][1], fminf(z.y, 0.f));
        add_exactly(pos[x][0][0], pos[x][0][1], fmaxf(z.x, 0.f));
        add_exactly(pos[x][1][0], pos[x][1][1], fmaxf(z.y, 0.f));
      }
    }
  }
  float s = 0.f, t = 0.f;  // this lane's block's score
  for (unsigned todo = at.among; todo != 0;) {
    const int j = __ffs(todo) - 1;
    todo &= todo - 1;
    float a = 0.f, b = 0.f;
    auto add = [&](const float (&q)[2], float k) {
      const float product = q[0] * k;
      b += fmaf(q[1], k, fmaf(q[0], k, -product));
      add_exactly(a, b, product);
    };
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (64 * x >= D) continue;
      const float2 l = pair_of(lo[x]), h = pair_of(hi[x]);
      add(neg[x][0], l.x);
      add(neg[x][1], l.y);
      add(pos[x][0], h.x);
      add(pos[x][1], h.y);
    }
    if (todo != 0) load_bounds(__ffs(todo) - 1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float other = __shfl_xor_sync(FULL, a, o);
      b += __shfl_xor_sync(FULL, b, o);
      add_exactly(a, b, other);
    }
    if (lane == j) {
      s = a + b;
      t = b - (s - a);
    }
  }
  // ordered by the first float, then by the second: the first is the sum rounded
  const unsigned long long key = static_cast<unsigned long long>(order_of(s)) << 32 | order_of(t);
  int before = 0;
  for (unsigned todo = at.among; todo != 0; todo &= todo - 1) {
    const int j = __ffs(todo) - 1;
    const unsigned long long y = __shfl_sync(FULL, key, j);
    const int k = __shfl_sync(FULL, at.block, j);
    before += y > key || (y == key && k < at.block) ? 1 : 0;
  }
  const int border = __ffs(__ballot_sync(FULL, at.close && before == at.rest - 1)) - 1;
  const float above = (s - __shfl_sync(FULL, s, border)) + (t - __shfl_sync(FULL, t, border));
  // In units of 2^-24 of 2^-24 of the terms' sum: errors of at most 23 of 2^-24 (16 sums a lane, 5 across lanes, products) are
  // added up in 42 additions, 966; the products with the queries' second floats, 2; those floats of G heads, G^2 / 2
  const float off = norms * (1.f / (1ull << 38) + static_cast<float>(G) * static_cast<float>(G) / (1ull << 48));
  const bool sure = at.close && above > 2.f * off, close = at.close && !sure && above >= -2.f * off;
  at.sure = at.sure || sure;
  at.close = close;
  at.among = __ballot_sync(FULL, close);
  at.rest -= __popc(__ballot_sync(FULL, sure));
  if (__popc(at.among) == at.rest) at.among = 0;
}

// The close blocks' scores in 64 bits, this lane's block's; of pages that are alike, mostly
__device__ __noinline__ unsigned long long exact_keys(const SelectBlocksParams& p, int r, int h, int n, int block, unsigned among,
                                                      int lane) {
  const int D = p.d, G = p.Hq / p.Hkv;
  const uint32_t* heads = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(r) * p.Hq + h * G) * D);
  unsigned long long key = 0;
  for (unsigned todo = among; todo != 0; todo &= todo - 1) {
    const int j = __ffs(todo) - 1;
    int id = p.block_table[static_cast<int64_t>(n) * p.max_blocks + __shfl_sync(FULL, block, j)];
    if (id < 0 || id >= p.num_blocks) id = 0;
    const uint32_t* from = reinterpret_cast<const uint32_t*>(p.bounds + (static_cast<int64_t>(id) * p.Hkv + h) * 2 * D);
    double sum = 0.0;
    for (int w = lane; w < D; w += 32) {  // terms 2 w and 2 w + 1 of the 2 d
      const bool low = 2 * w < D;
      double q[2] = {0.0, 0.0};
      for (int g = 0; g < G; ++g) {
        const float2 z = pair_of(heads[g * (D / 2) + (low ? w : w - D / 2)]);
        q[0] += low ? fminf(z.x, 0.f) : fmaxf(z.x, 0.f);
        q[1] += low ? fminf(z.y, 0.f) : fmaxf(z.y, 0.f);
      }
      const float2 k = pair_of(from[w]);
      sum = fma(q[0], static_cast<double>(k.x), fma(q[1], static_cast<double>(k.y), sum));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    if (lane == j) key = order_of(sum);
  }
  return key;
}

// The sums over heads in 64 bits, [2 d], channels begin, begin + step, ..
__device__ __forceinline__ void sum_heads(const SelectBlocksParams& p, const Row& row, double* sums, int begin, int step) {
  const int D = p.d, G = p.Hq / p.Hkv;
  for (int c = begin; c < D; c += step) {
    const __nv_bfloat16* q = p.q + (static_cast<int64_t>(row.r) * p.Hq + row.h * G) * D + c;
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
    sums[c] = neg;
    sums[D + c] = pos;
  }
}
// Block i's bounds, words 32 k + lane
__device__ __forceinline__ void load_bounds(const SelectBlocksParams& p, const Row& row, int i, uint32_t (&b)[8], int lane) {
  int id = p.block_table[static_cast<int64_t>(row.n) * p.max_blocks + i];
  if (id < 0 || id >= p.num_blocks) id = 0;
  const uint32_t* from = reinterpret_cast<const uint32_t*>(p.bounds + (static_cast<int64_t>(id) * p.Hkv + row.h) * 2 * p.d) + lane;
#pragma unroll
  for (int k = 0; k < 8; ++k) b[k] = 32 * k < p.d ? from[32 * k] : 0u;
}
// Their product with the sums, by a warp: the block's score in 64 bits
__device__ __forceinline__ double product(const SelectBlocksParams& p, const double* sums, const uint32_t (&b)[8], int lane) {
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (32 * k >= p.d) break;
    const float2 x = pair_of(b[k]);
    const int c = 32 * k + lane;
    sum = fma(sums[2 * c], static_cast<double>(x.x), fma(sums[2 * c + 1], static_cast<double>(x.y), sum));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
  return sum;
}

// Wild tiles, those with a bound that is no finite number or too large (of a norm from `cut` on), would leave every score of
// the row unsure.  Their blocks whose norm is above `limit`, the largest one of the other tiles, are scored in 64 bits, and
// take part with that score as a float, cut to what is above or below all others': `most`, twice ||Q|| times the limit.  That
// is off by less than the others' bound, keeps the order among wild blocks, and those that it makes equal are told apart by
// exact scores, like all that are close to the border.  By all threads of the row, between two barriers.
template <int T>
__device__ __noinline__ void tame(const SelectBlocksParams& p, int r, int h, int n, int nb, const float* norms, float cut,
                                  float limit, float most, double* sums, float* scores) {
  Row row;  // (a caller's would have to lie in memory)
  row.r = r;
  row.h = h;
  row.n = n;
  row.nb = nb;
  const int tid = T == 32 ? threadIdx.x & 31 : threadIdx.x, warp = tid >> 5, lane = tid & 31;
  sum_heads(p, row, sums, tid, T);
  sync_row<T>();
  for (int tile = warp; 16 * tile < nb; tile += T / 32) {
    if (norms[tile] < cut) continue;
    for (int i = 16 * tile; i < 16 * tile + 16; ++i) {
      if (!competes(p, i, nb)) continue;
      uint32_t b[8];
      load_bounds(p, row, i, b, lane);
      float squares = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 x = pair_of(b[k]);
        squares = fmaf(x.x, x.x, fmaf(x.y, x.y, squares));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) squares += __shfl_xor_sync(FULL, squares, o);
      if (sqrtf(squares) < 0.999f * limit) continue;  // as sure as the others' scores
      const double sum = product(p, sums, b, lane);
      if (lane == 0) scores[i] = sum < most ? (sum > -most ? static_cast<float>(sum) : -most) : most;  // a NaN is the highest
    }
  }
}

// Where too many blocks are unsure because a few tiles have norms far above the others' (16 times their geometric mean, at
// least), those are taken for wild ones.  Returns ||Q|| times the largest norm of the others, or 0 where there are none such.
// 512 rows of 2048 pages, 8 heads, of which one has bounds 10^4 times the others': 0.3 ms, by exact scores of all 14.4.
template <int T>
__device__ __noinline__ float leave_out(const SelectBlocksParams& p, int r, int h, int n, int nb, const float* norms, float q_norm,
                                        PickShared& sh, float* scores) {
  constexpr int NW = T / 32;
  const int tid = T == 32 ? threadIdx.x & 31 : threadIdx.x, warp = tid >> 5, lane = tid & 31, tiles = (nb + 15) / 16;
  auto reduce = [&](int a, int b, uint32_t most) {  // two sums and a maximum
    a = __reduce_add_sync(FULL, a);
    b = __reduce_add_sync(FULL, b);
    most = __reduce_max_sync(FULL, most);
    sync_row<T>();
    if (lane == 0) sh.red[warp] = make_uint4(a, b, most, 0);
    sync_row<T>();
    const uint4 x = lane < NW ? sh.red[lane] : make_uint4(0, 0, 0, 0);
    return make_int3(__reduce_add_sync(FULL, static_cast<int>(x.x)), __reduce_add_sync(FULL, static_cast<int>(x.y)),
                     static_cast<int>(__reduce_max_sync(FULL, x.z)));
  };
  int sum = 0, count = 0, large = 0;
  for (int i = tid; i < tiles; i += T)
    if (norms[i] > LEAST_NORM && norms[i] < INFINITY) {
      sum += static_cast<int>(__float_as_uint(norms[i]) >> 23);
      ++count;
    }
  const int3 all = reduce(sum, count, 0);
  if (all.y == 0) return 0.f;
  const float cut = __uint_as_float(static_cast<uint32_t>(min(all.x / all.y + 5, 254)) << 23);
  float most = LEAST_NORM;
  for (int i = tid; i < tiles; i += T) {
    if (norms[i] >= cut) large += norms[i] < INFINITY ? 1 : 0;
    else most = fmaxf(most, norms[i]);
  }
  const int3 rest = reduce(large, 0, __float_as_uint(most));
  if (rest.x == 0 || 16 * rest.x > tiles) return 0.f;
  most = __int_as_float(rest.z);
  const float bound = (q_norm < LEAST_NORM ? LEAST_NORM : q_norm) * most;
  tame<T>(p, r, h, n, nb, norms, cut, most, 2.f * bound, sh.q, scores);
  return bound;
}

// Picks the blocks of a row and KV head, by a CTA of T threads.  CACHED: shared memory holds its scores, else they are read
// again and again.  s_bits: [words] chosen blocks, [words] ties; the scores from word cache_at on.  EASY: false, and nothing
// done, where there is more to it than a few blocks about the border.
template <int T, bool CACHED, bool EASY>
__device__ __forceinline__ bool pick(const SelectBlocksParams& p, const Row& row, float eps, PickShared& sh, uint32_t* s_bits) {
  constexpr int NW = T / 32;
  const int nb = row.nb, K = p.K, r = row.r, h = row.h, n = row.n;
  const int tid = T == 32 ? threadIdx.x & 31 : threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* out = p.blocks + (static_cast<int64_t>(r) * p.Hkv + h) * K;
  const int c0 = p.first, c1 = nb - p.last;  // the blocks that compete
  const int want = K - p.first - p.last;     // for so many places: fewer than they are
  const int words = (nb + 31) / 32;
  uint32_t* ties = s_bits + words;
  for (int i = tid; i < BINS / 4; i += T) reinterpret_cast<int4*>(sh.hist[0])[i] = make_int4(0, 0, 0, 0);
  if (tid < 2) sh.open[tid] = sh.over[tid] = 0;

  // ---- how far a score may be off, and the scores' range
  float* sc = row.scores;
  float* cache = reinterpret_cast<float*>(s_bits + cache_at(p.max_blocks));
  const float none = __uint_as_float(0x7fffffffu);  // a NaN: neither above, below nor within a window
  auto competing = [&](int i) { return i >= c0 && i < c1; };
  auto score = [&](int i) {  // of a block that competes, else none
    if constexpr (CACHED) return cache[i];
    else return competing(i) ? sc[i] : none;
  };
  // four scores at a time, of blocks 4 v ..
  auto edge = [&](int v) { return 4 * v < c0 || 4 * v + 4 > c1; };
  auto read_four = [&](int v) {
    float4 x = *reinterpret_cast<const float4*>((CACHED && sc == nullptr ? cache : sc) + 4 * v);
    if (edge(v)) {
      x.x = competing(4 * v) ? x.x : none;
      x.y = competing(4 * v + 1) ? x.y : none;
      x.z = competing(4 * v + 2) ? x.z : none;
      x.w = competing(4 * v + 3) ? x.w : none;
    }
    return x;
  };
  auto four = [&](int v) {
    if constexpr (CACHED) return *reinterpret_cast<const float4*>(cache + 4 * v);
    else return read_four(v);
  };
  float low = INFINITY, high = -INFINITY, off;
  uint32_t most, wild;
  auto widen = [&](const float4& x) {
    low = fminf(fminf(low, fminf(x.x, x.y)), fminf(x.z, x.w));
    high = fmaxf(fmaxf(high, fmaxf(x.x, x.y)), fmaxf(x.z, x.w));
  };
  auto reduce = [&]() {
    most = __reduce_max_sync(FULL, __float_as_uint(row.b_norm));  // norms by their bits
    const uint32_t least = __reduce_min_sync(FULL, order_of(low)), top = __reduce_max_sync(FULL, order_of(high));
    wild = __any_sync(FULL, row.wild);
    if (lane == 0) sh.red[warp] = make_uint4(most, least, top, wild);
    sync_row<T>();
    const uint4 x = sh.red[lane % NW];
    most = __reduce_max_sync(FULL, x.x);
    low = from_order(__reduce_min_sync(FULL, x.y));
    high = from_order(__reduce_max_sync(FULL, x.z));
    wild = __any_sync(FULL, x.w != 0);
  };
  auto scores_changed = [&]() {
    sync_row<T>();
    for (int i = tid; i < BINS / 2; i += T) reinterpret_cast<int4*>(sh.hist[0])[i] = make_int4(0, 0, 0, 0);
    if (tid < 2) sh.open[tid] = sh.over[tid] = 0;
    low = INFINITY;
    high = -INFINITY;
    for (int v = tid; 4 * v < nb; v += T) widen(four(v));
    reduce();
  };
#pragma unroll 2
  for (int v = tid; 4 * v < (CACHED ? 32 * words : nb); v += T) {
    const float4 x = 4 * v < nb ? read_four(v) : make_float4(none, none, none, none);
    if constexpr (CACHED) *reinterpret_cast<float4*>(cache + 4 * v) = x;
    widen(x);
  }
  reduce();
  {
    const float b_norm = fmaxf(__uint_as_float(most), wild ? LEAST_NORM : 0.f), norms = norm_of_q(row, wild) * b_norm;
    off = eps * norms;
    if (EASY && (wild || !(off < INFINITY) || want == 0)) return false;
    if (wild && off < INFINITY) {
      tame<T>(p, r, h, n, nb, row.norms, INFINITY, b_norm, 2.f * norms, sh.q, CACHED ? cache : sc);
      scores_changed();
    }
  }
  const bool known = off < INFINITY;  // else a NaN or infinity is among the queries, and every score is taken again
  auto choose = [&](int i) { atomicOr(&s_bits[i >> 5], 1u << (i & 31)); };
  auto exact = [&](int i) {  // block i's score in 64 bits, by a warp
    uint32_t b[8];
    load_bounds(p, row, i, b, lane);
    return order_of(product(p, sh.q, b, lane));
  };

  // ---- Narrow the window [low, high] about the border, a bin of BINS at a time, until 32 blocks at most are in it.
  // A score far from the others (a first page's, say) costs a round.
  bool few = false;
  int open = 0, over = 0;  // in the window; above it
  for (bool tried = false; known && want > 0; tried = true) {
    for (int round = 0; !few; ++round) {
      int* hist = sh.hist[round & 1];
      const float range = high - low, per_step = (4 * BINS - 1) / range;
      if (!(range < INFINITY && per_step < INFINITY)) break;  // all alike, or past float32
      auto count = [&](float x) { count_step(hist, x, low, high, per_step); };
      for (int v = tid; 4 * v < nb; v += T) {
        const float4 x = four(v);
        count(x.x);
        count(x.y);
        count(x.z);
        count(x.w);
      }
      sync_row<T>();
      // a warp finds the bin of the border, each for itself where they are few: lane 0 holds the highest
      int bin = -1;
      if (NW <= 8 || warp == 0) bin = border_bin(hist, over, want, lane);
      if constexpr (NW > 8) {
        if (tid == 0) sh.digit = bin;
        sync_row<T>();
        bin = sh.digit;
      }
      narrow(bin, range, off, low, high);
      int above_high = 0;
      for (int w = warp; w < words; w += NW) {
        const float x = score(32 * w + lane);
        const bool above = x > high;
        if (x >= low && !above) {
          const int k = atomicAdd(&sh.open[round & 1], 1);
          if (k < 32) {
            sh.at[k] = 32 * w + lane;
            sh.score[k] = x;
          }
        }
        const unsigned bits = __ballot_sync(FULL, above);
        above_high += __popc(bits);
        if (lane == 0) s_bits[w] = bits;
      }
      if (lane == 0 && above_high > 0) atomicAdd(&sh.over[round & 1], above_high);
      sync_row<T>();
      open = sh.open[round & 1];
      over = sh.over[round & 1];
      few = open <= 32;
      if (!few) {
        if (!(high - low < 0.5f * range)) break;  // the error's width: they may as well be alike
        const int other = (round & 1) ^ 1;
        for (int i = tid; i < BINS; i += T) sh.hist[other][i] = 0;
        sync_row<T>();
        if (tid == 0) sh.open[round & 1] = sh.over[round & 1] = 0;
      }
    }
    if (EASY || few || tried || sc == nullptr || off == 0.f) break;  // (a row scored by its own CTA has no norms)
    const float norms = leave_out<T>(p, r, h, n, nb, row.norms, row.q_norm, sh, CACHED ? cache : sc);
    if (norms == 0.f) break;
    off = eps * norms;
    over = 0;
    scores_changed();
  }

  if (EASY && !few) return false;
  if (EASY || few) {
    // ---- a warp settles it, a lane a block
    const int places = want - over;  // 1 <= places <= open
    for (int i = tid; i < p.first + p.last; i += T) choose(i < p.first ? i : nb - p.last + i - p.first);
    Border at;
    if (warp == 0) {
      at = settle(sh, open, places, off, lane);
      if (lane == 0) sh.among = off == 0.f ? 0u : at.among;
      if (at.among == 0 && (at.sure || at.close)) choose(at.block);
    }
    sync_row<T>();
    if (sh.among != 0) {  // by the exact scores, a warp a block; the first one's bounds come while the heads are summed
      unsigned todo = sh.among;
      for (int k = 0; k < warp && todo != 0; ++k) todo &= todo - 1;
      uint32_t b[8];
      if (todo != 0) load_bounds(p, row, sh.at[__ffs(todo) - 1], b, lane);
      sum_heads(p, row, sh.q, tid, T);
      sync_row<T>();
      for (bool first = true; todo != 0; first = false) {
        const int j = __ffs(todo) - 1;
        const unsigned long long key = first ? order_of(product(p, sh.q, b, lane)) : exact(sh.at[j]);
        if (lane == 0) sh.key[j] = key;
        for (int k = 0; k < NW && todo != 0; ++k) todo &= todo - 1;
      }
      sync_row<T>();
    }
    if (warp == 0 && at.among != 0) {
      const unsigned long long key = at.close && off != 0.f ? sh.key[lane] : 0ull;  // where the bound is 0 every score is
      if (takes(at, key)) choose(at.block);
    }
  } else {
    // ---- Many at the border, or none: queries that are no finite numbers, pages that are alike, or no place but the kept
    // ones'.  The border digit by digit, of the scores and then, among those that they leave open, of the exact scores: of their
    // upper halves, which take the scores' places, and of the lower halves of those that then tie.  512 rows of 2048 pages,
    // 8 heads, of two kinds whose scores tie: 28 ms (125 where each digit had every score computed again).
    int* hist = sh.digits;
    auto digit = [&](int left) {  // the one that holds the left-th largest
      sync_row<T>();
      if (tid == 0) {
        int above = 0, at = 255;
        while (at > 0 && above + hist[at] < left) above += hist[at--];
        sh.digit = at;
        sh.above = above;
      }
      sync_row<T>();
    };
    auto clear = [&]() {
      sync_row<T>();
      for (int i = tid; i < 256; i += T) hist[i] = 0;
      sync_row<T>();
    };
    uint32_t border = 0;
    if (known && want > 0) {
      uint32_t mask = 0;
      int left = want;
      for (int shift = 24; shift >= 0; shift -= 8) {
        clear();
        for (int i = c0 + tid; i < c1; i += T) {
          const uint32_t u = order_of(score(i));
          if (((u ^ border) & mask) == 0) atomicAdd(&hist[u >> shift & 255], 1);
        }
        digit(left);
        border |= static_cast<uint32_t>(sh.digit) << shift;
        mask |= 255u << shift;
        left -= sh.above;
      }
    }
    const float at = from_order(border), most = known ? at + 2.f * off : INFINITY, least = known ? at - 2.f * off : -INFINITY;
    sync_row<T>();
    if (tid == 0) sh.open[0] = sh.over[0] = 0;
    sync_row<T>();
    int ins = 0, opens = 0;
    for (int w = warp; w < words; w += NW) {
      const int i = 32 * w + lane;
      const bool mine = want > 0 && competing(i), kept = i < nb && !competing(i), in = mine && known && score(i) > most;
      const unsigned open_bits = __ballot_sync(FULL, mine && !in && (!known || score(i) >= least));
      const unsigned in_bits = __ballot_sync(FULL, in), kept_bits = __ballot_sync(FULL, kept);
      ins += __popc(in_bits);
      opens += __popc(open_bits);
      if (lane == 0) {
        s_bits[w] = in_bits | kept_bits;
        ties[w] = open_bits;
      }
    }
    if (lane == 0) {
      atomicAdd(&sh.over[0], ins);
      atomicAdd(&sh.open[0], opens);
    }
    sync_row<T>();
    int left = want - sh.over[0];
    // with a bound of 0 every score is 0, with a NaN among the queries' sums every score is one
    bool score_again = left < sh.open[0] && !(known && off == 0.f) && row.q_norm == row.q_norm;
    if (score_again) {
      // Pages with the same bounds have the same score, and a cache that nothing was written to has no others: 512 rows of
      // 2048 such pages, 8 heads, take 1.2 ms this way.
      if (tid == 0) sh.among = 0;
      sync_row<T>();
      const uint32_t* bounds = reinterpret_cast<const uint32_t*>(p.bounds);
      auto page_of = [&](int i) {
        int id = p.block_table[static_cast<int64_t>(n) * p.max_blocks + i];
        if (id < 0 || id >= p.num_blocks) id = 0;
        return id;
      };
      int first = -1;  // the lowest of them
      for (int w = 0; first < 0; ++w)
        if (ties[w] != 0) first = page_of(32 * w + __ffs(ties[w]) - 1);
      uint32_t like[8], differs = 0;
      auto words_of = [&](int page, uint32_t (&x)[8]) {
        const uint32_t* from = bounds + (static_cast<int64_t>(page) * p.Hkv + h) * p.d + lane;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 32 * k < p.d ? from[32 * k] : 0u;
      };
      words_of(first, like);
      for (int w = warp; w < words; w += NW) {
        const int page = ties[w] >> lane & 1 ? page_of(32 * w + lane) : first;
        for (unsigned todo = ties[w]; todo != 0; todo &= todo - 1) {
          uint32_t x[8];
          words_of(__shfl_sync(FULL, page, __ffs(todo) - 1), x);
#pragma unroll
          for (int k = 0; k < 8; ++k) differs |= x[k] ^ like[k];
        }
        if (__any_sync(FULL, differs != 0)) break;
      }
      if (differs != 0) atomicOr(&sh.among, 1u);
      sync_row<T>();
      score_again = sh.among != 0;
    }
    if (score_again) sum_heads(p, row, sh.q, tid, T);
    uint32_t* keys = reinterpret_cast<uint32_t*>(CACHED ? cache : sc);
    for (int half = 0; score_again && half < 2; ++half) {
      sync_row<T>();
      for (int w = warp; w < words; w += NW)
        for (unsigned todo = ties[w]; todo != 0; todo &= todo - 1) {
          const int i = 32 * w + __ffs(todo) - 1;
          const unsigned long long key = exact(i);
          if (lane == 0) keys[i] = static_cast<uint32_t>(half == 0 ? key >> 32 : key);
        }
      uint32_t key_at = 0, mask = 0;
      for (int shift = 24; shift >= 0; shift -= 8) {
        clear();
        for (int w = warp; w < words; w += NW)
          if (ties[w] >> lane & 1) {
            const uint32_t u = keys[32 * w + lane];
            if (((u ^ key_at) & mask) == 0) atomicAdd(&hist[u >> shift & 255], 1);
          }
        digit(left);
        key_at |= static_cast<uint32_t>(sh.digit) << shift;
        mask |= 255u << shift;
        left -= sh.above;
      }
      score_again = left < hist[sh.digit];  // of those that tie, or all of them have a place
      for (int w = warp; w < words; w += NW) {
        const bool mine = ties[w] >> lane & 1;
        const uint32_t u = mine ? keys[32 * w + lane] : 0u;
        const unsigned above = __ballot_sync(FULL, mine && u > key_at), tie = __ballot_sync(FULL, mine && u == key_at);
        if (lane == 0) {
          s_bits[w] |= above;
          ties[w] = tie;
        }
      }
    }
    sync_row<T>();
    if (warp == 0)  // the lowest of those that tie
      for (int w = 0; w < words && left > 0; ++w) {
        unsigned tie = ties[w];
        while (__popc(tie) > left) tie &= ~(0x80000000u >> __clz(tie));
        left -= __popc(tie);
        if (lane == 0) s_bits[w] |= tie;
      }
  }
  sync_row<T>();

  // ---- in ascending order: every warp counts, each takes the words, a lane a word, of every NW-th group of 32
  int base = 0;
  for (int w0 = 0, group = 0; w0 < words; w0 += 32, ++group) {
    unsigned bits = w0 + lane < words ? s_bits[w0 + lane] : 0u;
    int upto = __popc(bits);
    if (group % NW != warp) {
      base += __reduce_add_sync(FULL, upto);
      continue;
    }
    int place = base - upto;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(FULL, upto, o);
      if (lane >= o) upto += x;
    }
    place += upto;
    base += __shfl_sync(FULL, upto, 31);
    for (; bits != 0; bits &= bits - 1, ++place)
      if (place < K) out[place] = 32 * (w0 + lane) + __ffs(bits) - 1;
  }
  return true;
}

// The other rows, apart: what they need of registers would cost the easy ones
template <int T, bool CACHED>
__device__ __noinline__ void pick_hard(const SelectBlocksParams& p, int r, int h, int n, int nb, float* scores, const float* norms,
                                       float q_norm, float b_norm, bool wild, float eps, PickShared& sh, uint32_t* s_bits) {
  Row row;
  row.r = r;
  row.h = h;
  row.n = n;
  row.nb = nb;
  row.scores = scores;
  row.norms = norms;
  row.q_norm = q_norm;
  row.b_norm = b_norm;
  row.wild = wild;
  sync_row<T>();
  pick<T, CACHED, false>(p, row, eps, sh, s_bits);
}
template <int T, bool CACHED>
__device__ __forceinline__ void pick_hard(const SelectBlocksParams& p, const Row& row, float eps, PickShared& sh, uint32_t* s_bits) {
  pick_hard<T, CACHED>(p, row.r, row.h, row.n, row.nb, row.scores, row.norms, row.q_norm, row.b_norm, row.wild, eps, sh, s_bits);
}

// The same by a warp that holds the scores in registers, 32 NR at most; wild tiles are tame.  norms: ||Q|| times the largest
// ||b||.  False, and nothing done, where there is more to it: queries that are no finite numbers, many alike at the
// border, or no place but the kept blocks'.
template <int NR>
__device__ __forceinline__ bool pick_warp(const SelectBlocksParams& p, const Row& row, float norms, bool wild, float eps,
                                          PickShared& sh) {
  constexpr int NW = (NR + 31) / 32;  // words of chosen blocks a lane: word 32 k + lane
  const int lane = threadIdx.x & 31, nb = row.nb, c0 = p.first, c1 = nb - p.last, want = p.K - p.first - p.last;
  if (want == 0) return false;
  const float* sc = row.scores;
  const float none = __uint_as_float(0x7fffffffu);  // a NaN: neither above, below nor within a window
  float x[NR], low = INFINITY, high = -INFINITY;
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    x[j] = none;
    if (32 * j < nb && static_cast<unsigned>(32 * j + lane - c0) < static_cast<unsigned>(c1 - c0)) x[j] = sc[32 * j + lane];
  }
  int* hist = sh.hist[0];
  auto clear = [&]() {
#pragma unroll
    for (int k = 0; k < BINS / 128; ++k) reinterpret_cast<int4*>(hist)[32 * k + lane] = make_int4(0, 0, 0, 0);
    __syncwarp();
  };
  clear();
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    low = fminf(low, x[j]);
    high = fmaxf(high, x[j]);
  }
  low = from_order(__reduce_min_sync(FULL, order_of(low)));
  high = from_order(__reduce_max_sync(FULL, order_of(high)));
  const float off = eps * norms;
  if (!(off < INFINITY)) return false;
  unsigned bits[NW], in[NW];  // of this lane's scores: bit j % 32 of number j / 32; above the window, within it
  int open = 0, over = 0;     // how many are in the window; above it
  for (;;) {
    const float range = high - low, per_step = (4 * BINS - 1) / range;
    if (!(range < INFINITY && per_step < INFINITY)) return false;
#pragma unroll
    for (int j = 0; j < NR; ++j) count_step(hist, x[j], low, high, per_step);
    __syncwarp();
    narrow(border_bin(hist, over, want, lane), range, off, low, high);
#pragma unroll
    for (int k = 0; k < NW; ++k) bits[k] = in[k] = 0;
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      if (x[j] > high) bits[j / 32] |= 1u << j % 32;
      if (x[j] >= low) in[j / 32] |= 1u << j % 32;
    }
    open = over = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      in[k] &= ~bits[k];
      open += __popc(in[k]);
      over += __popc(bits[k]);
    }
    int place = open;  // in the list of those in the window, after the lanes' before
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULL, place, o);
      if (lane >= o) place += y;
    }
    place -= open;
    open = __shfl_sync(FULL, place + open, 31);
    over = __reduce_add_sync(FULL, over);
    if (open <= 32) {
#pragma unroll
      for (int k = 0; k < NW; ++k)
        for (; in[k] != 0; in[k] &= in[k] - 1, ++place) {
          const int i = 32 * (32 * k + __ffs(in[k]) - 1) + lane;
          sh.at[place] = i;
          sh.score[place] = sc[i];
        }
      __syncwarp();
      break;
    }
    if (!(high - low < 0.5f * range)) return false;  // the error's width: they may as well be alike
    __syncwarp();
    clear();
  }
  // block 32 j + l is bit j of lane l's: to bit l of lane j's
#pragma unroll
  for (int k = 0; k < NW; ++k) bits[k] = transpose_32x32(bits[k], lane);
  Border at = settle(sh, open, want - over, off, lane);
  if (at.among != 0 && off != 0.f && !wild) refine(p, row, norms, at, lane);  // (wild blocks are past its range)
  bool chosen = at.sure || at.close;
  if (at.among != 0) {
    // where the bound is 0 every score is
    const unsigned long long key = off != 0.f ? exact_keys(p, row.r, row.h, row.n, at.block, at.among, lane) : 0ull;
    chosen = takes(at, key);
  }
  for (unsigned todo = __ballot_sync(FULL, chosen); todo != 0; todo &= todo - 1) {
    const int block = __shfl_sync(FULL, at.block, __ffs(todo) - 1);
#pragma unroll
    for (int k = 0; k < NW; ++k)
      if (block >> 5 == 32 * k + lane) bits[k] |= 1u << (block & 31);
  }
  int32_t* out = p.blocks + (static_cast<int64_t>(row.r) * p.Hkv + row.h) * p.K;
  int base = 0;
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    const int b0 = 32 * (32 * k + lane);  // the word's first block; the kept ones are those outside [c0, c1)
    unsigned word = bits[k] | ~below(c1 - b0) | below(c0 - b0);
    word &= below(nb - b0);
    int upto = __popc(word), place = base - upto;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULL, upto, o);
      if (lane >= o) upto += y;
    }
    place += upto;
    base += __shfl_sync(FULL, upto, 31);
    for (; word != 0; word &= word - 1, ++place)
      if (place < p.K) out[place] = b0 + __ffs(word) - 1;
  }
  return true;
}

// A warp a row and KV head, four a CTA.  The numbers of CTAs an SM leave 20 to 90 bytes a thread of the forms with 16 and 32
// scores a lane in local memory, and 50 of select_one_kernel's at d = 128.
template <int NR>
__global__ void __launch_bounds__(128, NR == 16 ? 6 : NR == 32 ? 5 : 4)
    select_warps_kernel(const __grid_constant__ SelectBlocksParams p, const Scratch ws) {
  extern __shared__ __align__(16) uint32_t s_words[];
  __shared__ PickShared shared[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + warp;
  const bool beyond = at >= static_cast<int64_t>(p.T) * p.Hkv;
  if (beyond) at = 0;
  Row row;
  row.r = static_cast<int>(static_cast<unsigned>(at) / static_cast<unsigned>(p.Hkv));  // rows times heads are below 2^31
  row.h = static_cast<int>(at - static_cast<int64_t>(row.r) * p.Hkv);
  row.n = p.cu == nullptr ? row.r : sequence_of(p.cu, p.N, row.r);
  const Span s = span_of(p, row.n, false);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores are there
  if (beyond || row.r < s.first || row.r >= s.end) return;  // of no sequence: left as it was
  row.nb = blocks_seen(s, row.r);
  if (row.nb <= p.K) {
    choose_all<32>(p, at, row.nb);
    return;
  }
  row.norms = ws.b_norm + (static_cast<int64_t>(row.n) * p.Hkv + row.h) * ws.tiles;
  row.q_norm = ws.q_norm[at];
  row.b_norm = 0.f;
  row.wild = false;
#pragma unroll
  for (int k = 0; k < (NR * 2 + 31) / 32; ++k)
    if (32 * k + lane < (row.nb + 15) / 16) count_norm(row, row.norms[32 * k + lane]);
  row.scores = ws.scores + at * ws.stride;
  const bool wild = __any_sync(FULL, row.wild);
  const float most = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(row.b_norm)));
  const float b_norm = fmaxf(most, wild ? LEAST_NORM : 0.f), norms = norm_of_q(row, wild) * b_norm;
  if (wild && norms < INFINITY) {
    tame<32>(p, row.r, row.h, row.n, row.nb, row.norms, INFINITY, b_norm, 2.f * norms, shared[warp].q, row.scores);
    __syncwarp();
  }
  if (!pick_warp<NR>(p, row, norms, wild, ws.eps, shared[warp]))
    pick_hard<32, false>(p, row, ws.eps, shared[warp], s_words + warp * cache_at(p.max_blocks));
}

template <int T, bool CACHED>
__global__ void __launch_bounds__(T, T == 128 ? 10 : 1)
    select_kernel(const __grid_constant__ SelectBlocksParams p, const Scratch ws) {
  extern __shared__ __align__(16) uint32_t s_bits[];
  __shared__ PickShared shared;
  Row row;
  row.r = blockIdx.x / p.Hkv;
  row.h = blockIdx.x % p.Hkv;
  row.n = p.cu == nullptr ? row.r : sequence_of(p.cu, p.N, row.r);
  const Span s = span_of(p, row.n, false);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores are there
  if (row.r < s.first || row.r >= s.end) return;       // of no sequence: left as it was
  row.nb = blocks_seen(s, row.r);
  if (row.nb <= p.K) {
    choose_all<T>(p, blockIdx.x, row.nb);
    return;
  }
  row.norms = ws.b_norm + (static_cast<int64_t>(row.n) * p.Hkv + row.h) * ws.tiles;
  row.q_norm = ws.q_norm[blockIdx.x];
  row.b_norm = 0.f;
  row.wild = false;
  for (int i = threadIdx.x; i < (row.nb + 15) / 16; i += T) count_norm(row, row.norms[i]);
  row.scores = ws.scores + static_cast<int64_t>(blockIdx.x) * ws.stride;
  if (!pick<T, CACHED, true>(p, row, ws.eps, shared, s_bits)) pick_hard<T, CACHED>(p, row, ws.eps, shared, s_bits);
}

// Short sequences of one row each: a CTA scores the blocks of a row and KV head and picks among them, in one launch.  A
// warp takes 16 blocks at a time, their bounds from HBM straight to registers, in the order of the matrix product's left
// operand.
template <int D, int T>
__global__ void __launch_bounds__(T, 512 / T) select_one_kernel(const __grid_constant__ SelectBlocksParams p, float eps) {
  constexpr int NW = T / 32, KK = 2 * D / 32, PART = KK < 8 ? KK : 8, PARTS = KK / PART;
  extern __shared__ __align__(16) uint32_t s_bits[];
  __shared__ PickShared shared;
  __shared__ __align__(16) uint32_t s_qb[KK * 2 * 16];  // Q-, Q+ as two bf16 numbers each: [KK][2 columns][16 words]
  __shared__ float s_squares[NW], s_norms[ONE_BLOCKS / 16];  // s_norms: infinite for wild tiles, else 0
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  Row row;
  const int n = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  const Span s = span_of(p, n, h == 0 && threadIdx.x == 0);
  if (s.end <= s.first) return;
  row.r = s.first;
  row.h = h;
  row.n = n;
  row.nb = blocks_seen(s, s.first);
  row.scores = nullptr;
  const int nb = row.nb;
  if (nb <= p.K) {
    choose_all<T>(p, static_cast<int64_t>(row.r) * p.Hkv + h, nb);
    return;
  }
  auto page_of = [&](int tile) {  // of block 16 tile + lane % 16; page 0 where there is none
    const int blk = tile * 16 + (lane & 15);
    int id = blk < nb ? p.block_table[static_cast<int64_t>(n) * p.max_blocks + blk] : 0;
    if (id < 0 || id >= p.num_blocks) {
      set_error(&g_select_blocks_status, kDevBadPage);
      id = 0;
    }
    return id;
  };
  uint32_t a[PART][2][4];
  auto load = [&](int id, int part) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t page = __shfl_sync(FULL, id, g + 8 * e);
      const __nv_bfloat16* from = p.bounds + (page * p.Hkv + h) * 2 * D + 32 * PART * part + 8 * t;
#pragma unroll
      for (int k = 0; k < PART; ++k) {
        const uint4 x = *reinterpret_cast<const uint4*>(from + 32 * k);
        a[k][e][0] = x.x; a[k][e][1] = x.y; a[k][e][2] = x.z; a[k][e][3] = x.w;
      }
    }
  };
  int tile = warp, id = tile * 16 < nb ? page_of(tile) : 0;
  // ---- the sums over heads, a pair of channels a thread; four heads' loads in flight
  const int G = p.Hq / p.Hkv;
  float squares = 0.f;
  uint32_t any = 0;
  if (threadIdx.x < D / 2) {
    const uint32_t* from = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(row.r) * p.Hq + h * G) * D) + threadIdx.x;
    float neg[2] = {0.f, 0.f}, pos[2] = {0.f, 0.f};
    for (int e0 = 0; e0 < G; e0 += 4) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = e0 + e < G ? from[(e0 + e) * (D / 2)] : 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) add_parts(w[e], neg, pos);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float* x = half ? pos : neg;
      const uint32_t hi = pack_bf16x2(x[0], x[1]);
      const float2 z = pair_of(hi);
      const int word = half * (D / 2) + threadIdx.x;
      s_qb[word / 16 * 32 + word % 16] = hi;
      s_qb[word / 16 * 32 + 16 + word % 16] = pack_bf16x2(x[0] - z.x, x[1] - z.y);
      squares = fmaf(x[0], x[0], fmaf(x[1], x[1], squares));
      any |= hi & 0x7fff7fffu;
    }
  }
  if (tile * 16 < nb) load(id, 0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) squares += __shfl_xor_sync(FULL, squares, o);
  if (__any_sync(FULL, any != 0) && squares < LEAST_NORM * LEAST_NORM) squares = LEAST_NORM * LEAST_NORM;
  if (lane == 0) s_squares[warp] = squares;
  __syncthreads();
  squares = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i) squares += s_squares[i];
  row.q_norm = sqrtf(squares);
  row.norms = s_norms;
  row.b_norm = 0.f;

  float* cache = reinterpret_cast<float*>(s_bits + cache_at(p.max_blocks));
  while (tile * 16 < nb) {
    const int next = tile + NW, next_id = next * 16 < nb ? page_of(next) : 0;
    float acc[2][4] = {}, norm[2] = {0.f, 0.f};
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      if (part > 0) load(id, part);
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
#pragma unroll
      for (int k = 0; k < PART; ++k) {
        uint4 b = make_uint4(0, 0, 0, 0);  // the columns behind the second are 0
        if (g < 2) b = *reinterpret_cast<const uint4*>(s_qb + (part * PART + k) * 32 + g * 16 + t * 4);
        mma_16816<false>(acc[0], a[k][0][0], a[k][1][0], a[k][0][1], a[k][1][1], b.x, b.y);
        mma_16816<false>(acc[1], a[k][0][2], a[k][1][2], a[k][0][3], a[k][1][3], b.z, b.w);
      }
    }
    const int blk = tile * 16 + g;
    if (t == 0) {
      if (blk < nb) cache[blk] = (acc[0][0] + acc[1][0]) + (acc[0][1] + acc[1][1]);
      if (blk + 8 < nb) cache[blk + 8] = (acc[0][2] + acc[1][2]) + (acc[0][3] + acc[1][3]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      norm[e] += __shfl_xor_sync(FULL, norm[e], 1);
      norm[e] += __shfl_xor_sync(FULL, norm[e], 2);
      if (!(norm[e] < MOST_SQUARES)) norm[e] = INFINITY;  // NaN too
      if (competes(p, blk + 8 * e, nb)) row.b_norm = fmaxf(row.b_norm, norm[e]);
    }
    tile = next;
    id = next_id;
    if (tile * 16 < nb) load(id, 0);
  }
  row.wild = !(row.b_norm < INFINITY);
  if (__syncthreads_or(row.wild)) {  // rare: which tiles, and the norms of the others; a block a thread
    for (int i = threadIdx.x; i < (nb + 15) / 16; i += T) s_norms[i] = 0.f;
    row.b_norm = 0.f;
    row.wild = false;
    __syncthreads();
    for (int i = p.first + threadIdx.x; i < nb - p.last; i += T) {
      int page = p.block_table[static_cast<int64_t>(n) * p.max_blocks + i];
      if (page < 0 || page >= p.num_blocks) page = 0;
      const uint4* from = reinterpret_cast<const uint4*>(p.bounds + (static_cast<int64_t>(page) * p.Hkv + h) * 2 * D);
      float norm = 0.f;
#pragma unroll 4
      for (int k = 0; k < D / 4; ++k) {
        const uint4 x = from[k];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 y = pair_of(w[c]);
          norm = fmaf(y.x, y.x, fmaf(y.y, y.y, norm));
        }
      }
      if (norm < MOST_SQUARES) {
        row.b_norm = fmaxf(row.b_norm, norm);
      } else {
        row.wild = true;
        s_norms[i / 16] = INFINITY;
      }
    }
    // a tile's blocks are wild together: the norm of one that is not by itself does no harm
    __syncthreads();
  }
  // the sum of squares may have been an eighth too small
  row.b_norm = fmaxf(1.1f * sqrtf(row.b_norm), LEAST_NORM);
  if (!pick<T, true, true>(p, row, eps, shared, s_bits)) pick_hard<T, true>(p, row, eps, shared, s_bits);
}

// A kernel's limit of dynamic shared memory belongs to the kernel on the device, not to the call: two host threads set it
// between each other's setting and launch.  So every call sets the same limit, the largest that any call needs.

// A launch as a programmatic dependent of the kernel before it
template <class... Params, class... Args>
cudaError_t launch_behind(void (*kernel)(Params...), unsigned grid, unsigned threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int T, bool CACHED>
cudaError_t select(const SelectBlocksParams& p, const Scratch& ws, cudaStream_t stream) {
  constexpr int MOST = pick_bytes(CACHED ? CACHED_BLOCKS : SELECT_MOST_BLOCKS, CACHED);
  const int smem = pick_bytes(p.max_blocks, CACHED);
  const cudaError_t e = cudaFuncSetAttribute(select_kernel<T, CACHED>, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
  if (e != cudaSuccess) return e;
  return launch_behind(select_kernel<T, CACHED>, static_cast<unsigned>(static_cast<int64_t>(p.T) * p.Hkv), T, smem, stream, p,
                       ws);
}

template <int NR>
cudaError_t select_warps(const SelectBlocksParams& p, const Scratch& ws, cudaStream_t stream) {
  const int smem = 4 * pick_bytes(p.max_blocks, false);
  return launch_behind(select_warps_kernel<NR>, static_cast<unsigned>((static_cast<int64_t>(p.T) * p.Hkv + 3) / 4), 128, smem,
                       stream, p, ws);
}

template <int D, int T>
cudaError_t select_one(const SelectBlocksParams& p, float eps, cudaStream_t stream) {
  // within the 48 KB that a launch may take without a limit of its own, beside sums, bins and norms
  static_assert(pick_bytes(ONE_BLOCKS, true) + sizeof(PickShared) + 4 * 1024 <= 48 * 1024, "shared memory budget");
  select_one_kernel<D, T><<<static_cast<unsigned>(static_cast<int64_t>(p.N) * p.Hkv), T, pick_bytes(p.max_blocks, true), stream>>>(
      p, eps);
  return cudaGetLastError();
}

template <int D>
cudaError_t score_few(const SelectBlocksParams& p, const Scratch& ws, int sms, cudaStream_t stream) {
  using C = FewCfg<D>;
  const int warps = C::warps(p.max_q), smem = warps * C::warp_bytes(p.max_q);
  const cudaError_t e = cudaFuncSetAttribute(score_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::most_bytes());
  if (e != cudaSuccess) return e;
  score_few_kernel<D><<<sms, warps * 32, smem, stream>>>(p, ws);
  return cudaGetLastError();
}

template <int D, bool SMALL>
cudaError_t score_many(const SelectBlocksParams& p, const Scratch& ws, int sms, cudaStream_t stream) {
  using C = ManyCfg<D, SMALL>;
  const int sum_tiles = (p.max_q + SUM_ROWS - 1) / SUM_ROWS, row_tiles = (p.max_q + C::RT - 1) / C::RT;
  const int64_t pairs = static_cast<int64_t>(p.N) * p.Hkv;
  sum_heads_kernel<D, SMALL><<<static_cast<unsigned>(pairs * sum_tiles), SUM_ROWS / 2 * 32, 0, stream>>>(p, ws, sum_tiles);
  cudaError_t e = cudaGetLastError();
  auto kern = score_many_kernel<D, SMALL>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t all = (p.max_blocks + 127) / 128, most = (SCORE_CTAS + pairs - 1) / pairs;
  const int chunks = static_cast<int>(all < most ? all : most);
  // where the device holds more CTAs than there are tiles: d = 128, a sequence of 8192 tokens, 8 KV heads, 512 rows 12.7 us
  // against 19.7, of 16384 tokens with 4096 rows 69.5 against 115.7
  const int64_t fit = static_cast<int64_t>(sms) * C::CTAS / (pairs * chunks), most_splits = fit < row_tiles ? fit : row_tiles;
  const int splits = most_splits > 1 ? static_cast<int>(most_splits) : 1;
  return launch_behind(kern, static_cast<unsigned>(pairs * chunks * splits), C::WARPS * 32, C::SMEM, stream, p, ws, chunks,
                       splits);
}

// How far scores may be off, relative to ||Q|| ||b||: Q as two bf16 numbers 2^-18, its sums over G heads 2^-24 each, and the
// matrix products.  Measured on sm_103a: a product aligns its terms and the accumulator to the largest one and drops what lies
// below 2^-25 of that one's power of two, then cuts the sum to 24 bits: it is off by (terms + 4) 2^-25 of the sum of |terms|
// at most.  mma.sync takes 8 terms at a time, two accumulators share the 2 d, and three additions join them with the second
// parts of Q; tcgen05 takes 16, for the second parts first.  One 2^-25 a product covers those parts, which are 2^-8 of the
// first at most.  Terms made to lose all that they can reach 0.41 to 0.63 of this with tcgen05, 0.26 to 0.46 with mma.sync;
// random ones 0.03.
template <int D, bool FEW_ROWS>
constexpr float score_error(int heads) {
  constexpr float U = 1.f / (1 << 25);
  return FEW_ROWS ? 1.f / (1 << 18) + static_cast<float>(heads + 3) * (2 * U) + static_cast<float>(D / 16 * (2 * (8 + 4) + 1)) * U
                  : 1.f / (1 << 18) + static_cast<float>(heads) * (2 * U) + static_cast<float>(D / 8 * (16 + 4 + 1)) * U;
}

template <int D>
cudaError_t launch(const SelectBlocksParams& p, Scratch& ws, cudaStream_t stream) {
  const float eps_few = score_error<D, true>(p.Hq / p.Hkv);
  const int64_t pairs = static_cast<int64_t>(p.N) * p.Hkv;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // One launch as long as every row and KV head has a CTA at once and tables are short enough for a CTA to read a row's
  // bounds alone.  Both sides at d = 128, one against two launches: 128 rows times heads of 250 blocks 10.4 and 14.9 us, of
  // 1000 26.3 and 26.1; 8 of 250 8.8 and 11.2, of 500 10.9 and 10.5, of 1000 17.2 and 12.3; 256 of 500 21.7 and 26.4.  Of
  // more, smaller CTAs: 512 of 125 12.1 and 18.3, of 250 22.0 and 26.5, of 32 to 512 30.9 and 27.5, where the longest is
  // waited for; 2048 of 125 45.0 and 43.2.
  if (p.max_q == 1 && pairs <= 2 * sms && p.max_blocks <= ONE_BLOCKS && p.max_blocks <= 250 + 8 * pairs)
    return select_one<D, 256>(p, eps_few, stream);
  if (p.max_q == 1 && pairs <= 4 * sms && p.max_blocks <= 256) return select_one<D, 128>(p, eps_few, stream);
  // few rows and more tiles of blocks than SMs: gathering the bounds counts, and two CTAs an SM overlap that
  const bool small = D == 128 && p.max_q <= SMALL_ROWS && pairs * ((p.max_blocks + 127) / 128) > sms;
  ws.eps = p.max_q <= FEW ? eps_few : score_error<D, false>(p.Hq / p.Hkv);
  e = p.max_q <= FEW ? score_few<D>(p, ws, sms, stream)
      : small        ? score_many<D, D == 128>(p, ws, sms, stream)
                     : score_many<D, false>(p, ws, sms, stream);
  if (e != cudaSuccess) return e;
  // Of few long rows the latency of one is to be shortened.  Of many, instructions count, which are fewer the fewer warps
  // do a row's common work: 4096 rows of 2048 blocks take 51 us with 128 threads, 55 with 64, which leave too few warps.
  // The whole call with 128 and with 1024 threads, d = 64: 128 rows of 2500 blocks 31.9 and 26.0 us, 256 47.6 and 46.1, 512
  // 80.8 and 89.3, 800 112 and 132; of 8125 128 71.8 and 59.3, 256 122.3 and 116.6, 512 220.8 and 228.2, 800 346 and 352.
  // A warp a row, its scores in registers, has no barriers and does a row's common work once; a CTA a row has more rows'
  // latencies under way where they are few.  Warp and CTA, us, d = 128: 16384 rows of 250 blocks 64 and 96, of 500 61 and 92,
  // of 2000 130 and 170, 32768 of 1000 143 and 220; 1024 of 1000 17.4 and 20.7, of 2000 20.6 and 23.8; decode steps of 2048
  // rows and heads, 1000 blocks 202 and 204, 2000 384 and 386; 512 of 375 33.0 and 32.1, of 1000 61.4 and 62.6; 64 of 2000
  // 26.3 and 23.7.
  if (static_cast<int64_t>(p.T) * p.Hkv >= WARP_ROWS) {
    if (p.max_blocks <= 512) return select_warps<16>(p, ws, stream);
    if (p.max_blocks <= 1024) return select_warps<32>(p, ws, stream);
    if (p.max_blocks <= 1536) return select_warps<48>(p, ws, stream);
    if (p.max_blocks <= 2048) return select_warps<64>(p, ws, stream);
    if (p.max_blocks <= 2560) return select_warps<80>(p, ws, stream);
  }
  if (p.max_blocks > CACHED_BLOCKS) return select<1024, false>(p, ws, stream);
  const bool many = static_cast<int64_t>(p.T) * p.Hkv > 2 * sms;  // more than 1024 threads each can take at once
  return many || p.max_blocks <= NARROW ? select<128, true>(p, ws, stream) : select<1024, true>(p, ws, stream);
}

}  // namespace

#ifdef ATTN_TEST_DROP_COPY
extern "C" int attn_test_drop_copy_select(int what) {
  return static_cast<int>(cudaMemcpyToSymbol(g_test_drop_copy_select, &what, sizeof(int)));
}
#endif

size_t select_blocks_workspace_bytes(int64_t T, int64_t N, int64_t max_q, int64_t Hkv, int d, int64_t max_blocks) {
  // (for any number of rows: the SMALL form takes no more)
  const int RT = d == 256 ? ManyCfg<256, false>::RT : ManyCfg<128, false>::RT;
  static_assert(ManyCfg<64, false>::RT == ManyCfg<128, false>::RT, "one size for both");
  const int64_t images = max_q <= FEW ? 0 : tile_place(T, N, 1, RT);
  return up256(T * Hkv * score_stride(max_blocks) * 4) + up256(T * Hkv * 4) + up256(N * Hkv * ((max_blocks + 15) / 16) * 4) +
         images * Hkv * RT * 8 * d;
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
  at += up256(static_cast<size_t>(p.N) * p.Hkv * ws.tiles * 4);
  ws.images = at;
  if (p.d == 64) return launch<64>(p, ws, stream);
  if (p.d == 128) return launch<128>(p, ws, stream);
  if (p.d == 256) return launch<256>(p, ws, stream);
  return cudaErrorInvalidValue;
}

cudaError_t select_blocks_status(uint32_t* out, bool clear) { return read_status(g_select_blocks_status, out, clear); }

}  // namespace attn
