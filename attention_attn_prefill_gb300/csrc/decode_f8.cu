// Attention over the 8-bit paged cache (format and layout: cache_f8.cuh), for single tokens: over all blocks of a
// sequence, or over a list of blocks that each query and KV head names.
//
// A page's keys are k = 2^a c and its values v = 2^b c with one exponent each, so the codes themselves are the
// operands: score = 2^a (q . c), and the values' exponent joins the probability's, p 2^b = 2^(score + b - reference).
// An e4m3 code is an fp16 number exactly, two to a conversion instruction.  The queries become fp16 by a power of two
// a head, which puts the largest channel at 2^14 .. 2^15: their 8 bits are kept down to 2^-28 of it.  p 2^b enters the
// product with V as fp16: 11 bits, off by 2^-12 at most, an eighth of the output's own rounding.  Its reference is
// one of its own, apart from the sum's, and moves with the largest p 2^b of a step: what fp16 drops is below 2^-22 of
// the largest weight times scale that the sequence has had in this warp.
//
// Both products have the codes as the left operand, S^T = K Q^T and O^T = V^T P^T, and 8 columns hold the query heads
// of a KV head.  With P = 2 a step takes two pages and the columns hold up to four heads of both, so that one round
// of exponentials and roundings serves both; a page's product with V has zeros in the other page's columns.
//
// Work: the (sequence, unit, step) list is cut into contiguous shares of equal weight, one a CTA (decode_shares.cuh),
// or where they are short a CTA takes each row and unit whole; the CTA's computing warps deal its steps among
// themselves.  One more warp requests the records (one bulk copy each) into the warps' rings, and merges the warps'
// states of a sequence when all have left it, so that the computing warps never wait for each other; the last sequence's
// states, behind which there is no work to hide the merge, all warps merge.  Where a share's
// end cuts a sequence, the CTA leaves a partial, which a second kernel, launched as a programmatic dependent, merges.
// With listed blocks a query token is what a sequence is otherwise, each of its units has the steps that the list's
// width takes, and the loading warp says how many tokens of each page the query sees.
//
// Bound by reading the records.  Measured (GB300, calls in a captured graph, copy rate 6796 GB/s): 64 sequences of 512
// to 8192, 32/8 heads, d = 128, 96.2 us, 5.96 TB/s; 8 of 6335 to 122863, 16/2 heads, d = 256, 87.3 us, 6.08 TB/s.  The
// kernel itself reads at 6.1 TB/s with 31% of the issue slots used; start, merge and CTAs that end earlier than others
// are the rest.  64 listed blocks of each row and head, 133 MB: 27.1 us, 4.92 TB/s, a CTA each; 1 sequence of 1009 8.6 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache_f8.cuh"
#include "decode_shares.cuh"
#include "sm103.cuh"
#include "step.h"

namespace attn {

__device__ uint32_t g_decode_f8_status;

#ifdef ATTN_TEST_DROP_COPY
// Test-only builds (never the product library), in the CTA that begins sequence 0: 1: the loading warp leaves out
// its first copy; 2: it leaves at once.  The waits for what is then missing run out after ATTN_WAIT_LIMIT_NS.
__device__ int g_test_drop_copy_f8;
#endif

namespace {

using f8::Record;
using namespace shares;

constexpr uint32_t FULL = 0xffffffffu;
constexpr int SEGMENT = 10;            // steps that starting on a (sequence, unit) and leaving it cost
constexpr float P_LIMIT = 1073741824.f;  // a probability above 2^30 moves the sum's reference to the maximum
constexpr float W_LIMIT = 16384.f;     // a weight p 2^b above 2^14 moves the output's reference ...
constexpr float W_ROOM = 8.f;          // ... to where the largest is 2^8: fp16 keeps 11 bits down to 2^-14
constexpr uint32_t Q_TOP = 14;         // a head's largest channel is put at 2^14 .. 2^15

// How the list is dealt out.  SHARES: equal shares of it, one a CTA, and a second kernel that merges what a share's end
// cuts.  Else a CTA takes all steps of one row and unit: ALONE with as many warps as an SM holds, WHOLE with the warps of
// a share, MANY with fewer, so that more CTAs fit.
enum Deal { SHARES, WHOLE, ALONE, MANY };

// P: pages a warp takes at a step; ROWS / P query heads.
template <int D, int P, int DEAL>
struct Cfg {
  // Warps that compute (one more loads), steps in flight a warp, and CTAs an SM: what shared memory holds.  SHARES, measured
  // in one series (in which the form that is used took 98.8 us; by itself it takes 96 to 97) on 64 sequences of 512 to 8192, 32/8
  // heads, d = 128, warps x steps x CTAs: 5 x 2 x 2 (used) 98.8 us, 3 x 2 x 3 100.4, 4 x 3 x 2
  // 103.9, 11 x 2 x 1 102.7 (more in flight is no faster), one page a step 7 x 2 x 2 100.6.  64 of 8704, d = 64, 64/8
  // heads: 5 x 3 x 3 116.3, 3 x 3 x 5 (FINE) 109.7; with 32/8 heads, two pages a step, 104.0 and 105.6.  64 of 512 to 8192,
  // 64/8 heads, d = 128: 7 x 2 x 2 105.0, 3 x 2 x 4 102.4, 3 x 3 x 4 101.0; MANY's 512 lists of 64 blocks with two steps
  // in flight 29.0, with three 27.9.
  static constexpr bool FINE = DEAL == SHARES && D <= 128 && P == 1;
  static constexpr int NW = DEAL == ALONE  ? (D == 256 ? 8 : D == 128 && P == 2 ? 11 : 13)
                            : DEAL == MANY || FINE ? (D == 256 ? 2 : 3)
                                                   : (D == 256 ? 4 : D == 128 && P == 1 ? 7 : 5);
  static constexpr int DEPTH = D == 64 || FINE || (DEAL == MANY && D == 128 && P == 1) ? 3 : 2;
  static constexpr int CTAS = DEAL == ALONE ? 1 : DEAL == MANY || FINE ? (D == 64 ? 5 : 4) : D == 64 ? 3 : 2;
  static constexpr int THREADS = (NW + 1) * 32;
  static constexpr int TILE = ROWS / P;  // query heads a tile
  static constexpr int SLOTS = NW * DEPTH;
  static constexpr int STAGE = (P * Record<D>::BYTES + 127) & ~127;
  static constexpr int OROW = D + 8;  // floats of a row in the merge buffer
  static constexpr int MERGE = 2 * ROWS + TILE * OROW;  // floats a warp: m, l, o
  static constexpr int MERGE_OFF = SLOTS * STAGE;
  static constexpr int BAR_OFF = MERGE_OFF + NW * MERGE * 4;
  static constexpr int ALLOC = BAR_OFF + (2 * SLOTS + 2) * 8;
  static_assert(CTAS * (ALLOC + 1024 + (DEAL == SHARES ? 24 * THREADS : 384)) <= 228 * 1024, "shared memory budget");
};

// 64-bit division costs over a hundred instructions, and the lists of all but the largest batches are counted in 32 bits
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if ((a | b) >> 32 == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Sequence of query row r (-1: none) and the tokens that it sees.
struct RowInfo {
  int n, seen;
};
__device__ __forceinline__ RowInfo row_info(const DecodeF8Params& p, int r) {
  RowInfo x{r, 0};
  int behind = 0;  // query tokens of the sequence behind this one
  // where each sequence has one row, row r is sequence r's: its length is read along with cu, not behind it
  const int guess = r < p.N ? clamped_len(p.seq_lens, r, p.max_blocks) : 0;
  if (p.cu != nullptr) {
    const int n = sequence_of(p.cu, p.N, r), end = p.cu[n + 1];
    x.n = p.cu[n] <= r && r < end ? n : -1;
    behind = end - 1 - r;
  }
  if (x.n >= 0) {
    const int seen = (x.n == r ? guess : clamped_len(p.seq_lens, x.n, p.max_blocks)) - behind;
    x.seen = seen > 0 ? seen : 0;
  }
  return x;
}

// Position in the list: of sequences' pages, or of query rows whose units all have `ns` steps.
template <int P, bool LISTED>
struct At : Cursor<P> {
  __device__ __forceinline__ void begin(const DecodeF8Params& p, int n, int u, int step) {
    this->n = n;
    this->u = u;
    this->step = step;
    if constexpr (LISTED) this->ns = (p.K + P - 1) / P;
    else this->enter(p.seq_lens, p.max_blocks);
  }
  __device__ __forceinline__ void go(int by, const DecodeF8Params& p, int units) {
    if constexpr (LISTED) {
      this->step += by;
      while (this->step >= this->ns) {
        this->step -= this->ns;
        if (++this->u == units) {
          this->u = 0;
          ++this->n;
        }
      }
    } else {
      this->advance(by, p.seq_lens, p.N, units, p.max_blocks);
    }
  }
};

template <int D, int P, bool LISTED, int DEAL>
__global__ void __launch_bounds__(Cfg<D, P, DEAL>::THREADS, Cfg<D, P, DEAL>::CTAS)
    decode_f8_kernel(const DecodeF8Params p, const Geometry geo) {
  using C = Cfg<D, P, DEAL>;
  using R = Record<D>;
  constexpr int NW = C::NW, THREADS = C::THREADS, TILE = C::TILE, SLOTS = C::SLOTS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_weight[NW + 1], s_steps[NW + 1], s_end[2], s_at;
  __shared__ longlong2 s_before[LISTED || DEAL != SHARES ? 1 : THREADS];  // weight and steps of the warp's sequences before a thread's
  __shared__ int3 s_start;
  __shared__ int s_valid[SLOTS][P];  // listed blocks: tokens of each page of a slot that the query sees
  float* merge = reinterpret_cast<float*>(smem + C::MERGE_OFF);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + SLOTS;
  uint64_t* rec_full = empty + SLOTS;  // every computing warp's state of a segment is in the merge buffer
  uint64_t* rec_free = rec_full + 1;   // the loading warp has read them
  const int warp = __shfl_sync(FULL, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, units = geo.units;
  const int rows = LISTED ? p.T : p.N;  // of the list

  if (threadIdx.x < SLOTS) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], 1);
    if (threadIdx.x == 0) {
      mbar_init(rec_full, NW);
      mbar_init(rec_free, 1);
    }
    fence_mbar_init();
  }
  // The list is cut by weight: a (row, unit) weighs its steps and SEGMENT more, what starting on it and
  // leaving its result cost.  Short lists make fewer shares than CTAs: of one step, they would only be more partials to
  // merge.  Share b is the weight from b * per on.
  const int b = blockIdx.x;
  long long W = 0, per = 1;
  auto cut_list = [&](long long steps) {
    const long long most = steps / 2, shares = most >= geo.grid ? geo.grid : most < 1 ? 1 : most;
    per = quotient(W + shares - 1, shares);
  };
  auto check_lens = [&]() {
    for (int n = threadIdx.x; n < p.N; n += THREADS) {
      const int L = p.seq_lens[n];
      if (L < 0 || L > p.max_blocks * PAGE) set_error(&g_decode_f8_status, kDevBadSplit);
      if (p.cu != nullptr) {
        const int c0 = p.cu[n], c1 = p.cu[n + 1];
        if (c0 < 0 || c1 < c0 || c1 > p.T) set_error(&g_decode_f8_status, kDevBadSeqlens);
      }
    }
  };
  if constexpr (DEAL != SHARES) {
    if (b == 0) check_lens();
    if (threadIdx.x == 0) {
      const int row = b / units;
      s_start = make_int3(row, b - row * units, 0);
      s_at = 0;
      s_end[0] = 0;
      s_end[1] = LISTED ? (p.K + P - 1) / P : steps_of<P>(p.seq_lens, row, p.max_blocks);
    }
  } else if constexpr (LISTED) {
    const int S = (p.K + P - 1) / P;
    const long long pairs = static_cast<long long>(rows) * units;
    W = pairs * (S + SEGMENT);
    cut_list(pairs * S);
    if (threadIdx.x < 2) {
      const long long x = per * (b + threadIdx.x) < W ? per * (b + threadIdx.x) : W;
      const long long pair = quotient(x, S + SEGMENT);
      const int in = static_cast<int>(x - pair * (S + SEGMENT)), step = in > SEGMENT ? in - SEGMENT : 0;
      s_end[threadIdx.x] = pair * S + step;  // steps before x
      if (threadIdx.x == 0) {
        const int row = static_cast<int>(quotient(pair, units));
        s_start = make_int3(row, static_cast<int>(pair - static_cast<long long>(row) * units), step);
        s_at = pair * (S + SEGMENT);
      }
    }
    if (b == 0) check_lens();
  } else {
    // ---- total steps, and the sequence that holds this share's first one
    const int N = p.N;
    const int chunk = (N + THREADS - 1) / THREADS;  // sequences a thread counts
    const int n_lo = static_cast<int>(threadIdx.x) * chunk < N ? threadIdx.x * chunk : N;
    const int n_hi = n_lo + chunk < N ? n_lo + chunk : N;
    long long my_weight = 0, my_steps = 0;
    for (int n = n_lo; n < n_hi; ++n) {
      const int L = p.seq_lens[n];
      if (b == 0 && (L < 0 || L > p.max_blocks * PAGE)) set_error(&g_decode_f8_status, kDevBadSplit);
      const int ns = steps_of<P>(p.seq_lens, n, p.max_blocks);
      my_steps += ns;
      my_weight += ns > 0 ? ns + SEGMENT : 0;
    }
    long long to_weight = my_weight, to_steps = my_steps;  // inclusive sums
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long a = __shfl_up_sync(FULL, to_weight, off), c = __shfl_up_sync(FULL, to_steps, off);
      if (lane >= off) {
        to_weight += a;
        to_steps += c;
      }
    }
    s_before[threadIdx.x] = make_longlong2(to_weight - my_weight, to_steps - my_steps);
    if (lane == 31) {
      s_weight[warp] = to_weight;
      s_steps[warp] = to_steps;
    }
    __syncthreads();
    long long weight = 0, steps = 0;
#pragma unroll
    for (int i = 0; i < NW + 1; ++i) {
      weight += s_weight[i];
      steps += s_steps[i];
    }
    W = weight * units;
    cut_list(steps * units);
    if (warp < 2) {  // where the share begins (warp 0) and ends
      const long long x = per * (b + warp);
      if (x >= W) {
        if (lane == 0) s_end[warp] = steps * units;
      } else {
        // the last warp, and of it the last thread, whose sequences begin at or before x
        long long at = 0, before = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          if ((at + s_weight[i]) * units > x) break;
          at += s_weight[i];
          before += s_steps[i];
        }
        int v = 0;
        long long upto = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          upto += s_weight[i];
          v += upto * units <= x ? 1 : 0;
        }
        const longlong2 mine = s_before[v * 32 + lane];
        const int u = 31 - __clz(__ballot_sync(FULL, (at + mine.x) * units <= x));
        at = (at + __shfl_sync(FULL, mine.x, u)) * units;
        before = (before + __shfl_sync(FULL, mine.y, u)) * units;
        int n = (v * 32 + u) * chunk, ns = 0;
        for (;; ++n) {
          ns = steps_of<P>(p.seq_lens, n, p.max_blocks);
          const long long w = ns > 0 ? static_cast<long long>(ns + SEGMENT) * units : 0;
          if (x < at + w) break;
          at += w;
          before += static_cast<long long>(ns) * units;
        }
        const int unit = static_cast<int>(quotient(x - at, ns + SEGMENT));
        const int in = static_cast<int>(x - at - static_cast<long long>(unit) * (ns + SEGMENT));
        const int step = in > SEGMENT ? in - SEGMENT : 0;
        if (lane == 0) {
          s_end[warp] = before + static_cast<long long>(unit) * ns + step;  // steps before x
          if (warp == 0) {
            s_start = make_int3(n, unit, step);
            s_at = at + static_cast<long long>(unit) * (ns + SEGMENT);
          }
        }
      }
    }
    // empty sequences: this CTA's part of them
    for (int n = b; n < N; n += gridDim.x) {
      if (p.seq_lens[n] > 0) continue;
      for (int i = threadIdx.x; i < p.Hq * (D / 8); i += THREADS)
        reinterpret_cast<uint4*>(p.o + static_cast<int64_t>(n) * p.Hq * D)[i] = make_uint4(0, 0, 0, 0);
      if (p.lse != nullptr)
        for (int i = threadIdx.x; i < p.Hq; i += THREADS) p.lse[static_cast<int64_t>(n) * p.Hq + i] = -INFINITY;
    }
  }
  __syncthreads();
  // every CTA of this grid is resident: the combine's CTAs may queue up behind them
  if constexpr (DEAL == SHARES) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Workspace ws = carve<D>(p.workspace, geo.grid);
  const int count = static_cast<int>(s_end[1] - s_end[0]);  // steps of this share
  if (count <= 0) {
    if constexpr (DEAL != SHARES) {  // an empty sequence
      const int kvh = s_start.y / geo.tiles, h0 = s_start.y % geo.tiles * TILE, heads = min(TILE, G - h0);
      const int64_t row = static_cast<int64_t>(s_start.x) * p.Hq + kvh * G + h0;
      for (int i = threadIdx.x; i < heads * (D / 8); i += THREADS)
        reinterpret_cast<uint4*>(p.o + row * D)[i] = make_uint4(0, 0, 0, 0);
      if (p.lse != nullptr && threadIdx.x < heads) p.lse[row + threadIdx.x] = -INFINITY;
    } else if (threadIdx.x == 0 && !geo.by_unit) {
      ws.desc[b] = make_int4(0, 0, -1, 0);
    }
    return;
  }

  // The warps' states of a segment, left in the merge buffer, become a result or a partial: threads `first` of `of`
  auto merge_states = [&](int n, int u, bool starts, bool ends, bool lives, int first, int of) {
    const int kvh = u / geo.tiles, h0 = u % geo.tiles * TILE;
    const int heads = G - h0 < TILE ? G - h0 : TILE;
    const int64_t part = 2 * static_cast<int64_t>(b) + (starts ? 1 : 0);
    // four at a time: one alone would wait for its loads (d = 256, 8 heads, by one warp: 9700 cycles one by one)
    constexpr int AT_ONCE = 4;
    for (int w0 = first; w0 < heads * (D / 4); w0 += of * AT_ONCE) {
      float M[AT_ONCE], L[AT_ONCE];
      float4 O[AT_ONCE];
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        const int w = w0 + of * k, r = w < heads * (D / 4) ? w / (D / 4) : 0, x = w % (D / 4) * 4;
        M[k] = -INFINITY;
#pragma unroll
        for (int v = 0; v < NW; ++v) M[k] = fmaxf(M[k], merge[v * C::MERGE + r]);
        L[k] = 0.f;
        O[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < NW; ++v) {
          const float* src = merge + v * C::MERGE;
          const float l = src[ROWS + r];
          const float wl = l == 0.f ? 0.f : l * ex2_approx(src[r] - M[k]);  // 0: a warp without tokens
          const float4 y = *reinterpret_cast<const float4*>(src + 2 * ROWS + r * C::OROW + x);
          L[k] += wl;
          O[k].x = fmaf(y.x, wl, O[k].x); O[k].y = fmaf(y.y, wl, O[k].y);
          O[k].z = fmaf(y.z, wl, O[k].z); O[k].w = fmaf(y.w, wl, O[k].w);
        }
        const float inv = L[k] == 0.f ? 0.f : 1.f / L[k];
        O[k].x *= inv; O[k].y *= inv; O[k].z *= inv; O[k].w *= inv;
      }
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        const int w = w0 + of * k, r = w / (D / 4), x = w % (D / 4) * 4;
        if (w >= heads * (D / 4)) break;
        if (DEAL != SHARES || (starts && ends)) {
          if (lives) {
            const int64_t row = static_cast<int64_t>(n) * p.Hq + kvh * G + h0 + r;
            *reinterpret_cast<uint2*>(p.o + row * D + x) = make_uint2(pack_bf16x2(O[k].x, O[k].y), pack_bf16x2(O[k].z, O[k].w));
            if (x == 0 && p.lse != nullptr) p.lse[row] = (M[k] + log2f(L[k])) * LN2;
          }
        } else {
          *reinterpret_cast<float4*>(ws.o + (part * ROWS + r) * D + x) = O[k];
          if (x == 0) {
            ws.m[part * ROWS + r] = M[k];
            ws.l[part * ROWS + r] = L[k];
          }
        }
      }
    }
  };

  At<P, LISTED> cur;  // the share's first step
  cur.begin(p, s_start.x, s_start.y, s_start.z);

  if (warp == NW) {
    // ---------------------------------------------------------- loads, and results
    // Lane w serves computing warp w: step i of the share belongs to warp i % NW and goes through that
    // warp's ring.  The lanes poll their rings together, so that no warp waits for another's slot, and
    // each reads the block table a step ahead of the copy that needs it.  When all warps have left
    // their states of a segment (the share's part of a row and unit), this warp merges them and
    // writes the result, while the others are at the next segment.
    bool ok = true;
    At<P, LISTED> seg = cur;  // the segment to merge next ...
    long long at = s_at;      // ... the weight before its (row, unit) ...
    int seg_i = 0;            // ... its first step's share index
    uint32_t seg_phase = 0;
    int4 cut = make_int4(0, 0, -1, 0);
    int i = lane;  // this lane's next step, with the pages' table entries and the tokens that are seen of them
    int ids[P] = {}, seen[P] = {};
    int listed[P] = {};           // listed blocks: the entries of the step behind, read a step ahead of their pages
    At<P, LISTED> behind = cur;
    int stage_k = 0;
    uint32_t phase = 1;  // a slot's first use waits for nothing
    int info_row = -1;
    RowInfo info{-1, 0};
    auto read_list = [&]() {  // entries of step `behind`
      const int32_t* list = p.blocks + (static_cast<int64_t>(behind.n) * p.Hkv + behind.u / geo.tiles) * p.K + behind.step * P;
#pragma unroll
      for (int a = 0; a < P; ++a) listed[a] = behind.step * P + a < p.K ? list[a] : -1;
    };
    // step `cur`: its pages and what is seen of them; `more`: another step of this lane follows
    auto fetch = [&](bool more) {
      if constexpr (LISTED) {
        if (info_row != cur.n) {
          info = row_info(p, cur.n);
          info_row = cur.n;
        }
#pragma unroll
        for (int a = 0; a < P; ++a) {
          seen[a] = 0;
          const int blk = info.n >= 0 ? listed[a] : -1;
          if (blk < 0 || blk >= p.max_blocks || blk * PAGE >= info.seen) continue;
          seen[a] = info.seen - blk * PAGE < PAGE ? info.seen - blk * PAGE : PAGE;
          ids[a] = p.block_table[static_cast<int64_t>(info.n) * p.max_blocks + blk];
        }
        if (more) {
          behind.go(NW, p, units);
          read_list();
        }
      } else {
        const int32_t* row = p.block_table + static_cast<int64_t>(cur.n) * p.max_blocks + cur.step * P;
        seen[0] = PAGE;
        ids[0] = row[0];
        if (P == 2) {
          seen[P - 1] = cur.step * P + 1 < cur.pages ? PAGE : 0;
          if (seen[P - 1] > 0) ids[P - 1] = row[1];
        }
      }
    };
    const bool serves = lane < NW;
    if (serves && i < count) {
      if (lane > 0) cur.go(lane, p, units);
      if constexpr (LISTED) {
        behind = cur;
        read_list();
      }
      fetch(i + NW < count);
    }
    uint64_t since = global_timer_ns();
#ifdef ATTN_TEST_DROP_COPY
    const int drop = s_start.x == 0 && s_start.y == 0 && s_start.z == 0 ? g_test_drop_copy_f8 : 0;
    ok = drop != 2;
#endif
    while (ok && seg_i < count) {
      const int slot = lane + NW * stage_k;
      const bool go = serves && i < count && mbar_test_wait(&empty[slot], phase);
      if (go) {
        int pages = 0;
#pragma unroll
        for (int a = 0; a < P; ++a) {
          pages += seen[a] > 0 ? 1 : 0;
          if constexpr (LISTED) s_valid[slot][a] = seen[a];
        }
        if (pages > 0) mbar_arrive_expect_tx(&full[slot], pages * R::BYTES);
        else mbar_arrive(&full[slot]);
#pragma unroll
        for (int a = 0; a < P; ++a) {
          if (seen[a] == 0) continue;
          int id = ids[a];
          if (id < 0 || id >= p.num_blocks) {
            set_error(&g_decode_f8_status, kDevBadPage);
            id = 0;
          }
#ifdef ATTN_TEST_DROP_COPY
          if (drop == 1 && i == 0) continue;
#endif
          bulk_load(smem + slot * C::STAGE + a * R::BYTES,
                    p.cache + (static_cast<int64_t>(id) * p.Hkv + cur.u / geo.tiles) * R::BYTES, R::BYTES, &full[slot]);
        }
        if (++stage_k == C::DEPTH) {
          stage_k = 0;
          phase ^= 1;
        }
        i += NW;
        if (i < count) {
          cur.go(NW, p, units);
          fetch(i + NW < count);
        }
      }
      const bool merge_now = __all_sync(FULL, mbar_test_wait(rec_full, seg_phase));
      if (merge_now) {
        seg_phase ^= 1;
        const int seg_steps = seg.ns - seg.step < count - seg_i ? seg.ns - seg.step : count - seg_i;
        const bool starts = seg.step == 0, ends = seg.step + seg_steps == seg.ns;
        // a row of no sequence has no result
        const bool lives = !LISTED || p.cu == nullptr || row_info(p, seg.n).n >= 0;
        // the last segment's states are merged by the warps that left them
        if (seg_i + seg_steps < count) merge_states(seg.n, seg.u, starts, ends, lives, lane, 32);
        __syncwarp();
        if (lane == 0) mbar_arrive(rec_free);
        if (starts && !ends && lives) {
          // the share that holds the last step
          cut = make_int4(seg.n, seg.u, b, static_cast<int>(quotient(at + SEGMENT + seg.ns - 1, per)));
        }
        if (DEAL == SHARES && geo.by_unit && starts && lane == 0)
          ws.desc[static_cast<int64_t>(seg.n) * units + seg.u] = ends || !lives ? make_int4(0, 0, -1, 0) : cut;
        at += SEGMENT + seg.ns;
        seg_i += seg_steps;
        if (seg_i < count) seg.go(seg_steps, p, units);
      }
      if (__any_sync(FULL, go) || merge_now) {
        since = global_timer_ns();
      } else {
        __nanosleep(50);
        ok = __all_sync(FULL, global_timer_ns() - since < ATTN_WAIT_LIMIT_NS);
      }
    }
    if (lane == 0) {
      if (DEAL == SHARES && !geo.by_unit) ws.desc[b] = cut;
      if (!ok) set_error(&g_decode_f8_status, kDevWaitTimeout);
    }
    // Copies in flight must land before the CTA's shared memory is given back: the newest of each slot.
    const int issued = serves ? (i - lane) / NW : 0;
    for (int k = issued > C::DEPTH ? issued - C::DEPTH : 0; k < issued; ++k)
      mbar_wait(&full[lane + NW * (k % C::DEPTH)], k / C::DEPTH & 1);
    return;
  }

  // ------------------------------------------------------------ attention
  const int g = lane >> 2, t = lane & 3;
  const int q_row = P == 2 ? g & 3 : g;     // the query head of the tile that this lane loads: column g
  const int my_page = P == 2 ? t >> 1 : 0;  // columns 2 t and 2 t + 1 are two heads of this page of the step
  bool ok = true;
  int i = warp;        // share index of this warp's next step
  int stage_k = 0;     // its ring stage: slot warp + NW stage_k ...
  uint32_t phase = 0;  // ... and the parity of that slot's barriers
  uint32_t free_phase = 0, seg_index = 0;
  for (int seg = 0; seg < count;) {
    const int seg_n = cur.n, seg_u = cur.u, first_step = cur.step;
    const int seg_steps = cur.ns - first_step < count - seg ? cur.ns - first_step : count - seg;
    const int seg_end = seg + seg_steps;
    const int len = LISTED ? 0 : clamped_len(p.seq_lens, seg_n, p.max_blocks);
    const int kvh = seg_u / geo.tiles, h0 = seg_u % geo.tiles * TILE;
    const int heads = G - h0 < TILE ? G - h0 : TILE;
    const __nv_bfloat16* q_head = p.q + (static_cast<int64_t>(seg_n) * p.Hq + kvh * G + h0) * D;
    // for the merge of the last segment, asked here, while the first records are on their way
    const bool lives = !LISTED || p.cu == nullptr || seg_end < count || row_info(p, seg_n).n >= 0;

    // ---- queries: channels 64 j + 16 t + 4 s .. + 3, in the order of the K words
    uint32_t qb[R::KJ][4][2];
    int q_exp[2];  // the power that columns 2 t and 2 t + 1 were multiplied by
    {
      uint32_t most2 = 0;
#pragma unroll
      for (int j = 0; j < R::KJ; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (q_row < heads) x = *reinterpret_cast<const uint4*>(q_head + q_row * D + 64 * j + 16 * t + 8 * e);
          qb[j][2 * e][0] = x.x; qb[j][2 * e][1] = x.y; qb[j][2 * e + 1][0] = x.z; qb[j][2 * e + 1][1] = x.w;
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t lo = w[k] & 0x7fffu, hi = w[k] >> 16 & 0x7fffu;
            most2 = max(most2, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));  // what is finite
          }
        }
      most2 = max(most2, __shfl_xor_sync(FULL, most2, 1));
      most2 = max(most2, __shfl_xor_sync(FULL, most2, 2));
      const int biased = min(254, 254 + static_cast<int>(Q_TOP) - static_cast<int>(most2 >> 7));
      const float f = f8::pow2(biased);
#pragma unroll
      for (int j = 0; j < R::KJ; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w = qb[j][s][k];
            qb[j][s][k] = pack_f16x2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
          }
      q_exp[0] = __shfl_sync(FULL, biased, 8 * t) - 127;
      q_exp[1] = __shfl_sync(FULL, biased, 8 * t + 4) - 127;
    }

    float mc[2] = {-1e38f, -1e38f};  // of columns 2 t, 2 t + 1, in log2 units: the reference of the sum ...
    float mo[2] = {-1e38f, -1e38f};  // ... and of the output
    float l[2] = {0.f, 0.f};         // this lane's share of the sum of probabilities
    float o[D / 16][4];  // channels B g + 2 x (0, 1) and + 1 (2, 3) of columns 2 t and 2 t + 1
#pragma unroll
    for (int x = 0; x < D / 16; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;

    for (; i < seg_end; i += NW) {
      const int slot = warp + NW * stage_k;
      ok = ok && __all_sync(FULL, mbar_wait(&full[slot], phase));
      if (++stage_k == C::DEPTH) {
        stage_k = 0;
        phase ^= 1;
      }
      if (!ok) continue;
      const uint8_t* stage = smem + slot * C::STAGE;
      // ---- S^T: rows are tokens g (0, 1) and g + 8 (2, 3), columns 2 t and 2 t + 1
      float acc[P][2][4];
#pragma unroll
      for (int a = 0; a < P; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) acc[a][e][0] = acc[a][e][1] = acc[a][e][2] = acc[a][e][3] = 0.f;
#pragma unroll
      for (int j = 0; j < R::KJ; ++j) {
        uint32_t kw[P][2][4];
#pragma unroll
        for (int a = 0; a < P; ++a)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint4 x = *reinterpret_cast<const uint4*>(stage + a * R::BYTES + R::K_OFF + (e * R::KJ + j) * 512 + lane * 16);
            kw[a][e][0] = x.x; kw[a][e][1] = x.y; kw[a][e][2] = x.z; kw[a][e][3] = x.w;
          }
        // consecutive products go to different accumulators: each would wait for the one before otherwise
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int a = 0; a < P; ++a)
            mma_16816<true>(acc[a][s & 1], f8::halves2(kw[a][0][s]), f8::halves2(kw[a][1][s]),
                            f8::halves2_upper(kw[a][0][s]), f8::halves2_upper(kw[a][1][s]), qb[j][s][0], qb[j][s][1]);
      }
      const float2 scales = *reinterpret_cast<const float2*>(stage + my_page * R::BYTES + R::S_OFF);
      const int k_exp = __float_as_uint(scales.x) >> 23;
      const float v_exp = static_cast<float>(static_cast<int>(__float_as_uint(scales.y) >> 23) - 127);
      float sc[4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float f = p.scale_log2 * f8::pow2(min(254, max(1, k_exp - q_exp[c])));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x0 = acc[0][0][2 * e + c] + acc[0][1][2 * e + c];
          const float x1 = acc[P - 1][0][2 * e + c] + acc[P - 1][1][2 * e + c];
          sc[2 * e + c] = (P == 2 && my_page ? x1 : x0) * f;
        }
      }
      // tokens of this lane's page that the query sees; the last step's second page may have none
      int valid[P];
#pragma unroll
      for (int a = 0; a < P; ++a) {
        if constexpr (LISTED) valid[a] = s_valid[slot][a];
        else valid[a] = len - ((first_step + i - seg) * P + a) * PAGE;
      }
      const bool whole = valid[0] >= PAGE && valid[P - 1] >= PAGE;
      if (!whole) {
        const int mine = P == 2 && my_page ? valid[P - 1] : valid[0];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (g + 8 * e >= mine) sc[2 * e] = sc[2 * e + 1] = -INFINITY;
      }
      // ---- online softmax against the references; a number past its limit moves them
      float pr[4], w[4];
      float mv[2] = {mo[0] - v_exp, mo[1] - v_exp};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        pr[x] = ex2_approx(sc[x] - mc[x & 1]);
        w[x] = ex2_approx(sc[x] - mv[x & 1]);
      }
      if (__any_sync(FULL, fmaxf(fmaxf(pr[0], pr[1]), fmaxf(pr[2], pr[3])) > P_LIMIT ||
                               fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])) > W_LIMIT)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(sc[c], sc[2 + c]);
          float mw = mx + v_exp;
#pragma unroll
          for (int off = P == 2 ? 2 : 4; off < 32; off <<= 1) {  // with two pages, a head's two columns share them
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, off));
            mw = fmaxf(mw, __shfl_xor_sync(FULL, mw, off));
          }
          const float to = fmaxf(mc[c], mx), f = ex2_approx(mc[c] - to);
          mc[c] = to;
          l[c] *= f;
          const float to_o = fmaxf(mo[c], mw - W_ROOM), fo = ex2_approx(mo[c] - to_o);
          mo[c] = to_o;
          mv[c] = to_o - v_exp;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            o[x][c] *= fo;
            o[x][2 + c] *= fo;
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          pr[x] = ex2_approx(sc[x] - mc[x & 1]);
          w[x] = ex2_approx(sc[x] - mv[x & 1]);
        }
      }
      l[0] += pr[0] + pr[2];
      l[1] += pr[1] + pr[3];
      // ---- O^T += V^T (p 2^b)^T
      const uint32_t pb0 = transpose_8x8(pack_f16x2(w[0], w[1])), pb1 = transpose_8x8(pack_f16x2(w[2], w[3]));
#pragma unroll
      for (int a = 0; a < P; ++a) {
        const bool on = P == 1 || (g >> 2) == a;  // as an operand, this lane holds column g
        const uint32_t b0 = on ? pb0 : 0u, b1 = on ? pb1 : 0u;
        uint32_t vw[R::VH][4][R::VB / 4];
#pragma unroll
        for (int h = 0; h < R::VH; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint8_t* from = stage + a * R::BYTES + R::V_OFF + ((k * R::VH + h) * 32 + lane) * R::VB;
            if constexpr (R::VB == 16) {
              const uint4 x = *reinterpret_cast<const uint4*>(from);
              vw[h][k][0] = x.x; vw[h][k][1] = x.y; vw[h][k][2] = x.z; vw[h][k][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(from);
              vw[h][k][0] = x.x; vw[h][k][1] = x.y;
            }
          }
        if (!whole) {  // whatever lies past the sequence is not to be multiplied with: 0 * NaN is not 0
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (8 * (k >> 1) + 2 * t + (k & 1) >= valid[a]) {
#pragma unroll
              for (int h = 0; h < R::VH; ++h)
#pragma unroll
                for (int x = 0; x < R::VB / 4; ++x) vw[h][k][x] = 0u;
            }
        }
#pragma unroll
        for (int h = 0; h < R::VH; ++h)
#pragma unroll
          for (int x = 0; x < R::VB / 2; ++x) {
            // tokens 2 t, 2 t + 1 and 2 t + 8, + 9 of channels 2 x (lower half) and 2 x + 1
            const uint32_t pick = x % 2 ? 0x7362 : 0x5140;
            const uint32_t u = __byte_perm(vw[h][0][x / 2], vw[h][1][x / 2], pick);
            const uint32_t v = __byte_perm(vw[h][2][x / 2], vw[h][3][x / 2], pick);
            mma_16816<true>(o[h * (R::VB / 2) + x], f8::halves2(u), f8::halves2_upper(u), f8::halves2(v),
                            f8::halves2_upper(v), b0, b1);
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
    }
    // A wait that ran out is this warp's last: waits of the others that need it run out once too, and not for
    // every segment that is left.
    if (!ok) break;

    // ---- this warp's state to shared memory, normalised, then the CTA's to global memory.  With two pages, a
    // head's sums are in columns c and c + 4, two lanes apart.
#pragma unroll
    for (int off = P == 2 ? 2 : 4; off < 32; off <<= 1) {
#pragma unroll
      for (int c = 0; c < 2; ++c) l[c] += __shfl_xor_sync(FULL, l[c], off);
    }
    if (P == 2) {
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[x][j] += __shfl_xor_sync(FULL, o[x][j], 2);
    }
    // the loading warp has merged the segment before this one
    if (seg > 0) {
      ok = __all_sync(FULL, mbar_wait(rec_free, free_phase));
      free_phase ^= 1;
      if (!ok) break;
    }
    float* my = merge + warp * C::MERGE;
    if (2 * t < TILE) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bool none = l[c] == 0.f;  // no tokens: no part in the maximum
        if (g == 0) {
          my[2 * t + c] = none ? -INFINITY : mc[c];
          my[ROWS + 2 * t + c] = l[c];
        }
        // 2^(mo - mc) in two halves: the values' scale may be near either end of the range
        const float half = ex2_approx(0.5f * (mo[c] - mc[c])), f = none ? 0.f : half / l[c];
#pragma unroll
        for (int h = 0; h < R::VH; ++h)
#pragma unroll
          for (int x = 0; x < R::VB / 2; ++x) {
            const float* y = o[h * (R::VB / 2) + x];
            *reinterpret_cast<float2*>(my + 2 * ROWS + (2 * t + c) * C::OROW + 8 * R::VB * h + R::VB * g + 2 * x) =
                make_float2(y[c] * f * half, y[2 + c] * f * half);
          }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(rec_full);
    if (seg_end == count) {  // nothing is left to do: all warps merge, in a fraction of the time that one takes
      ok = __all_sync(FULL, mbar_wait(rec_full, seg_index & 1));
      if (!ok) break;
      merge_states(seg_n, seg_u, first_step == 0, first_step + seg_steps == cur.ns, lives, warp * 32 + lane, NW * 32);
    }
    ++seg_index;
    seg = seg_end;
    if (seg < count) cur.go(seg_steps, p, units);
  }
  if (!ok && lane == 0) set_error(&g_decode_f8_status, kDevWaitTimeout);
}

int sms_of_device() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}
// CTAs of the largest grid that leaves partials, of either number of pages a step
template <int D>
constexpr int most_ctas() {
  constexpr int one = Cfg<D, 1, SHARES>::CTAS, two = Cfg<D, D == 256 ? 1 : 2, SHARES>::CTAS;
  return one > two ? one : two;
}

template <int D, int P, bool LISTED, int DEAL>
cudaError_t start(const DecodeF8Params& p, const Geometry& geo, int64_t grid, cudaStream_t stream) {
  using C = Cfg<D, P, DEAL>;
  auto kern = decode_f8_kernel<D, P, LISTED, DEAL>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::ALLOC);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(grid), C::THREADS, C::ALLOC, stream>>>(p, geo);
  return cudaGetLastError();
}

template <int D, int P, bool LISTED>
cudaError_t launch(const DecodeF8Params& p, cudaStream_t stream) {
  using C = Cfg<D, P, SHARES>;
  Geometry geo;
  const int sms = sms_of_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  geo.grid = sms * C::CTAS;  // every SM filled
  const int rows = LISTED ? p.T : p.N;
  geo.tile = C::TILE;
  geo.tiles = (p.Hq / p.Hkv + C::TILE - 1) / C::TILE;
  geo.units = p.Hkv * geo.tiles;
  const int64_t pairs = static_cast<int64_t>(rows) * geo.units;
  geo.by_unit = pairs * 8 <= geo.grid;
  // What the host knows of the lengths is the table's width, or the list's: the most pages of a row and unit.  A CTA to each
  // row and unit takes one launch instead of two, no scan of the lengths and no merge of partials, but where the last round
  // of CTAs is not a full one the GPU idles for its time: `lost`, in pages.  Measured, us, d = 128, 32/8 heads, equal lengths
  // (SHARES, ALONE, WHOLE, MANY):
  //     8 rows and units: 17 tokens 9.0 5.2 4.4 4.2, 500 8.2 6.7 7.1 7.6, 1000 8.5 8.4 9.8 10.9, 2000 9.1 12.4 15.4 17.8
  //   128: 100 tokens 8.4 5.6 4.8 5.1, 1000 13.6 8.7 10.0 11.2, 2000 19.9 16.0 19.5 24.9, 64 listed blocks 14.3 10.4 12.2 14.0
  //   256: 1000 tokens 21.0 19.7 15.6 17.6, 2000 30.7 29.0 25.2 29.0, 64 listed blocks 22.3 22.8 17.4 19.3
  //   512: 100 tokens 12.5 17.8 9.2 6.7, 1000 31.3 37.7 28.8 25.5, 2000 51.0 56.4 47.4 44.0, of 100 to 2000 32.9 36.3 33.3
  //        32.6, of 500 to 8000 93.7 98.9 109 113; 64 listed blocks 34.1 44.7 32.4 27.8, 128 54.5 65.8 52.3 47.2
  //   640: 64 listed blocks 40.2 54.6 45.1 41.7; 896: 50.9 67.7 51.0 49.4, 2000 tokens 80.1 87.5 76.0 79.5;
  //   1200: 64 listed blocks 63.5 89.3 66.9 57.8; 2400: 1000 tokens 104 142 111 99
  // A table that is wider than its sequences are long may lead to the slower side: 16 sequences of 1000 tokens take 8.6 us in a table
  // of 63 columns and 13.8 in one of 513 or more, 64 of them 25.3 and 31.
  const int64_t pages = LISTED ? p.K : p.max_blocks, steps = (pages + P - 1) / P;
  auto lost = [&](int64_t ctas) {  // with so many at a time
    const int64_t places = (pairs + ctas - 1) / ctas * ctas;
    return pages * (places - pairs) / ctas;
  };
  if (pairs <= sms && steps <= 8) return start<D, P, LISTED, WHOLE>(p, geo, pairs, stream);
  if (pairs <= sms && steps <= (LISTED ? 14 : 33) + pairs / 2) return start<D, P, LISTED, ALONE>(p, geo, pairs, stream);
  if ((LISTED || pages <= 128) && pairs < int64_t(1) << 31) {  // a table may be far wider than most of its sequences
    const int64_t fit = sms * Cfg<D, P, WHOLE>::CTAS, many = sms * Cfg<D, P, MANY>::CTAS, rounds = (pairs + many - 1) / many;
    if (pairs <= fit && lost(fit) <= (LISTED ? 56 : 45)) return start<D, P, LISTED, WHOLE>(p, geo, pairs, stream);
    if (pairs > fit && lost(many) <= 45 * (rounds > 2 ? rounds - 1 : 1))
      return start<D, P, LISTED, MANY>(p, geo, pairs, stream);
    if (pairs > fit && rounds <= 2 && lost(fit) <= 10) return start<D, P, LISTED, WHOLE>(p, geo, pairs, stream);
  }
  const cudaError_t e = start<D, P, LISTED, SHARES>(p, geo, geo.grid, stream);
  if (e != cudaSuccess) return e;
  return launch_combine<D, C::TILE>(
      MergeParams{p.workspace, p.o, p.lse, LISTED ? nullptr : p.seq_lens, rows, p.Hq, p.Hkv, p.max_blocks}, geo, stream);
}

template <int D>
cudaError_t launch_for(const DecodeF8Params& p, cudaStream_t stream) {
  if constexpr (D == 256) {
    // two pages a step do not leave room for two CTAs an SM
    return p.blocks != nullptr ? launch<D, 1, true>(p, stream) : launch<D, 1, false>(p, stream);
  } else {
    const bool pairs = p.Hq / p.Hkv <= ROWS / 2;
    if (p.blocks != nullptr) return pairs ? launch<D, 2, true>(p, stream) : launch<D, 1, true>(p, stream);
    return pairs ? launch<D, 2, false>(p, stream) : launch<D, 1, false>(p, stream);
  }
}

}  // namespace

#ifdef ATTN_TEST_DROP_COPY
extern "C" int attn_test_drop_copy_f8(int what) {
  return static_cast<int>(cudaMemcpyToSymbol(g_test_drop_copy_f8, &what, sizeof(int)));
}
#endif

size_t decode_f8_workspace_bytes(int d) {
  const int ctas = d == 64 ? most_ctas<64>() : d == 128 ? most_ctas<128>() : d == 256 ? most_ctas<256>() : 0;
  return workspace_bytes(sms_of_device() * ctas, d);
}

cudaError_t decode_f8_launch(int d, const DecodeF8Params& p, cudaStream_t stream) {
  if (d == 64) return launch_for<64>(p, stream);
  if (d == 128) return launch_for<128>(p, stream);
  if (d == 256) return launch_for<256>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t decode_f8_status(uint32_t* out, bool clear) { return read_status(g_decode_f8_status, out, clear); }

}  // namespace attn
