// Single-token attention over the 4-bit paged cache (format and layout: cache_q4.cuh).
//
// With K = s_g (c - z_g) and V likewise, per group g of 64 channels,
//   score = sum_g s_g (q . c - z_g sum q),     O = sum_tokens p s c - sum_tokens p s z,
// so the codes themselves are the matrix operands, and scales and zero points are applied to the scores of
// a page's 16 tokens and to their probabilities, not to the d values of a token.  Decoding is what the
// arithmetic pipe is busy with; a word of eight codes costs
//   K, as bf16 (the queries are): a mask and an or each, the nibble on the upper mantissa bits of 16.0,
//     and three rotations;
//   V, as fp16: a mask and an or each on 1024 or 64, whose mantissas take two nibbles without a shift,
//     one shift, and a subtraction in the float pipe, which leaves c - 8.
// p s enters that product as one fp16 number: 11 bits, off by 2^-12 at most, an eighth of the output's own
// rounding (a bf16 one would double the output's error).  fp16's range is kept by a power of two for each
// group of channels of a warp, moved when a scale grows past it, as the reference maximum is for p.
//
// Both products have the codes as the left operand, S^T = K Q^T and O^T = V^T P^T: their four registers
// are the decoded words themselves, and 8 columns hold the query heads of a KV head.  With up to four
// heads, a step takes two pages and the columns hold the heads of both, so that one round of
// exponentials and roundings serves both; a page's product with V has zeros in the other page's columns.
//
// Work: the (sequence, KV head, step) list is cut into contiguous shares of equal weight, one a CTA; the
// CTA's computing warps deal its steps among themselves.  One more warp requests the records (one
// bulk copy each) into the warps' rings, and merges the warps' states of a sequence when all have left
// it, so that the computing warps never wait for each other.  Where a share's end cuts a sequence, the
// CTA leaves a partial (normalised output, max, sum); a second kernel, launched as a programmatic
// dependent, merges the partials of each cut sequence.  At most two partials a CTA, so the workspace
// does not depend on the batch.
//
// Measured: 64 sequences of 512 to 8192 tokens, 32/8 heads, d = 128: 70 us for 304 MB (45 at the rate of a
// copy; the copies alone 58); 8 of up to 122,863, 16/2 heads, d = 256: 75 us for 281 MB.  No
// resource is full: of 600 instructions a step of two pages, 256 make operands and 32 are products, they depend on
// one another, and 16 warps an SM (10 at d = 256), all that the registers hold, use 56% of the issue slots.  With
// two pages a step at d = 256, 42 bytes a thread spill (8/2 heads: 64 us for the 75 above).  A lone sequence of
// 1009 tokens takes 9.5 us: two launches and six reads that wait for each other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache_q4.cuh"
#include "decode_shares.cuh"
#include "sm103.cuh"
#include "step.h"

namespace attn {

__device__ uint32_t g_decode_q4_status;

#ifdef ATTN_TEST_DROP_COPY
// Test-only builds (never the product library), in the CTA that begins sequence 0: 1: the loading warp leaves out
// its first copy; 2: it leaves at once.  The waits for what is then missing run out after ATTN_WAIT_LIMIT_NS.
__device__ int g_test_drop_copy_q4;
#endif

namespace {

using q4::Record;
using namespace shares;

constexpr int SEGMENT = 10;                   // steps that starting on a (sequence, unit) and leaving it cost
constexpr uint32_t CODE_MASK = 0x00780078u;   // a nibble on mantissa bits 3..6 of both halves
constexpr uint32_t K_MAGIC = 0x41804180u;     // 16 + c in both halves
constexpr uint32_t V_MASK0 = 0x000f000fu, V_MAGIC0 = 0x64006400u;  // fp16: 1024 + c
constexpr uint32_t V_MASK1 = 0x00f000f0u, V_MAGIC1 = 0x54005400u;  // 64 + c
// p s is at most P_LIMIT * 2^(V_BITS + V_ROOM + 1) = 2^15 as fp16, whose largest number is 65504, and keeps its
// 11 bits down to 2^-20 of the group's largest s (for p = 1)
constexpr float P_LIMIT = 64.f;               // a probability above it moves the reference maximum
constexpr uint32_t V_BITS = 6;                // where a group's unit puts the largest scale
constexpr uint32_t V_ROOM = 2;                // powers of two a scale may grow by before the unit moves
constexpr uint32_t PAST_ALL = 0x7f800000u;    // a float's bits from which on it is no finite number
constexpr uint32_t Z_MASK = 0x00780000u, Z_MAGIC = 0x41800000u;  // a zero point on the same bits of a float: 16 + z

// P: pages a warp takes at a step; ROWS / P query heads.
template <int D, int P>
struct Cfg {
  // Warps that compute (one more loads), and CTAs an SM: what shared memory holds with three steps in flight
  // a warp.  d = 256: 75 us with four warps, 77 with five (8 sequences of 58000, 16/2 heads).  d = 64: its
  // copies are small, and one loading warp for seven others cannot issue them fast enough; 64 sequences
  // of 8704, 32/8 heads: 93 us with 2 CTAs of seven warps, 83 with 3, 82 with 4 of five (64/8: 122, 103, 97).
  static constexpr int NW = D == 256 ? 4 : D == 128 ? 7 : 5;
  static constexpr int CTAS = D == 64 ? 4 : 2;
  static constexpr int THREADS = (NW + 1) * 32;
  static constexpr int TILE = ROWS / P;            // query heads a tile
  static constexpr int DEPTH = D == 256 && P == 2 ? 2 : 3;  // steps in flight a warp (two: 73 us for 70, d = 128)
  static constexpr int SLOTS = NW * DEPTH;
  static constexpr int STAGE = (P * Record<D>::BYTES + 127) & ~127;
  static constexpr int OROW = D + 8;               // floats of a row in the merge buffer
  static constexpr int MERGE = 2 * ROWS + TILE * OROW;  // floats a warp: m, l, o
  static constexpr int MERGE_OFF = SLOTS * STAGE;
  static constexpr int BAR_OFF = MERGE_OFF + NW * MERGE * 4;
  static constexpr int ALLOC = BAR_OFF + (2 * SLOTS + 2) * 8;
  static_assert(CTAS * (ALLOC + 1024 + 256) <= 228 * 1024, "shared memory budget");
};

struct Q4Geometry : shares::Geometry {
  // the magic numbers as arguments: a constant that the compiler knows would not stay in a register, and
  // decoding would take two instructions for the mask and the or
  uint32_t k_magic, v_magic0, v_magic1;
};

template <uint32_t MASK>
__device__ __forceinline__ uint32_t mask_or(uint32_t w, uint32_t magic) {
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(w), "n"(MASK), "r"(magic));
  return x;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}

// The 16-bit parameter words of a token's groups.
template <int NG>
struct Params {
  static constexpr int WORDS = (NG + 1) / 2;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const uint8_t* at) {
    if constexpr (NG == 1) {
      w[0] = *reinterpret_cast<const uint16_t*>(at);
    } else if constexpr (NG == 2) {
      w[0] = *reinterpret_cast<const uint32_t*>(at);
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(at);
      w[0] = x.x; w[1] = x.y;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float scale(int e) const {
    return __uint_as_float((e % 2 ? w[e / 2] : w[e / 2] << 16) & 0xfff00000u);
  }
  // the zero point, 16 + z
  __device__ __forceinline__ float zero(int e) const {
    return __uint_as_float(((e % 2 ? w[e / 2] << 3 : w[e / 2] << 19) & Z_MASK) | Z_MAGIC);
  }
};

template <int D, int P>
__global__ void __launch_bounds__(Cfg<D, P>::THREADS, Cfg<D, P>::CTAS)
    decode_q4_kernel(const DecodeQ4Params p, const Q4Geometry geo) {
  using C = Cfg<D, P>;
  using R = Record<D>;
  using VP = Params<R::NG>;
  constexpr int NW = C::NW, NG = R::NG, THREADS = C::THREADS, TILE = C::TILE, SLOTS = C::SLOTS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_weight[NW + 1], s_steps[NW + 1], s_end[2], s_at;
  __shared__ int3 s_start;
  float* merge = reinterpret_cast<float*>(smem + C::MERGE_OFF);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + SLOTS;
  uint64_t* rec_full = empty + SLOTS;  // every computing warp's state of a segment is in the merge buffer
  uint64_t* rec_free = rec_full + 1;   // the loading warp has read them
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int N = p.N, G = p.Hq / p.Hkv, units = geo.units;

  // ---- total steps, and the sequence that holds this share's first one
  if (threadIdx.x < SLOTS) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], 1);
    if (threadIdx.x == 0) {
      mbar_init(rec_full, NW);
      mbar_init(rec_free, 1);
    }
    fence_mbar_init();
  }
  // The list is cut by weight: a (sequence, unit) weighs its steps and SEGMENT more, what starting on it and
  // leaving its result cost.
  const int chunk = (N + THREADS - 1) / THREADS;
  const int n_lo = static_cast<int>(threadIdx.x) * chunk < N ? threadIdx.x * chunk : N;
  const int n_hi = n_lo + chunk < N ? n_lo + chunk : N;
  long long my_weight = 0, my_steps = 0;
  for (int n = n_lo; n < n_hi; ++n) {
    const int L = p.seq_lens[n];
    if (blockIdx.x == 0 && (L < 0 || L > p.max_blocks * PAGE)) set_error(&g_decode_q4_status, kDevBadSplit);
    const int ns = steps_of<P>(p.seq_lens, n, p.max_blocks);
    my_steps += ns;
    my_weight += ns > 0 ? ns + SEGMENT : 0;
  }
  long long to_weight = my_weight, to_steps = my_steps;  // inclusive sums
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, to_weight, off), c = __shfl_up_sync(0xffffffffu, to_steps, off);
    if (lane >= off) {
      to_weight += a;
      to_steps += c;
    }
  }
  if (lane == 31) {
    s_weight[warp] = to_weight;
    s_steps[warp] = to_steps;
  }
  __syncthreads();
  long long weight = 0, steps = 0;
#pragma unroll
  for (int i = 0; i < NW + 1; ++i) {
    if (i < warp) {
      to_weight += s_weight[i];
      to_steps += s_steps[i];
    }
    weight += s_weight[i];
    steps += s_steps[i];
  }
  const long long W = weight * units;
  // Short lists make fewer shares than CTAs: of one step, they would only be more partials to merge (a
  // sequence of 16 tokens: 10 us with two steps a share, 13 with four, 20 with seven)
  const long long most = steps * units / 2;
  const long long shares = most >= geo.grid ? geo.grid : most < 1 ? 1 : most;
  const int b = blockIdx.x;
  const long long lo = b < shares ? mul_div(b, W, shares) : W, hi = b < shares ? mul_div(b + 1, W, shares) : W;
  if (threadIdx.x == 0) s_end[0] = s_end[1] = steps * units;  // where the share's end is the list's
  __syncthreads();
  // the sequences in which the share begins and ends
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const long long x = side ? hi : lo;
    if (x < (to_weight - my_weight) * units || x >= to_weight * units) continue;
    long long at = (to_weight - my_weight) * units, before = (to_steps - my_steps) * units;
    int n = n_lo, ns = 0;
    for (;; ++n) {
      ns = steps_of<P>(p.seq_lens, n, p.max_blocks);
      const long long w = ns > 0 ? static_cast<long long>(ns + SEGMENT) * units : 0;
      if (x < at + w) break;
      at += w;
      before += static_cast<long long>(ns) * units;
    }
    const int u = static_cast<int>(mul_div(x - at, 1, ns + SEGMENT));
    const int in = static_cast<int>(x - at - static_cast<long long>(u) * (ns + SEGMENT));
    const int step = in > SEGMENT ? in - SEGMENT : 0;
    s_end[side] = before + static_cast<long long>(u) * ns + step;  // steps before x
    if (side == 0) {
      s_start = make_int3(n, u, step);
      s_at = at + static_cast<long long>(u) * (ns + SEGMENT);
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
  __syncthreads();
  // every CTA of this grid is resident: the combine's CTAs may queue up behind them
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Workspace ws = carve<D>(p.workspace, geo.grid);
  const int count = static_cast<int>(s_end[1] - s_end[0]);  // steps of this share
  if (count <= 0) {
    if (threadIdx.x == 0 && !geo.by_unit) ws.desc[b] = make_int4(0, 0, -1, 0);
    return;
  }

  Cursor<P> cur;  // the share's first step
  cur.n = s_start.x;
  cur.u = s_start.y;
  cur.step = s_start.z;
  cur.enter(p.seq_lens, p.max_blocks);

  if (warp == NW) {
    // ---------------------------------------------------------- loads, and results
    // Lane w serves computing warp w: step i of the share belongs to warp i % NW and goes through that
    // warp's ring.  The lanes poll their rings together, so that no warp waits for another's slot, and
    // each reads the block table a step ahead of the copy that needs it.  When all warps have left
    // their states of a segment (the share's part of a sequence and unit), this warp merges them and
    // writes the result, while the others are at the next segment.
    bool ok = true;
    Cursor<P> seg = cur;    // the segment to merge next ...
    long long at = s_at;    // ... the weight before its (sequence, unit) ...
    int seg_i = 0;          // ... its first step's share index
    uint32_t seg_phase = 0;
    int4 cut = make_int4(0, 0, -1, 0);
    int i = lane;      // this lane's next step, with the pages' table entries
    int ids[P] = {};
    int stage_k = 0;
    uint32_t phase = 1;  // a slot's first use waits for nothing
    auto fetch = [&]() {
      const int32_t* row = p.block_table + static_cast<int64_t>(cur.n) * p.max_blocks + cur.step * P;
      ids[0] = row[0];
      if (P == 2 && cur.step * P + 1 < cur.pages) ids[P - 1] = row[1];
    };
    if (lane > 0) cur.advance(lane, p.seq_lens, N, units, p.max_blocks);
    const bool serves = lane < NW;
    if (serves && i < count) fetch();
    uint64_t since = global_timer_ns();
#ifdef ATTN_TEST_DROP_COPY
    const int drop = s_start.x == 0 && s_start.y == 0 && s_start.z == 0 ? g_test_drop_copy_q4 : 0;
    ok = drop != 2;
#endif
    while (ok && seg_i < count) {
      const int slot = lane + NW * stage_k;
      const bool go = serves && i < count && mbar_test_wait(&empty[slot], phase);
      if (go) {
        const int pages = P == 2 && cur.step * P + 1 < cur.pages ? 2 : 1;
        mbar_arrive_expect_tx(&full[slot], pages * R::BYTES);
#pragma unroll
        for (int a = 0; a < P; ++a) {
          if (a >= pages) break;
          int id = ids[a];
          if (id < 0 || id >= p.num_blocks) {
            set_error(&g_decode_q4_status, kDevBadPage);
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
          cur.advance(NW, p.seq_lens, N, units, p.max_blocks);
          fetch();
        }
      }
      const bool merge_now = __all_sync(0xffffffffu, mbar_test_wait(rec_full, seg_phase));
      if (merge_now) {
        seg_phase ^= 1;
        const int seg_steps = seg.ns - seg.step < count - seg_i ? seg.ns - seg.step : count - seg_i;
        const bool starts = seg.step == 0, ends = seg.step + seg_steps == seg.ns;
        const int kvh = seg.u / geo.tiles, h0 = seg.u % geo.tiles * TILE;
        const int heads = G - h0 < TILE ? G - h0 : TILE;
        const int64_t part = 2 * b + (starts ? 1 : 0);
        for (int w = lane; w < heads * (D / 4); w += 32) {
          const int r = w / (D / 4), x = w % (D / 4) * 4;
          float M = -INFINITY;
#pragma unroll
          for (int v = 0; v < NW; ++v) M = fmaxf(M, merge[v * C::MERGE + r]);
          float L = 0.f;
          float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int v = 0; v < NW; ++v) {
            const float* src = merge + v * C::MERGE;
            const float wl = src[ROWS + r];
            if (wl == 0.f) continue;  // a warp without tokens
            const float f = ex2_approx(src[r] - M);
            const float4 y = *reinterpret_cast<const float4*>(src + 2 * ROWS + r * C::OROW + x);
            L = fmaf(wl, f, L);
            O.x = fmaf(y.x, f, O.x); O.y = fmaf(y.y, f, O.y);
            O.z = fmaf(y.z, f, O.z); O.w = fmaf(y.w, f, O.w);
          }
          const float inv = 1.f / L;
          O.x *= inv; O.y *= inv; O.z *= inv; O.w *= inv;
          if (starts && ends) {
            const int64_t row = static_cast<int64_t>(seg.n) * p.Hq + kvh * G + h0 + r;
            *reinterpret_cast<uint2*>(p.o + row * D + x) = make_uint2(pack_bf16x2(O.x, O.y), pack_bf16x2(O.z, O.w));
            if (x == 0 && p.lse != nullptr) p.lse[row] = (M + log2f(L)) * LN2;
          } else {
            *reinterpret_cast<float4*>(ws.o + (part * ROWS + r) * D + x) = O;
            if (x == 0) {
              ws.m[part * ROWS + r] = M;
              ws.l[part * ROWS + r] = L;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(rec_free);
        if (starts && !ends) {
          // the share that holds the last step: weight x lies in share ((x + 1) shares - 1) / W
          const long long past = at + SEGMENT + seg.ns;
          cut = make_int4(seg.n, seg.u, b, static_cast<int>(mul_div(past * shares - 1, 1, W)));
        }
        if (geo.by_unit && starts && lane == 0)
          ws.desc[seg.n * units + seg.u] = ends ? make_int4(0, 0, -1, 0) : cut;
        at += SEGMENT + seg.ns;
        seg_i += seg_steps;
        if (seg_i < count) seg.advance(seg_steps, p.seq_lens, N, units, p.max_blocks);
      }
      if (__any_sync(0xffffffffu, go) || merge_now) {
        since = global_timer_ns();
      } else {
        __nanosleep(50);
        ok = __all_sync(0xffffffffu, global_timer_ns() - since < ATTN_WAIT_LIMIT_NS);
      }
    }
    if (lane == 0) {
      if (!geo.by_unit) ws.desc[b] = cut;
      if (!ok) set_error(&g_decode_q4_status, kDevWaitTimeout);
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
  const float c2 = p.scale_log2;
  bool ok = true;
  int i = warp;    // share index of this warp's next step
  int stage_k = 0;         // its ring stage: slot warp + NW stage_k ...
  uint32_t phase = 0;      // ... and the parity of that slot's barriers
  uint32_t free_phase = 0;
  for (int seg = 0; seg < count;) {
    const int seg_n = cur.n, seg_u = cur.u, first_step = cur.step;
    const int seg_steps = cur.ns - first_step < count - seg ? cur.ns - first_step : count - seg;
    const int seg_end = seg + seg_steps;
    const int len = clamped_len(p.seq_lens, seg_n, p.max_blocks);
    const int kvh = seg_u / geo.tiles, h0 = seg_u % geo.tiles * TILE;
    const int heads = G - h0 < TILE ? G - h0 : TILE;
    const __nv_bfloat16* q_head = p.q + (static_cast<int64_t>(seg_n) * p.Hq + kvh * G + h0) * D;

    // ---- queries: channels 64 e + 16 t + 8 h .. + 7, paired as the K words pair them
    uint32_t qb[NG][2][4];
    float nqsum[NG][2];  // minus the sum over a group, of columns 2 t and 2 t + 1
#pragma unroll
    for (int e = 0; e < NG; ++e) {
      float sum = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (q_row < heads) x = *reinterpret_cast<const uint4*>(q_head + q_row * D + 64 * e + 16 * t + 8 * h);
        qb[e][h][0] = __byte_perm(x.x, x.z, 0x5410);  // channels 0, 4
        qb[e][h][1] = __byte_perm(x.x, x.z, 0x7632);  // 1, 5
        qb[e][h][2] = __byte_perm(x.y, x.w, 0x5410);  // 2, 6
        qb[e][h][3] = __byte_perm(x.y, x.w, 0x7632);  // 3, 7
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) sum -= __uint_as_float(w[j] << 16) + __uint_as_float(w[j] & 0xffff0000u);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      nqsum[e][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
      nqsum[e][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
    }

    float mc[2] = {-1e38f, -1e38f};  // of columns 2 t, 2 t + 1: the reference maximum, in log2 units
    float l[2] = {0.f, 0.f};         // this lane's share of the sum of probabilities
    float base[NG][2];               // sum of p s (z - 8) over this lane's tokens
    float v_unit[NG];                // s enters o and base times this power of two; 0: no scale seen yet
    uint32_t v_most[VP::WORDS];      // the largest parameter words that fit it, two groups a word
    float o[D / 16][4];              // channels 16 i + 2 g (0, 1) and + 1 (2, 3) of columns 2 t and 2 t + 1
#pragma unroll
    for (int x = 0; x < D / 16; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
#pragma unroll
    for (int e = 0; e < NG; ++e) base[e][0] = base[e][1] = v_unit[e] = 0.f;
#pragma unroll
    for (int x = 0; x < VP::WORDS; ++x) v_most[x] = 0x000f000fu;  // a scale of 0 and any zero point

    // S^T of a step whose records are at `stage`: rows are tokens g (0, 1) and g + 8 (2, 3), columns 2 t and
    // 2 t + 1
    auto scores = [&](const uint8_t* stage, float (&sc)[4]) {
      sc[0] = sc[1] = sc[2] = sc[3] = 0.f;
      Params<NG> kp[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) kp[j].load(stage + my_page * R::BYTES + R::KP_OFF + (g + 8 * j) * (2 * NG));
#pragma unroll
      for (int pr = 0; pr < NG / R::PAIR; ++pr) {
        float acc[R::PAIR][P][4];
        uint32_t kw[P][2][2 * R::PAIR];
#pragma unroll
        for (int a = 0; a < P; ++a) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint8_t* row =
                stage + a * R::BYTES + R::K_OFF + (g + 8 * j) * (D / 2) + pr * (32 * R::PAIR) + t * (8 * R::PAIR);
            if constexpr (R::PAIR == 2) {
              const uint4 x = *reinterpret_cast<const uint4*>(row);
              kw[a][j][0] = x.x; kw[a][j][1] = x.y; kw[a][j][2] = x.z; kw[a][j][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(row);
              kw[a][j][0] = x.x; kw[a][j][1] = x.y;
            }
          }
        }
        // consecutive products go to different accumulators: each would wait for the one before otherwise
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int a = 0; a < P; ++a)
#pragma unroll
            for (int ee = 0; ee < R::PAIR; ++ee) {
              const int e = pr * R::PAIR + ee, h = k / 2, s = k % 2 * 2;
              const uint32_t w0 = kw[a][0][ee * 2 + h], w1 = kw[a][1][ee * 2 + h];
              if (k == 0) acc[ee][a][0] = acc[ee][a][1] = acc[ee][a][2] = acc[ee][a][3] = 0.f;
              mma_16816<false>(acc[ee][a], mask_or<CODE_MASK>(__funnelshift_r(w0, w0, 4 * s), geo.k_magic),
                               mask_or<CODE_MASK>(__funnelshift_r(w1, w1, 4 * s), geo.k_magic),
                               mask_or<CODE_MASK>(__funnelshift_r(w0, w0, 4 * s + 4), geo.k_magic),
                               mask_or<CODE_MASK>(__funnelshift_r(w1, w1, 4 * s + 4), geo.k_magic), qb[e][h][s],
                               qb[e][h][s + 1]);
            }
#pragma unroll
        for (int ee = 0; ee < R::PAIR; ++ee) {
          const int e = pr * R::PAIR + ee;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float s = kp[j].scale(e), z = kp[j].zero(e);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float x = P == 2 && my_page ? acc[ee][P - 1][2 * j + c] : acc[ee][0][2 * j + c];
              sc[2 * j + c] = fmaf(s, fmaf(z, nqsum[e][c], x), sc[2 * j + c]);
            }
          }
        }
      }
    };
    for (; i < seg_end; i += NW) {
      const int slot = warp + NW * stage_k;
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&full[slot], phase));
      if (++stage_k == C::DEPTH) {
        stage_k = 0;
        phase ^= 1;
      }
      if (!ok) continue;
      float sc[4];
      scores(smem + slot * C::STAGE, sc);
      const uint8_t* stage = smem + slot * C::STAGE;
      // tokens of this lane's page that the sequence has; the last step's second page may have none
      const int valid = len - ((first_step + i - seg) * P + my_page) * PAGE;
      Params<NG> vp[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) vp[j].load(stage + my_page * R::BYTES + R::VP_OFF + (g + 8 * j) * (2 * NG));
      if (__any_sync(0xffffffffu, valid < PAGE)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (g + 8 * j >= valid) {
            sc[2 * j] = sc[2 * j + 1] = -INFINITY;
            vp[j].clear();  // whatever lies past the sequence is not to be multiplied with: 0 * NaN is not 0
          }
      }
      // ---- online softmax against the reference; a probability past the limit moves it to the maximum
      float pr[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) pr[x] = ex2_approx(fmaf(sc[x], c2, -mc[x & 1]));
      if (__any_sync(0xffffffffu, fmaxf(fmaxf(pr[0], pr[1]), fmaxf(pr[2], pr[3])) > P_LIMIT)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(sc[c], sc[2 + c]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          if (P == 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));  // a head's two pages share it
          const float to = fmaxf(mc[c], mx * c2), f = ex2_approx(mc[c] - to);
          mc[c] = to;
          l[c] *= f;
#pragma unroll
          for (int e = 0; e < NG; ++e) base[e][c] *= f;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            o[x][c] *= f;
            o[x][2 + c] *= f;
          }
          pr[c] = ex2_approx(fmaf(sc[c], c2, -to));
          pr[2 + c] = ex2_approx(fmaf(sc[2 + c], c2, -to));
        }
      }
      l[0] += pr[0] + pr[2];
      l[1] += pr[1] + pr[3];
      bool grown = false;
#pragma unroll
      for (int x = 0; x < VP::WORDS; ++x)
        grown |= __vmaxu2(__vmaxu2(vp[0].w[x], vp[1].w[x]), v_most[x]) != v_most[x];
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int e = 0; e < NG; ++e) {
          // the largest scale's bits; a NaN scale says nothing about the others' range
          const uint32_t s0 = __float_as_uint(vp[0].scale(e)), s1 = __float_as_uint(vp[1].scale(e));
          const uint32_t top = __reduce_max_sync(0xffffffffu, max(s0 < PAST_ALL ? s0 : 0u, s1 < PAST_ALL ? s1 : 0u));
          if (top == 0 && v_unit[e] == 0.f) continue;
          // its exponent.  Below 2^(V_BITS - 126), scales without one (subnormal) among them, the unit stays
          // 2^126, whose reciprocal is the smallest normal number.
          const uint32_t to = max(top >> 23, V_BITS + 1);
          const float unit = __uint_as_float((254 + V_BITS - to) << 23);  // the largest scale: [2^V_BITS, 2 of it)
          if (v_unit[e] != 0.f && unit >= v_unit[e]) continue;
          const float f = v_unit[e] == 0.f ? 0.f : unit / v_unit[e];
          v_unit[e] = unit;
          const uint32_t most = min((to + V_ROOM) << 7 | 127u, 0x7f7fu);
          v_most[e / 2] = e % 2 ? (v_most[e / 2] & 0xffffu) | most << 16 : (v_most[e / 2] & 0xffff0000u) | most;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            base[e][c] *= f;
#pragma unroll
            for (int x = 4 * e; x < 4 * e + 4; ++x) {
              o[x][c] *= f;
              o[x][2 + c] *= f;
            }
          }
        }
      }
      // ---- O^T += V^T (p s)^T
#pragma unroll
      for (int e = 0; e < NG; ++e) {
        uint32_t pb[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float s = vp[j].scale(e) * v_unit[e], z = vp[j].zero(e) - 24.f;
          const float x0 = pr[2 * j] * s, x1 = pr[2 * j + 1] * s;
          // the rounded product in both sums, so that a code equal to its zero point stands for exactly 0
          const uint32_t xh = pack_f16x2(x0, x1);
          const float2 xf = __half22float2(*reinterpret_cast<const __half2*>(&xh));
          base[e][0] = fmaf(xf.x, z, base[e][0]);
          base[e][1] = fmaf(xf.y, z, base[e][1]);
          pb[j] = transpose_8x8(xh);
        }
#pragma unroll
        for (int a = 0; a < P; ++a) {
          const bool on = P == 1 || (g >> 2) == a;  // as an operand, this lane holds column g
          const uint32_t b0 = on ? pb[0] : 0u, b1 = on ? pb[1] : 0u;
          const uint4 vw = *reinterpret_cast<const uint4*>(stage + a * R::BYTES + R::V_OFF + (e * 32 + lane) * 16);
          const uint32_t w4[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w = w4[j], w8 = w >> 8;
            mma_16816<true>(o[e * 4 + j], sub_f16x2(mask_or<V_MASK0>(w, geo.v_magic0), 0x64086408u),
                            sub_f16x2(mask_or<V_MASK1>(w, geo.v_magic1), 0x54805480u),
                            sub_f16x2(mask_or<V_MASK0>(w8, geo.v_magic0), 0x64086408u),
                            sub_f16x2(mask_or<V_MASK1>(w8, geo.v_magic1), 0x54805480u), b0, b1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
    }
    // A wait that ran out is this warp's last: waits of the others that need it run out once too, and not for
    // every segment that is left.
    if (!ok) break;

    // ---- this warp's state to shared memory, then the CTA's to global memory.  With two pages, a head's
    // sums are in columns c and c + 4, two lanes apart.
#pragma unroll
    for (int off = P == 2 ? 2 : 4; off < 32; off <<= 1) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[c] += __shfl_xor_sync(0xffffffffu, l[c], off);
#pragma unroll
        for (int e = 0; e < NG; ++e) base[e][c] += __shfl_xor_sync(0xffffffffu, base[e][c], off);
      }
    }
    if (P == 2) {
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[x][j] += __shfl_xor_sync(0xffffffffu, o[x][j], 2);
    }
    float v_back[NG];  // 1 / v_unit
#pragma unroll
    for (int e = 0; e < NG; ++e) v_back[e] = __uint_as_float((254u << 23) - __float_as_uint(v_unit[e]));
    // the loading warp has merged the segment before this one
    if (seg > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(rec_free, free_phase));
      free_phase ^= 1;
      if (!ok) break;
    }
    float* my = merge + warp * C::MERGE;
    if (2 * t < TILE) {
      if (g == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          my[2 * t + c] = l[c] == 0.f ? -INFINITY : mc[c];  // no tokens: no part in the maximum
          my[ROWS + 2 * t + c] = l[c];
        }
      }
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        float* at = my + 2 * ROWS + 2 * t * C::OROW + 16 * x + 2 * g;
        *reinterpret_cast<float2*>(at) =
            make_float2((o[x][0] - base[x / 4][0]) * v_back[x / 4], (o[x][2] - base[x / 4][0]) * v_back[x / 4]);
        *reinterpret_cast<float2*>(at + C::OROW) =
            make_float2((o[x][1] - base[x / 4][1]) * v_back[x / 4], (o[x][3] - base[x / 4][1]) * v_back[x / 4]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(rec_full);
    seg = seg_end;
    if (seg < count) cur.advance(seg_steps, p.seq_lens, N, units, p.max_blocks);
  }
  if (!ok && lane == 0) set_error(&g_decode_q4_status, kDevWaitTimeout);
}

// CTAs of the grid: every SM filled
template <int D>
int grid_of_device() {
  static_assert(Cfg<D, 1>::CTAS == Cfg<D, 2>::CTAS, "one size of workspace for a head dim");
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms * Cfg<D, 1>::CTAS;
}

template <int D, int P>
cudaError_t launch(const DecodeQ4Params& p, cudaStream_t stream) {
  using C = Cfg<D, P>;
  Q4Geometry geo;
  geo.grid = grid_of_device<D>();
  if (geo.grid <= 0) return cudaErrorInvalidDevice;
  geo.tile = C::TILE;
  geo.tiles = (p.Hq / p.Hkv + C::TILE - 1) / C::TILE;
  geo.units = p.Hkv * geo.tiles;
  geo.by_unit = static_cast<int64_t>(p.N) * geo.units * 8 <= geo.grid;
  geo.k_magic = K_MAGIC;
  geo.v_magic0 = V_MAGIC0;
  geo.v_magic1 = V_MAGIC1;
  auto kern = decode_q4_kernel<D, P>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::ALLOC);
  if (e != cudaSuccess) return e;
  kern<<<geo.grid, C::THREADS, C::ALLOC, stream>>>(p, geo);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return shares::launch_combine<D, C::TILE>(
      shares::MergeParams{p.workspace, p.o, p.lse, p.seq_lens, p.N, p.Hq, p.Hkv, p.max_blocks}, geo, stream);
}

template <int D>
cudaError_t launch_for(const DecodeQ4Params& p, cudaStream_t stream) {
  return p.Hq / p.Hkv <= ROWS / 2 ? launch<D, 2>(p, stream) : launch<D, 1>(p, stream);
}

}  // namespace

#ifdef ATTN_TEST_DROP_COPY
extern "C" int attn_test_drop_copy_q4(int what) {
  return static_cast<int>(cudaMemcpyToSymbol(g_test_drop_copy_q4, &what, sizeof(int)));
}
#endif

size_t decode_q4_workspace_bytes(int d) {
  const size_t grid = d == 64    ? grid_of_device<64>()
                      : d == 128 ? grid_of_device<128>()
                      : d == 256 ? grid_of_device<256>()
                                 : 0;
  return shares::workspace_bytes(static_cast<int>(grid), d);
}

cudaError_t decode_q4_launch(int d, const DecodeQ4Params& p, cudaStream_t stream) {
  if (d == 64) return launch_for<64>(p, stream);
  if (d == 128) return launch_for<128>(p, stream);
  if (d == 256) return launch_for<256>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t decode_q4_status(uint32_t* out, bool clear) { return read_status(g_decode_q4_status, out, clear); }

}  // namespace attn
