// Single-token attention over the 4-bit paged cache (format and layout: cache_q4.cuh).
//
// With K = s_g (c - z_g) and V likewise, per group g of 64 channels,
//   score = sum_g s_g (q . c - z_g sum q),     O = sum_tokens p s c - sum_tokens p s z,
// so the codes themselves are the matrix operands: a code becomes a bf16 number by one mask and one
// or (16 + c, exact, its nibble on the upper mantissa bits), and scales and zero points are applied
// to the 16 scores of a page's token tile and to its 16 probabilities, not to the d values of a token.
//
// Both products have the codes as the left operand, S^T = K Q^T and O^T = V^T P^T: their four registers
// are the decoded words themselves, and 8 columns hold the query heads of a KV head.  With up to four
// heads the columns take the heads of two pages, so that one step's scores, exponentials and
// roundings serve both.  p s is split into two bf16 numbers (16 bits together): one alone would add an
// error as large as the output's own rounding.  Odd tokens of V enter as c - 31 (one exclusive-or
// instead of the or), so that the offsets of the codes cancel in the running sums.
//
// Work: the (sequence, KV head, page) list is cut into equal contiguous shares, one a CTA; the CTA's
// warps deal its pages among themselves, each with its own ring of bulk copies (a record is one
// copy).  Where a share's end cuts a sequence, the CTA leaves a partial (normalised output, max, sum);
// a second kernel, launched as a programmatic dependent, merges the partials of each cut sequence.
// At most two partials a CTA, so the workspace does not depend on the batch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache_q4.cuh"
#include "sm103.cuh"
#include "step.h"

namespace attn {

__device__ uint32_t g_decode_q4_status;

namespace {

using q4::PAGE;
using q4::Record;

constexpr float LN2 = 0.693147180559945309f;
constexpr int ROWS = 8;                       // score columns of a warp: query heads, or heads of two pages
constexpr uint32_t CODE_MASK = 0x00780078u;   // a nibble on mantissa bits 3..6 of both halves
constexpr uint32_t K_MAGIC = 0x41804180u;     // 16 + c in both halves
constexpr uint32_t V_MAGIC = 0xc1f84180u;     // 16 + c in the lower half (an even token), c - 31 in the upper one
constexpr float P_LIMIT = 256.f;              // a probability above it moves the reference maximum
constexpr uint32_t Z_MASK = 0x00780000u;      // a zero point on the same bits of a float: 16 + z, z - 31
constexpr uint32_t Z_EVEN = 0x41800000u, Z_ODD = 0xc1f80000u;

// P: pages a warp takes at a step; ROWS / P query heads.
template <int D, int P>
struct Cfg {
  static constexpr int NW = D < 256 ? 7 : P == 2 ? 4 : 5;  // warps that compute (one more loads)
  static constexpr int NS = D == 256 ? 3 : D == 128 ? 3 : 4;  // pages in flight a warp
  static constexpr int CTAS = 2;                   // CTAs an SM
  static constexpr int THREADS = (NW + 1) * 32;
  static constexpr int TILE = ROWS / P;            // query heads a tile
  static constexpr int DEPTH = P == 2 ? 2 : NS;    // steps in flight a warp
  static constexpr int SLOTS = NW * DEPTH;
  static constexpr int STAGE = (P * Record<D>::BYTES + 127) & ~127;
  static constexpr int OROW = D + 8;               // floats of a row in the merge buffer
  static constexpr int MERGE = 2 * ROWS + ROWS * OROW;  // floats a warp: m, l, o
  static constexpr int MERGE_OFF = SLOTS * STAGE;
  static constexpr int BAR_OFF = MERGE_OFF + NW * MERGE * 4;
  static constexpr int ALLOC = BAR_OFF + 2 * SLOTS * 8;
  static_assert(CTAS * (ALLOC + 1024 + 256) <= 228 * 1024, "shared memory budget");
  static_assert(CTAS * THREADS * (D == 256 ? 168 : 128) <= 65536, "register budget");
};

// a * b / c with c > 0; the quotient is below 2^63.  64-bit division costs over a hundred instructions,
// and the shares of all but the largest batches are counted in 32 bits.
__device__ __forceinline__ long long mul_div(long long a, long long b, long long c) {
  const long long n = a * b;
  if ((n | c) >> 32 == 0) return static_cast<uint32_t>(n) / static_cast<uint32_t>(c);
  return n / c;
}

struct Q4Geometry {
  int grid, tiles, units;  // CTAs, head tiles a KV head, (KV head, tile) pairs a sequence
  // K_MAGIC and V_MAGIC as arguments: a constant that the compiler knows would not stay in a register,
  // and decoding a word half would take two instructions
  uint32_t k_magic, v_magic;
};

// What the workspace holds: the shares' descriptors, then the partials' o, m and l.
struct Workspace {
  int4* desc;    // [grid]: (sequence, unit, last share, 1) of the cut sequence that starts in share b, or w = 0
  float* o;      // [2 grid][ROWS][d]: index 2 b: continued from the share before, 2 b + 1: starts here
  float *m, *l;  // [2 grid][ROWS]
};

template <int D>
__device__ Workspace carve(void* ws, int grid) {
  Workspace w;
  w.desc = static_cast<int4*>(ws);
  w.o = reinterpret_cast<float*>(w.desc + grid);
  w.m = w.o + static_cast<size_t>(2) * grid * ROWS * D;
  w.l = w.m + static_cast<size_t>(2) * grid * ROWS;
  return w;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (w & CODE_MASK) ^ magic
__device__ __forceinline__ uint32_t decode(uint32_t w, uint32_t magic) {
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(x) : "r"(w), "n"(CODE_MASK), "r"(magic));
  return x;
}

// transposes an 8 x 8 tile of 16-bit values held as an accumulator's pairs
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ int clamped_len(const int32_t* lens, int n, int max_blocks) {
  const int L = lens[n];
  return L < 0 ? 0 : (L > max_blocks * PAGE ? max_blocks * PAGE : L);
}
// steps of P pages of sequence n
template <int P>
__device__ __forceinline__ int steps_of(const int32_t* lens, int n, int max_blocks) {
  return (clamped_len(lens, n, max_blocks) + P * PAGE - 1) / (P * PAGE);
}

// Position in the (sequence, unit, step) list.
template <int P>
struct Cursor {
  int n, u, step, ns;
  __device__ __forceinline__ void advance(int by, const int32_t* lens, int N, int units, int max_blocks) {
    step += by;
    while (step >= ns) {
      step -= ns;
      if (++u == units) {
        u = 0;
        do {
          if (++n >= N) {  // past the end of the list: nothing there is read
            n = N;
            ns = 0x7fffffff;
            return;
          }
          ns = steps_of<P>(lens, n, max_blocks);
        } while (ns == 0);
      }
    }
  }
};

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
  // the zero point z as `magic` makes a float of it: 16 + z or z - 31
  __device__ __forceinline__ float zero(int e, uint32_t magic) const {
    return __uint_as_float(((e % 2 ? w[e / 2] << 3 : w[e / 2] << 19) & Z_MASK) ^ magic);
  }
};

template <int D, int P>
__global__ void __launch_bounds__(Cfg<D, P>::THREADS, Cfg<D, P>::CTAS)
    decode_q4_kernel(const DecodeQ4Params p, const Q4Geometry geo) {
  using C = Cfg<D, P>;
  using R = Record<D>;
  constexpr int NW = C::NW, NG = R::NG, THREADS = C::THREADS, TILE = C::TILE, SLOTS = C::SLOTS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_warp[NW + 1];
  __shared__ long long s_before;
  __shared__ int s_n;
  float* merge = reinterpret_cast<float*>(smem + C::MERGE_OFF);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + SLOTS;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int N = p.N, G = p.Hq / p.Hkv, units = geo.units;

  // ---- total steps, and the sequence that holds this share's first one
  if (threadIdx.x < SLOTS) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], 1);
    fence_mbar_init();
  }
  const int chunk = (N + THREADS - 1) / THREADS;
  const int n_lo = static_cast<int>(threadIdx.x) * chunk < N ? threadIdx.x * chunk : N;
  const int n_hi = n_lo + chunk < N ? n_lo + chunk : N;
  long long mine = 0;
  for (int n = n_lo; n < n_hi; ++n) {
    const int L = p.seq_lens[n];
    if (blockIdx.x == 0 && (L < 0 || L > p.max_blocks * PAGE)) set_error(&g_decode_q4_status, kDevBadSplit);
    mine += steps_of<P>(p.seq_lens, n, p.max_blocks);
  }
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += a;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int i = 0; i < NW + 1; ++i) {
    if (i < warp) incl += s_warp[i];
    total += s_warp[i];
  }
  const long long W = total * units;
  // at least a step for each warp of a share
  const long long shares = W >= static_cast<long long>(geo.grid) * NW ? geo.grid : W < NW ? 1 : static_cast<int>(W) / NW;
  const int b = blockIdx.x;
  const long long lo = b < shares ? mul_div(b, W, shares) : W, hi = b < shares ? mul_div(b + 1, W, shares) : W;
  const int count = static_cast<int>(hi - lo);  // steps of this share
  const long long before_mine = (incl - mine) * units;
  if (count > 0 && before_mine <= lo && lo < incl * units) {
    long long at = before_mine;
    int n = n_lo;
    for (;; ++n) {
      const long long w = static_cast<long long>(steps_of<P>(p.seq_lens, n, p.max_blocks)) * units;
      if (lo < at + w) break;
      at += w;
    }
    s_n = n;
    s_before = at;
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
  if (count <= 0) {
    if (threadIdx.x == 0) ws.desc[b] = make_int4(0, 0, 0, 0);
    return;
  }

  Cursor<P> cur;  // the share's first step
  cur.n = s_n;
  cur.ns = steps_of<P>(p.seq_lens, cur.n, p.max_blocks);
  const long long rel = lo - s_before;
  cur.u = static_cast<int>(mul_div(rel, 1, cur.ns));
  cur.step = static_cast<int>(rel - static_cast<long long>(cur.u) * cur.ns);

  if (warp == NW) {
    // ---------------------------------------------------------- loads
    // Step i goes to slot i % SLOTS and to computing warp i % NW.  Each lane finds the records of one
    // of 32 steps (its table entries are read together with the other lanes'), then NW lanes at a
    // time wait for their slots and request their records, one copy a record.
    constexpr int ROUND = 32 / NW * NW;
    bool ok = true;
    int last = -1;   // this lane's last step whose copy was requested
    cur.advance(lane, p.seq_lens, N, units, p.max_blocks);
    for (int base = 0; base < count; base += ROUND) {
      const int i = base + lane;
      const bool live = lane < ROUND && i < count;
      const uint8_t* src[P];
      int pages = 0;
      if (live) {
        const int len = clamped_len(p.seq_lens, cur.n, p.max_blocks);
        const int32_t* row = p.block_table + static_cast<int64_t>(cur.n) * p.max_blocks + cur.step * P;
#pragma unroll
        for (int a = 0; a < P; ++a) {
          if ((cur.step * P + a) * PAGE >= len) continue;
          int id = row[a];
          if (id < 0 || id >= p.num_blocks) {
            set_error(&g_decode_q4_status, kDevBadPage);
            id = 0;
          }
          src[a] = p.cache + (static_cast<int64_t>(id) * p.Hkv + cur.u / geo.tiles) * R::BYTES;
          ++pages;
        }
      }
#pragma unroll 1
      for (int from = 0; from < ROUND && base + from < count; from += NW) {
        if (live && lane >= from && lane < from + NW) {
          const int slot = i % SLOTS;
          if (ok) ok = mbar_wait(&empty[slot], (i / SLOTS & 1) ^ 1);
          if (ok) {
            mbar_arrive_expect_tx(&full[slot], pages * R::BYTES);
            bulk_load(smem + slot * C::STAGE, src[0], R::BYTES, &full[slot]);
            if (P == 2 && pages == 2) bulk_load(smem + slot * C::STAGE + R::BYTES, src[P - 1], R::BYTES, &full[slot]);
            last = i;
          }
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      cur.advance(ROUND, p.seq_lens, N, units, p.max_blocks);
    }
    if (!ok) set_error(&g_decode_q4_status, kDevWaitTimeout);
    // Copies in flight must land before the CTA's shared memory is given back.  Only a slot's newest
    // copy is of the phase that its barrier is in; an older one was waited for before the newer left.
    static_assert(ROUND >= SLOTS, "a lane has at most one step among the newest of the slots");
    const int end = __reduce_max_sync(0xffffffffu, last) + 1;
    if (last >= 0 && last >= end - SLOTS) mbar_wait(&full[last % SLOTS], last / SLOTS & 1);
    return;
  }

  // ------------------------------------------------------------ attention
  const int g = lane >> 2, t = lane & 3;
  const int q_row = P == 2 ? g & 3 : g;     // the query head of the tile that this lane loads: column g
  const int my_page = P == 2 ? t >> 1 : 0;  // columns 2 t and 2 t + 1 are two heads of this page of the step
  const uint32_t z_magic = g & 1 ? Z_ODD : Z_EVEN;  // of tokens g and g + 8 of V
  const float c2 = p.scale_log2;
  bool ok = true;
  int i = warp;    // share index of this warp's next step
  int4 cut = make_int4(0, 0, 0, 0);
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
    float base[NG][2];               // sum of p s (16 + z) or p s (z - 31) over this lane's tokens
    float o[D / 16][4];              // channels 16 i + 2 g (0, 1) and + 1 (2, 3) of columns 2 t and 2 t + 1
#pragma unroll
    for (int x = 0; x < D / 16; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
#pragma unroll
    for (int e = 0; e < NG; ++e) base[e][0] = base[e][1] = 0.f;

    for (; i < seg_end; i += NW) {
      const int slot = i % SLOTS;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], i / SLOTS & 1));
      if (!ok) continue;
      const uint8_t* stage = smem + slot * C::STAGE;
      const uint8_t* mine_rec = stage + my_page * R::BYTES;
      // tokens of this lane's page that the sequence has; the last step's second page may have none
      const int valid = len - ((first_step + i - seg) * P + my_page) * PAGE;

      // ---- S^T: rows are tokens g (0, 1) and g + 8 (2, 3), columns 2 t and 2 t + 1
      float sc[4] = {0.f, 0.f, 0.f, 0.f};
      Params<NG> kp[2], vp[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        kp[j].load(mine_rec + R::KP_OFF + (g + 8 * j) * (2 * NG));
        vp[j].load(mine_rec + R::VP_OFF + (g + 8 * j) * (2 * NG));
      }
#pragma unroll
      for (int pr = 0; pr < NG / R::PAIR; ++pr) {
        float acc[R::PAIR][P][4];
#pragma unroll
        for (int a = 0; a < P; ++a) {
          uint32_t kw[2][2 * R::PAIR];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint8_t* row =
                stage + a * R::BYTES + R::K_OFF + (g + 8 * j) * (D / 2) + pr * (32 * R::PAIR) + t * (8 * R::PAIR);
            if constexpr (R::PAIR == 2) {
              const uint4 x = *reinterpret_cast<const uint4*>(row);
              kw[j][0] = x.x; kw[j][1] = x.y; kw[j][2] = x.z; kw[j][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(row);
              kw[j][0] = x.x; kw[j][1] = x.y;
            }
          }
#pragma unroll
          for (int ee = 0; ee < R::PAIR; ++ee) {
            const int e = pr * R::PAIR + ee;
            acc[ee][a][0] = acc[ee][a][1] = acc[ee][a][2] = acc[ee][a][3] = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w0 = kw[0][ee * 2 + h], w1 = kw[1][ee * 2 + h];
              mma_16816(acc[ee][a], decode(w0, geo.k_magic), decode(w1, geo.k_magic),
                        decode(__funnelshift_r(w0, w0, 4), geo.k_magic),
                        decode(__funnelshift_r(w1, w1, 4), geo.k_magic), qb[e][h][0], qb[e][h][1]);
              mma_16816(acc[ee][a], decode(__funnelshift_r(w0, w0, 8), geo.k_magic),
                        decode(__funnelshift_r(w1, w1, 8), geo.k_magic),
                        decode(__funnelshift_r(w0, w0, 12), geo.k_magic),
                        decode(__funnelshift_r(w1, w1, 12), geo.k_magic), qb[e][h][2], qb[e][h][3]);
            }
          }
        }
#pragma unroll
        for (int ee = 0; ee < R::PAIR; ++ee) {
          const int e = pr * R::PAIR + ee;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float s = kp[j].scale(e), z = kp[j].zero(e, Z_EVEN);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float x = P == 2 && my_page ? acc[ee][P - 1][2 * j + c] : acc[ee][0][2 * j + c];
              sc[2 * j + c] = fmaf(s, fmaf(z, nqsum[e][c], x), sc[2 * j + c]);
            }
          }
        }
      }
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
      // ---- O^T += V^T (p s)^T.  A page's product takes its own columns' probabilities, zeros for the other's.
#pragma unroll
      for (int e = 0; e < NG; ++e) {
        uint32_t ph[2], pl[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float s = vp[j].scale(e), z = vp[j].zero(e, z_magic);
          const float x0 = pr[2 * j] * s, x1 = pr[2 * j + 1] * s;
          base[e][0] = fmaf(x0, z, base[e][0]);
          base[e][1] = fmaf(x1, z, base[e][1]);
          const uint32_t hi = pack_bf16x2(x0, x1);
          ph[j] = transpose_8x8(hi);
          pl[j] = transpose_8x8(
              pack_bf16x2(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xffff0000u)));
        }
#pragma unroll
        for (int a = 0; a < P; ++a) {
          const bool on = P == 1 || (g >> 2) == a;  // as an operand, this lane holds column g
          const uint32_t h0_ = on ? ph[0] : 0u, h1_ = on ? ph[1] : 0u, l0_ = on ? pl[0] : 0u, l1_ = on ? pl[1] : 0u;
          const uint4 vw = *reinterpret_cast<const uint4*>(stage + a * R::BYTES + R::V_OFF + (e * 32 + lane) * 16);
          const uint32_t w4[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w = w4[j];
            const uint32_t a0 = decode(w << 3, geo.v_magic), a1 = decode(w >> 1, geo.v_magic);
            const uint32_t a2 = decode(w >> 5, geo.v_magic), a3 = decode(w >> 9, geo.v_magic);
            mma_16816(o[e * 4 + j], a0, a1, a2, a3, h0_, h1_);
            mma_16816(o[e * 4 + j], a0, a1, a2, a3, l0_, l1_);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
    }

    // ---- this warp's state to shared memory, then the CTA's to global memory
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[c] += __shfl_xor_sync(0xffffffffu, l[c], off);
#pragma unroll
        for (int e = 0; e < NG; ++e) base[e][c] += __shfl_xor_sync(0xffffffffu, base[e][c], off);
      }
    }
    float* my = merge + warp * C::MERGE;
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
      *reinterpret_cast<float2*>(at) = make_float2(o[x][0] - base[x / 4][0], o[x][2] - base[x / 4][0]);
      *reinterpret_cast<float2*>(at + C::OROW) = make_float2(o[x][1] - base[x / 4][1], o[x][3] - base[x / 4][1]);
    }
    named_barrier_sync(1, NW * 32);
    const bool starts = first_step == 0, ends = first_step + seg_steps == cur.ns;
    const int64_t slot = 2 * b + (starts ? 1 : 0);
    for (int w = threadIdx.x; w < heads * (D / 4); w += NW * 32) {
      const int r = w / (D / 4), x = w % (D / 4) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int v = 0; v < NW * P; ++v) M = fmaxf(M, merge[v / P * C::MERGE + v % P * TILE + r]);
      float L = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < NW * P; ++v) {
        const float* src = merge + v / P * C::MERGE;
        const int vr = v % P * TILE + r;
        const float wl = src[ROWS + vr];
        if (wl == 0.f) continue;  // a row without tokens
        const float f = ex2_approx(src[vr] - M);
        const float4 y = *reinterpret_cast<const float4*>(src + 2 * ROWS + vr * C::OROW + x);
        L = fmaf(wl, f, L);
        O.x = fmaf(y.x, f, O.x); O.y = fmaf(y.y, f, O.y);
        O.z = fmaf(y.z, f, O.z); O.w = fmaf(y.w, f, O.w);
      }
      const float inv = 1.f / L;
      O.x *= inv; O.y *= inv; O.z *= inv; O.w *= inv;
      if (starts && ends) {
        const int64_t row = static_cast<int64_t>(seg_n) * p.Hq + kvh * G + h0 + r;
        *reinterpret_cast<uint2*>(p.o + row * D + x) = make_uint2(pack_bf16x2(O.x, O.y), pack_bf16x2(O.z, O.w));
        if (x == 0 && p.lse != nullptr) p.lse[row] = (M + log2f(L)) * LN2;
      } else {
        *reinterpret_cast<float4*>(ws.o + (slot * ROWS + r) * D + x) = O;
        if (x == 0) {
          ws.m[slot * ROWS + r] = M;
          ws.l[slot * ROWS + r] = L;
        }
      }
    }
    if (starts && !ends) {
      // the share that holds the sequence's last step: step x lies in share ((x + 1) shares - 1) / W
      const long long past = lo + seg + cur.ns;
      cut = make_int4(seg_n, seg_u, static_cast<int>(mul_div(past * shares - 1, 1, W)), 1);
    }
    seg = seg_end;
    if (seg < count) {
      cur.advance(seg_steps, p.seq_lens, N, units, p.max_blocks);
      named_barrier_sync(1, NW * 32);  // the merge buffer is free again
    }
  }
  if (threadIdx.x == 0) ws.desc[b] = cut;
  if (!ok && lane == 0) set_error(&g_decode_q4_status, kDevWaitTimeout);
}

// One CTA a share: merges the partials of the cut sequence that starts there, if there is one.
// RS groups of threads take every RS-th partial.
template <int D, int P>
__global__ void __launch_bounds__(1024) combine_q4_kernel(const DecodeQ4Params p, const Q4Geometry geo) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int TILE = ROWS / P;
  constexpr int COLS = TILE * D / 4;  // threads that cover the outputs, 4 columns each
  constexpr int RS = 1024 / COLS;
  __shared__ float4 s_o[RS > 1 ? RS - 1 : 1][COLS];
  __shared__ float s_l[RS > 1 ? RS - 1 : 1][COLS];
  const Workspace ws = carve<D>(p.workspace, geo.grid);
  const int4 d = ws.desc[blockIdx.x];
  if (d.w == 0) return;
  const int G = p.Hq / p.Hkv, kvh = d.y / geo.tiles, h0 = d.y % geo.tiles * TILE;
  const int heads = G - h0 < TILE ? G - h0 : TILE;
  const int col = threadIdx.x % COLS, grp = threadIdx.x / COLS;
  const int r = col / (D / 4), x = col % (D / 4) * 4;
  const int first = blockIdx.x;
  const int count = d.z - first + 1;
  // partial j: the cut sequence's start, then the shares that continue it
  auto slot_of = [&](int j) { return static_cast<int64_t>(j == 0 ? 2 * first + 1 : 2 * (first + j)) * ROWS + r; };
  float M = -INFINITY, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < heads) {
    for (int j = 0; j < count; ++j) M = fmaxf(M, ws.m[slot_of(j)]);
#pragma unroll 4
    for (int j = grp; j < count; j += RS) {
      const int64_t s = slot_of(j);
      const float f = ws.l[s] * ex2_approx(ws.m[s] - M);
      const float4 y = *reinterpret_cast<const float4*>(ws.o + s * D + x);
      L += f;
      O.x = fmaf(y.x, f, O.x); O.y = fmaf(y.y, f, O.y);
      O.z = fmaf(y.z, f, O.z); O.w = fmaf(y.w, f, O.w);
    }
  }
  if constexpr (RS > 1) {
    if (grp > 0) {
      s_o[grp - 1][col] = O;
      s_l[grp - 1][col] = L;
    }
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int j = 0; j < RS - 1; ++j) {
      const float4 y = s_o[j][col];
      L += s_l[j][col];
      O.x += y.x; O.y += y.y; O.z += y.z; O.w += y.w;
    }
  }
  if (r >= heads) return;
  const float inv = 1.f / L;
  const int64_t row = static_cast<int64_t>(d.x) * p.Hq + kvh * G + h0 + r;
  *reinterpret_cast<uint2*>(p.o + row * D + x) =
      make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
  if (x == 0 && p.lse != nullptr) p.lse[row] = (M + log2f(L)) * LN2;
}

// CTAs of the grid: every SM filled (the same count for each variant)
int grid_of_device() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms * Cfg<128, 1>::CTAS;
}

template <int D, int P>
cudaError_t launch(const DecodeQ4Params& p, cudaStream_t stream) {
  using C = Cfg<D, P>;
  Q4Geometry geo;
  geo.grid = grid_of_device();
  if (geo.grid <= 0) return cudaErrorInvalidDevice;
  geo.tiles = (p.Hq / p.Hkv + C::TILE - 1) / C::TILE;
  geo.units = p.Hkv * geo.tiles;
  geo.k_magic = K_MAGIC;
  geo.v_magic = V_MAGIC;
  auto kern = decode_q4_kernel<D, P>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::ALLOC);
  if (e != cudaSuccess) return e;
  kern<<<geo.grid, C::THREADS, C::ALLOC, stream>>>(p, geo);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(geo.grid);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_q4_kernel<D, P>, p, geo);
}

template <int D>
cudaError_t launch_for(const DecodeQ4Params& p, cudaStream_t stream) {
  return p.Hq / p.Hkv <= ROWS / 2 ? launch<D, 2>(p, stream) : launch<D, 1>(p, stream);
}

}  // namespace

size_t decode_q4_workspace_bytes(int d) {
  const size_t grid = static_cast<size_t>(grid_of_device());
  return grid * 16 + 2 * grid * ROWS * (static_cast<size_t>(d) + 2) * sizeof(float);
}

cudaError_t decode_q4_launch(int d, const DecodeQ4Params& p, cudaStream_t stream) {
  if (d == 64) return launch_for<64>(p, stream);
  if (d == 128) return launch_for<128>(p, stream);
  if (d == 256) return launch_for<256>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t decode_q4_status(uint32_t* out, bool clear) { return read_status(g_decode_q4_status, out, clear); }

}  // namespace attn
