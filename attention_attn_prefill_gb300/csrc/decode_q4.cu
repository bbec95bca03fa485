// Single-token attention over the 4-bit paged cache (format and layout: cache_q4.cuh).
//
// With K = s_g (c - z_g) and V likewise, per group g of 64 channels,
//   score = sum_g s_g (q . c - z_g sum q),     O = sum_tokens p s c - sum_tokens p s z,
// so the codes themselves are the matrix operands: a code becomes a bf16 number by one mask and one
// or (16 + c, exact, its nibble on the upper mantissa bits), and scales and zero points are applied
// to the 16 scores of a page's token tile and to its 16 probabilities, not to the d values of a token.
//
// S = Q K^T has the query heads of a KV head as rows (up to 8 a tile) and tokens as columns; its
// accumulator layout is that of the right-hand operand of O^T = V^T P^T, so the probabilities go from
// one product to the next in registers.  p s is split into two bf16 numbers (16 bits together): one
// alone would add an error as large as the output's own rounding.
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

constexpr int TILE = 8;  // query heads a tile
constexpr float RESCALE_LOG2_THRESHOLD = 8.0f;
constexpr float LN2 = 0.693147180559945309f;
constexpr uint32_t CODE_MASK = 0x00780078u;   // a nibble on mantissa bits 3..6 of both halves
constexpr uint32_t CODE_MAGIC = 0x41804180u;  // 16.0: with the nibble, 16 + c
constexpr int MIN_SHARE = 8;                  // pages a CTA takes at least

template <int D>
struct Cfg {
  static constexpr int NW = D == 256 ? 6 : 8;     // warps a CTA
  static constexpr int NS = D == 256 ? 2 : 3;     // records in flight a warp
  static constexpr int CTAS = 2;                  // CTAs an SM
  static constexpr int STAGE = (Record<D>::BYTES + 127) & ~127;
  static constexpr int OROW = D + 8;              // floats of a head's row in the merge buffer
  static constexpr int MERGE = 2 * TILE + TILE * OROW;  // floats a warp: m, l, o
  static constexpr int MERGE_OFF = NW * NS * STAGE;
  static constexpr int BAR_OFF = MERGE_OFF + NW * MERGE * 4;
  static constexpr int ALLOC = BAR_OFF + NW * NS * 8;
  static_assert(CTAS * (ALLOC + 1024 + 256) <= 228 * 1024, "shared memory budget");
};

struct Q4Geometry {
  int grid, tiles, units;  // CTAs, head tiles a KV head, (KV head, tile) pairs a sequence
};

// What the workspace holds: the shares' descriptors, then the partials' o, m and l.
struct Workspace {
  int4* desc;    // [grid]: (sequence, unit, last share, 1) of the cut sequence that starts in share b, or w = 0
  float* o;      // [2 grid][TILE][d]: index 2 b: continued from the share before, 2 b + 1: starts here
  float *m, *l;  // [2 grid][TILE]
};

template <int D>
__device__ Workspace carve(void* ws, int grid) {
  Workspace w;
  w.desc = static_cast<int4*>(ws);
  w.o = reinterpret_cast<float*>(w.desc + grid);
  w.m = w.o + static_cast<size_t>(2) * grid * TILE * D;
  w.l = w.m + static_cast<size_t>(2) * grid * TILE;
  return w;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int clamped_len(const int32_t* lens, int n, int max_blocks) {
  const int L = lens[n];
  return L < 0 ? 0 : (L > max_blocks * PAGE ? max_blocks * PAGE : L);
}
__device__ __forceinline__ int pages_of(const int32_t* lens, int n, int max_blocks) {
  return (clamped_len(lens, n, max_blocks) + PAGE - 1) / PAGE;
}

// Position in the (sequence, unit, page) list.
struct Cursor {
  int n, u, page, np;
  __device__ __forceinline__ void advance(int step, const int32_t* lens, int N, int units, int max_blocks) {
    page += step;
    while (page >= np) {
      page -= np;
      if (++u == units) {
        u = 0;
        do {
          if (++n >= N) {  // past the end of the list: nothing there is read
            n = N;
            np = 0x7fffffff;
            return;
          }
          np = pages_of(lens, n, max_blocks);
        } while (np == 0);
      }
    }
  }
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::NW * 32, Cfg<D>::CTAS)
    decode_q4_kernel(const DecodeQ4Params p, const Q4Geometry geo) {
  using C = Cfg<D>;
  using R = Record<D>;
  constexpr int NW = C::NW, NS = C::NS, NG = R::NG, THREADS = NW * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_warp[NW];
  __shared__ long long s_before;
  __shared__ int s_n;
  float* merge = reinterpret_cast<float*>(smem + C::MERGE_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int N = p.N, G = p.Hq / p.Hkv, units = geo.units;

  // ---- total pages, and the sequence that holds this share's first page
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&bars[warp * NS + i], 1);
    fence_mbar_init();
  }
  const int chunk = (N + THREADS - 1) / THREADS;
  const int n_lo = static_cast<int>(threadIdx.x) * chunk < N ? threadIdx.x * chunk : N;
  const int n_hi = n_lo + chunk < N ? n_lo + chunk : N;
  long long mine = 0;
  for (int n = n_lo; n < n_hi; ++n) {
    const int L = p.seq_lens[n];
    if (blockIdx.x == 0 && (L < 0 || L > p.max_blocks * PAGE)) set_error(&g_decode_q4_status, kDevBadSplit);
    mine += pages_of(p.seq_lens, n, p.max_blocks);
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
  for (int i = 0; i < NW; ++i) {
    if (i < warp) incl += s_warp[i];
    total += s_warp[i];
  }
  const long long W = total * units;
  long long shares = W / MIN_SHARE;
  shares = shares < 1 ? 1 : (shares > geo.grid ? geo.grid : shares);
  const int b = blockIdx.x;
  const long long lo = b < shares ? b * W / shares : W, hi = b < shares ? (b + 1) * W / shares : W;
  const int npg = static_cast<int>(hi - lo);
  const long long before_mine = (incl - mine) * units;
  if (npg > 0 && before_mine <= lo && lo < incl * units) {
    long long at = before_mine;
    int n = n_lo;
    for (;; ++n) {
      const long long w = static_cast<long long>(pages_of(p.seq_lens, n, p.max_blocks)) * units;
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
  if (npg <= 0) {
    if (threadIdx.x == 0) ws.desc[b] = make_int4(0, 0, 0, 0);
    return;
  }

  Cursor cur;  // the share's first page, then each segment's
  cur.n = s_n;
  cur.np = pages_of(p.seq_lens, cur.n, p.max_blocks);
  const long long rel = lo - s_before;
  cur.u = static_cast<int>(rel / cur.np);
  cur.page = static_cast<int>(rel % cur.np);

  // ---- this warp's ring: page i of the share belongs to warp i % NW
  uint8_t* stages = smem + warp * NS * C::STAGE;
  uint64_t* my_bars = bars + warp * NS;
  const int n_my = npg > warp ? (npg - warp + NW - 1) / NW : 0;
  Cursor icur = cur;
  if (warp > 0) icur.advance(warp, p.seq_lens, N, units, p.max_blocks);
  int pid = 0;  // physical page at icur, fetched one page ahead of its use
  auto fetch_pid = [&](int k) {
    if (k < n_my) pid = p.block_table[static_cast<int64_t>(icur.n) * p.max_blocks + icur.page];
  };
  auto issue = [&](int k) {
    int id = pid;
    if (id < 0 || id >= p.num_blocks) {
      set_error(&g_decode_q4_status, kDevBadPage);
      id = 0;
    }
    mbar_arrive_expect_tx(&my_bars[k % NS], R::BYTES);
    bulk_load(stages + k % NS * C::STAGE,
              p.cache + (static_cast<int64_t>(id) * p.Hkv + icur.u / geo.tiles) * R::BYTES, R::BYTES, &my_bars[k % NS]);
    icur.advance(NW, p.seq_lens, N, units, p.max_blocks);
    fetch_pid(k + 1);
  };
  if (lane == 0) {
    fetch_pid(0);
    for (int k = 0; k < n_my && k < NS; ++k) issue(k);
  }
  __syncwarp();

  const float c2 = p.scale_log2;
  bool ok = true;
  int k = 0;       // pages this warp has taken
  int landed = 0;  // of which the copy was seen to land
  int i = warp;    // share index of its next page
  int4 cut = make_int4(0, 0, 0, 0);
  for (int seg = 0; seg < npg;) {
    const int seg_n = cur.n, seg_u = cur.u, first_page = cur.page;
    const int seg_pages = cur.np - first_page < npg - seg ? cur.np - first_page : npg - seg;
    const int seg_end = seg + seg_pages;
    const int len = clamped_len(p.seq_lens, seg_n, p.max_blocks);
    const int kvh = seg_u / geo.tiles, h0 = seg_u % geo.tiles * TILE;
    const int heads = G - h0 < TILE ? G - h0 : TILE;
    const __nv_bfloat16* q_head = p.q + (static_cast<int64_t>(seg_n) * p.Hq + kvh * G + h0) * D;

    // ---- queries: row g of the tile; channels 64 e + 16 t + 8 h .. + 7, paired as the K words pair them
    uint32_t qa[NG][2][4];
    float qsum[NG];
#pragma unroll
    for (int e = 0; e < NG; ++e) {
      qsum[e] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (g < heads) x = *reinterpret_cast<const uint4*>(q_head + g * D + 64 * e + 16 * t + 8 * h);
        qa[e][h][0] = __byte_perm(x.x, x.z, 0x5410);  // channels 0, 4
        qa[e][h][1] = __byte_perm(x.x, x.z, 0x7632);  // 1, 5
        qa[e][h][2] = __byte_perm(x.y, x.w, 0x5410);  // 2, 6
        qa[e][h][3] = __byte_perm(x.y, x.w, 0x7632);  // 3, 7
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) qsum[e] += __uint_as_float(w[j] << 16) + __uint_as_float(w[j] & 0xffff0000u);
      }
      qsum[e] += __shfl_xor_sync(0xffffffffu, qsum[e], 1);
      qsum[e] += __shfl_xor_sync(0xffffffffu, qsum[e], 2);
    }

    float m = -INFINITY, l = 0.f;  // of head g: raw-score max that o and l refer to, this lane's share of the sum
    float o[D / 16][4];            // channels 16 i + 2 g (0, 1) and + 1 (2, 3) of heads 2 t and 2 t + 1
    float base[NG];                // sum of p s (16 + z) of head g over this lane's tokens
#pragma unroll
    for (int x = 0; x < D / 16; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
#pragma unroll
    for (int e = 0; e < NG; ++e) base[e] = 0.f;
    bool first = true;

    for (; i < seg_end; i += NW, ++k) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&my_bars[k % NS], (k / NS) & 1));
      if (!ok) continue;
      landed = k + 1;
      const uint8_t* rec = stages + k % NS * C::STAGE;
      const int token0 = (first_page + i - seg) * PAGE;
      const int valid = len - token0 < PAGE ? len - token0 : PAGE;

      // ---- S: tokens 2 t, 2 t + 1 (tile 0) and + 8 (tile 1) of head g; K words of tokens g and g + 8
      float sc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int pr = 0; pr < NG / R::PAIR; ++pr) {
        uint32_t kw[2][2 * R::PAIR];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const uint8_t* row = rec + R::K_OFF + (g + 8 * nt) * (D / 2) + pr * (32 * R::PAIR) + t * (8 * R::PAIR);
          if constexpr (R::PAIR == 2) {
            const uint4 x = *reinterpret_cast<const uint4*>(row);
            kw[nt][0] = x.x; kw[nt][1] = x.y; kw[nt][2] = x.z; kw[nt][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(row);
            kw[nt][0] = x.x; kw[nt][1] = x.y;
          }
        }
#pragma unroll
        for (int ee = 0; ee < R::PAIR; ++ee) {
          const int e = pr * R::PAIR + ee;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w = kw[nt][ee * 2 + h];
              const uint32_t b0 = (w & CODE_MASK) | CODE_MAGIC;
              const uint32_t b1 = (__funnelshift_r(w, w, 4) & CODE_MASK) | CODE_MAGIC;
              const uint32_t b2 = (__funnelshift_r(w, w, 8) & CODE_MASK) | CODE_MAGIC;
              const uint32_t b3 = (__funnelshift_r(w, w, 12) & CODE_MASK) | CODE_MAGIC;
              mma_16816(acc, qa[e][h][0], 0u, qa[e][h][1], 0u, b0, b1);
              mma_16816(acc, qa[e][h][2], 0u, qa[e][h][3], 0u, b2, b3);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t par =
                  reinterpret_cast<const uint16_t*>(rec + R::KP_OFF)[(8 * nt + 2 * t + j) * NG + e];
              const float s = __uint_as_float((par & 0xfff0u) << 16);
              const float z16 = __uint_as_float(0x41800000u | (par & 15u) << 19);  // 16 + z
              sc[nt][j] = fmaf(s, fmaf(-z16, qsum[e], acc[j]), sc[nt][j]);
            }
          }
        }
      }
      // ---- online softmax of row g
      if (valid < PAGE) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (8 * nt + 2 * t + j >= valid) sc[nt][j] = -INFINITY;
      }
      float mx = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (first) {
        m = mx;
        first = false;
      } else {
        const bool grow = (mx - m) * c2 > RESCALE_LOG2_THRESHOLD;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2_approx((m - mx) * c2) : 1.f;
          if (grow) m = mx;
          l *= f;
#pragma unroll
          for (int e = 0; e < NG; ++e) base[e] *= f;
          const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            o[x][0] *= f0; o[x][1] *= f1;
            o[x][2] *= f0; o[x][3] *= f1;
          }
        }
      }
      const float mc = m * c2;
      float pr[2][2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          pr[nt][j] = ex2_approx(fmaf(sc[nt][j], c2, -mc));
          l += pr[nt][j];
        }
      // ---- O^T += V^T (p s)^T
#pragma unroll
      for (int e = 0; e < NG; ++e) {
        uint32_t hi[2], lo_[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          float x[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int token = 8 * nt + 2 * t + j;
            uint32_t par = reinterpret_cast<const uint16_t*>(rec + R::VP_OFF)[token * NG + e];
            if (token >= valid) par = 0;  // whatever lies past the sequence: 0 * NaN is not 0
            x[j] = pr[nt][j] * __uint_as_float((par & 0xfff0u) << 16);
            base[e] = fmaf(x[j], __uint_as_float(0x41800000u | (par & 15u) << 19), base[e]);
          }
          hi[nt] = pack_bf16x2(x[0], x[1]);
          lo_[nt] = pack_bf16x2(x[0] - __uint_as_float(hi[nt] << 16), x[1] - __uint_as_float(hi[nt] & 0xffff0000u));
        }
        const uint4 vw = *reinterpret_cast<const uint4*>(rec + R::V_OFF + (e * 32 + lane) * 16);
        const uint32_t w4[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = w4[j];
          const uint32_t a0 = ((w << 3) & CODE_MASK) | CODE_MAGIC;
          const uint32_t a1 = ((w >> 1) & CODE_MASK) | CODE_MAGIC;
          const uint32_t a2 = ((w >> 5) & CODE_MASK) | CODE_MAGIC;
          const uint32_t a3 = ((w >> 9) & CODE_MASK) | CODE_MAGIC;
          mma_16816(o[e * 4 + j], a0, a1, a2, a3, hi[0], hi[1]);
          mma_16816(o[e * 4 + j], a0, a1, a2, a3, lo_[0], lo_[1]);
        }
      }
      __syncwarp();
      if (lane == 0 && k + NS < n_my) {
        fence_proxy_async_smem();
        issue(k + NS);
      }
      __syncwarp();
    }

    // ---- this warp's state to shared memory, then the CTA's to global memory
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
#pragma unroll
    for (int e = 0; e < NG; ++e) {
      base[e] += __shfl_xor_sync(0xffffffffu, base[e], 1);
      base[e] += __shfl_xor_sync(0xffffffffu, base[e], 2);
    }
    float* my = merge + warp * C::MERGE;
    if (t == 0) {
      my[g] = first ? -INFINITY : m * c2;
      my[TILE + g] = l;
    }
#pragma unroll
    for (int e = 0; e < NG; ++e) {
      const float b0 = __shfl_sync(0xffffffffu, base[e], 8 * t), b1 = __shfl_sync(0xffffffffu, base[e], 8 * t + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = e * 4 + j;
        float* at = my + 2 * TILE + 2 * t * C::OROW + 16 * x + 2 * g;
        *reinterpret_cast<float2*>(at) = make_float2(o[x][0] - b0, o[x][2] - b0);
        *reinterpret_cast<float2*>(at + C::OROW) = make_float2(o[x][1] - b1, o[x][3] - b1);
      }
    }
    __syncthreads();
    const bool starts = first_page == 0, ends = first_page + seg_pages == cur.np;
    const int64_t slot = 2 * b + (starts ? 1 : 0);
    for (int w = threadIdx.x; w < heads * (D / 4); w += THREADS) {
      const int r = w / (D / 4), x = w % (D / 4) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int v = 0; v < NW; ++v) M = fmaxf(M, merge[v * C::MERGE + r]);
      float L = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        const float* src = merge + v * C::MERGE;
        const float wl = src[TILE + r];
        if (wl == 0.f) continue;  // a warp without pages
        const float f = ex2_approx(src[r] - M);
        const float4 y = *reinterpret_cast<const float4*>(src + 2 * TILE + r * C::OROW + x);
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
        *reinterpret_cast<float4*>(ws.o + (slot * TILE + r) * D + x) = O;
        if (x == 0) {
          ws.m[slot * TILE + r] = M;
          ws.l[slot * TILE + r] = L;
        }
      }
    }
    if (starts && !ends) {
      // the share that holds the sequence's last page: unit x lies in share ((x + 1) shares - 1) / W
      const long long past = lo + seg + cur.np;
      cut = make_int4(seg_n, seg_u, static_cast<int>((past * shares - 1) / W), 1);
    }
    seg = seg_end;
    if (seg < npg) cur.advance(seg_pages, p.seq_lens, N, units, p.max_blocks);
    __syncthreads();  // the merge buffer is free again
  }
  if (threadIdx.x == 0) ws.desc[b] = cut;
  if (!ok && lane == 0) {
    set_error(&g_decode_q4_status, kDevWaitTimeout);
    // copies in flight must land before the CTA's shared memory is given back
    for (int j = landed; j < n_my && j < landed + NS; ++j) mbar_wait(&my_bars[j % NS], (j / NS) & 1);
  }
}

// One CTA a share: merges the partials of the cut sequence that starts there, if there is one.
// RS groups of threads take every RS-th partial.
template <int D>
__global__ void __launch_bounds__(1024) combine_q4_kernel(const DecodeQ4Params p, const Q4Geometry geo) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  auto slot_of = [&](int j) { return static_cast<int64_t>(j == 0 ? 2 * first + 1 : 2 * (first + j)) * TILE + r; };
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

int grid_of_device(int d) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms * (d == 64 ? Cfg<64>::CTAS : d == 128 ? Cfg<128>::CTAS : Cfg<256>::CTAS);
}

template <int D>
cudaError_t launch(const DecodeQ4Params& p, cudaStream_t stream) {
  Q4Geometry geo;
  geo.grid = grid_of_device(D);
  if (geo.grid <= 0) return cudaErrorInvalidDevice;
  geo.tiles = (p.Hq / p.Hkv + TILE - 1) / TILE;
  geo.units = p.Hkv * geo.tiles;
  auto kern = decode_q4_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::ALLOC);
  if (e != cudaSuccess) return e;
  kern<<<geo.grid, Cfg<D>::NW * 32, Cfg<D>::ALLOC, stream>>>(p, geo);
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
  return cudaLaunchKernelEx(&cfg, combine_q4_kernel<D>, p, geo);
}

}  // namespace

size_t decode_q4_workspace_bytes(int d) {
  const size_t grid = static_cast<size_t>(grid_of_device(d));
  return grid * 16 + 2 * grid * TILE * (static_cast<size_t>(d) + 2) * sizeof(float);
}

cudaError_t decode_q4_launch(int d, const DecodeQ4Params& p, cudaStream_t stream) {
  if (d == 64) return launch<64>(p, stream);
  if (d == 128) return launch<128>(p, stream);
  if (d == 256) return launch<256>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t decode_q4_status(uint32_t* out, bool clear) { return read_status(g_decode_q4_status, out, clear); }

}  // namespace attn
