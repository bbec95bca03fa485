// What the decodes over quantised caches have in common: the (sequence, unit, step) list and its cursor, the matrix
// product of a warp, the partials of sequences that a share's end cuts, and the kernel that merges them.
//
// A unit is a tile of query heads of one KV head; a step is P pages of it.  The list is cut into contiguous shares,
// one a CTA.  At most two partials a CTA (continued from the share before, and cut at this one's end), so the
// workspace does not depend on the batch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm103.cuh"

namespace attn {
namespace shares {

constexpr int PAGE = 16;
constexpr int ROWS = 8;  // score columns of a warp: query heads, or heads of two pages
constexpr float LN2 = 0.693147180559945309f;

// a * b / c with c > 0; the quotient is below 2^63.  64-bit division costs over a hundred instructions,
// and the shares of all but the largest batches are counted in 32 bits.
__device__ __forceinline__ long long mul_div(long long a, long long b, long long c) {
  const long long n = a * b;
  if ((n | c) >> 32 == 0) return static_cast<uint32_t>(n) / static_cast<uint32_t>(c);
  return n / c;
}

// The sequence whose rows cu[n] .. cu[n + 1] - 1 would hold row r: the last n < N with cu[n] <= r (0: none).  Eight parts at
// a time, their loads in flight together: bisection would wait for log2 N of them one after another (64 sequences: 3.6 us).
// A step with one row a sequence finds it at once.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int N, int r) {
  if (r < N && cu[r] <= r && r < cu[r + 1]) return r;
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int step = (hi - lo + 7) >> 3;
    int parts = 0;
#pragma unroll
    for (int k = 1; k < 8; ++k) parts += lo + k * step < hi && cu[lo + k * step] <= r ? 1 : 0;
    lo += parts * step;
    hi = hi - lo < step ? hi : lo + step;
  }
  return lo;
}

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
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
  int n, u, step, ns, pages;  // ns steps and `pages` pages of sequence n
  __device__ __forceinline__ void enter(const int32_t* lens, int max_blocks) {
    pages = (clamped_len(lens, n, max_blocks) + PAGE - 1) / PAGE;
    ns = (pages + P - 1) / P;
  }
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
          enter(lens, max_blocks);
        } while (ns == 0);
      }
    }
  }
};

struct Geometry {
  int grid;          // CTAs
  bool by_unit;      // few (sequence, unit) pairs: a descriptor for each; else one for each share
  int tile;          // query heads a tile
  int tiles, units;  // tiles a KV head, (KV head, tile) pairs a sequence
};

// What the workspace holds: the shares' descriptors, then the partials' o, m and l.
struct Workspace {
  int4* desc;    // [grid]: (sequence, unit, first share, last share) of a cut sequence, or z = -1; of the one
                 // that starts in share b, or of pair sequence * units + unit
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

inline size_t workspace_bytes(int grid, int d) {
  const size_t g = grid;
  return g * 16 + 2 * g * ROWS * (static_cast<size_t>(d) + 2) * sizeof(float);
}

struct MergeParams {
  void* workspace;
  __nv_bfloat16* o;         // [N][Hq][d]
  float* lse;               // [N][Hq] or null
  const int32_t* seq_lens;  // [N], or null where every sequence has steps
  int N, Hq, Hkv, max_blocks;
};

// Merges the partials of descriptor blockIdx.x's sequence, if it was cut: a CTA of T threads takes HEADS query
// heads.  Each of RS groups of threads takes every RS-th partial, U of them in flight at a time, with a
// running maximum; then the groups' sums are merged.  A partial without tokens has the maximum -inf; a sequence of
// such partials alone gives 0 and -inf.
template <int D, int HEADS, int T>
__global__ void __launch_bounds__(T) combine_shares_kernel(const MergeParams p, const Geometry geo) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int COLS = HEADS * D / 4;  // threads that cover the heads' outputs, 4 columns each
  constexpr int RS = T / COLS;
  constexpr int U = RS > 4 ? 4 : 8;
  __shared__ float4 s_o[RS][COLS];
  __shared__ float s_m[RS][HEADS], s_l[RS][HEADS];
  const Workspace ws = carve<D>(p.workspace, geo.grid);
  const int col = threadIdx.x % COLS, grp = threadIdx.x / COLS;
  const int x = col % (D / 4) * 4, head = col / (D / 4);
  const int r = blockIdx.y * HEADS + head;
  // an empty sequence has no steps that could have written its pairs' descriptors
  if (geo.by_unit && p.seq_lens != nullptr && clamped_len(p.seq_lens, blockIdx.x / geo.units, p.max_blocks) == 0) return;
  const int4 d = ws.desc[blockIdx.x];
  const int G = p.Hq / p.Hkv, kvh = d.y / geo.tiles, h = d.y % geo.tiles * geo.tile + r;
  // after a wait that ran out (a recorded error) a descriptor may be missing: nothing of it is used
  if (d.z < 0 || d.w >= geo.grid || d.x < 0 || d.x >= p.N || d.y < 0 || d.y >= geo.units) return;
  const int first = d.z, count = h < G ? d.w - first + 1 : 0;
  float M = -INFINITY, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = grp; j0 < count; j0 += RS * U) {
    float m[U], l[U];
    float4 y[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int j = j0 + k * RS;
      m[k] = -INFINITY;
      if (j < count) {
        // partial j: the cut sequence's start, then the shares that continue it
        const int64_t s = static_cast<int64_t>(j == 0 ? 2 * first + 1 : 2 * (first + j)) * ROWS + r;
        m[k] = ws.m[s];
        l[k] = ws.l[s];
        y[k] = *reinterpret_cast<const float4*>(ws.o + s * D + x);
      }
    }
    float to = M;
#pragma unroll
    for (int k = 0; k < U; ++k) to = fmaxf(to, m[k]);
    if (to == -INFINITY) continue;  // no tokens so far
    const float f = ex2_approx(M - to);
    M = to;
    L *= f;
    O.x *= f; O.y *= f; O.z *= f; O.w *= f;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (j0 + k * RS >= count) break;
      const float fn = l[k] * ex2_approx(m[k] - to);
      L += fn;
      O.x = fmaf(y[k].x, fn, O.x); O.y = fmaf(y[k].y, fn, O.y);
      O.z = fmaf(y[k].z, fn, O.z); O.w = fmaf(y[k].w, fn, O.w);
    }
  }
  s_o[grp][col] = O;
  if (x == 0) {
    s_m[grp][head] = M;
    s_l[grp][head] = L;
  }
  __syncthreads();
  if (grp > 0 || h >= G) return;
#pragma unroll
  for (int k = 1; k < RS; ++k) {
    if (k >= count) break;  // the groups behind have no partials
    const float to = fmaxf(M, s_m[k][head]);
    if (to == -INFINITY) continue;
    const float fo = ex2_approx(M - to), fn = ex2_approx(s_m[k][head] - to);
    const float4 y = s_o[k][col];
    M = to;
    L = L * fo + s_l[k][head] * fn;
    O.x = O.x * fo + y.x * fn; O.y = O.y * fo + y.y * fn;
    O.z = O.z * fo + y.z * fn; O.w = O.w * fo + y.w * fn;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t row = static_cast<int64_t>(d.x) * p.Hq + kvh * G + h;
  *reinterpret_cast<uint2*>(p.o + row * D + x) =
      make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
  if (x == 0 && p.lse != nullptr) p.lse[row] = (M + log2f(L)) * LN2;
}

// The merge as a programmatic dependent of the kernel before it on `stream`.
// Few sequences and heads for many shares: many partials each, so every head gets a CTA (a sequence of
// 30000 tokens over the 4-bit cache, 16/2 heads, d = 256, 152 partials a head: 18 us against 40).  Else a cut
// sequence has two or three, and the CTAs that find nothing to do cost more (64 sequences of 4352, 32/8 heads: 71 us
// against 68).
template <int D, int TILE>
cudaError_t launch_combine(const MergeParams& p, const Geometry& geo, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (geo.by_unit) {
    const int heads = p.Hq / p.Hkv;
    cfg.gridDim = dim3(p.N * geo.units, heads < TILE ? heads : TILE);
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, combine_shares_kernel<D, 1, 256>, p, geo);
  }
  cfg.gridDim = dim3(geo.grid);
  cfg.blockDim = dim3(512);
  return cudaLaunchKernelEx(&cfg, combine_shares_kernel<D, TILE, 512>, p, geo);
}

}  // namespace shares
}  // namespace attn
