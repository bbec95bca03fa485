// Block tables, slot map, positions and sequence offsets of one serving step, from request lengths.
//
// Request n holds c_n cached tokens and brings w_n new ones.  It keeps its ceil(c_n / 16) pages and
// takes need_n = ceil((c_n + w_n) / 16) - ceil(c_n / 16) more from the free list, in request order, so
// both what a request's tokens are numbered from and which free pages it takes are exclusive prefix
// sums over the requests.  Token i of request n sits at position p = c_n + i of its sequence: slot
// page(p / 16) * 16 + p % 16.
//
// One launch: a decode step moves a few KB, so what it costs is latency.  Every CTA serves 1024
// consecutive tokens and scans the lengths itself (256 requests at a time, 8 bytes each, from L2)
// until the requests of its own tokens are behind it, instead of waiting for a scan kernel's result;
// it keeps the requests that own some of its tokens in shared memory, where each token finds its own
// by binary search.  CTA 0 goes through all requests and writes the per-request outputs.  64 requests of
// a token each take 2.7 us, an empty launch 2; 512 requests with 35,000 tokens 5.0 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "sm103.cuh"
#include "step.h"

namespace attn {

__device__ uint32_t g_step_tables_status;

namespace {

constexpr int PAGE = 16;
constexpr int THREADS = 256;
constexpr int TOKENS = 1024;  // per CTA

struct Owner {
  int start;   // first token of the request in the packed batch (may lie before this CTA's tokens)
  int request;
  int cached;
  int pages;   // index of the request's first free page (0 if it needs none), or -1: it takes part in nothing
};

__global__ void __launch_bounds__(THREADS) step_tables_kernel(const StepTablesParams p) {
  __shared__ Owner owners[TOKENS];  // each owns at least one of the CTA's tokens
  __shared__ long long warp_tok[THREADS / 32], warp_page[THREADS / 32], warp_used[THREADS / 32];
  __shared__ int warp_own[THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * TOKENS;
  const int t1 = p.T - t0 < TOKENS ? p.T : t0 + TOKENS;
  const long long room = static_cast<long long>(p.max_blocks) * PAGE;
  const bool all = blockIdx.x == 0;
  long long tok_base = 0, page_base = 0;  // sums over the requests before this round
  long long used = 0;                     // end of the free pages of this thread's last successful request
  int owned = 0;
  for (int base = 0; base < p.N && (all || tok_base < t1); base += THREADS) {
    const int n = base + threadIdx.x;
    int c = 0, w = 0;
    if (n < p.N) {
      c = p.cached_lens[n];
      w = p.new_lens[n];
    }
    const bool fits = c >= 0 && w >= 0 && static_cast<long long>(c) + w <= room;
    const long long rows = w > 0 ? w : 0;  // rows of the packed batch, also of a request that does not fit
    const long long need = fits ? (c + w + PAGE - 1) / PAGE - (c + PAGE - 1) / PAGE : 0;
    long long tok = rows, pg = need;  // inclusive sums within the warp
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, tok, off), b = __shfl_up_sync(0xffffffffu, pg, off);
      if (lane >= off) {
        tok += a;
        pg += b;
      }
    }
    if (lane == 31) {
      warp_tok[warp] = tok;
      warp_page[warp] = pg;
    }
    __syncthreads();
    long long tok_sum = 0, page_sum = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) {
        tok += warp_tok[i];
        pg += warp_page[i];
      }
      tok_sum += warp_tok[i];
      page_sum += warp_page[i];
    }
    const long long start = tok_base + tok - rows, first = page_base + pg - need;
    const bool ok = n < p.N && fits && (need == 0 || first + need <= p.num_free) && start + rows <= p.T;
    if (n < p.N && all) {
      if (!ok) set_error(&g_step_tables_status, kDevBadStep);
      p.seq_lens[n] = ok ? c + w : (c < 0 ? 0 : (c > room ? static_cast<int>(room) : c));
      const long long end = start + rows;
      p.cu_seqlens[n + 1] = end > 0x7fffffff ? 0x7fffffff : static_cast<int>(end);
      if (ok && need > 0) used = first + need;
    }
    const bool mine = n < p.N && rows > 0 && start < t1 && start + rows > t0;
    const unsigned vote = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) warp_own[warp] = __popc(vote);
    __syncthreads();  // also: the sums are read before the next round writes them
    int at = owned + __popc(vote & ((1u << lane) - 1u));
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) at += warp_own[i];
      owned += warp_own[i];
    }
    if (mine) owners[at] = Owner{static_cast<int>(start), n, c, ok ? (need > 0 ? static_cast<int>(first) : 0) : -1};
    tok_base += tok_sum;
    page_base += page_sum;
  }
  if (all) {
    // the ends grow with the request index: the largest over the threads is the last request's
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const long long a = __shfl_xor_sync(0xffffffffu, used, off);
      used = a > used ? a : used;
    }
    if (lane == 0) warp_used[warp] = used;
  }
  __syncthreads();  // owners and warp_used are complete
  if (all && threadIdx.x == 0) {
    for (int i = 1; i < THREADS / 32; ++i) used = warp_used[i] > used ? warp_used[i] : used;
    *p.pages_used = static_cast<int>(used);
    p.cu_seqlens[0] = 0;
  }
  for (int t = t0 + threadIdx.x; t < t1; t += THREADS) {
    int lo = 0, hi = owned;  // the last owner that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (owners[mid].start <= t) lo = mid + 1; else hi = mid;
    }
    int pos = 0, slot = -1;
    if (lo > 0 && t < tok_base) {
      const Owner o = owners[lo - 1];
      if (o.pages >= 0) {
        pos = o.cached + t - o.start;
        const int page = pos / PAGE, held = (o.cached + PAGE - 1) / PAGE;
        int32_t* row = p.block_table + static_cast<int64_t>(o.request) * p.max_blocks;
        const bool fresh = page >= held;
        const int id = fresh ? p.free_pages[o.pages + page - held] : row[page];
        if (id < 0 || id >= p.num_blocks) {
          set_error(&g_step_tables_status, kDevBadPage);
        } else {
          slot = id * PAGE + pos % PAGE;
          if (fresh && pos % PAGE == 0) row[page] = id;  // the page's first token enters it in the table
        }
      }
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
  }
}

}  // namespace

cudaError_t step_tables_launch(const StepTablesParams& p, cudaStream_t stream) {
  const int grid = p.T > TOKENS ? (p.T + TOKENS - 1) / TOKENS : 1;
  step_tables_kernel<<<grid, THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t step_tables_status(uint32_t* out, bool clear) { return read_status(g_step_tables_status, out, clear); }

}  // namespace attn
