// Argument checks that the entry points of the serving step share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "attn.h"

namespace attn {
namespace api {

constexpr int kPage = 16;
constexpr int64_t kMaxTokens = int64_t(1) << 30;

inline bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline bool given(const void* p, uintptr_t bytes) { return p != nullptr && aligned(p, bytes); }
inline attn_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }
inline bool head_dim(int d) { return d == 64 || d == 128 || d == 256; }
// tokens of heads x d values, `stride` elements apart: rows start on 16 bytes and do not overlap
inline bool token_stride(int64_t stride, int heads, int d) {
  return stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * d && stride <= (int64_t(1) << 32);
}

// Arguments shared by the entry points that read a quantised cache, or its key bounds, through a block table.
inline attn_status_t check_paged(const void* cache, const int32_t* block_table, const int32_t* seq_lens, int num_seqs,
                                 int Hkv, int d, int page_size, int max_blocks_per_seq, int num_blocks) {
  if (!given(cache, 16) || !given(block_table, 4) || !given(seq_lens, 4)) return ATTN_ERR_INVALID_ARG;
  if (num_seqs < 1 || num_seqs > 65535 || Hkv < 1 || Hkv > 65535 || max_blocks_per_seq < 1 || num_blocks < 1)
    return ATTN_ERR_INVALID_ARG;
  if (page_size != kPage || !head_dim(d)) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_blocks) * kPage > kMaxTokens ||
      static_cast<int64_t>(max_blocks_per_seq) * kPage > kMaxTokens)
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// the read-back numbers a sequence's records in 32 bits
inline bool records_fit(int max_blocks_per_seq, int Hkv) {
  return static_cast<int64_t>(max_blocks_per_seq) * Hkv <= (int64_t(1) << 31) - 1;
}

inline size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Prefill over a quantised cache reads the sequences back into the workspace: what attn_prefill_paged would refuse is
// refused before anything is enqueued, and `p` (GatherQ4Params or GatherF8Params) is filled in.
template <class Gather>
attn_status_t check_prefill_readback(const void* q, const void* cache, const int32_t* block_table,
                                     const int32_t* cu_seqlens_q, const int32_t* seq_lens, const void* o,
                                     const float* lse, int num_seqs, int max_seqlen_q, int total_q, int Hq, int Hkv,
                                     int d, int page_size, int max_blocks_per_seq, int num_blocks, float scale,
                                     void* workspace, size_t workspace_bytes, Gather& p) {
  const attn_status_t chk =
      check_paged(cache, block_table, seq_lens, num_seqs, Hkv, d, page_size, max_blocks_per_seq, num_blocks);
  if (chk != ATTN_OK) return chk;
  if (!given(q, 16) || !given(o, 16) || !aligned(lse, 4) || !given(cu_seqlens_q, 4)) return ATTN_ERR_INVALID_ARG;
  if (max_seqlen_q < 1 || total_q < 1 || total_q > kMaxTokens || Hq < 1 || Hq > 65535 || Hq % Hkv != 0 ||
      static_cast<int64_t>(Hq) * d > (1 << 30))
    return ATTN_ERR_INVALID_ARG;
  const int64_t q_tiles = (static_cast<int64_t>(max_seqlen_q) + 127) / 128;
  if (q_tiles > 65535 || q_tiles * num_seqs * Hq > (int64_t(1) << 30)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  const size_t need = attn_prefill_q4_workspace_bytes(num_seqs, Hkv, d, max_blocks_per_seq);
  if (need == 0) return ATTN_ERR_INVALID_ARG;
  if (!given(workspace, 256) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
  const size_t half = up256(static_cast<size_t>(num_seqs) * max_blocks_per_seq * kPage * Hkv * d * 2);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.cache = static_cast<const uint8_t*>(cache);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.k_out = reinterpret_cast<__nv_bfloat16*>(ws);
  p.v_out = reinterpret_cast<__nv_bfloat16*>(ws + half);
  p.out_table = reinterpret_cast<int32_t*>(ws + 2 * half);
  p.N = num_seqs;
  p.Hkv = Hkv;
  p.d = d;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  return ATTN_OK;
}

}  // namespace api
}  // namespace attn
