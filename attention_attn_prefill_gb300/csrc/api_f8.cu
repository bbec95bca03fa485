// C-ABI entry points of the 8-bit paged cache, attention over it, and block selection.  Argument checks and
// dispatch; see include/attn.h for the contract of each.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "attn.h"
#include "step.h"

using namespace attn::api;

namespace {

constexpr int kMostBlocks = attn::SELECT_MOST_BLOCKS;

// What both decodes over the 8-bit cache check and pass on
attn_status_t decode_f8(attn::DecodeF8Params& p, const void* q, const void* cache, const int32_t* block_table,
                        const int32_t* seq_lens, void* o, float* lse, int num_tokens, int num_seqs, int Hq, int Hkv, int d,
                        int page_size, int max_blocks_per_seq, int num_blocks, float scale, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const attn_status_t chk =
      check_paged(cache, block_table, seq_lens, num_seqs, Hkv, d, page_size, max_blocks_per_seq, num_blocks);
  if (chk != ATTN_OK) return chk;
  if (!given(q, 16) || !given(o, 16) || !aligned(lse, 4)) return ATTN_ERR_INVALID_ARG;
  if (Hq < 1 || Hq > 65535 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (!given(workspace, 16)) return ATTN_ERR_WORKSPACE;
  const size_t need = attn::decode_f8_workspace_bytes(d);
  if (need == 0) return ATTN_ERR_CUDA;
  if (workspace_bytes < need) return ATTN_ERR_WORKSPACE;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const uint8_t*>(cache);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.workspace = workspace;
  p.T = num_tokens;
  p.N = num_seqs;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * 1.4426950408889634f;
  return from_cuda(attn::decode_f8_launch(d, p, static_cast<cudaStream_t>(stream)));
}

bool select_fits(int num_tokens, int num_seqs, int Hkv, int max_blocks_per_seq) {
  return num_tokens >= 1 && num_tokens <= kMaxTokens && num_seqs >= 1 && num_seqs <= 65535 && Hkv >= 1 && Hkv <= 65535 &&
         max_blocks_per_seq >= 1 && max_blocks_per_seq <= kMostBlocks &&
         static_cast<int64_t>(num_tokens) * Hkv <= (int64_t(1) << 31) - 1 &&
         // the kernel numbers tiles of 16 blocks in 32 bits
         static_cast<int64_t>(num_seqs) * Hkv <= ((int64_t(1) << 31) - 1) / ((max_blocks_per_seq + 15) / 16);
}

}  // namespace

extern "C" {

size_t attn_cache_f8_record_bytes(int d) { return head_dim(d) ? static_cast<size_t>(32) * d + 16 : 0; }

attn_status_t attn_cache_append_f8(const void* k, long long k_stride, const void* v, long long v_stride,
                                   const int32_t* slots, void* cache, void* bounds, int num_tokens, int Hkv, int d,
                                   int page_size, int num_blocks, void* stream) {
  if (!given(k, 16) || !given(v, 16) || !given(slots, 4) || !given(cache, 16) || !aligned(bounds, 16))
    return ATTN_ERR_INVALID_ARG;
  if (num_tokens < 1 || num_tokens > kMaxTokens || Hkv < 1 || Hkv > 65535 || num_blocks < 1)
    return ATTN_ERR_INVALID_ARG;
  if (page_size != kPage || !head_dim(d)) return ATTN_ERR_UNSUPPORTED;
  if (!token_stride(k_stride, Hkv, d) || !token_stride(v_stride, Hkv, d) ||
      static_cast<int64_t>(num_blocks) * kPage > kMaxTokens)
    return ATTN_ERR_INVALID_ARG;
  attn::AppendF8Params p;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.slots = slots;
  p.cache = static_cast<uint8_t*>(cache);
  p.bounds = static_cast<__nv_bfloat16*>(bounds);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.num_slots = static_cast<int64_t>(num_blocks) * kPage;
  p.T = num_tokens;
  p.Hkv = Hkv;
  p.d = d;
  return from_cuda(attn::append_f8_launch(p, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_cache_gather_f8(const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                                   void* k_out, void* v_out, int num_seqs, int Hkv, int d, int page_size,
                                   int max_blocks_per_seq, int num_blocks, void* stream) {
  const attn_status_t chk =
      check_paged(cache, block_table, seq_lens, num_seqs, Hkv, d, page_size, max_blocks_per_seq, num_blocks);
  if (chk != ATTN_OK) return chk;
  if (!given(k_out, 16) || !given(v_out, 16) || !records_fit(max_blocks_per_seq, Hkv)) return ATTN_ERR_INVALID_ARG;
  attn::GatherF8Params p;
  p.cache = static_cast<const uint8_t*>(cache);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.out_table = nullptr;
  p.N = num_seqs;
  p.Hkv = Hkv;
  p.d = d;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  return from_cuda(attn::gather_f8_launch(p, static_cast<cudaStream_t>(stream)));
}

size_t attn_decode_f8_workspace_bytes(int d) { return head_dim(d) ? attn::decode_f8_workspace_bytes(d) : 0; }

attn_status_t attn_decode_paged_f8(const void* q, const void* cache, const int32_t* block_table,
                                   const int32_t* seq_lens, void* o, float* lse, int num_seqs, int Hq, int Hkv, int d,
                                   int page_size, int max_blocks_per_seq, int num_blocks, float scale,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  attn::DecodeF8Params p;
  p.cu = nullptr;
  p.blocks = nullptr;
  p.K = 0;
  return decode_f8(p, q, cache, block_table, seq_lens, o, lse, num_seqs, num_seqs, Hq, Hkv, d, page_size,
                   max_blocks_per_seq, num_blocks, scale, workspace, workspace_bytes, stream);
}

attn_status_t attn_decode_blocks_f8(const void* q, const void* cache, const int32_t* block_table,
                                    const int32_t* cu_seqlens_q, const int32_t* seq_lens, const int32_t* blocks,
                                    int num_selected, void* o, float* lse, int num_tokens, int num_seqs, int Hq, int Hkv,
                                    int d, int page_size, int max_blocks_per_seq, int num_blocks, float scale,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!given(blocks, 4) || !aligned(cu_seqlens_q, 4) || num_selected < 1 || num_selected > kMostBlocks ||
      num_tokens < 1 || num_tokens > kMaxTokens || (cu_seqlens_q == nullptr && num_tokens != num_seqs))
    return ATTN_ERR_INVALID_ARG;
  attn::DecodeF8Params p;
  p.cu = cu_seqlens_q;
  p.blocks = blocks;
  p.K = num_selected;
  return decode_f8(p, q, cache, block_table, seq_lens, o, lse, num_tokens, num_seqs, Hq, Hkv, d, page_size,
                   max_blocks_per_seq, num_blocks, scale, workspace, workspace_bytes, stream);
}

size_t attn_prefill_f8_workspace_bytes(int num_seqs, int Hkv, int d, int max_blocks_per_seq) {
  return attn_prefill_q4_workspace_bytes(num_seqs, Hkv, d, max_blocks_per_seq);  // the same pages in bf16
}

attn_status_t attn_prefill_paged_f8(const void* q, const void* cache, const int32_t* block_table,
                                    const int32_t* cu_seqlens_q, const int32_t* seq_lens, void* o, float* lse,
                                    int num_seqs, int max_seqlen_q, int total_q, int Hq, int Hkv, int d,
                                    int page_size, int max_blocks_per_seq, int num_blocks, float scale, int causal,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  attn::GatherF8Params p;
  const attn_status_t chk = check_prefill_readback(q, cache, block_table, cu_seqlens_q, seq_lens, o, lse, num_seqs,
                                                   max_seqlen_q, total_q, Hq, Hkv, d, page_size, max_blocks_per_seq,
                                                   num_blocks, scale, workspace, workspace_bytes, p);
  if (chk != ATTN_OK) return chk;
  const cudaError_t e = attn::gather_f8_launch(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  return attn_prefill_paged(q, p.k_out, p.v_out, p.out_table, cu_seqlens_q, seq_lens, o, lse, num_seqs, max_seqlen_q,
                            total_q, Hq, Hkv, d, page_size, max_blocks_per_seq, num_seqs * max_blocks_per_seq, scale,
                            causal, stream);
}

size_t attn_select_blocks_workspace_bytes(int num_tokens, int num_seqs, int max_seqlen_q, int Hkv, int d,
                                          int max_blocks_per_seq) {
  if (!head_dim(d) || max_seqlen_q < 1 || !select_fits(num_tokens, num_seqs, Hkv, max_blocks_per_seq)) return 0;
  return attn::select_blocks_workspace_bytes(num_tokens, num_seqs, max_seqlen_q, Hkv, d, max_blocks_per_seq);
}

attn_status_t attn_select_blocks(const void* q, const void* bounds, const int32_t* block_table,
                                 const int32_t* cu_seqlens_q, const int32_t* seq_lens, int32_t* blocks, int num_selected,
                                 int first, int last, int num_tokens, int num_seqs, int max_seqlen_q, int Hq, int Hkv,
                                 int d, int page_size, int max_blocks_per_seq, int num_blocks, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const attn_status_t chk =
      check_paged(bounds, block_table, seq_lens, num_seqs, Hkv, d, page_size, max_blocks_per_seq, num_blocks);
  if (chk != ATTN_OK) return chk;
  if (!given(q, 16) || !given(blocks, 4) || !aligned(cu_seqlens_q, 4)) return ATTN_ERR_INVALID_ARG;
  if (Hq < 1 || Hq > 65535 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  // the own block holds tokens behind the query: it is always among the last ones, and never chosen by its score
  if (first < 0 || last < 1 || num_selected < 1 || num_selected > kMostBlocks || first > num_selected ||
      last > num_selected - first)
    return ATTN_ERR_INVALID_ARG;
  if (max_seqlen_q < 1 || (cu_seqlens_q == nullptr && (num_tokens != num_seqs || max_seqlen_q != 1)))
    return ATTN_ERR_INVALID_ARG;
  if (max_blocks_per_seq > kMostBlocks) return ATTN_ERR_UNSUPPORTED;
  if (!select_fits(num_tokens, num_seqs, Hkv, max_blocks_per_seq)) return ATTN_ERR_INVALID_ARG;
  const int max_q = max_seqlen_q < num_tokens ? max_seqlen_q : num_tokens;
  const int64_t row_tiles = (static_cast<int64_t>(max_q) + 3) / 4;
  if (row_tiles * num_seqs * Hkv > (int64_t(1) << 30)) return ATTN_ERR_INVALID_ARG;
  if (!given(workspace, 256) ||
      workspace_bytes <
          attn::select_blocks_workspace_bytes(num_tokens, num_seqs, max_seqlen_q, Hkv, d, max_blocks_per_seq))
    return ATTN_ERR_WORKSPACE;
  attn::SelectBlocksParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.bounds = static_cast<const __nv_bfloat16*>(bounds);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu = cu_seqlens_q;
  p.blocks = blocks;
  p.workspace = workspace;
  p.T = num_tokens;
  p.N = num_seqs;
  p.max_q = max_q;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = d;
  p.K = num_selected;
  p.first = first;
  p.last = last;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  return from_cuda(attn::select_blocks_launch(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
