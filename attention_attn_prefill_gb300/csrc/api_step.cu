// C-ABI entry points of the serving step: tables from request lengths, query/key norm with rotation,
// the 4-bit paged cache, and attention over it.  Argument checks and dispatch; see include/attn.h for
// the contract of each.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "attn.h"
#include "step.h"

using namespace attn::api;

namespace {

struct Ints {
  const int32_t* at;
  int64_t n;
};
bool overlap(const Ints& a, const Ints& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.n > 0 && b.n > 0 && x < y + 4 * b.n && y < x + 4 * a.n;
}

}  // namespace

extern "C" {

attn_status_t attn_step_tables(const int32_t* cached_lens, const int32_t* new_lens, const int32_t* free_pages,
                               int32_t* block_table, int32_t* seq_lens, int32_t* cu_seqlens, int32_t* positions,
                               int32_t* slots, int32_t* pages_used, int num_seqs, int num_tokens, int num_free,
                               int page_size, int max_blocks_per_seq, int num_blocks, void* stream) {
  if (!given(cached_lens, 4) || !given(new_lens, 4) || !given(block_table, 4) || !given(seq_lens, 4) ||
      !given(cu_seqlens, 4) || !given(pages_used, 4))
    return ATTN_ERR_INVALID_ARG;
  if (num_seqs < 1 || num_tokens < 0 || num_free < 0 || max_blocks_per_seq < 1 || num_blocks < 1)
    return ATTN_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!given(positions, 4) || !given(slots, 4))) return ATTN_ERR_INVALID_ARG;
  if (num_free > 0 && !given(free_pages, 4)) return ATTN_ERR_INVALID_ARG;
  if (page_size != kPage) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_blocks) * kPage > kMaxTokens ||
      static_cast<int64_t>(max_blocks_per_seq) * kPage > kMaxTokens || num_tokens > kMaxTokens ||
      num_seqs > (1 << 24))
    return ATTN_ERR_INVALID_ARG;
  // every CTA reads the lengths while the first writes its outputs: none may lie in another tensor of the call
  const Ints outs[] = {{seq_lens, num_seqs},   {cu_seqlens, int64_t(num_seqs) + 1}, {positions, num_tokens},
                       {slots, num_tokens},    {pages_used, 1},
                       {block_table, static_cast<int64_t>(num_seqs) * max_blocks_per_seq}};
  const Ints ins[] = {{cached_lens, num_seqs}, {new_lens, num_seqs}, {free_pages, num_free}};
  for (const Ints& out : outs) {
    for (const Ints& in : ins)
      if (overlap(out, in)) return ATTN_ERR_INVALID_ARG;
    for (const Ints& other : outs)
      if (&other != &out && overlap(out, other)) return ATTN_ERR_INVALID_ARG;
  }
  attn::StepTablesParams p;
  p.cached_lens = cached_lens;
  p.new_lens = new_lens;
  p.free_pages = free_pages;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu_seqlens = cu_seqlens;
  p.positions = positions;
  p.slots = slots;
  p.pages_used = pages_used;
  p.N = num_seqs;
  p.T = num_tokens;
  p.num_free = num_free;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  return from_cuda(attn::step_tables_launch(p, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_rope_table(float* table, int max_positions, int rot, double theta, void* stream) {
  if (!given(table, 16) || max_positions < 1 || rot < 1 || !std::isfinite(theta) || !(theta > 0.0))
    return ATTN_ERR_INVALID_ARG;
  if (rot % 16 != 0 || rot > 256) return ATTN_ERR_UNSUPPORTED;
  return from_cuda(attn::rope_table_launch(table, max_positions, rot, theta, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_qk_norm_rope(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                                long long v_stride, const void* q_weight, const void* k_weight, float eps,
                                const int32_t* positions, const float* table, int max_positions, int rot,
                                int interleaved, void* q_out, long long q_out_stride, void* k_out,
                                long long k_out_stride, void* k_cache, void* v_cache, const int32_t* slots,
                                int num_tokens, int Hq, int Hkv, int d, int page_size, int num_blocks, void* stream) {
  if (!given(q, 16) || !given(k, 16) || !given(q_out, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) ||
      !aligned(k_out, 16))
    return ATTN_ERR_INVALID_ARG;
  if (num_tokens < 1 || num_tokens > kMaxTokens || Hq < 1 || Hkv < 1 || Hq > 65535 || Hkv > 65535)
    return ATTN_ERR_INVALID_ARG;
  if (!head_dim(d)) return ATTN_ERR_UNSUPPORTED;
  if (!token_stride(q_stride, Hq, d) || !token_stride(k_stride, Hkv, d) || !token_stride(q_out_stride, Hq, d))
    return ATTN_ERR_INVALID_ARG;
  if (k_out != nullptr && !token_stride(k_out_stride, Hkv, d)) return ATTN_ERR_INVALID_ARG;
  if ((q_weight != nullptr || k_weight != nullptr) && (!std::isfinite(eps) || eps < 0.f)) return ATTN_ERR_INVALID_ARG;
  if (rot < 0 || rot > d) return ATTN_ERR_INVALID_ARG;
  if (rot % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if (rot > 0 && (!given(positions, 4) || !given(table, 16) || max_positions < 1)) return ATTN_ERR_INVALID_ARG;
  // the kernel numbers its threads, one for 64 values, in 32 bits
  if (static_cast<int64_t>(num_tokens) * ((Hq + 7) / 8 + 2 * ((Hkv + 7) / 8)) * (d / 8) >= (int64_t(1) << 31))
    return ATTN_ERR_INVALID_ARG;
  const bool paged = k_cache != nullptr || v_cache != nullptr;
  if (!paged && k_out == nullptr) return ATTN_ERR_INVALID_ARG;
  if (paged) {
    if (!given(k_cache, 16) || !given(v_cache, 16) || !given(v, 16) || !given(slots, 4) || num_blocks < 1 ||
        !token_stride(v_stride, Hkv, d) || static_cast<int64_t>(num_blocks) * kPage > kMaxTokens)
      return ATTN_ERR_INVALID_ARG;
    if (page_size != kPage) return ATTN_ERR_UNSUPPORTED;
  }
  attn::QkRopeParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  p.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
  p.positions = positions;
  p.table = table;
  p.slots = slots;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.num_slots = paged ? static_cast<int64_t>(num_blocks) * kPage : 0;
  p.T = num_tokens;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = d;
  p.rot = rot;
  p.interleaved = interleaved ? 1 : 0;
  p.max_positions = max_positions;
  p.eps = eps;
  return from_cuda(attn::qk_rope_launch(p, static_cast<cudaStream_t>(stream)));
}

size_t attn_cache_q4_record_bytes(int d) { return head_dim(d) ? static_cast<size_t>(17) * d : 0; }

attn_status_t attn_cache_append_q4(const void* k, long long k_stride, const void* v, long long v_stride,
                                   const int32_t* slots, void* cache, int num_tokens, int Hkv, int d, int page_size,
                                   int num_blocks, void* stream) {
  if (!given(k, 16) || !given(v, 16) || !given(slots, 4) || !given(cache, 16)) return ATTN_ERR_INVALID_ARG;
  if (num_tokens < 1 || num_tokens > kMaxTokens || Hkv < 1 || Hkv > 65535 || num_blocks < 1)
    return ATTN_ERR_INVALID_ARG;
  if (page_size != kPage || !head_dim(d)) return ATTN_ERR_UNSUPPORTED;
  if (!token_stride(k_stride, Hkv, d) || !token_stride(v_stride, Hkv, d) ||
      static_cast<int64_t>(num_blocks) * kPage > kMaxTokens ||
      static_cast<int64_t>(num_tokens) * Hkv > (int64_t(1) << 32))
    return ATTN_ERR_INVALID_ARG;
  attn::AppendQ4Params p;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.slots = slots;
  p.cache = static_cast<uint8_t*>(cache);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.num_slots = static_cast<int64_t>(num_blocks) * kPage;
  p.T = num_tokens;
  p.Hkv = Hkv;
  p.d = d;
  return from_cuda(attn::append_q4_launch(p, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_cache_gather_q4(const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                                   void* k_out, void* v_out, int num_seqs, int Hkv, int d, int page_size,
                                   int max_blocks_per_seq, int num_blocks, void* stream) {
  const attn_status_t chk =
      check_paged(cache, block_table, seq_lens, num_seqs, Hkv, d, page_size, max_blocks_per_seq, num_blocks);
  if (chk != ATTN_OK) return chk;
  if (!given(k_out, 16) || !given(v_out, 16) || !records_fit(max_blocks_per_seq, Hkv)) return ATTN_ERR_INVALID_ARG;
  attn::GatherQ4Params p;
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
  return from_cuda(attn::gather_q4_launch(p, static_cast<cudaStream_t>(stream)));
}

size_t attn_decode_q4_workspace_bytes(int d) { return head_dim(d) ? attn::decode_q4_workspace_bytes(d) : 0; }

attn_status_t attn_decode_paged_q4(const void* q, const void* cache, const int32_t* block_table,
                                   const int32_t* seq_lens, void* o, float* lse, int num_seqs, int Hq, int Hkv, int d,
                                   int page_size, int max_blocks_per_seq, int num_blocks, float scale,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  const attn_status_t chk =
      check_paged(cache, block_table, seq_lens, num_seqs, Hkv, d, page_size, max_blocks_per_seq, num_blocks);
  if (chk != ATTN_OK) return chk;
  if (!given(q, 16) || !given(o, 16) || !aligned(lse, 4)) return ATTN_ERR_INVALID_ARG;
  if (Hq < 1 || Hq > 65535 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (!given(workspace, 16)) return ATTN_ERR_WORKSPACE;
  const size_t need = attn::decode_q4_workspace_bytes(d);
  if (need == 0) return ATTN_ERR_CUDA;
  if (workspace_bytes < need) return ATTN_ERR_WORKSPACE;
  attn::DecodeQ4Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const uint8_t*>(cache);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.workspace = workspace;
  p.N = num_seqs;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  return from_cuda(attn::decode_q4_launch(d, p, static_cast<cudaStream_t>(stream)));
}

size_t attn_prefill_q4_workspace_bytes(int num_seqs, int Hkv, int d, int max_blocks_per_seq) {
  if (num_seqs < 1 || Hkv < 1 || Hkv > 65535 || !head_dim(d) || max_blocks_per_seq < 1 ||
      !records_fit(max_blocks_per_seq, Hkv) || static_cast<int64_t>(num_seqs) * max_blocks_per_seq * kPage > kMaxTokens)
    return 0;
  const size_t pages = static_cast<size_t>(num_seqs) * max_blocks_per_seq;
  return 2 * up256(pages * kPage * Hkv * d * 2) + up256(pages * 4);
}

attn_status_t attn_prefill_paged_q4(const void* q, const void* cache, const int32_t* block_table,
                                    const int32_t* cu_seqlens_q, const int32_t* seq_lens, void* o, float* lse,
                                    int num_seqs, int max_seqlen_q, int total_q, int Hq, int Hkv, int d,
                                    int page_size, int max_blocks_per_seq, int num_blocks, float scale, int causal,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  attn::GatherQ4Params p;
  const attn_status_t chk = check_prefill_readback(q, cache, block_table, cu_seqlens_q, seq_lens, o, lse, num_seqs,
                                                   max_seqlen_q, total_q, Hq, Hkv, d, page_size, max_blocks_per_seq,
                                                   num_blocks, scale, workspace, workspace_bytes, p);
  if (chk != ATTN_OK) return chk;
  const cudaError_t e = attn::gather_q4_launch(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  return attn_prefill_paged(q, p.k_out, p.v_out, p.out_table, cu_seqlens_q, seq_lens, o, lse, num_seqs, max_seqlen_q,
                            total_q, Hq, Hkv, d, page_size, max_blocks_per_seq, num_seqs * max_blocks_per_seq, scale,
                            causal, stream);
}

}  // extern "C"
