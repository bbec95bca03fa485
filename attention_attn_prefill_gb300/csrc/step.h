// Internal interface between the C-ABI layer and the serving-step kernels: tables from request
// lengths, query/key norm with rotation, the 4-bit and the 8-bit paged cache, and block selection.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace attn {

struct StepTablesParams {
  const int32_t* cached_lens;  // [N] tokens already in the cache
  const int32_t* new_lens;     // [N] tokens of this step
  const int32_t* free_pages;   // [num_free], taken from the front
  int32_t* block_table;        // [N][max_blocks], in and out
  int32_t* seq_lens;           // [N]
  int32_t* cu_seqlens;         // [N + 1]
  int32_t* positions;          // [T]
  int32_t* slots;              // [T]
  int32_t* pages_used;         // [1]
  int N, T, num_free, max_blocks, num_blocks;
};
cudaError_t step_tables_launch(const StepTablesParams& p, cudaStream_t stream);

struct QkRopeParams {
  const __nv_bfloat16 *q, *k, *v;  // rows of d, heads dense, tokens q_stride / k_stride / v_stride apart
  const __nv_bfloat16 *q_weight, *k_weight;  // [d] or null (no norm)
  const int32_t* positions;        // [T]
  const float* table;              // [max_positions][rot]: cosines, then sines
  const int32_t* slots;            // [T] or null
  __nv_bfloat16 *q_out, *k_out;    // k_out may be null
  __nv_bfloat16 *k_cache, *v_cache;  // [num_blocks][16][Hkv][d], both or neither
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // elements
  int64_t num_slots;               // num_blocks * 16
  int T, Hq, Hkv, d, rot, interleaved, max_positions;
  float eps;
};
cudaError_t qk_rope_launch(const QkRopeParams& p, cudaStream_t stream);
cudaError_t rope_table_launch(float* table, int max_positions, int rot, double theta, cudaStream_t stream);

struct AppendQ4Params {
  const __nv_bfloat16 *k, *v;
  const int32_t* slots;
  uint8_t* cache;
  int64_t k_stride, v_stride, num_slots;
  int T, Hkv, d;
};
cudaError_t append_q4_launch(const AppendQ4Params& p, cudaStream_t stream);

struct GatherQ4Params {
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  __nv_bfloat16 *k_out, *v_out;  // [N][max_blocks * 16][Hkv][d]
  int32_t* out_table;            // [N][max_blocks] or null: the page of k_out that holds each page
  int N, Hkv, d, max_blocks, num_blocks;
};
cudaError_t gather_q4_launch(const GatherQ4Params& p, cudaStream_t stream);

struct DecodeQ4Params {
  const __nv_bfloat16* q;  // [N][Hq][d]
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  __nv_bfloat16* o;  // [N][Hq][d]
  float* lse;        // [N][Hq] or null
  void* workspace;
  int N, Hq, Hkv, max_blocks, num_blocks;
  float scale, scale_log2;
};
size_t decode_q4_workspace_bytes(int d);  // on the current device; 0 on error
cudaError_t decode_q4_launch(int d, const DecodeQ4Params& p, cudaStream_t stream);

struct AppendF8Params {
  const __nv_bfloat16 *k, *v;
  const int32_t* slots;
  uint8_t* cache;
  __nv_bfloat16* bounds;  // [num_blocks][Hkv][2][d] or null
  int64_t k_stride, v_stride, num_slots;
  int T, Hkv, d;
};
cudaError_t append_f8_launch(const AppendF8Params& p, cudaStream_t stream);

struct GatherF8Params {
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  __nv_bfloat16 *k_out, *v_out;  // [N][max_blocks * 16][Hkv][d]
  int32_t* out_table;            // [N][max_blocks] or null: the page of k_out that holds each page
  int N, Hkv, d, max_blocks, num_blocks;
};
cudaError_t gather_f8_launch(const GatherF8Params& p, cudaStream_t stream);

struct DecodeF8Params {
  const __nv_bfloat16* q;  // [T][Hq][d]
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu;      // [N + 1] or null: one query a sequence
  const int32_t* blocks;  // [T][Hkv][K] or null: all blocks
  __nv_bfloat16* o;       // [T][Hq][d]
  float* lse;             // [T][Hq] or null
  void* workspace;
  int T, N, Hq, Hkv, K, max_blocks, num_blocks;
  float scale_log2;
};
size_t decode_f8_workspace_bytes(int d);  // on the current device; 0 on error
cudaError_t decode_f8_launch(int d, const DecodeF8Params& p, cudaStream_t stream);

constexpr int SELECT_MOST_BLOCKS = 1 << 18;  // of a sequence: a bit each in shared memory, twice
struct SelectBlocksParams {
  const __nv_bfloat16* q;       // [T][Hq][d]
  const __nv_bfloat16* bounds;  // [num_blocks][Hkv][2][d]
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu;  // [N + 1] or null: one query a sequence
  int32_t* blocks;    // [T][Hkv][K]
  void* workspace;
  int T, N, max_q, Hq, Hkv, d, K, first, last, max_blocks, num_blocks;
};
size_t select_blocks_workspace_bytes(int64_t T, int64_t N, int64_t max_q, int64_t Hkv, int d, int64_t max_blocks);
cudaError_t select_blocks_launch(const SelectBlocksParams& p, cudaStream_t stream);

cudaError_t step_tables_status(uint32_t* out, bool clear);
cudaError_t qk_rope_status(uint32_t* out, bool clear);
cudaError_t cache_q4_status(uint32_t* out, bool clear);
cudaError_t decode_q4_status(uint32_t* out, bool clear);
cudaError_t cache_f8_status(uint32_t* out, bool clear);
cudaError_t decode_f8_status(uint32_t* out, bool clear);
cudaError_t select_blocks_status(uint32_t* out, bool clear);

// Reads (and optionally clears) a kernel file's device status word.
template <class Symbol>
cudaError_t read_status(Symbol& word, uint32_t* out, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(out, word, sizeof(uint32_t));
  if (e == cudaSuccess && clear) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(word, &zero, sizeof(uint32_t));
  }
  return e;
}

}  // namespace attn
