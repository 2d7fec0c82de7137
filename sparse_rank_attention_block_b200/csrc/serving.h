// Internal declarations of the serving operators: prompt attention and the
// 8-bit key/value cache (host side).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace sda {

// sda_api.cu: checks shared by the entry points.
int32_t require_device();  // the current device is sm_100 (SDA_ERR_DEVICE otherwise)

// Packed prompts, by value to the kernel.
struct Prompt {
  int n_seq, rows_q, rows_k, H, H_kv, d, causal;
  long long ld_q, ld_k, ld_v, ld_o;  // elements between rows
  float scale_log2;                  // softmax scale * log2(e)
};

// serving_api.cu
// Limit of the serving kernels' waits, as sda_set_attention_wait_limit_ns sets it.
uint64_t serving_wait_limit();
void set_serving_wait_limit(uint64_t limit_ns);

// prompt_attn_tc.cu
cudaError_t launch_prompt_attn(const Prompt& p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               const int32_t* seq_q, const int32_t* seq_k, uint16_t* o, float* lse, unsigned* status,
                               cudaStream_t stream);

// The cache and its sequences, by value to the kernels.
struct Cache {
  int B, H, H_kv, d, block, n_blocks, max_blocks, rows, max_new, weights, keep, recent;
  int g;                             // query heads of a key head
  int dst_blocks;                    // ceil(keep / block): width of the eviction's target table
  long long ld_q, ld_k, ld_v, ld_o;
  float scale_log2;
};

// Workspace regions of the cache calls (byte offsets).
struct CacheLayout {
  size_t status;                     // unsigned status word
  size_t line;                       // [B + 1] int32: the sequences' places in the order of work
  size_t part_o;                     // [2 * workers, tile_rows, d] fp32 partial outputs
  size_t part_ml;                    // [2 * workers, tile_rows, 4] fp32: their running maxima and sums
  size_t lse2;                       // [rows, H] fp32 (weights kept only)
  size_t scores;                     // [B, H_kv, max tokens, rows_pad] fp32 scores (weights kept only)
  size_t total;
  int workers;                       // CTAs that share the work
  int whole_row_tiles;               // > 0: a CTA per unit (short sequences), of so many row tiles per key head
  int tile_rows;                     // query rows of a tile: 8 or 16
  int rows_pad;                      // row slots per key head
  long long join_ctas;               // CTAs of the second kernel, at most
  long long line_places;             // the longest possible line of work
  int wide_join;                     // 1: the second kernel takes a CTA per row, 0: a warp per row
};
CacheLayout make_cache_layout(const Cache& c);

// cache.cu. Eviction keeps each target's source row in `rows` ([B, H_kv, keep], in the workspace behind the status).
cudaError_t launch_cache_append(const Cache& c, const uint16_t* k, const uint16_t* v, const int32_t* seq,
                                const int32_t* lens, const int32_t* table, uint8_t* k_codes, uint8_t* v_codes,
                                float* k_scale, float* v_scale, float* w, unsigned* status, cudaStream_t stream);
cudaError_t launch_cache_evict(const Cache& c, const int32_t* lens, const int32_t* table, uint8_t* k_codes,
                               uint8_t* v_codes, float* k_scale, float* v_scale, float* w, const int32_t* dst_table,
                               int32_t* kept, int32_t* dst_lens, int32_t* rows, unsigned* status, cudaStream_t stream);

// cache_attn.cu
cudaError_t launch_cache_attn(const Cache& c, const CacheLayout& y, void* ws, const uint16_t* q, const int32_t* seq,
                              const int32_t* lens, const int32_t* table, const uint8_t* k_codes,
                              const uint8_t* v_codes, const float* k_scale, const float* v_scale, const float* w_in,
                              float* w_out, uint16_t* o, cudaStream_t stream);

}  // namespace sda
