// Internal launchers of the head and paged-cache calls.  Arguments are already
// validated by the C-ABI layer (paged_api.cu).
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "rope.cuh"

namespace csa2 {

// csa2_heads with its strides filled in (heads == 0: absent)
struct HeadRows {
  void* data = nullptr;
  int heads = 0;
  int64_t token_stride = 0, head_stride = 0;
};

// csa2_paged_kv with its strides filled in, as the kernels read it
struct PagedView {
  const uint8_t *k, *v;              // v == k: shared rows
  const uint8_t *k_scales, *v_scales;
  int64_t page_stride, token_stride, head_stride;   // channels
  const int32_t* table;
  const int32_t* lens;
  int64_t table_stride;
  int64_t n_pages;
  int64_t capacity;                  // max_pages * page_size
  int page_shift, heads, B;
  int* err;

  // channel offset of row (page, slot, head)
  __device__ __forceinline__ int64_t row(int64_t page, int slot, int head) const {
    return page * page_stride + slot * token_stride + head * head_stride;
  }
};

csa2_status launch_head_norm(csa2_dtype dtype, const HeadRows& q, const float* q_weight,
                             const HeadRows& q_out, const HeadRows& k, const float* k_weight,
                             const HeadRows& k_out, int64_t T, int D, float eps,
                             const int32_t* positions, const rope::RopeArgs& rope, cudaStream_t stream);

csa2_status launch_paged_append(csa2_dtype dtype, const HeadRows& k, const HeadRows& v,
                                const int32_t* seq, const int32_t* pos, int64_t T, int D, bool fp4,
                                const rope::RopeArgs& rope, const PagedView& cache, cudaStream_t stream);

// One attention launch over a paged cache.
struct PagedAttn {
  csa2_kv_fmt fmt;
  int D, Hq, G;                      // head width, query heads, query heads per cache head
  const void* q;
  int64_t q_token, q_head;           // strides in elements
  float scale;
  int window, sinks;                 // window 0: none
  void* out;                         // [T, Hq, D]
  float* lse;                        // [T, Hq] or null
  PagedView kv;
};
size_t paged_decode_workspace(const PagedAttn& a, int64_t max_len, int chunk);
csa2_status launch_paged_decode(const PagedAttn& a, int64_t max_len, int chunk, void* ws,
                                cudaStream_t stream);
// The decode launch for rows of up to 256 channels, FP4 of 512 (paged_decode.cu); the caller
// joins the chunks.
bool paged_decode_stream_applies(const PagedAttn& a);
int paged_decode_heads(const PagedAttn& a);          // query heads per CTA
csa2_status launch_paged_decode_stream(const PagedAttn& a, int chunk, int chunks, float* part_o, float2* part_ml,
                                       cudaStream_t stream);
// Tensor map of 16-bit cache rows as [page][slot][head][channel] with the 128-byte
// swizzle: a box is 64 channels of box_rows slots of one head and page.
csa2_status make_tensor_map_paged(CUtensorMap* map, const void* base, int dim, int heads, int64_t head_stride,
                                  int page_size, int64_t token_stride, int64_t n_pages, int64_t page_stride,
                                  int box_rows);
// Tensor map of rows of heads as [token][head][channel]: a box is 64 channels of
// box_heads heads of box_tokens tokens.
csa2_status make_tensor_map_heads(CUtensorMap* map, const void* base, int dim, int heads, int64_t head_stride,
                                  int64_t tokens, int64_t token_stride, int box_heads, int box_tokens);
// Prompt attention on the tensor cores, rows of 64 or 128 channels (paged_window.cu).
bool paged_window_tc_applies(const PagedAttn& a);
csa2_status launch_paged_window_tc(const PagedAttn& a, const int32_t* cu_q, int64_t T, cudaStream_t stream);
// The decode launch on the tensor cores (paged_wide.cu): chunks of aligned tiles of
// 128 tokens; the caller joins them.
bool paged_wide_applies(const PagedAttn& a);
int paged_wide_heads(const PagedAttn& a);            // query heads per CTA
// A prompt by the same kernel, one CTA per token.
bool paged_wide_prompt_applies(const PagedAttn& a);
csa2_status launch_paged_wide_prompt(const PagedAttn& a, const int32_t* cu_q, int64_t T, cudaStream_t stream);
csa2_status launch_paged_wide(const PagedAttn& a, int chunk, int chunks, float* part_o, float2* part_ml,
                              cudaStream_t stream);
csa2_status launch_paged_window(const PagedAttn& a, const int32_t* cu_q, int64_t T, cudaStream_t stream);

}  // namespace csa2
