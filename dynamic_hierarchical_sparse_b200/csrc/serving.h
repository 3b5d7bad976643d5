// Internal arguments and launchers of the operators around the prefill path:
// rotary positions, paged append and paged attention (C++ linkage, not exported).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dhsa.h"

namespace dhsa {

// A packed [T, H, d] operand with its token stride resolved (elements).
struct TokensArg {
  void* data;
  long long stride;
};

// The paged cache and the batch step as the kernels see them (device pointers).
struct PagedArgs {
  int head_dim, num_kv_heads, page_size, num_pages;
  long long page_stride;  // elements
  void* k_pages;
  void* v_pages;
  int num_seqs, max_pages, table_stride, num_groups;
  const int* cu_q;
  const int* kv_lens;
  const int* block_table;
  const int* group_ptr;
  const int* prefix_lens;
  int total_q;    // cu_q[B]
  int uniform_q;  // n when every sequence brings n >= 1 tokens (the owner of token t is t / n), else 0
};

// Rotary positions of q and k (either may be absent: data null).
cudaError_t launch_rope(const dhsa_rope_table& rope, int dtype, int head_dim, int tokens, const int* positions,
                        TokensArg q, int num_q_heads, TokensArg q_out, TokensArg k, int num_kv_heads,
                        TokensArg k_out, cudaStream_t stream);

// Paged append; rope null: keys are stored as they are.
cudaError_t launch_kv_append(const PagedArgs& a, int dtype, const dhsa_rope_table* rope, const int* positions,
                             TokensArg k, TokensArg v, TokensArg k_out, TokensArg q, TokensArg q_out,
                             int num_q_heads, uint32_t* status, cudaStream_t stream);

// Paged attention.  The work of a call is a list of items, each a set of query
// tokens that walk one range of keys: the groups' shared prefixes first, then
// every sequence's own part.  An item has Hkv * ceil(rows / kTileRows-sized
// tiles) segments (rows = its tokens times Hq / Hkv), each of all its key
// tiles; the key tiles of all segments, in order, are cut evenly among `ctas`
// CTAs, and a CTA leaves one partial result (O unnormalised, running max, sum)
// for each segment that it touches.
struct PagedWork {
  PagedArgs p;
  const void* q;
  long long q_stride;
  void* out;
  long long out_stride;
  float* lse;  // may be null
  int num_q_heads;
  float scale;
  float* part_o;    // [rows of all partials, d]
  float2* part_ml;  // [rows of all partials]: running max (log2 units), sum
  long long* items; // [2 * num_items + 1]: first key tile of each item, the total, then first row of each item
  uint32_t* status;
};

// Rows of partials that a call may need at most, from the host mirrors.
struct PagedShape {
  int num_items;
  long long part_rows;
};
PagedShape paged_shape(const PagedArgs& p, const int* h_cu_q, const int* h_group_ptr, int num_q_heads, int dtype);

cudaError_t launch_paged_attention(const PagedWork& w, const PagedShape& shape, int dtype, cudaStream_t stream);

}  // namespace dhsa
