// Internal arguments and launchers of the operators around the prefill path:
// rotary positions, paged append and paged attention (C++ linkage, not exported).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dhsa.h"

namespace dhsa {

// n / d for 0 <= n < 2^31 by a product and a shift, the division by invariant
// integers of Granlund and Montgomery (1994) (a division by a number that
// is not known when compiling takes some forty instructions, which the first
// pass over a kernel's code, the whole of a short call, pays for in fetching).
struct FastDiv {
  uint32_t mul, shift, d;
  FastDiv() = default;
  explicit FastDiv(uint32_t by) : d(by) {
    shift = 0;
    while ((1u << shift) < by) ++shift;
    mul = static_cast<uint32_t>((((1ull << shift) - by) << 32) / by + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
#endif
};

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
  FastDiv by_uniform_q;
  int page_shift;  // log2(page_size)
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
// every sequence's own part.  An item has Hkv * ceil(rows / its tile's rows)
// segments (rows = its tokens times Hq / Hkv), each of all its key tiles; the
// key tiles of all segments, in order, are cut among the CTAs, by what they cost,
// and a CTA leaves one partial result (O unnormalised, running max, sum) for each segment
// that it touches.  One kernel works on one list: all items, or the prefixes
// and the sequences in a list each.
struct PagedList {
  int begin, end;    // items of the list
  FastDiv by_ctas;   // by the CTAs of its grid
  int extra;         // key tiles that a segment counts beside its own (see PagedCut)
  float* part_o;     // [rows of all its partials, d]
  float2* part_ml;   // [rows of all its partials]: running max (log2 units), sum
  int* items;        // [2 (end - begin) + 2]: first unit of each item, the total, the chunk
                     // (or minus the extra tiles), first row of each item
};

struct PagedWork {
  PagedArgs p;
  const void* q;
  long long q_stride;
  void* out;
  long long out_stride;
  float* lse;  // may be null
  int num_q_heads;
  FastDiv by_group;  // by Hq / Hkv
  float scale;
  PagedList prefix;  // the groups, where they are a list of their own; else empty
  PagedList list;    // the sequences, and the groups where `prefix` is empty
  uint32_t* status;
};

// How a call divides into lists, and the rows of partials that they may need at
// most (from the host mirrors).
struct PagedShape {
  bool own_prefix;  // the prefixes are a list of their own
  int prefix_items, list_items;
  int list_max;  // rows a tile of the list at most
  long long prefix_rows, list_rows;
  bool fits;     // units and rows within the kernels' 32-bit counts
};
PagedShape paged_shape(const PagedArgs& p, const int* h_cu_q, const int* h_group_ptr, int num_q_heads, int dtype);

cudaError_t launch_paged_attention(const PagedWork& w, const PagedShape& shape, int dtype, cudaStream_t stream);

// TMA view of a page array; one box is 128 bytes of up to `tile` tokens of a page.
CUresult encode_pages_map(CUtensorMap* map, const void* base, const PagedArgs& p, int tile, CUtensorMapDataType type);

// The prefixes' list on tcgen05 (bf16): key tiles of 128 and row tiles of up to
// 256, for d 256 of 64 and 128; one CTA an SM.
constexpr int paged_prefix_keys(int head_dim) { return head_dim == 256 ? 64 : 128; }
constexpr int paged_prefix_rows(int head_dim) { return head_dim == 256 ? 128 : 256; }
cudaError_t launch_paged_prefix(const PagedWork& w, cudaStream_t stream);

}  // namespace dhsa
