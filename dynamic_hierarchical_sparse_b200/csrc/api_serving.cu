// C ABI of the operators around the prefill path: checks of arguments,
// workspace layout and launches.  Every entry point returns a dhsa_status;
// nothing throws across the ABI.
#include <math.h>
#include <stdint.h>

#include <cmath>
#include <limits>

#include "serving.h"

namespace dhsa {
namespace {

constexpr size_t kAlign = 256;
constexpr size_t kStatusBytes = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
dhsa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DHSA_OK : DHSA_ERR_CUDA; }
long long elem_bytes(int dtype) { return dtype == DHSA_BF16 ? 2 : 4; }

dhsa_status check_dtype_dim(int dtype, int head_dim) {
  if (dtype != DHSA_BF16 && dtype != DHSA_F32) return DHSA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return head_dim > 0 ? DHSA_ERR_UNSUPPORTED : DHSA_ERR_INVALID_ARG;
  return DHSA_OK;
}

bool rope_ok(const dhsa_rope_table* r, int head_dim) {
  return r->rotary_dim >= 2 && r->rotary_dim <= head_dim && r->rotary_dim % 2 == 0 && isfinite(r->factor);
}

// A packed operand as the kernels take it: bytes of a token, token stride.
struct Rows {
  uintptr_t base;
  long long stride, row, tokens;  // bytes, bytes, count
  bool same_place(const Rows& o) const { return base == o.base && stride == o.stride && row == o.row; }
};

// Whether two packed operands share a byte.  With equal strides (slices of one
// fused tensor) the rows are compared within a stride, otherwise as whole ranges.
bool overlap(const Rows& a, const Rows& b) {
  if (a.tokens == 0 || b.tokens == 0 || a.base == 0 || b.base == 0) return false;
  const uintptr_t a1 = a.base + (a.tokens - 1) * a.stride + a.row, b1 = b.base + (b.tokens - 1) * b.stride + b.row;
  if (a1 <= b.base || b1 <= a.base) return false;
  if (a.stride != b.stride) return true;
  const uintptr_t d = (a.base < b.base ? b.base - a.base : a.base - b.base) % a.stride;
  const long long lead = a.base < b.base ? a.row : b.row, trail = a.base < b.base ? b.row : a.row;
  return d < static_cast<uintptr_t>(lead) || d + trail > static_cast<uintptr_t>(a.stride);
}

// Resolves a packed operand; false: misaligned, or rows that overlap each other.
bool resolve(const dhsa_tokens& t, int heads, int head_dim, int dtype, long long tokens, TokensArg* arg, Rows* rows) {
  const long long e = elem_bytes(dtype), row = static_cast<long long>(heads) * head_dim;
  const long long stride = t.token_stride == 0 ? row : t.token_stride;
  arg->data = t.data;
  arg->stride = stride;
  *rows = Rows{reinterpret_cast<uintptr_t>(t.data), stride * e, row * e, t.data == nullptr ? 0 : tokens};
  if (t.data == nullptr) return true;
  if (stride < row || stride > (1ll << 40)) return false;
  return aligned16(t.data) && (stride * e) % 16 == 0;
}

dhsa_status check_cache(const dhsa_paged_cache* c) {
  if (c == nullptr) return DHSA_ERR_INVALID_ARG;
  if (dhsa_status s = check_dtype_dim(c->dtype, c->head_dim); s != DHSA_OK) return s;
  if (c->num_kv_heads < 1 || c->num_pages < 1 || c->page_size < 1) return DHSA_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return DHSA_ERR_UNSUPPORTED;
  if (c->num_kv_heads > 65535) return DHSA_ERR_UNSUPPORTED;
  const long long page = static_cast<long long>(c->num_kv_heads) * c->page_size * c->head_dim;
  // V's element size is K's for both dtypes
  if (c->page_stride < page || (c->page_stride * elem_bytes(c->dtype)) % 16 != 0) return DHSA_ERR_INVALID_ARG;
  if (c->page_stride > (1ll << 36)) return DHSA_ERR_UNSUPPORTED;
  if (c->k_pages == nullptr || c->v_pages == nullptr || !aligned16(c->k_pages) || !aligned16(c->v_pages))
    return DHSA_ERR_INVALID_ARG;
  return DHSA_OK;
}

dhsa_status check_batch(const dhsa_paged_batch* b, const dhsa_paged_cache* c, bool groups) {
  if (b == nullptr) return DHSA_ERR_INVALID_ARG;
  if (b->num_seqs < 0 || b->num_groups < 0 || b->max_pages < 1 || b->table_stride < b->max_pages)
    return DHSA_ERR_INVALID_ARG;
  if (static_cast<long long>(b->max_pages) * c->page_size > (1ll << 30)) return DHSA_ERR_UNSUPPORTED;
  if (b->cu_q == nullptr || b->h_cu_q == nullptr) return DHSA_ERR_INVALID_ARG;
  if (b->num_seqs > 0 && (b->kv_lens == nullptr || b->block_table == nullptr)) return DHSA_ERR_INVALID_ARG;
  if (b->h_cu_q[0] != 0) return DHSA_ERR_INVALID_ARG;
  for (int i = 0; i < b->num_seqs; ++i)
    if (b->h_cu_q[i + 1] < b->h_cu_q[i]) return DHSA_ERR_INVALID_ARG;
  if (!groups || b->num_groups == 0) return DHSA_OK;
  if (b->group_ptr == nullptr || b->prefix_lens == nullptr || b->h_group_ptr == nullptr) return DHSA_ERR_INVALID_ARG;
  if (b->h_group_ptr[0] != 0 || b->h_group_ptr[b->num_groups] != b->num_seqs) return DHSA_ERR_INVALID_ARG;
  for (int g = 0; g < b->num_groups; ++g)
    if (b->h_group_ptr[g + 1] < b->h_group_ptr[g]) return DHSA_ERR_INVALID_ARG;
  return DHSA_OK;
}

PagedArgs paged_args(const dhsa_paged_cache* c, const dhsa_paged_batch* b) {
  PagedArgs a{};
  a.head_dim = c->head_dim;
  a.num_kv_heads = c->num_kv_heads;
  a.page_size = c->page_size;
  a.num_pages = c->num_pages;
  a.page_stride = c->page_stride;
  a.k_pages = c->k_pages;
  a.v_pages = c->v_pages;
  a.num_seqs = b->num_seqs;
  a.max_pages = b->max_pages;
  a.table_stride = b->table_stride;
  a.num_groups = b->num_groups;
  a.cu_q = b->cu_q;
  a.kv_lens = b->kv_lens;
  a.block_table = b->block_table;
  a.group_ptr = b->group_ptr;
  a.prefix_lens = b->prefix_lens;
  a.total_q = b->h_cu_q[b->num_seqs];
  a.uniform_q = b->num_seqs > 0 ? b->h_cu_q[1] : 0;
  for (int i = 1; i < b->num_seqs && a.uniform_q > 0; ++i)
    if (b->h_cu_q[i + 1] - b->h_cu_q[i] != a.uniform_q) a.uniform_q = 0;
  a.by_uniform_q = FastDiv(a.uniform_q > 0 ? static_cast<uint32_t>(a.uniform_q) : 1u);
  while ((1 << a.page_shift) < c->page_size) ++a.page_shift;
  return a;
}

struct AttentionLayout {
  PagedShape shape;
  size_t items[2], ml[2], o[2], total;  // of the prefixes' own list and of the other
};

dhsa_status attention_layout(const dhsa_paged_cache* c, const dhsa_paged_batch* b, int num_q_heads,
                             const PagedArgs& a, AttentionLayout* L) {
  if (num_q_heads < 1 || num_q_heads % c->num_kv_heads != 0) return DHSA_ERR_INVALID_ARG;
  if (num_q_heads > 65535) return DHSA_ERR_UNSUPPORTED;
  if (static_cast<long long>(a.total_q) * num_q_heads > INT32_MAX) return DHSA_ERR_UNSUPPORTED;
  L->shape = paged_shape(a, b->h_cu_q, b->h_group_ptr, num_q_heads, c->dtype);
  if (!L->shape.fits) return DHSA_ERR_UNSUPPORTED;
  size_t at = kStatusBytes;
  for (int x = 0; x < 2; ++x) {
    const size_t rows = static_cast<size_t>(x == 0 ? L->shape.prefix_rows : L->shape.list_rows);
    const size_t n = static_cast<size_t>(x == 0 ? L->shape.prefix_items : L->shape.list_items);
    L->items[x] = at;
    at += align_up((2 * n + 2) * sizeof(int));
    L->ml[x] = at;
    at += align_up(rows * sizeof(float2));
    L->o[x] = at;
    at += align_up(rows * c->head_dim * sizeof(float));
  }
  L->total = at;
  return DHSA_OK;
}

// Frequencies are worked out in 64 bits of mantissa, one more than a fraction of a
// turn keeps: in a double's 53 they would be off by up to 2^-55 turns a position,
// 2^-24 turns at the far end of the positions.
using Freq = long double;
static_assert(std::numeric_limits<Freq>::digits >= 64, "the fractions of a turn have 64 bits");
constexpr Freq kPi = 3.14159265358979323846264338327950288L;

// The frequencies (radians a position) as fractions of a turn, rounded to 64 bits.
dhsa_status fill_turns(dhsa_rope_table* rope, int32_t rotary_dim, int32_t interleaved, const Freq* freq,
                       double factor) {
  if (!isfinite(factor) || !isfinite(static_cast<float>(factor))) return DHSA_ERR_INVALID_ARG;
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!std::isfinite(freq[i])) return DHSA_ERR_INVALID_ARG;
  rope->rotary_dim = rotary_dim;
  rope->interleaved = interleaved != 0;
  rope->factor = static_cast<float>(factor);
  for (int i = 0; i < DHSA_ROPE_MAX_PAIRS; ++i) {
    rope->turns[i] = 0;
    if (i >= rotary_dim / 2) continue;
    Freq turn = freq[i] / (2 * kPi);
    turn -= std::floor(turn);
    turn = std::round(std::ldexp(turn, 64));  // 2^64, a whole turn, is none
    rope->turns[i] = turn >= std::ldexp(Freq(1), 64) ? 0 : static_cast<uint64_t>(turn);
  }
  return DHSA_OK;
}

}  // namespace
}  // namespace dhsa

using namespace dhsa;

extern "C" {

dhsa_status dhsa_rope_init_freq(dhsa_rope_table* rope, int32_t rotary_dim, int32_t interleaved,
                                const double* inv_freq, double factor) {
  if (rope == nullptr || inv_freq == nullptr) return DHSA_ERR_INVALID_ARG;
  if (rotary_dim < 2 || rotary_dim > 2 * DHSA_ROPE_MAX_PAIRS || rotary_dim % 2 != 0) return DHSA_ERR_INVALID_ARG;
  Freq freq[DHSA_ROPE_MAX_PAIRS];
  for (int i = 0; i < rotary_dim / 2; ++i) freq[i] = inv_freq[i];
  return fill_turns(rope, rotary_dim, interleaved, freq, factor);
}

dhsa_status dhsa_rope_init(dhsa_rope_table* rope, int32_t rotary_dim, int32_t interleaved, double base,
                           const dhsa_rope_scaling* sc) {
  if (rope == nullptr) return DHSA_ERR_INVALID_ARG;
  if (rotary_dim < 2 || rotary_dim > 2 * DHSA_ROPE_MAX_PAIRS || rotary_dim % 2 != 0) return DHSA_ERR_INVALID_ARG;
  if (!isfinite(base) || !(base > 1.0)) return DHSA_ERR_INVALID_ARG;
  const int kind = sc == nullptr ? DHSA_ROPE_UNSCALED : sc->kind;
  if (kind < DHSA_ROPE_UNSCALED || kind > DHSA_ROPE_YARN) return DHSA_ERR_INVALID_ARG;
  if (kind != DHSA_ROPE_UNSCALED && !(isfinite(sc->factor) && sc->factor >= 1.0)) return DHSA_ERR_INVALID_ARG;
  if ((kind == DHSA_ROPE_LLAMA3 || kind == DHSA_ROPE_YARN) && !(isfinite(sc->original_len) && sc->original_len > 0))
    return DHSA_ERR_INVALID_ARG;
  if (kind == DHSA_ROPE_LLAMA3 && !(sc->low_freq_factor > 0 && sc->high_freq_factor > sc->low_freq_factor &&
                                    isfinite(sc->high_freq_factor)))
    return DHSA_ERR_INVALID_ARG;
  if (kind == DHSA_ROPE_YARN &&
      !(sc->beta_slow > 0 && sc->beta_fast >= sc->beta_slow && isfinite(sc->beta_fast)))
    return DHSA_ERR_INVALID_ARG;
  Freq freq[DHSA_ROPE_MAX_PAIRS];
  double factor = 1.0, low = 0, high = 0;
  if (kind == DHSA_ROPE_YARN) {
    // the pair index that makes `turns` turns in the original length
    auto index = [&](double turns) {
      return rotary_dim * log(sc->original_len / (turns * 2 * static_cast<double>(kPi))) / (2 * log(base));
    };
    low = fmax(floor(index(sc->beta_fast)), 0.0);
    high = fmin(ceil(index(sc->beta_slow)), rotary_dim - 1.0);
    if (high == low) high += 0.001;
    factor = 0.1 * log(sc->factor) + 1.0;
  }
  const Freq one = 1, zero = 0, by = kind == DHSA_ROPE_UNSCALED ? 1.0 : sc->factor;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const Freq f = std::pow(static_cast<Freq>(base), -2 * static_cast<Freq>(i) / rotary_dim);
    Freq y = f;
    if (kind == DHSA_ROPE_LINEAR) {
      y = f / by;
    } else if (kind == DHSA_ROPE_LLAMA3) {
      const Freq turns = sc->original_len * f / (2 * kPi), lo = sc->low_freq_factor, hi = sc->high_freq_factor;
      const Freq keep = std::fmin(std::fmax((turns - lo) / (hi - lo), zero), one);
      y = keep * f + (1 - keep) * (f / by);
    } else if (kind == DHSA_ROPE_YARN) {
      const Freq share = std::fmin(std::fmax((i - static_cast<Freq>(low)) / (static_cast<Freq>(high) - low), zero), one);
      y = share * (f / by) + (1 - share) * f;
    }
    freq[i] = y;
  }
  return fill_turns(rope, rotary_dim, interleaved, freq, factor);
}

dhsa_status dhsa_rope(const dhsa_rope_table* rope, int32_t dtype, int32_t head_dim, int32_t total_tokens,
                      const int32_t* positions, dhsa_tokens q, int32_t num_q_heads, dhsa_tokens q_out, dhsa_tokens k,
                      int32_t num_kv_heads, dhsa_tokens k_out, void* stream) {
  if (rope == nullptr || total_tokens < 0) return DHSA_ERR_INVALID_ARG;
  if (dhsa_status s = check_dtype_dim(dtype, head_dim); s != DHSA_OK) return s;
  if (!rope_ok(rope, head_dim)) return DHSA_ERR_INVALID_ARG;
  const bool has_q = q.data != nullptr, has_k = k.data != nullptr;
  if ((has_q && num_q_heads < 1) || (has_k && num_kv_heads < 1)) return DHSA_ERR_INVALID_ARG;
  if ((has_q && num_q_heads > 65535) || (has_k && num_kv_heads > 65535)) return DHSA_ERR_UNSUPPORTED;
  if (has_q != (q_out.data != nullptr) || has_k != (k_out.data != nullptr)) return DHSA_ERR_INVALID_ARG;
  TokensArg aq, aqo, ak, ako;
  Rows rq, rqo, rk, rko;
  if (!resolve(q, num_q_heads, head_dim, dtype, total_tokens, &aq, &rq) ||
      !resolve(q_out, num_q_heads, head_dim, dtype, total_tokens, &aqo, &rqo) ||
      !resolve(k, num_kv_heads, head_dim, dtype, total_tokens, &ak, &rk) ||
      !resolve(k_out, num_kv_heads, head_dim, dtype, total_tokens, &ako, &rko))
    return DHSA_ERR_INVALID_ARG;
  if ((!rqo.same_place(rq) && overlap(rqo, rq)) || (!rko.same_place(rk) && overlap(rko, rk)) || overlap(rqo, rk) ||
      overlap(rko, rq) || overlap(rqo, rko))
    return DHSA_ERR_INVALID_ARG;
  if (total_tokens == 0 || (!has_q && !has_k)) return DHSA_OK;
  if (positions == nullptr) return DHSA_ERR_INVALID_ARG;
  return cuda_status(launch_rope(*rope, dtype, head_dim, total_tokens, positions, aq, num_q_heads, aqo, ak,
                                 num_kv_heads, ako, static_cast<cudaStream_t>(stream)));
}

dhsa_status dhsa_kv_append(const dhsa_paged_cache* cache, const dhsa_paged_batch* batch, const dhsa_rope_table* rope,
                           const int32_t* positions, dhsa_tokens k, dhsa_tokens v, dhsa_tokens k_out, dhsa_tokens q,
                           dhsa_tokens q_out, int32_t num_q_heads, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (dhsa_status s = check_cache(cache); s != DHSA_OK) return s;
  if (dhsa_status s = check_batch(batch, cache, false); s != DHSA_OK) return s;
  const int d = cache->head_dim, hkv = cache->num_kv_heads, dtype = cache->dtype;
  if (rope != nullptr && !rope_ok(rope, d)) return DHSA_ERR_INVALID_ARG;
  const bool has_q = q.data != nullptr;
  if (has_q != (q_out.data != nullptr) || (has_q && (rope == nullptr || num_q_heads < 1)))
    return DHSA_ERR_INVALID_ARG;
  if (has_q && num_q_heads > 65535) return DHSA_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < kStatusBytes || (reinterpret_cast<uintptr_t>(workspace) % 4) != 0)
    return DHSA_ERR_WORKSPACE;
  const PagedArgs a = paged_args(cache, batch);
  TokensArg aq, aqo, ak, ako, av;
  Rows rq, rqo, rk, rko, rv;
  if (!resolve(q, num_q_heads, d, dtype, a.total_q, &aq, &rq) ||
      !resolve(q_out, num_q_heads, d, dtype, a.total_q, &aqo, &rqo) ||
      !resolve(k, hkv, d, dtype, a.total_q, &ak, &rk) || !resolve(k_out, hkv, d, dtype, a.total_q, &ako, &rko) ||
      !resolve(v, hkv, d, dtype, a.total_q, &av, &rv))
    return DHSA_ERR_INVALID_ARG;
  if ((!rqo.same_place(rq) && overlap(rqo, rq)) || (!rko.same_place(rk) && overlap(rko, rk)) || overlap(rqo, rk) ||
      overlap(rko, rq) || overlap(rqo, rko) || overlap(rqo, rv) || overlap(rko, rv))
    return DHSA_ERR_INVALID_ARG;
  if (a.total_q == 0) return DHSA_OK;
  if (k.data == nullptr || v.data == nullptr) return DHSA_ERR_INVALID_ARG;
  return cuda_status(launch_kv_append(a, dtype, rope, positions, ak, av, ako, aq, aqo, num_q_heads,
                                      static_cast<uint32_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

dhsa_status dhsa_paged_attention_workspace_size(const dhsa_paged_cache* cache, const dhsa_paged_batch* batch,
                                                int32_t num_q_heads, size_t* bytes) {
  if (dhsa_status s = check_cache(cache); s != DHSA_OK) return s;
  if (dhsa_status s = check_batch(batch, cache, true); s != DHSA_OK) return s;
  if (bytes == nullptr) return DHSA_ERR_INVALID_ARG;
  AttentionLayout L;
  if (dhsa_status s = attention_layout(cache, batch, num_q_heads, paged_args(cache, batch), &L); s != DHSA_OK)
    return s;
  *bytes = L.total;
  return DHSA_OK;
}

dhsa_status dhsa_paged_attention(const dhsa_paged_cache* cache, const dhsa_paged_batch* batch, dhsa_tokens q,
                                 int32_t num_q_heads, float scale, dhsa_tokens out, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (dhsa_status s = check_cache(cache); s != DHSA_OK) return s;
  if (dhsa_status s = check_batch(batch, cache, true); s != DHSA_OK) return s;
  PagedWork w{};
  w.p = paged_args(cache, batch);
  AttentionLayout L;
  if (dhsa_status s = attention_layout(cache, batch, num_q_heads, w.p, &L); s != DHSA_OK) return s;
  if (workspace == nullptr || workspace_bytes < L.total || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0)
    return DHSA_ERR_WORKSPACE;
  TokensArg aq, ao;
  Rows rq, ro;
  if (!resolve(q, num_q_heads, cache->head_dim, cache->dtype, w.p.total_q, &aq, &rq) ||
      !resolve(out, num_q_heads, cache->head_dim, cache->dtype, w.p.total_q, &ao, &ro) || overlap(rq, ro))
    return DHSA_ERR_INVALID_ARG;
  if (w.p.total_q == 0) return DHSA_OK;
  if (q.data == nullptr || out.data == nullptr) return DHSA_ERR_INVALID_ARG;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  w.q = aq.data;
  w.q_stride = aq.stride;
  w.out = ao.data;
  w.out_stride = ao.stride;
  w.lse = lse;
  w.num_q_heads = num_q_heads;
  w.by_group = FastDiv(static_cast<uint32_t>(num_q_heads / cache->num_kv_heads));
  w.scale = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(cache->head_dim));
  w.status = reinterpret_cast<uint32_t*>(ws);
  const int groups = w.p.num_groups;
  w.prefix.begin = 0;
  w.prefix.end = L.shape.own_prefix ? groups : 0;
  w.list.begin = w.prefix.end;
  w.list.end = groups + w.p.num_seqs;
  for (int x = 0; x < 2; ++x) {
    PagedList& l = x == 0 ? w.prefix : w.list;
    l.items = reinterpret_cast<int*>(ws + L.items[x]);
    l.part_ml = reinterpret_cast<float2*>(ws + L.ml[x]);
    l.part_o = reinterpret_cast<float*>(ws + L.o[x]);
  }
  return cuda_status(launch_paged_attention(w, L.shape, cache->dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
