// Rotary positions of packed queries and keys, and the same rotation on the way
// into a paged cache (K rotated into its page slot, V converted into its page
// slot, Q rotated beside them), in one launch each.
//
// Pair i of a token at position p turns by p * f_i.  f_i / (2 pi) comes as a
// 64-bit binary fraction of a turn, so p times it modulo 2^64 is the exact
// phase of any position; the top 32 bits are split into the nearest quarter
// turn and a remainder of at most an eighth of a turn, whose sine and cosine
// are taken in fp32 (no loss at far positions, where an fp32 product p * f_i
// would be off by p * 2^-24 radians).
//
// Bound by HBM: every element is read once and written once.  A thread owns
// one pair of 16-byte vectors of a head (the two halves of its pairs) and walks
// kHeads heads of its token with it, so the sines and cosines are computed once
// for kHeads heads; kHeads loads are in flight before the first store.  With
// few tokens (a decode step) every thread takes one head instead: latency, not
// bandwidth, counts there.
#include "common.cuh"
#include "serving.h"

namespace dhsa {
namespace {

constexpr int kThreads = 256;

struct Section {
  const void* src;
  void* dst;  // packed output (may be null for K and V on their way into pages)
  long long src_stride, dst_stride;
  int heads;
};

struct RopeArgs {
  Section q, k, v;
  const int* positions;
  int tokens;
  int head_dim;
  PagedArgs page;  // append only
  uint32_t* status;
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ float from_float<float>(float x) {
  return x;
}

// Storage type of a V page: f16 for bf16 problems, fp32 for fp32 ones.
__device__ __forceinline__ __half to_v_page(__nv_bfloat16 x, bool& bad) {
  const float f = __bfloat162float(x);
  bad |= !(fabsf(f) <= 65504.f);
  unsigned short r;
  asm("{\n\t.reg .b32 t;\n\tcvt.rn.satfinite.f16x2.f32 t, %1, %1;\n\tcvt.u16.u32 %0, t;\n\t}" : "=h"(r) : "f"(f));
  return __ushort_as_half(r);
}
__device__ __forceinline__ float to_v_page(float x, bool&) { return x; }

template <typename T>
struct VPage {
  using type = float;
};
template <>
struct VPage<__nv_bfloat16> {
  using type = __half;
};

// cos and sin of position p on the pair whose turn fraction is `turn`.
__device__ __forceinline__ void phase(int p, uint64_t turn, float a, float& c, float& s) {
  const uint64_t ph = static_cast<uint64_t>(static_cast<int64_t>(p)) * turn;
  const uint32_t top = static_cast<uint32_t>(ph >> 32);  // turns * 2^32
  const uint32_t quarter = (top + 0x20000000u) >> 30;    // nearest quarter turn
  const int rest = static_cast<int>(top - (quarter << 30));  // |rest| <= 2^29
  float sn, cs;
  sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &sn, &cs);  // half turns: rest * 2^-31
  const bool swap = quarter & 1u;
  const float c0 = swap ? sn : cs, s0 = swap ? cs : sn;
  // quarter turns 1 and 2 have a negative cosine, 2 and 3 a negative sine
  c = ((quarter + 1u) & 2u) ? -a * c0 : a * c0;
  s = (quarter & 2u) ? -a * s0 : a * s0;
}

template <typename T, int VEC, int HEADS, bool PAGED>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const __grid_constant__ dhsa_rope_table rope, const __grid_constant__ RopeArgs a) {
  using V = Vec<T, VEC>;
  const int d = a.head_dim;
  const int items = d / (2 * VEC);  // vector pairs of a head, a power of two
  const int cq = (a.q.heads + HEADS - 1) / HEADS, ck = (a.k.heads + HEADS - 1) / HEADS;
  const int cv = PAGED ? (a.v.heads + HEADS - 1) / HEADS : 0;
  const unsigned chunks = cq + ck + cv;
  const unsigned block = blockIdx.x;
  const int chunk = block % chunks;
  const int per_block = kThreads / items;
  const long long t64 = static_cast<long long>(block / chunks) * per_block + threadIdx.x / items;
  const int item = threadIdx.x % items;
  if (t64 >= a.tokens) return;
  const int t = static_cast<int>(t64);

  const int kind = chunk < cq ? 0 : chunk < cq + ck ? 1 : 2;
  const Section& sec = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
  const int h0 = (chunk - (kind == 0 ? 0 : kind == 1 ? cq : cq + ck)) * HEADS;
  const int nh = min(HEADS, sec.heads - h0);

  const int rd = rope.rotary_dim;
  const int nrot = rd / (2 * VEC);
  const bool rot = kind != 2 && item < nrot;
  int e0, e1;  // the two vectors of this item
  if (rot && !rope.interleaved) {
    e0 = item * VEC;
    e1 = rd / 2 + item * VEC;
  } else {
    e0 = 2 * item * VEC;
    e1 = e0 + VEC;
  }
  if (!PAGED && !rot && sec.src == sec.dst) return;  // in place, behind the rotated part

  const T* src = static_cast<const T*>(sec.src) + t * sec.src_stride + static_cast<long long>(h0) * d;
  V x0[HEADS], x1[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    if (h < nh) {
      x0[h] = *reinterpret_cast<const V*>(src + h * d + e0);
      x1[h] = *reinterpret_cast<const V*>(src + h * d + e1);
    }
  }

  // position, and (append) the page slot
  int pos = 0;
  long long slot_off = -1;  // element offset of the token's (head 0) slot in the pages, -1: not stored
  if (PAGED) {
    const PagedArgs& g = a.page;
    int b;
    if (g.uniform_q > 0) {
      b = t / g.uniform_q;
    } else {  // the last b with cu_q[b] <= t (its sequence is not empty: cu_q[b + 1] > t)
      int lo = 0, hi = g.num_seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.cu_q[mid] <= t) lo = mid; else hi = mid;
      }
      b = lo;
    }
    // in unsigned arithmetic: a length that is out of range must not overflow
    const int held = g.kv_lens[b];
    const int at = static_cast<int>(static_cast<unsigned>(held) - static_cast<unsigned>(g.cu_q[b + 1] - t));
    pos = a.positions != nullptr ? a.positions[t] : at;
    if (kind != 0) {
      bool ok = at >= 0 && at < g.max_pages * g.page_size;
      if (ok) {
        const int pg = g.block_table[static_cast<long long>(b) * g.table_stride + at / g.page_size];
        ok = static_cast<unsigned>(pg) < static_cast<unsigned>(g.num_pages);
        if (ok)
          slot_off = pg * g.page_stride + (static_cast<long long>(h0) * g.page_size + at % g.page_size) * d;
      }
      // a negative position is padding, unless the length itself is negative
      if (!ok && (at >= 0 || held < 0) && item == 0) report(a.status, kDevCheck);
    }
  } else {
    pos = a.positions[t];
  }

  if (PAGED && kind == 2) {
    using VP = typename VPage<T>::type;
    if (slot_off < 0) return;
    VP* dst = static_cast<VP*>(a.page.v_pages) + slot_off;
    const int hs = a.page.page_size * d;
    bool bad = false;
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      if (h < nh) {
        Vec<VP, VEC> y0, y1;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          y0.v[e] = to_v_page(x0[h].v[e], bad);
          y1.v[e] = to_v_page(x1[h].v[e], bad);
        }
        *reinterpret_cast<Vec<VP, VEC>*>(dst + h * hs + e0) = y0;
        *reinterpret_cast<Vec<VP, VEC>*>(dst + h * hs + e1) = y1;
      }
    }
    if (bad) report(a.status, kDevCheck);
    return;
  }

  if (rot) {
    float c[VEC], s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) phase(pos, rope.turns[item * VEC + e], rope.factor, c[e], s[e]);
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      V y0, y1;
      if (!rope.interleaved) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float u = to_float(x0[h].v[e]), w = to_float(x1[h].v[e]);
          y0.v[e] = from_float<T>(u * c[e] - w * s[e]);
          y1.v[e] = from_float<T>(w * c[e] + u * s[e]);
        }
        x0[h] = y0;
        x1[h] = y1;
      } else {
        // element 2e of the 2 * VEC adjacent ones pairs with element 2e + 1
        T z[2 * VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          z[e] = x0[h].v[e];
          z[VEC + e] = x1[h].v[e];
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float u = to_float(z[2 * e]), w = to_float(z[2 * e + 1]);
          z[2 * e] = from_float<T>(u * c[e] - w * s[e]);
          z[2 * e + 1] = from_float<T>(w * c[e] + u * s[e]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x0[h].v[e] = z[e];
          x1[h].v[e] = z[VEC + e];
        }
      }
    }
  }

  if (sec.dst != nullptr && (rot || sec.dst != sec.src)) {
    T* dst = static_cast<T*>(sec.dst) + t * sec.dst_stride + static_cast<long long>(h0) * d;
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      if (h < nh) {
        *reinterpret_cast<V*>(dst + h * d + e0) = x0[h];
        *reinterpret_cast<V*>(dst + h * d + e1) = x1[h];
      }
    }
  }
  if (PAGED && kind == 1 && slot_off >= 0) {
    T* dst = static_cast<T*>(a.page.k_pages) + slot_off;
    const int hs = a.page.page_size * d;
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      if (h < nh) {
        *reinterpret_cast<V*>(dst + h * hs + e0) = x0[h];
        *reinterpret_cast<V*>(dst + h * hs + e1) = x1[h];
      }
    }
  }
}

template <typename T, int VEC, int HEADS, bool PAGED>
cudaError_t run(const dhsa_rope_table& rope, const RopeArgs& a, cudaStream_t stream) {
  const int per_block = kThreads / (a.head_dim / (2 * VEC));
  const long long chunks = (a.q.heads + HEADS - 1) / HEADS + (a.k.heads + HEADS - 1) / HEADS +
                           (PAGED ? (a.v.heads + HEADS - 1) / HEADS : 0);
  const long long blocks = (a.tokens + per_block - 1LL) / per_block * chunks;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  rope_kernel<T, VEC, HEADS, PAGED><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(rope, a);
  return cudaGetLastError();
}

template <typename T, int W, bool PAGED>
cudaError_t pick(const dhsa_rope_table& rope, const RopeArgs& a, cudaStream_t stream) {
  // 16-byte vectors need both halves of the rotated part on vector borders;
  // any other even rotary_dim goes element by element
  if (rope.rotary_dim % (2 * W) != 0) return run<T, 1, 4, PAGED>(rope, a, stream);
  constexpr int kMany = 8;
  const long long threads =
      static_cast<long long>(a.tokens) * (a.q.heads + a.k.heads + a.v.heads) * (a.head_dim / (2 * W));
  if (threads <= 148LL * 2048) return run<T, W, 1, PAGED>(rope, a, stream);  // one head a thread still fits one wave
  return run<T, W, kMany, PAGED>(rope, a, stream);
}

template <bool PAGED>
cudaError_t dispatch(const dhsa_rope_table& rope, int dtype, const RopeArgs& a, cudaStream_t stream) {
  if (a.tokens <= 0 || a.q.heads + a.k.heads + a.v.heads == 0) return cudaSuccess;
  return dtype == DHSA_BF16 ? pick<__nv_bfloat16, 8, PAGED>(rope, a, stream) : pick<float, 4, PAGED>(rope, a, stream);
}

Section section(TokensArg in, TokensArg out, int heads) {
  return Section{in.data, out.data, in.stride, out.stride, in.data != nullptr ? heads : 0};
}

}  // namespace

cudaError_t launch_rope(const dhsa_rope_table& rope, int dtype, int head_dim, int tokens, const int* positions,
                        TokensArg q, int num_q_heads, TokensArg q_out, TokensArg k, int num_kv_heads,
                        TokensArg k_out, cudaStream_t stream) {
  RopeArgs a{};
  a.q = section(q, q_out, num_q_heads);
  a.k = section(k, k_out, num_kv_heads);
  a.positions = positions;
  a.tokens = tokens;
  a.head_dim = head_dim;
  return dispatch<false>(rope, dtype, a, stream);
}

cudaError_t launch_kv_append(const PagedArgs& p, int dtype, const dhsa_rope_table* rope, const int* positions,
                             TokensArg k, TokensArg v, TokensArg k_out, TokensArg q, TokensArg q_out,
                             int num_q_heads, uint32_t* status, cudaStream_t stream) {
  RopeArgs a{};
  a.q = section(q, q_out, num_q_heads);
  a.k = section(k, k_out, p.num_kv_heads);
  a.v = section(v, TokensArg{nullptr, 0}, p.num_kv_heads);
  a.positions = positions;
  a.tokens = p.total_q;
  a.head_dim = p.head_dim;
  a.page = p;
  a.status = status;
  dhsa_rope_table none{};  // rotary_dim 0: every number is passed on
  return dispatch<true>(rope != nullptr ? *rope : none, dtype, a, stream);
}

}  // namespace dhsa
