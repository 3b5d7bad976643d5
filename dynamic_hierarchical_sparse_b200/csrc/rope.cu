// Rotary positions of packed queries and keys, and the same rotation on the way
// into a paged cache (K rotated into its page slot, V converted into its page
// slot, Q rotated beside them), in one launch each.
//
// Pair i of a token at position p turns by p * f_i.  f_i / (2 pi) comes as a
// 64-bit binary fraction of a turn, so p times it modulo 2^64 is the phase of
// any position (to |p| 2^-63 turns); the top 32 bits are split into the nearest quarter
// turn and a remainder of at most an eighth of a turn, whose sine and cosine
// are taken in fp32 (no loss at far positions, where an fp32 product p * f_i
// would be off by p * 2^-24 radians).
//
// Bound by HBM: every element is read once and written once.  A thread owns
// one pair of 16-byte vectors of a head (the two halves of its pairs) for two
// heads of its token, both loads in flight together; the lanes of a warp that
// have the same pairs of other heads share the sines and cosines, each
// computing a part.  With few tokens (a decode step) every thread takes one
// head: latency, not bandwidth, counts there.  More heads a thread (4, 8) save
// phases and lose to the registers and the longer serial walk: at 131072
// tokens, 32 + 8 heads of 128, 2 / 4 / 8 heads took 397 / 403 / 397 us at best,
// and appending 40960 tokens 166 / 180 / 184 us.  Measured: 397 us for 2.68 GB
// (6.76 TB/s, 1.03 of the measured copy rate), the append 167 us for 1.09 GB.
// A rotary_dim whose halves do not start on 16-byte borders takes vectors of 8,
// 4 or 2 bytes (rotary_dim 104 / 108 / 90 of 128, 32768 tokens: 112 / 145 / 208
// us against 102 us of bytes).
// What the arithmetic costs shows in how it is written: taking bf16 apart and
// together by 32-bit words instead of numbers took 909 to 464 us at 8 heads,
// and reading the table by generic address instead of through the constant
// bank (one lane at a time) another 10 to 20 % at 2 and 4.
#include "common.cuh"
#include "launch_early.cuh"
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

// A vector as fp32 numbers, and back (each rounded once).
template <typename T, int N>
__device__ __forceinline__ void unpack(const Vec<T, N>& v, float (&f)[N]) {
  if constexpr (sizeof(T) == 2 && N % 2 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = to_float(v.v[e]);
  }
}
template <typename T, int N>
__device__ __forceinline__ void pack(const float (&f)[N], Vec<T, N>& v) {
  if constexpr (sizeof(T) == 2 && N % 2 == 0) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) w[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v.v[e] = from_float<T>(f[e]);
  }
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

// An entry of the table by its generic address: every lane asks for another
// entry, which the constant bank would serve one lane at a time.
__device__ __forceinline__ uint64_t turn_of(const dhsa_rope_table& rope, int pair) {
  uint64_t v;
  asm volatile("ld.u64 %0, [%1];" : "=l"(v) : "l"(rope.turns + pair));
  return v;
}

// One warp's share of a head: D / (2 VEC) lanes, one vector pair each, so a
// warp takes kWide heads at a time (VEC 1: a head takes D / 64 warps).
template <typename T, int D, int VEC, int HEADS, bool PAGED>
struct RopeCfg {
  static constexpr int kItems = D / (2 * VEC);
  static constexpr int kWide = kItems < 32 ? 32 / kItems : 1;
  static constexpr int kLanes = kItems * kWide;            // threads of a unit (token, chunk)
  static constexpr int kChunk = kWide * HEADS;             // heads of a unit
  static constexpr int kBatch = HEADS < 2 ? HEADS : 2;     // heads in flight together
  static constexpr int kUnits = kThreads / kLanes;         // units of a block
  static constexpr int kPhases = VEC / kWide > 0 ? VEC / kWide : 1;  // pairs whose phase a lane computes
};

template <typename T, int D, int VEC, int HEADS, bool PAGED>
__global__ void __launch_bounds__(kThreads, 4)
    rope_kernel(const __grid_constant__ dhsa_rope_table rope, const __grid_constant__ RopeArgs a) {
  using C = RopeCfg<T, D, VEC, HEADS, PAGED>;
  using V = Vec<T, VEC>;
  let_next_start();
  wait_for_previous();
  const int cq = (a.q.heads + C::kChunk - 1) / C::kChunk, ck = (a.k.heads + C::kChunk - 1) / C::kChunk;
  const int cv = PAGED ? (a.v.heads + C::kChunk - 1) / C::kChunk : 0;
  const unsigned chunks = cq + ck + cv;
  const unsigned unit = blockIdx.x * static_cast<unsigned>(C::kUnits) + threadIdx.x / C::kLanes;
  const int t = static_cast<int>(unit / chunks);
  if (t >= a.tokens) return;  // uniform for the lanes of a unit, and for a warp
  const int chunk = static_cast<int>(unit % chunks);
  const int in_unit = threadIdx.x % C::kLanes;
  const int item = in_unit % C::kItems;

  const int kind = chunk < cq ? 0 : chunk < cq + ck ? 1 : 2;
  const Section& sec = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
  const int h0 = (chunk - (kind == 0 ? 0 : kind == 1 ? cq : cq + ck)) * C::kChunk + in_unit / C::kItems;

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
  const bool in_place = sec.src == sec.dst;
  const bool put = sec.dst != nullptr && (rot || !in_place);

  const T* src = static_cast<const T*>(sec.src) + t * sec.src_stride;
  T* dst = static_cast<T*>(sec.dst) + t * sec.dst_stride;
  V x0[C::kBatch], x1[C::kBatch];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < C::kBatch; ++i) {
      const int h = h0 + (i0 + i) * C::kWide;
      if (h < sec.heads) {
        x0[i] = *reinterpret_cast<const V*>(src + h * D + e0);
        x1[i] = *reinterpret_cast<const V*>(src + h * D + e1);
      }
    }
  };
  load(0);

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
        if (ok) slot_off = pg * g.page_stride + static_cast<long long>(at % g.page_size) * D;
      }
      // a negative position is padding, unless the length itself is negative
      if (!ok && (at >= 0 || held < 0) && in_unit == 0) report(a.status, kDevCheck);
    }
  } else {
    pos = a.positions[t];
  }

  // cos and sin of the item's pairs: the kWide lanes that share an item compute
  // kPhases of them each and hand them round
  float c[VEC], s[VEC];
  if (kind != 2 && nrot > 0) {
    const int sub = in_unit / C::kItems;
    float cc[C::kPhases], ss[C::kPhases];
#pragma unroll
    for (int e = 0; e < C::kPhases; ++e) {
      const int pair = item * VEC + (C::kWide > 1 ? sub * C::kPhases : 0) + e;
      phase(pos, rot ? turn_of(rope, pair) : 0, rope.factor, cc[e], ss[e]);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (C::kWide > 1) {
        const int from = (e / C::kPhases) * C::kItems + item;
        c[e] = __shfl_sync(0xffffffffu, cc[e % C::kPhases], from);
        s[e] = __shfl_sync(0xffffffffu, ss[e % C::kPhases], from);
      } else {
        c[e] = cc[e];
        s[e] = ss[e];
      }
    }
  }

  bool bad = false;
  const long long head_step = PAGED ? static_cast<long long>(a.page.page_size) * D : 0;
#pragma unroll 1
  for (int i0 = 0; i0 < HEADS; i0 += C::kBatch) {
    if (i0 > 0) {
      if (h0 + i0 * C::kWide >= sec.heads) break;
      load(i0);
    }
#pragma unroll
    for (int i = 0; i < C::kBatch; ++i) {
      const int h = h0 + (i0 + i) * C::kWide;
      if (h >= sec.heads) break;
      if (PAGED && kind == 2) {
        using VP = typename VPage<T>::type;
        if (slot_off < 0) break;
        VP* page = static_cast<VP*>(a.page.v_pages) + slot_off + h * head_step;
        Vec<VP, VEC> y0, y1;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          y0.v[e] = to_v_page(x0[i].v[e], bad);
          y1.v[e] = to_v_page(x1[i].v[e], bad);
        }
        *reinterpret_cast<Vec<VP, VEC>*>(page + e0) = y0;
        *reinterpret_cast<Vec<VP, VEC>*>(page + e1) = y1;
        continue;
      }
      if (rot) {
        float u[VEC], w[VEC], y0[VEC], y1[VEC];
        unpack(x0[i], u);
        unpack(x1[i], w);
        if (!rope.interleaved) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            y0[e] = u[e] * c[e] - w[e] * s[e];
            y1[e] = w[e] * c[e] + u[e] * s[e];
          }
        } else {
          // of the 2 VEC adjacent numbers, 2e pairs with 2e + 1 (VEC 1: the two vectors themselves)
          auto at = [](auto& lo, auto& hi, int e) -> float& { return e < VEC ? lo[e] : hi[e - VEC]; };
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float g = at(u, w, 2 * e), h2 = at(u, w, 2 * e + 1);
            at(y0, y1, 2 * e) = g * c[e] - h2 * s[e];
            at(y0, y1, 2 * e + 1) = h2 * c[e] + g * s[e];
          }
        }
        pack(y0, x0[i]);
        pack(y1, x1[i]);
      }
      if (put) {
        *reinterpret_cast<V*>(dst + h * D + e0) = x0[i];
        *reinterpret_cast<V*>(dst + h * D + e1) = x1[i];
      }
      if (PAGED && kind == 1 && slot_off >= 0) {
        T* page = static_cast<T*>(a.page.k_pages) + slot_off + h * head_step;
        *reinterpret_cast<V*>(page + e0) = x0[i];
        *reinterpret_cast<V*>(page + e1) = x1[i];
      }
    }
  }
  if (bad) report(a.status, kDevCheck);
}

template <typename T, int D, int VEC, int HEADS, bool PAGED>
cudaError_t run(const dhsa_rope_table& rope, const RopeArgs& a, cudaStream_t stream) {
  using C = RopeCfg<T, D, VEC, HEADS, PAGED>;
  const long long chunks = (a.q.heads + C::kChunk - 1) / C::kChunk + (a.k.heads + C::kChunk - 1) / C::kChunk +
                           (PAGED ? (a.v.heads + C::kChunk - 1) / C::kChunk : 0);
  const long long blocks = (a.tokens * chunks + C::kUnits - 1) / C::kUnits;
  if (blocks * C::kUnits > INT32_MAX) return cudaErrorInvalidValue;
  return launch_early(rope_kernel<T, D, VEC, HEADS, PAGED>, static_cast<unsigned>(blocks), kThreads, 0, stream, rope,
                      a);
}

// W: numbers of a 16-byte vector.
template <typename T, int D, int W, bool PAGED>
cudaError_t pick(const dhsa_rope_table& rope, const RopeArgs& a, cudaStream_t stream) {
  // the halves of the rotated part have to start on vector borders
  const int half = rope.rotary_dim / 2;
  if (half % W == 0) {
    const long long threads =
        static_cast<long long>(a.tokens) * (a.q.heads + a.k.heads + a.v.heads) * (D / (2 * W));
    if (threads <= 148LL * 1024) return run<T, D, W, 1, PAGED>(rope, a, stream);  // one head a thread fits one wave
    return run<T, D, W, 2, PAGED>(rope, a, stream);
  }
  if (half % (W / 2) == 0) return run<T, D, W / 2, 4, PAGED>(rope, a, stream);
  if (W > 4 && half % 2 == 0) return run<T, D, 2, 8, PAGED>(rope, a, stream);
  return run<T, D, 1, 8, PAGED>(rope, a, stream);
}

template <typename T, int W, bool PAGED>
cudaError_t pick_dim(const dhsa_rope_table& rope, const RopeArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return pick<T, 64, W, PAGED>(rope, a, stream);
    case 128: return pick<T, 128, W, PAGED>(rope, a, stream);
    default: return pick<T, 256, W, PAGED>(rope, a, stream);
  }
}

template <bool PAGED>
cudaError_t dispatch(const dhsa_rope_table& rope, int dtype, const RopeArgs& a, cudaStream_t stream) {
  if (a.tokens <= 0 || a.q.heads + a.k.heads + a.v.heads == 0) return cudaSuccess;
  return dtype == DHSA_BF16 ? pick_dim<__nv_bfloat16, 8, PAGED>(rope, a, stream)
                            : pick_dim<float, 4, PAGED>(rope, a, stream);
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
