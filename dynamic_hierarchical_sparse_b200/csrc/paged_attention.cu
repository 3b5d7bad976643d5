// Attention of new query tokens over a paged cache: a shared prefix is read once
// for the rows of all the sequences that share it, then every sequence's own
// keys, and a last kernel joins the partial results of each row.
//
//   out[t, h] = sum_{s < L} exp(x_s - m) v_s / l,  x_s = q . k_s * scale,
//   l = sum_s exp(x_s - m)
// is associative over sets of keys: a set's (m, l, O = sum exp(x - m) v) joins
// with another's by scaling both to the larger m.  So the key tiles of all
// items (prefixes with all their group's rows, sequences with their own) form
// one list that is cut evenly among the CTAs, wherever that falls, and every
// CTA leaves (m, l, O) for each segment that it touches.
//
// paged_mma_kernel (bf16): bound by HBM as long as a tile's rows are few.  One
// warp brings 64-key tiles of K and V from the pages by TMA (128-byte swizzle)
// into a ring, ahead across pieces; four warps run S = Q K^T and O += P V on
// mma.sync m16n8k16 fragments.  With 16 rows or fewer the four warps split a
// tile's keys (each with its own running max and O, joined when the piece
// ends), with 32 two split them, with 64 every warp has 16 rows of its own.
// Q stays in registers, P goes from the S fragments straight into the A
// operand of P V (f16, as V).  Measured: 48 unshared sequences of 100 to 8192
// keys, 32 + 8 heads of 128: 135 us for 839 MB, 6.2 TB/s (0.95 of the measured copy
// rate), of which the join has 4.  A short call (4 sequences, 128 rows, 9.3 us)
// is latency: the first pass over the code, one round of loads, the join.
//
// paged_f32_kernel (fp32): the same with 32-key tiles and 16 rows, on tf32
// fragments in pairs.  Bound by latency, of loads and of its own instructions.
// Measured: 4 sequences on 14117 keys, 32 + 8 heads: 64 us with d 256, 38 with d
// 128 (231 and 116 MB).
#include "launchers.h"
#include "paged.cuh"

namespace dhsa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// The prefixes are a list of their own, for the tcgen05 kernel, where a group
// has more than 32 rows (query tokens times Hq / Hkv) and the prefixes may be
// long: rows x Hkv x d x the tokens that a table row has room for (their lengths
// are on the device) of 2^30 or more.  That kernel costs a few us more to start
// and end; 32 + 8 heads of 128, page 16, up to 512 own keys, one kernel / two, in
// us: 16 sequences on 1024 keys 15.5 / 22.5, on 16384 36.1 / 36.0, 32 on 2048
// 22.9 / 30.2, on 8192 37.6 / 35.0, 12 on 32768 53.8 / 47.5, 32 on 32768 100 /
// 58.8, 64 on 131072 587 / 193; 64 of d 64 on 1024 22.6 / 28.3, 16 of d 256 on
// 8000 50.5 / 40.7; 12 sequences of 5 tokens in two groups, 8 + 4 heads of 256,
// on 4097 50.1 / 39.4.  In all of these the table has room for what is held and no
// more.  With room for 131072 tokens the rule takes the second kernel at any length,
// and short prefixes lose by it: 16 sequences on 1024 keys 23.0 instead of 15.6, on
// 4096 27.4 instead of 21.6, 32 on 2048 30.7 instead of 23.6.  One group with more
// than 32 rows takes all groups' prefixes there.
constexpr int kOwnPrefixRows = 32;
constexpr long long kOwnPrefixWork = 1ll << 30;

// ------------------------------------------------------------------ bf16
constexpr int kBN = 64;        // keys a tile
constexpr int kMmaThreads = 160;  // four compute warps, one producer
constexpr int kProducer = 4;

template <int D>
struct MmaCfg {
  static constexpr int kSlices = D / 64;             // 64-column (128-byte) slices of a row
  static constexpr int kTileBytes = kBN * D * 2;     // one K or V tile
  static constexpr int kStages = D == 64 ? 4 : 3;
  static constexpr int kCtas = D == 64 ? 3 : D == 128 ? 2 : 1;  // resident on an SM
  static constexpr int kJoinStride = D / 4 + 8;      // floats; + 8: the fragment writes of a half-warp hit all banks
  static constexpr int kOffJoin = kStages * 2 * kTileBytes;
  static constexpr int kOffMl = kOffJoin + 4 * 16 * kJoinStride * 4;
  static constexpr int kOffScan = kOffMl + 4 * 16 * 8;
  static constexpr int kOffBar = kOffScan + ((static_cast<int>(sizeof(PagedScan)) + 15) / 16) * 16;
  static constexpr int kSmemBytes = kOffBar + 8 * 2 * kStages + 16 + 1024;
  static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "shared memory budget");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A CTA's ring of key tiles (K, then V, in each stage) and where this warp is in it.
struct Ring {
  uint32_t sbase, bar0;
  unsigned char* smem;
  volatile int* abort_flag;
  int stage;
  uint32_t phase;
  template <int kStages>
  __device__ __forceinline__ void next() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ uint32_t bar_full(const Ring& c, int s) { return c.bar0 + 8u * s; }
template <int kStages>
__device__ __forceinline__ uint32_t bar_empty(const Ring& c, int s) {
  return c.bar0 + 8u * (kStages + s);
}

// The producer warp: brings the key tiles of all the CTA's pieces into the ring,
// by slices of kCols columns (128 bytes, swizzled), a lane for each box (page
// part, slice, K or V).
template <int BN, int kCols, int kSlices, int kStages, typename Walk>
__device__ __forceinline__ void page_producer(const PagedWork& w, Walk& walk, const CUtensorMap* tm_k,
                                              const CUtensorMap* tm_v, Ring& ring) {
  constexpr int kTileBytes = kSlices * BN * 128;
  const int lane = threadIdx.x & 31;
  const int ps = w.p.page_size, psh = w.p.page_shift;
  const int box = ps < BN ? ps : BN;
  const int kv = lane & 1, sl = (lane >> 1) % kSlices, pp = (lane >> 1) / kSlices;
  const bool mine = pp * box < BN;
  const CUtensorMap* map = kv ? tm_v : tm_k;
  const uint32_t dst0 = ring.sbase + kv * kTileBytes + sl * (BN * 128) + pp * box * 128;
  int issued = 0;
  bool ok = true;
  do {
    const int h = walk.h;
    const int* table = w.p.block_table + static_cast<long long>(walk.it.row) * w.p.table_stride;
    // the page of this lane's part of a tile, -1 where the item has no key in it
    auto page_at = [&](int kt) -> int {
      const int key = (walk.first + walk.kt + kt) * BN + pp * box;
      if (kt >= walk.count || !mine || key >= walk.it.hi || key + box <= walk.it.lo) return -1;
      const int pg = table[key >> psh];
      if (static_cast<unsigned>(pg) < static_cast<unsigned>(w.p.num_pages)) return pg;
      report(w.status, kDevCheck);
      return w.p.num_pages;  // outside the map: the box arrives as zeros
    };
    int page = page_at(0);
    for (int kt = 0; kt < walk.count; ++kt) {
      const int page_next = page_at(kt + 1);
      const int s = ring.stage;
      if (issued >= kStages)
        ok = paged_wait_warp(bar_empty<kStages>(ring, s), ring.phase ^ 1u, ring.abort_flag);
      if (!ok) break;
      const unsigned active = __ballot_sync(0xffffffffu, page >= 0);
      if (lane == 0) mbar_arrive_expect_tx(bar_full(ring, s), __popc(active) * box * 128);
      __syncwarp();
      if (page >= 0) {
        const int key = (walk.first + walk.kt + kt) * BN + pp * box;
        tma_load_4d(dst0 + s * 2 * kTileBytes, map, bar_full(ring, s), sl * kCols, key & (ps - 1), h, page);
      }
      ++issued;
      page = page_next;
      ring.template next<kStages>();
    }
  } while (ok && walk.next());
  if (*ring.abort_flag && lane == 0) {
    // let copies already in flight land before the CTA exits (bounded)
    volatile int never = 0;
    for (int x = max(0, issued - kStages); x < issued; ++x)
      mbar_wait(bar_full(ring, x % kStages), (x / kStages) & 1, &never, nullptr, 10000000ull);
  }
}

// A barrier of the compute warps (N threads), and the same saying whether any of
// the threads says so: every warp takes the same way out.
template <int N>
__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ bool compute_sync_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "n"(N)
      : "memory");
  return r != 0;
}

// Storage types of the pages, and which partials are made again (see paged_rows_again).
struct Bf16Pages {
  using K = __nv_bfloat16;
  using V = __half;
  static constexpr bool kAll = false;
};
struct F32Pages {
  using K = float;
  using V = float;
  static constexpr bool kAll = true;
};

// The end of a piece: false if a warp's wait gave up; `odd`: this thread met a number
// of the piece's partials that is not finite.  One barrier where neither is so.
template <int D, typename P, typename Walk>
__device__ __forceinline__ bool close_piece(const PagedWork& w, const Walk& k, int valid, int part, bool ok, bool odd) {
  if (!compute_sync_or<128>(!ok || odd)) return true;
  if (compute_sync_or<128>(!ok)) return false;
  paged_rows_again<D, typename P::K, typename P::V, P::kAll>(w, w.list, k.it, k.i, k.h, k.row0(), valid, k.key_begin(),
                                                             k.key_end(), part);
  return true;
}

// The end of a piece on the four compute warps: joins the WN warps of each row
// group, a quarter of the columns at a time, in the order of the warps, and
// leaves the piece's partial.  o: m16n8 fragments of the warp's 16 rows.  false: a
// warp's wait gave up.  With kFew rows or fewer (a decode step of as many query heads
// a KV head) all columns go at once, two barriers instead of nine: 8 unshared
// sequences 11.2 -> 10.8 us, of d 64 7.5 -> 7.2, two answers of d 256 9.7 -> 9.3, of
// fp32 12.7 -> 12.3 (a call that has both kinds, 4 answers to 2500 tokens, 13.7 ->
// 13.9: more code to fetch).
constexpr int kFew = 4;
template <int D, typename C, typename P, int kMax, int WM, int WN, typename Walk>
__device__ __forceinline__ bool finish_piece(const PagedWork& w, const Walk& k, const Ring& ctx, float (&o)[D / 8][4],
                                             const float (&m)[2], float (&l)[2], bool ok) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wm = warp / WN;
  float* join = reinterpret_cast<float*>(ctx.smem + C::kOffJoin);
  float2* ml = reinterpret_cast<float2*>(ctx.smem + C::kOffMl);
  const int part = paged_part_row(blockIdx.x, kMax, k.item_row, k.seg(), k.ts);
  const int valid = min(k.rows() - k.row0(), WM * 16);
  float mark = 0.f;
  if constexpr (kMax == 16) {
    if (valid <= kFew) {
      constexpr int kStride = D + 8;  // floats; four rows' writes hit all banks
      const int row = lane >> 2;
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], 2);
      if (row < valid) {
        if ((lane & 3) == 0) ml[warp * kFew + row] = make_float2(m[0], l[0]);
        float* dst = join + (warp * kFew + row) * kStride + 2 * (lane & 3);
#pragma unroll
        for (int j = 0; j < D / 8; ++j) *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(o[j][0], o[j][1]);
      }
      compute_sync<128>();
      for (int x = threadIdx.x; x < valid * (D / 4); x += 128) {
        const int r = x / (D / 4), v = x % (D / 4);
        float top = -INFINITY, sum = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < 4; ++y) top = fmaxf(top, ml[y * kFew + r].x);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float2 z = ml[y * kFew + r];
          const float f = top == -INFINITY ? 1.f : ex2_approx(z.x - top);
          const float4 u = *reinterpret_cast<const float4*>(join + (y * kFew + r) * kStride + 4 * v);
          sum = fmaf(z.y, f, sum);
          a.x = fmaf(u.x, f, a.x);
          a.y = fmaf(u.y, f, a.y);
          a.z = fmaf(u.z, f, a.z);
          a.w = fmaf(u.w, f, a.w);
        }
        mark = odd_mark(a.x, a.y, odd_mark(a.z, a.w, mark));
        *reinterpret_cast<float4*>(w.list.part_o + static_cast<long long>(part + r) * D + 4 * v) = a;
        if (v == 0) w.list.part_ml[part + r] = make_float2(top, sum);
      }
      return close_piece<D, P>(w, k, valid, part, ok, is_odd(mark));
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    if ((lane & 3) == 0) ml[warp * 16 + (lane >> 2) + 8 * e] = make_float2(m[e], l[e]);
  }
  compute_sync<128>();
  float f[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float top = -INFINITY;
#pragma unroll
    for (int x = 0; x < WN; ++x) top = fmaxf(top, ml[(wm * WN + x) * 16 + (lane >> 2) + 8 * e].x);
    f[e] = top == -INFINITY ? 1.f : ex2_approx(m[e] - top);
  }
  if (threadIdx.x < WM * 16 && static_cast<int>(threadIdx.x) < valid) {
    const int g = threadIdx.x >> 4, r = threadIdx.x & 15;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int x = 0; x < WN; ++x) top = fmaxf(top, ml[(g * WN + x) * 16 + r].x);
#pragma unroll
    for (int x = 0; x < WN; ++x) {
      const float2 v = ml[(g * WN + x) * 16 + r];
      sum += v.y * (top == -INFINITY ? 1.f : ex2_approx(v.x - top));
    }
    w.list.part_ml[part + threadIdx.x] = make_float2(top, sum);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const int jj = c * (D / 32) + j;
      float* dst = join + (warp * 16 + (lane >> 2)) * C::kJoinStride + 8 * j + 2 * (lane & 3);
      *reinterpret_cast<float2*>(dst) = make_float2(o[jj][0] * f[0], o[jj][1] * f[0]);
      *reinterpret_cast<float2*>(dst + 8 * C::kJoinStride) = make_float2(o[jj][2] * f[1], o[jj][3] * f[1]);
    }
    compute_sync<128>();
    constexpr int kVecs = D / 16;  // float4s of a row's quarter
    for (int x = threadIdx.x; x < valid * kVecs; x += 128) {
      const int r = x / kVecs, v = x % kVecs;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < WN; ++y) {
        const float4 u = *reinterpret_cast<const float4*>(
            join + (((r >> 4) * WN + y) * 16 + (r & 15)) * C::kJoinStride + 4 * v);
        a.x += u.x;
        a.y += u.y;
        a.z += u.z;
        a.w += u.w;
      }
      mark = odd_mark(a.x, a.y, odd_mark(a.z, a.w, mark));
      *reinterpret_cast<float4*>(w.list.part_o + static_cast<long long>(part + r) * D + c * (D / 4) + 4 * v) = a;
    }
    if (c < 3) compute_sync<128>();
  }
  return close_piece<D, P>(w, k, valid, part, ok, is_odd(mark));
}

// The same where every warp has 16 rows of its own: the fragments go out as they
// are, a row's 32-byte sector from four lanes (16 answers to 1000 tokens of d 256
// 29.9 -> 29.0 us, 4 of 4 tokens of d 64 to 2567 16.0 -> 15.4, against the way above).
template <int D, typename P, int kMax, typename Walk>
__device__ __forceinline__ bool finish_apart(const PagedWork& w, const Walk& k, const float (&o)[D / 8][4],
                                             const float (&m)[2], float (&l)[2], bool ok) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = paged_part_row(blockIdx.x, kMax, k.item_row, k.seg(), k.ts);
  const int valid = k.rows() - k.row0();
  float mark = 0.f;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    const int r = warp * 16 + (lane >> 2) + 8 * e;
    if (r < valid) {
      if ((lane & 3) == 0) w.list.part_ml[part + r] = make_float2(m[e], l[e]);
      float* dst = w.list.part_o + static_cast<long long>(part + r) * D + 2 * (lane & 3);
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        mark = odd_mark(o[j][2 * e], o[j][2 * e + 1], mark);
        *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(o[j][2 * e], o[j][2 * e + 1]);
      }
    }
  }
  return close_piece<D, P>(w, k, min(valid, 64), part, ok, is_odd(mark));
}

// One piece on the four compute warps: WM warps along the rows, WN along a
// tile's keys.  false: a warp's wait gave up.
template <int D, int kMax, int WM, int WN>
__device__ __forceinline__ bool mma_piece(const PagedWork& w, const PagedWalk<kBN, kMax>& k, Ring& ctx) {
  using C = MmaCfg<D>;
  constexpr int kWarpKeys = kBN / WN;
  constexpr int kSub = WN == 4 ? 16 : (D == 256 ? 16 : 32);  // keys of one softmax step
  constexpr int kPairs = kSub / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp / WN, wn = warp % WN;
  const int gh = k.group_heads;
  const int h = k.h, rows = k.rows(), row0 = k.row0();
  const float scale_log2 = w.scale * kLog2e;

  // the warp's 16 rows, one a lane (one copy of the code for both of a thread's rows)
  int my_lim = 0;
  long long my_q = -1;
  {
    const int r = row0 + wm * 16 + (lane & 15);
    if (r < rows) {
      const int tr = w.by_group(r), t = k.it.t0 + tr;
      const int b = k.i < w.p.num_groups ? paged_seq_of(w.p, t) : k.it.row;
      my_lim = min(k.it.hi, paged_limit(w.p, b, t));
      my_q = t * w.q_stride + static_cast<long long>((h - tr) * gh + r) * D;
    }
  }
  // the smallest and largest limit over the valid rows
  const int lim_min = __reduce_min_sync(0xffffffffu, my_q < 0 ? INT_MAX : my_lim);
  const int lim_max = __reduce_max_sync(0xffffffffu, my_lim);
  // this thread's two rows: lane / 4 and + 8
  int lim[2];
  const __nv_bfloat16* qrow[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    lim[e] = __shfl_sync(0xffffffffu, my_lim, (lane >> 2) + 8 * e);
    const long long at = __shfl_sync(0xffffffffu, my_q, (lane >> 2) + 8 * e);
    qrow[e] = at < 0 ? nullptr : static_cast<const __nv_bfloat16*>(w.q) + at;
  }

  uint32_t qf[D / 16][4];
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat16* q = qrow[e & 1];
      qf[s][e] = q == nullptr ? 0u : *reinterpret_cast<const uint32_t*>(q + 16 * s + (e >> 1) * 8 + (lane & 3) * 2);
    }
  }

  float o[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  const int krow = (lane & 7) + ((lane >> 4) << 3);        // K fragment rows: two 8-key groups
  const int kchunk = (lane >> 3) & 1;
  const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3);  // V fragment rows (transposed): 16 keys
  const int vchunk = lane >> 4;

  bool ok = true;  // a warp whose wait gave up still takes part in the barriers below
  for (int kt = 0; kt < k.count; ++kt) {
    ok = paged_wait_warp(bar_full(ctx, ctx.stage), ctx.phase, ctx.abort_flag);
    if (!ok) break;
    const uint32_t sk = ctx.sbase + ctx.stage * 2 * C::kTileBytes, sv = sk + C::kTileBytes;
    const int tile0 = (k.first + k.kt + kt) * kBN;
    if (lim_max > 0) {
#pragma unroll 1
      for (int sub = 0; sub < kWarpKeys; sub += kSub) {
        const int r0 = wn * kWarpKeys + sub;  // first key within the tile
        const int key0 = tile0 + r0;
        if (key0 >= lim_max || key0 + kSub <= k.it.lo) continue;
        float s[kSub / 8][4];
#pragma unroll
        for (int j = 0; j < kSub / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
          for (int pr = 0; pr < kPairs; ++pr) {
            const int row = r0 + pr * 16 + krow;
            const int chunk = (ks & 3) * 2 + kchunk;
            uint32_t b[4];
            ldsm4(b, sk + (ks >> 2) * (kBN * 128) + row * 128 + ((chunk ^ (row & 7)) << 4));
            mma_bf16(s[2 * pr], qf[ks], b[0], b[1]);
            mma_bf16(s[2 * pr + 1], qf[ks], b[2], b[3]);
          }
        }
        const bool edge = key0 < k.it.lo || key0 + kSub > lim_min;
        if (edge) {
#pragma unroll
          for (int j = 0; j < kSub / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + 8 * j + 2 * (lane & 3) + (e & 1);
              if (key < k.it.lo || key >= lim[e >> 1]) s[j][e] = -INFINITY;
            }
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < kSub / 8; ++j) {
          mx[0] = fmax3(mx[0], s[j][0], s[j][1]);
          mx[1] = fmax3(mx[1], s[j][2], s[j][3]);
        }
        bool grew = false;
        float mnew[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
          mnew[e] = fmaxf(m[e], weight_base(mx[e], scale_log2, kTopLog2));
          grew |= mnew[e] > m[e];
        }
        if (__any_sync(0xffffffffu, grew)) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            al[e] = mnew[e] > m[e] ? ex2_approx(m[e] - mnew[e]) : 1.f;
            m[e] = mnew[e];
            l[e] *= al[e];
          }
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[j][0] *= al[0];
            o[j][1] *= al[0];
            o[j][2] *= al[1];
            o[j][3] *= al[1];
          }
        }
        const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
        uint32_t pa[kPairs][4];
#pragma unroll
        for (int j = 0; j < kSub / 8; ++j) {
          const float p0 = ex2_approx(fmaf(s[j][0], scale_log2, -mu[0]));
          const float p1 = ex2_approx(fmaf(s[j][1], scale_log2, -mu[0]));
          const float p2 = ex2_approx(fmaf(s[j][2], scale_log2, -mu[1]));
          const float p3 = ex2_approx(fmaf(s[j][3], scale_log2, -mu[1]));
          l[0] += p0 + p1;
          l[1] += p2 + p3;
          pa[j >> 1][(j & 1) * 2] = pack_f16(p0, p1);
          pa[j >> 1][(j & 1) * 2 + 1] = pack_f16(p2, p3);
        }
#pragma unroll
        for (int pr = 0; pr < kPairs; ++pr) {
          // slots that hold no key of this item may hold anything, NaN
          // included, and 0 * NaN is NaN: such V rows are taken as zero
          uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
          if (edge) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + pr * 16 + e * 8 + 2 * (lane & 3);
              keep[e] = (key >= k.it.lo && key < k.it.hi ? 0xffffu : 0u) |
                        (key + 1 >= k.it.lo && key + 1 < k.it.hi ? 0xffff0000u : 0u);
            }
          }
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const int row = r0 + pr * 16 + vrow;
            const int chunk = (j & 3) * 2 + vchunk;
            uint32_t b[4];
            ldsm4_t(b, sv + (j >> 2) * (kBN * 128) + row * 128 + ((chunk ^ (row & 7)) << 4));
            mma_f16(o[2 * j], pa[pr], b[0] & keep[0], b[1] & keep[1]);
            mma_f16(o[2 * j + 1], pa[pr], b[2] & keep[0], b[3] & keep[1]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_empty<C::kStages>(ctx, ctx.stage));
    ctx.template next<C::kStages>();
  }

  if constexpr (WN == 1) {
    return finish_apart<D, Bf16Pages, kMax>(w, k, o, m, l, ok);
  } else {
    return finish_piece<D, C, Bf16Pages, kMax, WM, WN>(w, k, ctx, o, m, l, ok);
  }
}

// The start of a list's kernel: the ring's barriers and the CTA's first piece.
// false (for the whole CTA): no work.
template <typename C, int BN, int kMax>
__device__ __forceinline__ bool open_list(const PagedWork& w, unsigned char* smem_raw, Ring& ctx,
                                          PagedWalk<BN, kMax>& walk) {
  ctx.smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  ctx.sbase = smem_u32(ctx.smem);
  ctx.bar0 = ctx.sbase + C::kOffBar;
  ctx.abort_flag = reinterpret_cast<volatile int*>(ctx.smem + C::kOffBar + 8 * 2 * C::kStages);
  ctx.stage = 0;
  ctx.phase = 0;
  PagedScan* sc = reinterpret_cast<PagedScan*>(ctx.smem + C::kOffScan);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full(ctx, s), 1);
      mbar_init(bar_empty<C::kStages>(ctx, s), 4);
    }
    *ctx.abort_flag = 0;
    fence_mbar_init();
  }
  // The prefixes' kernel before this one, if any, has waited for what the call
  // reads, and writes nothing that this kernel reads or writes: no need to wait
  // for its end before this kernel's own (whose completion then stands for both).
  if (w.prefix.end == 0) wait_for_previous();
  paged_schedule<BN, kMax, kMmaThreads, 0>(w.p, w.by_group.d, w.list, sc, w.status);
  __syncthreads();
  let_next_start();
  return walk.init(&w.p, w.by_group.d, w.list, sc);
}

// kMax: rows a tile at most, 64, or 16 for a list without more (decode steps
// mostly), whose kernel then is a third of the code.
template <int D, int kMax>
__global__ void __launch_bounds__(kMmaThreads, MmaCfg<D>::kCtas)
    paged_mma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ PagedWork w) {
  using C = MmaCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Ring ctx;
  PagedWalk<kBN, kMax> walk;
  if (threadIdx.x == 32 * kProducer) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (!open_list<C, kBN, kMax>(w, smem_raw, ctx, walk)) {
    wait_for_previous();
    return;
  }
  if (threadIdx.x / 32 == kProducer) {
    page_producer<kBN, 64, C::kSlices, C::kStages>(w, walk, &tm_k, &tm_v, ctx);
  } else {
    bool ok;
    do {
      if (kMax == 16 || walk.ts == 4) {
        ok = mma_piece<D, kMax, 1, 4>(w, walk, ctx);
      } else if constexpr (kMax > 16) {
        ok = walk.ts == 5 ? mma_piece<D, kMax, 2, 2>(w, walk, ctx) : mma_piece<D, kMax, 4, 1>(w, walk, ctx);
      }
    } while (ok && walk.next());
  }
  report_abort(ctx.abort_flag, w.status);
  wait_for_previous();  // the prefixes' kernel, see open_list
}

// ------------------------------------------------------------------ fp32
// fp32 products on tf32 fragments, each number as the sum of two: x = h + l with
// h the tf32 (11 bits) nearest to x and l = x - h, 12 bits, without its last where
// it has them all: h + l is x to 2^-23, and a b = h h' + h l' + l h' to about 2^-21
// of |a b|, accumulated in fp32.  The split takes integer instructions, which takes
// 4 sequences on 14117 keys from 74 to 64 us with d 256 and from 42 to 38 with d
// 128 against the conversion's own.  An infinity, and a number that rounds to one, has
// no l that adds up to it: its products cancel to NaN, and the row is made again (see
// paged_rows_again).  A NaN whose bits the rounding carries past the sign leaves
// itself in l.  (The same in FFMA is bound by shared memory: 16 rows are too few for
// a register block that would feed it.)  A tile is 16 rows and 32 keys; the four
// warps split the keys.
constexpr int kFBN = 32;    // keys a tile
constexpr int kFRows = 16;  // rows a tile

template <int D>
struct F32Cfg {
  static constexpr int kSlices = D / 32;  // 32-column (128-byte) slices of a row
  static constexpr int kTileBytes = kFBN * D * 4;
  static constexpr int kStages = D == 64 ? 3 : 2;
  static constexpr int kCtas = D == 64 ? 3 : D == 128 ? 2 : 1;  // resident on an SM
  static constexpr int kQStride = D + 4;  // floats; + 4: 16-byte reads of 8 rows hit all banks
  static constexpr int kJoinStride = D / 4 + 8;
  static constexpr int kOffQ = kStages * 2 * kTileBytes;           // h, then l of Q
  static constexpr int kOffJoin = kOffQ + 2 * kFRows * kQStride * 4;
  static constexpr int kOffMl = kOffJoin + 4 * 16 * kJoinStride * 4;
  static constexpr int kOffScan = kOffMl + 4 * 16 * 8;
  static constexpr int kOffBar = kOffScan + ((static_cast<int>(sizeof(PagedScan)) + 15) / 16) * 16;
  static constexpr int kSmemBytes = kOffBar + 8 * 2 * kStages + 16 + 1024;
  static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "shared memory budget");
};

__device__ __forceinline__ void split_tf32(float x, uint32_t& h, uint32_t& l) {
  h = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  l = __float_as_uint(x - __uint_as_float(h)) & 0xffffe000u;
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One piece on the four compute warps.
template <int D>
__device__ __forceinline__ bool f32_piece(const PagedWork& w, const PagedWalk<kFBN, kFRows>& k, Ring& ctx) {
  using C = F32Cfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gh = k.group_heads, h = k.h, rows = k.rows(), row0 = k.row0();
  const float scale_log2 = w.scale * kLog2e;
  uint32_t* qh = reinterpret_cast<uint32_t*>(ctx.smem + C::kOffQ);
  uint32_t* ql = qh + kFRows * C::kQStride;
  // (the previous piece's last barrier is behind its reads of Q)
#pragma unroll 4
  for (int x = threadIdx.x; x < kFRows * (D / 4); x += 128) {
    const int tr = x / (D / 4), c = x % (D / 4), r = row0 + tr;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      const int t = w.by_group(r);
      v = *reinterpret_cast<const float4*>(static_cast<const float*>(w.q) + (k.it.t0 + t) * w.q_stride +
                                           static_cast<long long>((h - t) * gh + r) * D + 4 * c);
    }
    uint4 vh, vl;
    split_tf32(v.x, vh.x, vl.x);
    split_tf32(v.y, vh.y, vl.y);
    split_tf32(v.z, vh.z, vl.z);
    split_tf32(v.w, vh.w, vl.w);
    *reinterpret_cast<uint4*>(qh + tr * C::kQStride + 4 * c) = vh;
    *reinterpret_cast<uint4*>(ql + tr * C::kQStride + 4 * c) = vl;
  }
  int my_lim = 0;  // the 16 rows, one a lane
  {
    const int r = row0 + (lane & 15);
    if (r < rows) {
      const int t = k.it.t0 + w.by_group(r);
      const int b = k.i < w.p.num_groups ? paged_seq_of(w.p, t) : k.it.row;
      my_lim = min(k.it.hi, paged_limit(w.p, b, t));
    }
  }
  const int lim[2] = {__shfl_sync(0xffffffffu, my_lim, lane >> 2), __shfl_sync(0xffffffffu, my_lim, (lane >> 2) + 8)};
  float o[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const int r0 = 8 * warp;  // the warp's first key within a tile
  const int key7 = lane & 7;
  const uint32_t qa = smem_u32(qh) + (((lane & 7) + ((lane >> 3) & 1) * 8) * C::kQStride + (lane >> 4) * 4) * 4;
  constexpr uint32_t kLow = kFRows * C::kQStride * 4;
  compute_sync<128>();  // Q is there
  bool ok = true;  // a warp whose wait gave up still takes part in the barriers at the end
  for (int kt = 0; kt < k.count; ++kt) {
    ok = paged_wait_warp(bar_full(ctx, ctx.stage), ctx.phase, ctx.abort_flag);
    if (!ok) break;
    const uint32_t sk = ctx.sbase + ctx.stage * 2 * C::kTileBytes, sv = sk + C::kTileBytes;
    const int key0 = (k.first + k.kt + kt) * kFBN + r0;
    // six independent sums (products of h, and both kinds of cross products, of
    // even and odd steps): one chain of dependent MMAs would be all latency
    float sh[2][4], sx[2][4], sy[2][4];
#pragma unroll
    for (int e = 0; e < 8; ++e) sh[e >> 2][e & 3] = sx[e >> 2][e & 3] = sy[e >> 2][e & 3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {  // 16 columns
      uint32_t kr[4];
      const int chunk = (ks * 4 + (lane >> 3)) & 7;
      ldsm4(kr, sk + (ks >> 1) * (kFBN * 128) + (r0 + key7) * 128 + ((chunk ^ key7) << 4));
      uint32_t kh[4], kl[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split_tf32(__uint_as_float(kr[e]), kh[e], kl[e]);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t ah[4], al[4];
        ldsm4(ah, qa + (ks * 16 + half * 8) * 4);
        ldsm4(al, qa + kLow + (ks * 16 + half * 8) * 4);
        mma_tf32(sx[half], ah, kl[2 * half], kl[2 * half + 1]);
        mma_tf32(sh[half], ah, kh[2 * half], kh[2 * half + 1]);
        mma_tf32(sy[half], al, kh[2 * half], kh[2 * half + 1]);
      }
    }
    const int q2 = 2 * (lane & 3);
    float s[4], mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = key0 + q2 + (e & 1);
      const float dot = (sh[0][e] + sh[1][e]) + ((sx[0][e] + sx[1][e]) + (sy[0][e] + sy[1][e]));
      s[e] = key < k.it.lo || key >= lim[e >> 1] ? -INFINITY : dot * scale_log2;
      mx[e >> 1] = fmaxf(mx[e >> 1], s[e]);
    }
    bool grew = false;
    float mnew[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
      mnew[e] = fmaxf(m[e], mx[e]);
      grew |= mnew[e] > m[e];
    }
    if (__any_sync(0xffffffffu, grew)) {
      float al[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        al[e] = mnew[e] > m[e] ? ex2_approx(m[e] - mnew[e]) : 1.f;
        m[e] = mnew[e];
        l[e] *= al[e];
      }
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[j][0] *= al[0];
        o[j][1] *= al[0];
        o[j][2] *= al[1];
        o[j][3] *= al[1];
      }
    }
    // P as the A operand: k index q of the fragment stands for key 2q, q + 4 for key 2q + 1
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = ex2_approx(s[e] - (m[e >> 1] == -INFINITY ? 0.f : m[e >> 1]));
      l[e >> 1] += x;
      split_tf32(x, ph[(e & 1) * 2 + (e >> 1)], pl[(e & 1) * 2 + (e >> 1)]);
    }
    // slots that hold no key of this item may hold anything, NaN included: taken as zero
    const bool keep0 = key0 + q2 >= k.it.lo && key0 + q2 < k.it.hi;
    const bool keep1 = key0 + q2 + 1 >= k.it.lo && key0 + q2 + 1 < k.it.hi;
    const int row_a = q2, row_b = q2 + 1;  // (r0 is a multiple of 8: the swizzle goes by these alone)
    const int g = lane >> 2;
#pragma unroll
    for (int j0 = 0; j0 < D / 8; j0 += 4) {  // four 8-column blocks of O between dependent MMAs
      uint32_t vh[4][2], vl[4][2];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int j = j0 + x;
        const int chunk = (2 * j + (g >> 2)) & 7;
        const uint32_t at = sv + (j >> 2) * (kFBN * 128) + r0 * 128 + (g & 3) * 4;
        float v0, v1;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v0) : "r"(at + row_a * 128 + ((chunk ^ row_a) << 4)) : "memory");
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v1) : "r"(at + row_b * 128 + ((chunk ^ row_b) << 4)) : "memory");
        split_tf32(keep0 ? v0 : 0.f, vh[x][0], vl[x][0]);
        split_tf32(keep1 ? v1 : 0.f, vh[x][1], vl[x][1]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) mma_tf32(o[j0 + x], ph, vl[x][0], vl[x][1]);
#pragma unroll
      for (int x = 0; x < 4; ++x) mma_tf32(o[j0 + x], pl, vh[x][0], vh[x][1]);
#pragma unroll
      for (int x = 0; x < 4; ++x) mma_tf32(o[j0 + x], ph, vh[x][0], vh[x][1]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_empty<C::kStages>(ctx, ctx.stage));
    ctx.template next<C::kStages>();
  }
  return finish_piece<D, C, F32Pages, kFRows, 1, 4>(w, k, ctx, o, m, l, ok);
}

template <int D>
__global__ void __launch_bounds__(kMmaThreads, F32Cfg<D>::kCtas)
    paged_f32_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ PagedWork w) {
  using C = F32Cfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Ring ctx;
  PagedWalk<kFBN, kFRows> walk;
  if (!open_list<C, kFBN, kFRows>(w, smem_raw, ctx, walk)) return;
  if (threadIdx.x / 32 == kProducer) {
    page_producer<kFBN, 32, C::kSlices, C::kStages>(w, walk, &tm_k, &tm_v, ctx);
  } else {
    while (f32_piece<D>(w, walk, ctx) && walk.next()) {
    }
  }
  report_abort(ctx.abort_flag, w.status);
}

// ------------------------------------------------------------------ join
// The partials of a row (token, head): its prefix segment's and its own
// segment's, in the order of the CTAs that made them.  WARPS warps take a row,
// each a share of its partials, and join in the order of the warps: 4 where the
// rows are few, so that a row's partials are all in flight at once, and 1 where they
// are many, so that the CTAs are few enough to be there, their places
// looked up, when the kernel before ends.  The whole call with 4 / 1, in us: 128
// rows 9.3 / 11.1, 512 rows 15.6 / 17.1, 1024 rows 57.6 / 61.9, 1536 rows 138.4 /
// 136.3, 2048 rows 187.0 / 187.9.
// What it reads before it waits (offsets, lengths, groups) is the call's input, which
// the kernel that let it start does not write, and which is complete: that kernel had
// waited for the one before it, or was itself let start by the prefixes' kernel, which had.
template <int N>
struct __align__(N >= 4 ? 16 : 8) Cols {  // consecutive numbers, read and written together
  float x[N];
};
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void store2(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}

template <int D, typename T, int BN, int kMax, int WARPS>
__global__ void __launch_bounds__(128) paged_join_kernel(const __grid_constant__ PagedWork w) {
  let_next_start();
  constexpr int kCols = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x, h = blockIdx.y * (4 / WARPS) + warp / WARPS;
  const int part = warp % WARPS;
  const int gh = w.by_group.d;
  const int b = paged_seq_of(w.p, t);
  // a row's partials of one item: rows at + j * kStep for j < count
  struct Place {
    int seg, nt, ts, in_tile;  // segment, its key tiles, log2 rows a tile, row in the tile
    int j, n;                  // item of its list, items
  };
  auto place = [&](auto span, const PagedList& l, int i) -> Place {
    using Span = decltype(span);
    const PagedItem it = paged_item(w.p, i);
    const Span sp(it, gh);
    const int g = w.by_group(h), r = (t - it.t0 - g) * gh + h;
    return Place{g * sp.rt + (r >> sp.ts), sp.nt, sp.ts, r & ((1 << sp.ts) - 1), i - l.begin, l.end - l.begin};
  };
  constexpr int kPrefixRows = paged_prefix_rows(D);
  const bool own_list = w.prefix.end > 0;
  const int limit = paged_limit(w.p, b, t);
  Place pp{0, 0, 0, 0, 0, 0};
  if (w.p.num_groups > 0) {
    const int g = paged_group_of(w.p, b);
    pp = own_list ? place(PagedSpan<paged_prefix_keys(D), kPrefixRows>(), w.prefix, g)
                  : place(PagedSpan<BN, kMax>(), w.list, g);
  }
  const Place po = place(PagedSpan<BN, kMax>(), w.list, w.p.num_groups + b);
  wait_for_previous();
  const bool live = h < w.num_q_heads;
  // the first and last partial of the prefix's segment (lanes 0 and 1 of four) and of
  // the row's own (2 and 3), found side by side: divisions are long code to fetch
  const PagedList& pl = own_list ? w.prefix : w.list;
  const int pstep = own_list ? kPrefixRows : kMax;
  int first, owner;
  {
    const bool own = (lane & 2) != 0, last = (lane & 1) != 0;
    const int* items = own ? w.list.items : pl.items;
    const int seg = own ? po.seg : pp.seg, nt = own ? po.nt : pp.nt, ts = own ? po.ts : pp.ts;
    const int j = own ? po.j : pp.j, n = own ? po.n : pp.n;
    const int how = items[n + 1];
    PagedCut cut{items[n], max(how, 0), max(-how, 0), w.list.by_ctas};
    if (!own) cut.by_ctas = pl.by_ctas;
    // (the prefixes' own list has no extra tiles: there a tile is one unit)
    const int wt = cut.tile_units<kMax>(ts);
    const int u0 = items[j] + seg * cut.padded(nt, wt);
    owner = cut.owner(last ? u0 + (nt - 1) * wt : u0);
    first = paged_part_row(owner, own ? kMax : pstep, items[n + 2 + j], seg, ts) + (own ? po.in_tile : pp.in_tile);
  }
  const int pfirst = __shfl_sync(0xffffffffu, first, 0), ofirst = __shfl_sync(0xffffffffu, first, 2);
  const int spans = __shfl_down_sync(0xffffffffu, owner, 1) - owner + 1;
  const bool sees = limit > 0 && live;
  const int pcount = sees && pp.nt > 0 ? __shfl_sync(0xffffffffu, spans, 0) : 0;
  const int ocount = sees && po.nt > 0 ? __shfl_sync(0xffffffffu, spans, 2) : 0;
  const int all = pcount + ocount;
  float m = -INFINITY, sum = 0.f;
  __align__(16) float acc[kCols];  // columns lane * kCols and on
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
  // partials in flight a warp (4 / 8, in us: 4 short answers 9.6 / 9.2, 16 to 8192
  // tokens 27.3 / 26.4; d 256, 5 tokens on 4097 keys, 38.2 / 40.4)
  constexpr int kBatch = D == 256 ? 4 : 8;
#pragma unroll 1
  for (int j0 = part; j0 < all; j0 += WARPS * kBatch) {
    float2 ml[kBatch];
    __align__(16) float x[kBatch][kCols];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + WARPS * i;
      ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int c = 0; c < kCols; ++c) x[i][c] = 0.f;
      if (j < all) {
        const bool pre = j < pcount;
        const int r = pre ? pfirst + j * pstep : ofirst + (j - pcount) * kMax;
        ml[i] = (pre ? pl.part_ml : w.list.part_ml)[r];
        const float* o = (pre ? pl.part_o : w.list.part_o) + static_cast<long long>(r) * D;
        *reinterpret_cast<Cols<kCols>*>(x[i]) = *reinterpret_cast<const Cols<kCols>*>(o + lane * kCols);
      }
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[i].x);
    const float base = top == -INFINITY ? 0.f : top;
    const float f = ex2_approx(m - base);
    m = top;
    sum *= f;
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] *= f;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float g = ex2_approx(ml[i].x - base);
      sum = fmaf(ml[i].y, g, sum);
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = fmaf(x[i][c], g, acc[c]);
    }
  }
  if constexpr (WARPS == 4) {
    __shared__ __align__(16) float acc_s[4][D];
    __shared__ float2 ml_s[4];
    *reinterpret_cast<Cols<kCols>*>(&acc_s[warp][lane * kCols]) = *reinterpret_cast<const Cols<kCols>*>(acc);
    if (lane == 0) ml_s[warp] = make_float2(m, sum);
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY, f[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) top = fmaxf(top, ml_s[x].x);
    const float base = top == -INFINITY ? 0.f : top;
    sum = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      f[x] = ex2_approx(ml_s[x].x - base);
      sum = fmaf(ml_s[x].y, f[x], sum);
    }
    m = top;
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      acc[c] = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[c] = fmaf(acc_s[x][lane * kCols + c], f[x], acc[c]);
    }
  }
  if (!live) return;
  T* out = static_cast<T*>(w.out) + t * w.out_stride + static_cast<long long>(h) * D;
  const float inv = limit > 0 ? 1.f / sum : 0.f;  // a row that sees no key: acc is 0
#pragma unroll
  for (int c = 0; c < kCols; c += 2)
    store2(out + lane * kCols + c, acc[c] * inv, acc[c + 1] * inv);
  if (w.lse != nullptr && lane == 0) {
    // (f16 weights are lifted by up to 2^15: taken out of both, the logarithm is of a number near the plain sum)
    constexpr float kLift = sizeof(T) == 2 ? kTopLog2 : 0.f, kDown = sizeof(T) == 2 ? 0x1p-15f : 1.f;
    w.lse[static_cast<long long>(t) * w.num_q_heads + h] =
        limit > 0 ? ((m + kLift) + log2f(sum * kDown)) * kLn2 : -INFINITY;
  }
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Key tiles that a segment counts beside its own, for its Q, its first tile's
// latency and its end.  With 1 / 2 / 3 / 4, in us: 32 answers to 32K 57.9 / 57.7 /
// 58.3 / 58.6, 5 tokens on 4097 keys, d 256, 39.5 / 38.6 / 39.3 / 40.3, 7 tokens of
// 16 unshared sequences 28.2 / 26.5 / 26.0 / 26.9, 16 answers to 8192 tokens 28.3 /
// 26.5 / 26.1 / 26.1, 32 to 2048 24.1 / 22.9 / 23.7 / 23.6, fp32 with 14117 shared
// and up to 13 own tokens 67.8 / 64.6 / 65.2 / 66.5.
constexpr int kSegmentTiles = 2;
static_assert(kSegmentTiles > 0, "extra tiles are also the mark that tiles count their units");

// CTAs of a grid at most: what the partials are sized for.
constexpr int kMaxCtas = 148 * 3;

constexpr int kFewRows = 1024;  // of the join, see there

template <int D, typename T, int BN, int kMax>
cudaError_t join(const PagedWork& w, cudaStream_t stream) {
  const long long rows = static_cast<long long>(w.p.total_q) * w.num_q_heads;
  if (rows <= kFewRows)
    return launch_early(paged_join_kernel<D, T, BN, kMax, 4>, dim3(w.p.total_q, w.num_q_heads), 128, 0, stream, w);
  return launch_early(paged_join_kernel<D, T, BN, kMax, 1>, dim3(w.p.total_q, (w.num_q_heads + 3) / 4), 128, 0, stream,
                      w);
}

template <int D, int kMax>
cudaError_t run_mma(PagedWork w, cudaStream_t stream) {
  using C = MmaCfg<D>;
  CUtensorMap mk, mv;
  if (encode_pages_map(&mk, w.p.k_pages, w.p, kBN, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) != CUDA_SUCCESS ||
      encode_pages_map(&mv, w.p.v_pages, w.p, kBN, CU_TENSOR_MAP_DATA_TYPE_FLOAT16) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaError_t e =
      cudaFuncSetAttribute(paged_mma_kernel<D, kMax>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  w.list.by_ctas = FastDiv(sms * C::kCtas < kMaxCtas ? sms * C::kCtas : kMaxCtas);
  w.list.extra = kSegmentTiles;
  if (w.prefix.end > 0) {
    w.prefix.by_ctas = FastDiv(sms < kMaxCtas ? sms : kMaxCtas);
    if ((e = launch_paged_prefix(w, stream)) != cudaSuccess) return e;
  }
  e = launch_early(paged_mma_kernel<D, kMax>, w.list.by_ctas.d, kMmaThreads, C::kSmemBytes, stream, mk, mv, w);
  if (e != cudaSuccess) return e;
  return join<D, __nv_bfloat16, kBN, kMax>(w, stream);
}

template <int D>
cudaError_t run_f32(PagedWork w, cudaStream_t stream) {
  using C = F32Cfg<D>;
  CUtensorMap mk, mv;
  if (encode_pages_map(&mk, w.p.k_pages, w.p, kFBN, CU_TENSOR_MAP_DATA_TYPE_FLOAT32) != CUDA_SUCCESS ||
      encode_pages_map(&mv, w.p.v_pages, w.p, kFBN, CU_TENSOR_MAP_DATA_TYPE_FLOAT32) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(paged_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  w.list.by_ctas = FastDiv(sms * C::kCtas < kMaxCtas ? sms * C::kCtas : kMaxCtas);
  w.list.extra = kSegmentTiles;
  e = launch_early(paged_f32_kernel<D>, w.list.by_ctas.d, kMmaThreads, C::kSmemBytes, stream, mk, mv, w);
  if (e != cudaSuccess) return e;
  return join<D, float, kFBN, kFRows>(w, stream);
}

}  // namespace

// (d, page_size, Hkv, pages) view of a page array; one box is 128 bytes of up
// to `tile` tokens of a page, as rows of 128 bytes, swizzled.
CUresult encode_pages_map(CUtensorMap* map, const void* base, const PagedArgs& p, int tile,
                          CUtensorMapDataType type) {
  const TensorMapEncodeFn fn = tensor_map_encode_fn();
  if (fn == nullptr) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t bytes = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.head_dim), static_cast<cuuint64_t>(p.page_size),
                              static_cast<cuuint64_t>(p.num_kv_heads), static_cast<cuuint64_t>(p.num_pages)};
  const cuuint64_t strides[3] = {p.head_dim * bytes, static_cast<cuuint64_t>(p.page_size) * p.head_dim * bytes,
                                 static_cast<cuuint64_t>(p.page_stride) * bytes};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / bytes),
                             static_cast<cuuint32_t>(p.page_size < tile ? p.page_size : tile), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, type, 4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

PagedShape paged_shape(const PagedArgs& p, const int* h_cu_q, const int* h_group_ptr, int num_q_heads, int dtype) {
  PagedShape s{};
  const int gh = num_q_heads / p.num_kv_heads, G = p.num_groups, cap = p.max_pages * p.page_size;
  const bool bf16 = dtype == DHSA_BF16, wide = paged_prefix_rows(p.head_dim) == 256;
  auto group_rows = [&](int g) -> long long {
    return static_cast<long long>(h_cu_q[h_group_ptr[g + 1]] - h_cu_q[h_group_ptr[g]]) * gh;
  };
  auto seq_rows = [&](int b) -> long long { return static_cast<long long>(h_cu_q[b + 1] - h_cu_q[b]) * gh; };
  long long most_g = 0, all_g = 0, most_s = 0;
  for (int g = 0; g < G; ++g) {
    const long long r = group_rows(g);
    most_g = r > most_g ? r : most_g;
    all_g += r;
  }
  for (int b = 0; b < p.num_seqs; ++b) most_s = seq_rows(b) > most_s ? seq_rows(b) : most_s;
  const double work = static_cast<double>(all_g) * p.num_kv_heads * p.head_dim * cap;
  s.own_prefix = bf16 && most_g > kOwnPrefixRows && work >= static_cast<double>(kOwnPrefixWork);
  s.prefix_items = s.own_prefix ? G : 0;
  s.list_items = G + p.num_seqs - s.prefix_items;
  const long long most = s.own_prefix || most_s > most_g ? most_s : most_g;
  s.list_max = !bf16 || most <= 16 ? 16 : 64;
  // row tiles of an item, by the list's largest tile
  long long units[2] = {0, 0};
  auto add = [&](long long r, int max, int x, long long& rows) {
    const int ts = max == 256   ? paged_tile_shift<256>(static_cast<int>(r))
                   : max == 128 ? paged_tile_shift<128>(static_cast<int>(r))
                   : max == 64  ? paged_tile_shift<64>(static_cast<int>(r))
                                : paged_tile_shift<16>(static_cast<int>(r));
    const long long tiles = (r + (1 << ts) - 1) >> ts;
    rows += tiles * p.num_kv_heads << ts;
    units[x] += tiles * p.num_kv_heads * (cap / (x == 0 ? paged_prefix_keys(p.head_dim) : bf16 ? kBN : kFBN) + 4) *
                (max == 64 ? paged_tile_units<64>(ts) : 1);
  };
  for (int g = 0; g < G; ++g)
    s.own_prefix ? add(group_rows(g), wide ? 256 : 128, 0, s.prefix_rows)
                 : add(group_rows(g), s.list_max, 1, s.list_rows);
  for (int b = 0; b < p.num_seqs; ++b) add(seq_rows(b), s.list_max, 1, s.list_rows);
  if (s.own_prefix) s.prefix_rows += static_cast<long long>(kMaxCtas) * paged_prefix_rows(p.head_dim);
  s.list_rows += static_cast<long long>(kMaxCtas) * s.list_max;
  s.fits = units[0] < (1ll << 30) && units[1] < (1ll << 30) && s.prefix_rows < INT32_MAX && s.list_rows < INT32_MAX;
  return s;
}

cudaError_t launch_paged_attention(const PagedWork& w, const PagedShape& shape, int dtype, cudaStream_t stream) {
  if (w.p.total_q <= 0) return cudaSuccess;
  if (dtype == DHSA_BF16) {
    const bool small = shape.list_max == 16;
    switch (w.p.head_dim) {
      case 64: return small ? run_mma<64, 16>(w, stream) : run_mma<64, 64>(w, stream);
      case 128: return small ? run_mma<128, 16>(w, stream) : run_mma<128, 64>(w, stream);
      default: return small ? run_mma<256, 16>(w, stream) : run_mma<256, 64>(w, stream);
    }
  }
  switch (w.p.head_dim) {
    case 64: return run_f32<64>(w, stream);
    case 128: return run_f32<128>(w, stream);
    default: return run_f32<256>(w, stream);
  }
}

}  // namespace dhsa
