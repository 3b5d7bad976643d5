// The work list of paged attention, shared by its kernels: items, segments,
// pieces, and where their partial results lie (see PagedWork in serving.h).
#pragma once

#include "common.cuh"
#include "launch_early.cuh"
#include "serving.h"

namespace dhsa {

// 4-D tiled load (no multicast) into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  const int n = take ? 16 : 0;  // 0: the destination is zeroed
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// Waits of these kernels are on their own CTA's warps and copies.  One that runs out
// sets the CTA's abort flag, which ends the CTA's work and no other's, and is reported
// at the end (report_abort).  The status word gathers reports across calls, so no wait
// looks there: they get none to look at.
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait(bar, parity, abort_flag, nullptr);
}
__device__ __forceinline__ bool paged_wait_spin(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait_spin(bar, parity, abort_flag, nullptr);
}
// By a whole warp with one answer: where a lane gives up, all do, and the warp goes on
// together (votes and shuffles behind a wait count on all its lanes).
__device__ __forceinline__ bool paged_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, paged_wait(bar, parity, abort_flag));
}
// By every warp (or a thread behind a barrier of all) that has done its last wait.
__device__ __forceinline__ void report_abort(volatile int* abort_flag, uint32_t* status) {
  if (*abort_flag) report(status, kDevTimeout);
}

constexpr float kLog2e = 1.4426950408889634f;

// The base that a row's weights 2^(x - base) are taken against, by its largest
// logit so far (scores times scale, in log2 units): the largest weight becomes
// 2^lift, so that those far below it keep their bits in f16, where numbers are
// normal from 2^-14 and come in steps of 2^-24 below.  A weight is off by 2^-11 of
// itself, or by 2^-(25 + lift) of the row's largest where that is more.  The sums of
// weights carry the same factor.  Rounded up, so that x - base never passes lift.
__device__ __forceinline__ float weight_base(float top_score, float scale_log2, float lift) {
  return __fadd_ru(__fmul_ru(top_score, scale_log2), -lift);
}
constexpr float kTopLog2 = 15.f;  // f16 weights are 2^15 at most

// One item: the query tokens [t0, t1) over the keys [lo, hi) of a table row.
struct PagedItem {
  int t0, t1, lo, hi, row;
};

__device__ __forceinline__ int paged_clamp_len(const PagedArgs& p, int n) {
  return min(max(n, 0), p.max_pages * p.page_size);
}

// The group that holds sequence b (the last g with group_ptr[g] <= b).
__device__ __forceinline__ int paged_group_of(const PagedArgs& p, int b) {
  int lo = 0, hi = p.num_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.group_ptr[mid] <= b) lo = mid; else hi = mid;
  }
  return lo;
}

// The sequence that brings token t < total_q.
__device__ __forceinline__ int paged_seq_of(const PagedArgs& p, int t) {
  if (p.uniform_q > 0) return p.by_uniform_q(t);
  int lo = 0, hi = p.num_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_q[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Keys visible to token t of sequence b.
__device__ __forceinline__ int paged_limit(const PagedArgs& p, int b, int t) {
  return paged_clamp_len(p, p.kv_lens[b]) - (p.cu_q[b + 1] - 1 - t);
}

// Item i: the groups come first, then the sequences.  A kernel's list is the
// items begin .. end - 1 of them.
__device__ __forceinline__ PagedItem paged_item(const PagedArgs& p, int i) {
  PagedItem it;
  if (i < p.num_groups) {
    const int s0 = min(max(p.group_ptr[i], 0), p.num_seqs), s1 = min(max(p.group_ptr[i + 1], s0), p.num_seqs);
    it.t0 = p.cu_q[s0];
    it.t1 = p.cu_q[s1];
    it.lo = 0;
    it.hi = paged_clamp_len(p, p.prefix_lens[i]);
    it.row = s0;
    if (s0 == s1) it.hi = 0;
  } else {
    const int b = i - p.num_groups;
    it.t0 = p.cu_q[b];
    it.t1 = p.cu_q[b + 1];
    it.hi = paged_clamp_len(p, p.kv_lens[b]);
    it.lo = p.num_groups > 0 ? min(paged_clamp_len(p, p.prefix_lens[paged_group_of(p, b)]), it.hi) : 0;
    it.row = b;
  }
  return it;
}

// log2 of the rows of one segment's tile: a power of two from 16 to kMax that
// the item's rows fill, so that few rows (one decode step of one sequence) take
// the form in which all four warps split the keys, and many are worked on together.
template <int kMax>
__host__ __device__ __forceinline__ int paged_tile_shift(int rows) {
  int m = 4;
  while ((1 << m) < kMax && (1 << m) < rows) ++m;
  return m;
}

// Units that a key tile counts, by log2 of its rows (see PagedCut): in the kernel
// with tiles of up to 64 rows one of 64 takes about 2.6 times as long as one of
// 16.  Counting every tile alike / 1, 2, 3, in us (32 + 8 heads of 128, up to 512
// own keys): 16 sequences on 1024 shared keys 18.8 / 15.4, on 8192 29.4 / 26.5, 32
// on 2048 29.7 / 22.9; of d 256, 16 on 1000 43.4 / 28.1.
template <int kMax>
__host__ __device__ __forceinline__ constexpr int paged_tile_units(int ts) {
  return kMax != 64 ? 1 : ts - 3;
}

// An item's segments and key tiles.
template <int BN, int kMaxRows>
struct PagedSpan {
  static constexpr int kMax = kMaxRows;
  int rows, ts, rt, first, nt;  // rows; log2 rows a tile, row tiles; first key tile, key tiles
  PagedSpan() = default;
  __device__ __forceinline__ PagedSpan(const PagedItem& it, int group_heads) {
    rows = (it.t1 - it.t0) * group_heads;
    ts = paged_tile_shift<kMaxRows>(rows);
    rt = (rows + (1 << ts) - 1) >> ts;
    first = it.lo / BN;
    nt = it.hi > it.lo && rows > 0 ? (it.hi + BN - 1) / BN - first : 0;
  }
};

// How a list's units (fewer than 2^30) are cut among the CTAs.  chunk 0: the
// units are cut evenly, wherever that falls, and a key tile belongs to the CTA
// that holds its first unit.  extra > 0: a tile counts paged_tile_units, and a
// segment the units of `extra` more tiles behind its own, for what its start and
// end cost; every CTA has at least as many units as any tile counts.  extra 0
// (short lists): a tile is one unit, and with fewer units than CTAs the first
// `total` CTAs take one each.  Either way every CTA between the owners of a
// segment's first and last tile has a partial of it.
// chunk > 0: every segment counts as a whole number of chunks, a CTA takes one
// chunk, and none has two segments.
struct PagedCut {
  int total, chunk, extra;
  FastDiv by_ctas;
  template <int kMax>
  __device__ __forceinline__ int tile_units(int ts) const {
    return extra > 0 ? paged_tile_units<kMax>(ts) : 1;
  }
  __device__ __forceinline__ int padded(int nt, int wt) const {  // a segment's units
    return chunk > 0 ? (nt + chunk - 1) / chunk * chunk : nt > 0 ? (nt + extra) * wt : 0;
  }
  __device__ __forceinline__ int first(int c) const {  // the first unit of CTA c: c * total / ctas
    if (chunk > 0) return min(c * chunk, total);
    const int n = by_ctas.d;
    if (total <= n) return min(c, total);
    const int q = by_ctas(total);
    return c * q + by_ctas(c * (total - q * n));
  }
  __device__ __forceinline__ int owner(int unit) const {  // the CTA that holds a unit
    if (chunk > 0) return unit / chunk;
    const int n = by_ctas.d;
    if (total <= n) return unit;
    // ((unit + 1) * ctas - 1) / total; 32 bits divide several times faster than 64
    const unsigned long long x = static_cast<unsigned long long>(unit + 1) * n - 1;
    return static_cast<int>(x >> 32 == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(total) : x / total);
  }
};

// Where CTA c's partial of a segment starts (rows): c steps by the largest
// tile, a segment by its own rows, and along the list either c or the segment moves
// on, so no two partials overlap.
__device__ __forceinline__ int paged_part_row(int c, int max_rows, int item_row, int seg, int ts) {
  return c * max_rows + item_row + (seg << ts);
}

// Shared-memory words of the block-wide scan.
struct PagedScan {
  int warp_units[8], warp_rows[8], warp_segs[8];
  PagedCut cut;
  int item_unit, item_row;
  PagedItem it;
  int item;
};

// Every CTA counts the units of all items (each thread a run of them) and finds
// the item that holds its first unit.  CTA 0 writes the items' first units and
// rows, and the cut, for the join.  kSnap > 0: where the segments are fewer than
// half of the CTAs, they are cut into chunks, unless the longest share then is
// more than kSnap units (what a second piece costs a CTA) above the even one.
// Called by the CTA's last kThreads threads, which meet at barrier 1; the result
// is for the whole CTA after its next __syncthreads.
template <int BN, int kMaxRows, int kThreads, int kSnap>
__device__ __forceinline__ void paged_schedule(const PagedArgs& p, int group_heads, const PagedList& list,
                                               PagedScan* sc, uint32_t* status) {
  const int n = list.end - list.begin;
  const int per = (n + kThreads - 1) / kThreads;
  const int thread = threadIdx.x - (blockDim.x - kThreads);
  const int i0 = min(thread * per, n), i1 = min(i0 + per, n);
  const int lane = thread & 31, warp = thread >> 5;
  auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); };
  PagedCut cut{0, 0, 0, list.by_ctas};
  int base_u = 0, base_r = 0;
  // rounds (one body, so that its code comes in once): the plain count with
  // its segments (kSnap), the padded count, then the finding of this CTA's item
#pragma unroll 1
  for (int round = kSnap > 0 ? 0 : 1; round < 3; ++round) {
    const bool find = round == 2;
    const int mine = find ? cut.first(blockIdx.x) : 0;
    int units = base_u, rows = base_r;
    if (!find) units = rows = 0;
    int segs = 0;
    bool bad = false;
    for (int i = i0; i < i1; ++i) {
      const PagedItem it = paged_item(p, list.begin + i);
      const PagedSpan<BN, kMaxRows> sp(it, group_heads);
      const int tiles = p.num_kv_heads * sp.rt;
      const int du = tiles * cut.padded(sp.nt, cut.tile_units<kMaxRows>(sp.ts));
      const int dr = tiles << sp.ts;
      if (find) {
        if (du > 0 && units <= mine && mine < units + du) {
          sc->item = list.begin + i;
          sc->it = it;
          sc->item_unit = units;
          sc->item_row = rows;
        }
        if (blockIdx.x == 0) {
          list.items[i] = units;
          list.items[n + 2 + i] = rows;
        }
      } else if (blockIdx.x == 0 && round == 1) {
        const int g = list.begin + i;
        if (g < p.num_groups) {
          bad |= it.t1 > it.t0 && p.prefix_lens[g] != paged_clamp_len(p, p.prefix_lens[g]);
        } else {
          bad |= p.kv_lens[g - p.num_groups] != it.hi;
        }
      }
      units += du;
      rows += dr;
      // segments, or (no chunks) the units that they count beside their tiles
      segs += sp.nt == 0 ? 0
              : kSnap > 0 ? tiles
                          : tiles * ((sp.nt + list.extra) * paged_tile_units<kMaxRows>(sp.ts) - sp.nt);
    }
    if (find) break;
    if (bad) report(status, kDevCheck);
    int iu = units, ir = rows, is = segs;
#pragma unroll 1
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(0xffffffffu, iu, o), r = __shfl_up_sync(0xffffffffu, ir, o);
      const int g = __shfl_up_sync(0xffffffffu, is, o);
      if (lane >= o) {
        iu += u;
        ir += r;
        is += g;
      }
    }
    if (lane == 31) {
      sc->warp_units[warp] = iu;
      sc->warp_rows[warp] = ir;
      sc->warp_segs[warp] = is;
    }
    meet();
    base_u = iu - units;
    base_r = ir - rows;
    const int mine_s = segs;
    int base_s = is - segs;
    cut.total = 0;
    segs = 0;
#pragma unroll 1
    for (int x = 0; x < kThreads / 32; ++x) {
      const int u = sc->warp_units[x], g = sc->warp_segs[x];
      if (x < warp) {
        base_u += u;
        base_r += sc->warp_rows[x];
        base_s += g;
      }
      cut.total += u;
      segs += g;
    }
    if (kSnap > 0 && round == 0) {
      const int ctas = list.by_ctas.d;
      if (2 * segs < ctas && cut.total > 0) {
        const int chunk = (cut.total + ctas - segs - 1) / (ctas - segs);
        if (chunk <= list.by_ctas(cut.total) + kSnap) cut.chunk = chunk;
      }
      meet();  // the words above are read before the next round writes them
    }
    // threads without the first unit have no more to do (CTA 0's write the items)
    if (round == 1) {
      const int ctas = list.by_ctas.d;
      if (kSnap == 0 && cut.total > ctas && cut.total + segs >= paged_tile_units<kMaxRows>(6) * ctas) {
        cut.extra = list.extra;
        cut.total += segs;
        base_u += base_s;
        units += mine_s;
      }
      if (thread == 0) {
        sc->cut = cut;
        if (blockIdx.x == 0) {
          list.items[n] = cut.total;
          list.items[n + 1] = cut.chunk > 0 ? cut.chunk : -cut.extra;
        }
      }
      const int first = cut.first(blockIdx.x);
      if (blockIdx.x != 0 && !(units > 0 && base_u <= first && first < base_u + units)) break;
    }
  }
}

// A CTA's walk over its pieces: consecutive key tiles of one segment each.
template <int BN, int kMaxRows>
struct PagedWalk {
  const PagedArgs* p;
  int group_heads, end;
  bool one;  // one piece a CTA
  int i;
  PagedItem it;
  int ts, rt, first, nt;
  int item_row, left, extra;
  int wt, ntp;    // units of a key tile, of a segment
  int skip;       // units of the segment before this CTA's
  int h, ri;      // current piece: KV head, row tile,
  int kt, count;  // first key tile (of the item), tiles

  __device__ __forceinline__ void measure() {
    const PagedSpan<BN, kMaxRows> sp(it, group_heads);
    ts = sp.ts;
    rt = sp.rt;
    first = sp.first;
    nt = sp.nt;
  }
  __device__ __forceinline__ int seg() const { return h * rt + ri; }
  __device__ __forceinline__ int row0() const { return ri << ts; }  // the tile's first row
  __device__ __forceinline__ int rows() const { return (it.t1 - it.t0) * group_heads; }
  // the piece's keys
  __device__ __forceinline__ int key_begin() const { return max((first + kt) * BN, it.lo); }
  __device__ __forceinline__ int key_end() const { return min((first + kt + count) * BN, it.hi); }
  // false: no work for this CTA
  __device__ __forceinline__ bool init(const PagedArgs* args, int gh, const PagedList& list, const PagedScan* sc) {
    p = args;
    group_heads = gh;
    end = list.end;
    const PagedCut& cut = sc->cut;
    const int u0 = cut.first(blockIdx.x);
    left = cut.first(blockIdx.x + 1) - u0;
    if (left <= 0) return false;
    one = cut.chunk > 0;
    i = sc->item;
    it = sc->it;
    item_row = sc->item_row;
    measure();
    extra = cut.extra;
    wt = cut.tile_units<kMaxRows>(ts);
    ntp = cut.padded(nt, wt);
    const int off = u0 - sc->item_unit, s = off / ntp;
    skip = off - s * ntp;
    h = rt == 1 ? s : s / rt;
    ri = s - h * rt;
    kt = tiles(skip);
    count = min(nt, tiles(skip + left)) - kt;
    return count > 0 || next();  // (the first units may be those behind a segment's tiles)
  }
  // key tiles whose first unit is among the segment's first n
  __device__ __forceinline__ int tiles(int n) const {
    return kMaxRows == 64 ? (n + wt - 1) / wt : n;
  }
  __device__ __forceinline__ bool next() {
    left -= ntp - skip;
    if (one || left <= 0) return false;
    kt = 0;
    skip = 0;
    if (++ri == rt) {
      ri = 0;
      if (++h == p->num_kv_heads) {
        h = 0;
        do {
          item_row += p->num_kv_heads * rt << ts;
          if (++i >= end) return false;
          it = paged_item(*p, i);
          measure();
          if (kMaxRows == 64 && extra > 0) wt = paged_tile_units<kMaxRows>(ts);
          ntp = (nt + extra) * wt;
        } while (nt == 0);
      }
    }
    count = min(nt, tiles(left));
    return true;
  }
};

// ---------------------------------------------------------- rows once more
// The kernels take rows together, so a value that a row does not see, or that its
// products cannot take, can still reach its sums: a weight of 0 times a NaN or an
// infinity in V is NaN, and in fp32 the parts of an infinity (or of a number that
// rounds to one) cancel to NaN.  What came out so of a partial is made again for its
// row alone, in plain fp32 products over the keys that the row sees; the rest stays.
// Finite data pays for the check alone (a three-way maximum for two numbers of a
// partial: up to 0.8 us of 39 where a call is all latency).  4 sequences on 14117 fp32
// keys whose queries are NaN, every row made again from L2: 0.59 ms with d 128 and 1.4
// with d 256, against 0.039 and 0.067 finite.

// N consecutive numbers as fp32.
template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&x)[N]) {
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 v = *reinterpret_cast<const float2*>(p + c);
    x[c] = v.x;
    x[c + 1] = v.y;
  }
}
template <int N>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&x)[N]) {
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p + c));
    x[c] = v.x;
    x[c + 1] = v.y;
  }
}
template <int N>
__device__ __forceinline__ void load_row(const __half* p, float (&x)[N]) {
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(p + c));
    x[c] = v.x;
    x[c + 1] = v.y;
  }
}

template <int D>
struct RowAgain {
  float m, l, o[D / 32];  // m: largest logit (log2 units); o: columns lane * D / 32 and on
};

// Query row `q` (its head's first number) over the keys [k0, k1) of a table row and
// KV head, by one warp: a lane has its columns of q, k, v and O, and the logit of one
// of 32 keys.
template <int D, typename T, typename TV>
__device__ __noinline__ RowAgain<D> paged_row_again(const PagedWork& w, int table_row, int h, const T* q, int k0,
                                                    int k1) {
  constexpr int kCols = D / 32;
  const int lane = threadIdx.x & 31;
  const float scale_log2 = w.scale * kLog2e;
  RowAgain<D> r;
  r.m = -INFINITY;
  r.l = 0.f;
  float qx[kCols];
  load_row(q + lane * kCols, qx);
#pragma unroll
  for (int c = 0; c < kCols; ++c) r.o[c] = 0.f;
  const int* table = w.p.block_table + static_cast<long long>(table_row) * w.p.table_stride;
#pragma unroll 1
  for (int kb = k0; kb < k1; kb += 32) {
    const int key = kb + lane, n = min(k1 - kb, 32);
    const int pg = lane < n ? table[key >> w.p.page_shift] : -1;
    long long at = -1;  // the key's first number in the pages; a page outside the cache reads as zeros
    if (static_cast<unsigned>(pg) < static_cast<unsigned>(w.p.num_pages))
      at = pg * w.p.page_stride + (static_cast<long long>(h) * w.p.page_size + (key & (w.p.page_size - 1))) * D;
    float dot = 0.f;  // of this lane's key
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const long long k_at = __shfl_sync(0xffffffffu, at, j);
      float k[kCols], d = 0.f;
      load_row(static_cast<const T*>(w.p.k_pages) + max(k_at, 0ll) + lane * kCols, k);
#pragma unroll
      for (int c = 0; c < kCols; ++c) d = fmaf(qx[c], k_at < 0 ? 0.f : k[c], d);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
      if (lane == j) dot = d;
    }
    const float x = lane < n ? dot * scale_log2 : -INFINITY;
    float top = fmaxf(r.m, x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    const float base = top == -INFINITY ? 0.f : top;
    const float f = ex2_approx(r.m - base), p = ex2_approx(x - base);
    float sum = p;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    r.m = top;
    r.l = fmaf(r.l, f, sum);
#pragma unroll
    for (int c = 0; c < kCols; ++c) r.o[c] *= f;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const long long v_at = __shfl_sync(0xffffffffu, at, j);
      const float pj = __shfl_sync(0xffffffffu, p, j);
      float v[kCols];
      load_row(static_cast<const TV*>(w.p.v_pages) + max(v_at, 0ll) + lane * kCols, v);
#pragma unroll
      for (int c = 0; c < kCols; ++c) r.o[c] = fmaf(pj, v_at < 0 ? 0.f : v[c], r.o[c]);
    }
  }
  return r;
}

// Marks of numbers that are not finite: the largest magnitude, or NaN.
__device__ __forceinline__ float odd_mark(float a, float b, float mark) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(mark));
  return r;
}
__device__ __forceinline__ bool is_odd(float mark) { return !(fabsf(mark) < INFINITY); }

// This lane's columns of a partial that are not finite, from the row made again,
// against the base that the partial's sum of weights has.
template <int D>
__device__ __forceinline__ void put_again(const RowAgain<D>& a, float base, float* o) {
  const float f = base == -INFINITY ? 0.f : ex2_approx(a.m - base);
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    if (is_odd(o[c])) o[c] = a.o[c] * f;
}

// The rows of a piece whose partials in `list` are not finite, by four warps: segment
// of KV head h and first row row0 of item i, `valid` rows, keys [k0, k1) of it, partial
// rows from `part` on.  kAll: every such row, else those that do not see all the keys.
template <int D, typename T, typename TV, bool kAll>
__device__ __noinline__ void paged_rows_again(const PagedWork& w, const PagedList& list, const PagedItem it, int i,
                                              int h, int row0, int valid, int k0, int k1, int part) {
  constexpr int kCols = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gh = w.by_group.d;
#pragma unroll 1
  for (int x = warp; x < valid; x += 4) {
    float* o = list.part_o + static_cast<long long>(part + x) * D + lane * kCols;
    float mark = 0.f;
#pragma unroll
    for (int c = 0; c < kCols; c += 2) mark = odd_mark(o[c], o[c + 1], mark);
    const int r = row0 + x, tr = w.by_group(r), t = it.t0 + tr;
    const int b = i < w.p.num_groups ? paged_seq_of(w.p, t) : it.row;
    const int lim = paged_limit(w.p, b, t);
    if (!__any_sync(0xffffffffu, is_odd(mark)) || lim <= 0 || (!kAll && lim >= k1)) continue;
    const T* q = static_cast<const T*>(w.q) + t * w.q_stride + static_cast<long long>((h - tr) * gh + r) * D;
    const RowAgain<D> a = paged_row_again<D, T, TV>(w, it.row, h, q, k0, min(lim, k1));
    const float2 ml = list.part_ml[part + x];
    if (!is_odd(ml.y)) {  // the weights are right: the columns that are not finite, to their base
      put_again<D>(a, ml.x, o);
    } else {
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[c] = a.o[c];
      __syncwarp();
      if (lane == 0) list.part_ml[part + x] = make_float2(a.m, a.l);
    }
  }
}

}  // namespace dhsa
