// The work list of paged attention, shared by its kernels: items, segments,
// pieces, and where their partial results lie (see PagedWork in serving.h).
#pragma once

#include "common.cuh"
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

constexpr float kLog2e = 1.4426950408889634f;

// Programmatic dependent launch: a call's later kernels are launched while the
// earlier ones run.  `let_next_start` is given by every CTA of a kernel (or by
// its exit); `wait_for_previous` returns when the kernel before has completed
// and its writes are visible.  The prefixes' kernel and the list's kernel read
// the call's inputs only, so the second need not wait for the first to begin,
// but it waits before it ends: its completion then stands for both.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

template <int kMaxRows>
__host__ __device__ __forceinline__ int paged_part_shift(int shift) {
  return kMaxRows == 256 && shift < 8 ? shift + 1 : shift;
}

// An item's segments and key tiles.  Lists whose row tiles reach 256 (the
// prefixes' own, for d 64 and 128) leave two partials of tiles of up to 128 rows.
template <int BN, int kMaxRows>
struct PagedSpan {
  static constexpr int kMax = kMaxRows;
  int rows, ts, rt, first, nt;  // rows; log2 rows a tile, row tiles; first key tile, key tiles
  int ps;                       // log2 rows of a segment's partials
  PagedSpan() = default;
  __device__ __forceinline__ PagedSpan(const PagedItem& it, int group_heads) {
    rows = (it.t1 - it.t0) * group_heads;
    ts = paged_tile_shift<kMaxRows>(rows);
    rt = (rows + (1 << ts) - 1) >> ts;
    ps = paged_part_shift<kMaxRows>(ts);
    first = it.lo / BN;
    nt = it.hi > it.lo && rows > 0 ? (it.hi + BN - 1) / BN - first : 0;
  }
  __device__ __forceinline__ long long units(int num_kv_heads) const {
    return static_cast<long long>(num_kv_heads) * rt * nt;
  }
  __device__ __forceinline__ long long part_rows(int num_kv_heads) const {
    return static_cast<long long>(num_kv_heads) * rt << ps;
  }
};

// First unit (key tile of the whole list) of CTA c, and the CTA that holds a
// unit.  With fewer units than CTAs the first `total` CTAs take one each, so
// every CTA between the first and the last owner of a segment has a partial of it.
__device__ __forceinline__ int paged_ctas(long long total, int ctas) {
  return static_cast<int>(min(total, static_cast<long long>(ctas)));
}
// (Products within 32 bits, the usual case, divide several times faster.)
__device__ __forceinline__ long long paged_divide(long long a, long long b) {
  if ((a | b) >> 32 == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
__device__ __forceinline__ long long paged_first_unit(long long c, long long total, int ctas) {
  const int n = paged_ctas(total, ctas);
  return c < n ? paged_divide(c * total, n) : total;
}
__device__ __forceinline__ int paged_owner(long long unit, long long total, int ctas) {
  return static_cast<int>(paged_divide((unit + 1) * paged_ctas(total, ctas) - 1, total));
}

// Where CTA c's partial of a segment starts (rows): c steps by the largest
// tile, a segment by its own rows, and along the list either c or the segment moves
// on, so no two partials overlap.
__device__ __forceinline__ long long paged_part_row(int c, int max_rows, long long item_row, int seg, int ps) {
  return static_cast<long long>(c) * max_rows + item_row + (static_cast<long long>(seg) << ps);
}

// Shared-memory words of the block-wide scan.
struct PagedScan {
  long long warp_units[32], warp_rows[32];
  long long total, item_unit, item_row;
  int item;
};

// Every CTA counts the units of all items (each thread a run of them) and finds
// the item that holds its first unit.  CTA 0 writes the items' first units and
// rows for the join.  Called by the CTA's last kThreads threads, which meet at
// barrier 1; the result is for the whole CTA after its next __syncthreads.
template <int BN, int kMaxRows, int kThreads>
__device__ __forceinline__ void paged_schedule(const PagedArgs& p, int group_heads, const PagedList& list,
                                               PagedScan* sc, uint32_t* status) {
  const int n = list.end - list.begin;
  const int per = (n + kThreads - 1) / kThreads;
  const int thread = threadIdx.x - (blockDim.x - kThreads);
  const int i0 = min(thread * per, n), i1 = min(i0 + per, n);
  long long units = 0, rows = 0;
  bool bad = false;
  for (int i = i0; i < i1; ++i) {
    const PagedItem it = paged_item(p, list.begin + i);
    const PagedSpan<BN, kMaxRows> sp(it, group_heads);
    units += sp.units(p.num_kv_heads);
    rows += sp.part_rows(p.num_kv_heads);
    if (blockIdx.x == 0) {
      const int g = list.begin + i;
      if (g < p.num_groups) {
        bad |= it.t1 > it.t0 && p.prefix_lens[g] != paged_clamp_len(p, p.prefix_lens[g]);
      } else {
        bad |= p.kv_lens[g - p.num_groups] != it.hi;
      }
    }
  }
  if (bad) report(status, kDevCheck);
  const int lane = thread & 31, warp = thread >> 5;
  long long iu = units, ir = rows;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long u = __shfl_up_sync(0xffffffffu, iu, o), r = __shfl_up_sync(0xffffffffu, ir, o);
    if (lane >= o) {
      iu += u;
      ir += r;
    }
  }
  if (lane == 31) {
    sc->warp_units[warp] = iu;
    sc->warp_rows[warp] = ir;
  }
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
  long long base_u = iu - units, base_r = ir - rows, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long u = sc->warp_units[w];
    if (w < warp) {
      base_u += u;
      base_r += sc->warp_rows[w];
    }
    total += u;
  }
  const long long mine = paged_first_unit(blockIdx.x, total, gridDim.x);
  if (thread == 0) sc->total = total;
  const bool find = units > 0 && base_u <= mine && mine < base_u + units;
  if (find || blockIdx.x == 0) {
    long long u = base_u, r = base_r;
    for (int i = i0; i < i1; ++i) {
      const PagedItem it = paged_item(p, list.begin + i);
      const PagedSpan<BN, kMaxRows> sp(it, group_heads);
      const long long du = sp.units(p.num_kv_heads);
      if (du > 0 && u <= mine && mine < u + du) {
        sc->item = list.begin + i;
        sc->item_unit = u;
        sc->item_row = r;
      }
      if (blockIdx.x == 0) {
        list.items[i] = u;
        list.items[n + 1 + i] = r;
      }
      u += du;
      r += sp.part_rows(p.num_kv_heads);
    }
  }
  if (blockIdx.x == 0 && thread == 0) list.items[n] = total;
}

// A CTA's walk over its pieces: consecutive key tiles of one segment each.
template <int BN, int kMaxRows>
struct PagedWalk {
  const PagedArgs* p;
  int group_heads, end;
  int i;
  PagedItem it;
  int ts, ps, rt, first, nt;
  long long item_row, left;
  int h, ri;      // current piece: KV head, row tile,
  int kt, count;  // first key tile (of the item), tiles

  __device__ __forceinline__ void load() {
    it = paged_item(*p, i);
    const PagedSpan<BN, kMaxRows> sp(it, group_heads);
    ts = sp.ts;
    ps = sp.ps;
    rt = sp.rt;
    first = sp.first;
    nt = sp.nt;
  }
  __device__ __forceinline__ int seg() const { return h * rt + ri; }
  __device__ __forceinline__ int row0() const { return ri << ts; }  // the tile's first row
  __device__ __forceinline__ int rows() const { return (it.t1 - it.t0) * group_heads; }
  // false: no work for this CTA
  __device__ __forceinline__ bool init(const PagedArgs* args, int gh, const PagedList& list, const PagedScan* sc) {
    p = args;
    group_heads = gh;
    end = list.end;
    const long long u0 = paged_first_unit(blockIdx.x, sc->total, gridDim.x);
    left = paged_first_unit(blockIdx.x + 1, sc->total, gridDim.x) - u0;
    if (left <= 0) return false;
    i = sc->item;
    item_row = sc->item_row;
    load();
    const long long off = u0 - sc->item_unit;
    const int s = static_cast<int>(paged_divide(off, nt));
    kt = static_cast<int>(off - static_cast<long long>(s) * nt);
    h = rt == 1 ? s : s / rt;
    ri = s - h * rt;
    count = static_cast<int>(min(static_cast<long long>(nt - kt), left));
    return true;
  }
  __device__ __forceinline__ bool next() {
    left -= count;
    if (left <= 0) return false;
    kt = 0;
    if (++ri == rt) {
      ri = 0;
      if (++h == p->num_kv_heads) {
        h = 0;
        do {
          item_row += static_cast<long long>(p->num_kv_heads) * rt << ps;
          if (++i >= end) return false;
          load();
        } while (nt == 0);
      }
    }
    count = static_cast<int>(min(static_cast<long long>(nt), left));
    return true;
  }
};

}  // namespace dhsa
