// The shared prefixes of paged attention on tcgen05 tensor cores (bf16): the
// query rows of all the sequences of a group, up to 128 at a time, against the
// prefix's keys, each key tile brought from its pages once for the tile of rows.
//
// A CTA works on pieces of the prefixes' list (see PagedWork): consecutive
// 128-key tiles of one (group, KV head, row tile), and leaves each piece's
// (O unnormalised, running max, sum) for the join.  Per 128 rows and key tile
//   S = Q K^T       tcgen05.mma, 128 x 128, into TMEM;
//   P = exp2(S - m) by four softmax warps, a thread a row, written as f16 over
//                   S's own columns;
//   O += P V        tcgen05.mma with A from TMEM, V as stored (f16).
// That chain has nothing of its own to overlap, so a CTA runs two of them, its
// lanes, each with its own softmax warpgroup, S, O and issuing thread: the
// tensor core works for one while the other's softmax runs.  A row tile of more
// than 128 rows gives each lane half of them and every key tile feeds both; with
// 128 rows or fewer, where the call is bound by reading keys, both lanes have
// the same rows and take every other key tile, and join when the piece ends.  K and V
// tiles come into rings of 2 and 3 (4 and 4 for d 64).  P is handed over in two
// halves of 64 keys, so the first half's products run beside the second half's
// exponentials.  d 256 has TMEM and shared memory for one lane, with key tiles of
// 64 in the same rings: S of the next tile then runs beside this tile's softmax, and
// loads are in flight all the time (32 answers to 32000 tokens: a call of 82 us
// against 106 with key tiles of 128 in rings of one).
//
// The two issuing threads take turns, a tile's P V and the next S to a turn:
// with MMAs of both lanes mixed, one by one, a call of 64 answers to 128K tokens
// took 244 us instead of 211.
//
// Measured: 64 answers (256 rows) to 128K tokens, 8 KV heads of 128: 137 GFLOP
// in about 140 us, 0.98 PFLOP/s (0.6 of the measured matrix rate): 2.25 us for
// 256 rows x 128 keys on an SM, of which the exponentials of 2^15 weights, 16 a
// cycle, are half.  With 128 rows (32 answers to 32K tokens) both lanes' two key
// tiles, 131 KB, take 2.9 us: 6.5 TB/s over all SMs (0.99 of the measured copy
// rate) between the kernel's start and its end.
//
// Warp roles: a warpgroup for each lane's softmax, epilogue and Q (cp.async);
// then a warpgroup of the producer of K tiles (TMA, a lane for each page part
// and 64-column slice), a warp for each lane's MMAs, and the producer of V tiles.
#include "launchers.h"
#include "paged.cuh"

namespace dhsa {
namespace {

constexpr int kBM = 128;  // rows of a lane's tile
// O is rescaled only when a row's maximum grew by more than 2^4 since the last
// time, so that most tiles skip the pass over O: the largest weight is 2^11 when
// the base is set and 2^15 before it moves (see weight_base).  The slack costs range
// below; with 2^8 / 2^4 / 2^2 / 2^1 a call of 64 answers to 128K tokens takes 189.4 /
// 191.0 / 192.6 / 194.2 us, others the same within their noise.
constexpr float kRescaleLog2 = 4.0f;
constexpr float kLift = kTopLog2 - kRescaleLog2;

// A lane's two 32-bit columns, stored and loaded.
__device__ __forceinline__ void tmem_st2(uint32_t taddr, uint32_t x, uint32_t y) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void tmem_ld2(uint32_t taddr, uint32_t& x, uint32_t& y) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x), "=r"(y)
      : "r"(taddr)
      : "memory");
}

// Eight fp32 numbers of a row, a whole 32-byte sector, in one store.
__device__ __forceinline__ void store_row8(float* dst, const uint32_t* o) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(o[0]), "r"(o[1]), "r"(o[2]),
               "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
               : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A warp's rows (a lane each) marked `mine`, where the `cols` columns of their partial
// at dst, from col0 on, are not finite: made again for the keys [k0, k1) that each sees,
// against the base that the row's stored sum has.
template <int D>
__device__ __noinline__ void short_rows_again(const PagedWork& w, bool mine, const __nv_bfloat16* q, float* dst,
                                              int col0, int cols, float base, int table_row, int h, int k0, int k1) {
  constexpr int kCols = D / 32;
  const int lane = threadIdx.x & 31;
  const bool own = lane * kCols >= col0 && lane * kCols < col0 + cols;
  __syncwarp();  // the rows' stores, read and written here by other lanes
  uint32_t rows = __ballot_sync(0xffffffffu, mine);
#pragma unroll 1
  for (; rows != 0u; rows &= rows - 1u) {
    const int src = __ffs(rows) - 1;
    float* o = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), src)) +
               lane * kCols;
    const auto* q_row = reinterpret_cast<const __nv_bfloat16*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(q), src));
    const int end = __shfl_sync(0xffffffffu, k1, src);
    const float to = __shfl_sync(0xffffffffu, base, src);
    float mark = 0.f;
    if (own) {
#pragma unroll
      for (int c = 0; c < kCols; c += 2) mark = odd_mark(o[c], o[c + 1], mark);
    }
    if (!__any_sync(0xffffffffu, is_odd(mark))) continue;
    const RowAgain<D> r = paged_row_again<D, __nv_bfloat16, __half>(w, table_row, h, q_row, k0, end);
    if (own) put_again<D>(r, to, o);
  }
  __syncwarp();
}

enum {
  kBarKFull = 0,    // + stage
  kBarVFull = 4,    // + stage
  kBarKFree = 8,    // + stage: S of the tile done (one commit a lane, or two of one lane)
  kBarVFree = 12,   // + stage: P V of the tile done
  kBarSFull = 16,   // + lane
  kBarPHalf = 18,   // + lane: first 64 keys of P written, O rescaled
  kBarPFull = 20,   // + lane
  kBarQFull = 22,   // + lane: a piece's Q in shared memory
  kBarODone = 24,   // + lane: a piece's last P V done
  kBarDrain = 26,   // + lane
  kBarTurn = 28,    // + lane: that lane's thread ended a turn
  kBarCross = 30,   // + lane: its (m, l) is in TMEM and its O complete
  kBarPiece = 32,   // both lanes have read a piece's results
  kNumBars = 33
};

// A second piece costs a CTA about as much as this many key tiles (8 us of
// epilogue, Q and first tiles against 1.5 to 2 us a tile).
constexpr int kSnapTiles = 4;

template <int D>
struct PrefixCfg {
  static constexpr int kBN = paged_prefix_keys(D);
  static constexpr int kLanes = D == 256 ? 1 : 2;
  static constexpr int kRows = paged_prefix_rows(D);  // of a row tile
  static constexpr int kThreads = 128 * (kLanes + 1);
  static constexpr int kProducer = 4 * kLanes;
  static constexpr int kMma = kProducer + 1;  // + lane
  static constexpr int kProducerV = kProducer + 3;
  static constexpr int kKStages = D == 64 ? 4 : 2;
  static constexpr int kVStages = D == 64 ? 4 : 3;
  static constexpr int kSlices = D / 64;
  static constexpr int kSub = kBN * 128;  // one 64-column slice of a tile
  static constexpr int kTile = kSlices * kSub;
  static constexpr int kSubQ = kBM * 128;
  static constexpr int kTileQ = kSlices * kSubQ;
  static constexpr int kOffQ = 0;  // + lane
  static constexpr int kOffK = kLanes * kTileQ;
  static constexpr int kOffV = kOffK + kKStages * kTile;
  static constexpr int kOffScan = kOffV + kVStages * kTile;
  static constexpr int kOffBar = kOffScan + ((static_cast<int>(sizeof(PagedScan)) + 15) / 16) * 16;
  static constexpr int kSmemBytes = kOffBar + 8 * kNumBars + 16 + 1024;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0;         // + kBN * (lane, or the tile's parity with one lane)
  static constexpr uint32_t kColO = 2 * kBN;   // + D * lane
  static_assert(2 * kBN + kLanes * D <= 512, "TMEM budget");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(PrefixCfg<D>::kThreads, 1)
    paged_prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedWork w) {
  using C = PrefixCfg<D>;
  constexpr int kBN = C::kBN;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kOffBar;
  auto bar = [&](int idx) { return bar0 + 8u * static_cast<uint32_t>(idx); };
  int* misc = reinterpret_cast<int*>(smem + C::kOffBar + 8 * kNumBars);  // TMEM base, abort flag
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  PagedScan* sc = reinterpret_cast<PagedScan*>(smem + C::kOffScan);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gh = w.by_group.d;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(kBarKFull + s), 1);
      mbar_init(bar(kBarVFull + s), 1);
      mbar_init(bar(kBarKFree + s), C::kLanes);
      mbar_init(bar(kBarVFree + s), C::kLanes);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar(kBarSFull + a), 1);
      mbar_init(bar(kBarPHalf + a), 4);  // one arrival per softmax warp
      mbar_init(bar(kBarPFull + a), 4);
      mbar_init(bar(kBarQFull + a), 4);
      mbar_init(bar(kBarODone + a), 1);
      mbar_init(bar(kBarDrain + a), 1);
      mbar_init(bar(kBarTurn + a), 1);
      mbar_init(bar(kBarCross + a), 4);
    }
    mbar_init(bar(kBarPiece), 4 * C::kLanes);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kMma) {
    tmem_alloc(smem_u32(misc), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  PagedWalk<kBN, C::kRows> walk{};
  // Two lanes on one set of rows take every other key tile of a piece
  // (`apart`): lane a's tiles are a, a + 2, ...; otherwise every one.
  auto apart = [&]() -> bool { return C::kLanes == 2 && walk.ts < 8; };
  // The S and P of a lane's tile n, counted across pieces: two lanes have a place
  // and barriers each, one lane takes two by turns (S of the next tile is done
  // before P V of this one is sent, and neither side gets two tiles ahead on one).
  auto p_bar = [](int a, int n) { return C::kLanes == 2 ? a : n & 1; };
  auto p_phase = [](int n) { return static_cast<uint32_t>((C::kLanes == 2 ? n : n >> 1) & 1); };

  if (warp >= C::kProducer) {
    // 8 warps x 224 + 4 x 56 registers = the launch's 12 x 168
    if constexpr (C::kLanes == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // this warpgroup lays out the CTA's work while the softmax warps warm up
    wait_for_previous();
    paged_schedule<kBN, C::kRows, 128, kSnapTiles>(w.p, gh, w.prefix, sc, w.status);
    let_next_start();
    __syncthreads();
    const bool work = walk.init(&w.p, gh, w.prefix, sc);
    if (work && (warp == C::kProducer || warp == C::kProducerV)) {
      // ------------------------------------------------- K and V producers
      // a lane for each box of a tile: (page part, 64-column slice)
      const bool is_k = warp == C::kProducer;
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      const int full = is_k ? kBarKFull : kBarVFull, free = is_k ? kBarKFree : kBarVFree;
      const int stages = is_k ? C::kKStages : C::kVStages;
      const int ps = w.p.page_size, psh = w.p.page_shift;
      const int box = ps < kBN ? ps : kBN;
      const int sl = lane % C::kSlices, pp = lane / C::kSlices;
      const bool mine = pp * box < kBN;
      const uint32_t dst0 = sbase + (is_k ? C::kOffK : C::kOffV) + sl * C::kSub + pp * box * 128;
      int slot = 0, round = 0, issued = 0;
      bool ok = true;
      do {
        const int h = walk.h;
        const int* table = w.p.block_table + static_cast<long long>(walk.it.row) * w.p.table_stride;
        auto page_at = [&](int kt) -> int {
          const int key = (walk.first + walk.kt + kt) * kBN + pp * box;
          if (kt >= walk.count || !mine || key >= walk.it.hi) return -1;
          const int pg = table[key >> psh];
          if (static_cast<unsigned>(pg) < static_cast<unsigned>(w.p.num_pages)) return pg;
          report(w.status, kDevCheck);
          return w.p.num_pages;  // outside the map: the box arrives as zeros
        };
        int page = page_at(0);
        for (int kt = 0; kt < walk.count; ++kt) {
          const int page_next = page_at(kt + 1);
          const unsigned bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * box * 128;
          const int in_page = ((walk.first + walk.kt + kt) * kBN + pp * box) & (ps - 1);
          if (round > 0) ok = paged_wait_warp(bar(free + slot), (round - 1) & 1, abort_flag);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(full + slot), bytes);
          __syncwarp();
          if (page >= 0) tma_load_4d(dst0 + slot * C::kTile, map, bar(full + slot), sl * 64, in_page, h, page);
          ++issued;
          page = page_next;
          if (++slot == stages) {
            slot = 0;
            ++round;
          }
        }
      } while (ok && walk.next());
      if (*abort_flag && lane == 0) {
        // let copies already in flight land before the CTA exits (bounded)
        volatile int never = 0;
        for (int x = max(0, issued - stages); x < issued; ++x)
          mbar_wait(bar(full + x % stages), (x / stages) & 1, &never, nullptr, 10000000ull);
      }
    } else if (work && warp < C::kMma + C::kLanes) {
      // ------------------------------------------------------------- MMA
      if (lane == 0) {
        const int a = warp - C::kMma;
        constexpr uint32_t idesc_s = idesc_bf16_f32(kBM, kBN, 0);
        constexpr uint32_t idesc_o = idesc_f16_f32(kBM, D, 1);  // P and V in f16
        const uint32_t tS0 = tmem + C::kColS, tO = tmem + C::kColO + D * a;
        const uint32_t qbase = sbase + C::kOffQ + a * C::kTileQ;
        // turn x (counted across pieces): lane 1 waits for lane 0's turn x, lane 0 for lane 1's turn x - 1
        auto wait_turn = [&](int x) -> bool {
          if (C::kLanes == 1) return true;
          if (a == 1) return paged_wait_spin(bar(kBarTurn + 0), x & 1, abort_flag);
          return x == 0 || paged_wait_spin(bar(kBarTurn + 1), (x - 1) & 1, abort_flag);
        };
        auto end_turn = [&]() {
          if (C::kLanes == 2) mbar_arrive(bar(kBarTurn + a));
        };
        // a tile's slot is free for reloading once this lane's products on it
        // are done (a lane on its own tiles stands for the other one, too)
        auto release = [&](int idx, bool ap) {
          umma_commit(bar(idx));
          if (ap) umma_commit(bar(idx));
        };
        int n0 = 0, mine = 0, piece = 0, turn = 0;  // key tiles, this lane's tiles: across pieces
        bool ok = true;
        do {
          const bool ap = apart();
          const int step = ap ? 2 : 1, kt0 = ap ? a : 0;
          // one turn for the first S, then one for each of the tiles (of the lane that has more)
          const int turns = 1 + (ap ? (walk.count + 1) / 2 : walk.count);
          ok = paged_wait(bar(kBarQFull + a), piece & 1, abort_flag);
          // turn x: P V of the lane's tile x - 1 and S of its tile x
          for (int x = 0; ok && x < turns; ++x, ++turn) {
            const int kt = kt0 + (x - 1) * step;  // of P V
            const bool pv = x > 0 && kt < walk.count, sn = kt + step < walk.count;
            const int np = n0 + kt, ns = np + step;
            const int vs = np % C::kVStages, ks = ns % C::kKStages;
            auto k_there = [&]() {
              return paged_wait_spin(bar(kBarKFull + ks), (ns / C::kKStages) & 1, abort_flag);
            };
            auto p_there = [&]() {
              return paged_wait_spin(bar(kBarVFull + vs), (np / C::kVStages) & 1, abort_flag) &&
                     paged_wait_spin(bar(kBarPHalf + p_bar(a, mine)), p_phase(mine), abort_flag);
            };
            auto send_s = [&]() {
              const uint32_t kbase = sbase + C::kOffK + ks * C::kTile, tS = tS0 + kBN * p_bar(a, ns);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t so = (kk >> 2) * C::kSubQ + (kk & 3) * 32, ko = (kk >> 2) * C::kSub + (kk & 3) * 32;
                umma_f16_ss(tS, smem_desc_sw128(qbase + so, 16, 1024), smem_desc_sw128(kbase + ko, 16, 1024),
                            idesc_s, kk > 0 ? 1u : 0u);
              }
              umma_commit(bar(kBarSFull + p_bar(a, ns)));
            };
            auto send_pv = [&]() -> bool {
              const uint32_t vbase = sbase + C::kOffV + vs * C::kTile, tP = tS0 + kBN * p_bar(a, mine);
#pragma unroll
              for (int kk = 0; kk < kBN / 16; ++kk) {
                if (kk == kBN / 32) {
                  if (!paged_wait_spin(bar(kBarPFull + p_bar(a, mine)), p_phase(mine), abort_flag))
                    return false;
                  tc_fence_after();
                }
                umma_f16_ts(tO, tP + kk * 8, smem_desc_sw128(vbase + kk * 16 * 128, C::kSub, 1024), idesc_o,
                            (x > 1 || kk > 0) ? 1u : 0u);
              }
              ++mine;
              return true;
            };
            if constexpr (C::kLanes == 2) {
              if (pv && !(ok = p_there())) break;
              if (sn && !(ok = k_there())) break;
              if (!(ok = wait_turn(turn))) break;
              tc_fence_after();
              if (pv && !(ok = send_pv())) break;
              // S over the columns that these products read as P: the tensor core takes them in order
              if (sn) send_s();
            } else {
              // S into the other of two places first: it is done before this tile's softmax is
              if (sn) {
                if (!(ok = k_there())) break;
                tc_fence_after();
                send_s();
                umma_commit(bar(kBarKFree + ks));
              }
              if (pv) {
                if (!(ok = p_there())) break;
                tc_fence_after();
                if (!(ok = send_pv())) break;
              }
            }
            end_turn();
            if (C::kLanes == 2 && sn) release(kBarKFree + ks, ap);
            if (pv) {
              if (!sn) umma_commit(bar(kBarODone + a));
              release(kBarVFree + vs, ap);
            }
          }
          n0 += walk.count;
          ++piece;
        } while (ok && walk.next());
        // every MMA issued above completes before TMEM is released
        umma_commit(bar(kBarDrain + a));
        volatile int never = 0;
        mbar_wait(bar(kBarDrain + a), 0, &never, nullptr);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    if constexpr (C::kLanes == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int a = warp >> 2;            // the lane
    const int row = threadIdx.x & 127;  // the TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS0 = tmem + lane_base + C::kColS, tO = tmem + lane_base + C::kColO + D * a;
    const float scale_log2 = w.scale * kLog2e;
    // key tiles and this lane's tiles; pieces, those in which lane 1 has a tile, those with lanes apart: so far
    int n0 = 0, mine = 0, done[2] = {0, 0}, joins = 0;
    bool ok = true;
    // The first round is a rehearsal: the code below comes a cache line at a
    // time from L2 the first time that it runs (6 us for a tile's softmax,
    // against 1.2 us later), which is over before the first S is there when it
    // is spent on whatever TMEM holds while the work is laid out and K and Q
    // are on their way.  Nothing of it is kept.
    bool rehearsal = true;
    int kt0 = 0, step = 1, count = 1, in_tile = 0, lim = INT_MAX, hi = INT_MAX, first = 0;
    bool ap = false, valid = false, warp_valid = true;
    // Sends for a piece's Q (16 bytes a copy, a row's copies next to each
    // other, rows without a query zero): its arrival is waited for by land_q.
    // The lane's last S of the piece before is done by then.
    auto send_q = [&](const PagedWalk<kBN, C::kRows>& k) {
      const int tile_row = C::kLanes == 2 && k.ts < 8 ? row : a * kBM + row;
      const int r = k.row0() + tile_row;
      long long off = -1;
      if (tile_row >> k.ts == 0 && r < k.rows()) {
        const int tr = w.by_group(r);
        off = (k.it.t0 + tr) * w.q_stride + static_cast<long long>((k.h - tr) * gh + r) * D;
      }
      constexpr int kVecs = D / 8, kPer = 32 / kVecs;  // copies of a row, rows a step
      const int c = lane % kVecs;
#pragma unroll 4
      for (int i = 0; i < kVecs; ++i) {
        const int src = kPer > 0 ? i * kPer + lane / kVecs : i;
        const long long o = __shfl_sync(0xffffffffu, off, src);
        const int rr = (warp & 3) * 32 + src;
        cp_async16(sbase + C::kOffQ + a * C::kTileQ + (c >> 3) * C::kSubQ + rr * 128 + (((c & 7) ^ (rr & 7)) << 4),
                   static_cast<const __nv_bfloat16*>(w.q) + (o < 0 ? 0 : o + 8 * c), o >= 0);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto land_q = [&]() {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarQFull + a));
    };
    do {
      if (!rehearsal) {
        ap = apart();
        step = ap ? 2 : 1;
        kt0 = ap ? a : 0;
        count = walk.count;
        first = walk.first + walk.kt;
        hi = walk.it.hi;
        in_tile = ap ? row : a * kBM + row;
        const int r = walk.row0() + in_tile;
        valid = in_tile >> walk.ts == 0 && r < walk.rows();
        warp_valid = __any_sync(0xffffffffu, valid);
        lim = 0;
        if (valid) {
          const int t = walk.it.t0 + w.by_group(r);
          lim = min(hi, paged_limit(w.p, paged_seq_of(w.p, t), t));
        }
        land_q();
      }
      float m_run = -INFINITY;  // base of the weights, see weight_base
      float l_run = 0.f;
      for (int kt = kt0; kt < count; kt += step) {
        const int k0 = (first + kt) * kBN, pb = p_bar(a, mine);
        const uint32_t tS = tS0 + kBN * pb;
        if (!rehearsal) {
          if (!(ok = paged_wait_warp(bar(kBarSFull + pb), p_phase(mine), abort_flag))) break;
          ++mine;
          tc_fence_after();
          if (k0 + kBN > hi) {
            // slots behind the prefix may hold anything, NaN included, and 0 *
            // NaN is NaN: V's rows there are zeroed (a thread a row; lanes that share
            // the tile write the same zeros)
            const int n = n0 + kt, s = n % C::kVStages;
            if (!(ok = paged_wait_warp(bar(kBarVFull + s), (n / C::kVStages) & 1, abort_flag))) break;
            if (row < kBN && k0 + row >= hi) {
#pragma unroll 1
              for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4*>(smem + C::kOffV + s * C::kTile + (c >> 3) * C::kSub + row * 128 +
                                          ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();  // before this warp's arrival on PHalf, which takes all four
          }
          if (!warp_valid) {  // no row of this warp counts: its P may be anything
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(kBarPHalf + pb));
              mbar_arrive(bar(kBarPFull + pb));
            }
            continue;
          }
        }
        float s[kBN];
        float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const int cols = lim - k0;  // valid columns: c < cols
        auto take = [&](int base, uint32_t (&ra)[32], uint32_t (&rb)[32]) {  // 64 columns
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            s[base + e] = __uint_as_float(ra[e]);
            s[base + 32 + e] = __uint_as_float(rb[e]);
          }
          if (cols < base + 64) {
#pragma unroll
            for (int c = base; c < base + 64; ++c)
              if (c >= cols) s[c] = -INFINITY;
          }
#pragma unroll
          for (int c = base; c < base + 64; c += 8) {
#pragma unroll
            for (int x = 0; x < 4; ++x) mp[x] = fmax3(mp[x], s[c + x], s[c + 4 + x]);
          }
        };
        {
          uint32_t ra[32], rb[32], rc[32], rd[32];
          tmem_ld32(tS + 0, ra);
          tmem_ld32(tS + 32, rb);
          tmem_wait_ld();
          reg_dep32(ra);
          reg_dep32(rb);
          if constexpr (kBN == 128) {
            tmem_ld32(tS + 64, rc);
            tmem_ld32(tS + 96, rd);
          }
          take(0, ra, rb);
          if constexpr (kBN == 128) {
            tmem_wait_ld();
            reg_dep32(rc);
            reg_dep32(rd);
            take(64, rc, rd);
          }
        }
        // m_run is the base: this tile's largest weight is 2^(tile_base + kLift - m_run)
        const float tile_base =
            weight_base(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])), scale_log2, kLift);
        const bool any = __any_sync(0xffffffffu, tile_base - m_run > kRescaleLog2);
        float alpha = 1.f;
        if (any) {
          const float m_new = fmaxf(m_run, tile_base);
          alpha = m_new == -INFINITY ? 1.f : ex2_approx(m_run - m_new);
          m_run = m_new;
        }
        const float m_use = m_run == -INFINITY ? 0.f : m_run;
        uint64_t ps2[2] = {0ull, 0ull};
        const uint64_t scale2 = f2_pack(scale_log2, scale_log2);
        const uint64_t shift2 = f2_pack(-m_use, -m_use);
        // P of half of the columns, cb and up, over the TMEM columns cb / 2 .. (S is in registers)
        auto exp_cols = [&](int cb) {
#pragma unroll
          for (int q = cb; q < cb + kBN / 2; q += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(s[q + c], s[q + c + 1]), scale2, shift2), x0, x1);
              const float e0 = ex2_approx(x0);
              const float e1 = ex2_approx(x1);
              ps2[(c / 2) & 1] = f2_add(ps2[(c / 2) & 1], f2_pack(e0, e1));
              pk[c / 2] = pack_f16(e0, e1);
            }
            tmem_st16(tS + q / 2, pk);
          }
        };
        exp_cols(0);
        if (any && (kt > kt0 || rehearsal)) {
          // O is rescaled before this tile's products; the last tile's are
          // done, since this S was issued after them (with one lane: waited for)
          if (C::kLanes == 1 && !rehearsal) {
            const int n = n0 + kt - 1;
            ok = paged_wait_warp(bar(kBarVFree + n % C::kVStages), (n / C::kVStages) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
          }
          const uint64_t alpha2 = f2_pack(alpha, alpha);
#pragma unroll 1
          for (int c = 0; c < D / 32; c += 2) {
            uint32_t o0[32], o1[32];
            tmem_ld32(tO + 32 * c, o0);
            tmem_ld32(tO + 32 * (c + 1), o1);
            tmem_wait_ld();
            reg_dep32(o0);
            reg_dep32(o1);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(o0[e]), __uint_as_float(o0[e + 1])), alpha2), x0, x1);
              o0[e] = __float_as_uint(x0);
              o0[e + 1] = __float_as_uint(x1);
              f2_unpack(f2_mul(f2_pack(__uint_as_float(o1[e]), __uint_as_float(o1[e + 1])), alpha2), x0, x1);
              o1[e] = __float_as_uint(x0);
              o1[e + 1] = __float_as_uint(x1);
            }
            tmem_st32(tO + 32 * c, o0);
            tmem_st32(tO + 32 * (c + 1), o1);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !rehearsal) mbar_arrive(bar(kBarPHalf + pb));
        exp_cols(kBN / 2);
        {
          float a0, a1, b0, b1;
          f2_unpack(ps2[0], a0, a1);
          f2_unpack(ps2[1], b0, b1);
          l_run = l_run * alpha + ((a0 + a1) + (b0 + b1));
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !rehearsal) mbar_arrive(bar(kBarPFull + pb));
      }
      if (!ok) break;
      if (rehearsal) {
        rehearsal = false;
        wait_for_previous();
        __syncthreads();  // the schedule is there; what the rehearsal wrote to TMEM is behind tc_fence_before
        if (!walk.init(&w.p, gh, w.prefix, sc)) break;
        send_q(walk);
        continue;
      }
      const int part = paged_part_row(blockIdx.x, C::kRows, walk.item_row, walk.seg(), walk.ts) + in_tile;
      float* dst = w.prefix.part_o + static_cast<long long>(part) * D;
      // rows that do not see all of the piece's keys may have met values that are not theirs: what
      // making them again takes (see paged_rows_again)
      const int key_begin = walk.key_begin(), key_end = walk.key_end(), table_row = walk.it.row, head = walk.h;
      const bool short_row = valid && lim > 0 && lim < key_end;
      const __nv_bfloat16* q_row = nullptr;
      if (short_row) {
        const int r = walk.row0() + in_tile, tr = w.by_group(r);
        q_row = static_cast<const __nv_bfloat16*>(w.q) + (walk.it.t0 + tr) * w.q_stride +
                static_cast<long long>((head - tr) * gh + r) * D;
      }
      const bool some = kt0 < count;  // lanes apart: lane 1 has no tile in a piece of one
      const bool more = walk.next();
      if (more) send_q(walk);
      if (some) {
        if (!(ok = paged_wait_warp(bar(kBarODone + a), done[a] & 1, abort_flag))) break;
        tc_fence_after();
      }
      if (!ap) {
        if (warp_valid) {
          if (valid) w.prefix.part_ml[part] = make_float2(m_run, l_run);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
            reg_dep32(o);
            if (valid) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) store_row8(dst + 32 * c + e, o + e);
            }
          }
          if (__any_sync(0xffffffffu, short_row))
            short_rows_again<D>(w, short_row, q_row, dst, 0, D, m_run, table_row, head, key_begin, min(lim, key_end));
          tc_fence_before();  // the next piece's P V overwrites O after this warp's next arrival
        }
      } else {
        // Lanes apart: their results of a row join here, each lane finishing
        // half of the columns.  A thread of either lane sees the row's both O in
        // TMEM; (m, l) cross over there, too, in columns that P has left.
        tmem_st2(tS0 + kBN * a, __float_as_uint(m_run), __float_as_uint(l_run));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarCross + a));
        if (!(ok = paged_wait_warp(bar(kBarCross + 1 - a), joins & 1, abort_flag))) break;
        tc_fence_after();
        if (warp_valid) {
          uint32_t xm, xl;
          tmem_ld2(tS0 + kBN * (1 - a), xm, xl);
          const float om = __uint_as_float(xm), ol = __uint_as_float(xl);
          const float top = fmaxf(m_run, om);
          const float base = top == -INFINITY ? 0.f : top;
          const float f = ex2_approx(m_run - base), g = ex2_approx(om - base);
          const float f0 = a == 0 ? f : g, f1 = a == 0 ? g : f;  // of lane 0's and lane 1's O
          const bool both = count > 1;
          if (valid && a == 0) w.prefix.part_ml[part] = make_float2(top, fmaf(l_run, f, ol * g));
          constexpr int kHalf = D / 2;
#pragma unroll 1
          for (int c = 0; c < kHalf / 32; ++c) {
            uint32_t o0[32], o1[32];
            const uint32_t at = tmem + lane_base + C::kColO + a * kHalf + 32 * c;
            tmem_ld32(at, o0);
            tmem_ld32(at + D, o1);
            tmem_wait_ld();
            reg_dep32(o0);
            reg_dep32(o1);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o0[e] = __float_as_uint(
                  fmaf(__uint_as_float(o0[e]), f0, both ? __uint_as_float(o1[e]) * f1 : 0.f));
            if (valid) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) store_row8(dst + a * kHalf + 32 * c + e, o0 + e);
            }
          }
          if (__any_sync(0xffffffffu, short_row))
            short_rows_again<D>(w, short_row, q_row, dst, a * kHalf, kHalf, top, table_row, head, key_begin,
                                min(lim, key_end));
          tc_fence_before();
        }
        ++joins;
      }
      if constexpr (C::kLanes == 2) {
        if (!more) break;
        // no product of the next piece starts before both lanes have read TMEM
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPiece));
        if (!(ok = paged_wait_warp(bar(kBarPiece), (done[0]) & 1, abort_flag))) break;
      } else {
        if (!more) break;
      }
      // lane 0 has a tile in every piece
      ++done[0];
      if (!ap || count > 1) ++done[1];
      n0 += count;
    } while (true);
    asm volatile("cp.async.wait_all;" ::: "memory");  // (a Q sent for and not landed, where a wait gave up)
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMma) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0) report_abort(abort_flag, w.status);
}

template <int D>
cudaError_t run(const PagedWork& w, cudaStream_t stream) {
  using C = PrefixCfg<D>;
  CUtensorMap mk, mv;
  if (encode_pages_map(&mk, w.p.k_pages, w.p, C::kBN, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) != CUDA_SUCCESS ||
      encode_pages_map(&mv, w.p.v_pages, w.p, C::kBN, CU_TENSOR_MAP_DATA_TYPE_FLOAT16) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaError_t e =
      cudaFuncSetAttribute(paged_prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_early(paged_prefix_kernel<D>, w.prefix.by_ctas.d, C::kThreads, C::kSmemBytes, stream, mk, mv, w);
}

}  // namespace

cudaError_t launch_paged_prefix(const PagedWork& w, cudaStream_t stream) {
  switch (w.p.head_dim) {
    case 64: return run<64>(w, stream);
    case 128: return run<128>(w, stream);
    default: return run<256>(w, stream);
  }
}

}  // namespace dhsa
