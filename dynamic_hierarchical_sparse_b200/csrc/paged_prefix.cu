// The shared prefixes of paged attention on tcgen05 tensor cores (bf16): the
// query rows of all the sequences of a group, up to 128 at a time, against the
// prefix's keys, each key tile brought from its pages once for the tile of rows.
//
// A CTA works on pieces of the prefixes' list (see PagedWork): consecutive
// 128-key tiles of one (group, KV head, 128-row tile), and leaves each piece's
// (O unnormalised, running max, sum) for the join.  Per key tile
//   S = Q K^T       tcgen05.mma, 128 x 128, into TMEM;
//   P = exp2(S - m) by four softmax warps, a thread a row, written as f16 over
//                   S's own columns;
//   O += P V        tcgen05.mma with A from TMEM, V as stored (f16).
// One CTA's chain S, softmax, P V has nothing of its own to overlap, so two
// CTAs share an SM (half of TMEM and of shared memory each for d 64 and 128)
// and the tensor core works for one while the other's softmax runs; K of the
// next tile loads during the softmax and V during the next S.  P is handed over
// in two halves of 64 keys, so the first half's products run beside the second
// half's exponentials.  d 256 fills TMEM and shared memory alone.
//
// Warp roles (256 threads): warps 0-3 softmax and the partials' epilogue, warp
// 4 the TMA producer (a lane for each page part and 64-column slice), warp 5
// the issue of every MMA; 6 and 7 only give their registers away.
#include "launchers.h"
#include "paged.cuh"

namespace dhsa {
namespace {

constexpr int kBM = kPrefixRows;
constexpr int kBN = kPrefixBN;
constexpr int kThreads = 256;
constexpr int kProducer = 4;
constexpr int kMma = 5;
// O is rescaled only when a row's maximum grew by more than 2^8 since the last
// time: weights then reach 256 instead of 1, which f16 holds with the same
// relative rounding (2^-11), and most tiles skip the pass over O.
constexpr float kRescaleLog2 = 8.0f;

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

template <int D>
struct PrefixCfg {
  static constexpr int kCtas = D == 256 ? 1 : 2;  // on an SM
  static constexpr int kStages = D == 64 ? 2 : 1;  // of the K ring and of the V ring
  static constexpr int kSlices = D / 64;
  static constexpr int kSub = kBN * 128;           // one 64-column slice of a tile
  static constexpr int kTile = kSlices * kSub;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffScan = kOffV + kStages * kTile;
  static constexpr int kOffBar = kOffScan + ((static_cast<int>(sizeof(PagedScan)) + 15) / 16) * 16;
  static constexpr int kSmemBytes = kOffBar + 256 + 1024;
  static constexpr uint32_t kTmemCols = D == 256 ? 512 : 256;
  static constexpr uint32_t kColO = D == 256 ? 256 : 128;
  static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "shared memory budget");
};

enum {
  kBarKFull = 0,   // + stage
  kBarVFull = 2,   // + stage
  kBarKFree = 4,   // + stage: S of the tile done
  kBarVFree = 6,   // + stage: P V of the tile done
  kBarSFull = 8,
  kBarPHalf = 9,   // first 64 keys of P written, O rescaled
  kBarPFull = 10,
  kBarQFull = 11,  // a piece's Q in shared memory
  kBarODone = 12,  // a piece's last P V done
  kBarDrain = 13,
  kNumBars = 14
};

template <int D>
__global__ void __launch_bounds__(kThreads, PrefixCfg<D>::kCtas)
    paged_prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedWork w) {
  using C = PrefixCfg<D>;
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
  const int gh = w.num_q_heads / w.p.num_kv_heads;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kBarSFull; ++s) mbar_init(bar(s), 1);
    mbar_init(bar(kBarSFull), 1);
    mbar_init(bar(kBarPHalf), 4);  // one arrival per softmax warp
    mbar_init(bar(kBarPFull), 4);
    mbar_init(bar(kBarQFull), 4);
    mbar_init(bar(kBarODone), 1);
    mbar_init(bar(kBarDrain), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  paged_schedule<kBN, kBM, kThreads>(w.p, gh, w.prefix, sc, w.status);  // syncs the CTA
  let_next_start();
  PagedWalk<kBN, kBM> walk;
  if (!walk.init(&w.p, gh, w.prefix, sc)) return;  // uniform for the CTA
  if (warp == kMma) {
    tmem_alloc(smem_u32(misc), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);

  if (warp >= 4) {
    if constexpr (D != 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == kProducer) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      // a lane for each box of a tile: (page part, 64-column slice)
      const int ps = w.p.page_size;
      const int box = ps < kBN ? ps : kBN;
      const int sl = lane % C::kSlices, pp = lane / C::kSlices;
      const bool mine = pp < kBN / box;
      const uint32_t dst0 = sbase + sl * C::kSub + pp * box * 128;
      int n = 0;  // key tiles, across pieces
      bool ok = true;
      do {
        const int h = walk.seg / walk.rt;
        const int* table = w.p.block_table + static_cast<long long>(walk.it.row) * w.p.table_stride;
        auto page_at = [&](int kt) -> int {
          const int key = (walk.first + walk.kt + kt) * kBN + pp * box;
          if (kt >= walk.count || !mine || key >= walk.it.hi) return -1;
          const int pg = table[key / ps];
          if (static_cast<unsigned>(pg) < static_cast<unsigned>(w.p.num_pages)) return pg;
          report(w.status, kDevCheck);
          return w.p.num_pages;  // outside the map: the box arrives as zeros
        };
        int page = page_at(0);
        for (int kt = 0; kt < walk.count; ++kt, ++n) {
          const int page_next = page_at(kt + 1);
          const int s = n % C::kStages;
          const uint32_t round = static_cast<uint32_t>(n / C::kStages);
          const unsigned bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * box * 128;
          const int in_page = ((walk.first + walk.kt + kt) * kBN + pp * box) % ps;
          if (round > 0) ok = mbar_wait(bar(kBarKFree + s), (round - 1) & 1, abort_flag, w.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(kBarKFull + s), bytes);
          __syncwarp();
          if (page >= 0)
            tma_load_4d(dst0 + C::kOffK + s * C::kTile, &tm_k, bar(kBarKFull + s), sl * 64, in_page, h, page);
          if (round > 0) ok = mbar_wait(bar(kBarVFree + s), (round - 1) & 1, abort_flag, w.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) {
            ++n;  // this tile's K is under way
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(kBarVFull + s), bytes);
          __syncwarp();
          if (page >= 0)
            tma_load_4d(dst0 + C::kOffV + s * C::kTile, &tm_v, bar(kBarVFull + s), sl * 64, in_page, h, page);
          page = page_next;
        }
      } while (ok && walk.next());
      if (*abort_flag && lane == 0) {
        // let copies already in flight land before the CTA exits (bounded)
        volatile int never = 0;
        for (int x = max(0, n - C::kStages); x < n; ++x) {
          mbar_wait(bar(kBarKFull + x % C::kStages), (x / C::kStages) & 1, &never, nullptr, 10000000ull);
          mbar_wait(bar(kBarVFull + x % C::kStages), (x / C::kStages) & 1, &never, nullptr, 10000000ull);
        }
      }
    } else if (warp == kMma) {
      if (lane == 0) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(kBM, kBN, 0);
        constexpr uint32_t idesc_o = idesc_f16_f32(kBM, D, 1);  // P and V in f16
        int n = 0, piece = 0;
        bool ok = true;
        do {
          ok = mbar_wait(bar(kBarQFull), piece & 1, abort_flag, w.status);
          for (int kt = 0; ok && kt < walk.count; ++kt, ++n) {
            const int s = n % C::kStages;
            const uint32_t ph = static_cast<uint32_t>(n / C::kStages) & 1u;
            if (!(ok = mbar_wait_spin(bar(kBarKFull + s), ph, abort_flag, w.status))) break;
            tc_fence_after();
            const uint32_t kbase = sbase + C::kOffK + s * C::kTile;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::kSub + (kk & 3) * 32;
              umma_f16_ss(tmem, smem_desc_sw128(sbase + C::kOffQ + off, 16, 1024),
                          smem_desc_sw128(kbase + off, 16, 1024), idesc_s, kk > 0 ? 1u : 0u);
            }
            umma_commit(bar(kBarSFull));
            umma_commit(bar(kBarKFree + s));
            const uint32_t vbase = sbase + C::kOffV + s * C::kTile;
            auto issue_pv = [&](int kk0, int kk1) {
#pragma unroll
              for (int kk = kk0; kk < kk1; ++kk)
                umma_f16_ts(tmem + C::kColO, tmem + kk * 8, smem_desc_sw128(vbase + kk * 16 * 128, C::kSub, 1024),
                            idesc_o, (kt > 0 || kk > 0) ? 1u : 0u);
            };
            if (!(ok = mbar_wait_spin(bar(kBarVFull + s), ph, abort_flag, w.status))) break;
            if (!(ok = mbar_wait_spin(bar(kBarPHalf), n & 1, abort_flag, w.status))) break;
            tc_fence_after();
            issue_pv(0, kBN / 32);
            if (!(ok = mbar_wait_spin(bar(kBarPFull), n & 1, abort_flag, w.status))) break;
            tc_fence_after();
            issue_pv(kBN / 32, kBN / 16);
            umma_commit(bar(kBarVFree + s));
            if (kt + 1 == walk.count) umma_commit(bar(kBarODone));
          }
          ++piece;
        } while (ok && walk.next());
        // every MMA issued above completes before TMEM is released
        umma_commit(bar(kBarDrain));
        volatile int never = 0;
        mbar_wait(bar(kBarDrain), 0, &never, nullptr);
      }
    }
  } else {
    if constexpr (D != 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int row = threadIdx.x;  // 0..127, the TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tS = tmem + lane_base, tO = tmem + lane_base + C::kColO;
    const float scale_log2 = w.scale * kLog2e;
    int n = 0, piece = 0;
    bool ok = true;
    do {
      const int h = walk.seg / walk.rt, rt = walk.seg - h * walk.rt;
      const int rows = (walk.it.t1 - walk.it.t0) * gh;
      const int r = rt * walk.tm + row;
      const bool valid = row < walk.tm && r < rows;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      // Q of the piece (the previous piece's last S is done: its SFull was waited for)
      int lim = 0;
      {
        const __nv_bfloat16* q = nullptr;
        if (valid) {
          const int t = walk.it.t0 + r / gh;
          lim = min(walk.it.hi, paged_limit(w.p, paged_seq_of(w.p, t), t));
          q = static_cast<const __nv_bfloat16*>(w.q) + t * w.q_stride +
              static_cast<long long>(h * gh + r % gh) * D;
        }
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = valid ? *reinterpret_cast<const uint4*>(q + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(smem + C::kOffQ + (c >> 3) * C::kSub + row * 128 + (((c & 7) ^ (row & 7)) << 4)) =
              v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarQFull));
      }
      float m_run = -INFINITY;  // maximum that the weights are taken against (log2 units)
      float l_run = 0.f;
      for (int kt = 0; kt < walk.count; ++kt, ++n) {
        const int k0 = (walk.first + walk.kt + kt) * kBN;
        if (!(ok = mbar_wait(bar(kBarSFull), n & 1, abort_flag, w.status))) break;
        tc_fence_after();
        if (k0 + kBN > walk.it.hi) {
          // slots behind the prefix may hold anything, NaN included, and 0 *
          // NaN is NaN: V's rows there are zeroed (a thread a row)
          const int s = n % C::kStages;
          if (!(ok = mbar_wait(bar(kBarVFull + s), static_cast<uint32_t>(n / C::kStages) & 1u, abort_flag, w.status)))
            break;
          if (k0 + row >= walk.it.hi) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              *reinterpret_cast<uint4*>(smem + C::kOffV + s * C::kTile + (c >> 3) * C::kSub + row * 128 +
                                        ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();  // before this warp's arrival on PHalf, which takes all four
        }
        if (!warp_valid) {  // no row of this warp counts: its P may be anything
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(kBarPHalf));
            mbar_arrive(bar(kBarPFull));
          }
          continue;
        }
        float s[kBN];
        float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const int cols = lim - k0;  // valid columns: c < cols
        auto take_half = [&](int base, uint32_t (&ra)[32], uint32_t (&rb)[32]) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            s[base + e] = __uint_as_float(ra[e]);
            s[base + 32 + e] = __uint_as_float(rb[e]);
          }
          if (cols < base + kBN / 2) {
#pragma unroll
            for (int c = base; c < base + kBN / 2; ++c)
              if (c >= cols) s[c] = -INFINITY;
          }
#pragma unroll
          for (int c = base; c < base + kBN / 2; c += 8) {
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
          tmem_ld32(tS + 64, rc);
          tmem_ld32(tS + 96, rd);
          take_half(0, ra, rb);
          tmem_wait_ld();
          reg_dep32(rc);
          reg_dep32(rd);
          take_half(kBN / 2, rc, rd);
        }
        const float m_tile = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])) * scale_log2;
        const bool any = __any_sync(0xffffffffu, m_tile > m_run + kRescaleLog2);
        float alpha = 1.f;
        if (any) {
          const float m_new = fmaxf(m_run, m_tile);
          alpha = m_new == -INFINITY ? 1.f : ex2_approx(m_run - m_new);
          m_run = m_new;
        }
        const float m_use = m_run == -INFINITY ? 0.f : m_run;
        uint64_t ps2[2] = {0ull, 0ull};
        const uint64_t scale2 = f2_pack(scale_log2, scale_log2);
        const uint64_t shift2 = f2_pack(-m_use, -m_use);
        // P of columns cb .. cb + 63 over the TMEM columns cb / 2 .. (S is in registers)
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
        if (any && kt > 0) {
          // O is rescaled before this tile's products; the last tile's are
          // done, since this S was issued after them
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
        if (lane == 0) mbar_arrive(bar(kBarPHalf));
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
        if (lane == 0) mbar_arrive(bar(kBarPFull));
      }
      if (!ok) break;
      if (!(ok = mbar_wait(bar(kBarODone), piece & 1, abort_flag, w.status))) break;
      tc_fence_after();
      if (warp_valid) {
        const long long part = paged_part_row(blockIdx.x, kBM, walk.item_row, walk.seg, walk.tm) + row;
        if (valid) w.prefix.part_ml[part] = make_float2(m_run, l_run);
        float* dst = w.prefix.part_o + part * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld();
          reg_dep32(o);
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(dst + 32 * c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        tc_fence_before();  // the next piece's P V overwrites O after this warp's next arrival
      }
      ++piece;
    } while (walk.next());
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, C::kTmemCols);
}

template <int D>
cudaError_t run(const PagedWork& w, cudaStream_t stream) {
  using C = PrefixCfg<D>;
  CUtensorMap mk, mv;
  if (encode_pages_map(&mk, w.p.k_pages, w.p, kBN, false) != CUDA_SUCCESS ||
      encode_pages_map(&mv, w.p.v_pages, w.p, kBN, true) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaError_t e =
      cudaFuncSetAttribute(paged_prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  paged_prefix_kernel<D><<<w.prefix.ctas, kThreads, C::kSmemBytes, stream>>>(mk, mv, w);
  return cudaGetLastError();
}

}  // namespace

int paged_prefix_ctas(int head_dim, int sms) {
  return sms * (head_dim == 256 ? PrefixCfg<256>::kCtas : PrefixCfg<128>::kCtas);
}

cudaError_t launch_paged_prefix(const PagedWork& w, cudaStream_t stream) {
  switch (w.p.head_dim) {
    case 64: return run<64>(w, stream);
    case 128: return run<128>(w, stream);
    default: return run<256>(w, stream);
  }
}

}  // namespace dhsa
