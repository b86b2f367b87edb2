// Decode over shared prefixes, the prefixes' part in bf16 on tcgen05 (sm_103a):
// the query rows of a whole group of sequences against the keys that they share
// (full_shared.cuh says what an item and a part are).
//
//   m_r = max_j s_rj,  l_r = sum_j exp(s_rj - m_r),  o_r = sum_j exp(s_rj - m_r) v_j,
//   s_rj = scale q_r . k_j,  j < prefix_len
//
// A CTA works on two row tiles of 128 at a time, so that one's softmax runs
// under the other's products:
//   S_w = Q K^T -> TMEM; softmax w: P_w = exp2(S scale - m) back over S as bf16
//   pairs; O_w += P_w V with A = P from TMEM.
// Either the tiles are different rows and take every key tile in turn (one copy
// of it serves both), or, where the rows fit into one tile, they are the same
// rows and take the key tiles alternately, each with a maximum, sum and output
// of its own; the two warpgroups then join them, half the columns each. K and V
// tiles come through one ring in the order in which the products need them. The maximum only moves when a tile exceeds it by more than 2^8;
// P is rounded to bf16 for its product, the sum takes it unrounded: the operands of a
// product have one type, and a second term for what that drops would be a second product with V. Prefill and decode
// do the same (outputs 0.0023 from 64 bits, 0.0017 of it their own rounding).
//
// Bound: HBM for up to 128 rows (64 KB of keys and values for 2 d 128^2 products
// of each kind), the tensor cores and the chain from scores to weights above.
// Measured alone, caches cold (Hq 32, Hkv 8, d 128): 24 sequences behind 128 K keys
// 87 us, 6.2 TB/s (tensor pipe 40 %); 96 behind three prefixes, 20 K keys, 77 us.
//
// Warps: 0 loads (TMA; zeroes value rows behind the prefix's end), 1 MMA issue
// and TMEM, 2 the parts of this CTA's run (3 idles), 4-7 and 8-11 the two
// softmax warpgroups, one thread per row. Every wait is bounded. Nothing waits
// for another CTA: a grid of their own joins the parts.
#include "full_shared.cuh"
#include "full_tc.cuh"

namespace msa {
namespace {

constexpr int kPxThreads = 384;
// As in the prefill: 168 registers a thread at launch, of which the load / MMA
// warpgroup hands 2 x 48 to the softmax warpgroups, once.
constexpr uint32_t kRegsLaunch = 168, kRegsFew = 72, kRegsMany = 216;
static_assert(kRegsFew + 2 * kRegsMany <= 3 * kRegsLaunch, "the shares come out of the launch's registers");
constexpr float kLazy = 8.f;  // log2 of the largest weight
static_assert(kPxKeys == kKeys, "key tiles");

struct PxParams {
  SharedParams s;
  PageMap pages;
  int Hkv, hpg, tpt;
  float scale_log2;
  uint32_t* status;
  int inject_timeout;  // test hook: every second CTA waits on a barrier nothing completes
};
struct PxItem {
  PrefixPart d;
  int mode;  // 0: to compute, 2: bad pages, 3: no more
};

template <int D>
struct PxSmem {
  static constexpr int kStages = D == 128 ? 5 : 10;  // ring of K and V tiles
  static constexpr int kItems = 2;
  static constexpr uint32_t kTile = kRows * D * 2;
  static constexpr uint32_t oQ = 0, oRing = 2 * kTile, oStat = oRing + kStages * kTile;
  static constexpr uint32_t kStat = 2 * kRows * sizeof(float2);  // [half][row]: maximum, sum
  static constexpr uint32_t oItem = oStat + kStat, oBar = (oItem + kItems * sizeof(PxItem) + 15) & ~15u;
  static constexpr int kBars = 4 + 2 * kStages + 8 + 2 * kItems + 4;
  static constexpr uint32_t kTotal = oBar + kBars * 8 + 16;
};
// The order of a part's 2 n tiles in the ring: K_0 V_0 K_1 V_1 ..., or, where the
// halves take key tiles alternately, K_0 K_1 V_0 K_2 V_1 ... V_(n-1): the
// scores of tile t + 2 follow the products with V_t.
__device__ __forceinline__ int k_place(bool alt, int j) { return !alt ? 2 * j : j < 2 ? j : 2 * j - 1; }
__device__ __forceinline__ int v_place(bool alt, int j, int n) { return !alt || j == n - 1 ? 2 * j + 1 : 2 * j + 2; }
// the key tile of a place; whether it is V's
__device__ __forceinline__ int at_place(bool alt, int x, int n, bool& is_v) {
  if (!alt || x == 2 * n - 1) {
    is_v = x & 1;
    return x >> 1;
  }
  is_v = x >= 2 && !(x & 1);
  return is_v ? (x - 2) >> 1 : x < 2 ? x : (x + 1) >> 1;
}
// Eight floats to global memory: one whole 32-byte sector
__device__ __forceinline__ void store8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void arrive_twice(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 2;" ::"r"(tc::smem_u32(bar)) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kPxThreads, 1)
    full_prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PxParams p) {
  using SM = PxSmem<D>;
  constexpr int NH = D / 64, NS = SM::kStages, NI = SM::kItems;
  constexpr uint32_t kIdS = tc::idesc_bf16_f32(kRows, kKeys);
  constexpr uint32_t kIdO = tc::idesc_bf16_f32(kRows, D, true);  // B = V, MN-major
  constexpr uint32_t kColO = 256;
  extern __shared__ __align__(1024) uint8_t px_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (tc::smem_u32(px_smem) & 1023u) {  // the swizzled operands need 1024-byte alignment
    if (threadIdx.x == 0) set_status(p.status, MSA_ERR_CUDA);
    return;
  }
  PxItem* items = reinterpret_cast<PxItem*>(px_smem + SM::oItem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(px_smem + SM::oBar);
  uint64_t* q_full = bars;                // [2]
  uint64_t* q_empty = bars + 2;           // [2]
  uint64_t* t_full = bars + 4;            // [NS]
  uint64_t* t_empty = t_full + NS;        // [NS]
  uint64_t* s_full = t_empty + NS;        // [2]
  uint64_t* p_full = s_full + 2;          // [2]
  uint64_t* o_full = p_full + 2;          // [2]
  uint64_t* o_empty = o_full + 2;         // [2]
  uint64_t* item_full = o_empty + 2;      // [NI]
  uint64_t* item_empty = item_full + NI;  // [NI]
  uint64_t* both_bar = item_empty + NI;   // both halves' outputs, maxima and sums are there
  uint64_t* tail_bar = both_bar + 1;      // the copies of a value tile whose last rows are then zeroed
  uint64_t* done_bar = tail_bar + 1;
  uint64_t* never_bar = done_bar + 1;     // no thread arrives on it (timeout injection)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + SM::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  if (threadIdx.x == 0) {
    auto init = [](uint64_t* b, int n, uint32_t arrivals) {
#pragma unroll
      for (int x = 0; x < n; ++x) tc::mbar_init(b + x, arrivals);
    };
    init(bars, int(p_full - bars), 1);
    init(p_full, 2, 4);  // a row tile's softmax warps
    init(o_full, 2, 1);
    init(o_empty, 2, 8);  // both softmax warpgroups, or one twice
    init(item_full, NI, 1);
    init(item_empty, NI, 10);  // loads, MMA, 8 softmax warps
    init(both_bar, 1, 8);
    init(tail_bar, 3, 1);      // tail, done, never
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  tc::griddep_wait();               // the plan
  tc::griddep_launch_dependents();  // behind it, so that the decode grid, which may start now, has it as well
  auto fail = [&]() {
    *abort_flag = 1;
    set_status(p.status, MSA_ERR_TIMEOUT);
  };

  if (warp < 4) {
    tc::regs_dec<kRegsFew>();
    if (warp == 0) {
      // ------------------------------ loads ------------------------------
      if (lane == 0) {
        tc::tma_prefetch(&tmQ);
        tc::tma_prefetch(&tmK);
        tc::tma_prefetch(&tmV);
      }
      const int psz = 1 << p.pages.page_log2;
      const int per = kKeys >> p.pages.page_log2;  // boxes of a tile (lane x issues box x)
      auto boxes = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int g, int row) {
        const int cnt = __popc(__ballot_sync(0xffffffffu, row >= 0));
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, uint32_t(cnt * psz) * D * 2);
        __syncwarp();
        if (row >= 0) {
#pragma unroll
          for (int h = 0; h < NH; ++h) tc::tma_load_3d(dst + h * kHalfTile + lane * psz * 128, map, bar, h * 64, g, row);
        }
      };
      bool ok = true;
      int z = 0, issued = 0, tails = 0, nq0 = 0, nq1 = 0;  // z: places so far; the rest: loads issued
      for (int it = 0; ok; ++it) {
        if (!(ok = warp_wait(&item_full[it % NI], (it / NI) & 1, abort_flag))) break;
        const PrefixPart s = items[it % NI].d;
        const int mode = items[it % NI].mode;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&item_empty[it % NI]);
        if (mode == 3) break;
        if (mode == 2) continue;
        const int np = s.Lk >> p.pages.page_log2;
        const int32_t* table = p.pages.table + int64_t(s.leader) * p.pages.max_pages;
        bool is_v;
        auto first_row = [&](int x) {  // this lane's box of the tile at place x: its first row, -1 if it has none
          const int pi = (s.jb + at_place(s.alt, x, s.n, is_v)) * per + lane;
          return lane < per && pi < np ? table[pi] << p.pages.page_log2 : -1;
        };
        auto load_q = [&](int w, int use) {
          if (!(ok = warp_wait(&q_empty[w], (use & 1) ^ 1, abort_flag))) return;
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(&q_full[w], uint32_t(p.tpt * p.hpg) * D * 2);
#pragma unroll
            for (int h = 0; h < NH; ++h)
              tc::tma_load_4d(px_smem + SM::oQ + w * SM::kTile + h * kHalfTile, &tmQ, &q_full[w], h * 64, 0, s.g,
                              s.b0 + w * p.tpt);
          }
        };
        int row = first_row(0);
        load_q(0, nq0);
        if (!ok) break;
        ++nq0;
        for (int x = 0; x < 2 * s.n; ++x, ++z) {
          const int st = z % NS;
          const int next = x + 1 < 2 * s.n ? first_row(x + 1) : -1;  // in flight while this tile is issued
          const int j = s.jb + at_place(s.alt, x, s.n, is_v);
          if (!(ok = warp_wait(&t_empty[st], ((z / NS) & 1) ^ 1, abort_flag))) break;
          uint8_t* dst = px_smem + SM::oRing + st * SM::kTile;
          const int valid = s.Lk - j * kKeys;
          if (!is_v || valid >= kKeys) {
            boxes(dst, is_v ? &tmV : &tmK, &t_full[st], s.g, row);
            issued = z + 1;
          } else {
            // weight 0 does not silence an infinity or NaN that an earlier tile left: those rows become zeros
            boxes(dst, &tmV, tail_bar, s.g, row);
            if (!(ok = warp_wait(tail_bar, tails & 1, abort_flag))) {
              int zero = 0;
              tc::mbar_wait(tail_bar, tails & 1, &zero);
              break;
            }
            ++tails;
            zero_rows<NH>(dst, valid, kKeys);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&t_full[st]);
            issued = z + 1;
          }
          row = next;
          if (x == 0 && !s.alt) {
            load_q(1, nq1);
            if (!ok) break;
            ++nq1;
          }
          if (p.inject_timeout && z == 0 && blockIdx.x % 2 == 0 &&
              !(ok = __all_sync(0xffffffffu, tc::mbar_wait_for(never_bar, 0, abort_flag, tc::kInjectedWaitCycles))))
            break;
        }
      }
      if (!ok) {  // let the copies land before the CTA gives its shared memory up
        fail();
        int zero = 0;
        if (nq0 > 0) tc::mbar_wait(&q_full[0], (nq0 - 1) & 1, &zero);
        if (nq1 > 0) tc::mbar_wait(&q_full[1], (nq1 - 1) & 1, &zero);
        for (int x = max(issued - NS, 0); x < issued; ++x) tc::mbar_wait(&t_full[x % NS], (x / NS) & 1, &zero);
      }
    } else if (warp == 1) {
      // ----------------------------- MMA issue -----------------------------
      // A part is steps t = 0, 1, ..., whose row tile is t & 1: of key tile t / 2,
      // or of key tile t where the halves take them alternately.
      if (lane == 0) {
        constexpr uint32_t kHi = tc::smem_desc_hi(1024, 2);
        const uint32_t qa = tc::smem_desc_lo(tc::smem_u32(px_smem + SM::oQ), 16);
        const uint32_t ka = tc::smem_desc_lo(tc::smem_u32(px_smem + SM::oRing), 16);
        const uint32_t va = tc::smem_desc_lo(tc::smem_u32(px_smem + SM::oRing), kHalfTile);
        bool ok = true;
        uint32_t z = 0, qu0 = 0, qu1 = 0, ou0 = 0, ou1 = 0, sp0 = 0, sp1 = 0;  // places; uses of Q, of O; steps
        for (int it = 0; ok; ++it) {
          if (!(ok = tc::mbar_wait(&item_full[it % NI], (it / NI) & 1, abort_flag))) break;
          const int mode = items[it % NI].mode, n = items[it % NI].d.n;
          const bool alt = items[it % NI].d.alt;
          tc::mbar_arrive(&item_empty[it % NI]);
          if (mode == 3) break;
          if (mode == 2) continue;
          const int steps = alt ? n : 2 * n;
          auto k_at = [&](int t) { return z + uint32_t(k_place(alt, alt ? t : t >> 1)); };
          auto v_at = [&](int t) { return z + uint32_t(v_place(alt, alt ? t : t >> 1, n)); };
          auto full = [&](uint32_t x) { return tc::mbar_wait(&t_full[x % NS], (x / NS) & 1, abort_flag); };
          auto scores = [&](int t) {  // S_w = Q K^T, and what it is the last to read falls free
            const uint32_t w = t & 1, st = k_at(t) % NS;
            const uint32_t q0 = qa + (alt ? 0u : (w * SM::kTile) >> 4), k0 = ka + ((st * SM::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * kHalfTile + (kk & 3) * 32) >> 4;
              tc::mma_f16_ss_lo<kHi>(tmem + w * 128, q0 + off, k0 + off, kIdS, kk > 0 ? 1u : 0u);
            }
            tc::mma_commit(&s_full[w]);
            if (alt || w == 1) tc::mma_commit(&t_empty[st]);
            if (alt ? t + 1 == steps : t + 2 >= steps) tc::mma_commit(&q_empty[alt ? 0 : w]);
          };
          for (int t = 0; t < 2 && t < steps; ++t) {
            // the first scores go over the last weights of the part before, behind the products that read them
            if (!(ok = (t == 1 && alt ? true : tc::mbar_wait(&q_full[t], (t ? qu1 : qu0) & 1, abort_flag)) && full(k_at(t))))
              break;
            tc::fence_after_sync();
            scores(t);
          }
          ++qu0;
          if (!alt) ++qu1;
          for (int t = 0; t < steps && ok; ++t) {
            const uint32_t w = t & 1, st = v_at(t) % NS;
            // what is ready early is waited for first: every wait between products costs the pipe
            if (!(ok = full(v_at(t)) && (t + 2 >= steps || full(k_at(t + 2))))) break;
            const uint32_t v0 = va + ((st * SM::kTile) >> 4);
            // O of the part before has been read
            if (t < 2 && !(ok = tc::mbar_wait(&o_empty[w], ((w ? ou1 : ou0) & 1) ^ 1, abort_flag))) break;
            if (!(ok = tc::mbar_wait(&p_full[w], (w ? sp1 : sp0) & 1, abort_flag))) break;
            w ? ++sp1 : ++sp0;
            tc::fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)  // O_w += P_w V
              tc::mma_f16_ts_lo<kHi>(tmem + kColO + w * D, tmem + w * 128 + kk * 8, v0 + ((kk * 16 * 128) >> 4), kIdO,
                                     t > 1 || kk > 0 ? 1u : 0u);
            if (alt || w == 1) tc::mma_commit(&t_empty[st]);
            if (t + 2 < steps) {
              scores(t + 2);  // in issue order behind the product that reads P: S may go over it
            } else {
              tc::mma_commit(&o_full[w]);
              w ? ++ou1 : ++ou0;
            }
          }
          z += 2 * n;
        }
        if (!ok) fail();
        int zero = 0;
        tc::mma_commit(done_bar);
        tc::mbar_wait(done_bar, 0, &zero);
      }
    } else if (warp == 2) {
      // ------------------------------ parts ------------------------------
      PrefixRuns plan{p.s, p.Hkv};
      bool ok = true;
      int it = 0;
      auto publish = [&](const PxItem& d) {
        if (!(ok = warp_wait(&item_empty[it % NI], ((it / NI) & 1) ^ 1, abort_flag))) return;
        if (lane == 0) {
          items[it % NI] = d;
          tc::mbar_arrive(&item_full[it % NI]);
        }
        ++it;
      };
      if (plan.init(p.s.get_head(), blockIdx.x)) {
        while (ok && plan.at < plan.end) {
          PxItem d;
          d.d = plan.next();
          // the part's own pages in range; if not, the joins find its rows marked
          const int32_t* row = p.pages.table + int64_t(d.d.leader) * p.pages.max_pages;
          const int per = kKeys >> p.pages.page_log2, to = min((d.d.jb + d.d.n) * per, d.d.Lk >> p.pages.page_log2);
          bool bad = false;
#pragma unroll 4
          for (int x = d.d.jb * per + lane; x < to; x += 32) bad |= row[x] < 0 || row[x] >= p.pages.num_pages;
          d.mode = __any_sync(0xffffffffu, bad) ? 2 : 0;
          if (d.mode == 2 && lane == 0) set_status(p.status, MSA_ERR_BOUNDS);
          publish(d);
        }
      }
      if (ok) {
        PxItem d{};
        d.mode = 3;
        publish(d);
      }
      if (!ok) fail();
    }
  } else {
    // ------------------------------ softmax ------------------------------
    tc::regs_inc<kRegsMany>();
    const int w = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t sbase = tmem + (uint32_t(quarter * 32) << 16) + w * 128;
    const uint32_t obase = tmem + (uint32_t(quarter * 32) << 16) + kColO + w * D;
    float2* stats = reinterpret_cast<float2*>(px_smem + SM::oStat);
    const int row_seq = r / p.hpg;
    bool ok = true;
    int z = 0, used = 0, alts = 0;  // steps and parts of this row tile; parts of alternate key tiles
    for (int it = 0; ok; ++it) {
      if (!(ok = warp_wait(&item_full[it % NI], (it / NI) & 1, abort_flag))) break;
      // the item's slot is given back at its end: what is only wanted there is read there
      const PxItem* sp = items + it % NI;
      const int n = sp->d.n, mode = sp->mode, alt = sp->d.alt;
      auto give_back = [&]() {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&item_empty[it % NI]);
      };
      if (mode == 3) break;
      auto my_row = [&](bool& valid) {
        valid = r < p.tpt * p.hpg && row_seq + (alt ? 0 : w * p.tpt) < sp->d.count;
        return sp->d.row + (alt ? 0 : w * p.tpt) * p.hpg + r;  // of the part's
      };
      if (mode == 2) {
        bool valid;
        const int64_t row = my_row(valid);
        if (valid) p.s.stat[row] = make_float2(-INFINITY, -1.f);
        give_back();
        continue;
      }
      int lim = sp->d.Lk - (sp->d.jb + (alt ? w : 0)) * kKeys;  // columns of the tile below it are keys
      float m = -INFINITY, l = 0.f;
      const int steps = alt ? (n - w + 1) / 2 : n;
      for (int i = 0; i < steps; ++i, ++z, lim -= alt ? 2 * kKeys : kKeys) {
        if (!(ok = warp_wait(&s_full[w], z & 1, abort_flag))) break;
        tc::fence_after_sync();
        // O follows a raised maximum: S is complete, so is the product before it, and O is at rest
        auto raise = [&](float mt) {
          if (i == 0) {
            m = mt;
          } else if (__any_sync(0xffffffffu, mt > m + kLazy)) {
            const float mn = mt > m + kLazy ? mt : m;
            const float a = mn == m ? 1.f : ex2(m - mn);
            l *= a;
            m = mn;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tc::tmem_ld_32x32b_x32(obase + c * 32, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * a);
              tc::tmem_st_32x32b_x32(obase + c * 32, o);
            }
          }
          return m == -INFINITY ? 0.f : -m;
        };
        auto hand_over = [&]() {
          tc::tmem_st_wait();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&p_full[w]);
        };
        if (lim >= kKeys) {
          uint32_t v[kKeys];
          float m4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) m4[c] = tc::tmem_ld_max_32x32b_x32(sbase + c * 32, v + c * 32);
          tc::tmem_ld_wait();
          const float neg = raise(fmaxf(tc::fmax3(m4[0], m4[1], m4[2]), m4[3]) * p.scale_log2);
          const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), neg2 = pair(neg, neg);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              uint32_t* e = v + c * 64 + 2 * x;
              const float2 t = split(fma2(pair(__uint_as_float(e[0]), __uint_as_float(e[1])), scale2, neg2));
              const float p0 = ex2(t.x), p1 = ex2(t.y);
              e[0] = __float_as_uint(p0);
              e[1] = __float_as_uint(p1);
              pk[x] = pack_bf16(p0, p1);
            }
            tc::tmem_st_32x32b_x32(sbase + c * 32, pk);
          }
          hand_over();
          // the sum, off the tensor cores' path
          uint64_t l2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
          for (int x = 0; x < kKeys / 2; ++x)
            l2[x & 1] = add2(l2[x & 1], pair(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])));
          const float2 ls = split(add2(l2[0], l2[1]));
          l += ls.x + ls.y;
        } else {
          // the prefix's end, 32 columns at a time; those behind it are only zeroed
          const int chunks = (lim + 31) >> 5;
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            uint32_t v[32];
            tc::tmem_ld_32x32b_x32(sbase + c * 32, v);
            tc::tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) mx = fmaxf(mx, c * 32 + x < lim ? __uint_as_float(v[x]) : -INFINITY);
          }
          const float neg = raise(mx * p.scale_log2);
          float l2[2] = {0.f, 0.f};
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32], pk[16];
            if (c < chunks) {  // P of chunk c goes over S of chunk c / 2
              tc::tmem_ld_32x32b_x32(sbase + c * 32, v);
              tc::tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                float p0 = ex2(fmaf(__uint_as_float(v[2 * x]), p.scale_log2, neg));
                float p1 = ex2(fmaf(__uint_as_float(v[2 * x + 1]), p.scale_log2, neg));
                if (c * 32 + 2 * x >= lim) p0 = 0.f;
                if (c * 32 + 2 * x + 1 >= lim) p1 = 0.f;
                l2[0] += p0;
                l2[1] += p1;
                pk[x] = pack_bf16(p0, p1);
              }
            } else {
#pragma unroll
              for (int x = 0; x < 16; ++x) pk[x] = 0u;
            }
            tc::tmem_st_32x32b_x16(sbase + c * 16, pk);
          }
          hand_over();
          l += l2[0] + l2[1];
        }
      }
      if (!ok) break;
      if (steps > 0) {
        if (!(ok = warp_wait(&o_full[w], used & 1, abort_flag))) break;
        ++used;
        tc::fence_after_sync();
      }
      bool valid;
      const int64_t row = my_row(valid);
      give_back();
      if (!alt) {
        if (valid) p.s.stat[row] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          float o[64];
          tc::tmem_ld_32x32b_x32(obase + c * 64, reinterpret_cast<uint32_t*>(o));
          tc::tmem_ld_32x32b_x32(obase + c * 64 + 32, reinterpret_cast<uint32_t*>(o + 32));
          tc::tmem_ld_wait();
          if (valid) {
#pragma unroll
            for (int x = 0; x < 8; ++x) store8(p.s.part + row * D + c * 64 + x * 8, o + x * 8);
          }
        }
        tc::fence_before_sync();  // the next part's products may go over O
        __syncwarp();
        if (lane == 0) arrive_twice(&o_empty[w]);
        continue;
      }
      // ---- both halves' states of the same rows: joined, each warpgroup half the columns ----
      // A half writes its statistics behind products that waited for everybody to release its last output,
      // which they do behind reading the last statistics; a half without steps, which waits for nothing, writes none.
      if (steps > 0) stats[w * kRows + r] = make_float2(m, l);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(both_bar);
      if (!(ok = warp_wait(both_bar, alts & 1, abort_flag))) break;
      ++alts;
      tc::fence_after_sync();
      const float2 s0 = stats[r], s1 = n > 1 ? stats[kRows + r] : make_float2(-INFINITY, 0.f);
      const float M = fmaxf(s0.x, s1.x);
      const float a0 = s0.x == M ? 1.f : ex2(s0.x - M), a1 = s1.x == M ? 1.f : ex2(s1.x - M);
      if (valid && w == 0) p.s.stat[row] = make_float2(M, s0.y * a0 + s1.y * a1);
      const uint32_t o0 = tmem + (uint32_t(quarter * 32) << 16) + kColO + w * (D / 2), o1 = o0 + D;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        float x0[32], x1[32];
        tc::tmem_ld_32x32b_x32(o0 + c * 32, reinterpret_cast<uint32_t*>(x0));
        tc::tmem_ld_32x32b_x32(o1 + c * 32, reinterpret_cast<uint32_t*>(x1));  // anything, if n == 1
        tc::tmem_ld_wait();
        if (valid) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float o[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) o[y] = n > 1 ? fmaf(x1[8 * x + y], a1, x0[8 * x + y] * a0) : x0[8 * x + y];
            store8(p.s.part + row * D + w * (D / 2) + c * 32 + x * 8, o);
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&o_empty[0]);
        if (n > 1) tc::mbar_arrive(&o_empty[1]);
      }
    }
    if (!ok) fail();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t prefix(const SharedArgs& a, cudaStream_t stream) {
  const FullArgs& f = a.f;
  PxParams p{};
  p.s = a.s;
  p.pages = f.pages;
  p.Hkv = f.Hkv;
  p.hpg = f.Hq / f.Hkv;
  p.tpt = kRows / p.hpg;
  p.scale_log2 = f.scale * kLog2e;
  p.status = &static_cast<WsHeader*>(f.ws)->status;
  p.inject_timeout = debug_inject_timeout() ? 1 : 0;
  const uint64_t krows = uint64_t(f.pages.num_pages) << f.pages.page_log2;
  const int box = 1 << f.pages.page_log2;
  CUtensorMap tmQ, tmK, tmV;
  if (!map_rows(&tmQ, f.q, f.seq.B, f.Hq, f.Hkv, D, p.tpt) || !map_keys(&tmK, f.k, krows, f.Hkv, D, box) ||
      !map_keys(&tmV, f.v, krows, f.Hkv, D, box))
    return cudaErrorInvalidValue;
  auto kern = full_prefix_kernel<D>;
  constexpr int bytes = int(PxSmem<D>::kTotal);
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  // a launch with other registers could not cover the warpgroups' shares
  static KernelReady ready;
  if (cudaError_t e = ready.on_device(reinterpret_cast<const void*>(kern), bytes, int(kRegsLaunch))) return e;
  ProfScope pf("full_prefix", stream);
  return launch_early(kern, kNumSMs, kPxThreads, bytes, stream, tmQ, tmK, tmV, p);
}

}  // namespace

PrefixGeometry prefix_geometry_tc(int hpg) {
  const int tpt = kRows / hpg;
  return {hpg, 1, 2 * tpt, tpt, 2 * kRows, kNumSMs, 2, 24, 4};
}

cudaError_t launch_prefix_tc(const SharedArgs& a, cudaStream_t stream) {
  return a.f.d == 128 ? prefix<128>(a, stream) : prefix<64>(a, stream);
}

}  // namespace msa
