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
// of its own. The maximum only moves when a tile exceeds it by more than 2^8;
// P is rounded to bf16 for its product, the sum takes it unrounded.
//
// Bound: HBM for up to 128 rows (64 KB of keys and values for 2 d 128^2 products
// of each kind), the tensor cores and the chain from scores to weights above.
//
// Warps: 0 loads (TMA; zeroes value rows behind the prefix's end), 1 MMA issue
// and TMEM, 2 the parts of this CTA's run (3 idles), 4-7 and 8-11 the two
// softmax warpgroups, one thread per row. Every wait is bounded. Nothing waits
// for another CTA: the decode grid joins the parts.
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
  const int32_t* kv_len;
  int Hkv, hpg, tpt, cap;
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
  static constexpr int kStages = D == 128 ? 2 : 4;  // K ring and V ring
  static constexpr int kItems = 2;
  static constexpr uint32_t kTile = kRows * D * 2;
  static constexpr uint32_t oQ = 0, oK = 2 * kTile, oV = oK + kStages * kTile, oStore = oV + kStages * kTile;
  static constexpr uint32_t kStore = 32 * 128;  // per softmax warp: 32 rows x 32 columns
  static constexpr uint32_t oItem = oStore + 8 * kStore, oBar = (oItem + kItems * sizeof(PxItem) + 15) & ~15u;
  static constexpr int kBars = 4 + 4 * kStages + 8 + 2 * kItems + 3;
  static constexpr uint32_t kTotal = oBar + kBars * 8 + 16;
};

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
  tc::griddep_launch_dependents();  // the decode grid may start as SMs fall free; it waits for this one's parts
  if (tc::smem_u32(px_smem) & 1023u) {  // the swizzled operands need 1024-byte alignment
    if (threadIdx.x == 0) set_status(p.status, MSA_ERR_CUDA);
    return;
  }
  if (!cta_in_order(p.s.groups, p.s.disorder)) return;  // the decode grid reports it
  PxItem* items = reinterpret_cast<PxItem*>(px_smem + SM::oItem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(px_smem + SM::oBar);
  uint64_t* q_full = bars;                // [2]
  uint64_t* q_empty = bars + 2;           // [2]
  uint64_t* k_full = bars + 4;            // [NS]
  uint64_t* k_empty = k_full + NS;        // [NS]
  uint64_t* v_full = k_empty + NS;        // [NS]
  uint64_t* v_empty = v_full + NS;        // [NS]
  uint64_t* s_full = v_empty + NS;        // [2]
  uint64_t* p_full = s_full + 2;          // [2]
  uint64_t* o_full = p_full + 2;          // [2]
  uint64_t* o_empty = o_full + 2;         // [2]
  uint64_t* item_full = o_empty + 2;      // [NI]
  uint64_t* item_empty = item_full + NI;  // [NI]
  uint64_t* tail_bar = item_empty + NI;   // the copies of a value tile whose last rows are then zeroed
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
    init(o_empty, 2, 4);
    init(item_full, NI, 1);
    init(item_empty, NI, 10);  // loads, MMA, 8 softmax warps
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
      int z = 0, nv = 0, nk = 0, tails = 0, nq0 = 0, nq1 = 0;  // z: tiles so far; the rest: loads issued
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
        auto first_row = [&](int j) {  // this lane's box of the part's tile j: its first row, -1 if it has none
          const int pi = (s.jb + j) * per + lane;
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
        for (int j = 0; j < s.n; ++j, ++z) {
          const int st = z % NS, ph = (z / NS) & 1;
          const int next = j + 1 < s.n ? first_row(j + 1) : -1;  // in flight while this tile is issued
          if (!(ok = warp_wait(&k_empty[st], ph ^ 1, abort_flag))) break;
          boxes(px_smem + SM::oK + st * SM::kTile, &tmK, &k_full[st], s.g, row);
          nk = z + 1;
          if (j == 0 && !s.alt) {
            load_q(1, nq1);
            if (!ok) break;
            ++nq1;
          }
          if (!(ok = warp_wait(&v_empty[st], ph ^ 1, abort_flag))) break;
          uint8_t* vt = px_smem + SM::oV + st * SM::kTile;
          const int valid = s.Lk - (s.jb + j) * kKeys;
          if (valid >= kKeys) {
            boxes(vt, &tmV, &v_full[st], s.g, row);
            nv = z + 1;
          } else {
            // weight 0 does not silence an infinity or NaN that an earlier tile left: those rows become zeros
            boxes(vt, &tmV, tail_bar, s.g, row);
            if (!(ok = warp_wait(tail_bar, tails & 1, abort_flag))) {
              int zero = 0;
              tc::mbar_wait(tail_bar, tails & 1, &zero);
              break;
            }
            ++tails;
            zero_rows<NH>(vt, valid, kKeys);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&v_full[st]);
          }
          row = next;
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
        for (int x = max(nk - NS, 0); x < nk; ++x) tc::mbar_wait(&k_full[x % NS], (x / NS) & 1, &zero);
        for (int x = max(nv - NS, 0); x < nv; ++x) tc::mbar_wait(&v_full[x % NS], (x / NS) & 1, &zero);
      }
    } else if (warp == 1) {
      // ----------------------------- MMA issue -----------------------------
      // A part is steps t = 0, 1, ..., whose row tile is t & 1: of key tile t / 2,
      // or of key tile t where the halves take them alternately.
      if (lane == 0) {
        constexpr uint32_t kHi = tc::smem_desc_hi(1024, 2);
        const uint32_t qa = tc::smem_desc_lo(tc::smem_u32(px_smem + SM::oQ), 16);
        const uint32_t ka = tc::smem_desc_lo(tc::smem_u32(px_smem + SM::oK), 16);
        const uint32_t va = tc::smem_desc_lo(tc::smem_u32(px_smem + SM::oV), kHalfTile);
        bool ok = true;
        uint32_t z = 0, qu0 = 0, qu1 = 0, ou0 = 0, ou1 = 0, sp0 = 0, sp1 = 0;  // tiles; uses of Q, of O; steps
        for (int it = 0; ok; ++it) {
          if (!(ok = tc::mbar_wait(&item_full[it % NI], (it / NI) & 1, abort_flag))) break;
          const int mode = items[it % NI].mode, n = items[it % NI].d.n, alt = items[it % NI].d.alt;
          tc::mbar_arrive(&item_empty[it % NI]);
          if (mode == 3) break;
          if (mode == 2) continue;
          const int steps = alt ? n : 2 * n;
          auto tile = [&](int t) { return z + uint32_t(alt ? t : t >> 1); };
          auto scores = [&](int t) {  // S_w = Q K^T, and what it is the last to read falls free
            const uint32_t w = t & 1, st = tile(t) % NS;
            const uint32_t q0 = qa + (alt ? 0u : (w * SM::kTile) >> 4), k0 = ka + ((st * SM::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * kHalfTile + (kk & 3) * 32) >> 4;
              tc::mma_f16_ss_lo<kHi>(tmem + w * 128, q0 + off, k0 + off, kIdS, kk > 0 ? 1u : 0u);
            }
            tc::mma_commit(&s_full[w]);
            if (alt || w == 1) tc::mma_commit(&k_empty[st]);
            if (alt ? t + 1 == steps : t + 2 >= steps) tc::mma_commit(&q_empty[alt ? 0 : w]);
          };
          for (int t = 0; t < 2 && t < steps; ++t) {
            // the first scores go over the last weights of the part before, behind the products that read them
            if (!(ok = (t == 1 && alt ? true : tc::mbar_wait(&q_full[t], (t ? qu1 : qu0) & 1, abort_flag)) &&
                       tc::mbar_wait(&k_full[tile(t) % NS], (tile(t) / NS) & 1, abort_flag)))
              break;
            tc::fence_after_sync();
            scores(t);
          }
          ++qu0;
          if (!alt) ++qu1;
          for (int t = 0; t < steps && ok; ++t) {
            const uint32_t w = t & 1, st = tile(t) % NS;
            // what is ready early is waited for first: every wait between products costs the pipe
            if (!(ok = tc::mbar_wait(&v_full[st], (tile(t) / NS) & 1, abort_flag) &&
                       (t + 2 >= steps || tc::mbar_wait(&k_full[tile(t + 2) % NS], (tile(t + 2) / NS) & 1, abort_flag))))
              break;
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
            if (t + 2 < steps) {
              scores(t + 2);  // in issue order behind the product that reads P: S may go over it
            } else {
              tc::mma_commit(&o_full[w]);
              w ? ++ou1 : ++ou0;
            }
            if (alt || w == 1) tc::mma_commit(&v_empty[st]);
          }
          z += n;
        }
        if (!ok) fail();
        int zero = 0;
        tc::mma_commit(done_bar);
        tc::mbar_wait(done_bar, 0, &zero);
      }
    } else if (warp == 2) {
      // ------------------------------ parts ------------------------------
      PrefixPlan plan{p.s, p.kv_len, p.Hkv, p.cap, (1 << p.pages.page_log2) - 1};
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
      if (plan.init(blockIdx.x, blockIdx.x == 0)) {
        while (ok && plan.at < plan.end) {
          PxItem d;
          d.d = plan.next(blockIdx.x);
          // the part's own pages in range; if not, the decode grid finds its rows marked
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
    const uint32_t stage = tc::smem_u32(px_smem + SM::oStore + (warp - 4) * SM::kStore);
    const int row_seq = r / p.hpg;
    bool ok = true;
    int z = 0, used = 0;  // steps and parts of this row tile
    for (int it = 0; ok; ++it) {
      if (!(ok = warp_wait(&item_full[it % NI], (it / NI) & 1, abort_flag))) break;
      const PxItem* sp = items + it % NI;
      const int n = sp->d.n, mode = sp->mode, jb = sp->d.jb, alt = sp->d.alt, Lk = sp->d.Lk, count = sp->d.count;
      const int64_t row0 = sp->d.row;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&item_empty[it % NI]);
      if (mode == 3) break;
      const bool valid = r < p.tpt * p.hpg && row_seq + (alt ? 0 : w * p.tpt) < count;
      const int64_t row = row0 + (alt ? w * count : w * p.tpt) * p.hpg + r;  // of the part's
      if (mode == 2) {
        if (valid) p.s.stat[row] = make_float2(-INFINITY, -1.f);
        continue;
      }
      float m = -INFINITY, l = 0.f;
      const int steps = alt ? (n - w + 1) / 2 : n;
      for (int i = 0; i < steps; ++i, ++z) {
        const int lim = Lk - (jb + (alt ? 2 * i + w : i)) * kKeys;  // columns below it are keys
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
      if (valid) p.s.stat[row] = make_float2(m, l);
      if (steps > 0) {
        if (!(ok = warp_wait(&o_full[w], used & 1, abort_flag))) break;
        ++used;
        tc::fence_after_sync();
      }
      // the rows' output, 32 columns at a time through shared memory, so that 8 lanes store 128 contiguous bytes
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        if (steps > 0) {
          tc::tmem_ld_32x32b_x32(obase + c * 32, reinterpret_cast<uint32_t*>(o));
          tc::tmem_ld_wait();
        } else {  // a single key tile: the other half has none, and 0 counts for nothing
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + (uint32_t(x ^ (lane & 7)) << 4)),
                       "f"(o[4 * x]), "f"(o[4 * x + 1]), "f"(o[4 * x + 2]), "f"(o[4 * x + 3])
                       : "memory");
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int rr = x * 4 + (lane >> 3), cc = lane & 7;
          const int64_t to = __shfl_sync(0xffffffffu, valid ? row : int64_t(-1), rr);
          float4 f;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                       : "r"(stage + rr * 128 + (uint32_t(cc ^ (rr & 7)) << 4))
                       : "memory");
          if (to >= 0) reinterpret_cast<float4*>(p.s.part + to * D + c * 32)[cc] = f;
        }
        __syncwarp();
      }
      if (steps > 0) {  // the next part's products may go over O
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&o_empty[w]);
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
  p.kv_len = f.seq.kv_len;
  p.Hkv = f.Hkv;
  p.hpg = f.Hq / f.Hkv;
  p.tpt = kRows / p.hpg;
  p.cap = f.seq.Tk;
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
  kern<<<kNumSMs, kPxThreads, bytes, stream>>>(tmQ, tmK, tmV, p);
  return cudaGetLastError();
}

}  // namespace

PrefixGeometry prefix_geometry_tc(int hpg) {
  const int tpt = kRows / hpg;
  return {hpg, 1, 2 * tpt, tpt, 2 * kRows, kNumSMs, 2};
}

cudaError_t launch_prefix_tc(const SharedArgs& a, cudaStream_t stream) {
  return a.f.d == 128 ? prefix<128>(a, stream) : prefix<64>(a, stream);
}

}  // namespace msa
