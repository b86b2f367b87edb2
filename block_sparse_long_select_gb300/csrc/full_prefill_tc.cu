// Full attention, prefill, bf16 on tcgen05 (sm_103a): causal attention of
// packed query rows over packed or paged keys.
//
//   out_i = sum_j exp(s_ij - lse_i) v_j,  s_ij = scale q_i . k_j,  j <= Lk - Lq + i
//
// An item is 2 x 128 rows of one (sequence, key/value head) that walk its keys
// in tiles of 128. A row tile is 128 / hpg consecutive tokens x the hpg query
// heads that share the key/value head, token by token, so short sequences and
// chunks fill the 128 rows of an MMA, the causal edge is cut at 128 / hpg
// tokens, and one K/V tile serves every head of the group.
// The two row tiles alternate: while one's scores go through the softmax, the
// tensor cores run the other's products:
//   S_w(j) = Q_w K_j^T -> TMEM; softmax w: P_w(j) = exp2(S scale - m) back over
//   S as bf16 pairs; O_w += P_w(j) V_j with A = P from TMEM.
// The running maximum m only moves when a tile exceeds it by more than 2^8
// (then O and the sum are rescaled): weights stay below 2^8, and dividing by
// their sum at the end takes the common factor out again. P is rounded to
// bf16 for its product (2^-8 of each weight, which averages out over the keys);
// the sum takes the unrounded weights in fp32.
//
// The grid is persistent, one CTA per SM: the loads and first scores of the next
// item run under the end of the one before. Many items are handed out whole,
// long ones first; few or very long ones are divided into equal shares
// (full_sched.cuh), and the rows of an item that several CTAs share are joined
// by the last of them to arrive.
//
// Bound: the tensor cores (4 Hq d FLOPs per visible pair); in fact the chain from
// a tile's scores to its weights, about 1.4 us a tile of 2 x 128 rows where the
// products alone take 1.05. Measured (Hq 32, Hkv 8, d 128): 8192 tokens 393 us
// alone, 405 us in a loop (71 % of the measured tensor rate).
//
// Warps: 0 loads (TMA; zeroes the value rows behind a sequence's end, which
// may hold anything), 1 MMA issue and TMEM, 2 the items and the rows
// that see no key (3 idles), 4-7 and 8-11 the two softmax warpgroups, one thread per
// row. Every wait is bounded.
#include "full_sched.cuh"
#include "full_tc.cuh"

namespace msa {
namespace {

constexpr int kPfThreads = 384;
// Registers per thread: 168 at launch (3 warpgroups x 128 threads x 168), of
// which the load / MMA warpgroup hands 2 x 48 to the softmax warpgroups, whose
// threads hold a row of 128 scores. Given once, never taken back: a warp that
// asked for registers again could get them before the softmax warps do, and
// those would wait for good.
constexpr uint32_t kRegsLaunch = 168, kRegsFew = 72, kRegsMany = 216;
static_assert(kRegsFew + 2 * kRegsMany <= 3 * kRegsLaunch, "the shares come out of the launch's registers");
constexpr float kLazy = 8.f;  // log2 of the largest weight
// Shares, in keys: an item's start and end cost about two tiles; four tiles are
// the least that pays for a CTA of its own, and items up to eight are left whole
// (a join writes and reads 2 x 64 KB of partials, about three tiles).
constexpr int kPfFixed = 256, kPfLeast = 4 * kKeys + kPfFixed, kPfWhole = 8 * kKeys;

struct PfParams {
  SeqMap seq;
  PageMap pages;
  int Hq, Hkv, hpg, tpt, nslots;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  float* part;    // [2 * grid][D / 4][256][4] fp32: unnormalised rows of split items
  float2* stat;   // [2 * grid][256]: their maximum (log2 units) and sum
  uint32_t* arrivals;  // a byte per CTA, zero between calls: the parts of the split item that it holds the first of
  uint32_t* queue;     // next item to hand out, zero between calls
  uint32_t* status;
  int inject_timeout;  // test hook: every second CTA waits on a barrier nothing completes
};

struct PfItem {
  int b, g, i0, i1;          // rows (tokens) [i0, i1) of the sequence
  int jb, n;                 // key tiles [jb, jb + n)
  int q0, k0, Lq, Lk;
  int mode;                  // 0: whole, 1: part of a split item, 2: bad pages (zero rows), 3: no more items
  int c0, parts, slot;       // split: first CTA with tiles, number of parts, this part's slot
  int tiles, pad;            // of the whole item
};

template <int D>
struct PfSmem {
  static constexpr int kStages = D == 128 ? 2 : 4;  // K ring and V ring
  static constexpr int kItems = 2;
  static constexpr uint32_t kTile = kRows * D * 2;
  static constexpr uint32_t oQ = 0, oK = 2 * kTile, oV = oK + kStages * kTile, oStore = oV + kStages * kTile;
  static constexpr uint32_t kStore = 32 * 128;  // per softmax warp: 32 rows x 64 columns
  static constexpr uint32_t oItem = oStore + 8 * kStore, oBar = oItem + kItems * sizeof(PfItem);
  static constexpr int kBars = 4 + 4 * kStages + 2 + 2 + 4 + 2 * kItems + 2 + 3;
  static constexpr uint32_t kTotal = oBar + kBars * 8 + 16;
};

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1)
    full_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const PfParams p) {
  using SM = PfSmem<D>;
  constexpr int NH = D / 64, NS = SM::kStages, NI = SM::kItems;
  constexpr uint32_t kIdS = tc::idesc_bf16_f32(kRows, kKeys);
  constexpr uint32_t kIdO = tc::idesc_bf16_f32(kRows, D, true);  // B = V, MN-major
  constexpr uint32_t kColO = 256;
  extern __shared__ __align__(1024) uint8_t pf_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (tc::smem_u32(pf_smem) & 1023u) {  // the swizzled operands need 1024-byte alignment
    if (threadIdx.x == 0) set_status(p.status, MSA_ERR_CUDA);
    return;
  }
  PfItem* items = reinterpret_cast<PfItem*>(pf_smem + SM::oItem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(pf_smem + SM::oBar);
  uint64_t* q_full = bars;              // [2]
  uint64_t* q_empty = bars + 2;         // [2]
  uint64_t* k_full = bars + 4;          // [NS]
  uint64_t* k_empty = k_full + NS;      // [NS]
  uint64_t* v_full = k_empty + NS;      // [NS]
  uint64_t* v_empty = v_full + NS;      // [NS]
  uint64_t* s_full = v_empty + NS;      // [2]
  uint64_t* p_full = s_full + 2;        // [2]
  uint64_t* o_full = p_full + 2;        // [2]
  uint64_t* o_empty = o_full + 2;       // [2]
  uint64_t* item_full = o_empty + 2;    // [NI]
  uint64_t* item_empty = item_full + NI;  // [NI]
  uint64_t* part_bar = item_empty + NI;   // the warps' partials are written
  uint64_t* flag_bar = part_bar + 1;      // whether this CTA is the last of the item's
  uint64_t* tail_bar = flag_bar + 1;      // the copies of a value tile whose last rows are then zeroed
  uint64_t* done_bar = tail_bar + 1;
  uint64_t* never_bar = done_bar + 1;     // no thread arrives on it (timeout injection)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + SM::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = abort_flag + 1;
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
    init(part_bar, 1, 8);
    init(flag_bar, 4, 1);  // flag, tail, done, never
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
      const bool paged = p.pages.table != nullptr;
      const int psz = 1 << p.pages.page_log2;
      const int per = paged ? kKeys >> p.pages.page_log2 : 1;  // boxes of a tile (lane x issues box x)
      const int box_rows = paged ? psz : kKeys;
      auto boxes = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int g, int row) {
        const int cnt = __popc(__ballot_sync(0xffffffffu, row >= 0));
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, uint32_t(cnt * box_rows) * D * 2);
        __syncwarp();
        if (row >= 0) {
#pragma unroll
          for (int h = 0; h < NH; ++h)
            tc::tma_load_3d(dst + h * kHalfTile + lane * box_rows * 128, map, bar, h * 64, g, row);
        }
      };
      bool ok = true;
      int z = 0, nv = 0, nk = 0, tails = 0, nq0 = 0, nq1 = 0;  // z: tiles so far; the rest: loads issued
      for (int it = 0; ok; ++it) {
        if (!(ok = warp_wait(&item_full[it % NI], (it / NI) & 1, abort_flag))) break;
        const PfItem s = items[it % NI];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&item_empty[it % NI]);
        if (s.mode == 3) break;
        if (s.n == 0) continue;
        const int np = paged ? (s.Lk + psz - 1) >> p.pages.page_log2 : 0;
        const int32_t* table = paged ? p.pages.table + int64_t(s.b) * p.pages.max_pages : nullptr;
        auto first_row = [&](int j) {  // this lane's box of the item's tile j: its first row, -1 if it has none
          if (!paged) return lane == 0 ? s.k0 + (s.jb + j) * kKeys : -1;
          const int pi = (s.jb + j) * per + lane;
          return lane < per && pi < np ? table[pi] << p.pages.page_log2 : -1;
        };
        auto load_q = [&](int w, int use) {
          if (!(ok = warp_wait(&q_empty[w], (use & 1) ^ 1, abort_flag))) return;
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(&q_full[w], uint32_t(p.tpt * p.hpg) * D * 2);
#pragma unroll
            for (int h = 0; h < NH; ++h)
              tc::tma_load_4d(pf_smem + SM::oQ + w * SM::kTile + h * kHalfTile, &tmQ, &q_full[w], h * 64, 0, s.g,
                              s.q0 + s.i0 + w * p.tpt);
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
          boxes(pf_smem + SM::oK + st * SM::kTile, &tmK, &k_full[st], s.g, row);
          nk = z + 1;
          if (j == 0) {
            load_q(1, nq1);
            if (!ok) break;
            ++nq1;
          }
          if (!(ok = warp_wait(&v_empty[st], ph ^ 1, abort_flag))) break;
          uint8_t* vt = pf_smem + SM::oV + st * SM::kTile;
          const int valid = s.Lk - (s.jb + j) * kKeys;
          if (valid >= kKeys) {
            boxes(vt, &tmV, &v_full[st], s.g, row);
            nv = z + 1;
          } else {
            // rows behind the sequence's end belong to others: weight 0 does not
            // silence an infinity or NaN there, so they become zeros
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
      // One thread for both row tiles: issued by a thread each, their products
      // interleave and both finish late (504 us instead of 431 at 8K tokens).
      if (lane == 0) {
        constexpr uint32_t kHi = tc::smem_desc_hi(1024, 2);
        const uint32_t qa = tc::smem_desc_lo(tc::smem_u32(pf_smem + SM::oQ), 16);
        const uint32_t ka = tc::smem_desc_lo(tc::smem_u32(pf_smem + SM::oK), 16);
        const uint32_t va = tc::smem_desc_lo(tc::smem_u32(pf_smem + SM::oV), kHalfTile);
        auto scores = [&](int w, uint32_t st) {  // S_w = Q_w K^T
          const uint32_t q0 = qa + ((w * SM::kTile) >> 4), k0 = ka + ((st * SM::kTile) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * kHalfTile + (kk & 3) * 32) >> 4;
            tc::mma_f16_ss_lo<kHi>(tmem + w * 128, q0 + off, k0 + off, kIdS, kk > 0 ? 1u : 0u);
          }
          tc::mma_commit(&s_full[w]);
        };
        bool ok = true;
        uint32_t z = 0, used = 0;  // tiles and items so far
        for (int it = 0; ok; ++it) {
          if (!(ok = tc::mbar_wait(&item_full[it % NI], (it / NI) & 1, abort_flag))) break;
          const int mode = items[it % NI].mode, n = items[it % NI].n;
          tc::mbar_arrive(&item_empty[it % NI]);
          if (mode == 3) break;
          if (n == 0) continue;
          // the first scores go over the last weights of the item before, behind the products that read them
          if (!(ok = tc::mbar_wait(&q_full[0], used & 1, abort_flag) &&
                     tc::mbar_wait(&k_full[z % NS], (z / NS) & 1, abort_flag)))
            break;
          tc::fence_after_sync();
          scores(0, z % NS);
          if (n == 1) tc::mma_commit(&q_empty[0]);
          if (!(ok = tc::mbar_wait(&q_full[1], used & 1, abort_flag))) break;
          scores(1, z % NS);
          if (n == 1) tc::mma_commit(&q_empty[1]);
          tc::mma_commit(&k_empty[z % NS]);
          for (int j = 0; j < n && ok; ++j, ++z) {
            const uint32_t st = z % NS, st1 = (z + 1) % NS;
            // what is ready early is waited for first: every wait between products costs the pipe
            if (!(ok = tc::mbar_wait(&v_full[st], (z / NS) & 1, abort_flag) &&
                       (j + 1 == n || tc::mbar_wait(&k_full[st1], ((z + 1) / NS) & 1, abort_flag))))
              break;
            const uint32_t v0 = va + ((st * SM::kTile) >> 4);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              // O of the item before has been read
              if (j == 0 && !(ok = tc::mbar_wait(&o_empty[w], (used & 1) ^ 1, abort_flag))) break;
              if (!(ok = tc::mbar_wait(&p_full[w], z & 1, abort_flag))) break;
              tc::fence_after_sync();
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)  // O_w += P_w V
                tc::mma_f16_ts_lo<kHi>(tmem + kColO + w * D, tmem + w * 128 + kk * 8, v0 + ((kk * 16 * 128) >> 4), kIdO,
                                       j > 0 || kk > 0 ? 1u : 0u);
              if (j + 1 < n)
                scores(w, st1);  // in issue order behind the product that reads P: S may go over it
              else
                tc::mma_commit(&o_full[w]);
              if (w == 1) tc::mma_commit(&v_empty[st]);
              if (j + 1 < n) {
                if (w == 1) tc::mma_commit(&k_empty[st1]);
                if (j + 2 == n) tc::mma_commit(&q_empty[w]);
              }
            }
          }
          ++used;
        }
        if (!ok) fail();
        int zero = 0;
        tc::mma_commit(done_bar);
        tc::mbar_wait(done_bar, 0, &zero);
      }
    } else if (warp == 2) {
      // ------------------------------ items ------------------------------
      const int w2 = 2 * p.tpt;
      bool disorder = false;  // whether offsets are out of order (full_internal.cuh), known once all work is measured
      auto work = [&](int b) {  // items of 2 tpt rows that see keys
        const SeqSpan s = seq_span(p.seq, b);
        disorder |= !span_in_order(p.seq, s);
        if (!s.ok || s.Lq == 0 || s.Lk == 0) return SeqWork{0, 0, 0, 0};
        const int off = s.Lk - s.Lq, s0 = off < 0 ? -off / w2 : 0;
        return seq_work((s.Lq + w2 - 1) / w2 - s0, int(min(int64_t(off) + int64_t(s0 + 1) * w2, int64_t(s.Lk))), s.Lk, w2);
      };
      Share<decltype(work)> sh{work, {w2, kKeys, kPfFixed, kPfLeast, kPfWhole}, p.seq.B, p.Hkv};
      bool ok = true;
      int it = 0, checked = -1;
      bool bad = false;
      auto publish = [&](const PfItem& d) {
        if (!(ok = warp_wait(&item_empty[it % NI], ((it / NI) & 1) ^ 1, abort_flag))) return;
        if (lane == 0) {
          items[it % NI] = d;
          tc::mbar_arrive(&item_full[it % NI]);
        }
        ++it;
      };
      // an item's description; mode 2 if its pages are out of range
      auto describe = [&](PfItem& d, int sb, int g, int slot_tile, const SeqSpan& s) {
        d.b = sb;
        d.g = g;
        d.i0 = slot_tile * w2;
        d.i1 = min(d.i0 + w2, s.Lq);
        d.q0 = s.q0;
        d.k0 = s.k0;
        d.Lq = s.Lq;
        d.Lk = s.Lk;
        d.tiles = (s.Lk - s.Lq + d.i1 + kKeys - 1) / kKeys;
        if (p.pages.table && checked != sb) {  // every page of the sequence in range, for all its rows alike
          checked = sb;
          const int32_t* row = p.pages.table + int64_t(sb) * p.pages.max_pages;
          const int np = (s.Lk + (1 << p.pages.page_log2) - 1) >> p.pages.page_log2;
          bad = false;
#pragma unroll 4
          for (int x = lane; x < np; x += 32) bad |= row[x] < 0 || row[x] >= p.pages.num_pages;
          bad = __any_sync(0xffffffffu, bad);
          if (bad && lane == 0) set_status(p.status, MSA_ERR_BOUNDS);
        }
        if (bad) d.mode = 2;
      };
      const bool some_work = sh.measure(gridDim.x);
      disorder = __any_sync(0xffffffffu, disorder);
      if (!some_work) {
        // no row sees a key
      } else if (disorder) {  // items dealt out, each found sequence by sequence
        for (int i = blockIdx.x; ok && i < p.nslots * p.Hkv; i += gridDim.x) {
          int tile;
          SeqSpan s;
          const int sb = scan_tile(p.seq, false, w2, 1, i / p.Hkv, tile, s);
          if (sb < 0) break;  // nor are there any further on
          if (!s.ok || s.Lk - s.Lq + min((tile + 1) * w2, s.Lq) <= 0) continue;  // no keys: below
          PfItem d{};
          describe(d, sb, i % p.Hkv, tile, s);
          d.n = d.mode == 2 ? 0 : d.tiles;
          publish(d);
        }
      } else if (sh.hand_out()) {
        // Up to 32 sequences: a lane each, items by their place x in their sequence,
        // the last places (the longest walks) first. More: by slots, where the
        // last places of a sequence come first.
        const bool few = p.seq.B <= 32;
        const int mine = few && lane < p.seq.B ? work(lane).items : 0;
        const int all = (few ? __reduce_add_sync(0xffffffffu, mine) : p.nslots) * p.Hkv;
        int x = __reduce_max_sync(0xffffffffu, mine) - 1, before = 0;  // place; items before it
        for (int next = 0; ok && next < all;) {
          if (lane == 0) {
            next = int(atomicAdd(p.queue, 1u));
            // the last of the calls that find the queue empty leaves it ready for the next launch
            if (next == all + int(gridDim.x) - 1) atomicExch(p.queue, 0u);
          }
          next = __shfl_sync(0xffffffffu, next, 0);
          if (next >= all) break;
          int tile, sb, g = next % p.Hkv;
          SeqSpan s;
          if (few) {
            uint32_t longer = __ballot_sync(0xffffffffu, mine > x);
            while (next >= before + __popc(longer) * p.Hkv) {
              before += __popc(longer) * p.Hkv;
              --x;
              longer = __ballot_sync(0xffffffffu, mine > x);
            }
            const int nth = (next - before) / p.Hkv;  // of the sequences that reach this place
            g = (next - before) % p.Hkv;
            sb = __ffs(__ballot_sync(0xffffffffu, mine > x && __popc(longer & ((1u << lane) - 1u)) == nth)) - 1;
            s = seq_span(p.seq, sb);
            tile = x + (s.Lk < s.Lq ? (s.Lq - s.Lk) / w2 : 0);
          } else {
            sb = find_slot_tile(p.seq.cu_q, p.seq.B, w2, p.nslots - 1 - next / p.Hkv, tile);
            if (sb < 0) continue;
            s = seq_span(p.seq, sb);
            if (!s.ok || s.Lk - s.Lq + min((tile + 1) * w2, s.Lq) <= 0) continue;  // no keys: below
          }
          PfItem d{};
          describe(d, sb, g, tile, s);
          d.n = d.mode == 2 ? 0 : d.tiles;
          publish(d);
        }
      } else if (sh.init(blockIdx.x)) {
        for (; ok && !sh.done(); sh.next()) {
          const SeqSpan s = seq_span(p.seq, sh.cur.b);
          const int off = s.Lk - s.Lq;
          PfItem d{};
          describe(d, sh.cur.b, sh.cur.g, (off < 0 ? -off / w2 : 0) + sh.cur.x, s);
          int to;
          sh.tiles(d.tiles, d.jb, to);
          d.n = to - d.jb;
          if (d.n == 0) continue;
          if (d.mode == 2) {
            if (d.jb > 0) continue;  // whoever holds the first tile writes the rows
            d.n = 0;
          } else if (d.n < d.tiles) {
            d.mode = 1;
            // its CTAs are consecutive; the first may hold no more than the fixed cost
            d.c0 = sh.first_cta();
            while (!sh.holds(d.c0, d.tiles)) ++d.c0;
            while (d.c0 + d.parts < sh.G && sh.holds(d.c0 + d.parts, d.tiles)) ++d.parts;
            d.slot = 2 * int(blockIdx.x) + (d.c0 == int(blockIdx.x) ? 1 : 0);
          }
          publish(d);
        }
      }
      if (ok) {
        PfItem d{};
        d.mode = 3;
        publish(d);
      }
      if (!ok) fail();
      // --------------------- rows that see no key ---------------------
      // Up to as many sequences as CTAs: each sequence's rows are dealt out to all CTAs. More: whole
      // sequences are, so that no CTA reads every span again (4096 sequences, a third without keys:
      // 614 us with rows dealt out, 367 us with sequences).
      const int ctas = gridDim.x, me = blockIdx.x;
      const bool by_row = disorder || p.seq.B <= ctas;
      SpanFloor floor;
      const int lane_step = by_row ? 1 : ctas;
      const int seqs = disorder && p.seq.B > kMostScanned ? 0 : p.seq.B;
      if (disorder && lane == 0) set_status(p.status, MSA_ERR_BOUNDS);
      for (int64_t b0 = by_row ? 0 : me; b0 < seqs; b0 += 32 * lane_step) {
        const int64_t b = b0 + int64_t(lane) * lane_step;
        SeqSpan s{};
        int rows = 0;  // of the sequence, from its first on
        if (b < seqs) s = seq_span(p.seq, int(b));
        if (disorder) floor.apply(p.seq, s);
        if (b < seqs) {
          if (!s.ok) set_status(p.status, MSA_ERR_BOUNDS);
          if (s.rows_ok) rows = !s.ok || s.Lk == 0 ? s.Lq : s.Lk < s.Lq ? (s.Lq - s.Lk) / w2 * w2 : 0;
        }
        uint32_t some = __ballot_sync(0xffffffffu, rows > 0);
        for (; some; some &= some - 1) {
          const int src = __ffs(some) - 1;
          const int q0 = __shfl_sync(0xffffffffu, s.q0, src), cnt = __shfl_sync(0xffffffffu, rows, src);
          for (int r = by_row ? me : 0; r < cnt; r += by_row ? ctas : 1) {
            const int64_t row = int64_t(q0 + r) * p.Hq;
            uint4* dst = reinterpret_cast<uint4*>(p.out + row * D);
            for (int x = lane; x < p.Hq * (D / 8); x += 32) dst[x] = make_uint4(0, 0, 0, 0);
            if (p.lse)
              for (int x = lane; x < p.Hq; x += 32) p.lse[row + x] = -INFINITY;
          }
        }
      }
    }
  } else {
    // ------------------------------ softmax ------------------------------
    tc::regs_inc<kRegsMany>();
    const int w = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t sbase = tmem + (uint32_t(quarter * 32) << 16) + w * 128;
    const uint32_t obase = tmem + (uint32_t(quarter * 32) << 16) + kColO + w * D;
    const uint32_t stage = tc::smem_u32(pf_smem + SM::oStore + (warp - 4) * SM::kStore);
    const int row_tok = r / p.hpg, row_head = r % p.hpg;
    // Writes the warp's 32 rows: 64 columns at a time through shared memory, so
    // that 8 lanes store 128 contiguous bytes (a thread's own row alone would
    // make every store touch 32 sectors). get(c, o): the thread's columns [32 c, 32 c + 32).
    auto store_rows = [&](int64_t row, bool valid, float mul, bool some, auto get) {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float o[32];
          get(h * 2 + c, o);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t u[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              u[y] = some ? pack_bf16(o[x * 8 + 2 * y] * mul, o[x * 8 + 2 * y + 1] * mul) : 0u;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             stage + lane * 128 + (uint32_t((c * 4 + x) ^ (lane & 7)) << 4)),
                         "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3])
                         : "memory");
          }
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int rr = x * 4 + (lane >> 3), c = lane & 7;
          const int64_t to = __shfl_sync(0xffffffffu, valid ? row : int64_t(-1), rr);
          uint4 u;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                       : "r"(stage + rr * 128 + (uint32_t(c ^ (rr & 7)) << 4))
                       : "memory");
          if (to >= 0) reinterpret_cast<uint4*>(p.out + to * D + h * 64)[c] = u;
        }
        __syncwarp();
      }
    };
    bool ok = true;
    int z = 0, used = 0, splits = 0;
    for (int it = 0; ok; ++it) {
      if (!(ok = warp_wait(&item_full[it % NI], (it / NI) & 1, abort_flag))) break;
      const PfItem* sp = items + it % NI;
      const int n = sp->n, mode = sp->mode, jb = sp->jb, off = sp->Lk - sp->Lq;
      const int first = sp->i0 + w * p.tpt, i = first + row_tok;  // the tile's and this row's token
      const bool valid = r < p.tpt * p.hpg && i < sp->i1;
      const int64_t row = int64_t(sp->q0 + i) * p.Hq + sp->g * p.hpg + row_head;
      const int c0 = sp->c0, parts = sp->parts, slot = sp->slot;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&item_empty[it % NI]);
      if (mode == 3) break;
      float m = -INFINITY, l = 0.f;
      if (mode == 2) {
        store_rows(row, valid, 0.f, false, [](int, float(&o)[32]) {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0.f;
        });
        if (valid && p.lse) p.lse[row] = -INFINITY;
        continue;
      }
      const int vis = off + i + 1;  // keys this row sees
      // a row without any is 0; one whose scores are all -inf divides 0 by 0, as its formula does
      const bool some = vis > 0;
      const int j_mask = max(off + first + 1, 0) / kKeys;  // tiles below it are seen whole by every row of the tile
      for (int j = jb; j < jb + n; ++j, ++z) {
        if (!(ok = warp_wait(&s_full[w], z & 1, abort_flag))) break;
        tc::fence_after_sync();
        // O follows a raised maximum: S(j) is complete, so is the product before it, and O is at rest
        auto raise = [&](float mt) {
          if (j == jb) {
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
        if (j < j_mask) {  // every row sees the whole tile
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
          // the causal edge, 32 columns at a time; those that no row of the warp sees are only zeroed
          const int lim = vis - j * kKeys;  // columns below it are seen
          const int chunks = (__reduce_max_sync(0xffffffffu, min(max(valid ? lim : 0, 0), kKeys)) + 31) >> 5;
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
      if (!ok || !(ok = warp_wait(&o_full[w], used & 1, abort_flag))) break;
      ++used;
      tc::fence_after_sync();
      auto from_tmem = [&](int c, float(&o)[32]) {
        tc::tmem_ld_32x32b_x32(obase + c * 32, reinterpret_cast<uint32_t*>(o));
        tc::tmem_ld_wait();
      };
      auto release = [&]() {  // the next item's products may go over O
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&o_empty[w]);
      };
      if (mode == 0) {
        store_rows(row, valid, some ? 1.f / l : 0.f, some, from_tmem);
        release();
        if (valid && p.lse) p.lse[row] = some ? (m + log2f(l)) * kLn2f : -INFINITY;
        continue;
      }
      // ---- part of a split item: leave it, and join all parts if it is the last to arrive ----
      const int pr = w * kRows + r;  // row of the partial
      float4* po = reinterpret_cast<float4*>(p.part) + int64_t(slot) * (D / 4) * 256 + pr;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        from_tmem(c, o);
#pragma unroll
        for (int x = 0; x < 8; ++x)
          po[(c * 8 + x) * 256] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
      }
      p.stat[int64_t(slot) * 256 + pr] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(part_bar);
      if (warp == 4) {
        if (!(ok = warp_wait(part_bar, splits & 1, abort_flag))) break;
        if (lane == 0) {
          // one byte per CTA; releases the CTA's partial, acquires the others'
          const int sh = 8 * (c0 & 3);
          uint32_t old;
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
                       : "=r"(old)
                       : "l"(p.arrivals + (c0 >> 2)), "r"(1u << sh)
                       : "memory");
          const bool all = int((old >> sh) & 0xffu) == parts - 1;
          *last_flag = all;
          if (all) atomicSub(p.arrivals + (c0 >> 2), uint32_t(parts) << sh);  // ready for the next call
          tc::mbar_arrive(flag_bar);
        }
        __syncwarp();
      }
      if (!(ok = warp_wait(flag_bar, splits & 1, abort_flag))) break;
      ++splits;
      const bool last = *last_flag != 0;
      // everybody has read the flag before the next split item's can be set: that one waits for all partials
      if (!last) {
        release();
        continue;
      }
      // the parts are those of consecutive CTAs from c0 on, in the order of the keys
      auto slot_of = [&](int y) { return int64_t(2 * (c0 + y) + (y == 0 ? 1 : 0)); };
      float M = -INFINITY, den = 0.f;
      for (int y0 = 0; y0 < parts; y0 += 4) {
        float2 ml[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) ml[y] = __ldcg(p.stat + slot_of(min(y0 + y, parts - 1)) * 256 + pr);
        const float mn = fmaxf(tc::fmax3(ml[0].x, ml[1].x, ml[2].x), fmaxf(ml[3].x, M));
        den *= M == mn ? 1.f : ex2(M - mn);
        M = mn;
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (y0 + y < parts) den = fmaf(ml[y].x == M ? 1.f : ex2(ml[y].x - M), ml[y].y, den);
      }
      float acc[D];
#pragma unroll
      for (int x = 0; x < D; ++x) acc[x] = 0.f;
      for (int y = 0; y < parts; ++y) {
        const float mx = __ldcg(p.stat + slot_of(y) * 256 + pr).x, a = mx == M ? 1.f : ex2(mx - M);
        if (slot_of(y) == slot) {  // this CTA's own part is still in TMEM
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            from_tmem(c, o);
#pragma unroll
            for (int x = 0; x < 32; ++x) acc[c * 32 + x] = fmaf(a, o[x], acc[c * 32 + x]);
          }
        } else {
          const float4* src = reinterpret_cast<const float4*>(p.part) + slot_of(y) * (D / 4) * 256 + pr;
#pragma unroll
          for (int x0 = 0; x0 < D / 4; x0 += 16) {
            float4 f[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) f[x] = __ldcg(src + (x0 + x) * 256);
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const int e = 4 * (x0 + x);
              acc[e] = fmaf(a, f[x].x, acc[e]);
              acc[e + 1] = fmaf(a, f[x].y, acc[e + 1]);
              acc[e + 2] = fmaf(a, f[x].z, acc[e + 2]);
              acc[e + 3] = fmaf(a, f[x].w, acc[e + 3]);
            }
          }
        }
      }
      store_rows(row, valid, some ? 1.f / den : 0.f, some, [&](int c, float(&o)[32]) {
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = acc[c * 32 + x];
      });
      release();
      if (valid && p.lse) p.lse[row] = some ? (M + log2f(den)) * kLn2f : -INFINITY;
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

size_t pf_part_bytes(int d) { return size_t(2) * kNumSMs * 256 * d * sizeof(float); }
// Whether some item may be split: its keys are the packed ones, or those a table row holds.
bool pf_splits(int64_t most_keys) { return most_keys > kPfWhole; }

template <int D>
cudaError_t prefill(const FullArgs& a, cudaStream_t stream) {
  PfParams p{};
  p.seq = a.seq;
  p.pages = a.pages;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.hpg = a.Hq / a.Hkv;
  p.tpt = kRows / p.hpg;
  p.nslots = a.seq.Tq / (2 * p.tpt) + a.seq.B;
  p.scale_log2 = a.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  WsHeader* header = static_cast<WsHeader*>(a.ws);
  p.status = &header->status;
  p.arrivals = header->arrivals;
  p.queue = &header->queue;
  p.inject_timeout = debug_inject_timeout() ? 1 : 0;
  if (int64_t(p.nslots) * a.Hkv >= (int64_t(1) << 30)) return cudaErrorInvalidValue;
  if (pf_splits(a.seq.Tk)) {
    char* w = static_cast<char*>(a.ws) + kWsHeader;
    p.part = reinterpret_cast<float*>(w);
    p.stat = reinterpret_cast<float2*>(w + pf_part_bytes(D));
  }
  const bool paged = a.pages.table != nullptr;
  const uint64_t krows = paged ? uint64_t(a.pages.num_pages) << a.pages.page_log2 : uint64_t(a.seq.Tk);
  const int box = paged ? 1 << a.pages.page_log2 : kKeys;
  CUtensorMap tmQ, tmK, tmV;
  if (!map_rows(&tmQ, a.q, a.seq.Tq, a.Hq, a.Hkv, D, p.tpt) || !map_keys(&tmK, a.k, krows, a.Hkv, D, box) ||
      !map_keys(&tmV, a.v, krows, a.Hkv, D, box))
    return cudaErrorInvalidValue;
  auto kern = full_prefill_kernel<D>;
  constexpr int bytes = int(PfSmem<D>::kTotal);
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  // a launch with other registers could not cover the warpgroups' shares
  static KernelReady ready;
  if (cudaError_t e = ready.on_device(reinterpret_cast<const void*>(kern), bytes, int(kRegsLaunch))) return e;
  ProfScope pf("full_prefill", stream);
  kern<<<kNumSMs, kPfThreads, bytes, stream>>>(tmQ, tmK, tmV, p);
  return cudaGetLastError();
}

}  // namespace

size_t full_prefill_ws_bytes(int d, int64_t most_keys) {
  return pf_splits(most_keys) ? pf_part_bytes(d) + size_t(2) * kNumSMs * 256 * sizeof(float2) : 0;
}

cudaError_t launch_full_prefill_tc(const FullArgs& a, cudaStream_t stream) {
  return a.d == 128 ? prefill<128>(a, stream) : prefill<64>(a, stream);
}

}  // namespace msa
