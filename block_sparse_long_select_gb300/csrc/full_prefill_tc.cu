// Full attention, prefill, bf16 on tcgen05 (sm_103a): causal attention of
// packed query rows over packed or paged keys.
//
//   out_i = sum_j exp(s_ij - lse_i) v_j,  s_ij = scale q_i . k_j,  j <= Lk - Lq + i
//
// One CTA takes 2 x kRows rows of one (sequence, key/value head) and walks its
// keys in tiles of 128. A row tile is 128 / hpg consecutive tokens x the hpg
// query heads that share the key/value head, token by token, so short
// sequences and chunks fill the 128 rows of an MMA, the causal edge is cut at
// 128 / hpg tokens, and one K/V tile serves every head of the group.
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
// Bound: the tensor cores (4 Hq d FLOPs per visible pair).
//
// Warps: 0 loads (TMA; zeroes the value rows behind a sequence's end, which
// may hold anything), 1 MMA issue and TMEM, 4-7 and 8-11 the two softmax
// warpgroups, one thread per row. Every wait is bounded.
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

struct PfParams {
  SeqMap seq;
  PageMap pages;
  int Hq, Hkv, hpg, tpt, nslots;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
};

template <int D>
struct PfSmem {
  static constexpr int kStages = D == 128 ? 2 : 4;   // K ring and V ring
  static constexpr uint32_t kTile = kRows * D * 2;
  static constexpr uint32_t oQ = 0, oK = 2 * kTile, oV = oK + kStages * kTile, oBar = oV + kStages * kTile;
  static constexpr int kBars = 2 + 4 * kStages + 2 + 4 + 2 + 1 + 1;
  static constexpr uint32_t oStat = (oBar + kBars * 8 + 16 + 15) & ~15u;
  static constexpr uint32_t kTotal = oStat + 2 * kRows * 8;
  static_assert(2 * kRows * D * 4 <= oBar, "the partial fits where the operands were");
};

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1)
    full_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const PfParams p) {
  using SM = PfSmem<D>;
  constexpr int NH = D / 64, NS = SM::kStages;
  constexpr uint32_t kIdS = tc::idesc_bf16_f32(kRows, kKeys);
  constexpr uint32_t kIdO = tc::idesc_bf16_f32(kRows, D, true);  // B = V, MN-major
  constexpr uint32_t kColO = 256;
  extern __shared__ __align__(1024) uint8_t pf_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (tc::smem_u32(pf_smem) & 1023u) {  // the swizzled operands need 1024-byte alignment
    if (threadIdx.x == 0) set_status(p.status, MSA_ERR_CUDA);
    return;
  }

  // ---- which rows: heavy (late) tiles of a sequence first ----
  const int cl = cluster_size(), rank = cluster_rank(), work = blockIdx.x / cl;
  const int g = work % p.Hkv;
  int tile;
  const int b = find_slot_tile(p.seq.cu_q, p.seq.B, 2 * p.tpt, p.nslots - 1 - work / p.Hkv, tile);
  if (b < 0) return;
  const SeqSpan s = seq_span(p.seq, b);
  if (!s.rows_ok) {
    if (threadIdx.x == 0) set_status(p.status, MSA_ERR_BOUNDS);
    return;
  }
  const int i0 = tile * 2 * p.tpt;                  // first row (token) of the CTA within the sequence
  const int i1 = min(i0 + 2 * p.tpt, s.Lq);         // behind the last
  bool bad = !s.ok;
  if (!bad && p.pages.table) {  // every page of the sequence in range, for all its rows alike
    const int32_t* row = p.pages.table + int64_t(b) * p.pages.max_pages;
    const int np = (s.Lk + (1 << p.pages.page_log2) - 1) >> p.pages.page_log2;
    for (int x = threadIdx.x; x < np; x += kPfThreads) bad |= row[x] < 0 || row[x] >= p.pages.num_pages;
  }
  bad = __syncthreads_or(bad);
  const int vis_last = bad ? 0 : s.Lk - s.Lq + i1;  // keys the last row sees
  const int tiles = vis_last > 0 ? (vis_last + kKeys - 1) / kKeys : 0;
  if (tiles == 0) {  // no row sees a key
    if (bad && threadIdx.x == 0) set_status(p.status, MSA_ERR_BOUNDS);
    if (rank > 0) return;
    const int chunks = (i1 - i0) * p.hpg * (D / 8);
    for (int x = threadIdx.x; x < chunks; x += kPfThreads) {
      const int r = x / (D / 8), tok = s.q0 + i0 + r / p.hpg, h = g * p.hpg + r % p.hpg;
      const int64_t row = int64_t(tok) * p.Hq + h;
      reinterpret_cast<uint4*>(p.out + row * D)[x % (D / 8)] = make_uint4(0, 0, 0, 0);
      if (p.lse && x % (D / 8) == 0) p.lse[row] = -INFINITY;
    }
    return;
  }

  // this CTA's key tiles [jb, jb + n)
  const int jb = int(int64_t(tiles) * rank / cl), n = int(int64_t(tiles) * (rank + 1) / cl) - jb;

  uint64_t* bars = reinterpret_cast<uint64_t*>(pf_smem + SM::oBar);
  uint64_t* q_full = bars;             // [2]
  uint64_t* k_full = bars + 2;         // [NS]
  uint64_t* k_empty = k_full + NS;     // [NS]
  uint64_t* v_full = k_empty + NS;     // [NS]
  uint64_t* v_empty = v_full + NS;     // [NS]
  uint64_t* s_full = v_empty + NS;     // [2]
  uint64_t* p_full = s_full + 2;       // [2][2]: row tile, half of the keys
  uint64_t* o_full = p_full + 4;       // [2]
  uint64_t* tail_bar = o_full + 2;     // the copies of a value tile whose last rows are then zeroed
  uint64_t* done_bar = tail_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + SM::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float2* stats = reinterpret_cast<float2*>(pf_smem + SM::oStat);  // [2][128] maximum, sum (clusters only)
  if (threadIdx.x == 0) {
    for (int x = 0; x < SM::kBars; ++x) tc::mbar_init(bars + x, 1);
    for (int x = 0; x < 4; ++x) tc::mbar_init(p_full + x, 4);
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
    const int np = paged ? (s.Lk + psz - 1) >> p.pages.page_log2 : 0;
    const int32_t* table = paged ? p.pages.table + int64_t(b) * p.pages.max_pages : nullptr;
    auto first_row = [&](int j) {  // this lane's box of tile j: its first row, -1 if it has none
      if (!paged) return lane == 0 ? s.k0 + (jb + j) * kKeys : -1;
      const int pi = (jb + j) * per + lane;
      return lane < per && pi < np ? table[pi] << p.pages.page_log2 : -1;
    };
    auto boxes = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int row) {
      const int cnt = __popc(__ballot_sync(0xffffffffu, row >= 0));
      if (lane == 0) tc::mbar_arrive_expect_tx(bar, uint32_t(cnt * box_rows) * D * 2);
      __syncwarp();
      if (row >= 0) {
#pragma unroll
        for (int h = 0; h < NH; ++h)
          tc::tma_load_3d(dst + h * kHalfTile + lane * box_rows * 128, map, bar, h * 64, g, row);
      }
    };
    auto load_q = [&](int w) {
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(&q_full[w], uint32_t(p.tpt * p.hpg) * D * 2);
#pragma unroll
        for (int h = 0; h < NH; ++h)
          tc::tma_load_4d(pf_smem + SM::oQ + w * SM::kTile + h * kHalfTile, &tmQ, &q_full[w], h * 64, 0, g,
                          s.q0 + i0 + w * p.tpt);
      }
    };
    int row = first_row(0);
    bool ok = true;
    int nk = 0, nv = 0, tails = 0;
    if (n > 0) load_q(0);
    for (int j = 0; j < n && ok; ++j) {
      const int st = j % NS, ph = (j / NS) & 1;
      const int next = j + 1 < n ? first_row(j + 1) : -1;  // in flight while this tile is issued
      if (!(ok = warp_wait(&k_empty[st], ph ^ 1, abort_flag))) break;
      boxes(pf_smem + SM::oK + st * SM::kTile, &tmK, &k_full[st], row);
      ++nk;
      if (j == 0) load_q(1);
      if (!(ok = warp_wait(&v_empty[st], ph ^ 1, abort_flag))) break;
      uint8_t* vt = pf_smem + SM::oV + st * SM::kTile;
      const int valid = s.Lk - (jb + j) * kKeys;
      if (valid >= kKeys) {
        boxes(vt, &tmV, &v_full[st], row);
        ++nv;
      } else {
        // rows behind the sequence's end belong to others: weight 0 does not
        // silence an infinity or NaN there, so they become zeros
        boxes(vt, &tmV, tail_bar, row);
        ++tails;
        if (!(ok = warp_wait(tail_bar, 0, abort_flag))) break;
        zero_rows<NH>(vt, valid, kKeys);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&v_full[st]);
      }
      row = next;
    }
    if (!ok) {  // let the copies land before the CTA gives its shared memory up
      fail();
      int zero = 0;
      tc::mbar_wait(&q_full[0], 0, &zero);  // n > 0 here
      if (nk > 0) tc::mbar_wait(&q_full[1], 0, &zero);
      for (int x = max(nk - NS, 0); x < nk; ++x) tc::mbar_wait(&k_full[x % NS], (x / NS) & 1, &zero);
      for (int x = max(nv - NS, 0); x < nv; ++x) tc::mbar_wait(&v_full[x % NS], (x / NS) & 1, &zero);
      if (tails) tc::mbar_wait(tail_bar, 0, &zero);
    }
  } else if (warp == 1) {
    // ----------------------------- MMA issue -----------------------------
    if (lane == 0 && n > 0) {
      constexpr uint32_t kHi = tc::smem_desc_hi(1024, 2);
      const uint32_t qa = tc::smem_desc_lo(tc::smem_u32(pf_smem + SM::oQ), 16);
      const uint32_t ka = tc::smem_desc_lo(tc::smem_u32(pf_smem + SM::oK), 16);
      const uint32_t va = tc::smem_desc_lo(tc::smem_u32(pf_smem + SM::oV), kHalfTile);
      auto scores = [&](int w, int j) {  // S_w = Q_w K_j^T
        const uint32_t q0 = qa + ((w * SM::kTile) >> 4), k0 = ka + (((j % NS) * SM::kTile) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kHalfTile + (kk & 3) * 32) >> 4;
          tc::mma_f16_ss_lo<kHi>(tmem + w * 128, q0 + off, k0 + off, kIdS, kk > 0 ? 1u : 0u);
        }
        tc::mma_commit(&s_full[w]);
      };
      auto values = [&](int w, int j, int half) {  // O_w += P_w V_j over half of the keys
        const uint32_t v0 = va + (((j % NS) * SM::kTile) >> 4);
#pragma unroll
        for (int x = 0; x < kKeys / 32; ++x) {
          const int kk = half * (kKeys / 32) + x;
          tc::mma_f16_ts_lo<kHi>(tmem + kColO + w * D, tmem + w * 128 + kk * 8, v0 + ((kk * 16 * 128) >> 4), kIdO,
                                 (j > 0 || kk > 0) ? 1u : 0u);
        }
      };
      bool ok = tc::mbar_wait(&q_full[0], 0, abort_flag) && tc::mbar_wait(&k_full[0], 0, abort_flag);
      if (ok) {
        tc::fence_after_sync();
        scores(0, 0);
        ok = tc::mbar_wait(&q_full[1], 0, abort_flag);
      }
      if (ok) {
        scores(1, 0);
        tc::mma_commit(&k_empty[0]);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int st = j % NS, ph = (j / NS) & 1;
        if (!(ok = tc::mbar_wait(&v_full[st], ph, abort_flag))) break;
        const int st1 = (j + 1) % NS, ph1 = ((j + 1) / NS) & 1;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          // the first half's product runs while the softmax forms the second half
          if (!(ok = tc::mbar_wait(&p_full[2 * w], j & 1, abort_flag))) break;
          tc::fence_after_sync();
          values(w, j, 0);
          if (!(ok = tc::mbar_wait(&p_full[2 * w + 1], j & 1, abort_flag))) break;
          tc::fence_after_sync();
          values(w, j, 1);
          if (w == 1) tc::mma_commit(&v_empty[st]);
          if (j + 1 < n) {
            // in issue order behind the product that reads P: S may go over it
            if (w == 0 && !(ok = tc::mbar_wait(&k_full[st1], ph1, abort_flag))) break;
            scores(w, j + 1);
            if (w == 1) tc::mma_commit(&k_empty[st1]);
          } else {
            tc::mma_commit(&o_full[w]);
          }
        }
      }
      if (!ok) fail();
      int zero = 0;
      tc::mma_commit(done_bar);
      tc::mbar_wait(done_bar, 0, &zero);
    }
  }
  } else {
    // ------------------------------ softmax
    tc::regs_inc<kRegsMany>();
    const int w = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t sbase = tmem + (uint32_t(quarter * 32) << 16) + w * 128;
    const uint32_t obase = tmem + (uint32_t(quarter * 32) << 16) + kColO + w * D;
    const int i = i0 + w * p.tpt + r / p.hpg;  // this row's token within the sequence
    const bool valid = r < p.tpt * p.hpg && i < i1;
    const int vis = s.Lk - s.Lq + i + 1;       // keys it sees
    // tiles below j_mask are seen whole by every row of the tile (its first sees least)
    const int j_mask = max(s.Lk - s.Lq + i0 + w * p.tpt + 1, 0) / kKeys - jb;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!(ok = warp_wait(&s_full[w], j & 1, abort_flag))) break;
      tc::fence_after_sync();
      uint32_t v[kKeys];
      float mx;
      if (j < j_mask) {
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) m4[c] = tc::tmem_ld_max_32x32b_x32(sbase + c * 32, v + c * 32);
        tc::tmem_ld_wait();
        mx = fmaxf(tc::fmax3(m4[0], m4[1], m4[2]), m4[3]);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld_32x32b_x32(sbase + c * 32, v + c * 32);
        tc::tmem_ld_wait();
        const int lim = vis - (jb + j) * kKeys;
        mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) {
          if (c >= lim) v[c] = 0xff800000u;  // -inf
          mx = fmaxf(mx, __uint_as_float(v[c]));
        }
      }
      const float mt = mx * p.scale_log2;
      if (j == 0) {
        m = mt;
      } else if (__any_sync(0xffffffffu, mt > m + kLazy)) {
        // S(j) is complete, so is the product before it: O is at rest
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
      const float neg = m == -INFINITY ? 0.f : -m;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float p0 = ex2(fmaf(__uint_as_float(v[c * 64 + 2 * x]), p.scale_log2, neg));
          const float p1 = ex2(fmaf(__uint_as_float(v[c * 64 + 2 * x + 1]), p.scale_log2, neg));
          v[c * 64 + x] = __float_as_uint(p0 + p1);
          pk[x] = pack_bf16(p0, p1);
        }
        tc::tmem_st_32x32b_x32(sbase + c * 32, pk);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[2 * w + c]);
      }
      // the sum, off the tensor cores' path
      float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int x = 0; x < 32; ++x) l4[x & 3] += __uint_as_float(v[c * 64 + x]);
      l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
    }
    if (ok && n > 0) {
      ok = warp_wait(&o_full[w], 0, abort_flag);
      // a partial goes where the operands were: the other tile's products have to be done, too
      if (ok && cl > 1) ok = warp_wait(&o_full[w ^ 1], 0, abort_flag);
    }
    if (!ok) fail();
    if (ok && cl > 1) {
      tc::fence_after_sync();
      const uint32_t part = tc::smem_u32(pf_smem);
      if (n > 0) put_partial<D>(part, w * kRows + r, 0, obase, D);
      stats[w * kRows + r] = n > 0 ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
    } else if (ok) {
      tc::fence_after_sync();
      const int64_t row = int64_t(s.q0 + i) * p.Hq + g * p.hpg + r % p.hpg;
      const bool some = l > 0.f || l != l;
      const float inv = some ? 1.f / l : 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tc::tmem_ld_32x32b_x32(obase + c * 32, o);
        tc::tmem_ld_wait();
        if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + row * D + c * 32);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t u[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float a = __uint_as_float(o[x * 8 + 2 * y]) * inv, c2 = __uint_as_float(o[x * 8 + 2 * y + 1]) * inv;
              u[y] = some ? pack_bf16(a, c2) : 0u;
            }
            dst[x] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
      }
      if (valid && p.lse) p.lse[row] = some ? (m + log2f(l)) * kLn2f : -INFINITY;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  if (cl == 1) return;
  // ---- the ranks' partials of the 256 rows, a slice of rows per rank ----
  cluster_sync();
  const uint32_t part = tc::smem_u32(pf_smem), stat = tc::smem_u32(stats);
  const int per = 2 * kRows / cl;
  // the softmax warpgroups, which have the registers
  for (int x = int(threadIdx.x) - 128; x >= 0 && x < per * (D / 8); x += 256) {
    const int r = rank * per + x / (D / 8), c = x % (D / 8), w = r / kRows, rr = r % kRows;
    const int i = i0 + w * p.tpt + rr / p.hpg;
    if (rr >= p.tpt * p.hpg || i >= i1) continue;
    float M = -INFINITY, den = 0.f, o[8] = {};
    for (int y = 0; y < cl; ++y) M = fmaxf(M, ld_peer2(peer_addr(stat + r * 8, y)).x);
    for (int y = 0; y < cl; ++y) {
      const float2 ml = ld_peer2(peer_addr(stat + r * 8, y));
      if (!(ml.y > 0.f) && ml.y == ml.y) continue;  // no key there (its partial may hold nothing)
      const float a = ml.x == M ? 1.f : ex2(ml.x - M);
      const float4 u = ld_peer4(peer_addr(part_at<D>(part, r, 2 * c), y));
      const float4 v = ld_peer4(peer_addr(part_at<D>(part, r, 2 * c + 1), y));
      den = fmaf(a, ml.y, den);
      o[0] = fmaf(a, u.x, o[0]), o[1] = fmaf(a, u.y, o[1]), o[2] = fmaf(a, u.z, o[2]), o[3] = fmaf(a, u.w, o[3]);
      o[4] = fmaf(a, v.x, o[4]), o[5] = fmaf(a, v.y, o[5]), o[6] = fmaf(a, v.z, o[6]), o[7] = fmaf(a, v.w, o[7]);
    }
    const bool some = den > 0.f || den != den;
    const float inv = some ? 1.f / den : 0.f;
    const int64_t row = int64_t(s.q0 + i) * p.Hq + g * p.hpg + rr % p.hpg;
    reinterpret_cast<uint4*>(p.out + row * D)[c] =
        make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                   pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
    if (p.lse && c == 0) p.lse[row] = some ? (M + log2f(den)) * kLn2f : -INFINITY;
  }
  cluster_sync();  // nobody leaves while its partial is read
}

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
  p.status = &static_cast<WsHeader*>(a.ws)->status;
  const bool paged = a.pages.table != nullptr;
  const uint64_t krows = paged ? uint64_t(a.pages.num_pages) << a.pages.page_log2 : uint64_t(a.seq.Tk);
  const int box = paged ? 1 << a.pages.page_log2 : kKeys;
  CUtensorMap tmQ, tmK, tmV;
  if (!map_rows(&tmQ, a.q, a.seq.Tq, a.Hq, a.Hkv, D, p.tpt) || !map_keys(&tmK, a.k, krows, a.Hkv, D, box) ||
      !map_keys(&tmV, a.v, krows, a.Hkv, D, box))
    return cudaErrorInvalidValue;
  const int64_t ctas = int64_t(p.nslots) * a.Hkv;
  // a launch with other registers could not cover the warpgroups' shares
  cudaFuncAttributes fa;
  if (cudaError_t e = cudaFuncGetAttributes(&fa, full_prefill_kernel<D>)) return e;
  if (fa.numRegs != int(kRegsLaunch)) return cudaErrorInvalidConfiguration;
  ProfScope pf("full_prefill", stream);
  return launch_clusters(full_prefill_kernel<D>, ctas, cluster_split(ctas, (int64_t(a.seq.Tk) + kKeys - 1) / kKeys),
                         kPfThreads, int(PfSmem<D>::kTotal), stream, tmQ, tmK, tmV, p);
}

}  // namespace

cudaError_t launch_full_prefill_tc(const FullArgs& a, cudaStream_t stream) {
  return a.d == 128 ? prefill<128>(a, stream) : prefill<64>(a, stream);
}

}  // namespace msa
