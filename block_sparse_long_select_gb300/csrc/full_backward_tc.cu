// Full attention, backward, bf16 on tcgen05 (sm_103a), packed sequences:
//   P_ij = exp(s_ij - lse_i),  delta_i = dout_i . out_i
//   dS_ij = P_ij (dout_i . v_j - delta_i)
//   dv_j = sum_i P_ij dout_i;  dk_j = scale sum_i dS_ij q_i;  dq_i = scale sum_j dS_ij k_j
//
// Two kinds of CTAs in one launch, each of which owns what it sums, so that
// nothing is added atomically and every run gives the same bits: dk and dv per
// key tile over the rows that see it, dq per row tile over the keys it sees. That is seven
// products per tile pair instead of the five that one kernel with atomic dq
// sums would take; the order of its sums would change from run to run, and
// each pair would send 64 KB of fp32 adds to L2. Row tiles are 128 / hpg tokens x
// the hpg heads of a group, as in the forward: the sum over a group's heads is
// part of the product.
//
// Bound: the tensor cores. Both kinds split their epilogue in two so that the
// tensor cores work through it: from the scores to P (kept in registers) while
// the products of the tile before and dP run, then from dP to dS while the next
// scores run. P and dS are rounded to bf16 for the products that read them
// (2^-8 each, averaging out over the sums); sums stay in fp32.
//
// Measured (Hq 32, Hkv 8, d 128): 8192 tokens 1.38 ms in a loop (73 % of the
// measured tensor rate on the seven products, 52 % on five).
//
// Warps of both: 0 loads (TMA; zeroes rows of other sequences, whose
// infinities a weight of 0 would not silence), 1 MMA issue and TMEM, 4-11
// epilogue: two threads per TMEM lane, 64 columns each. dkv: 2-3 fetch the
// rows' lse and delta. Every wait is bounded.
#include <type_traits>

#include "full_tc.cuh"

namespace msa {
namespace {

constexpr int kFbThreads = 384;

struct FbParams {
  SeqMap seq;
  int Hq, Hkv, hpg, tpt, kslots, qslots;
  float scale, scale_log2;
  const float2* rows;  // [Hkv][Tq][hpg]: lse in log2 units, delta (full_common.cu)
  __nv_bfloat16 *dq, *dk, *dv;
  uint32_t* status;
  const uint32_t* disorder;
  int inject_timeout;  // test hook: every second CTA waits on a barrier nothing completes
};

template <int D>
struct FbSmem {
  static constexpr uint32_t kTile = 128 * D * 2;
  static constexpr int kRowSlots = 4;  // row data of four tiles (dkv)
  // two resident tiles, then a ring of two slots for each of two streamed operands
  static constexpr uint32_t oA = 0, oB = kTile, oC = 2 * kTile, oE = 4 * kTile, oRow = 6 * kTile;
  static constexpr uint32_t oBar = oRow + kRowSlots * 2 * kRows * 4;
  static constexpr int kBars = 1 + 8 + 4 + 2 * kRowSlots + 4;
  static constexpr uint32_t kTotal = oBar + kBars * 8 + 16;
};
struct FbBars {
  uint64_t *res_full, *c_full, *c_empty, *e_full, *e_empty, *s_full, *p_full, *dp_full, *ds_full, *r_full, *r_empty,
      *acc_full, *tail, *done, *never;
  __device__ __forceinline__ FbBars(uint64_t* b, int slots) {
    res_full = b;
    c_full = b + 1;
    c_empty = b + 3;
    e_full = b + 5;
    e_empty = b + 7;
    s_full = b + 9;
    p_full = b + 10;
    dp_full = b + 11;
    ds_full = b + 12;
    r_full = b + 13;
    r_empty = r_full + slots;
    acc_full = r_empty + slots;
    tail = acc_full + 1;
    done = tail + 1;
    never = done + 1;  // no thread arrives on it (timeout injection)
  }
  // One thread per barrier (of `bars`, from b on). 8 epilogue warps hand over P,
  // dS and the row data's slots, 2 warps fill those; else one arrival.
  __device__ __forceinline__ void init(uint64_t* b, int slots, int bars) const {
    if (threadIdx.x >= bars) return;
    const uint64_t* x = b + threadIdx.x;
    const bool by_epilogue = x == p_full || x == ds_full || (x >= r_empty && x < r_empty + slots);
    tc::mbar_init(b + threadIdx.x, by_epilogue ? 8 : x >= r_full && x < r_full + slots ? 2 : 1);
    tc::fence_barrier_init();
  }
};

// bf16 pairs of 64 columns go over the first half of the 64 columns they came
// from, so neither epilogue warpgroup writes where the other still reads.
__device__ __forceinline__ uint32_t a_col(int kk) { return uint32_t((kk >> 2) * 64 + (kk & 3) * 8); }
// Walks of up to this many tiles keep what the rounding of dS to bf16 leaves off
// as a second bf16 term with a product of its own. With few terms to average
// over, the rounding can cost a gradient half of its last bit again; and here a
// product more costs nothing, the time is latency. Long walks would pay a
// quarter (dk) or a third (dq) more tensor work for an error that stays below
// that of rounding the result.
constexpr int kFineTiles = 4;
// 64 columns of dP become dS (in pr, by `make` 32 at a time) and go back over
// them: bf16 pairs in the first half, their remainders, if wanted, in the second.
template <typename F>
__device__ __forceinline__ void put_ds(uint32_t taddr, float (&pr)[64], bool fine, F make) {
  if (!fine) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t v[32], pk[16];
      tc::tmem_ld_32x32b_x32(taddr + c * 32, v);
      tc::tmem_ld_wait();
      make(c, v);
#pragma unroll
      for (int x = 0; x < 16; ++x) pk[x] = pack_bf16(pr[c * 32 + 2 * x], pr[c * 32 + 2 * x + 1]);
      tc::tmem_st_32x32b_x16(taddr + c * 16, pk);
    }
    return;
  }
  // the remainders go where the second half of dP is: all of it is read first
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t v[32];
    tc::tmem_ld_32x32b_x32(taddr + c * 32, v);
    tc::tmem_ld_wait();
    make(c, v);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t pk[16], lo[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const float a = pr[c * 32 + 2 * x], b = pr[c * 32 + 2 * x + 1];
      pk[x] = pack_bf16(a, b);
      lo[x] = pack_bf16(a - __uint_as_float(pk[x] << 16), b - __uint_as_float(pk[x] & 0xffff0000u));
    }
    tc::tmem_st_32x32b_x16(taddr + c * 16, pk);
    tc::tmem_st_32x32b_x16(taddr + 32 + c * 16, lo);
  }
}

template <int D>
__device__ __forceinline__ void store_acc(uint32_t taddr, int cols, __nv_bfloat16* dst, float mul, bool in) {
  for (int c = 0; c < cols; c += 32) {
    uint32_t o[32];
    tc::tmem_ld_32x32b_x32(taddr + c, o);
    tc::tmem_ld_wait();
    if (in) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t u[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          u[y] = pack_bf16(__uint_as_float(o[x * 8 + 2 * y]) * mul, __uint_as_float(o[x * 8 + 2 * y + 1]) * mul);
        reinterpret_cast<uint4*>(dst + c)[x] = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16* row, int c, const float (&o)[8], float mul) {
  reinterpret_cast<uint4*>(row)[c] =
      make_uint4(pack_bf16(o[0] * mul, o[1] * mul), pack_bf16(o[2] * mul, o[3] * mul),
                 pack_bf16(o[4] * mul, o[5] * mul), pack_bf16(o[6] * mul, o[7] * mul));
}
// This rank's slice of `rows` rows summed over the ranks that had tiles, in
// rank order: f(row, chunk of 8 columns, sums).
template <int D, typename F>
__device__ __forceinline__ void sum_partials(uint32_t part, int rows, int rank, int cl, int tiles, F f) {
  const int per = rows / cl;
  for (int x = threadIdx.x; x < per * (D / 8); x += kFbThreads) {
    const int r = rank * per + x / (D / 8), c = x % (D / 8);
    float o[8] = {};
    for (int y = 0; y < cl; ++y) {
      if (int64_t(tiles) * y / cl == int64_t(tiles) * (y + 1) / cl) continue;
      const float4 u = ld_peer4(peer_addr(part_at<D>(part, r, 2 * c), y));
      const float4 v = ld_peer4(peer_addr(part_at<D>(part, r, 2 * c + 1), y));
      o[0] += u.x, o[1] += u.y, o[2] += u.z, o[3] += u.w;
      o[4] += v.x, o[5] += v.y, o[6] += v.z, o[7] += v.w;
    }
    f(r, c, o);
  }
}

// ---------------------------------------------------------------------------------
// dk, dv of 128 keys of one (sequence, key/value head)
// TMEM: S^T [0, 128) (P^T over it), dP^T [128, 256) (dS^T over it), dV, dK
// ---------------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void bwd_dkv(const CUtensorMap& tmQ, const CUtensorMap& tmO, const CUtensorMap& tmK,
                                        const CUtensorMap& tmV, const FbParams& p, bool in_order, uint8_t* fb_smem,
                                        int work, int cl, int rank) {
  using SM = FbSmem<D>;
  constexpr int NH = D / 64, NR = SM::kRowSlots;
  constexpr uint32_t kIdS = tc::idesc_bf16_f32(128, 128), kIdA = tc::idesc_bf16_f32(128, D, true);
  constexpr uint32_t kColDv = 256, kColDk = 256 + D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = work % p.Hkv;
  int kt;
  SeqSpan s;
  const int b = find_tile(p.seq, in_order, true, kKeys, 1, work / p.Hkv, kt, s);  // early keys: most rows
  if (b < 0) return;
  const int j0 = kt * kKeys;
  const int off = s.Lk - s.Lq;              // row i sees keys j <= off + i
  const int rf = max(j0 - off, 0) / p.tpt;  // first row tile that sees one of these keys
  const int tiles = s.ok ? max((s.Lq + p.tpt - 1) / p.tpt - rf, 0) : 0;
  if (tiles == 0) {  // no row sees them
    if (rank > 0) return;
    for (int x = threadIdx.x; x < min(kKeys, s.Lk - j0) * (D / 8); x += kFbThreads) {
      const int64_t o = ((int64_t(s.k0) + j0 + x / (D / 8)) * p.Hkv + g) * (D / 8) + x % (D / 8);
      reinterpret_cast<uint4*>(p.dk)[o] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(p.dv)[o] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  // this CTA's row tiles [r0, r0 + n)
  const int r0 = rf + int(int64_t(tiles) * rank / cl), n = rf + int(int64_t(tiles) * (rank + 1) / cl) - r0;
  const bool fine = tiles <= kFineTiles;
  uint64_t* bars = reinterpret_cast<uint64_t*>(fb_smem + SM::oBar);
  const FbBars bar(bars, NR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + SM::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* rowd = reinterpret_cast<float*>(fb_smem + SM::oRow);  // slot x: -lse2 [128], -delta [128]
  bar.init(bars, NR, SM::kBars);
  if (threadIdx.x == 0) *abort_flag = 0;
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

  if (warp == 0) {
    // ------------------------------ loads ------------------------------
    const int rows = p.tpt * p.hpg;
    if (rows < kRows) {  // rows that no box fills: zero for good
#pragma unroll
      for (int x = 0; x < 4; ++x) zero_rows<NH>(fb_smem + SM::oC + x * SM::kTile, rows, kRows);
      tc::fence_proxy_async_smem();
      __syncwarp();
    }
    auto keys = [&]() {
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(bar.res_full, 2 * SM::kTile);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          tc::tma_load_3d(fb_smem + SM::oA + h * kHalfTile, &tmK, bar.res_full, h * 64, g, s.k0 + j0);
          tc::tma_load_3d(fb_smem + SM::oB + h * kHalfTile, &tmV, bar.res_full, h * 64, g, s.k0 + j0);
        }
      }
    };
    auto box = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* full, int tok) {
#pragma unroll
      for (int h = 0; h < NH; ++h) tc::tma_load_4d(dst + h * kHalfTile, map, full, h * 64, 0, g, tok);
    };
    if (n > 0) keys();
    bool ok = true;
    int nc = 0, ne = 0, tails = 0;
    for (int i = 0; i < n && ok; ++i) {
      const int st = i & 1, ph = (i >> 1) & 1, t0 = (r0 + i) * p.tpt;
      uint8_t* qd = fb_smem + SM::oC + st * SM::kTile;
      uint8_t* od = fb_smem + SM::oE + st * SM::kTile;
      const uint32_t bytes = uint32_t(rows) * D * 2;
      if (!(ok = warp_wait(bar.c_empty + st, ph ^ 1, abort_flag))) break;
      const int valid = (s.Lq - t0) * p.hpg;
      if (valid >= rows) {
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar.c_full + st, bytes);
          box(&tmQ, qd, bar.c_full + st, s.q0 + t0);
        }
        ++nc;
        if (!(ok = warp_wait(bar.e_empty + st, ph ^ 1, abort_flag))) break;
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar.e_full + st, bytes);
          box(&tmO, od, bar.e_full + st, s.q0 + t0);
        }
        ++ne;
      } else {  // the sequence ends in this tile: the rows behind it become zeros
        if (!(ok = warp_wait(bar.e_empty + st, ph ^ 1, abort_flag))) break;
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar.tail, 2 * bytes);
          box(&tmQ, qd, bar.tail, s.q0 + t0);
          box(&tmO, od, bar.tail, s.q0 + t0);
        }
        ++tails;
        if (!(ok = warp_wait(bar.tail, 0, abort_flag))) break;
        zero_rows<NH>(qd, valid, rows);
        zero_rows<NH>(od, valid, rows);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(bar.c_full + st);
          tc::mbar_arrive(bar.e_full + st);
        }
      }
      if (p.inject_timeout && i == 0 && blockIdx.x % 2 == 0)
        ok = __all_sync(0xffffffffu, tc::mbar_wait_for(bar.never, 0, abort_flag, tc::kInjectedWaitCycles));
    }
    if (!ok) {
      fail();
      int zero = 0;
      tc::mbar_wait(bar.res_full, 0, &zero);
      for (int x = max(nc - 2, 0); x < nc; ++x) tc::mbar_wait(bar.c_full + (x & 1), (x >> 1) & 1, &zero);
      for (int x = max(ne - 2, 0); x < ne; ++x) tc::mbar_wait(bar.e_full + (x & 1), (x >> 1) & 1, &zero);
      if (tails) tc::mbar_wait(bar.tail, 0, &zero);
    }
  } else if (warp == 1) {
    // ----------------------------- MMA issue -----------------------------
    if (lane == 0 && n > 0) {
      constexpr uint32_t kHi = tc::smem_desc_hi(1024, 2);
      const uint32_t sb = tc::smem_u32(fb_smem);
      auto major = [&](uint32_t o) { return tc::smem_desc_lo(sb + o, 16); };           // K-major along d
      auto minor = [&](uint32_t o) { return tc::smem_desc_lo(sb + o, kHalfTile); };    // rows along K
      auto dots = [&](uint32_t col, uint32_t a0, uint32_t b0) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * kHalfTile + (kk & 3) * 32) >> 4;
          tc::mma_f16_ss_lo<kHi>(tmem + col, a0 + o, b0 + o, kIdS, kk > 0 ? 1u : 0u);
        }
      };
      auto sums = [&](uint32_t dst, uint32_t src, uint32_t b0, bool first) {
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk)
          tc::mma_f16_ts_lo<kHi>(tmem + dst, tmem + src + a_col(kk), b0 + ((kk * 16 * 128) >> 4), kIdA,
                                 first && kk == 0 ? 0u : 1u);
      };
      const uint32_t ka = major(SM::oA), va = major(SM::oB);
      bool ok = tc::mbar_wait(bar.res_full, 0, abort_flag) && tc::mbar_wait(bar.c_full, 0, abort_flag);
      if (ok) {
        tc::fence_after_sync();
        dots(0, ka, major(SM::oC));
        tc::mma_commit(bar.s_full);
        ok = tc::mbar_wait(bar.e_full, 0, abort_flag);
      }
      if (ok) {
        dots(128, va, major(SM::oE));
        tc::mma_commit(bar.dp_full);
      }
      // a loop of its own for walks with the second term: a branch in the issuing thread's loop costs 8 %
      auto walk = [&](auto second) {
        for (int i = 0; i < n && ok; ++i) {
          const uint32_t st = i & 1, q = SM::oC + st * SM::kTile, o = SM::oE + st * SM::kTile;
          const uint32_t st1 = st ^ 1, ph1 = ((i + 1) >> 1) & 1;
          const uint32_t q1 = SM::oC + st1 * SM::kTile, o1 = SM::oE + st1 * SM::kTile;
          if (!(ok = tc::mbar_wait(bar.p_full, i & 1, abort_flag))) break;
          tc::fence_after_sync();
          sums(kColDv, 0, minor(o), i == 0);
          tc::mma_commit(bar.e_empty + st);  // dP and dV of this tile have read dO
          if (i + 1 < n) {  // over P, behind the product that reads it
            if (!(ok = tc::mbar_wait(bar.c_full + st1, ph1, abort_flag))) break;
            dots(0, ka, major(q1));
            tc::mma_commit(bar.s_full);
          }
          if (!(ok = tc::mbar_wait(bar.ds_full, i & 1, abort_flag))) break;
          tc::fence_after_sync();
          sums(kColDk, 128, minor(q), i == 0);
          if constexpr (decltype(second)::value) sums(kColDk, 128 + 32, minor(q), false);
          tc::mma_commit(bar.c_empty + st);
          if (i + 1 < n) {
            if (!(ok = tc::mbar_wait(bar.e_full + st1, ph1, abort_flag))) break;
            dots(128, va, major(o1));
            tc::mma_commit(bar.dp_full);
          } else {
            tc::mma_commit(bar.acc_full);
          }
        }
      };
      if (fine)
        walk(std::true_type{});
      else
        walk(std::false_type{});
      if (!ok) fail();
      int zero = 0;
      tc::mma_commit(bar.done);
      tc::mbar_wait(bar.done, 0, &zero);
    }
  } else if (warp < 4) {
    // --------------------------- lse and delta ---------------------------
    const int x0 = (warp - 2) * 64 + lane;
    tc::griddep_wait();  // the rows' data are the previous grid's
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int sl = i % NR, t0 = (r0 + i) * p.tpt;
      const int valid = min(s.Lq - t0, p.tpt) * p.hpg;
      const float2* src = p.rows + (int64_t(g) * p.seq.Tq + s.q0 + t0) * p.hpg;
      float2 v[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) v[y] = x0 + 32 * y < valid ? src[x0 + 32 * y] : make_float2(INFINITY, 0.f);
      if (!(ok = warp_wait(bar.r_empty + sl, ((i / NR) & 1) ^ 1, abort_flag))) break;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        rowd[sl * 2 * kRows + x0 + 32 * y] = -v[y].x;
        rowd[sl * 2 * kRows + kRows + x0 + 32 * y] = -v[y].y;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar.r_full + sl);
    }
    if (!ok) fail();
  } else {
    // ------------------------------ epilogue ------------------------------
    const int w = (warp - 4) >> 2, quarter = warp & 3, key = quarter * 32 + lane;
    const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);
    const uint32_t sbase = tmem + (uint32_t(quarter * 32) << 16);
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int sl = i % NR;
      // row r (token t0 + r / hpg) sees this key from row rmin on
      const int rmin = (j0 + key - off - (r0 + i) * p.tpt) * p.hpg - w * 64;
      const bool mask = j0 + kKeys - 1 - off > (r0 + i) * p.tpt;  // some key of the tile is hidden from its first row
      if (!(ok = warp_wait(bar.r_full + sl, (i / NR) & 1, abort_flag) && warp_wait(bar.s_full, i & 1, abort_flag)))
        break;
      tc::fence_after_sync();
      const float4* l4 = reinterpret_cast<const float4*>(rowd + sl * 2 * kRows + w * 64);
      const float4* d4 = reinterpret_cast<const float4*>(rowd + sl * 2 * kRows + kRows + w * 64);
      float pr[64];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32], pk[16];
        tc::tmem_ld_32x32b_x32(sbase + w * 64 + c * 32, v);
        tc::tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float4 l = l4[c * 8 + x];  // negated
          const float2 t0 = split(fma2(pair(__uint_as_float(v[4 * x]), __uint_as_float(v[4 * x + 1])), scale2, pair(l.x, l.y)));
          const float2 t1 =
              split(fma2(pair(__uint_as_float(v[4 * x + 2]), __uint_as_float(v[4 * x + 3])), scale2, pair(l.z, l.w)));
          pr[c * 32 + 4 * x] = ex2(t0.x);
          pr[c * 32 + 4 * x + 1] = ex2(t0.y);
          pr[c * 32 + 4 * x + 2] = ex2(t1.x);
          pr[c * 32 + 4 * x + 3] = ex2(t1.y);
        }
        if (mask) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (c * 32 + x < rmin) pr[c * 32 + x] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) pk[x] = pack_bf16(pr[c * 32 + 2 * x], pr[c * 32 + 2 * x + 1]);
        tc::tmem_st_32x32b_x16(sbase + w * 64 + c * 16, pk);
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar.p_full);
      if (!(ok = warp_wait(bar.dp_full, i & 1, abort_flag))) break;
      tc::fence_after_sync();
      auto ds_of = [&](int c, const uint32_t* v) {  // over P
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float4 d = d4[c * 8 + x];  // negated
          float* q = pr + c * 32 + 4 * x;
          const float2 t0 = split(mul2(pair(q[0], q[1]), add2(pair(__uint_as_float(v[4 * x]), __uint_as_float(v[4 * x + 1])), pair(d.x, d.y))));
          const float2 t1 = split(
              mul2(pair(q[2], q[3]), add2(pair(__uint_as_float(v[4 * x + 2]), __uint_as_float(v[4 * x + 3])), pair(d.z, d.w))));
          q[0] = t0.x, q[1] = t0.y, q[2] = t1.x, q[3] = t1.y;
        }
      };
      put_ds(sbase + 128 + w * 64, pr, fine, ds_of);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(bar.ds_full);
        tc::mbar_arrive(bar.r_empty + sl);
      }
    }
    if (ok && n > 0) ok = warp_wait(bar.acc_full, 0, abort_flag);
    if (!ok) fail();
    if (ok && n > 0) {
      tc::fence_after_sync();
      const int64_t row = (int64_t(s.k0) + j0 + key) * p.Hkv + g;
      if (cl > 1)  // w 0: dv, w 1: dk; every product is done, the operands' space is free
        put_partial<D>(tc::smem_u32(fb_smem), w * kKeys + key, 0, sbase + (w == 0 ? kColDv : kColDk), D);
      else if (w == 0)
        store_acc<D>(sbase + kColDv, D, p.dv + row * D, 1.f, j0 + key < s.Lk);
      else
        store_acc<D>(sbase + kColDk, D, p.dk + row * D, p.scale, j0 + key < s.Lk);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  if (cl == 1) return;
  cluster_sync();
  sum_partials<D>(tc::smem_u32(fb_smem), 2 * kKeys, rank, cl, tiles, [&](int r, int c, float (&o)[8]) {
    const int key = r % kKeys;
    if (j0 + key >= s.Lk) return;
    const int64_t row = (int64_t(s.k0) + j0 + key) * p.Hkv + g;
    store8(r < kKeys ? p.dv + row * D : p.dk + row * D, c, o, r < kKeys ? 1.f : p.scale);
  });
  cluster_sync();  // nobody leaves while its partial is read
}

// ---------------------------------------------------------------------------------
// dq of one row tile over its keys
// TMEM: S of even tiles [0, 128), dP [128, 256) (dS over it), dQ [256, 256 + D), S of odd tiles [384, 512)
// ---------------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void bwd_dq(const CUtensorMap& tmQ, const CUtensorMap& tmO, const CUtensorMap& tmK,
                                       const CUtensorMap& tmV, const FbParams& p, bool in_order, uint8_t* fb_smem,
                                       int work) {
  using SM = FbSmem<D>;
  constexpr int NH = D / 64;
  constexpr uint32_t kIdS = tc::idesc_bf16_f32(128, 128), kIdA = tc::idesc_bf16_f32(128, D, true);
  constexpr uint32_t kColDq = 256;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = work % p.Hkv;
  int rt;
  SeqSpan s;
  const int b = find_tile(p.seq, in_order, false, p.tpt, 1, p.qslots - 1 - work / p.Hkv, rt, s);  // late rows first
  if (b < 0) return;
  const int i0 = rt * p.tpt, i1 = min(i0 + p.tpt, s.Lq);
  const int vis_last = s.ok ? s.Lk - s.Lq + i1 : 0;
  const int n = vis_last > 0 ? (vis_last + kKeys - 1) / kKeys : 0;
  if (n == 0) {
    for (int x = threadIdx.x; x < (i1 - i0) * p.hpg * (D / 8); x += kFbThreads) {
      const int r = x / (D / 8);
      const int64_t row = (int64_t(s.q0) + i0 + r / p.hpg) * p.Hq + g * p.hpg + r % p.hpg;
      reinterpret_cast<uint4*>(p.dq + row * D)[x % (D / 8)] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const bool fine = n <= kFineTiles;
  uint64_t* bars = reinterpret_cast<uint64_t*>(fb_smem + SM::oBar);
  const FbBars bar(bars, SM::kRowSlots);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + SM::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  bar.init(bars, SM::kRowSlots, SM::kBars);
  if (threadIdx.x == 0) *abort_flag = 0;
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
  auto s_col = [](int j) { return (j & 1) ? 384u : 0u; };

  if (warp == 0) {
    // ------------------------------ loads ------------------------------
    auto box = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* full, int row) {
#pragma unroll
      for (int h = 0; h < NH; ++h) tc::tma_load_3d(dst + h * kHalfTile, map, full, h * 64, g, row);
    };
    if (lane == 0) {
      tc::mbar_arrive_expect_tx(bar.res_full, 2 * uint32_t(p.tpt * p.hpg) * D * 2);
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        tc::tma_load_4d(fb_smem + SM::oA + h * kHalfTile, &tmQ, bar.res_full, h * 64, 0, g, s.q0 + i0);
        tc::tma_load_4d(fb_smem + SM::oB + h * kHalfTile, &tmO, bar.res_full, h * 64, 0, g, s.q0 + i0);
      }
    }
    bool ok = true;
    int nc = 0, ne = 0, tails = 0;
    for (int j = 0; j < n && ok; ++j) {
      const int st = j & 1, ph = (j >> 1) & 1, valid = s.Lk - j * kKeys;
      uint8_t* kd = fb_smem + SM::oC + st * SM::kTile;
      uint8_t* vd = fb_smem + SM::oE + st * SM::kTile;
      if (!(ok = warp_wait(bar.c_empty + st, ph ^ 1, abort_flag))) break;
      if (valid >= kKeys) {
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar.c_full + st, SM::kTile);
          box(&tmK, kd, bar.c_full + st, s.k0 + j * kKeys);
        }
        ++nc;
        if (!(ok = warp_wait(bar.e_empty + st, ph ^ 1, abort_flag))) break;
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar.e_full + st, SM::kTile);
          box(&tmV, vd, bar.e_full + st, s.k0 + j * kKeys);
        }
        ++ne;
      } else {  // the keys behind the sequence's end become zeros
        if (!(ok = warp_wait(bar.e_empty + st, ph ^ 1, abort_flag))) break;
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar.tail, 2 * SM::kTile);
          box(&tmK, kd, bar.tail, s.k0 + j * kKeys);
          box(&tmV, vd, bar.tail, s.k0 + j * kKeys);
        }
        ++tails;
        if (!(ok = warp_wait(bar.tail, 0, abort_flag))) break;
        zero_rows<NH>(kd, valid, kKeys);
        zero_rows<NH>(vd, valid, kKeys);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(bar.c_full + st);
          tc::mbar_arrive(bar.e_full + st);
        }
      }
      if (p.inject_timeout && j == 0 && blockIdx.x % 2 == 0)
        ok = __all_sync(0xffffffffu, tc::mbar_wait_for(bar.never, 0, abort_flag, tc::kInjectedWaitCycles));
    }
    if (!ok) {
      fail();
      int zero = 0;
      tc::mbar_wait(bar.res_full, 0, &zero);
      for (int x = max(nc - 2, 0); x < nc; ++x) tc::mbar_wait(bar.c_full + (x & 1), (x >> 1) & 1, &zero);
      for (int x = max(ne - 2, 0); x < ne; ++x) tc::mbar_wait(bar.e_full + (x & 1), (x >> 1) & 1, &zero);
      if (tails) tc::mbar_wait(bar.tail, 0, &zero);
    }
  } else if (warp == 1) {
    // ----------------------------- MMA issue -----------------------------
    if (lane == 0 && n > 0) {
      constexpr uint32_t kHi = tc::smem_desc_hi(1024, 2);
      const uint32_t sb = tc::smem_u32(fb_smem);
      auto major = [&](uint32_t o) { return tc::smem_desc_lo(sb + o, 16); };
      auto minor = [&](uint32_t o) { return tc::smem_desc_lo(sb + o, kHalfTile); };
      auto dots = [&](uint32_t col, uint32_t a0, uint32_t b0) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * kHalfTile + (kk & 3) * 32) >> 4;
          tc::mma_f16_ss_lo<kHi>(tmem + col, a0 + o, b0 + o, kIdS, kk > 0 ? 1u : 0u);
        }
      };
      const uint32_t qa = major(SM::oA), oa = major(SM::oB);
      bool ok = tc::mbar_wait(bar.res_full, 0, abort_flag) && tc::mbar_wait(bar.c_full, 0, abort_flag);
      if (ok) {
        tc::fence_after_sync();
        dots(s_col(0), qa, major(SM::oC));
        tc::mma_commit(bar.s_full);
        ok = tc::mbar_wait(bar.e_full, 0, abort_flag);
      }
      if (ok) {
        dots(128, oa, major(SM::oE));
        tc::mma_commit(bar.dp_full);
        tc::mma_commit(bar.e_empty);
      }
      auto walk = [&](auto second) {
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t st = j & 1, st1 = st ^ 1, ph1 = ((j + 1) >> 1) & 1;
          if (j + 1 < n) {
            // the other S buffer: its tile j - 1 was read before dS(j - 1), whose product is issued
            if (!(ok = tc::mbar_wait(bar.c_full + st1, ph1, abort_flag))) break;
            dots(s_col(j + 1), qa, major(SM::oC + st1 * SM::kTile));
            tc::mma_commit(bar.s_full);
          }
          if (!(ok = (j + 1 == n || tc::mbar_wait(bar.e_full + st1, ph1, abort_flag)) &&
                     tc::mbar_wait(bar.ds_full, j & 1, abort_flag)))
            break;
          tc::fence_after_sync();
          const uint32_t kb = minor(SM::oC + st * SM::kTile);
          auto sums = [&](uint32_t src, bool first) {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              tc::mma_f16_ts_lo<kHi>(tmem + kColDq, tmem + src + a_col(kk), kb + ((kk * 16 * 128) >> 4), kIdA,
                                     first && kk == 0 ? 0u : 1u);
          };
          sums(128, j == 0);
          if constexpr (decltype(second)::value) sums(128 + 32, false);
          tc::mma_commit(bar.c_empty + st);
          if (j + 1 < n) {
            dots(128, oa, major(SM::oE + st1 * SM::kTile));
            tc::mma_commit(bar.dp_full);
            tc::mma_commit(bar.e_empty + st1);
          } else {
            tc::mma_commit(bar.acc_full);
          }
        }
      };
      if (fine)
        walk(std::true_type{});
      else
        walk(std::false_type{});
      if (!ok) fail();
      int zero = 0;
      tc::mma_commit(bar.done);
      tc::mbar_wait(bar.done, 0, &zero);
    }
  } else if (warp >= 4) {
    // ------------------------------ epilogue ------------------------------
    const int w = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lbase = tmem + (uint32_t(quarter * 32) << 16);
    const int i = i0 + r / p.hpg;
    const bool valid = r < p.tpt * p.hpg && i < i1;
    tc::griddep_wait();  // the rows' data are the previous grid's
    float2 rd = make_float2(INFINITY, 0.f);
    if (valid) rd = p.rows[(int64_t(g) * p.seq.Tq + s.q0 + i) * p.hpg + r % p.hpg];
    const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), lse2 = pair(-rd.x, -rd.x), dlt2 = pair(-rd.y, -rd.y);
    const int vis = s.Lk - s.Lq + i + 1;
    const int j_mask = max(s.Lk - s.Lq + i0 + 1, 0) / kKeys;  // tiles below it are seen whole by every row
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!(ok = warp_wait(bar.s_full, j & 1, abort_flag))) break;
      tc::fence_after_sync();
      const int lim = vis - j * kKeys - w * 64;  // columns below it are seen
      float pr[64];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
        tc::tmem_ld_32x32b_x32(lbase + s_col(j) + w * 64 + c * 32, v);
        tc::tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float2 t = split(fma2(pair(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])), scale2, lse2));
          pr[c * 32 + 2 * x] = ex2(t.x);
          pr[c * 32 + 2 * x + 1] = ex2(t.y);
        }
      }
      if (j >= j_mask) {
#pragma unroll
        for (int x = 0; x < 64; ++x)
          if (x >= lim) pr[x] = 0.f;
      }
      if (!(ok = warp_wait(bar.dp_full, j & 1, abort_flag))) break;
      tc::fence_after_sync();
      put_ds(lbase + 128 + w * 64, pr, fine, [&](int c, const uint32_t* v) {  // over P
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          float* q = pr + c * 32 + 2 * x;
          const float2 t = split(mul2(pair(q[0], q[1]), add2(pair(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])), dlt2)));
          q[0] = t.x, q[1] = t.y;
        }
      });
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar.ds_full);
    }
    if (ok) ok = warp_wait(bar.acc_full, 0, abort_flag);
    if (ok) {
      tc::fence_after_sync();
      const int64_t row = (int64_t(s.q0) + i) * p.Hq + g * p.hpg + r % p.hpg;
      store_acc<D>(lbase + kColDq + w * (D / 2), D / 2, p.dq + row * D + w * (D / 2), p.scale, valid);
    } else {
      fail();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Key tiles first (their walks over rows x heads are the longest), then row
// tiles, which fill the SMs as the former run out.
template <int D>
__global__ void __launch_bounds__(kFbThreads, 1)
    full_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ FbParams p) {
  extern __shared__ __align__(1024) uint8_t fb_smem[];
  if (tc::smem_u32(fb_smem) & 1023u) {  // the swizzled operands need 1024-byte alignment
    if (threadIdx.x == 0) set_status(p.status, MSA_ERR_CUDA);
    return tc::griddep_wait();
  }
  const bool in_order = cta_in_order(p.seq, p.disorder);
  if (!in_order && threadIdx.x == 0) set_status(p.status, MSA_ERR_BOUNDS);
  // a cluster shares a key tile; row tiles are a CTA each
  const int cl = cluster_size(), nk = p.kslots * p.Hkv, row = int(blockIdx.x) - nk * cl;
  if (row < 0)
    bwd_dkv<D>(tmQ, tmO, tmK, tmV, p, in_order, fb_smem, blockIdx.x / cl, cl, cluster_rank());
  else if (row < p.qslots * p.Hkv)  // the last cluster may have CTAs to spare
    bwd_dq<D>(tmQ, tmO, tmK, tmV, p, in_order, fb_smem, row);
  // Also CTAs without work: this grid must not be over before the one that still
  // writes the rows' data, or the workspace's next user would run beside it.
  tc::griddep_wait();
}

template <int D>
cudaError_t backward(const FullBwdArgs& a, cudaStream_t stream) {
  const FullArgs& f = a.f;
  FbParams p{};
  p.seq = f.seq;
  p.Hq = f.Hq;
  p.Hkv = f.Hkv;
  p.hpg = f.Hq / f.Hkv;
  p.tpt = kRows / p.hpg;
  p.scale = f.scale;
  p.scale_log2 = f.scale * kLog2e;
  p.rows = reinterpret_cast<float2*>(static_cast<char*>(f.ws) + kWsHeader);
  p.dq = static_cast<__nv_bfloat16*>(a.dq);
  p.dk = static_cast<__nv_bfloat16*>(a.dk);
  p.dv = static_cast<__nv_bfloat16*>(a.dv);
  p.status = &static_cast<WsHeader*>(f.ws)->status;
  p.disorder = &static_cast<WsHeader*>(f.ws)->disorder;
  p.inject_timeout = debug_inject_timeout() ? 1 : 0;
  p.qslots = f.seq.Tq / p.tpt + f.seq.B;
  p.kslots = f.seq.Tk / kKeys + f.seq.B;
  const int64_t kc = int64_t(p.kslots) * f.Hkv, qc = int64_t(p.qslots) * f.Hkv;
  CUtensorMap tmQ, tmO, tmK, tmV;
  if (!map_rows(&tmQ, f.q, f.seq.Tq, f.Hq, f.Hkv, D, p.tpt) || !map_rows(&tmO, a.dout, f.seq.Tq, f.Hq, f.Hkv, D, p.tpt) ||
      !map_keys(&tmK, f.k, f.seq.Tk, f.Hkv, D, kKeys) || !map_keys(&tmV, f.v, f.seq.Tk, f.Hkv, D, kKeys))
    return cudaErrorInvalidValue;
  constexpr int bytes = FbSmem<D>::kTotal;
  cudaError_t e;
  if ((e = launch_order_check(f.seq, f.ws, stream)) || (e = launch_full_bwd_rows(a, stream))) return e;
  ProfScope pf("full_bwd", stream);
  const int c = cluster_split(kc, f.seq.Tq / f.seq.B / p.tpt);
  static KernelReady ready;
  return launch_clusters(ready, full_bwd_kernel<D>, kc + (qc + c - 1) / c, c, kFbThreads, bytes, true, stream, tmQ, tmO,
                         tmK, tmV, p);
}

}  // namespace

cudaError_t launch_full_backward_tc(const FullBwdArgs& a, cudaStream_t stream) {
  return a.f.d == 128 ? backward<128>(a, stream) : backward<64>(a, stream);
}

}  // namespace msa
