// Decode kernels of full attention: the walk over the keys of a batch, the ring
// of copies, the joins. What a warp does with 16 keys (element types, products)
// is its core, which the including file defines. With SHARED the keys that a
// group of sequences has in common are left to another grid, and what a warp has
// of an item goes to a third that joins it all (full_shared.cuh): warps then work
// alone throughout, each on an equal run of the steps (of 16 keys) of all items.
//
// Work: the keys of every (sequence, key/value head, group of up to 16 query
// heads) -- an item -- are cut into units of 128 (16 per warp; 64 for fp32 of d
// 128, which has four warps; caches in 8 bits: 16 to 64 per warp), the units of
// all items are numbered through, and each CTA of a fixed grid (one per SM) takes
// an equal run of them, so ragged lengths balance whatever they are, without the
// host knowing them.
// In a unit each warp takes 16 keys, which lie in one page (in 8 bits one to four such tiles), and works alone:
// its own ring of copies (cp.async, keys past the end arriving as zeros, or TMA
// with bounded waits), scores, running maximum and sum, products. Warps meet only where an item ends in the
// CTA: their states are joined in shared memory. An item that lies in several
// CTAs leaves a partial (maximum, sum, unnormalised output) per CTA, and the
// CTA that arrives last joins them in the order of the keys.
// Many short items: their ends would cost more than their keys (a join takes as
// long as a unit), so single warps take whole items instead, with nothing to join, or
// (caches in 8 bits) equal runs of the steps of all items: at the end each CTA joins
// the items that lie in several of its warps, and the last CTA those that lie in several.
#pragma once

#include "full_shared.cuh"
#include "tc_utils.cuh"

namespace msa {
namespace {

constexpr int kSub = 16;                  // keys of a tile: never across a page
constexpr int kFdMaxHeads = 16;           // query heads of an item
// What an item's beginning and end count beside its steps where warps take runs of
// them (1000 sequences of 10 to 120 keys: 0 steps 74 us, 2 57, 4 58, 7 59).
constexpr int kFdItemSteps = 2;
constexpr float kFdLog2e = 1.4426950408889634f, kFdLn2 = 0.6931471805599453f;
// The maximum only moves when a step exceeds it by 2^8: weights stay below
// 2^8 and their common factor drops out in the division by their sum.
constexpr float kFdLazy = 8.f;

__device__ __forceinline__ float ex2d(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8x8 b16 matrix across the warp, transposed
__device__ __forceinline__ uint32_t trans8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float qmax(float x) {  // over the 8 lanes that share lane & 3
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float qsum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Address of 16-byte chunk c of row r in a [rows][row_bytes] tile whose chunks
// are exchanged within 128 bytes by the row's low bits (conflict-free ldmatrix
// and vector reads down a column).
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int row_bytes, int r, int c) {
  return base + uint32_t(r * row_bytes) + (uint32_t(c ^ (r & 7)) << 4);
}

struct FdParams {
  const void *q, *k, *v;
  const float *k_scale, *v_scale;  // caches in 8 bits
  const int32_t* kv_len;
  PageMap pages;
  int B, Hq, Hkv, hpg, ngr, cap;  // ngr: head groups (items) per key/value head; cap: most keys
  float scale_log2;
  // Partials. Slots: two of 16 heads for each CTA; caches in 8 bits: two for each warp, SHARED: one for
  // each item and warp, of as many heads as an item has.
  float* part_o;   // [slots][heads][D]
  float* part_ml;  // [slots][heads][2]: maximum (log2 units), sum; a negative sum marks a page out of range
  uint32_t* arrivals;  // a byte per CTA, zero between calls: the parts of the split item that it holds the first of
  void* out;
  float* lse;
  uint32_t* status;
  SharedParams shared;  // SHARED only
};

// The keys of sequence b that its items walk: [from, L). SHARED: from is where its
// group's prefix ends, if that is left to the other grid, and x the group (-1:
// none); else the prefix's keys, up to `upto`, are found by the leader's page table.
struct Own {
  int from, L, x, leader, upto;
  bool ok;
  __device__ __forceinline__ int units(int unit_log2) const { return ok && L > from ? ((L - from - 1) >> unit_log2) + 1 : 0; }
};
template <bool SHARED>
__device__ __forceinline__ Own own_of(const FdParams& p, int b) {
  Own o{0, p.kv_len[b], -1, 0, 0, true};
  if constexpr (SHARED) {
    const SharedSeq q = p.shared.get_seq(b);
    o.from = q.from;
    o.x = q.group;
    o.leader = q.leader;
    o.upto = q.upto;
    o.ok = q.from >= 0;
  } else {
    o.ok = o.L >= 0 && o.L <= p.cap;
  }
  return o;
}
template <bool SHARED>
__device__ __forceinline__ int units_of(const FdParams& p, int b, int unit_log2) {
  return own_of<SHARED>(p, b).units(unit_log2);
}

// Four values of each of ROWS heads joined over `parts` parts, in order, and their
// lse. A negative sum marks a head without a result.
template <typename T, int kBatch = 8, int ROWS = 1, typename F>  // kBatch: parts in flight, the loads of which do not wait for each other
__device__ __forceinline__ void join_head(const FdParams& p, int64_t row, int D, int dim, int parts, F part_of) {
  float M[ROWS], den[ROWS], sum[ROWS][4];
  bool spoilt[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    M[r] = -INFINITY;
    den[r] = sum[r][0] = sum[r][1] = sum[r][2] = sum[r][3] = 0.f;
    spoilt[r] = false;
  }
  for (int y0 = 0; y0 < parts; y0 += kBatch) {
    float2 ml[ROWS][kBatch];
    float4 v[ROWS][kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const bool in = y0 + x < parts;  // places behind the last part hold zeros: weight 0 does not silence an infinity
      const PartAt s = part_of(in ? y0 + x : 0);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        ml[r][x] = in ? __ldcg(reinterpret_cast<const float2*>(s.ml) + r) : make_float2(-INFINITY, 0.f);
        v[r][x] = in ? __ldcg(reinterpret_cast<const float4*>(s.o + r * D + dim)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      float mn = M[r];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        spoilt[r] |= ml[r][x].y < 0.f;
        mn = fmaxf(mn, ml[r][x].x);
      }
      const float a = M[r] == mn ? 1.f : ex2d(M[r] - mn);
      M[r] = mn;
      den[r] *= a;
#pragma unroll
      for (int y = 0; y < 4; ++y) sum[r][y] *= a;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const float w = ml[r][x].x == mn ? 1.f : ex2d(ml[r][x].x - mn);
        den[r] = fmaf(w, ml[r][x].y, den[r]);
        sum[r][0] = fmaf(w, v[r][x].x, sum[r][0]);
        sum[r][1] = fmaf(w, v[r][x].y, sum[r][1]);
        sum[r][2] = fmaf(w, v[r][x].z, sum[r][2]);
        sum[r][3] = fmaf(w, v[r][x].w, sum[r][3]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const float inv = 1.f / den[r];
    T* dst = static_cast<T*>(p.out) + (row + r) * D + dim;
#pragma unroll
    for (int y = 0; y < 4; ++y) dst[y] = from_f<T>(spoilt[r] ? 0.f : sum[r][y] * inv);
    if (p.lse && dim == 0) p.lse[row + r] = spoilt[r] ? -INFINITY : (M[r] + log2f(den[r])) * kFdLn2;
  }
}

// A walk over units in order: those of a CTA's run, or (SOLO) of every hop-th item.
template <bool SHARED>
struct Walk {
  int b, g, hg, u, n;  // sequence, key/value head, head group, unit within the item, units of the item
  Own own;             // the sequence's keys
  __device__ __forceinline__ int from() const { return SHARED ? own.from : 0; }
  __device__ __forceinline__ int arrive(const FdParams& p, int unit_log2) {  // at sequence b: its units
    own = own_of<SHARED>(p, b);
    return own.units(unit_log2);
  }
  template <bool SOLO>
  __device__ __forceinline__ void next(const FdParams& p, int hop, int unit_log2) {
    if (++u < n) return;
    u = 0;
    if constexpr (SOLO) return seek(p, hop, hop, unit_log2);
    if (++hg < p.ngr) return;
    hg = 0;
    if (++g < p.Hkv) return;
    g = 0;
    do {
      n = ++b < p.B ? arrive(p, unit_log2) : 1;  // past the last sequence the walk is over
    } while (n == 0);
  }
  // To the first item with keys among those `by`, `by` + hop, ... further on.
  __device__ __forceinline__ void seek(const FdParams& p, int by, int hop, int step_log2) {
    const int items = p.Hkv * p.ngr;
    int it = g * p.ngr + hg;
    do {
      it += by;
      b += it / items;
      it %= items;
      by = hop;
      n = b < p.B ? arrive(p, step_log2) : 1;
    } while (n == 0);
    g = it / p.ngr;
    hg = it % p.ngr;
  }
};

// One CTA per SM: the copies in flight are what covers HBM's latency.
template <typename C>
struct FdShape {
  static constexpr int kWarps = C::kWarps, kThreads = kWarps * 32;
  static constexpr int kStep = C::kTiles * kSub, kUnit = kWarps * kStep;  // keys of a warp's step, of a unit
  static constexpr int kStepLog2 = C::kTiles == 1 ? 4 : C::kTiles == 2 ? 5 : 6, kUnitLog2 = kStepLog2 + (kWarps == 8 ? 3 : 2);
  static_assert(1 << kStepLog2 == kStep && 1 << kUnitLog2 == kUnit, "keys of a step and of a unit");
  static constexpr int kStages = C::kStages;
  static constexpr int kRing = kStages * C::kStage;      // per warp
  static constexpr int kState = (C::kAcc + 2 * C::kM + 1) * 32;  // floats of a warp's state
  // A slot per hand-over, but that the last of three takes the slot that its
  // warp read itself: it is not written again before the next item's first barrier.
  // Bulk copies: the values go through the stage just used, which is not filled
  // again before a barrier, and only the rest through a slot per warp.
  static constexpr int kSlots = kWarps == 8 ? 6 : kWarps - 1, kRest = (2 * C::kM + 1) * 32;
  static constexpr int kJoin = C::kBulk ? kWarps * kRest * 4 : kSlots * kState * 4;
  static_assert(!C::kBulk || C::kAcc * 128 <= C::kStage, "a stage holds a warp's values");
  // barriers of the copies' stages, one that nothing completes; two flags
  static constexpr int kBars = C::kBulk ? (kWarps * kStages + 1) * 8 : 0;
  static constexpr int kFlags = kWarps * (kRing + C::kExtra) + kJoin + kBars;
  static constexpr int kBytes = kFlags + 16;
};

// Steps of a warp's run of `total`
template <typename C>
__device__ __forceinline__ int64_t run_steps(int64_t total) {
  const int64_t runs = int64_t(gridDim.x) * C::kWarps;
  return (total + runs - 1) / runs;
}
// An item of which a warp has the beginning or (the CTA's first warp) a later part.
struct SplitItem {
  int run, parts;  // the run that it begins in; the runs that it lies in, 0: no item
  int row, heads;  // its first row of the output, its heads
};

// SOLO: whole items for single warps; SHARED, RUNS: the warp's run of the `total`
// steps; else the CTA's run of the `total` units. RUNS: `begun` is the item that
// begins in the run and goes on behind it, `came` the one that goes on into it.
template <typename C, bool SOLO, bool SHARED, bool RUNS>
__device__ __forceinline__ void decode_run(const typename C::Params& p, int64_t total, SplitItem& came, SplitItem& begun) {
  using SH = FdShape<C>;
  using T = typename C::T;
  constexpr int D = C::kD;
  constexpr int NS = SH::kStages, kFdWarps = SH::kWarps, kFdThreads = SH::kThreads;
  extern __shared__ __align__(1024) uint8_t fd_smem[];
  int& last_s = *reinterpret_cast<int*>(fd_smem + SH::kFlags);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = tc::smem_u32(fd_smem) + warp * SH::kRing;
  const uint32_t extra = tc::smem_u32(fd_smem) + kFdWarps * SH::kRing + warp * C::kExtra;
  float* join = reinterpret_cast<float*>(fd_smem + kFdWarps * (SH::kRing + C::kExtra));
  const int items = p.Hkv * p.ngr;
  T* out = static_cast<T*>(p.out);

  constexpr bool ALONE = SOLO || SHARED || RUNS;
  constexpr int ulog = ALONE ? SH::kStepLog2 : SH::kUnitLog2;
  const int hop = SOLO ? int(gridDim.x) * kFdWarps : 0, sub0 = ALONE ? 0 : warp * SH::kStep;
  // SHARED: runs in the order of the SMs, so that few of them lie on many; other SMs may be the prefixes'
  int run = blockIdx.x;
  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  if constexpr (RUNS) {
    run = blockIdx.x * kFdWarps + warp;
    per = run_steps<C>(total);
  }
  if constexpr (SHARED) {
    const SharedHead head = p.shared.get_head();
    if (head.disorder || int(blockIdx.x) >= head.own_ctas) return;
    run = warp * head.own_ctas + int(blockIdx.x);
    per = head.own_per;
    total = head.steps;
  }
  const int64_t run0 = SOLO ? 0 : run * per, run1 = SOLO ? INT64_MAX : min(run0 + per, total);
  if (run0 >= run1) return;
  Walk<SHARED> at{};
  int64_t first = 0;  // number of the walk's sequence's first unit
  int64_t item_first = 0;  // number of the item's first unit
  constexpr int E = RUNS ? kFdItemSteps : SHARED ? kOwnItemSteps : 0;  // counted ahead of an item's own
  int skip = 0;            // of those at the run's beginning
  if constexpr (SOLO) {
    at.seek(p, warp * int(gridDim.x) + int(blockIdx.x), hop, ulog);
  } else {
    if constexpr (SHARED) {
      // the last sequence that starts at or before the run: those without steps are passed over
      at.b = warp_count_true(p.B - 1, [&](int i) { return __ldcg(p.shared.step0 + i) <= run0; });
      first = __ldcg(p.shared.step0 + at.b);
    } else {
      int ahead = lane < p.B ? units_of<SHARED>(p, lane, ulog) : 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int mine = ahead;
        ahead = b0 + 32 + lane < p.B ? units_of<SHARED>(p, b0 + 32 + lane, ulog) : 0;  // in flight during the scan
        int64_t incl = mine > 0 ? int64_t(mine + E) * items : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, first + incl > run0);
        if (hit) {
          const int src = __ffs(hit) - 1;
          at.b = b0 + src;
          at.n = __shfl_sync(0xffffffffu, mine, src);
          first += __shfl_sync(0xffffffffu, incl, src) - int64_t(at.n + E) * items;
          break;
        }
        first += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    at.own = own_of<SHARED>(p, at.b);
    if constexpr (SHARED) at.n = at.own.units(ulog);
    const int it = int((run0 - first) / (at.n + E));
    at.g = it / p.ngr;
    at.hg = it % p.ngr;
    const int in_item = int((run0 - first) % (at.n + E));
    at.u = max(in_item - E, 0);
    skip = max(E - in_item, 0);
    item_first = first + int64_t(it) * (at.n + E) + E;
    if ((RUNS || SHARED) && run0 + skip >= run1) return;
  }

  // ---- copies: the walk `ld` runs ahead of `at` ----
  Walk<SHARED> ld = at;
  int64_t ld_left = !SOLO || ld.b < p.B ? run1 - run0 - skip : 0;
  uint32_t bad_ring = 0;  // stage x's page was out of range
  int page[C::kTiles];
  auto pages_of = [&](const Walk<SHARED>& w) {
    const int key = w.from() + (w.u << ulog) + sub0;
#pragma unroll
    for (int x = 0; x < C::kTiles; ++x)
      page[x] = key + x * kSub < w.own.L
                    ? p.pages.table[int64_t(SHARED && key < w.own.upto ? w.own.leader : w.b) * p.pages.max_pages +
                                    ((key + x * kSub) >> p.pages.page_log2)]
                    : 0;
  };
  if (ld_left > 0) pages_of(ld);
  [[maybe_unused]] uint64_t* bars = reinterpret_cast<uint64_t*>(fd_smem + SH::kFlags - SH::kBars) + warp * NS;
  [[maybe_unused]] volatile int* abort_flag = &last_s + 1;
  [[maybe_unused]] int64_t issued = 0, landed = 0;  // bulk copies' stages
  if constexpr (C::kBulk) {
    if (lane == 0) {
#pragma unroll
      for (int x = 0; x < NS; ++x) tc::mbar_init(bars + x, 1);
      tc::fence_barrier_init();
    }
    __syncwarp();
  }
  auto issue = [&](int st) {
    if (ld_left > 0) {
      const int key0 = ld.from() + (ld.u << ulog) + sub0, g = ld.g;
      bool spoilt = false, in[C::kTiles];
#pragma unroll
      for (int x = 0; x < C::kTiles; ++x) {
        const int valid = ld.own.L - key0 - x * kSub;
        const bool bad = valid > 0 && (page[x] < 0 || page[x] >= p.pages.num_pages);
        spoilt |= bad;
        in[x] = valid > 0 && !bad;
        if constexpr (!C::kBulk)
          C::copy(p, ring + st * C::kStage + x * (C::kStage / C::kTiles), in[x] ? page[x] : 0,
                  (key0 + x * kSub) & ((1 << p.pages.page_log2) - 1), g, in[x] ? valid : 0);
      }
      if constexpr (C::kBulk) {
        if (lane == 0) {
          const int box = C::kTiles == 1 ? 1 : 1 << (C::box_of(p) - 4);  // tiles of a copy, which lie in one page
          int boxes = 0;
#pragma unroll
          for (int x = 0; x < C::kTiles; ++x) boxes += in[x] && (x & (box - 1)) == 0;
          if (boxes)
            tc::mbar_arrive_expect_tx(bars + st, boxes * box * C::kTileBytes);
          else
            tc::mbar_arrive(bars + st);
#pragma unroll
          for (int x = 0; x < C::kTiles; ++x)
            if (in[x] && (x & (box - 1)) == 0)
              C::copy(p, ring + st * C::kStage, extra, st, x, bars + st, page[x],
                      (key0 + x * kSub) & ((1 << p.pages.page_log2) - 1), g);
        }
        ++issued;
      }
      bad_ring = spoilt ? bad_ring | (1u << st) : bad_ring & ~(1u << st);
      if (--ld_left > 0) {
        ld.template next<SOLO>(p, hop, ulog);
        if ((RUNS || SHARED) && ld.u == 0) ld_left = max(ld_left - E, int64_t(0));
        if (RUNS || SHARED ? ld_left > 0 : !SOLO || ld.b < p.B)
          pages_of(ld);
        else
          ld_left = 0;
      }
    }
    if constexpr (!C::kBulk) cp_commit_group();
  };
#pragma unroll
  for (int st = 0; st < NS - 1; ++st) issue(st);

  C c;
  bool fresh = true, bad = false;
  int st = 0;
  [[maybe_unused]] uint32_t parity = 0;
  [[maybe_unused]] bool dead = false;  // a wait ran out: nothing more is copied or read, but everybody is met
  if constexpr (C::kBulk) {
    if (p.inject_timeout && blockIdx.x % 2 == 0 && warp == 0)
      dead = !tc::mbar_wait_for(reinterpret_cast<uint64_t*>(fd_smem + SH::kFlags) - 1, 0, abort_flag, tc::kInjectedWaitCycles);
  }
  int h0 = 0, heads = 0;
  for (int64_t z = run0 + skip; z < run1 && (!SOLO || at.b < p.B); ++z) {
    if (fresh) {
      h0 = at.g * p.hpg + at.hg * kFdMaxHeads;
      heads = min(p.hpg - at.hg * kFdMaxHeads, kFdMaxHeads);
      c.start(p, static_cast<const T*>(p.q) + (int64_t(at.b) * p.Hq + h0) * D, heads, extra);
      fresh = bad = false;
    }
    if constexpr (C::kBulk) {
      if (!dead) {
        issue((st + NS - 1) % NS);
        dead = !__all_sync(0xffffffffu, tc::mbar_wait(bars + st, parity, abort_flag));
        if (dead)
          *abort_flag = 1;
        else
          ++landed;
      }
      if (st == NS - 1) parity ^= 1;
    } else {
      issue((st + NS - 1) % NS);
      cp_wait<NS - 1>();
      __syncwarp();
    }
    bad |= (bad_ring >> st) & 1u;
    int valid = at.own.L - (at.from() + (at.u << ulog) + sub0);
    if (C::kBulk && dead) valid = 0;
    if (valid > 0) c.step(p, ring + st * C::kStage, extra, st, valid);
    __syncwarp();
    st = (st + 1) % NS;
    const int b = at.b, n = at.n;
    const bool ends = at.u + 1 == at.n;
    if (!ends && z + 1 < run1) {
      ++at.u;
      continue;
    }
    // ---- the item ends here: join the warps' states, halving their number ----
    fresh = true;
    c.finish();
    // values to or from v, maxima, sums and whether a page was out of range to or from r
    auto put = [&](float* v, float* r) {
#pragma unroll
      for (int x = 0; x < C::kAcc; ++x) v[x * 32 + lane] = c.acc[x];
#pragma unroll
      for (int x = 0; x < C::kM; ++x) {
        r[x * 32 + lane] = c.m[x];
        r[(C::kM + x) * 32 + lane] = c.l[x];
      }
      r[2 * C::kM * 32 + lane] = bad ? 1.f : 0.f;
    };
    auto take = [&](const float* v, const float* r) {
      float wa[C::kM], wb[C::kM];
#pragma unroll
      for (int x = 0; x < C::kM; ++x) {
        const float mo = r[x * 32 + lane], mn = fmaxf(c.m[x], mo);
        wa[x] = c.m[x] == mn ? 1.f : ex2d(c.m[x] - mn);
        wb[x] = mo == mn ? 1.f : ex2d(mo - mn);
        c.m[x] = mn;
        c.l[x] = c.l[x] * wa[x] + r[(C::kM + x) * 32 + lane] * wb[x];
      }
#pragma unroll
      for (int x = 0; x < C::kAcc; ++x)
        c.acc[x] = c.acc[x] * wa[C::m_index(x)] + v[x * 32 + lane] * wb[C::m_index(x)];
      bad |= r[2 * C::kM * 32 + lane] != 0.f;
    };
    if constexpr (!ALONE && C::kBulk) {
      float* mine = reinterpret_cast<float*>(fd_smem + warp * SH::kRing + (st == 0 ? NS - 1 : st - 1) * C::kStage);
#pragma unroll
      for (int half = kFdWarps / 2; half > 0; half >>= 1) {
        if (warp >= half && warp < 2 * half) put(mine, join + warp * SH::kRest);
        __syncthreads();
        if (warp < half) take(mine + half * (SH::kRing / 4), join + (warp + half) * SH::kRest);
      }
      tc::fence_proxy_async_smem();  // before the next copy into the stage
      __syncthreads();
    } else if constexpr (!ALONE) {
      // Every hand-over has a slot of its own: the upper warps may be at the next
      // item's end while the lower ones still read this one's.
#pragma unroll
      for (int half = kFdWarps / 2, slot0 = 0; half > 0; slot0 += half, half >>= 1) {
        if (half == 1) slot0 = SH::kSlots - 1;
        float* slot = join + (slot0 + warp % half) * SH::kState;
        if (warp >= half && warp < 2 * half) put(slot, slot + C::kAcc * 32);
        __syncthreads();
        if (warp < half) take(slot, slot + C::kAcc * 32);
      }
    }
    const bool whole = SOLO || (item_first >= run0 && ends);
    // SHARED: parts in the order of the items, those of one item in the order of the runs
    const int item = at.b * items + at.g * p.ngr + at.hg, item_heads = SHARED || C::kBulk ? min(p.hpg, kFdMaxHeads) : kFdMaxHeads;
    const int slot = SHARED ? item + run : 2 * run + (item_first >= run0 ? 1 : 0);
    if (ALONE || warp == 0) {
      c.sum_l();
      if (__any_sync(0xffffffffu, bad)) {
        bad = true;
        if (lane == 0) set_status(p.status, MSA_ERR_BOUNDS);
      }
      if (whole && !SHARED) {
        float inv[C::kM];
#pragma unroll
        for (int x = 0; x < C::kM; ++x) inv[x] = bad ? 0.f : 1.f / c.l[x];
        if constexpr (C::kBulk) {
          c.each_run([&](int h, int x, int dim, float(&val)[C::kRunDims]) {
            if (h >= heads) return;
            uint4 w[C::kRunDims * sizeof(T) / 16];
#pragma unroll
            for (int y = 0; y < C::kRunDims; ++y) reinterpret_cast<T*>(w)[y] = from_f<T>(bad ? 0.f : val[y] * inv[x]);
            uint4* dst = reinterpret_cast<uint4*>(out + (int64_t(b) * p.Hq + h0 + h) * D + dim);
#pragma unroll
            for (int y = 0; y < int(sizeof(w) / 16); ++y) dst[y] = w[y];
          });
        } else {
          c.each([&](int h, int x, int dim, float val) {
            if (h < heads)
              out[(int64_t(b) * p.Hq + h0 + h) * D + dim] = from_f<T>(bad ? 0.f : val * inv[x]);
          });
        }
        if (p.lse)
          c.each_head([&](int h, int x) {
            if (h < heads) p.lse[int64_t(b) * p.Hq + h0 + h] = bad ? -INFINITY : (c.m[x] + log2f(c.l[x])) * kFdLn2;
          });
      } else {
        float* po = p.part_o + int64_t(slot) * item_heads * D;
        float* pm = p.part_ml + int64_t(slot) * item_heads * 2;
        if constexpr (C::kBulk) {
          c.each_run([&](int h, int, int dim, float(&val)[C::kRunDims]) {
            if (h >= heads) return;
            float4* dst = reinterpret_cast<float4*>(po + h * D + dim);
#pragma unroll
            for (int y = 0; y < C::kRunDims / 4; ++y)
              dst[y] = make_float4(val[4 * y], val[4 * y + 1], val[4 * y + 2], val[4 * y + 3]);
          });
        } else {
          c.each([&](int h, int, int dim, float val) {
            if (h < heads) po[h * D + dim] = val;
          });
        }
        c.each_head([&](int h, int x) {
          if (h < heads) {
            pm[2 * h] = c.m[x];
            pm[2 * h + 1] = bad ? -1.f : c.l[x];
          }
        });
      }
    }
    if constexpr (RUNS) {
      if (!whole) {
        const int r0 = int(item_first / per);
        (item_first >= run0 ? begun : came) = SplitItem{r0, int((item_first + n - 1) / per) - r0 + 1, b * p.Hq + h0, heads};
      }
    }
    if (!ALONE && !whole) {
      // the item's units lie in CTAs c0..c1: the last to arrive joins them
      const int c0 = int(item_first / per), c1 = int((item_first + n - 1) / per);
      if (warp == 0) {
        __syncwarp();
        if (lane == 0) {
          // releases the warp's stores (ordered by __syncwarp), acquires the others'
          const int sh = 8 * (c0 & 3);
          uint32_t old;
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
                       : "=r"(old)
                       : "l"(p.arrivals + (c0 >> 2)), "r"(1u << sh)
                       : "memory");
          last_s = int((old >> sh) & 0xffu) == c1 - c0;
          if (last_s) atomicSub(p.arrivals + (c0 >> 2), uint32_t(c1 - c0 + 1) << sh);  // ready for the next call
        }
      }
      __syncthreads();
      if (last_s)
        for (int o = threadIdx.x * 4; o < heads * D; o += kFdThreads * 4)
          join_head<T>(p, int64_t(b) * p.Hq + h0 + o / D, D, o % D, c1 - c0 + 1, [&](int y) {
            const int cta = c0 + y, s = 2 * cta + (cta == c0 && item_first >= c0 * per ? 1 : 0);
            const int64_t head = int64_t(s) * item_heads + o / D;
            return PartAt{p.part_o + head * D, p.part_ml + head * 2};
          });
      __syncthreads();  // last_s is read before the next item sets it
    }
    if (ends) item_first += n + E;
    const int was = at.b;
    at.template next<SOLO>(p, hop, ulog);
    if (at.b != was) item_first = z + 1 + E;
    z += E;
  }
  if constexpr (C::kBulk) {
    if (dead && issued > 0) {  // let the copies land before the CTA gives its shared memory up
      if (lane == 0) set_status(p.status, MSA_ERR_TIMEOUT);
      int zero = 0;
      for (int64_t x = landed; x < issued; ++x) tc::mbar_wait(bars + x % NS, uint32_t(x / NS) & 1, &zero);
    }
  } else {
    cp_wait<0>();
  }
}

// RUNS: joins the items that lie in several warps' runs: those that
// lie in this CTA, and of those that lie in several CTAs the ones that it is the last of.
template <typename C>
__device__ __forceinline__ void join_runs(const typename C::Params& p, const SplitItem& came, const SplitItem& begun) {
  using T = typename C::T;
  constexpr int D = C::kD, W = C::kWarps;
  extern __shared__ __align__(1024) uint8_t fd_smem[];
  int& last_s = *reinterpret_cast<int*>(fd_smem + FdShape<C>::kFlags);
  // where warps' states would be joined: each warp's item in this CTA; the one from before, the one to behind
  SplitItem* split = reinterpret_cast<SplitItem*>(fd_smem + W * (FdShape<C>::kRing + C::kExtra));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, heads = min(p.hpg, kFdMaxHeads);
  auto join = [&](const SplitItem& s, int o) {  // four values
    join_head<T, 4>(p, s.row + o / D, D, o % D, s.parts, [&](int y) {
      const int64_t head = int64_t(2 * (s.run + y) + (y == 0 ? 1 : 0)) * heads + o / D;
      return PartAt{p.part_o + head * D, p.part_ml + head * 2};
    });
  };
  if (lane == 0) {
    const bool here = begun.parts > 0 && (begun.run + begun.parts - 1) / W == int(blockIdx.x);
    const SplitItem none{};
    split[warp] = here ? begun : none;
    if (warp == 0) split[W] = came;  // the CTA's first step is its first warp's
    if (warp == 0) split[W + 1] = none;
  }
  __syncthreads();
  if (lane == 0 && begun.parts > 0 && split[warp].parts == 0) split[W + 1] = begun;
  const int each = heads * (D / 4);
  for (int o = threadIdx.x; o < W * each; o += W * 32) {
    const SplitItem s = split[o / each];
    if (s.parts > 0 && o % each < s.heads * (D / 4)) join(s, o % each * 4);
  }
  __syncthreads();
  for (int x = 0; x < 2; ++x) {
    const SplitItem s = split[W + x];
    if (s.parts == 0) continue;
    const int c0 = s.run / W, c1 = (s.run + s.parts - 1) / W;
    if (threadIdx.x == 0) {
      // releases the CTA's stores (ordered by the barrier), acquires the others'
      const int sh = 8 * (c0 & 3);
      uint32_t old;
      asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
                   : "=r"(old)
                   : "l"(p.arrivals + (c0 >> 2)), "r"(1u << sh)
                   : "memory");
      last_s = int((old >> sh) & 0xffu) == c1 - c0;
      if (last_s) atomicSub(p.arrivals + (c0 >> 2), uint32_t(c1 - c0 + 1) << sh);  // ready for the next call
    }
    __syncthreads();
    if (last_s)
      for (int o = threadIdx.x; o < s.heads * (D / 4); o += W * 32) join(s, o * 4);
    __syncthreads();  // last_s is read before it is set again
  }
}

template <typename C>
__global__ void __launch_bounds__(FdShape<C>::kThreads, 1) full_decode_shared_kernel(const __grid_constant__ typename C::Params p) {
  tc::griddep_launch_dependents();  // the joins' grid, which waits for this one
  SplitItem none{};
  decode_run<C, false, true, false>(p, 0, none, none);
  tc::griddep_wait();  // this grid is not over before the prefixes' grid is
}

template <typename C>
__global__ void __launch_bounds__(FdShape<C>::kThreads, 1) full_decode_kernel(const __grid_constant__ typename C::Params p) {
  using SH = FdShape<C>;
  using T = typename C::T;
  constexpr int D = C::kD;
  constexpr int kFdWarps = SH::kWarps, kFdThreads = SH::kThreads;
  const int lane = threadIdx.x & 31, items = p.Hkv * p.ngr;
  T* out = static_cast<T*>(p.out);
  if constexpr (C::kBulk) {
    extern __shared__ __align__(1024) uint8_t fd_smem[];
    if (tc::smem_u32(fd_smem) & 1023u) {  // the swizzled tiles need 1024-byte alignment
      if (threadIdx.x == 0) set_status(p.status, MSA_ERR_CUDA);
      return;
    }
    if (threadIdx.x == 0) {
      tc::mbar_init(reinterpret_cast<uint64_t*>(fd_smem + SH::kFlags) - 1, 1);
      reinterpret_cast<int*>(fd_smem + SH::kFlags)[1] = 0;  // no wait has run out
      tc::fence_barrier_init();
      C::prefetch(p);
    }
    __syncthreads();
  }

  // ---- all units (every warp counts alone) ----
  int64_t total = 0, steps = 0;
  int longest = 0;  // in warps' steps
#pragma unroll 8
  for (int b = lane; b < p.B; b += 32) {
    const int n = units_of<false>(p, b, SH::kStepLog2);
    total += (n + kFdWarps - 1) / kFdWarps;
    if (n > 0) steps += n + kFdItemSteps;
    longest = max(longest, n);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total *= items;
  const int64_t all = int64_t(p.B) * items;
  bool alone;  // warps work alone, on whole items or (kBulk) on runs of steps
  if constexpr (C::kBulk) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) steps += __shfl_xor_sync(0xffffffffu, steps, o);
    steps *= items;
    // Runs of steps for single warps, or shared-out units? In runs warps meet once, at
    // the end; units cost a join by all warps per item. Measured both ways (d 128, bf16):
    //   200 sequences of 100 to 500 keys, 800 items   41 (runs) : 78 us
    //   128 of 2000 to 8000, 512                      226 : 240 us
    //   64 of 4096, 256                               100 : 100 us     40 of 2000, 160    45 : 41 us
    //   128 of 50 to 4000, one head, 128               39 :  33 us     1 of 777, 4        17 : 10 us
    //   16 of 4 K to 128 K, 64 (long runs of warps lie far apart in memory)  338 : 320 us
    alone = all >= int64_t(gridDim.x) && total <= 64 * all;
  } else {
    // Whole items for single warps, or shared-out units? A unit and a warp's step
    // both take about 1.1 us, and so does an item's end or start; single warps
    // come out ahead from 1.25 times the other count on. Measured both ways (Hq 32,
    // Hkv 8, d 128, bf16; lengths within a factor of 2):
    //   1280 items up to 64 keys   19 (single) : 29 us     2560 up to 256   65 :  70 us
    //   10240 items up to 128      99 : 177 us             2560 up to 512  119 : 109 us
    //   640 items up to 128        18 :  20 us              320 up to 128   17 :  16 us
    longest = __reduce_max_sync(0xffffffffu, longest);
    const int warps = int(gridDim.x) * kFdWarps;
    const int64_t rounds = (all + warps - 1) / warps;
    alone = 4 * rounds * (1 + longest) * int64_t(gridDim.x) <= 5 * (total + all);
  }
  // sequences without keys: nobody's run holds them
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const Own o = own_of<false>(p, b);
    if (o.units(SH::kStepLog2) > 0) continue;
    if (threadIdx.x == 0 && !o.ok) set_status(p.status, MSA_ERR_BOUNDS);
    for (int x = threadIdx.x; x < p.Hq * D; x += kFdThreads) out[int64_t(b) * p.Hq * D + x] = from_f<T>(0.f);
    if (p.lse)
      for (int x = threadIdx.x; x < p.Hq; x += kFdThreads) p.lse[int64_t(b) * p.Hq + x] = -INFINITY;
  }
  SplitItem came{}, begun{};
  if (!alone) {
    decode_run<C, false, false, false>(p, total, came, begun);
  } else if constexpr (!C::kBulk) {
    decode_run<C, true, false, false>(p, total, came, begun);
  } else {
    decode_run<C, false, false, true>(p, steps, came, begun);
    join_runs<C>(p, came, begun);
  }
}

int fd_grid() { return kNumSMs; }

// SHARED: the grid may start while the one before it ends
template <typename C, bool SHARED>
cudaError_t decode(const typename C::Params& p, const char* name, cudaStream_t stream) {
  constexpr auto kern = [] {
    if constexpr (SHARED)
      return full_decode_shared_kernel<C>;
    else
      return full_decode_kernel<C>;
  }();
  constexpr int bytes = FdShape<C>::kBytes;
  static_assert(bytes <= 227 * 1024 - 16, "shared memory of one CTA");
  static KernelReady ready;
  if (cudaError_t e = ready.on_device(reinterpret_cast<const void*>(kern), bytes)) return e;
  ProfScope pf(name, stream);
  if constexpr (SHARED) {
    return launch_early(kern, fd_grid(), FdShape<C>::kThreads, bytes, stream, p);
  } else {
    kern<<<fd_grid(), FdShape<C>::kThreads, bytes, stream>>>(p);
    return cudaGetLastError();
  }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
int head_groups(int hpg) { return (hpg + kFdMaxHeads - 1) / kFdMaxHeads; }
// partials of `slots` slots
size_t fd_part_bytes(int slots, int d) { return up256(size_t(slots) * kFdMaxHeads * d * 4) + up256(size_t(slots) * kFdMaxHeads * 8); }
FdParams fd_params(const FullArgs& a, int slots) {
  FdParams p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.kv_len = a.seq.kv_len;
  p.pages = a.pages;
  p.B = a.seq.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.hpg = a.Hq / a.Hkv;
  p.ngr = head_groups(p.hpg);
  p.cap = a.seq.Tk;
  p.scale_log2 = a.scale * kFdLog2e;
  char* w = static_cast<char*>(a.ws) + kWsHeader;
  p.part_o = reinterpret_cast<float*>(w);
  p.part_ml = reinterpret_cast<float*>(w + up256(size_t(slots) * kFdMaxHeads * a.d * 4));
  p.arrivals = static_cast<WsHeader*>(a.ws)->arrivals;
  p.out = a.out;
  p.lse = a.lse;
  p.status = &static_cast<WsHeader*>(a.ws)->status;
  return p;
}

}  // namespace
}  // namespace msa
