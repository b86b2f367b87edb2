// Decode over shared prefixes, the plan (full_shared.cuh): one CTA looks at all
// sequences and groups, so that the grids behind it find their work by a search.
// Latency: its barriers and a chain of four loads, under which the next grid's CTAs
// start; few sequences get a CTA of few warps.
#include "full_shared.cuh"
#include "tc_utils.cuh"

namespace msa {
namespace {

constexpr int kStepKeys = 16;  // keys of a step of the decode grid
constexpr int kOwnLeast = 2;   // steps of a warp at least: each item of its run is a part to be joined
// Both grids side by side: the sequences' own keys are bound by HBM, which three
// quarters of the SMs keep busy, the prefixes of many rows by the chain from
// scores to weights. So each grid gets as many SMs as its work says: the
// prefixes' other CTAs leave at once, the decode grid's take their place and share
// out what there is among as many as fit. Measured, one after the other and side
// by side (bf16, Hq 32, Hkv 8, d 128; no other heads):
//   97 sequences, 1300 own keys behind 3 prefixes, 20 K   117 : 109 us
//   32 sequences, 100 behind 8 K                           27 :  24 us
//   64 sequences, 500 behind 8 K                           58 :  47 us
//   64 sequences, 4000 behind 8 K                         197 : 184 us
//   4000 sequences, 100 in 1000 groups behind 512         703 : 794 us
// (`beside` 24; 13 leaves the prefixes too few, 169, 24, 57, 248, 705 us; 42: 112, 24, 53, 184, 1028.
// The fp32 grid has two CTAs to an SM and counts no SMs of its own: one after the other.)
constexpr int kLeastOwn = 8;  // SMs of the decode grid

// Sums over the CTA: what the threads before this one have, and all (whole CTA).
template <int NT, int N>
__device__ __forceinline__ void scan(int64_t (&x)[N], int64_t (&all)[N]) {
  __shared__ int64_t warps_s[N][NT / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();  // the last sums are read
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t own = x[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x[i], o);
      if (lane >= o) x[i] += y;
    }
    if (lane == 31) warps_s[i][warp] = x[i];
    x[i] -= own;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int64_t w = lane < NT / 32 ? warps_s[i][lane] : 0, own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    all[i] = __shfl_sync(0xffffffffu, w, 31);
    x[i] += __shfl_sync(0xffffffffu, w - own, warp);
  }
}

struct PlanParams {
  SharedParams s;
  const int32_t* kv_len;
  int Hkv, items, warps, cap, page_mask;
};

template <int NT>
__global__ void __launch_bounds__(NT) shared_plan_kernel(const PlanParams p) {
  const SharedParams& s = p.s;
  const int groups = s.groups.B, seqs = s.groups.Tq;
  tc::griddep_launch_dependents();
  // in flight under the look at the offsets
  const int first_len = int(threadIdx.x) < seqs ? p.kv_len[threadIdx.x] : 0;
  bool bad = false;
  for (int x = threadIdx.x; x < groups; x += NT) bad |= !span_in_order(s.groups, seq_span(s.groups, x));
  if (__syncthreads_or(bad)) {  // whose keys these are is not known
    if (threadIdx.x == 0) *s.head = SharedHead{0, 0, 1, 1, 1, 0, 0, kNumSMs};
    return;
  }
  // ---- groups ----
  struct Group {
    int b0, count, n, leader;  // n: key tiles that its items walk, 0 if its sequences do that themselves
  };
  // The first of the sequences of [b, to) that see `len` keys, or `to`.
  auto sees = [&](int b, int to, int len) {
    for (; b < to; b += 8) {  // eight loads in flight: a batch's finished samples have none
      int L[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) L[i] = p.kv_len[min(b + i, to - 1)];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (L[i] >= len && L[i] <= p.cap) return min(b + i, to - 1);
    }
    return to;
  };
  // Whether a prefix of n key tiles is worth an item's start and end (bf16: about 7 us
  // beside 1.1 us a tile; a sequence walks a tile in as much by itself, out of L2
  // from the second on). 512 sequences of 200 keys, each a group behind 512: 298 us
  // as items, 258 by themselves; 4000 of 100 keys in 1000 groups of about four behind
  // 256: 580 with all groups of three as items (`worth` 4), 672 (8), 828 (16).
  auto worth = [&](int count, int n) { return int64_t(n) * (count - 1) >= s.geo.worth; };
  auto look = [&](int x) {
    Group g{0, 0, 0, 0};
    if (x >= groups) return g;
    g.b0 = s.groups.cu_q[x];
    g.count = s.groups.cu_q[x + 1] - g.b0;
    const int len = s.prefix_len[x], n = (len - 1) / kPxKeys + 1;
    if (len <= 0 || len > p.cap || (len & p.page_mask) || !worth(g.count, n)) return g;
    g.leader = sees(g.b0, g.b0 + g.count, len);
    if (g.leader < g.b0 + g.count) g.n = n;
    return g;
  };
  const Group first = look(threadIdx.x);  // in flight under the sequences
  // ---- sequences ----
  auto group_of = [&](int b) {  // the last group that starts at or before it, so that empty ones are passed over
    int lo = 0, n = groups;
    while (n > 1) {
      const int mid = n / 2;
      if (s.groups.cu_q[lo + mid] <= b) {
        lo += mid;
        n -= mid;
      } else {
        n = mid;
      }
    }
    return s.groups.cu_q[lo] <= b && b < s.groups.cu_q[lo + 1] ? lo : -1;
  };
  int64_t steps = 0;
  for (int b0 = 0; b0 < seqs; b0 += NT) {
    const int b = b0 + int(threadIdx.x);
    int64_t mine[1] = {0}, all[1];
    if (b < seqs) {
      const int L = b0 == 0 ? first_len : p.kv_len[b];
      SharedSeq q{0, -1, b, 0};
      if (L != 0) {  // 0: a padded entry, in a group or not
        q.group = group_of(b);
        const int len = q.group >= 0 ? s.prefix_len[q.group] : 0;
        if (L < 0 || L > p.cap || len < 0 || len > L || (len & p.page_mask)) {
          q.from = q.group = -1;
        } else if (len > 0) {
          const int g0 = s.groups.cu_q[q.group], g1 = s.groups.cu_q[q.group + 1];
          if (worth(g1 - g0, (len - 1) / kPxKeys + 1)) {
            q.from = len;
          } else {
            q.group = -1;
            q.leader = sees(g0, g1, len);
            q.upto = len;
          }
        }
      }
      s.seqs[b] = q;
      if (q.from >= 0 && L > q.from) mine[0] = int64_t((L - q.from - 1) / kStepKeys + 1 + kOwnItemSteps) * p.items;
    }
    scan<NT>(mine, all);
    if (b < seqs) s.step0[b] = steps + mine[0];
    steps += all[0];
  }
  const int all_heads = p.Hkv * s.geo.groups;
  int64_t work[2] = {0, 0}, sums[2];  // units, items
  for (int x = threadIdx.x; x < groups; x += NT) {
    const Group g = x == int(threadIdx.x) ? first : look(x);
    if (g.n == 0) continue;
    const PrefixTiles t = prefix_tiles(s.geo, g.count, g.n, 1);
    work[0] += t.units * all_heads;
    work[1] += int64_t(t.tiles) * all_heads;
  }
  scan<NT>(work, sums);
  const int64_t units = sums[0], items = sums[1];
  int64_t ctas = s.geo.grid;
  const bool beside = s.geo.beside > 0 && units > 0 && steps > 0;
  if (beside)
    ctas = max(min(ctas * units * s.geo.beside / (units * s.geo.beside + steps), ctas - kLeastOwn), int64_t(1));
  // Few items: no CTA has two runs (its second starts behind the end of its first, about 3 us).
  // Many: runs of half a CTA's share. Either way at most 2 ctas runs beyond the items.
  const int64_t want = 2 * items <= ctas ? ctas - items : 2 * ctas;
  // (an item has up to 2^23 units)
  const int per = int(min(max((units + want - 1) / want, int64_t(s.geo.least)), int64_t(1) << 24));
  int64_t runs = 0, rows = 0, more = 0;
  for (int x0 = 0; x0 < groups; x0 += NT) {
    const int x = x0 + int(threadIdx.x);
    const Group g = x0 == 0 ? first : look(x);
    int64_t mine[3] = {0, 0, 0}, all[3];
    if (g.n > 0) {
      const PrefixTiles t = prefix_tiles(s.geo, g.count, g.n, per);
      mine[0] = t.runs * all_heads;
      mine[1] = t.rows * all_heads;
      mine[2] = (t.runs - t.tiles) * all_heads;
    }
    scan<NT>(mine, all);
    if (x < groups) s.recs[x] = PrefixRec{runs + mine[0], rows + mine[1], more + mine[2], g.b0, g.count, g.n, g.leader, 0};
    runs += all[0];
    rows += all[1];
    more += all[2];
  }
  if (threadIdx.x == 0) {
    SharedHead h{};
    h.runs = runs;
    h.steps = steps;
    h.per = per;
    h.each = int((runs + ctas - 1) / ctas);
    h.ctas = h.each ? int((runs + h.each - 1) / h.each) : 0;
    h.own_ctas = beside ? kNumSMs - h.ctas : kNumSMs;
    const int64_t own_runs = int64_t(h.own_ctas) * p.warps;
    h.own_per = max((steps + own_runs - 1) / own_runs, int64_t(kOwnLeast));
    *s.head = h;
  }
}

}  // namespace

cudaError_t launch_shared_plan(const SharedArgs& a, int warps, int items, cudaStream_t stream) {
  const PlanParams p{a.s, a.f.seq.kv_len, a.f.Hkv, items, warps, a.f.seq.Tk, (1 << a.f.pages.page_log2) - 1};
  ProfScope pf("shared_plan", stream);
  if (a.f.seq.B <= 128)
    shared_plan_kernel<128><<<1, 128, 0, stream>>>(p);
  else
    shared_plan_kernel<1024><<<1, 1024, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace msa
