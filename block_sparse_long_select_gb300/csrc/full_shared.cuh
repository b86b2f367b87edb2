// Decode over shared prefixes: how the work on the prefixes is cut, and where
// its partial results lie. One grid computes them (full_prefix_tc.cu for bf16,
// full_prefix_fp32.cu), the decode grid behind it joins them to each
// sequence's own keys.
//
// Group x holds the consecutive sequences [cu[x], cu[x+1]); its prefix is the
// first prefix_len[x] keys of the page-table row of its leader, the group's
// first sequence with keys. An item is a tile of the group's rows (sequences x
// heads of one key/value head) and walks the prefix in tiles of kPxKeys keys. All
// items' steps are numbered through as units and dealt out to the CTAs in equal
// runs, so an item may lie in several consecutive CTAs; each leaves a part: its
// rows' maximum (log2 units), sum and unnormalised output. The reader finds the
// parts in closed form, so nothing is counted, and nothing waits, inside the grid.
// The decode grid leaves parts of the sequences' own keys, and a third grid
// joins them all, a thread per four values: joined at each item's end inside the
// decode grid, 97 sequences of 1300 own keys behind 12 K shared ones took 190 us,
// of which its copies stood still for half.
#pragma once

#include "full_internal.cuh"

namespace msa {

constexpr int kPxKeys = 128;  // keys of a tile

// How rows are cut into items. bf16: two row tiles of `half` sequences, which
// share each key tile; an item whose sequences fit into one takes the key tiles
// two at a time instead, one per half (`alt`).
struct PrefixGeometry {
  int heads, groups;  // heads of an item; items' head groups per key/value head
  int seqs, half;     // sequences of an item; of a row tile (0: an item is one row tile)
  int block;          // most rows of a part
  int grid;           // CTAs
  int least;          // units that a CTA takes at least
  int beside;         // what a unit takes in the decode grid's steps of all SMs together; 0: no grids side by side
};
// A group's items.
struct PrefixRec {
  int64_t unit0, row0;  // units and rows of the groups before it
  int64_t per;          // units of a CTA
  int b0, count;        // first sequence, sequences
  int n, leader;        // key tiles (0: nothing to compute), whose page table
};
static_assert(sizeof(PrefixRec) == 40, "read as five 8-byte words");

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }
// Of an item of `count` sequences whose prefix has n key tiles
struct PrefixItem {
  int units, rows;
  bool alt;
};
__host__ __device__ __forceinline__ PrefixItem prefix_item(const PrefixGeometry& g, int count, int n) {
  const bool alt = g.half > 0 && count <= g.half;
  return {alt ? (n + 1) / 2 : n, count * g.heads, alt};
}
// Of all items of a group for one key/value head and head group
struct PrefixTiles {
  int tiles;
  int64_t units, rows;
};
__host__ __device__ __forceinline__ PrefixTiles prefix_tiles(const PrefixGeometry& g, int count, int n) {
  const int tiles = ceil_div(count, g.seqs);
  const PrefixItem last = prefix_item(g, count - (tiles - 1) * g.seqs, n), full = prefix_item(g, g.seqs, n);
  return {tiles, int64_t(tiles - 1) * full.units + last.units, int64_t(tiles - 1) * full.rows + last.rows};
}

// A part of some heads' results: heads x D unnormalised values; a maximum (log2
// units) and a sum per head, negative where there is no result.
struct PartAt {
  const float *o, *ml;
};
// The parts that concern one sequence's heads [h, ...) of one item.
template <int D>
struct PrefixRows;

struct SharedParams {
  SeqMap groups;  // cu_q: cu_prefix, kv_len: prefix_len, B: groups, Tq: sequences
  const int32_t* prefix_len;
  const uint32_t* disorder;
  PrefixGeometry geo;
  PrefixRec* recs;
  float* part;   // [rows][D]
  float2* stat;  // [rows]: maximum, sum (negative: a page out of range)

  // The group of sequence b, or -1. Offsets in order.
  __device__ __forceinline__ int group_of(int b) const {
    int lo = 0, n = groups.B;  // cu[lo] <= b, if any; the last such group, so that empty ones are passed over
    while (n > 1) {
      const int mid = n / 2;
      if (groups.cu_q[lo + mid] <= b) {
        lo += mid;
        n -= mid;
      } else {
        n = mid;
      }
    }
    return groups.cu_q[lo] <= b && b < groups.cu_q[lo + 1] ? lo : -1;
  }
  template <int D>
  __device__ __forceinline__ PrefixRows<D> rows(int x, int b, int g, int h) const;
};

template <int D>
struct PrefixRows {
  const float* o;
  const float2* ml;
  int n, block;  // parts; rows from one to the next
  __device__ __forceinline__ PartAt part(int y) const {
    return {o + int64_t(y) * block * D, reinterpret_cast<const float*>(ml + int64_t(y) * block)};
  }
};

// Behind the prefixes' grid (griddepcontrol.wait).
template <int D>
__device__ __forceinline__ PrefixRows<D> SharedParams::rows(int x, int b, int g, int h) const {
  PrefixRows<D> r{nullptr, nullptr, 0, 0};
  if (x < 0) return r;
  const int64_t* w = reinterpret_cast<const int64_t*>(recs + x);
  const int64_t unit0 = __ldcg(w), row0 = __ldcg(w + 1), per = __ldcg(w + 2), bc = __ldcg(w + 3), nl = __ldcg(w + 4);
  const int b0 = int(bc), count = int(bc >> 32), n = int(nl);
  if (n <= 0) return r;
  const PrefixTiles t = prefix_tiles(geo, count, n);
  const int s = b - b0, i = s / geo.seqs, hg = h / geo.heads, gi = g * geo.groups + hg;
  const PrefixItem full = prefix_item(geo, geo.seqs, n), mine = prefix_item(geo, min(geo.seqs, count - i * geo.seqs), n);
  const int64_t u0 = unit0 + gi * t.units + int64_t(i) * full.units;
  const int64_t c0 = u0 / per, c1 = (u0 + mine.units - 1) / per;
  const int64_t row = row0 + gi * t.rows + int64_t(i) * full.rows + c0 * geo.block + (s - i * geo.seqs) * geo.heads + h -
                      hg * geo.heads;
  r.o = part + row * D;
  r.ml = stat + row;
  r.block = geo.block;
  r.n = int(c1 - c0 + 1);
  return r;
}

// ---- both grids side by side -------------------------------------------------------
// The sequences' own keys are bound by HBM, which three quarters of the SMs keep
// busy; the prefixes are bound by the chain from scores to weights. So where the
// former take much longer, the latter get as few CTAs as still end with them, and
// the decode grid, whose other CTAs start at once, only uses the SMs left (97
// sequences of 1300 own keys behind three prefixes, 20 K keys: 130 us one after the
// other, BESIDE us with the prefixes on a fifth of the SMs). Else every SM serves both in turn.
constexpr int kLeastOwn = 8;  // SMs
struct PrefixLoad {
  int64_t units;  // of all groups
  int ctas;       // that work on them
  int64_t per;    // units of each but the last
};
// Group i's key tiles (0: nothing to compute), sequences and leader.
__device__ __forceinline__ void look_at_group(const SharedParams& p, const int32_t* kv_len, int cap, int page_mask, int i,
                                              int& tiles, int& first, int& cnt, int& lead) {
  first = p.groups.cu_q[i];
  cnt = p.groups.cu_q[i + 1] - first;
  const int len = p.prefix_len[i];
  tiles = 0;
  lead = first;
  if (cnt <= 0 || len <= 0 || len > cap || (len & page_mask)) return;
  for (int b = first; b < first + cnt; ++b) {
    const int L = kv_len[b];
    if (L >= len && L <= cap) {  // the others see nothing of it
      lead = b;
      tiles = (len - 1) / kPxKeys + 1;
      return;
    }
  }
}
// Whole warp. `heads`: key/value heads. t, f, c, l: of group `lane`, where there are up to 32.
__device__ __forceinline__ PrefixLoad prefix_load(const SharedParams& p, const int32_t* kv_len, int heads, int cap,
                                                  int page_mask, int& t, int& f, int& c, int& l) {
  const int lane = threadIdx.x & 31;
  int64_t units = 0, own = 0;
  if (p.geo.beside)
#pragma unroll 4
    for (int b = lane; b < p.groups.Tq; b += 32) own += min(max(kv_len[b], 0), cap);
  for (int x0 = 0; x0 < p.groups.B; x0 += 32) {
    t = 0;
    if (x0 + lane < p.groups.B) look_at_group(p, kv_len, cap, page_mask, x0 + lane, t, f, c, l);
    if (t > 0) {
      units += prefix_tiles(p.geo, c, t).units * heads * p.geo.groups;
      own -= int64_t(c) * t * kPxKeys;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    units += __shfl_xor_sync(0xffffffffu, units, o);
    own += __shfl_xor_sync(0xffffffffu, own, o);
  }
  PrefixLoad r{units, p.geo.grid, max((units + p.geo.grid - 1) / p.geo.grid, int64_t(p.geo.least))};
  if (p.geo.beside && own > 0 && units > 0) {
    const int64_t work = units * p.geo.beside, steps = own / 16 * heads + 1;
    const int64_t most = max(min(kNumSMs * work / (work + steps), int64_t(kNumSMs - kLeastOwn)), int64_t(1));
    r.per = max((units + most - 1) / most, int64_t(p.geo.least));
    r.ctas = int((units + r.per - 1) / r.per);
  }
  return r;
}

// ---- the prefixes' grid: a CTA's run of units ------------------------------------
// One part to compute.
struct PrefixPart {
  int x, g, hg;       // group, key/value head, head group
  int b0, count;      // its rows' sequences
  int leader, Lk;     // whose page table, keys of the prefix
  int jb, n;          // key tiles [jb, jb + n)
  int alt;
  int64_t row;        // of its first row
};
struct PrefixPlan {
  const SharedParams& p;
  const int32_t* kv_len;
  int Hkv, cap, page_mask;
  // where the run stands
  int64_t at, end, per, unit0, row0;
  int x, n, b0, count, leader;

  // Whole warp: measures all groups, leaves their records (`write`), and finds
  // this CTA's run. False: it has none.
  __device__ __forceinline__ bool init(int cta, bool write) {
    const int lane = threadIdx.x & 31, all = Hkv * p.geo.groups;
    int t = 0, f = 0, c = 0, l = 0;
    const PrefixLoad load = prefix_load(p, kv_len, Hkv, cap, page_mask, t, f, c, l);
    const int64_t total = load.units;
    per = load.per;
    at = int64_t(cta) * per;
    end = min(at + per, total);
    bool found = false;
    int64_t units = 0, rows = 0;
    for (int x0 = 0; x0 < p.groups.B && (write || !found); x0 += 32) {
      if (p.groups.B > 32) {  // else they are in hand
        t = 0;
        if (x0 + lane < p.groups.B) look_at_group(p, kv_len, cap, page_mask, x0 + lane, t, f, c, l);
      }
      PrefixTiles pt{0, 0, 0};
      if (t > 0) pt = prefix_tiles(p.geo, c, t);
      int64_t u = pt.units * all, r = pt.rows * all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t yu = __shfl_up_sync(0xffffffffu, u, o), yr = __shfl_up_sync(0xffffffffu, r, o);
        if (lane >= o) u += yu, r += yr;
      }
      const int64_t u0 = units + u - pt.units * all, r0 = rows + r - pt.rows * all;
      if (write && x0 + lane < p.groups.B) p.recs[x0 + lane] = PrefixRec{u0, r0, per, f, c, t, l};
      const uint32_t hit = __ballot_sync(0xffffffffu, t > 0 && u0 + pt.units * all > at);
      if (hit && !found && at < end) {
        const int src = __ffs(hit) - 1;
        found = true;
        x = x0 + src;
        unit0 = __shfl_sync(0xffffffffu, u0, src);
        row0 = __shfl_sync(0xffffffffu, r0, src);
        n = __shfl_sync(0xffffffffu, t, src);
        b0 = __shfl_sync(0xffffffffu, f, src);
        count = __shfl_sync(0xffffffffu, c, src);
        leader = __shfl_sync(0xffffffffu, l, src);
      }
      units += __shfl_sync(0xffffffffu, u, 31);
      rows += __shfl_sync(0xffffffffu, r, 31);
    }
    return found;
  }
  // The next part of the run (at < end), the same in all lanes.
  __device__ __forceinline__ PrefixPart next(int cta) {
    const int all = Hkv * p.geo.groups;
    PrefixTiles t = prefix_tiles(p.geo, count, n);
    while (at >= unit0 + t.units * all) {  // on to the next group with work
      unit0 += t.units * all;
      row0 += t.rows * all;
      do {
        look_at_group(p, kv_len, cap, page_mask, ++x, n, b0, count, leader);
      } while (n == 0);
      t = prefix_tiles(p.geo, count, n);
    }
    const int gi = int((at - unit0) / t.units);
    const int64_t in = (at - unit0) % t.units;
    const PrefixItem full = prefix_item(p.geo, p.geo.seqs, n);
    const int i = min(int(in / full.units), t.tiles - 1);
    PrefixPart d;
    d.x = x;
    d.g = gi / p.geo.groups;
    d.hg = gi % p.geo.groups;
    d.b0 = b0 + i * p.geo.seqs;
    d.count = min(p.geo.seqs, count - i * p.geo.seqs);
    d.leader = leader;
    d.Lk = p.prefix_len[x];
    const PrefixItem mine = prefix_item(p.geo, d.count, n);
    const int64_t u0 = in - int64_t(i) * full.units, to = min(int64_t(mine.units), u0 + (end - at));
    d.alt = mine.alt;
    d.jb = int(mine.alt ? 2 * u0 : u0);
    d.n = int(mine.alt ? min(2 * to, int64_t(n)) : to) - d.jb;
    d.row = row0 + gi * t.rows + int64_t(i) * full.rows + int64_t(cta) * p.geo.block;
    at += to - u0;
    return d;
  }
};

// bf16: full_prefix_tc.cu; fp32: full_prefix_fp32.cu. Behind the call's offsets check.
struct SharedArgs {
  FullArgs f;
  SharedParams s;
};
PrefixGeometry prefix_geometry_tc(int hpg);
PrefixGeometry prefix_geometry_f32(int hpg);
cudaError_t launch_prefix_tc(const SharedArgs& a, cudaStream_t stream);
cudaError_t launch_prefix_f32(const SharedArgs& a, cudaStream_t stream);

}  // namespace msa
