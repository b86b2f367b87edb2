// Decode over shared prefixes: how the work on the prefixes is cut, and where
// its partial results lie. One grid computes them (full_prefix_tc.cu for bf16,
// full_prefix_fp32.cu), the decode grid beside or behind it walks the sequences'
// own keys, and a third joins what both leave, a thread per four values. (Joined
// at each item's end inside the decode grid, 97 sequences of 1300 own keys behind
// 20 K shared ones took 190 us, of which its copies stood still for half.)
//
// Group x holds the consecutive sequences [cu[x], cu[x+1]); its prefix is the
// first prefix_len[x] keys of the page-table row of its leader, the group's
// first sequence with keys. An item is a tile of the group's rows (sequences x
// heads of one key/value head) and walks the prefix in tiles of kPxKeys keys. Each
// item is cut into equal runs, which are numbered through and dealt out to the
// CTAs, and leaves a part per run: its rows' maximum (log2 units), sum and
// unnormalised output. The reader finds the parts in closed form, so nothing is
// counted, and nothing waits, inside the grid.
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
  int least;          // units of a run at least, 2 or more
  int beside;         // what a unit takes in steps of the decode grid; 0: no grids side by side
};
// A group's items, for the reader.
struct PrefixRec {
  int64_t row0, more0;  // rows and parts beyond the first ones of the items of the groups before it
  int b0, count;        // first sequence, sequences
  int n, per;           // key tiles (0: nothing to compute), units of a run at most
};
static_assert(sizeof(PrefixRec) == 32, "read as two 16-byte words");

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }
// Of an item of `count` sequences whose prefix has n key tiles: a unit is a key
// tile, as what a unit takes is mostly its copy; alt items count an even number.
struct PrefixItem {
  int units, rows, runs;
  bool alt;
};
__host__ __device__ __forceinline__ PrefixItem prefix_item(const PrefixGeometry& g, int count, int n, int per) {
  const bool alt = g.half > 0 && count <= g.half;
  const int units = alt ? (n + 1) / 2 * 2 : n;
  return {units, count * g.heads, int(uint32_t(units + per - 1) / uint32_t(per)), alt};
}
// Of all items of a group for one key/value head and head group
struct PrefixTiles {
  int tiles;
  int64_t units, rows, runs;
};
__host__ __device__ __forceinline__ PrefixTiles prefix_tiles(const PrefixGeometry& g, int count, int n, int per) {
  const int tiles = ceil_div(count, g.seqs);
  const PrefixItem last = prefix_item(g, count - (tiles - 1) * g.seqs, n, per), full = prefix_item(g, g.seqs, n, per);
  return {tiles, int64_t(tiles - 1) * full.units + last.units, int64_t(tiles - 1) * full.rows + last.rows,
          int64_t(tiles - 1) * full.runs + last.runs};
}
// most parts beyond the items' first ones: see prefix_load
__host__ __device__ __forceinline__ int prefix_most_parts(const PrefixGeometry& g) { return 2 * g.grid; }

// A part of some heads' results: heads x D unnormalised values; a maximum (log2
// units) and a sum per head, negative where there is no result.
struct PartAt {
  const float *o, *ml;
};
// The parts that concern one sequence's heads [h, ...) of one item.
template <int D>
struct PrefixRows {
  const float* o;
  const float2* ml;
  int n, block;  // parts; rows from one to the next
  __device__ __forceinline__ PartAt part(int y) const {
    return {o + int64_t(y) * block * D, reinterpret_cast<const float*>(ml + int64_t(y) * block)};
  }
};

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
  // The parts of heads [h, ...) of key/value head g for sequence b of group x (-1:
  // none). Behind the prefixes' grid (griddepcontrol.wait).
  template <int D>
  __device__ __forceinline__ PrefixRows<D> rows(int x, int b, int g, int h) const {
    PrefixRows<D> r{nullptr, nullptr, 0, 0};
    if (x < 0) return r;
    const longlong2 before = __ldcg(reinterpret_cast<const longlong2*>(recs + x));
    const int4 mine4 = __ldcg(reinterpret_cast<const int4*>(recs + x) + 1);
    const int64_t row0 = before.x, more0 = before.y;
    const int b0 = mine4.x, count = mine4.y, n = mine4.z, per = mine4.w;
    if (n <= 0) return r;
    const PrefixTiles t = prefix_tiles(geo, count, n, per);
    const int s = b - b0, i = s / geo.seqs, hg = h / geo.heads, gi = g * geo.groups + hg;
    const PrefixItem full = prefix_item(geo, geo.seqs, n, per);
    const PrefixItem mine = prefix_item(geo, min(geo.seqs, count - i * geo.seqs), n, per);
    const int64_t more = more0 + gi * (t.runs - t.tiles) + int64_t(i) * (full.runs - 1);
    const int64_t row = row0 + gi * t.rows + int64_t(i) * full.rows + more * geo.block + (s - i * geo.seqs) * geo.heads + h -
                        hg * geo.heads;
    r.o = part + row * D;
    r.ml = stat + row;
    r.block = geo.block;
    r.n = mine.runs;
    return r;
  }
};

// ---- how much there is to do -------------------------------------------------------
// Group i's key tiles (0: nothing to compute), sequences and leader.
struct PrefixGroup {
  int n, b0, count, leader;
};
__device__ __forceinline__ PrefixGroup look_at_group(const SharedParams& p, const int32_t* kv_len, int cap, int page_mask,
                                                     int i) {
  PrefixGroup g;
  g.b0 = p.groups.cu_q[i];
  g.count = p.groups.cu_q[i + 1] - g.b0;
  const int len = p.prefix_len[i];
  g.n = 0;
  g.leader = g.b0;
  if (g.count <= 0 || len <= 0 || len > cap || (len & page_mask)) return g;
  for (int b = g.b0; b < g.b0 + g.count; ++b) {
    const int L = kv_len[b];
    if (L >= len && L <= cap) {  // the others see nothing of it
      g.leader = b;
      g.n = (len - 1) / kPxKeys + 1;
      return g;
    }
  }
  return g;
}
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// The runs, and both grids side by side: the sequences' own keys are bound by
// HBM, which three quarters of the SMs keep busy, the prefixes of many rows by the
// chain from scores to weights. So each grid gets as many SMs as its work says:
// the prefixes' other CTAs leave at once, the decode grid's take their place and
// share out what there is among as many as fit. Measured, one after the other
// and side by side (Hq 32, Hkv 8, d 128):
//   97 sequences, 1300 own keys behind 3 prefixes, 20 K   130 : 112 us
//   32 sequences, 100 behind 8 K                           36 :  29 us
//   64 sequences, 500 behind 8 K                           64 :  50 us
//   64 sequences, 4000 behind 8 K                         204 : 189 us
// (`beside` 24; 13 leaves the prefixes too few, 144, 29, 52, 247 us; 42: 115, 35, 54, 190.)
constexpr int kLeastOwn = 8;  // SMs of the decode grid
struct PrefixLoad {
  int per;  // units of a run, at most
  int64_t runs;
  int each, ctas;  // runs of a CTA, CTAs that have any
  bool beside;     // the decode grid has the other SMs to itself
};
// Whole warp. `heads`: key/value heads; mine: group `lane`, where there are up to 32.
__device__ __forceinline__ PrefixLoad prefix_load(const SharedParams& p, const int32_t* kv_len, int heads, int cap,
                                                  int page_mask, PrefixGroup& mine) {
  const int lane = threadIdx.x & 31, all = heads * p.geo.groups;
  int64_t units = 0, items = 0, own = 0;
  if (p.geo.beside)
#pragma unroll 4
    for (int b = lane; b < p.groups.Tq; b += 32) {
      const int L = kv_len[b], x = p.group_of(b), from = x >= 0 ? p.prefix_len[x] : 0;
      if (L <= cap && from >= 0 && L > from) own += L - from;
    }
  mine.n = 0;
  for (int x0 = 0; x0 < p.groups.B; x0 += 32) {
    PrefixGroup g{0, 0, 0, 0};
    if (x0 + lane < p.groups.B) g = look_at_group(p, kv_len, cap, page_mask, x0 + lane);
    if (x0 == 0) mine = g;
    if (g.n > 0) {
      const PrefixTiles t = prefix_tiles(p.geo, g.count, g.n, 1);
      units += t.units * all;
      items += int64_t(t.tiles) * all;
    }
  }
  units = warp_sum(units);
  items = warp_sum(items);
  own = warp_sum(own);
  int64_t ctas = p.geo.grid;
  const int64_t work = units * p.geo.beside;
  const bool beside = work > 0 && own > 0;
  if (beside) ctas = max(min(ctas * work / (work + own / 16 * heads + 1), ctas - kLeastOwn), int64_t(1));
  // Few items: no CTA has two runs (its second starts behind the end of its first, about 3 us).
  // Many: runs of half a CTA's share. Either way at most 2 ctas runs beyond the items.
  const int64_t want = 2 * items <= ctas ? ctas - items : 2 * ctas;
  // (an item has up to 2^23 units)
  PrefixLoad r{int(min(max((units + want - 1) / want, int64_t(p.geo.least)), int64_t(1) << 24)), 0, 0, 0, beside};
  for (int x0 = 0; x0 < p.groups.B; x0 += 32) {
    PrefixGroup g = mine;
    if (p.groups.B > 32) {
      g.n = 0;
      if (x0 + lane < p.groups.B) g = look_at_group(p, kv_len, cap, page_mask, x0 + lane);
    }
    if (g.n > 0) r.runs += prefix_tiles(p.geo, g.count, g.n, r.per).runs * all;
  }
  r.runs = warp_sum(r.runs);
  r.each = int((r.runs + ctas - 1) / ctas);
  r.ctas = r.each ? int((r.runs + r.each - 1) / r.each) : 0;
  return r;
}

// ---- the prefixes' grid: a CTA's runs ------------------------------------------------
// One part to compute.
struct PrefixPart {
  int g, hg;       // key/value head, head group
  int b0, count;   // its rows' sequences
  int leader, Lk;  // whose page table, keys of the prefix
  int jb, n;       // key tiles [jb, jb + n)
  int alt;
  int64_t row;     // of its first row
};
struct PrefixPlan {
  const SharedParams& p;
  const int32_t* kv_len;
  int Hkv, cap, page_mask;
  // where it stands
  int64_t at, end, run0, row0, more0;
  int x, per;
  PrefixGroup g;

  // Whole warp: measures all groups, leaves their records (`write`), and finds
  // this CTA's runs [at, end). False: it has none.
  __device__ __forceinline__ bool init(int cta, bool write) {
    const int lane = threadIdx.x & 31, all = Hkv * p.geo.groups;
    PrefixGroup mine;
    const PrefixLoad load = prefix_load(p, kv_len, Hkv, cap, page_mask, mine);
    per = load.per;
    at = int64_t(cta) * load.each;
    end = min(at + load.each, load.runs);
    bool found = false;
    int64_t runs = 0, rows = 0, more = 0;
    for (int x0 = 0; x0 < p.groups.B && (write || (!found && at < end)); x0 += 32) {
      if (p.groups.B > 32) {  // else they are in hand
        mine.n = 0;
        if (x0 + lane < p.groups.B) mine = look_at_group(p, kv_len, cap, page_mask, x0 + lane);
      }
      PrefixTiles t{0, 0, 0, 0};
      if (mine.n > 0) t = prefix_tiles(p.geo, mine.count, mine.n, per);
      const int64_t own_u = t.runs * all, own_r = t.rows * all, own_m = (t.runs - t.tiles) * all;
      int64_t u = own_u, r = own_r, m = own_m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t yu = __shfl_up_sync(0xffffffffu, u, o), yr = __shfl_up_sync(0xffffffffu, r, o),
                      ym = __shfl_up_sync(0xffffffffu, m, o);
        if (lane >= o) u += yu, r += yr, m += ym;
      }
      const int64_t u0 = runs + u - own_u, r0 = rows + r - own_r, m0 = more + m - own_m;
      if (write && x0 + lane < p.groups.B)
        p.recs[x0 + lane] = PrefixRec{r0, m0, mine.b0, mine.count, mine.n, per};
      const uint32_t hit = __ballot_sync(0xffffffffu, mine.n > 0 && u0 + own_u > at);
      if (hit && !found && at < end) {
        const int src = __ffs(hit) - 1;
        found = true;
        x = x0 + src;
        run0 = __shfl_sync(0xffffffffu, u0, src);
        row0 = __shfl_sync(0xffffffffu, r0, src);
        more0 = __shfl_sync(0xffffffffu, m0, src);
        g.n = __shfl_sync(0xffffffffu, mine.n, src);
        g.b0 = __shfl_sync(0xffffffffu, mine.b0, src);
        g.count = __shfl_sync(0xffffffffu, mine.count, src);
        g.leader = __shfl_sync(0xffffffffu, mine.leader, src);
      }
      runs += __shfl_sync(0xffffffffu, u, 31);
      rows += __shfl_sync(0xffffffffu, r, 31);
      more += __shfl_sync(0xffffffffu, m, 31);
    }
    return found;
  }
  // The next part (at < end), the same in all lanes.
  __device__ __forceinline__ PrefixPart next() {
    const int all = Hkv * p.geo.groups;
    PrefixTiles t = prefix_tiles(p.geo, g.count, g.n, per);
    while (at >= run0 + t.runs * all) {  // on to the next group with work
      run0 += t.runs * all;
      row0 += t.rows * all;
      more0 += (t.runs - t.tiles) * all;
      do {
        g = look_at_group(p, kv_len, cap, page_mask, ++x);
      } while (g.n == 0);
      t = prefix_tiles(p.geo, g.count, g.n, per);
    }
    const int gi = int((at - run0) / t.runs), in = int((at - run0) % t.runs);
    const PrefixItem full = prefix_item(p.geo, p.geo.seqs, g.n, per);
    const int i = min(in / full.runs, t.tiles - 1), j = in - i * full.runs;
    PrefixPart d;
    d.g = gi / p.geo.groups;
    d.hg = gi % p.geo.groups;
    d.b0 = g.b0 + i * p.geo.seqs;
    d.count = min(p.geo.seqs, g.count - i * p.geo.seqs);
    d.leader = g.leader;
    d.Lk = p.prefix_len[x];
    const PrefixItem mine = prefix_item(p.geo, d.count, g.n, per);
    // units [from, to); an alt item's runs start with even ones (each has one, as runs have two units or more)
    int from = int(int64_t(j) * mine.units / mine.runs), to = int(int64_t(j + 1) * mine.units / mine.runs);
    if (mine.alt) from = (from + 1) & ~1, to = (to + 1) & ~1;
    d.alt = mine.alt;
    d.jb = from;
    d.n = min(to, g.n) - from;
    d.row = row0 + gi * t.rows + int64_t(i) * full.rows +
            (more0 + gi * (t.runs - t.tiles) + int64_t(i) * (full.runs - 1) + j) * p.geo.block;
    ++at;
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
