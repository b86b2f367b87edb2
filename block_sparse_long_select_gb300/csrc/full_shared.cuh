// Decode over shared prefixes: how the work is cut, and where its partial
// results lie. Four grids, each of which starts while the one before it ends:
// one CTA plans (full_shared_plan.cu); one grid computes the prefixes
// (full_prefix_tc.cu for bf16, full_prefix_fp32.cu); the decode grid, beside it
// or behind it, walks the sequences' own keys; the last joins what both leave, a
// thread per four values. (Joined at each item's end inside the decode grid, 97
// sequences of 1300 own keys behind 20 K shared ones took 190 us, of which its
// copies stood still for half.)
//
// Group x holds the consecutive sequences [cu[x], cu[x+1]); its prefix is the
// first prefix_len[x] keys of the page-table row of its leader, the group's
// first sequence with keys. An item is a tile of the group's rows (sequences x
// heads of one key/value head) and walks the prefix in tiles of kPxKeys keys. Each
// item is cut into equal runs, which are numbered through and dealt out to the
// CTAs, and leaves a part per run: its rows' maximum (log2 units), sum and
// unnormalised output. The decode grid's steps are numbered through and dealt out
// to its warps likewise. The reader finds all parts in closed form, so nothing is
// counted, and nothing waits, inside a grid.
#pragma once

#include "full_internal.cuh"

namespace msa {

constexpr int kPxKeys = 128;  // keys of a tile
// What an item's beginning and end count beside its steps in the decode grid (4000
// sequences of 100 keys in 1000 groups behind 512: 0 steps 866 us, 2 794, 4 800).
constexpr int kOwnItemSteps = 2;

// How rows are cut into items. bf16: two row tiles of `half` sequences, which
// share each key tile; an item whose sequences fit into one takes the key tiles
// two at a time instead, one per half (`alt`).
struct PrefixGeometry {
  int heads, groups;  // heads of an item; items' head groups per key/value head
  int seqs, half;     // sequences of an item; of a row tile (0: an item is one row tile)
  int block;          // most rows of a part
  int grid;           // CTAs
  int least;          // units of a run at least; 2 or more where there are alt items
  int beside;         // what a unit takes in steps of the decode grid; 0: no grids side by side
  int worth;          // key tiles times sequences beyond the first that make an item
};
// A group's items; runs, rows and parts beyond the items' first ones of the groups before it.
struct PrefixRec {
  int64_t run0, row0, more0;
  int b0, count;  // first sequence, sequences
  int n, leader;  // key tiles (0: nothing to compute), whose page table
  int64_t unused;
};
static_assert(sizeof(PrefixRec) == 48, "read as three 16-byte words");
// What the planning CTA says of the whole call.
struct SharedHead {
  int64_t runs, steps;            // prefixes' runs; own keys' steps of all items, what their ends count among them
  int64_t own_per, disorder;      // steps of a warp; whether cu_prefix is out of order: then nothing else counts
  int per, each, ctas, own_ctas;  // units of a prefix's run at most; runs of a CTA, CTAs with runs; of the decode grid
};
static_assert(sizeof(SharedHead) == 48, "read as three 16-byte words");
// A sequence: where the keys that it walks by itself begin (-1: its length is out
// of range), the group whose parts it takes (-1: none), and whose page table holds
// its first keys, up to where.
struct SharedSeq {
  int from, group, leader, upto;
};

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
// most parts beyond the items' first ones (full_shared_plan.cu)
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
  PrefixGeometry geo;
  SharedHead* head;
  SharedSeq* seqs;  // [sequences]
  int64_t* step0;   // [sequences]: steps of the sequences before it
  PrefixRec* recs;  // [groups]
  float* part;      // [rows][D]
  float2* stat;     // [rows]: maximum, sum (negative: a page out of range)

  // The plan is read past L1: the grids that read it may have started before it was made.
  __device__ __forceinline__ SharedHead get_head() const {
    const longlong2* w = reinterpret_cast<const longlong2*>(head);
    const longlong2 a = __ldcg(w), b = __ldcg(w + 1);
    const int4 c = __ldcg(reinterpret_cast<const int4*>(w + 2));
    return {a.x, a.y, b.x, b.y, c.x, c.y, c.z, c.w};
  }
  __device__ __forceinline__ SharedSeq get_seq(int b) const {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(seqs + b));
    return {v.x, v.y, v.z, v.w};
  }
  __device__ __forceinline__ PrefixRec get_rec(int x) const {
    const int4* w = reinterpret_cast<const int4*>(recs + x);
    const longlong2 a = __ldcg(reinterpret_cast<const longlong2*>(w));
    const int4 b = __ldcg(w + 1), c = __ldcg(w + 2);
    PrefixRec r;
    r.run0 = a.x, r.row0 = a.y;
    r.more0 = int64_t(uint32_t(b.x)) | int64_t(b.y) << 32;
    r.b0 = b.z, r.count = b.w;
    r.n = c.x, r.leader = c.y;
    return r;
  }
  // The parts of heads [h, ...) of key/value head g for sequence b of group x (-1: none).
  template <int D>
  __device__ __forceinline__ PrefixRows<D> rows(int x, int b, int g, int h, int per) const {
    PrefixRows<D> r{nullptr, nullptr, 0, 0};
    if (x < 0) return r;
    const PrefixRec c = get_rec(x);
    if (c.n <= 0) return r;
    const PrefixTiles t = prefix_tiles(geo, c.count, c.n, per);
    const int s = b - c.b0, i = s / geo.seqs, hg = h / geo.heads, gi = g * geo.groups + hg;
    const PrefixItem full = prefix_item(geo, geo.seqs, c.n, per);
    const PrefixItem mine = prefix_item(geo, min(geo.seqs, c.count - i * geo.seqs), c.n, per);
    const int64_t more = c.more0 + gi * (t.runs - t.tiles) + int64_t(i) * (full.runs - 1);
    const int64_t row = c.row0 + gi * t.rows + int64_t(i) * full.rows + more * geo.block + (s - i * geo.seqs) * geo.heads +
                        h - hg * geo.heads;
    r.o = part + row * D;
    r.ml = stat + row;
    r.block = geo.block;
    r.n = mine.runs;
    return r;
  }
};

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
struct PrefixRuns {
  const SharedParams& p;
  int Hkv;
  int64_t at, end;  // runs left
  int x, per;
  PrefixRec g;  // group x

  // Whole warp. False: the CTA has none.
  __device__ __forceinline__ bool init(const SharedHead& h, int cta) {
    per = h.per;
    at = int64_t(cta) * h.each;
    end = min(at + h.each, h.runs);
    if (h.disorder || at >= end) return false;
    // the last group that starts at or before the run: groups without runs are passed over
    x = warp_count_true(p.groups.B - 1, [&](int i) { return __ldcg(&p.recs[i].run0) <= at; });
    g = p.get_rec(x);
    return true;
  }
  // The next part (at < end), the same in all lanes.
  __device__ __forceinline__ PrefixPart next() {
    const int all = Hkv * p.geo.groups;
    PrefixTiles t = prefix_tiles(p.geo, g.count, g.n, per);
    while (at >= g.run0 + t.runs * all) {  // on to the next group with work
      do {
        g = p.get_rec(++x);
      } while (g.n == 0);
      t = prefix_tiles(p.geo, g.count, g.n, per);
    }
    const int gi = int((at - g.run0) / t.runs), in = int((at - g.run0) % t.runs);
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
    d.row = g.row0 + gi * t.rows + int64_t(i) * full.rows +
            (g.more0 + gi * (t.runs - t.tiles) + int64_t(i) * (full.runs - 1) + j) * p.geo.block;
    ++at;
    return d;
  }
};

struct SharedArgs {
  FullArgs f;
  SharedParams s;
};
// A launch that starts while the grid before it in the stream ends (which it waits for itself).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), int64_t ctas, int threads, int smem, cudaStream_t stream, A... args) {
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
// `warps`: of a decode CTA; `items`: of a sequence in the decode grid
cudaError_t launch_shared_plan(const SharedArgs& a, int warps, int items, cudaStream_t stream);
PrefixGeometry prefix_geometry_tc(int hpg);
PrefixGeometry prefix_geometry_f32(int hpg);
cudaError_t launch_prefix_tc(const SharedArgs& a, cudaStream_t stream);
cudaError_t launch_prefix_f32(const SharedArgs& a, cudaStream_t stream);

}  // namespace msa
