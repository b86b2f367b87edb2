// Even division of attention work over a persistent grid.
//
// An item is one tile of a sequence and key/value head (query rows, or keys in
// dk/dv) with all it has to walk on the other side; its cost is that length
// plus a constant for its start and end. Items of a sequence grow linearly up
// to a bound, so costs add up in closed form: every CTA finds its equal share
// [T i / G, T (i + 1) / G) of the total T by itself, whatever the lengths, and
// no host or second kernel needs to know them. A share may begin or end inside
// an item: the item is then split, and the CTAs that hold its parts leave
// partials in the workspace for the last of them to join in order. Items that
// are short are not split: a share's border inside one moves to its nearer end.
#pragma once

#include "full_internal.cuh"

namespace msa {

// Items x = 0 .. items - 1 of a sequence, each for every key/value head:
// length min(most, first + x * step); the first `below` are below the bound.
struct SeqWork {
  int items, first, most, below;
};
__device__ __forceinline__ SeqWork seq_work(int items, int first, int most, int step) {
  return SeqWork{items, first, most, most > first ? int((unsigned(most) - unsigned(first) + step - 1) / step) : 0};
}

struct SchedParams {
  int step;       // growth of the length from item to item
  int tile;       // lengths are walked in tiles of this
  int fixed;      // cost of an item beside its length
  int least_run;  // a share is at least this long (fewer CTAs work then)
  int whole;      // items up to this length are not split
};

__device__ __forceinline__ int item_len(const SeqWork& s, int step, int x) {
  return int(min(int64_t(s.most), s.first + int64_t(x) * step));
}
// Cost of items [0, x) of one head.
__device__ __forceinline__ int64_t items_cost(const SeqWork& s, const SchedParams& p, int x) {
  if (x <= 0) return 0;
  const int64_t m = min(s.below, x);
  return m * s.first + p.step * (m * (m - 1) / 2) + (x - m) * int64_t(s.most) + x * int64_t(p.fixed);
}

// A place in the order (sequence, head, item).
struct Place {
  int b, g, x;
  SeqWork w;
  int64_t at;  // cost before the item
};

// One CTA's share; computed and walked by one warp (f(b): the work of sequence b).
template <typename F>
struct Share {
  F f;
  SchedParams p;
  int B, Hkv;
  int64_t total, each;  // all cost; a share's (the first `more` shares have one more)
  int G, more;
  int64_t lo, hi;  // the share, in cost
  int longest;     // cost of the longest item
  Place cur;

  __device__ __forceinline__ int64_t border(int i) const { return each * i + min(i, more); }
  __device__ __forceinline__ int64_t item_cost(const Place& q) const {
    return item_len(q.w, p.step, q.x) + int64_t(p.fixed);
  }
  __device__ __forceinline__ Place locate(int64_t pos) const {
    const int lane = threadIdx.x & 31;
    Place r{};
    int64_t before = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const SeqWork w = b0 + lane < B ? f(b0 + lane) : SeqWork{0, 0, 0, 0};
      int64_t incl = items_cost(w, p, w.items) * Hkv;
      const int64_t mine = incl;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + incl > pos);
      if (hit) {
        const int src = __ffs(hit) - 1;
        r.b = b0 + src;
        r.w.items = __shfl_sync(0xffffffffu, w.items, src);
        r.w.first = __shfl_sync(0xffffffffu, w.first, src);
        r.w.most = __shfl_sync(0xffffffffu, w.most, src);
        r.w.below = __shfl_sync(0xffffffffu, w.below, src);
        r.at = before + __shfl_sync(0xffffffffu, incl - mine, src);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    const int64_t head = items_cost(r.w, p, r.w.items);
    // the head: no 64-bit division on a CTA's way to its first item
    r.g = warp_count_true(Hkv - 1, [&](int x) { return r.at + x * head <= pos; });
    r.at += r.g * head;
    const int64_t in = pos - r.at;
    r.x = warp_count_true(r.w.items - 1, [&](int x) { return items_cost(r.w, p, x) <= in; });
    r.at += items_cost(r.w, p, r.x);
    return r;
  }
  // A border moved off the short item that it would split.
  __device__ __forceinline__ int64_t settle(int64_t pos, Place* place) const {
    if (pos >= total) return total;
    *place = locate(pos);
    if (pos == place->at) return pos;
    const int64_t c = item_cost(*place);
    if (item_len(place->w, p.step, place->x) > p.whole) return pos;
    return pos - place->at < c / 2 ? place->at : place->at + c;
  }
  // All cost, and whether there is any.
  __device__ __forceinline__ bool measure(int ctas) {
    total = 0;
    longest = 0;
#pragma unroll 1  // unrolled by 4 it costs few long sequences 4 us (279 -> 283) and many short ones as much
    for (int b = threadIdx.x & 31; b < B; b += 32) {
      const SeqWork w = f(b);
      total += items_cost(w, p, w.items);
      longest = max(longest, w.items > 0 ? item_len(w, p.step, w.items - 1) : 0);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    longest = __reduce_max_sync(0xffffffffu, longest);
    total *= Hkv;
    G = int(max(min(total / p.least_run, int64_t(ctas)), int64_t(1)));
    each = total / G;
    more = int(total - each * G);
    return total > 0;
  }
  // Where equal shares would hold several items each, items are handed out
  // whole, one after the other, long ones first: no joins, and the last ones
  // are short. Equal shares serve few or very long items.
  __device__ __forceinline__ bool hand_out() const { return longest + p.fixed <= each / 2; }
  // The CTA's share (measure first).
  __device__ __forceinline__ bool init(int cta) {
    if (cta >= G) return false;
    Place other;
    lo = settle(border(cta), &cur);
    hi = settle(border(cta + 1), &other);
    if (lo >= hi) return false;
    if (lo > cur.at) {
      // settled on the end of a short item: begin with the next one
      if (item_len(cur.w, p.step, cur.x) <= p.whole) next();
    }
    return true;
  }
  // To the next item; sequences without items are passed over.
  __device__ __forceinline__ void next() {
    cur.at += item_cost(cur);
    if (++cur.x < cur.w.items) return;
    cur.x = 0;
    if (++cur.g < Hkv) return;
    cur.g = 0;
    do {
      if (++cur.b >= B) {
        cur.w = SeqWork{1, 0, 0, 0};
        return;
      }
      cur.w = f(cur.b);
    } while (cur.w.items == 0);
  }
  __device__ __forceinline__ bool done() const { return cur.at >= hi || cur.b >= B; }
  // First tile, of an item's n, behind a place `pos` in the order.
  __device__ __forceinline__ int tile_at(int64_t pos, int n) const {
    const int64_t in = pos - cur.at;
    if (in >= item_cost(cur)) return n;
    return in <= p.fixed ? 0 : int(min((in - p.fixed + p.tile - 1) / p.tile, int64_t(n)));
  }
  // This share's tiles [from, to) of the current item's n.
  __device__ __forceinline__ void tiles(int n, int& from, int& to) const {
    from = tile_at(lo, n);
    to = tile_at(hi, n);
  }
  // The CTA that holds the start of the current, split item.
  __device__ __forceinline__ int first_cta() const {
    return warp_count_true(G - 1, [&](int i) { return border(i) <= cur.at; });
  }
  // Whether CTA i holds tiles of the current, split item.
  __device__ __forceinline__ bool holds(int i, int n) const {
    return tile_at(border(i + 1), n) > tile_at(max(border(i), cur.at), n);
  }
};

}  // namespace msa
