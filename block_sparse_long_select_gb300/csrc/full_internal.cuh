// Shared by the full-attention and paged-cache kernels: where a sequence's
// rows and keys lie, the searches over packed offsets, and the launchers.
#pragma once

#include <atomic>

#include "msa_internal.cuh"

namespace msa {

constexpr int kMaxFullHpg = 64;  // query heads per key/value head
constexpr int kMaxFullHeads = 1 << 16;  // a row's elements are counted in 32 bits

// Pages of a cache [num_pages, page_size, Hkv, d] and the table that maps
// sequences to them. table == nullptr: keys are packed rows instead.
struct PageMap {
  const int32_t* table;
  int num_pages, page_log2, max_pages;
};

// Rows and keys of a batch: query rows packed by cu_q (nullptr: row b is
// sequence b's only one); keys packed by cu_k, or kv_len[b] keys in pages.
struct SeqMap {
  const int32_t* cu_q;
  const int32_t* cu_k;    // packed keys
  const int32_t* kv_len;  // paged keys
  int B, Tq, Tk;          // Tk: packed key rows, or max_pages * page_size
};
struct SeqSpan {
  int q0, Lq, k0, Lk;  // k0: first packed key row (0 for paged keys)
  bool rows_ok, keys_ok;  // q0 and Lq, k0 and Lk can be trusted
  bool ok;                // both
};
__device__ __forceinline__ SeqSpan seq_span(const SeqMap& m, int b) {
  SeqSpan s;
  s.q0 = b;
  s.Lq = 1;
  if (m.cu_q) {
    const int a = m.cu_q[b], e = m.cu_q[b + 1];
    s.q0 = a;
    s.rows_ok = a >= 0 && a <= e && e <= m.Tq;
    s.Lq = e - a;
  } else {
    s.rows_ok = true;
  }
  if (m.kv_len) {
    s.k0 = 0;
    s.Lk = m.kv_len[b];
    s.keys_ok = s.Lk >= 0 && s.Lk <= m.Tk;
  } else {
    const int a = m.cu_k[b], e = m.cu_k[b + 1];
    s.k0 = a;
    s.keys_ok = a >= 0 && a <= e && e <= m.Tk;
    s.Lk = e - a;
  }
  s.ok = s.rows_ok && s.keys_ok;
  return s;
}

// ---- offsets out of order ------------------------------------------------------
// The searches below take packed offsets as ordered, 0 <= cu[0] <= ... <= cu[B]
// <= T: one offset that is not can lead them past tiles of every other sequence.
// So all offsets are looked at first, and where they are not in order the
// sequences are gone through one after the other instead: slow, but none is lost.
// Up to kSelfChecked sequences each CTA looks by itself, beside its search's
// loads; for more, a grid of one CTA does it ahead of the call's (about 2 us;
// append of 67614 tokens of 4096 sequences: 144 us unchecked, 232 us if every CTA
// looks, 148 us with the grid; 30446 of 1000: 66, 74 and 70; 12473 of 256: 21, then
// 25 either way).
constexpr int kSelfChecked = 256;
// Every CTA goes through the sequences, so that the time grows with their square
// (estimated at a second or two for gradients of 65536). More than that many out
// of order are left alone: no sequence counts as found.
constexpr int kMostScanned = 1 << 16;
__device__ __forceinline__ bool span_in_order(const SeqMap& m, const SeqSpan& s) {
  return s.rows_ok && (m.kv_len || s.keys_ok);  // a wrong kv_len misleads no search
}
// Whole CTA (a barrier): whether all packed offsets are in order. `disorder` is
// what launch_order_check left, ahead of the grid, for batches that it serves.
__device__ __forceinline__ bool cta_in_order(const SeqMap& m, const uint32_t* disorder) {
  if (m.B > kSelfChecked) return *disorder == 0;
  bool bad = false;
  for (int b = threadIdx.x; b < m.B; b += blockDim.x) bad |= !span_in_order(m, seq_span(m, b));
  bad = __any_sync(0xffffffffu, bad);  // the compiler then knows that warps go one way (append: 30 registers, 50 without)
  return !__syncthreads_or(bad);
}
// Whole warp, 32 sequences at a time from the first on, a lane each: offsets
// below an earlier one within [0, T] are out of range too, so that no two
// sequences in range own the same row.
struct SpanFloor {
  int q = 0, k = 0;  // largest offsets within range so far
  // the largest of the earlier lanes' x and `most`, which then takes in all lanes'
  __device__ __forceinline__ static int before(int x, int& most) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = max(x, y);
    }
    const int up = __shfl_up_sync(0xffffffffu, x, 1), r = lane > 0 ? max(up, most) : most;
    most = max(most, __shfl_sync(0xffffffffu, x, 31));
    return r;
  }
  __device__ __forceinline__ void apply(const SeqMap& m, SeqSpan& s) {
    if (m.cu_q) s.rows_ok &= s.q0 >= before(s.q0 >= 0 && s.q0 <= m.Tq ? s.q0 : 0, q);
    if (!m.kv_len) s.keys_ok &= s.k0 >= before(s.k0 >= 0 && s.k0 <= m.Tk ? s.k0 : 0, k);
    s.ok = s.rows_ok && s.keys_ok;
  }
};
// f(b, span) with the whole warp for 32 sequences at a time (b >= B: an empty
// span out of range), until it returns true. Not at all beyond kMostScanned.
template <typename F>
__device__ __forceinline__ void each_32_seqs(const SeqMap& m, F f) {
  if (m.B > kMostScanned) return;
  SpanFloor floor;
  for (int b0 = 0; b0 < m.B; b0 += 32) {
    const int b = b0 + int(threadIdx.x & 31);
    SeqSpan s{};
    if (b < m.B) s = seq_span(m, b);
    floor.apply(m, s);
    if (b >= m.B) s.rows_ok = s.keys_ok = s.ok = false;
    if (f(b, s)) return;
  }
}

// Warp-wide 32-ary search: the number of indices i in [1, n] with f(i) true,
// for f true up to some index and false after it (2 rounds of loads up to
// n = 1023). Terminates with a value in [0, n] whatever f says.
template <typename F>
__device__ __forceinline__ int warp_count_true(int n, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 0) {
    const int step = (n + 31) >> 5;
    const int probe = min((lane + 1) * step, n);
    const int c = __popc(__ballot_sync(0xffffffffu, f(lo + probe)));
    if (c == 32) return lo + n;
    const int from = min(c * step, n), to = min((c + 1) * step, n);
    lo += from;
    n = max(to - from - 1, 0);
  }
  return lo;
}

// The sequence that owns packed row t, or -1 (whole warp; offsets in order).
__device__ __forceinline__ int find_row_seq(const int32_t* cu, int B, int t) {
  const int b = warp_count_true(B, [&](int i) { return cu[i] <= t; });
  return b < B && cu[b] <= t && t < cu[b + 1] ? b : -1;
}

// The same whatever the offsets are; a row's owner is in range.
__device__ __forceinline__ int scan_row_seq(const SeqMap& m, bool keys, int t) {
  int r = -1;
  each_32_seqs(m, [&](int b, const SeqSpan& s) {
    const int from = keys ? s.k0 : s.q0, n = keys ? s.Lk : s.Lq;
    const uint32_t hit = __ballot_sync(0xffffffffu, (keys ? s.keys_ok : s.rows_ok) && from <= t && t < from + n);
    if (hit) r = __shfl_sync(0xffffffffu, b, __ffs(hit) - 1);
    return hit != 0;
  });
  return r;
}

// Tiles of `tt` rows that start at each sequence's first row, in slots: a
// sequence's token count times `mul` rows, cut into tiles. Tile j of sequence b
// has slot cu[b] * mul / tt + b + j. Slots are unique (a sequence of n rows
// needs at most ceil(n / tt) of them and the + b leaves room for its ragged
// end), so T * mul / tt + B slots cover every tile and a slot's tile is found
// by one search; some slots hold none. Returns the sequence of slot `i` and
// its tile (-1: none). Whole warp; offsets in order.
__device__ __forceinline__ int find_slot_tile(const int32_t* cu, int B, int tt, int i, int& tile, int mul = 1) {
  auto slot0 = [&](int x) { return int64_t(cu[x]) * mul / tt + x; };
  // largest b whose first slot is at most i
  const int b = warp_count_true(B, [&](int x) { return x < B && slot0(x) <= i; });
  const int64_t j = i - slot0(b);
  tile = int(j);
  return j >= 0 && j < (int64_t(cu[b + 1] - cu[b]) * mul + tt - 1) / tt ? b : -1;
}

// The same whatever the offsets are: the i-th tile (`keys`: key tile) of the
// sequences in range, which own no row together, so that as many slots do.
__device__ __forceinline__ int scan_tile(const SeqMap& m, bool keys, int tt, int mul, int i, int& tile, SeqSpan& s) {
  const int lane = threadIdx.x & 31;
  int r = -1;
  int64_t before = 0;
  each_32_seqs(m, [&](int b, const SeqSpan& x) {
    const int64_t n = (keys ? x.keys_ok : x.rows_ok) ? (int64_t(keys ? x.Lk : x.Lq) * mul + tt - 1) / tt : 0;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, before + incl > i);
    if (hit) {
      const int src = __ffs(hit) - 1;
      auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
      r = of(b);
      tile = i - int(__shfl_sync(0xffffffffu, before + incl - n, src));
      s = SeqSpan{of(x.q0), of(x.Lq), of(x.k0), of(x.Lk), of(x.rows_ok) != 0, of(x.keys_ok) != 0, of(x.ok) != 0};
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
    return hit != 0;
  });
  return r;
}

// A CTA's tile by either way, and its sequence's span (`keys`: a key tile).
__device__ __forceinline__ int find_tile(const SeqMap& m, bool in_order, bool keys, int tt, int mul, int i, int& tile,
                                         SeqSpan& s) {
  if (!in_order) return scan_tile(m, keys, tt, mul, i, tile, s);
  const int b = find_slot_tile(keys ? m.cu_k : m.cu_q, m.B, tt, i, tile, mul);
  if (b >= 0) s = seq_span(m, b);
  return b;
}

// ---- launchers ---------------------------------------------------------------
// Prepares a kernel once per device: its dynamic shared memory, and, where its
// warpgroups exchange registers, that it was built with `regs` per thread (0:
// not checked). One instance per kernel; safe from several threads.
class KernelReady {
 public:
  cudaError_t on_device(const void* kern, int smem, int regs = 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
    if (regs) {
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
      if (fa.numRegs != regs) return cudaErrorInvalidConfiguration;
    }
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    done_.fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

struct FullArgs {
  const void *q, *k, *v;
  SeqMap seq;
  PageMap pages;
  int Hq, Hkv, d, dtype;
  float scale;
  void* out;
  float* lse;
  void* ws;
};
struct FullBwdArgs {
  FullArgs f;  // out: the forward's output (read)
  const void* dout;
  void *dq, *dk, *dv;
};
size_t full_decode_ws_bytes(int d);  // behind the header
size_t full_backward_ws_bytes(int Tq, int Hq);  // behind the header
size_t full_prefill_ws_bytes(int d, int64_t most_keys);  // bf16, behind the header
// WsHeader::disorder for the calls of more than kSelfChecked sequences
cudaError_t launch_order_check(const SeqMap& m, void* ws, cudaStream_t stream);
// fp32 prefill and backward
cudaError_t launch_full_f32(const FullArgs& a, cudaStream_t stream);
cudaError_t launch_full_f32_backward(const FullBwdArgs& a, cudaStream_t stream);
// the backward's per-row lse and delta, into the workspace behind the header
cudaError_t launch_full_bwd_rows(const FullBwdArgs& a, cudaStream_t stream);
// every sequence's rows (or keys) of a (and b, if given) zero, lse (if given) -inf
cudaError_t launch_full_zero(const SeqMap& m, bool keys, int heads, int d, int dtype, void* a, void* b, float* lse,
                             void* ws, cudaStream_t stream);
// decode over pages, any dtype
cudaError_t launch_full_decode(const FullArgs& a, cudaStream_t stream);
// tcgen05 prefill (bf16); needs Tk > 0
cudaError_t launch_full_prefill_tc(const FullArgs& a, cudaStream_t stream);
// tcgen05 backward (bf16); needs Tq, Tk > 0
cudaError_t launch_full_backward_tc(const FullBwdArgs& a, cudaStream_t stream);
struct AppendArgs {
  const void *q, *k_new, *v_new;
  const float* rope;
  const int32_t *cu_new, *kv_len;
  PageMap pages;
  int B, T, Hq, Hkv, d, rot, interleaved, max_pos, dtype;
  void *q_out, *k_cache, *v_cache;
  WsHeader* ws;
};
cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t stream);

}  // namespace msa
