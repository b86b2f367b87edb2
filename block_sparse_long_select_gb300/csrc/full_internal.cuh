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

// The sequence that owns packed row t, or -1 (whole warp).
__device__ __forceinline__ int find_row_seq(const int32_t* cu, int B, int t) {
  const int b = warp_count_true(B, [&](int i) { return cu[i] <= t; });
  return b < B && cu[b] <= t && t < cu[b + 1] ? b : -1;
}

// Tiles of `tt` rows that start at each sequence's first row, in slots: a
// sequence's token count times `mul` rows, cut into tiles. Tile j of sequence b
// has slot cu[b] * mul / tt + b + j. Slots are unique (a sequence of n rows
// needs at most ceil(n / tt) of them and the + b leaves room for its ragged
// end), so T * mul / tt + B slots cover every tile and a slot's tile is found
// by one search; some slots hold none. Returns the sequence of slot `i` and
// its tile (-1: none). Whole warp. cu[x] is not checked here: out of range
// values give a tile whose sequence seq_span refuses.
__device__ __forceinline__ int find_slot_tile(const int32_t* cu, int B, int tt, int i, int& tile, int mul = 1) {
  auto slot0 = [&](int x) { return int64_t(cu[x]) * mul / tt + x; };
  // largest b whose first slot is at most i
  const int b = warp_count_true(B, [&](int x) { return x < B && slot0(x) <= i; });
  const int64_t j = i - slot0(b);
  tile = int(j);
  return j >= 0 && j < (int64_t(cu[b + 1] - cu[b]) * mul + tt - 1) / tt ? b : -1;
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
// fp32 prefill and backward
cudaError_t launch_full_f32(const FullArgs& a, cudaStream_t stream);
cudaError_t launch_full_f32_backward(const FullBwdArgs& a, cudaStream_t stream);
// the backward's per-row lse and delta, into the workspace behind the header
cudaError_t launch_full_bwd_rows(const FullBwdArgs& a, cudaStream_t stream);
// every sequence's rows of a (and b, if given) zero, lse (if given) -inf
cudaError_t launch_full_zero(const int32_t* cu, int B, int T, int heads, int d, int dtype, void* a, void* b, float* lse,
                             cudaStream_t stream);
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
  uint32_t* status;
};
cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t stream);

}  // namespace msa
