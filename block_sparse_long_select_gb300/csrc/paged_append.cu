// Appends new tokens' keys and values to a paged cache and rotates keys and
// queries by their positions on the way:
//   (x, y) -> (x cos - y sin, y cos + x sin) on the pairs of the first `rot`
// dims, fp32 inside, rounded once.
//
// Streaming work, bound by HBM at 5.64 TB/s for 20924 tokens (or, for a step of single tokens, by launch
// latency): one CTA per token; a thread's unit is one 16-byte chunk of a head
// row and, for split pairs, the chunk rot / 2 dims further, so both elements
// of every pair are in one thread's registers and q may be rotated in place.
// A few tokens (a decode step) get as many threads as a token has units, so that
// all loads are in flight at once (64 tokens: 7.4 us instead of 8.7 with 128
// threads); with more tokens than fill the SMs, 128 threads each, which share
// the search for the sequence among fewer warps (20924 tokens: 93 us instead of
// 160).
#include "full_internal.cuh"

namespace msa {
namespace {

constexpr int kAppThreads = 128, kAppMostThreads = 512, kAppFewTokens = 4 * kNumSMs;

// x / d, exact while x d is below 2^32, by the rounded-up reciprocal 2^32 / d
struct SmallDiv {
  uint32_t m, d;
  __host__ __device__ explicit SmallDiv(int n) : m(n > 1 ? uint32_t(0x100000000ull / uint32_t(n)) + 1u : 0u), d(n) {}
  __device__ __forceinline__ int of(int x) const { return d == 1 ? x : int(__umulhi(uint32_t(x), m)); }
};

template <typename T>
struct Chunk {
  static constexpr int N = 16 / sizeof(T);  // elements of a 16-byte chunk
  float x[N];
  __device__ __forceinline__ void load(const T* p) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f(e[i]);
  }
  __device__ __forceinline__ void store(T* p) const {
    uint4 raw;
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = from_f<T>(x[i]);
    *reinterpret_cast<uint4*>(p) = raw;
  }
};

// rows by cu_new; lengths are looked at token by token
__host__ __device__ SeqMap seqs_of(const AppendArgs& a) { return SeqMap{a.cu_new, nullptr, a.kv_len, a.B, a.T, 0}; }

template <typename T>
__global__ void __launch_bounds__(kAppMostThreads) paged_append_kernel(const AppendArgs a, const SmallDiv by_units,
                                                                  const SmallDiv by_chunks) {
  constexpr int N = Chunk<T>::N;
  const int t = blockIdx.x;
  int b = t;
  if (a.cu_new) {  // every warp finds the token's sequence itself
    const SeqMap m = seqs_of(a);
    if (cta_in_order(m, &a.ws->disorder)) {
      b = find_row_seq(a.cu_new, a.B, t);
    } else {
      if (threadIdx.x == 0) set_status(&a.ws->status, MSA_ERR_BOUNDS);
      b = scan_row_seq(m, false, t);
    }
    if (b < 0) return;
  }
  const int last = a.cu_new ? a.cu_new[b + 1] : t + 1;
  const int64_t pos = int64_t(a.kv_len[b]) - (last - t);
  const int psz = 1 << a.pages.page_log2;
  int64_t row = -1;
  if (pos >= 0 && pos < (int64_t(a.pages.max_pages) << a.pages.page_log2) &&
      (a.rot == 0 || pos < a.max_pos)) {
    const int page = a.pages.table[int64_t(b) * a.pages.max_pages + (pos >> a.pages.page_log2)];
    if (page >= 0 && page < a.pages.num_pages) row = int64_t(page) * psz + (pos & (psz - 1));
  }
  if (row < 0 && threadIdx.x == 0) set_status(&a.ws->status, MSA_ERR_BOUNDS);
  const int qh = a.q ? a.Hq : 0;
  if (row < 0 && !a.q) return;
  // units of a head row: rot / 2 / N pair units (two chunks each; adjacent
  // chunks if interleaved), then the unrotated chunks
  const int half = a.rot / 2, pu = half / N, units = pu + (a.d - a.rot) / N, chunks = a.d / N;
  const int qk = (qh + a.Hkv) * units, total = qk + a.Hkv * chunks;
  const float* cs = a.rope ? a.rope + pos * a.rot : nullptr;
  for (int u = threadIdx.x; u < total; u += blockDim.x) {
    if (u >= qk) {  // values: copied
      if (row < 0) continue;
      const int h = by_chunks.of(u - qk), c = (u - qk) - h * chunks;
      *reinterpret_cast<uint4*>(static_cast<T*>(a.v_cache) + (row * a.Hkv + h) * a.d + c * N) =
          *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v_new) + (int64_t(t) * a.Hkv + h) * a.d + c * N);
      continue;
    }
    const int hh = by_units.of(u), w = u - hh * units;
    const bool is_q = hh < qh;
    const int h = is_q ? hh : hh - qh;
    const T* src = is_q ? static_cast<const T*>(a.q) + (int64_t(t) * a.Hq + h) * a.d
                        : static_cast<const T*>(a.k_new) + (int64_t(t) * a.Hkv + h) * a.d;
    T* dst = is_q ? static_cast<T*>(a.q_out) + (int64_t(t) * a.Hq + h) * a.d
                  : static_cast<T*>(a.k_cache) + (row * a.Hkv + h) * a.d;
    if (row < 0) {
      if (!is_q) continue;
      const uint4 z = make_uint4(0, 0, 0, 0);
      if (w < pu) {
        *reinterpret_cast<uint4*>(dst + (a.interleaved ? 2 * w * N : w * N)) = z;
        *reinterpret_cast<uint4*>(dst + (a.interleaved ? 2 * w * N + N : half + w * N)) = z;
      } else {
        *reinterpret_cast<uint4*>(dst + a.rot + (w - pu) * N) = z;
      }
      continue;
    }
    if (w >= pu) {  // past the rotated dims
      const int o = a.rot + (w - pu) * N;
      *reinterpret_cast<uint4*>(dst + o) = *reinterpret_cast<const uint4*>(src + o);
      continue;
    }
    const int o0 = a.interleaved ? 2 * w * N : w * N, o1 = a.interleaved ? o0 + N : half + o0;
    Chunk<T> c0, c1;
    c0.load(src + o0);
    c1.load(src + o1);
    const float4* r4 = reinterpret_cast<const float4*>(cs + 2 * w * N);  // N (cos, sin) pairs
    float cc[N], ss[N];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float4 f = __ldg(r4 + i);
      cc[2 * i] = f.x;
      ss[2 * i] = f.y;
      cc[2 * i + 1] = f.z;
      ss[2 * i + 1] = f.w;
    }
    if (a.interleaved) {  // pairs (2i, 2i + 1) of the two adjacent chunks
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float x = c0.x[2 * i], y = c0.x[2 * i + 1];
        c0.x[2 * i] = x * cc[i] - y * ss[i];
        c0.x[2 * i + 1] = y * cc[i] + x * ss[i];
        const float z = c1.x[2 * i], w1 = c1.x[2 * i + 1];
        c1.x[2 * i] = z * cc[N / 2 + i] - w1 * ss[N / 2 + i];
        c1.x[2 * i + 1] = w1 * cc[N / 2 + i] + z * ss[N / 2 + i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x = c0.x[i], y = c1.x[i];
        c0.x[i] = x * cc[i] - y * ss[i];
        c1.x[i] = y * cc[i] + x * ss[i];
      }
    }
    c0.store(dst + o0);
    c1.store(dst + o1);
  }
}

}  // namespace

namespace {
template <typename T>
cudaError_t append(const AppendArgs& a, cudaStream_t stream) {
  constexpr int N = Chunk<T>::N;
  const int units = a.rot / 2 / N + (a.d - a.rot) / N, chunks = a.d / N;
  const int total = ((a.q ? a.Hq : 0) + a.Hkv) * units + a.Hkv * chunks;
  const int threads = a.T > kAppFewTokens ? kAppThreads : total >= kAppMostThreads ? kAppMostThreads : (total + 31) / 32 * 32;
  if (a.cu_new)
    if (cudaError_t e = launch_order_check(seqs_of(a), a.ws, stream)) return e;
  ProfScope pf("paged_append", stream);
  paged_append_kernel<T><<<a.T, threads, 0, stream>>>(a, SmallDiv(units), SmallDiv(chunks));
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t stream) {
  return a.dtype == MSA_BF16 ? append<__nv_bfloat16>(a, stream) : append<float>(a, stream);
}

}  // namespace msa
