// Full attention: what every element type shares. Whether offsets are in order,
// the rows' lse and delta for the backward, and the outputs of calls without any key or any query row.
#include "full_internal.cuh"
#include "tc_utils.cuh"

namespace msa {
namespace {

// Per row: lse in log2 units (+inf where no key is seen, so that the row's
// weights are 0; NaN where the output is NaN as well, the weights being
// undefined) and delta = dout . out, laid out as the backward's row tiles,
// [Hkv][Tq][hpg]. A thread per 16-byte chunk; bound by HBM (out and dout once).
constexpr int kRowsPer = 4;
template <typename T, int D>
__global__ void __launch_bounds__(256) full_bwd_rows_kernel(const uint4* __restrict__ out, const uint4* __restrict__ dout,
                                                            const float* __restrict__ lse, int Tq, int Hq, int hpg,
                                                            float2* __restrict__ rows) {
  constexpr int kPer = 16 / sizeof(T), kLanes = D / kPer, kStep = 256 / kLanes;
  const int64_t n = int64_t(Tq) * Hq, x0 = int64_t(blockIdx.x) * kStep * kRowsPer + threadIdx.x / kLanes;
  const int c = threadIdx.x % kLanes;
  tc::griddep_launch_dependents();  // the next grid waits for this one's writes
  uint4 a[kRowsPer], b[kRowsPer];  // all loads in flight at once
#pragma unroll
  for (int r = 0; r < kRowsPer; ++r) {
    const int64_t x = min(x0 + r * kStep, n - 1);
    a[r] = out[x * kLanes + c];
    b[r] = dout[x * kLanes + c];
  }
#pragma unroll
  for (int r = 0; r < kRowsPer; ++r) {
    const int64_t x = x0 + r * kStep;
    const T *ta = reinterpret_cast<const T*>(&a[r]), *tb = reinterpret_cast<const T*>(&b[r]);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s = fmaf(to_f(ta[i]), to_f(tb[i]), s);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (x < n && c == 0) {
      // rows are counted in 32 bits: a 64-bit division would cost more than the row's bytes
      const uint32_t t = uint32_t(x) / uint32_t(Hq), h = uint32_t(x) % uint32_t(Hq);
      const float l = lse[x];
      rows[(int64_t(h / uint32_t(hpg)) * Tq + t) * hpg + h % uint32_t(hpg)] =
          make_float2(l != -INFINITY ? l * 1.4426950408889634f : s == s ? INFINITY : NAN, s);
    }
  }
}

template <typename T, int D>
cudaError_t bwd_rows(const FullBwdArgs& a, cudaStream_t stream) {
  const FullArgs& f = a.f;
  const int64_t threads = (int64_t(f.seq.Tq) * f.Hq + kRowsPer - 1) / kRowsPer * (D * int(sizeof(T)) / 16);
  ProfScope pf("full_bwd_rows", stream);
  full_bwd_rows_kernel<T, D><<<unsigned((threads + 255) / 256), 256, 0, stream>>>(
      static_cast<const uint4*>(f.out), static_cast<const uint4*>(a.dout), f.lse, f.seq.Tq, f.Hq, f.Hq / f.Hkv,
      reinterpret_cast<float2*>(static_cast<char*>(f.ws) + kWsHeader));
  return cudaGetLastError();
}

__global__ void __launch_bounds__(1024) full_order_kernel(const SeqMap m, uint32_t* disorder) {
  bool bad = false;
#pragma unroll 4
  for (int b = threadIdx.x; b < m.B; b += 1024) bad |= !span_in_order(m, seq_span(m, b));
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *disorder = bad;
}

// Zeroes the rows (`keys`: key rows) of every sequence whose own offsets are in
// range, one warp per row of row_bytes; lse, if given, becomes -inf.
__global__ void __launch_bounds__(128) full_zero_kernel(const SeqMap m, bool keys, int row_bytes, uint4* __restrict__ a,
                                                        uint4* __restrict__ b, float* __restrict__ lse, int heads,
                                                        WsHeader* ws) {
  const int t = blockIdx.x * 4 + int(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const bool in_order = cta_in_order(m, &ws->disorder);
  if (!in_order && threadIdx.x == 0) set_status(&ws->status, MSA_ERR_BOUNDS);
  if (t >= (keys ? m.Tk : m.Tq)) return;
  if ((in_order ? find_row_seq(keys ? m.cu_k : m.cu_q, m.B, t) : scan_row_seq(m, keys, t)) < 0) return;
  for (int x = lane; x < row_bytes / 16; x += 32) {
    const int64_t o = int64_t(t) * (row_bytes / 16) + x;
    a[o] = make_uint4(0, 0, 0, 0);
    if (b) b[o] = make_uint4(0, 0, 0, 0);
  }
  if (lse)
    for (int x = lane; x < heads; x += 32) lse[int64_t(t) * heads + x] = -INFINITY;
}

}  // namespace

size_t full_backward_ws_bytes(int Tq, int Hq) { return (size_t(Tq) * Hq * sizeof(float2) + 255) & ~size_t(255); }

cudaError_t launch_order_check(const SeqMap& m, void* ws, cudaStream_t stream) {
  if (m.B <= kSelfChecked) return cudaSuccess;
  ProfScope pf("full_order", stream);
  full_order_kernel<<<1, 1024, 0, stream>>>(m, &static_cast<WsHeader*>(ws)->disorder);
  return cudaGetLastError();
}

cudaError_t launch_full_bwd_rows(const FullBwdArgs& a, cudaStream_t stream) {
  if (a.f.dtype == MSA_BF16)
    return a.f.d == 128 ? bwd_rows<__nv_bfloat16, 128>(a, stream) : bwd_rows<__nv_bfloat16, 64>(a, stream);
  return a.f.d == 128 ? bwd_rows<float, 128>(a, stream) : bwd_rows<float, 64>(a, stream);
}

cudaError_t launch_full_zero(const SeqMap& m, bool keys, int heads, int d, int dtype, void* a, void* b, float* lse,
                             void* ws, cudaStream_t stream) {
  if (cudaError_t e = launch_order_check(m, ws, stream)) return e;
  ProfScope pf("full_zero", stream);
  full_zero_kernel<<<((keys ? m.Tk : m.Tq) + 3) / 4, 128, 0, stream>>>(
      m, keys, heads * d * (dtype == MSA_BF16 ? 2 : 4), static_cast<uint4*>(a), static_cast<uint4*>(b), lse, heads,
      static_cast<WsHeader*>(ws));
  return cudaGetLastError();
}

}  // namespace msa
