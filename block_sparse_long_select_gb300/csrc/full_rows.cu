// Full attention on CUDA cores, one warp per (row, head): forward over packed
// or paged keys, and the two halves of the backward.
//
//   out_i = sum_j exp(s_ij - lse_i) v_j,  s_ij = scale q_i . k_j,  j <= Lk - Lq + i
//   dS_ij = P_ij (dout_i . v_j - delta_i);  dq_i = scale sum_j dS_ij k_j
//   dk_j = scale sum_i dS_ij q_i;  dv_j = sum_i P_ij dout_i
//
// A lane holds d / 32 dims of its row; a score is one warp sum. The running
// maximum and sum of the softmax, and every accumulator, are fp32.
#include "full_internal.cuh"

namespace msa {
namespace {

constexpr int kRowWarps = 4;

template <int N>
__device__ __forceinline__ float dot_warp(const float (&a)[N], const float (&b)[N]) {
  float s = 0.f;
#pragma unroll
  for (int x = 0; x < N; ++x) s = fmaf(a[x], b[x], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* p, float (&r)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int x = 0; x < N; ++x) r[x] = to_f(p[lane + 32 * x]);
}
template <typename T, int N>
__device__ __forceinline__ void store_row(T* p, const float (&r)[N], float mul) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int x = 0; x < N; ++x) p[lane + 32 * x] = from_f<T>(r[x] * mul);
}

// Row (in units of Hkv heads) of key j, or -1 if its page is out of range.
__device__ __forceinline__ int64_t key_row(const PageMap& pg, int b, int k0, int j) {
  if (!pg.table) return int64_t(k0) + j;
  const int page = pg.table[int64_t(b) * pg.max_pages + (j >> pg.page_log2)];
  if (page < 0 || page >= pg.num_pages) return -1;
  return (int64_t(page) << pg.page_log2) + (j & ((1 << pg.page_log2) - 1));
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowWarps * 32)
    full_rows_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, SeqMap m, PageMap pg,
                     int Hq, int Hkv, float scale, T* __restrict__ out, float* __restrict__ lse, uint32_t* status) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (item >= int64_t(m.Tq) * Hq) return;
  const int t = int(item / Hq), h = int(item % Hq), g = h / (Hq / Hkv);
  const int b = m.cu_q ? find_row_seq(m.cu_q, m.B, t) : t;
  if (b < 0) return;
  const SeqSpan s = seq_span(m, b);
  if (!s.rows_ok) {
    if (lane == 0) set_status(status, MSA_ERR_BOUNDS);
    return;
  }
  bool ok = s.ok;
  const int n = ok ? min(s.Lk, s.Lk - s.Lq + (t - s.q0) + 1) : 0;  // visible keys
  float qr[N], acc[N], mx = -INFINITY, den = 0.f;
  load_row(q + item * D, qr);
#pragma unroll
  for (int x = 0; x < N; ++x) acc[x] = 0.f;
  for (int j = 0; j < n; ++j) {
    const int64_t row = key_row(pg, b, s.k0, j);
    if (row < 0) {
      ok = false;
      break;
    }
    float kr[N], vr[N];
    load_row(k + (row * Hkv + g) * D, kr);
    load_row(v + (row * Hkv + g) * D, vr);
    const float sc = dot_warp(qr, kr) * scale;
    const float mn = fmaxf(mx, sc);
    const float a = mx == -INFINITY ? 0.f : expf(mx - mn);
    const float p = mn == -INFINITY ? 0.f : expf(sc - mn);
    den = den * a + p;
#pragma unroll
    for (int x = 0; x < N; ++x) acc[x] = fmaf(acc[x], a, p * vr[x]);
    mx = mn;
  }
  if (!ok && lane == 0) set_status(status, MSA_ERR_BOUNDS);
  const bool some = ok && den != 0.f;
#pragma unroll
  for (int x = 0; x < N; ++x)
    if (!some) acc[x] = 0.f;
  store_row(out + item * D, acc, some ? 1.f / den : 0.f);
  if (lse && lane == 0) lse[item] = some ? mx + logf(den) : -INFINITY;
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowWarps * 32)
    full_rows_dq_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                        const T* __restrict__ out, const T* __restrict__ dout, const float* __restrict__ lse, SeqMap m,
                        int Hq, int Hkv, float scale, T* __restrict__ dq, uint32_t* status) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (item >= int64_t(m.Tq) * Hq) return;
  const int t = int(item / Hq), g = int(item % Hq) / (Hq / Hkv);
  const int b = find_row_seq(m.cu_q, m.B, t);
  if (b < 0) return;
  const SeqSpan s = seq_span(m, b);
  if (!s.ok && lane == 0) set_status(status, MSA_ERR_BOUNDS);
  if (!s.rows_ok) return;
  const int n = s.ok ? min(s.Lk, s.Lk - s.Lq + (t - s.q0) + 1) : 0;
  float qr[N], go[N], orow[N], acc[N];
  load_row(q + item * D, qr);
  load_row(dout + item * D, go);
  load_row(out + item * D, orow);
  const float delta = dot_warp(go, orow), l = lse[item];
#pragma unroll
  for (int x = 0; x < N; ++x) acc[x] = 0.f;
  for (int j = 0; j < n; ++j) {
    float kr[N], vr[N];
    const int64_t row = (int64_t(s.k0 + j) * Hkv + g) * D;
    load_row(k + row, kr);
    load_row(v + row, vr);
    const float p = expf(dot_warp(qr, kr) * scale - l);
    const float ds = p * (dot_warp(go, vr) - delta);
#pragma unroll
    for (int x = 0; x < N; ++x) acc[x] = fmaf(ds, kr[x], acc[x]);
  }
  store_row(dq + item * D, acc, scale);
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowWarps * 32)
    full_rows_dkv_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                         const T* __restrict__ out, const T* __restrict__ dout, const float* __restrict__ lse, SeqMap m,
                         int Hq, int Hkv, float scale, T* __restrict__ dk, T* __restrict__ dv, uint32_t* status) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (item >= int64_t(m.Tk) * Hkv) return;
  const int r = int(item / Hkv), g = int(item % Hkv), hpg = Hq / Hkv;
  const int b = find_row_seq(m.cu_k, m.B, r);
  if (b < 0) return;
  const SeqSpan s = seq_span(m, b);
  if (!s.ok) {
    if (lane == 0) set_status(status, MSA_ERR_BOUNDS);
    return;
  }
  const int j = r - s.k0;
  float kr[N], vr[N], ak[N], av[N];
  load_row(k + item * D, kr);
  load_row(v + item * D, vr);
#pragma unroll
  for (int x = 0; x < N; ++x) ak[x] = av[x] = 0.f;
  for (int i = max(0, j - (s.Lk - s.Lq)); i < s.Lq; ++i)
    for (int hh = 0; hh < hpg; ++hh) {
      const int64_t row = int64_t(s.q0 + i) * Hq + g * hpg + hh;
      float qr[N], go[N], orow[N];
      load_row(q + row * D, qr);
      load_row(dout + row * D, go);
      load_row(out + row * D, orow);
      const float p = expf(dot_warp(qr, kr) * scale - lse[row]);
      const float ds = p * (dot_warp(go, vr) - dot_warp(go, orow));
#pragma unroll
      for (int x = 0; x < N; ++x) {
        ak[x] = fmaf(ds, qr[x], ak[x]);
        av[x] = fmaf(p, go[x], av[x]);
      }
    }
  store_row(dk + item * D, ak, scale);
  store_row(dv + item * D, av, 1.f);
}

inline unsigned row_blocks(int64_t items) { return unsigned((items + kRowWarps - 1) / kRowWarps); }

template <typename T, int D>
cudaError_t rows_fwd(const FullArgs& a, cudaStream_t stream) {
  ProfScope pf("full_rows", stream);
  full_rows_kernel<T, D><<<row_blocks(int64_t(a.seq.Tq) * a.Hq), kRowWarps * 32, 0, stream>>>(
      static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.seq, a.pages, a.Hq, a.Hkv,
      a.scale, static_cast<T*>(a.out), a.lse, &static_cast<WsHeader*>(a.ws)->status);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t rows_bwd(const FullBwdArgs& a, cudaStream_t stream) {
  const FullArgs& f = a.f;
  uint32_t* status = &static_cast<WsHeader*>(f.ws)->status;
  const T *q = static_cast<const T*>(f.q), *k = static_cast<const T*>(f.k), *v = static_cast<const T*>(f.v);
  const T *out = static_cast<const T*>(f.out), *dout = static_cast<const T*>(a.dout);
  if (f.seq.Tq > 0) {
    ProfScope pf("full_rows_dq", stream);
    full_rows_dq_kernel<T, D><<<row_blocks(int64_t(f.seq.Tq) * f.Hq), kRowWarps * 32, 0, stream>>>(
        q, k, v, out, dout, f.lse, f.seq, f.Hq, f.Hkv, f.scale, static_cast<T*>(a.dq), status);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  if (f.seq.Tk > 0) {
    ProfScope pf("full_rows_dkv", stream);
    full_rows_dkv_kernel<T, D><<<row_blocks(int64_t(f.seq.Tk) * f.Hkv), kRowWarps * 32, 0, stream>>>(
        q, k, v, out, dout, f.lse, f.seq, f.Hq, f.Hkv, f.scale, static_cast<T*>(a.dk), static_cast<T*>(a.dv), status);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_full_rows(const FullArgs& a, cudaStream_t stream) {
  if (a.dtype == MSA_BF16)
    return a.d == 128 ? rows_fwd<__nv_bfloat16, 128>(a, stream) : rows_fwd<__nv_bfloat16, 64>(a, stream);
  return a.d == 128 ? rows_fwd<float, 128>(a, stream) : rows_fwd<float, 64>(a, stream);
}
cudaError_t launch_full_rows_backward(const FullBwdArgs& a, cudaStream_t stream) {
  if (a.f.dtype == MSA_BF16)
    return a.f.d == 128 ? rows_bwd<__nv_bfloat16, 128>(a, stream) : rows_bwd<__nv_bfloat16, 64>(a, stream);
  return a.f.d == 128 ? rows_bwd<float, 128>(a, stream) : rows_bwd<float, 64>(a, stream);
}

}  // namespace msa
