// Paged caches in 8 bits: new tokens' keys and values written as e4m3 codes with
// a scale per (token, head), and cached rows read back.
//
//   y: a head's row of d values (keys: rotated, see paged_append.cu), in fp32
//   scale = the smallest power of two >= 2^-126 with max|y| / scale <= 448
//   code = e4m3(y / scale), to nearest even;   the row stands for code * scale
// A power of two divides exactly, so a code is one rounding of y: at most half
// a step, 2^-4 of it (2^-10 scale below 2^-6 scale). e4m3's own exponent
// covers 2^-6 to 448, so that the finest scale max|y| / 448 would not round the
// larger values of a row less. A row of zeros has scale 0; one with an infinity
// or NaN (also of the rotation) has scale NaN, so that it stands out wherever it is read.
// Whether a key lies on one side of a code's border or the other must not depend
// on the order of two roundings: keys are rotated with the products' and sums'
// errors carried along and rounded to fp32 once.
//
// Append: streaming, bound by HBM. A head's row is L = d e / 16 lanes with 16
// bytes each, so that its maximum is L - 1 exchanges, and a lane's pairs of the
// rotation are the same for every row of the token: their cosines are loaded
// once. One CTA per token; a decode step's tokens get a thread per 16 bytes.
// Read: streaming. A CTA has 16 packed rows, whose cache rows 16 threads look up
// at once; a thread's unit is 16 bytes of output.
#include "full_internal.cuh"

namespace msa {
namespace {

constexpr int kAppThreads = 128, kAppMostThreads = 512, kAppFewTokens = 4 * kNumSMs;
constexpr int kReadThreads = 256, kReadRows = 16;

// x / d, exact while x d is below 2^32, by the rounded-up reciprocal 2^32 / d
struct SmallDiv {
  uint32_t m, d;
  __host__ __device__ explicit SmallDiv(int n) : m(n > 1 ? uint32_t(0x100000000ull / uint32_t(n)) + 1u : 0u), d(n) {}
  __device__ __forceinline__ int of(int x) const { return d == 1 ? x : int(__umulhi(uint32_t(x), m)); }
};

// a b + c d, rounded to fp32 once but for errors below 2^-45 of the larger product
__device__ __forceinline__ float dot2(float a, float b, float c, float d) {
  const float p = __fmul_rn(a, b), q = __fmul_rn(c, d);
  const float ep = __fmaf_rn(a, b, -p), eq = __fmaf_rn(c, d, -q);  // exact errors of the products
  const float s = __fadd_rn(p, q), t = __fsub_rn(s, p);
  const float es = __fadd_rn(__fsub_rn(p, __fsub_rn(s, t)), __fsub_rn(q, t));  // exact error of their sum
  return __fadd_rn(s, __fadd_rn(es, __fadd_rn(ep, eq)));
}

// two codes, the first in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// rows by cu_new; lengths are looked at token by token
__host__ __device__ SeqMap seqs_of(const AppendArgs& a) { return SeqMap{a.cu_new, nullptr, a.kv_len, a.B, a.T, 0}; }

// The cache row of a packed token: page * page_size + row, -1 if it is out of range.
__device__ __forceinline__ int64_t cache_row(const PageMap& m, int b, int64_t pos) {
  if (pos < 0 || pos >= int64_t(m.max_pages) << m.page_log2) return -1;
  const int page = m.table[int64_t(b) * m.max_pages + (pos >> m.page_log2)];
  if (page < 0 || page >= m.num_pages) return -1;
  return (int64_t(page) << m.page_log2) + (pos & ((1 << m.page_log2) - 1));
}

template <typename T, int D>
__global__ void __launch_bounds__(kAppMostThreads)
    paged_append_fp8_kernel(const AppendArgs a, float* __restrict__ k_scale, float* __restrict__ v_scale) {
  constexpr int N = 16 / int(sizeof(T)), L = D / N, kPer = 32 / L;  // elements of a lane, lanes of a row, rows of a warp
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
  const int64_t row = a.rot == 0 || pos < a.max_pos ? cache_row(a.pages, b, pos) : -1;
  if (row < 0 && threadIdx.x == 0) set_status(&a.ws->status, MSA_ERR_BOUNDS);
  const int qh = a.q ? a.Hq : 0;
  if (row < 0 && !a.q) return;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L, c = lane % L;
  const int half = a.rot / 2 / N;  // 16-byte chunks of half the rotated dims
  // this lane's part of the rotation: out = x cc + partner ss
  const bool turns = c < 2 * half && row >= 0;
  const int partner = turns && !a.interleaved ? (c < half ? lane + half : lane - half) : lane;
  float cc[N], ss[N];
  if (turns) {
    const float* cs = a.rope + pos * a.rot;
    if (a.interleaved) {  // pairs (2i, 2i + 1) of the chunk
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float2 f = __ldg(reinterpret_cast<const float2*>(cs) + c * (N / 2) + i);
        cc[2 * i] = cc[2 * i + 1] = f.x;
        ss[2 * i] = -f.y;
        ss[2 * i + 1] = f.y;
      }
    } else {
      const float sign = c < half ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(cs + 2 * (c < half ? c : c - half) * N) + i);
        cc[2 * i] = f.x;
        ss[2 * i] = sign * f.y;
        cc[2 * i + 1] = f.z;
        ss[2 * i + 1] = sign * f.w;
      }
    }
  }
  const int64_t page = row >> a.pages.page_log2, in_page = row & ((1 << a.pages.page_log2) - 1);
  const int rows = qh + 2 * a.Hkv, step = int(blockDim.x >> 5) * kPer;
  constexpr int kBatch = 4;  // rows in flight
  for (int r0 = warp * kPer; r0 < rows; r0 += kBatch * step) {
    uint4 raw[kBatch];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int r = r0 + y * step + sub;
      const T* src = r < qh ? static_cast<const T*>(a.q) + (int64_t(t) * a.Hq + r) * D
                     : r < qh + a.Hkv ? static_cast<const T*>(a.k_new) + (int64_t(t) * a.Hkv + r - qh) * D
                                      : static_cast<const T*>(a.v_new) + (int64_t(t) * a.Hkv + r - qh - a.Hkv) * D;
      raw[y] = r < rows ? reinterpret_cast<const uint4*>(src)[c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      if (r0 + y * step >= rows) break;  // the whole warp's
      const int r = r0 + y * step + sub;
      const bool is_q = r < qh, is_k = !is_q && r < qh + a.Hkv;
      uint4 other = raw[y];
      if (!a.interleaved) {
        other.x = __shfl_sync(0xffffffffu, raw[y].x, partner);
        other.y = __shfl_sync(0xffffffffu, raw[y].y, partner);
        other.z = __shfl_sync(0xffffffffu, raw[y].z, partner);
        other.w = __shfl_sync(0xffffffffu, raw[y].w, partner);
      }
      const T *e = reinterpret_cast<const T*>(&raw[y]), *eo = reinterpret_cast<const T*>(&other);
      float x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = to_f(e[i]);
        if (turns && (is_q || is_k)) {
          const float z = to_f(a.interleaved ? e[i ^ 1] : eo[i]);
          x[i] = is_k ? dot2(x[i], cc[i], z, ss[i]) : fmaf(x[i], cc[i], z * ss[i]);
        }
      }
      uint32_t top = 0;  // as bits: a NaN is above infinity above all else
#pragma unroll
      for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (r >= rows) continue;
      if (is_q) {
        uint4 u;
        T* w = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = from_f<T>(row < 0 ? 0.f : x[i]);
        if (row >= 0 && !turns) u = raw[y];  // copied
        reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + (int64_t(t) * a.Hq + r) * D)[c] = u;
        continue;
      }
      if (row < 0) continue;
      const int h = r - qh - (is_k ? 0 : a.Hkv);
      // 448 = 1.75 * 2^8: the exponent field of top, one more if its fraction is above 1.75, less 8
      const uint32_t field = max(int((top + 0x1fffffu) >> 23) - 8, 1);
      const bool fine = top < 0x7f800000u;
      const float inv = __uint_as_float((254u - field) << 23);
      uint8_t* dst = static_cast<uint8_t*>(is_k ? a.k_cache : a.v_cache) + (row * a.Hkv + h) * D + c * N;
      uint32_t w[N / 4];
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        w[i] = !fine ? 0u : e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) | e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16;
      if constexpr (N == 8)
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(dst) = w[0];
      if (c == 0)
        (is_k ? k_scale : v_scale)[((page * a.Hkv + h) << a.pages.page_log2) + in_page] =
            !fine ? __uint_as_float(0x7fc00000u) : top == 0 ? 0.f : __uint_as_float(field << 23);
    }
  }
}

template <typename T, int D>
cudaError_t append(const AppendArgs& a, float* k_scale, float* v_scale, cudaStream_t stream) {
  constexpr int L = D * int(sizeof(T)) / 16;
  const int total = ((a.q ? a.Hq : 0) + 2 * a.Hkv) * L;
  const int threads = a.T > kAppFewTokens ? kAppThreads : total >= kAppMostThreads ? kAppMostThreads : (total + 31) / 32 * 32;
  if (a.cu_new)
    if (cudaError_t e = launch_order_check(seqs_of(a), a.ws, stream)) return e;
  ProfScope pf("paged_append_fp8", stream);
  paged_append_fp8_kernel<T, D><<<a.T, threads, 0, stream>>>(a, k_scale, v_scale);
  return cudaGetLastError();
}

__host__ __device__ SeqMap seqs_of(const ReadArgs& a) { return SeqMap{a.cu, nullptr, a.kv_len, a.B, a.T, 0}; }

template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) paged_read_fp8_kernel(const ReadArgs a, const SmallDiv by_rows) {
  constexpr int N = 16 / int(sizeof(T)), L = D / N;  // elements of a unit, units of a head's row
  __shared__ int64_t row_s[kReadRows];               // cache row; -1: out of range, -2: nobody's
  const int t0 = blockIdx.x * kReadRows, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool in_order = !a.cu || cta_in_order(seqs_of(a), &a.ws->disorder);
  auto look = [&](int t, int b) {
    if (b < 0) return int64_t(-2);
    const int64_t row = cache_row(a.pages, b, int64_t(a.kv_len[b]) - ((a.cu ? a.cu[b + 1] : t + 1) - t));
    if (row < 0) set_status(&a.ws->status, MSA_ERR_BOUNDS);
    return row;
  };
  if (in_order) {
    const int t = t0 + int(threadIdx.x);
    if (threadIdx.x < kReadRows) {
      int b = t < a.T ? t : -1;
      if (a.cu && t < a.T) {  // the last sequence that starts at or before t
        int n = a.B;
        b = 0;
        while (n > 1) {
          const int mid = n / 2;
          if (a.cu[b + mid] <= t) {
            b += mid;
            n -= mid;
          } else {
            n = mid;
          }
        }
        if (a.cu[b] > t || t >= a.cu[b + 1]) b = -1;
      }
      row_s[threadIdx.x] = look(t, b);
    }
  } else {
    if (threadIdx.x == 0) set_status(&a.ws->status, MSA_ERR_BOUNDS);
    for (int x = warp; x < kReadRows; x += kReadThreads / 32) {
      const int t = t0 + x, b = t < a.T ? scan_row_seq(seqs_of(a), false, t) : -1;
      if (lane == 0) row_s[x] = look(t, b);
    }
  }
  __syncthreads();
  const int heads = 2 * a.Hkv, c = threadIdx.x % L;
  constexpr int kBatch = 8, kStep = kReadThreads / L;  // units in flight; head rows of a pass
  const int all = kReadRows * heads;
  for (int r0 = threadIdx.x / L; r0 < all; r0 += kBatch * kStep) {
    uint32_t code[kBatch][N / 4];
    float scale[kBatch];
    int64_t to[kBatch];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int r = min(r0 + y * kStep, all - 1);
      int x = by_rows.of(r);
      x -= x * heads > r;  // beyond 8192 key/value heads the reciprocal's quotient can be one too large
      const int hh = r - x * heads;
      const bool is_v = hh >= a.Hkv;
      const int h = is_v ? hh - a.Hkv : hh;
      const int64_t row = row_s[x], src = max(row, int64_t(0));
      const uint8_t* p = static_cast<const uint8_t*>(is_v ? a.v_cache : a.k_cache) + (src * a.Hkv + h) * D + c * N;
      if constexpr (N == 8) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        code[y][0] = u.x, code[y][1] = u.y;
      } else {
        code[y][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      }
      const int64_t s = (((src >> a.pages.page_log2) * a.Hkv + h) << a.pages.page_log2) + (src & ((1 << a.pages.page_log2) - 1));
      scale[y] = __ldg((is_v ? a.v_scale : a.k_scale) + s);
      if (row < 0) {  // out of range: zeros
        scale[y] = 0.f;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) code[y][i] = 0;
      }
      to[y] = row == -2 || r0 + y * kStep >= all ? -1 : (int64_t(t0 + x) * a.Hkv + h) * 2 + is_v;
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      if (to[y] < 0) continue;
      uint4 u;
      T* w = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        uint32_t f;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(uint16_t(code[y][i / 2] >> (16 * (i & 1)))));
        float lo, hi;
        asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(lo), "=f"(hi) : "r"(f));
        w[2 * i] = from_f<T>(lo * scale[y]);
        w[2 * i + 1] = from_f<T>(hi * scale[y]);
      }
      reinterpret_cast<uint4*>(static_cast<T*>(to[y] & 1 ? a.v_out : a.k_out) + (to[y] >> 1) * D)[c] = u;
    }
  }
}

template <typename T, int D>
cudaError_t read(const ReadArgs& a, cudaStream_t stream) {
  if (a.cu)
    if (cudaError_t e = launch_order_check(seqs_of(a), a.ws, stream)) return e;
  ProfScope pf("paged_read_fp8", stream);
  paged_read_fp8_kernel<T, D><<<(a.T + kReadRows - 1) / kReadRows, kReadThreads, 0, stream>>>(a, SmallDiv(2 * a.Hkv));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append_fp8(const AppendArgs& a, float* k_scale, float* v_scale, cudaStream_t stream) {
  if (a.dtype == MSA_BF16)
    return a.d == 128 ? append<__nv_bfloat16, 128>(a, k_scale, v_scale, stream)
                      : append<__nv_bfloat16, 64>(a, k_scale, v_scale, stream);
  return a.d == 128 ? append<float, 128>(a, k_scale, v_scale, stream) : append<float, 64>(a, k_scale, v_scale, stream);
}

cudaError_t launch_paged_read_fp8(const ReadArgs& a, cudaStream_t stream) {
  if (a.dtype == MSA_BF16) return a.d == 128 ? read<__nv_bfloat16, 128>(a, stream) : read<__nv_bfloat16, 64>(a, stream);
  return a.d == 128 ? read<float, 128>(a, stream) : read<float, 64>(a, stream);
}

}  // namespace msa
